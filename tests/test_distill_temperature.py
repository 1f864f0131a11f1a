"""hqq_distill's smallest temperatures: refused on the host where log2(e) / t, by which
the kernel multiplies, is beyond fp32 (no GPU needed)."""
import ctypes
import math

import numpy as np
import pytest

LIMIT = math.log2(math.e) / float(np.finfo(np.float32).max)        # 4.24e-39


@pytest.mark.parametrize("t", [1e-45, 1e-39, 2.9e-39, 2.95e-39, 3.5e-39, 4.2e-39, 0.999 * LIMIT])
def test_tiny_temperatures_are_refused(t):
    import weight_only_quantization_b200 as hqq
    P = ctypes.c_void_p
    st = hqq._lib.hqq_distill(P(256), 1000, 0, 4, 1000, P(256), 2, P(256), 8, 8, t, None, None,
                              P(256), P(256), P(512), 1000, None)
    assert st == 4


@pytest.mark.gpu
@pytest.mark.parametrize("t", [1.001 * LIMIT, 2.0 ** -100, 2.0 ** 100, 3e38])
def test_temperatures_at_the_ends_of_the_range(t):
    """Accepted temperatures give what their formula tends to: towards 0 the largest
    logit takes all, towards infinity every one has the same share."""
    torch = pytest.importorskip("torch")
    import weight_only_quantization_b200 as hqq
    V = 64
    z = torch.randperm(V, generator=torch.Generator().manual_seed(1)).float()[None].cuda()
    top, at = torch.topk(z, 2, dim=1)
    loss, _, grad = hqq.hqq_distill(z, top.contiguous(), at.contiguous(), t, weight=torch.tensor(
        [min(t, 1.0)], device="cuda"), grad=True)
    assert bool(torch.isfinite(grad).all())
    if t < 1:                  # teacher and student agree: all on the same entry
        assert float(loss) == 0.0 and float(grad.abs().max()) <= 2.0 ** -22
    else:                      # uniform over 2 against uniform over 64
        assert abs(float(loss) - math.log(32.0)) <= 64 * 2.0 ** -24 * math.log(64.0)
