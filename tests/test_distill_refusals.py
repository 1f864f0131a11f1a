"""Argument checks of hqq_distill: bad calls are refused on the host before
anything is enqueued (no GPU needed)."""
import ctypes

import pytest

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    import weight_only_quantization_b200 as m
    return m


def call(lib, logits=256, ls=1000, dtype=0, T=4, V=1000, top=256, tdt=2, at=256, ib=8, K=8,
         temp=1.0, tl=None, w=None, loss=256, lse=256, grad=512, gs=1000):
    ptr = lambda v: P(v) if v else None  # noqa: E731
    return lib._lib.hqq_distill(ptr(logits), ls, dtype, T, V, ptr(top), tdt, ptr(at), ib, K, temp,
                                ptr(tl), ptr(w), ptr(loss), ptr(lse), ptr(grad), gs, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), 2), (dict(T=1 << 27), 2), (dict(V=0), 2), (dict(V=1 << 31, ls=1 << 31), 2),
    (dict(K=0), 2), (dict(K=1025), 2), (dict(ls=999), 2), (dict(gs=999), 2),
    (dict(grad=256, gs=1008), 2), (dict(dtype=3), 3), (dict(tdt=-1), 3), (dict(ib=2), 3),
    (dict(temp=0.0), 4), (dict(temp=-1.0), 4), (dict(temp=float("nan")), 4),
    (dict(temp=float("inf")), 4), (dict(temp=1e-39), 4),
    (dict(logits=0), 1), (dict(top=0), 1), (dict(at=0), 1),
    (dict(logits=257), 5), (dict(logits=258, dtype=2), 5), (dict(top=258), 5), (dict(at=260), 5),
    (dict(grad=513), 5), (dict(tl=258), 5), (dict(w=258), 5), (dict(loss=258), 5),
    (dict(lse=258), 5),
    (dict(T=0, logits=0, top=0, at=0), 0), (dict(loss=0, lse=0, grad=0), 0),
])
def test_distill_refusals(lib, kw, want):
    assert call(lib, **kw) == want


def test_distill_binding_refusals(lib):
    torch = pytest.importorskip("torch")
    z = torch.zeros(2, 10, dtype=torch.float16)
    with pytest.raises(ValueError):                    # no CPU path
        lib.hqq_distill(z, torch.zeros(2, 3), torch.zeros(2, 3, dtype=torch.int64))
