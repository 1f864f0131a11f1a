"""The wait of hqq_distill for a row's copy, run out: the kernel is built here from its
source without the copy, so that nothing ever reports to the barrier.  The wait ends by
its own limit (about a second), every output of the tokens that wait is NaN, and the
GPU carries on."""
import ctypes
import importlib.util
import os
import re
import subprocess

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "weight_only_quantization_b200")

CALL = """
extern "C" int without_copy(const void* logits, void* grad, const void* top, const void* at,
                            const float* weight, float* loss, float* lse, long tokens, long vocab,
                            int k, int dtype) {
    hqq::DistillParams p = {};
    p.logits = logits;
    p.grad = grad;
    p.top = top;
    p.at = at;
    p.weight = weight;
    p.loss = loss;
    p.lse = lse;
    p.T = tokens;
    p.V = p.logits_stride = p.grad_stride = vocab;
    p.K = k;
    p.top_dtype = 2;
    p.at64 = 1;
    p.hash_mask = 63;
    p.inv_t = 1.0f;
    p.log2e_t = 1.44269504f;
    return (int)hqq::launch_distill(p, dtype, nullptr);
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    spec = importlib.util.spec_from_file_location("hqq_build", os.path.join(PKG, "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    src = open(os.path.join(PKG, "csrc", "hqq_distill.cu")).read()
    src, n = re.subn(r'if \(bytes\)\s*asm volatile\(\s*"cp\.async\.bulk\..*?: "memory"\);', "", src,
                     flags=re.S)
    assert n == 1
    out = tmp_path_factory.mktemp("wait")
    path = str(out / "without_copy.cu")
    with open(path, "w") as f:
        f.write(src + CALL)
    so = str(out / "without_copy.so")
    res = subprocess.run(["nvcc", *build.COMPILE_FLAGS, "-I", os.path.join(PKG, "csrc"), "-shared",
                          "-cudart", "static", path, "-o", so], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    return ctypes.CDLL(so)


@pytest.mark.parametrize("tokens,vocab", [(3, 2000), (3, 300007)])
def test_a_row_that_never_arrives_gives_nan(lib, tokens, vocab):
    g = torch.Generator().manual_seed(1)
    z = torch.randn(tokens, vocab, generator=g).bfloat16().cuda()
    top, at = torch.topk(z.float(), 4, dim=1)
    top, at = top.contiguous(), at.contiguous()
    weight = torch.tensor([1.0, 0.0, 2.0], device="cuda")
    loss, lse = (torch.full((tokens,), 5.0, device="cuda") for _ in range(2))
    grad = torch.full_like(z, 5.0)
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    torch.cuda.synchronize()
    st = lib.without_copy(p(z), p(grad), p(top), p(at), p(weight), p(loss), p(lse),
                          ctypes.c_long(tokens), ctypes.c_long(vocab), 4, 1)
    assert st == 0
    torch.cuda.synchronize()
    for i in (0, 2):
        assert bool(torch.isnan(loss[i])) and bool(torch.isnan(lse[i]))
        assert bool(torch.isnan(grad[i]).all())
    # a token of weight 0 waits for nothing
    assert float(loss[1]) == 0.0 and float(lse[1]) == 0.0 and bool((grad[1] == 0).all())
    # the context is usable
    import weight_only_quantization_b200 as hqq
    out = hqq.hqq_distill(z, top, at, weight=weight, grad=True)
    assert all(bool(torch.isfinite(o).all()) for o in out)
