"""Calls given a stream of their own beside work queued on the current one: neither side
gets memory that the other still uses."""
import pytest

from test_adapters_gpu import adapters, indices, matrix, tokens

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

CYCLES = 20_000_000            # of a queued delay: about 10 ms


@pytest.fixture(scope="module")
def calls():
    """name -> the call (stream=None) with inputs made beforehand."""
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import weight_only_quantization_b200 as hqq
    rows, cols, count, M = 264, 512, 3, 300
    q, _ = matrix(hqq, rows, cols, 3, 64, seed=7)
    ad = adapters(hqq, count, 16, rows, cols, torch.float32, seed=7)
    index = indices(M, count, "mixed", 4).cuda()
    X, dY = tokens(M, cols, 6).cuda(), tokens(M, rows, 7).cuda()
    z = torch.randn(M, 4000, generator=torch.Generator().manual_seed(1)).half().cuda()
    top, at = torch.topk(z.float(), 9, dim=1)
    top, at = top.contiguous(), at.contiguous()
    return {
        "adapters": lambda s=None: (hqq.hqq_linear_adapters(X, q, ad, index, stream=s),),
        "few": lambda s=None: (hqq.hqq_linear_adapters(X[:4], q, ad, index[:4], stream=s),),
        "backward": lambda s=None: hqq.hqq_linear_adapters_backward(dY, X, q, ad, index, stream=s),
        "distill": lambda s=None: hqq.hqq_distill(z, top, at, grad=True, stream=s),
    }


@pytest.mark.parametrize("name", ["adapters", "few", "backward", "distill"])
def test_memory_of_a_call_that_waits(calls, name):
    """The call's kernels wait behind a delay while the current stream allocates and
    fills blocks of every size that the call can have had."""
    want = calls[name]()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(CYCLES)
        got = calls[name](side)
        junk = [torch.full((n,), 0x5a, dtype=torch.uint8, device="cuda")
                for n in [256 << k for k in range(16)] * 3]
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(bool((j == 0x5a).all()) for j in junk)
        del got, junk


@pytest.mark.parametrize("name", ["adapters", "few", "backward", "distill"])
def test_memory_that_the_current_stream_still_reads(calls, name):
    """Blocks of the results' sizes are freed while the current stream has reads of them
    queued behind a delay; the call must not write them first.  Then results are freed
    with reads queued, and the side stream's next call must not take them."""
    want = calls[name]()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        old = [torch.full_like(w, 3.0) for w in want for _ in range(4)]
        kept = [torch.empty_like(o) for o in old]
        torch.cuda.synchronize()
        torch.cuda._sleep(CYCLES)
        for k, o in zip(kept, old):
            k.copy_(o)
        del old, o
        got = calls[name](side)
        torch.cuda.synchronize()
        assert all(bool((k == 3).all()) for k in kept)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        copies = [torch.empty_like(g) for g in got]
        torch.cuda.synchronize()
        torch.cuda._sleep(CYCLES)
        for c, g in zip(copies, got):
            c.copy_(g)
        del got, g
        with torch.cuda.stream(side):
            junk = [torch.full_like(w, 5.0) for w in want for _ in range(4)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(copies, want))
        del junk


def test_a_stream_as_a_bare_handle(calls):
    """Any object that has a stream's handle is taken as that stream."""
    import types

    import weight_only_quantization_b200 as hqq
    side = torch.cuda.Stream()
    bare = types.SimpleNamespace(cuda_stream=side.cuda_stream)
    for call in calls.values():
        want = call()
        torch.cuda.synchronize()
        got = call(bare)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    q, _ = matrix(hqq, 264, 512, 3, 64, seed=7)
    X = tokens(4, 512, 6).cuda()
    want = hqq.hqq_linear(X, q)
    torch.cuda.synchronize()
    got = hqq.hqq_linear(X, q, stream=bare)
    side.synchronize()
    assert torch.equal(got, want)
