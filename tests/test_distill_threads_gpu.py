"""hqq_distill from several host threads at once, each on a stream of its own."""
import ctypes
import threading

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def test_rows_of_different_lengths_from_several_threads():
    """Short rows (little shared memory) and long ones beside each other, as calls of
    the library with the arguments made beforehand: the threads spend their time inside
    it, where the interpreter's lock is free.  Every call is accepted and gives the bits
    it gives alone."""
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import weight_only_quantization_b200 as hqq
    work = []
    for tokens, vocab, k in ((2, 1000, 2), (200, 32000, 64), (2, 200, 1), (200, 24000, 5)):
        g = torch.Generator().manual_seed(vocab)
        z = torch.randn(tokens, vocab, generator=g).bfloat16().cuda()
        top, at = torch.topk(z.float(), k, dim=1)
        top, at = top.contiguous(), at.contiguous()
        want = hqq.hqq_distill(z, top, at, grad=True)
        stream = torch.cuda.Stream()
        outs = [torch.empty_like(w) for w in want]
        p = ctypes.c_void_p
        i = ctypes.c_int64
        args = (p(z.data_ptr()), i(vocab), 1, i(tokens), i(vocab), p(top.data_ptr()), 2,
                p(at.data_ptr()), 8, i(k), ctypes.c_float(1.0), None, None,
                p(outs[0].data_ptr()), p(outs[1].data_ptr()), p(outs[2].data_ptr()), i(vocab),
                p(stream.cuda_stream))
        work.append((args, stream, (z, top, at), outs, want))
    torch.cuda.synchronize()
    statuses = [[] for _ in work]
    go = threading.Barrier(len(work))

    def caller(which):
        args, fn = work[which][0], hqq._lib.hqq_distill
        go.wait()
        statuses[which] = [fn(*args) for _ in range(4000)]

    threads = [threading.Thread(target=caller, args=(n,)) for n in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert all(len(s) == 4000 for s in statuses)
    assert [sum(v != 0 for v in s) for s in statuses] == [0] * len(work)
    for _, _, _, outs, want in work:
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
