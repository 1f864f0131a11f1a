"""GPU tests of the linear layer with low-rank adapters and of its gradients
(hqq_linear_adapters, hqq_linear_adapters_backward, through the C ABI) against
their formulas in 64 bits on the oracle's dequantized weights.

Tolerances, from the kernels' arithmetic (u = 2^-23, one fp32 addition of a tensor
core, truncating or rounding; D(n) = ceil(n / 16) + 40 additions on any path of a
sum over n, as for hqq_linear):
- quantized product over n terms: 1.001 D(n) u sum |x w|;
- T = s A X: products exact up to the split of an fp32 factor (2^-22), so
  eT = |s| (D(n) u + 2^-21) sum |A X| per element (P = s B^T dY likewise);
- low-rank term: sum_j |F_j| eT_j + (rank + 16) u sum_j |T_j F_j|, and one
  addition to the quantized sum;
- output: half an fp16 step, 2^-11 of the value, or 2^-25;
- dA = P^T X over m tokens: sum |X| eP + (2^-21 + (40 + m / 64) u) sum |P X|: a
  chunk of 64 tokens adds at most 40 times inside the MMAs, and the chunks, token
  halves and cluster parts follow (m / 64 in all); the factor 2^-21 covers the two
  tf32 halves of P; the same for dB.
A defect in a group's scale or an adapter's row moves an output by far more than
these; on small-integer data, where every partial sum is exact, results must be
equal."""
import math

import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -23
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def hqq():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import weight_only_quantization_b200 as m
    return m


def matrix(hqq, rows, cols, nbits, group, seed, integer=False):
    """A quantized matrix of random codes and its W_hat in 64 bits."""
    L = (1 << nbits) - 1
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, L + 1, rows * cols).astype(np.uint8)
    ng = rows * cols // group
    if integer:
        scale = rng.choice(np.array([0.5, 1.0, 2.0], np.float16), ng)
        zero = rng.integers(0, L + 1, ng).astype(np.float16)
    else:
        scale = (0.02 + 0.05 * rng.random(ng)).astype(np.float16)
        zero = (L * rng.random(ng)).astype(np.float16)
    q = hqq.QuantizedMatrix(torch.from_numpy(oracle.pack(codes, nbits)).cuda(),
                            torch.from_numpy(scale.reshape(rows, cols // group)).cuda(),
                            torch.from_numpy(zero.reshape(rows, cols // group)).cuda(),
                            rows, cols, nbits, group)
    Wh = oracle.dequantize(codes, scale, zero, group).reshape(rows, cols)
    return q, torch.from_numpy(Wh.astype(np.float64))


def adapters(hqq, count, rank, rows, cols, dtype, seed, scaling=True):
    g = torch.Generator().manual_seed(seed)
    A = (torch.randn(count, rank, cols, generator=g) / math.sqrt(cols)).to(dtype)
    B = torch.randn(count, rows, rank, generator=g).to(dtype)
    s = torch.rand(count, generator=g) + 0.5 if scaling else None
    return hqq.Adapters(A.cuda(), B.cuda(), None if s is None else s.cuda())


def tokens(M, n, seed, scale=1.0):
    return (scale * torch.randn(M, n, generator=torch.Generator().manual_seed(seed))).half()


def indices(M, count, kind, seed):
    """None; one adapter for each; runs; any, with a quarter of the tokens without."""
    g = torch.Generator().manual_seed(seed)
    if kind == "one":
        return None
    if kind == "none":
        return torch.full((M,), -1, dtype=torch.int32)
    if kind == "runs":
        return (torch.arange(M) * count // M).to(torch.int32)
    i = torch.randint(0, count, (M,), generator=g, dtype=torch.int32)
    off = torch.rand(M, generator=g)
    i[off < 0.15] = -1
    i[off > 0.9] = count + int(seed) % 5               # past the last: none too
    return i


def D(n):
    return -(-n // 16) + 40


def small(X, F, s, index, count):
    """T[m] = s_a F[a] X[m] ([M, rank]) and its tolerance; F [count, rank, n]."""
    M, n = X.shape
    i = torch.zeros(M, dtype=torch.long) if index is None else index.long()
    T = torch.zeros(M, F.shape[1], dtype=torch.float64)
    tol = torch.zeros_like(T)
    for a in range(count):
        at = (i == a).nonzero().view(-1)
        if len(at):
            T[at] = s[a] * (X[at] @ F[a].T)
            tol[at] = abs(s[a]) * (D(n) * U + 2.0 ** -21) * (X[at].abs() @ F[a].abs().T)
    return T, tol, i


def big(X, W, T, eT, i, F, count):
    """X W^T + T_m F[a]^T with its tolerance; F [count, features, rank]."""
    Y = X @ W.T
    tol = 1.001 * D(W.shape[1]) * U * (X.abs() @ W.abs().T)
    for a in range(count):
        at = (i == a).nonzero().view(-1)
        if len(at):
            Y[at] += T[at] @ F[a].T
            tol[at] += eT[at] @ F[a].abs().T + \
                (F.shape[2] + 16) * U * (T[at].abs() @ F[a].abs().T)
    return Y, tol + U * Y.abs() + 2.0 ** -11 * (Y.abs() + tol) + 2.0 ** -25


def data(ad):
    count = ad.A.shape[0]
    s = torch.ones(count, dtype=torch.float64) if ad.scaling is None else ad.scaling.double().cpu()
    return ad.A.double().cpu(), ad.B.double().cpu(), s


def forward_ref(X, W, ad, index):
    A, B, s = data(ad)
    X = X.double()
    T, eT, i = small(X, A, s, index, len(s))
    return big(X, W, T, eT, i, B, len(s))


def backward_ref(dY, X, W, ad, index):
    A, B, s = data(ad)
    X, dY = X.double(), dY.double()
    n = len(s)
    T, eT, i = small(X, A, s, index, n)
    P, eP, _ = small(dY, B.transpose(1, 2), s, index, n)
    dX = big(dY, W.T, P, eP, i, A.transpose(1, 2), n)
    dA, dB = torch.zeros_like(A), torch.zeros_like(B)
    tA, tB = torch.zeros_like(A), torch.zeros_like(B)
    for a in range(n):
        at = (i == a).nonzero().view(-1)
        if not len(at):
            continue
        e = 2.0 ** -21 + (40 + len(at) / 64) * U
        dA[a] = P[at].T @ X[at]
        tA[a] = eP[at].T @ X[at].abs() + e * (P[at].abs().T @ X[at].abs())
        dB[a] = dY[at].T @ T[at]
        tB[a] = dY[at].abs().T @ eT[at] + e * (dY[at].abs().T @ T[at].abs())
    return dX, (dA, tA), (dB, tB)


def close(got, want, what):
    y, tol = want
    err = (got.double().cpu() - y).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), float((err / tol).max()),
                                 bad.nonzero()[:4].tolist())


def to_gpu(i):
    return None if i is None else i.cuda()


def check_both(hqq, q, W, ad, M, index, seed):
    X, dY = tokens(M, q.cols, seed), tokens(M, q.rows, seed + 1, 0.25)
    Y = hqq.hqq_linear_adapters(X.cuda(), q, ad, to_gpu(index))
    got = hqq.hqq_linear_adapters_backward(dY.cuda(), X.cuda(), q, ad, to_gpu(index))
    torch.cuda.synchronize()
    close(Y, forward_ref(X, W, ad, index), "Y")
    for g, w, nm in zip(got, backward_ref(dY, X, W, ad, index), ("dX", "dA", "dB")):
        close(g, w, nm)


@pytest.mark.parametrize("nbits,group", [(3, 64), (4, 64), (2, 32), (8, 128), (1, 16)])
@pytest.mark.parametrize("M", [1, 7, 16, 33, 300])
@pytest.mark.parametrize("kind", ["one", "mixed"])
def test_formats_and_token_counts(hqq, nbits, group, M, kind):
    rows, cols, count = 264, 512, 1 if kind == "one" else 5
    q, W = matrix(hqq, rows, cols, nbits, group, seed=nbits)
    ad = adapters(hqq, count, 16, rows, cols, torch.float16, seed=M)
    check_both(hqq, q, W, ad, M, indices(M, count, kind, M), seed=M)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rank", [1, 5, 8, 16, 24, 33, 64, 100])
@pytest.mark.parametrize("M", [3, 70])
def test_ranks_and_types(hqq, dtype, rank, M):
    rows, cols, count = 200, 320, 3
    q, W = matrix(hqq, rows, cols, 3, 64, seed=rank)
    ad = adapters(hqq, count, rank, rows, cols, TYPES[dtype], seed=rank, scaling=rank % 2 == 0)
    check_both(hqq, q, W, ad, M, indices(M, count, "mixed", rank), seed=rank + M)


@pytest.mark.parametrize("rows,cols,M,nbits,group", [
    (1, 16, 1, 3, 16), (7, 48, 2, 4, 16), (129, 320, 17, 3, 64), (77, 1040, 40, 2, 16),
    (300, 208, 129, 8, 16), (1001, 192, 260, 1, 64), (130, 4112, 9, 3, 16),
    (4100, 64, 90, 3, 64), (64, 8192, 31, 4, 128), (515, 512, 1030, 3, 32)])
@pytest.mark.parametrize("kind", ["runs", "mixed"])
def test_ragged_shapes(hqq, rows, cols, M, nbits, group, kind):
    """Sizes off every tile, rows that are not whole 16-byte runs of dY, one
    token and one row."""
    q, W = matrix(hqq, rows, cols, nbits, group, seed=rows)
    count = 4
    ad = adapters(hqq, count, 8, rows, cols, torch.float16, seed=cols)
    check_both(hqq, q, W, ad, M, indices(M, count, kind, M), seed=rows + M)


@pytest.mark.parametrize("M,kind", [(64, "mixed"), (64, "none"), (200, "runs"), (2, "mixed")])
@pytest.mark.parametrize("count", [1, 40, 300])
def test_many_adapters(hqq, M, kind, count):
    """More adapters than tokens and fewer; adapters without a token get zero
    gradients; a call in which no token has one."""
    rows, cols = 136, 256
    q, W = matrix(hqq, rows, cols, 4, 64, seed=count)
    ad = adapters(hqq, count, 8, rows, cols, torch.float16, seed=count)
    index = indices(M, count, kind, count)
    check_both(hqq, q, W, ad, M, index, seed=count + M)
    if kind == "none":
        X = tokens(M, cols, 5).cuda()
        assert torch.equal(hqq.hqq_linear_adapters(X, q, ad, index.cuda()), hqq.hqq_linear(X, q))


@pytest.mark.parametrize("M", [1, 9, 16, 40, 256, 1100])
@pytest.mark.parametrize("nbits", [3, 4])
def test_exact_on_integer_data(hqq, M, nbits):
    """Small integers: every partial sum is exact in fp32 (and every T and P in
    the tf32 halves), so all outputs equal the exact ones rounded once."""
    rows, cols, count, rank = 264, 2048, 3, 8
    q, W = matrix(hqq, rows, cols, nbits, 64, seed=M, integer=True)
    g = torch.Generator().manual_seed(M)
    A = torch.randint(-1, 2, (count, rank, cols), generator=g).half()
    B = torch.randint(-1, 2, (count, rows, rank), generator=g).half()
    ad = hqq.Adapters(A.cuda(), B.cuda(), torch.tensor([1.0, 2.0, -1.0]).cuda())
    index = indices(M, count, "mixed", M)
    X = torch.randint(-2, 3, (M, cols), generator=g).half()
    dY = torch.randint(-2, 3, (M, rows), generator=g).half()
    Y = hqq.hqq_linear_adapters(X.cuda(), q, ad, index.cuda())
    got = hqq.hqq_linear_adapters_backward(dY.cuda(), X.cuda(), q, ad, index.cuda())
    want = forward_ref(X, W, ad, index)[0]
    assert float(want.abs().max()) < 65504
    assert torch.equal(Y.cpu(), want.half())
    ref = backward_ref(dY, X, W, ad, index)
    for x, (w, _) in zip(got, ref):
        assert float(w.abs().max()) < (65504 if x.dtype == torch.float16 else 2 ** 24)
        assert torch.equal(x.cpu(), w.to(x.dtype))


@pytest.mark.parametrize("rows,cols", [(2048, 200 * 16), (8192, 272)])
@pytest.mark.parametrize("nbits", [1, 2, 3, 4, 8])
@pytest.mark.parametrize("M", [5, 24, 64, 100, 300, 1030])
def test_input_gradient_exact(hqq, rows, cols, nbits, M):
    """dX = dY W_hat alone, bit for bit on small integers, at long reductions,
    columns off the 128-wide tile and every token tile (24: split reduction)."""
    q, W = matrix(hqq, rows, cols, nbits, 16, seed=M + nbits, integer=True)
    g = torch.Generator().manual_seed(M)
    lim = 1 if nbits == 8 else 2
    dY = torch.randint(-lim, lim + 1, (M, rows), generator=g).half()
    dX, dA, dB = hqq.hqq_linear_adapters_backward(dY.cuda(), None, q)
    assert dA is None and dB is None
    want = dY.double() @ W
    assert float((dY.abs().double() @ W.abs()).max()) * 2 < 2 ** 24
    assert torch.equal(dX.cpu(), want.half())


def test_lowrank_residual_as_adapter(hqq):
    """The data-free residual of the quantization error (2-D fp32 factors) moves
    the layer's output towards the unquantized one, as the formula says."""
    g = torch.Generator().manual_seed(3)
    W16 = (0.02 * torch.randn(256, 512, generator=g)).half().cuda()
    q = hqq.hqq_quantize(W16, nbits=2, group=64)
    B, A, _ = hqq.hqq_lowrank(W16, q, 16, torch.randn(512, 32, generator=g).cuda())
    ad = hqq.Adapters(A, B)
    X = tokens(48, 512, 4)
    W = hqq.hqq_dequantize(q).double().cpu()
    full = hqq.Adapters(A.unsqueeze(0), B.unsqueeze(0))
    close(hqq.hqq_linear_adapters(X.cuda(), q, ad), forward_ref(X, W, full, None), "Y")
    got = hqq.hqq_linear_adapters_backward(tokens(48, 256, 5).cuda(), X.cuda(), q, ad)
    for x, w in zip(got, backward_ref(tokens(48, 256, 5), X, W, full, None)):
        close(x, w, "gradients")


@pytest.mark.parametrize("M", [4, 50])
def test_meta_8bit(hqq, M):
    """Zero points and scales in 8-bit form: the result of the restored matrix."""
    rows, cols, group = 128, 512, 64
    q, _ = matrix(hqq, rows, cols, 3, group, seed=1)
    zq = hqq.hqq_meta_quantize(q.zero.view(-1), 0)
    sq = hqq.hqq_meta_quantize(q.scale.view(-1), 128)
    W = hqq.hqq_dequantize_meta(q.packed, zq, rows, cols, 3, group, scale_q=sq).double().cpu()
    ad = adapters(hqq, 2, 16, rows, cols, torch.float16, seed=2)
    index = indices(M, 2, "mixed", 3)
    bare = hqq.QuantizedMatrix(q.packed, None, None, rows, cols, 3, group)
    X, dY = tokens(M, cols, 6), tokens(M, rows, 7)
    Y = hqq.hqq_linear_adapters(X.cuda(), bare, ad, index.cuda(), zero_q=zq, scale_q=sq)
    close(Y, forward_ref(X, W, ad, index), "Y")
    got = hqq.hqq_linear_adapters_backward(dY.cuda(), X.cuda(), bare, ad, index.cuda(),
                                           zero_q=zq, scale_q=sq)
    for x, w in zip(got, backward_ref(dY, X, W, ad, index)):
        close(x, w, "gradients")


@pytest.mark.parametrize("M", [6, 80])
def test_strides_offsets_and_parts(hqq, M):
    """Adapters in a larger pool (strided, not 16-byte aligned), packed codes off
    16 bytes, outputs left out one at a time, and guard values behind outputs."""
    rows, cols, rank, count = 137, 272, 16, 3
    q, W = matrix(hqq, rows, cols, 3, 16, seed=9)
    pool = torch.randn(count, rank * cols + 3, generator=torch.Generator().manual_seed(1))
    poolB = torch.randn(count, rows * rank + 1, generator=torch.Generator().manual_seed(2))
    for dt in TYPES.values():
        a, b = pool.to(dt).cuda(), poolB.to(dt).cuda()
        ad = hqq.Adapters(a[:, 1:1 + rank * cols].unflatten(1, (rank, cols)),
                          b[:, 1:].unflatten(1, (rows, rank)),
                          torch.tensor([0.5, 1.0, 2.0]).cuda())
        check_both(hqq, q, W, ad, M, indices(M, count, "mixed", 2), seed=3)
    raw = torch.zeros(q.packed.numel() + 64, dtype=torch.uint8, device="cuda")
    off = (16 - raw.data_ptr() % 16) % 16 + 4
    raw[off:off + q.packed.numel()] = q.packed
    q2 = hqq.QuantizedMatrix(raw[off:off + q.packed.numel()], q.scale, q.zero, rows, cols, 3, 16)
    check_both(hqq, q2, W, ad, M, indices(M, count, "runs", 2), seed=4)
    X, dY = tokens(M, cols, 6).cuda(), tokens(M, rows, 7).cuda()
    index = indices(M, count, "mixed", 5).cuda()
    dX, dA, dB = hqq.hqq_linear_adapters_backward(dY, X, q, ad, index)
    only = hqq.hqq_linear_adapters_backward(dY, None, q, ad, index, need_factors=False)
    assert torch.equal(only[0], dX) and only[1] is None and only[2] is None
    only = hqq.hqq_linear_adapters_backward(dY, X, q, ad, index, need_dX=False)
    assert only[0] is None and torch.equal(only[1], dA) and torch.equal(only[2], dB)
    # what lies behind the outputs and the workspace stays as it was
    need = hqq._lib.hqq_linear_adapters_workspace_bytes(M, rows, cols, rank, count, 1)
    ws = torch.full((need + 512,), 77, dtype=torch.uint8, device="cuda")
    bufs = [torch.full((t.numel() + 32,), 5.0, dtype=t.dtype, device="cuda") for t in (dX, dA, dB)]
    outs = [b[:t.numel()].view(t.shape) for b, t in zip(bufs, (dX, dA, dB))]
    hqq.hqq_linear_adapters_backward(dY, X, q, ad, index, dX=outs[0], dA=outs[1], dB=outs[2],
                                     workspace=ws[:need])
    assert all(torch.equal(o, t) for o, t in zip(outs, (dX, dA, dB)))
    assert all(bool((b[-32:] == 5).all()) for b in bufs) and bool((ws[need:] == 77).all())
    Y = hqq.hqq_linear_adapters(X, q, ad, index)
    buf = torch.full((Y.numel() + 32,), 5.0, dtype=Y.dtype, device="cuda")
    out = hqq.hqq_linear_adapters(X, q, ad, index, out=buf[:Y.numel()].view(Y.shape))
    assert torch.equal(out, Y) and bool((buf[-32:] == 5).all())


@pytest.mark.parametrize("M", [12, 90])
def test_tokens_do_not_reach_each_other(hqq, M):
    """A token of NaN and infinities leaves the other tokens' outputs and, where
    it has another adapter, the other adapters' gradients as they were; adapters
    of NaN that no token has are not used."""
    rows, cols, count = 200, 256, 4
    q, W = matrix(hqq, rows, cols, 4, 64, seed=4)
    ad = adapters(hqq, count, 16, rows, cols, torch.float16, seed=8)
    index = torch.arange(M, dtype=torch.int32) % 3           # adapter 3: no token
    index[5] = -1
    X, dY = tokens(M, cols, 6).cuda(), tokens(M, rows, 7).cuda()
    Y = hqq.hqq_linear_adapters(X, q, ad, index.cuda())
    base = hqq.hqq_linear_adapters_backward(dY, X, q, ad, index.cuda())
    ad.A[3] = math.nan
    ad.B[3] = math.inf
    X2, dY2 = X.clone(), dY.clone()
    X2[1] = math.nan
    dY2[1] = math.inf
    X2[5] = math.inf
    Y2 = hqq.hqq_linear_adapters(X2, q, ad, index.cuda())
    got = hqq.hqq_linear_adapters_backward(dY2, X2, q, ad, index.cuda())
    keep = torch.ones(M, dtype=torch.bool)
    keep[[1, 5]] = False
    assert torch.equal(Y2[keep], Y[keep])
    keep[5] = True
    assert torch.equal(got[0][keep], base[0][keep])
    for a in (0, 2):
        assert torch.equal(got[1][a], base[1][a]) and torch.equal(got[2][a], base[2][a])
    assert bool((got[1][3] == 0).all()) and bool((got[2][3] == 0).all())
    assert not bool(torch.isfinite(got[1][1]).all())


def test_results_do_not_depend_on_order_of_adapters(hqq):
    """The same bits whatever the adapters are numbered, and from call to call."""
    rows, cols, M, count = 264, 512, 150, 6
    q, _ = matrix(hqq, rows, cols, 3, 64, seed=5)
    ad = adapters(hqq, count, 16, rows, cols, torch.float16, seed=5)
    index = indices(M, count, "mixed", 1).cuda()
    X, dY = tokens(M, cols, 6).cuda(), tokens(M, rows, 7).cuda()
    Y = hqq.hqq_linear_adapters(X, q, ad, index)
    g = hqq.hqq_linear_adapters_backward(dY, X, q, ad, index)
    flip = hqq.Adapters(ad.A.flip(0).contiguous(), ad.B.flip(0).contiguous(),
                        ad.scaling.flip(0).contiguous())
    index2 = torch.where((index >= 0) & (index < count), count - 1 - index, index)
    assert torch.equal(hqq.hqq_linear_adapters(X, q, flip, index2), Y)
    g2 = hqq.hqq_linear_adapters_backward(dY, X, q, flip, index2)
    assert torch.equal(g2[0], g[0])
    assert torch.equal(g2[1].flip(0), g[1]) and torch.equal(g2[2].flip(0), g[2])
    for _ in range(3):
        again = hqq.hqq_linear_adapters_backward(dY, X, q, ad, index)
        assert all(torch.equal(a, b) for a, b in zip(again, g))


def test_gradients_against_differences(hqq):
    """sum(dY * Y) is linear in X, A and B each, so its difference along a
    direction equals the gradient's product with it, up to the rounding of the
    fp16 outputs: half a step (2^-11) of every |Y| and dX, each weighted."""
    rows, cols, M, count = 136, 256, 40, 2
    q, _ = matrix(hqq, rows, cols, 4, 64, seed=6)
    ad = adapters(hqq, count, 8, rows, cols, torch.float32, seed=6)
    index = indices(M, count, "mixed", 2).cuda()
    X, dY = tokens(M, cols, 6).cuda(), tokens(M, rows, 7).cuda()
    dX, dA, dB = (t.double() for t in hqq.hqq_linear_adapters_backward(dY, X, q, ad, index))

    def value(X, A, B):
        Y = hqq.hqq_linear_adapters(X, q, hqq.Adapters(A, B, ad.scaling), index).double()
        return float((dY.double() * Y).sum()), float((dY.double() * Y).abs().sum())
    g = torch.Generator().manual_seed(1)
    for wrt in range(3):
        args = [X, ad.A, ad.B]
        d = torch.randint(0, 2, args[wrt].shape, generator=g).cuda() * 2 - 1
        step = d.to(args[wrt].dtype) * 2.0 ** -2
        up, dn = list(args), list(args)
        up[wrt], dn[wrt] = args[wrt] + step, args[wrt] - step
        move = (up[wrt].double() - dn[wrt].double())           # what the rounded steps are
        (a, sa), (b, sb) = value(*up), value(*dn)
        grad = (dX, dA, dB)[wrt]
        want = float((grad * move).sum())
        tol = 2.0 ** -11 * (sa + sb + float((grad * move).abs().sum())) * 1.01
        assert abs((a - b) - want) <= tol, (wrt, a - b, want, tol)


def test_streams_graphs_and_workspaces(hqq):
    """A side stream, two captured graphs with a workspace each replayed side by
    side, and eager calls between them: the same bits everywhere."""
    rows, cols, count = 264, 512, 3
    q, _ = matrix(hqq, rows, cols, 3, 64, seed=7)
    ad = adapters(hqq, count, 16, rows, cols, torch.float16, seed=7)
    for M in (5, 100):
        index = indices(M, count, "mixed", 4).cuda()
        X, dY = tokens(M, cols, 6).cuda(), tokens(M, rows, 7).cuda()
        Y = hqq.hqq_linear_adapters(X, q, ad, index)
        g = hqq.hqq_linear_adapters_backward(dY, X, q, ad, index)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            Y2 = hqq.hqq_linear_adapters(X, q, ad, index, status=status)
            g2 = hqq.hqq_linear_adapters_backward(dY, X, q, ad, index, status=status)
        side.synchronize()
        assert torch.equal(Y, Y2) and all(torch.equal(a, b) for a, b in zip(g, g2))
        assert int(status) == 0
        graphs, outs = [], []
        Xg, dYg, ig = torch.zeros_like(X), torch.zeros_like(dY), torch.full_like(index, -1)
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                outs.append((hqq.hqq_linear_adapters(Xg, q, ad, ig),
                             *hqq.hqq_linear_adapters_backward(dYg, Xg, q, ad, ig)))
            graphs.append(graph)
        Xg.copy_(X)
        dYg.copy_(dY)
        ig.copy_(index)
        torch.cuda.synchronize()
        for _ in range(3):
            for graph, s in zip(graphs, (side, torch.cuda.Stream())):
                with torch.cuda.stream(s):
                    graph.replay()
            mid = hqq.hqq_linear_adapters(X, q, ad, index)
            torch.cuda.synchronize()
            assert torch.equal(mid, Y)
            for o in outs:
                assert torch.equal(o[0], Y) and all(torch.equal(a, b) for a, b in zip(o[1:], g))


def test_empty_calls(hqq):
    rows, cols, count = 128, 256, 2
    q, _ = matrix(hqq, rows, cols, 4, 64, seed=8)
    ad = adapters(hqq, count, 8, rows, cols, torch.float16, seed=8)
    X = torch.zeros(0, cols, dtype=torch.float16, device="cuda")
    dY = torch.zeros(0, rows, dtype=torch.float16, device="cuda")
    index = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert hqq.hqq_linear_adapters(X, q, ad, index).shape == (0, rows)
    dA = torch.full((count, 8, cols), 3.0, device="cuda")
    dB = torch.full((count, rows, 8), 3.0, device="cuda")
    dX, _, _ = hqq.hqq_linear_adapters_backward(dY, X, q, ad, index, dA=dA, dB=dB)
    assert dX.shape == (0, cols) and bool((dA == 0).all()) and bool((dB == 0).all())


def test_distilled_step(hqq):
    """The operators as they are used together: student logits from a quantized
    head with adapters, the teacher's top logits from the fp16 head, the loss and
    its gradient, the adapters' gradients and the hidden gradient for the layer
    below, and a step along them, against the same run in 64 bits."""
    V, H, M, K = 1000, 256, 24, 16
    g = torch.Generator().manual_seed(11)
    Wh = (0.08 * torch.randn(V, H, generator=g)).half().cuda()
    q = hqq.hqq_quantize(Wh, nbits=3, group=64)
    ad = adapters(hqq, 2, 8, V, H, torch.float32, seed=12)
    ad.B *= 0.05
    index = (torch.arange(M) % 2).to(torch.int32)
    h = tokens(M, H, 13)
    top, at = torch.topk(h.cuda().float() @ Wh.float().T, K, dim=1)
    weight = torch.full((M,), 64.0, device="cuda")
    weight[3] = 0.0
    logits = hqq.hqq_linear_adapters(h.cuda(), q, ad, index.cuda())
    loss, _, dlogits = hqq.hqq_distill(logits, top, at, 1.0, weight=weight, grad=True)
    dX, dA, dB = hqq.hqq_linear_adapters_backward(dlogits, h.cuda(), q, ad, index.cuda())
    step = hqq.Adapters(ad.A - 1e-3 * dA, ad.B - 1e-3 * dB, ad.scaling)
    after = hqq.hqq_linear_adapters(h.cuda(), q, step, index.cuda())
    torch.cuda.synchronize()
    # each stage against 64 bits on the stage's own (rounded) inputs
    W = hqq.hqq_dequantize(q).double().cpu()
    close(logits, forward_ref(h, W, ad, index), "logits")
    z = logits.double().cpu().requires_grad_()
    t, a = top.double().cpu(), at.cpu()
    p = torch.softmax(t, 1)
    kl = (p * (torch.log(p) - torch.log_softmax(z, 1).gather(1, a))).sum(1) * weight.double().cpu()
    kl.sum().backward()
    # fp32 arithmetic with |logits| < 16, 1000 + 16 terms: below 2^-16 of the weights
    assert float((loss.double().cpu() - kl.detach()).abs().max()) <= 64 * 2.0 ** -16
    err = (dlogits.double().cpu() - z.grad).abs()
    assert bool((err <= 2.0 ** -11 * z.grad.abs() + 64 * 2.0 ** -16 * z.grad.abs() + 2.0 ** -14
                 * (p.sum(1).max() * 2.0 ** -4)).all())
    for x, w, nm in zip((dX, dA, dB), backward_ref(dlogits.cpu(), h, W, ad, index), "XAB"):
        close(x, w, "d" + nm)
    close(after, forward_ref(h, W, step, index), "after")


@pytest.mark.parametrize("rows,cols,M", [(3200, 2048, 300), (3200, 2064, 777), (4103, 1024, 2048),
                                         (2176, 8192, 1030), (1024, 4112, 129)])
@pytest.mark.parametrize("nbits", [3, 4])
def test_large_tiles_exact(hqq, rows, cols, M, nbits):
    """Token tiles of up to 512, pairs of CTAs, reductions split over a cluster
    and their combinations, bit for bit on small integers."""
    count, rank = 3, 8
    q, W = matrix(hqq, rows, cols, nbits, 16, seed=M, integer=True)
    g = torch.Generator().manual_seed(M)
    A = torch.randint(-1, 2, (count, rank, cols), generator=g).half()
    B = torch.randint(-1, 2, (count, rows, rank), generator=g).half()
    ad = hqq.Adapters(A.cuda(), B.cuda(), torch.tensor([1.0, 2.0, -1.0]).cuda())
    index = indices(M, count, "mixed" if nbits == 3 else "runs", M)
    X = torch.randint(-1, 2, (M, cols), generator=g).half()
    dY = torch.randint(-1, 2, (M, rows), generator=g).half()
    Y = hqq.hqq_linear_adapters(X.cuda(), q, ad, index.cuda())
    got = hqq.hqq_linear_adapters_backward(dY.cuda(), X.cuda(), q, ad, index.cuda())
    on = (index >= 0) & (index < count)
    i = torch.where(on, index, 0).long()
    s = ad.scaling.cpu().double()[i] * on
    x, y, w = X.double().cuda(), dY.double().cuda(), W.cuda()
    hot = (torch.nn.functional.one_hot(i, count) * s[:, None]).cuda()
    T = torch.einsum("mk,ajk,ma->maj", x, A.double().cuda(), hot)
    P = torch.einsum("mn,anj,ma->maj", y, B.double().cuda(), hot)
    want = x @ w.T + torch.einsum("maj,anj->mn", T, B.double().cuda())
    assert float(want.abs().max()) < 65504 and torch.equal(Y, want.half())
    want = y @ w + torch.einsum("maj,ajk->mk", P, A.double().cuda())
    assert float(want.abs().max()) < 65504 and torch.equal(got[0], want.half())
    dA, dB = torch.einsum("maj,mk->ajk", P, x), torch.einsum("maj,mn->anj", T, y)
    assert max(float(dA.abs().max()), float(dB.abs().max())) < 2 ** 24
    assert torch.equal(got[1], dA.float()) and torch.equal(got[2], dB.float())


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rank", [40, 104, 512])
@pytest.mark.parametrize("kind", ["one", "runs", "mixed"])
def test_high_ranks_on_many_tokens(hqq, dtype, rank, kind):
    """Several passes of 16 ranks over the sums, in tiles of one adapter and of
    several; 512 ranks do not fit beside the tile in shared memory."""
    rows, cols, M, count = 264, 528, 300, 1 if kind == "one" else 3
    q, W = matrix(hqq, rows, cols, 4, 16, seed=rank)
    ad = adapters(hqq, count, rank, rows, cols, TYPES[dtype], seed=rank)
    check_both(hqq, q, W, ad, M, indices(M, count, kind, rank), seed=rank)


@pytest.mark.parametrize("M", [12, 70, 300, 700])
@pytest.mark.parametrize("rank", [16, 40])
def test_a_token_does_not_depend_on_the_others_adapters(hqq, M, rank):
    """The same bits for a token whether its neighbours have its adapter, others
    or none."""
    rows, cols, count = 264, 512, 4
    q, _ = matrix(hqq, rows, cols, 3, 64, seed=M)
    ad = adapters(hqq, count, rank, rows, cols, torch.float16, seed=rank)
    X, dY = tokens(M, cols, 6).cuda(), tokens(M, rows, 7).cuda()
    other = indices(M, count, "mixed", 3).cuda()
    pick = int(other[(other >= 0) & (other < count)][0])        # an adapter that some have
    same = torch.full((M,), pick, dtype=torch.int32, device="cuda")
    Y = hqq.hqq_linear_adapters(X, q, ad, same)
    Z = hqq.hqq_linear_adapters(X, q, ad, other)
    dX = hqq.hqq_linear_adapters_backward(dY, None, q, ad, same, need_factors=False)[0]
    dZ = hqq.hqq_linear_adapters_backward(dY, None, q, ad, other, need_factors=False)[0]
    at = other == pick
    assert torch.equal(Y[at], Z[at]) and torch.equal(dX[at], dZ[at])
