"""GPU tests of the adapter calls on values that are not finite: an output is NaN
where its formula gives NaN, not finite where that is not, and keeps its bits where
the formula does not see the bad value.

The NaNs are those that the GPU's own arithmetic makes (all bits but the sign set),
besides the ones of a literal: what splits a value into halves by its bits has to
keep both."""
import math

import pytest

from test_adapters_gpu import (TYPES, adapters, backward_ref, forward_ref, indices, matrix, to_gpu,
                               tokens)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

# NaN of fp32 arithmetic, of a literal, with the sign set, and signalling in the lowest bit
NANS = {torch.float32: (0x7fffffff, 0x7fc00000, -1, 0x7f800001),
        torch.float16: (0x7fff, 0x7e00, -1, 0x7c01),
        torch.bfloat16: (0x7fff, 0x7fc0, -1, 0x7f81)}


@pytest.fixture(scope="module")
def hqq():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import weight_only_quantization_b200 as m
    return m


def nan_of(dtype, which):
    bits = torch.int32 if dtype == torch.float32 else torch.int16
    return torch.tensor([NANS[dtype][which]], dtype=bits, device="cuda").view(dtype)


def run(hqq, q, ad, index, X, dY):
    Y = hqq.hqq_linear_adapters(X, q, ad, index)
    return (Y, *hqq.hqq_linear_adapters_backward(dY, X, q, ad, index))


def check(hqq, q, W, ad, index, X, dY, clean):
    """NaN where the formulas in 64 bits give it, not finite where they are not; the
    clean call's bits elsewhere."""
    got = run(hqq, q, ad, to_gpu(index), X.cuda(), dY.cuda())
    torch.cuda.synchronize()
    want = [forward_ref(X.cpu(), W, ad, index)[0]]
    want += [w for w, _ in backward_ref(dY.cpu(), X.cpu(), W, ad, index)]
    seen = 0
    for g, w, c, name in zip(got, want, clean, ("Y", "dX", "dA", "dB")):
        g = g.cpu()
        nan, same = torch.isnan(w), torch.isfinite(w)
        # (an infinity times the two halves of an fp32 value may be inf - inf)
        assert torch.equal(torch.isfinite(g), same), (name, int((~same).sum()),
                                                      int((~torch.isfinite(g)).sum()))
        assert bool(torch.isnan(g)[nan].all()), name
        assert torch.equal(g[same], c.cpu()[same]), name
        seen += int(nan.sum())
    assert seen > 0


def setup(hqq, dtype, M, rank, kind="mixed"):
    rows, cols, count = 200, 320, 1 if kind == "one" else 3
    q, W = matrix(hqq, rows, cols, 4, 64, seed=rank)
    ad = adapters(hqq, count, rank, rows, cols, TYPES[dtype], seed=rank)
    index = indices(M, count, kind, 3)
    if index is not None:
        index[1] = 1                                     # the token that tests change
    X, dY = tokens(M, cols, 6), tokens(M, rows, 7, 0.25)
    clean = run(hqq, q, ad, to_gpu(index), X.cuda(), dY.cuda())
    return q, W, ad, index, X, dY, clean


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("M", [4, 70, 300])
@pytest.mark.parametrize("rank", [5, 16, 40])
@pytest.mark.parametrize("which", range(4))
def test_nan_in_a_factor(hqq, dtype, M, rank, which):
    """In A: its tokens' T, hence their whole rows of Y and a column of dB, and one
    column of dX; in B: one feature of Y, and P, hence rows of dX and dA."""
    q, W, ad, index, X, dY, clean = setup(hqq, dtype, M, rank)
    for name, place in (("A", (1, rank - 1, 37)), ("B", (1, 11, rank // 2))):
        F = getattr(ad, name)
        old = F[place].clone()
        F[place] = nan_of(F.dtype, which)[0]
        check(hqq, q, W, ad, index, X, dY, clean)
        F[place] = old


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("M", [4, 70])
def test_nan_in_the_one_adapter(hqq, dtype, M):
    """One adapter for every token (no index): no block of tokens is mixed."""
    q, W, ad, index, X, dY, clean = setup(hqq, dtype, M, 16, "one")
    for name in ("A", "B"):
        F = getattr(ad, name)
        old = F[0, 7, 9].clone()
        F[0, 7, 9] = nan_of(F.dtype, 0)[0]
        check(hqq, q, W, ad, index, X, dY, clean)
        F[0, 7, 9] = old


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("M", [4, 70])
@pytest.mark.parametrize("which", range(3))
def test_nan_in_one_operand_alone(hqq, dtype, M, which):
    """NaN in X alone reaches dB through T, NaN in dY alone reaches dA through P."""
    q, W, ad, index, X, dY, clean = setup(hqq, dtype, M, 16)
    X2, dY2 = X.clone(), dY.clone()
    X2[1, 100] = nan_of(torch.float16, which)[0].cpu()
    check(hqq, q, W, ad, index, X2, dY, clean)
    dY2[1, 100] = nan_of(torch.float16, which)[0].cpu()
    check(hqq, q, W, ad, index, X, dY2, clean)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("M", [4, 70])
def test_infinities_of_both_signs_in_the_gradient(hqq, dtype, M):
    """An overflowed dY: B's rows at its two places are equal, so P = inf - inf is NaN
    and with it the token's dX and its adapter's whole dA; dB has infinities at the two
    rows alone."""
    q, W, ad, index, X, dY, clean = setup(hqq, dtype, M, 16)
    ad.B[1, 20] = ad.B[1, 150]
    clean = run(hqq, q, ad, to_gpu(index), X.cuda(), dY.cuda())
    dY2 = dY.clone()
    dY2[1, 20], dY2[1, 150] = math.inf, -math.inf
    check(hqq, q, W, ad, index, X, dY2, clean)
    dA, dB = hqq.hqq_linear_adapters_backward(dY2.cuda(), X.cuda(), q, ad, to_gpu(index))[1:]
    assert bool(torch.isnan(dA[1]).all()) and not bool(torch.isfinite(dB[1, [20, 150]]).any())


def test_factor_near_the_largest_value(hqq):
    """A value that rounding to eleven bits would carry to infinity: T = A X and
    dB = dY T are exact here."""
    rows, cols = 128, 256
    q, _ = matrix(hqq, rows, cols, 4, 64, seed=1)
    big = torch.tensor([0x7f7ff800], dtype=torch.int32).view(torch.float32)[0]
    ad = hqq.Adapters(torch.zeros(1, 8, cols).cuda(), torch.zeros(1, rows, 8).cuda())
    ad.A[0, 3, 17] = big
    X, dY = torch.zeros(2, cols).half().cuda(), torch.zeros(2, rows).half().cuda()
    X[1, 17], dY[1, 5] = 1.0, 2.0 ** -10
    dB = hqq.hqq_linear_adapters_backward(dY, X, q, ad)[2].cpu()
    assert float(dB[0, 5, 3]) == float(big) * 2.0 ** -10
    dB[0, 5, 3] = 0.0
    assert bool((dB == 0).all())


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M", [4, 70])
@pytest.mark.parametrize("rank", [1, 5, 8, 13, 16, 40])
def test_an_infinity_among_positive_values(hqq, dtype, M, rank):
    """With every weight and factor positive an infinite X gives a row of infinities,
    and an infinite dY one of dX, whether or not the rank fills the rows of 16 that T
    and P are kept in."""
    rows, cols, count = 200, 320, 3
    q, _ = matrix(hqq, rows, cols, 4, 64, seed=rank)
    q.zero.fill_(-1.0)
    ad = adapters(hqq, count, rank, rows, cols, TYPES[dtype], seed=rank)
    for F in (ad.A, ad.B):
        F.abs_().add_(0.5)
    index = torch.arange(M, dtype=torch.int32) % count
    X, dY = tokens(M, cols, 6), tokens(M, rows, 7, 0.25)
    clean = run(hqq, q, ad, index.cuda(), X.cuda(), dY.cuda())
    X[1, 100] = dY[1, 33] = math.inf
    got = run(hqq, q, ad, index.cuda(), X.cuda(), dY.cuda())
    for g, c in zip(got[:2], clean[:2]):
        assert bool((g[1] == math.inf).all())
        g[1] = c[1] = 0.0
        assert torch.equal(g, c)
