"""GPU tests of the distillation loss (hqq_distill, through the C ABI) against
its definition in 64 bits.

Tolerances, from the kernel's arithmetic, with u = 2^-24 (one fp32 rounding)
and a = |z - max| log2(e) / t:
- an exponential 2^a is formed from a difference, a product and a rounded
  constant (3 u of a each) and ex2.approx (2^-22): relative error
  (3 ln2 a + 4) u <= (2.1 a + 4) u;
- a thread's sum takes 16 pair additions and 4 more per four packs of 16 bytes, at
  most 4 times for a 64 KiB share of the row (12 for the longest kept share),
  then 5 + 3 + 3 joining steps of 2: at most 102 roundings, 262 for rows of more
  than 131072 values; D = 174, and 64 per 16384 values + 110 above, cover
  both, so the sum's relative error is es = (2.1 R + 4 + D) u, with R the
  largest a whose term matters (terms beyond a = 40 are below 2^-40 of the sum);
- p_k likewise: ep = (2.1 Rt + 8 + K / 32 + 8) u + 4 u (|t_k| / t + |L|), the
  second part the rounded difference of two logits;
- loss terms: p_k (log p_k - log q_k), each logarithm a difference of values
  rounded to u, summed in at most K / 32 + 6 steps;
- gradient: w / t (psum q - mass), q to 2 es, mass to ep, then one rounding to
  the output type: at most half a step, eps / 2 of the value, or half the
  smallest subnormal.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -127, torch.float32: 2.0 ** -127}


@pytest.fixture(scope="module")
def hqq():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import weight_only_quantization_b200 as m
    return m


def reference(z, top, at, temp, teacher_lse=None, weight=None):
    """loss, lse, gradient and their tolerances (before the rounding of the
    output type), in 64 bits, from the definition."""
    z = z.double().cpu()
    top, at = top.double().cpu(), at.long().cpu()
    T, V = z.shape
    K = top.shape[1]
    w = torch.ones(T, dtype=torch.float64) if weight is None else weight.double().cpu()
    zt = z / temp
    m = zt.amax(1, keepdim=True)
    d = zt - m
    # softmax and its logarithm from z - max: with values of 1e38, z - lse would
    # lose log(sum) even in 64 bits
    logs = torch.log(torch.exp(d).sum(1))
    lse = m.squeeze(1) + logs
    q = torch.exp(d - logs[:, None])
    valid = (at >= 0) & (at < V) & (top != -math.inf)
    t = torch.where(valid, top / temp, torch.tensor(-math.inf, dtype=torch.float64))
    if teacher_lse is None:
        L = torch.logsumexp(t, 1)
    else:
        L = teacher_lse.double().cpu()
    lp = torch.where(valid, t - L[:, None], torch.zeros_like(t))
    p = torch.where(valid, torch.exp(lp), torch.zeros_like(t))
    place = at.clamp(0, V - 1)
    lq = d.gather(1, place) - logs[:, None]
    terms = torch.where(p > 0, p * (lp - lq), torch.zeros_like(p))
    loss = w * terms.sum(1)
    mass = torch.zeros_like(z).scatter_add_(1, place, p)
    psum = p.sum(1, keepdim=True)
    grad = (w / temp)[:, None] * (psum * q - mass)
    # tolerances
    R = 1.4427 * d.abs().nan_to_num(0.0, posinf=0.0).clamp(max=28.0).amax(1)
    rounds = max(1, -(-V // 16384)) if V > 131072 else 1
    es = (2.1 * R + 4 + 64 * rounds + 110) * U
    tabs = torch.where(valid, t.abs(), torch.zeros_like(t))
    peak = torch.where(valid, t, torch.full_like(t, -math.inf)).amax(1)
    Rt = 1.4427 * torch.where(valid, (t - peak[:, None]).abs(), torch.zeros_like(t)).clamp(max=28.0).amax(1)
    Lf = torch.where(torch.isfinite(L), L.abs(), torch.zeros_like(L))
    ep = ((2.1 * Rt + 16 + K / 32)[:, None] + 4 * (tabs + Lf[:, None])) * U
    dabs = d.gather(1, place).abs()
    per_term = p * ((lp - lq).abs() * (ep + (K / 32 + 8) * U) + 4 * U * (tabs + Lf[:, None])
                    + 4 * U * dabs + (es + 4 * U * (1 + logs.abs()))[:, None] + ep)
    loss_tol = w.abs() * torch.where(p > 0, per_term, torch.zeros_like(p)).sum(1) + 2.0 ** -126
    # (elements beyond a = 40 have their own relative error up to 2.1 a u)
    ea = 2.1 * 1.4427 * d.abs().nan_to_num(0.0, posinf=0.0) * U
    qt = q * psum * (2 * es[:, None] + ea + 4 * U + (ep * p).sum(1, keepdim=True)
                     / psum.clamp(min=1e-300))
    mt = torch.zeros_like(z).scatter_add_(1, place, p * (ep + (K + 4) * U))
    grad_tol = (w.abs() / temp)[:, None] * (qt + mt) + 2.0 ** -126
    lse_tol = es + 4 * U * (1 + lse.abs() + m.squeeze(1).abs() + logs.abs())
    skip = w == 0
    for x in (loss, lse):
        x[skip] = 0.0
    grad[skip] = 0.0
    return loss, lse, grad, loss_tol, lse_tol, grad_tol


def close(got, want, tol, dtype=None):
    got = got.double().cpu()
    if dtype is not None:
        tol = tol * (1 + torch.finfo(dtype).eps) + torch.finfo(dtype).eps / 2 * want.abs() + TINY[dtype]
    nan = torch.isnan(want)
    assert torch.equal(nan, torch.isnan(got))
    inf = torch.isinf(want)
    assert torch.equal(want[inf], got[inf])
    ok = nan | inf | ((got - want).abs() <= tol)
    assert bool(ok.all()), (int((~ok).sum()),
                            float(((got - want).abs() / tol)[~ok].max()))


def inputs(T, V, K, dtype, index, temp, tail, seed, top_dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    z = (torch.randn(T, V, generator=g) * 2 + 6 * (torch.rand(T, V, generator=g) < 0.002)).to(dtype)
    teacher = z.float() + 0.7 * torch.randn(T, V, generator=g)
    top, at = torch.topk(teacher, K, dim=1)
    lse = torch.logsumexp(teacher.double() / temp, 1).float() if tail else None
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    return cuda(z), cuda(top.to(top_dtype)), cuda(at.to(index)), cuda(lse)


SHAPES = [(1, 1, 1), (3, 7, 3), (5, 1000, 32), (2, 1000, 1000), (37, 4100, 65), (2, 32000, 64),
          (300, 32000, 16), (3, 32001, 20), (2, 50001, 128), (2, 131072, 256), (1, 300007, 5),
          (2, 270336, 9)]


@pytest.mark.parametrize("T,V,K", SHAPES)
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("temp,tail", [(1.0, False), (2.0, True)])
def test_distill_shapes_and_types(hqq, T, V, K, dtype, temp, tail):
    index = torch.int64 if tail else torch.int32
    top_dtype = DTYPES[dtype] if V % 2 else torch.float32
    z, top, at, lse = inputs(T, V, K, DTYPES[dtype], index, temp, tail, 1000 * T + V, top_dtype)
    loss, glse, grad = hqq.hqq_distill(z, top, at, temp, teacher_lse=lse, grad=True)
    torch.cuda.synchronize()
    want = reference(z, top, at, temp, lse)
    close(loss, want[0], want[3])
    close(glse, want[1], want[4])
    close(grad, want[2], want[5], DTYPES[dtype])


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_distill_without_gradient_gives_the_same_loss(hqq, dtype):
    z, top, at, _ = inputs(9, 5003, 17, DTYPES[dtype], torch.int64, 1.5, False, 3)
    a = hqq.hqq_distill(z, top, at, 1.5, grad=True)
    b = hqq.hqq_distill(z, top, at, 1.5)
    assert b[2] is None
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("V", [640, 40000, 300000])
def test_distill_masked_logits_and_entries(hqq, dtype, V):
    """Logits masked with -inf or the type's lowest value (whole CTA shares of
    them), equal rows, unused, repeated and massless entries, weights."""
    dt = DTYPES[dtype]
    T, K = 9, 12
    z, top, at, _ = inputs(T, V, K, dt, torch.int64, 1.0, False, 7)
    low = torch.finfo(dt).min
    z[1, V // 3:] = -math.inf
    at[1] %= V // 3
    z[2, V // 8:] = low
    at[2] %= V // 8
    z[3, :] = low                              # a row whose mask leaves nothing: uniform
    z[4, :] = 1.25
    at[5, 3] = -1
    at[5, 4] = V
    at[5, 5] = at[5, 0]                        # the same index three times
    at[5, 9] = at[5, 0]
    at[6, :] = -1                              # no entry at all
    top[7, 2] = -math.inf
    top[7, 5:] = -math.inf
    weight = torch.tensor([1, 0.5, 2, 1, 1, 1, 1, 1, -0.25], device="cuda")
    loss, lse, grad = hqq.hqq_distill(z, top, at, 1.0, weight=weight, grad=True)
    torch.cuda.synchronize()
    want = reference(z, top, at, 1.0, weight=weight)
    if dtype != "fp16":
        # one fp32 rounding of a value of 1e38 and the sum beside it
        want[4][3] = want[1][3].abs() * 2.0 ** -22
    close(loss, want[0], want[3])
    close(lse, want[1], want[4])
    close(grad, want[2], want[5], dt)
    assert float(loss[6]) == 0.0 and bool((grad[6] == 0).all())


def test_distill_nan_and_infinity_stay_in_their_token(hqq):
    z, top, at, _ = inputs(6, 3001, 8, torch.float32, torch.int32, 1.0, False, 9)
    clean = hqq.hqq_distill(z, top, at, 1.0, grad=True)
    bad = z.clone()
    bad[1, 2000] = math.nan
    bad[3, 5] = math.inf
    bad[4, :] = -math.inf
    loss, lse, grad = hqq.hqq_distill(bad, top, at, 1.0, grad=True)
    for i in (0, 2, 5):
        assert torch.equal(loss[i], clean[0][i]) and torch.equal(grad[i], clean[2][i])
    for i in (1, 3, 4):
        assert math.isnan(float(loss[i])) and bool(torch.isnan(grad[i]).all())
    # the student gives no probability to an entry that the teacher does
    bad = z.clone()
    bad[2, at[2, 0].long()] = -math.inf
    loss, _, grad = hqq.hqq_distill(bad, top, at, 1.0, grad=True)
    assert float(loss[2]) == math.inf and bool(torch.isfinite(grad).all())


@pytest.mark.parametrize("V", [4096, 4097, 300000])
def test_distill_weight_zero_is_not_read(hqq, V):
    z, top, at, _ = inputs(5, V, 6, torch.bfloat16, torch.int64, 1.0, False, 11)
    weight = torch.tensor([1.0, 0.0, 3.0, 0.0, 1.0], device="cuda")
    z[1, :] = math.nan
    z[3, :] = -math.inf
    loss, lse, grad = hqq.hqq_distill(z, top, at, 1.0, weight=weight, grad=True)
    want = reference(z, top, at, 1.0, weight=weight)
    for i in (1, 3):
        assert float(loss[i]) == 0.0 and float(lse[i]) == 0.0 and bool((grad[i] == 0).all())
    for i in (0, 2, 4):
        close(loss[i:i + 1], want[0][i:i + 1], want[3][i:i + 1])
        close(grad[i], want[2][i], want[5][i], torch.bfloat16)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("V", [2000, 2001, 40000, 300000])
def test_distill_strided_rows_and_in_place(hqq, dtype, V):
    dt = DTYPES[dtype]
    z, top, at, _ = inputs(4, V, 10, dt, torch.int32, 1.0, False, 13)
    ref = hqq.hqq_distill(z, top, at, 1.0, grad=True)
    wide = torch.full((4, V + 24), 7.0, dtype=dt, device="cuda")
    gwide = torch.full((4, V + 40), 9.0, dtype=dt, device="cuda")
    wide[:, :V] = z
    out = hqq.hqq_distill(wide[:, :V], top, at, 1.0, grad=gwide[:, 3:V + 3])
    want = reference(z, top, at, 1.0)
    close(out[0], want[0], want[3])
    close(out[2], want[2], want[5], dt)
    assert bool((gwide[:, :3] == 9).all()) and bool((gwide[:, V + 3:] == 9).all())
    out = hqq.hqq_distill(wide[:, :V], top, at, 1.0, grad=wide[:, :V])      # in place
    assert bool((wide[:, V:] == 7).all())
    close(out[2], want[2], want[5], dt)
    out = hqq.hqq_distill(z, top, at, 1.0, grad=z)
    assert torch.equal(out[2], ref[2]) and torch.equal(out[0], ref[0])


def test_distill_gradient_against_differences(hqq):
    """(L(z + h d) - L(z - h d)) / 2h along random directions d of unit entries;
    the loss is smooth with third derivatives of at most about 1 per unit
    direction entry, so the difference is within h^2 + (loss tolerance) / h."""
    T, V, K = 4, 600, 20
    z, top, at, _ = inputs(T, V, K, torch.float32, torch.int64, 1.0, False, 17)
    weight = torch.tensor([1.0, 2.0, 0.5, 0.0], device="cuda")
    grad = hqq.hqq_distill(z, top, at, 1.0, weight=weight, grad=True)[2].double()
    tol = reference(z, top, at, 1.0, weight=weight)[3].cuda()
    h = 2.0 ** -6
    for seed in range(4):
        g = torch.Generator().manual_seed(seed)
        d = (torch.randint(0, 2, (T, V), generator=g) * 2 - 1).float().cuda()
        up = hqq.hqq_distill(z + h * d, top, at, 1.0, weight=weight)[0].double()
        dn = hqq.hqq_distill(z - h * d, top, at, 1.0, weight=weight)[0].double()
        # z + h d is rounded: 2^-24 of values below 32, through a gradient of 1-norm <= 2 w
        slack = 2 * weight.double() * 32 * U / h
        diff = (up - dn) / (2 * h)
        assert bool(((diff - (grad * d.double()).sum(1)).abs() <=
                     weight.double() * h * h + tol / h + slack + 1e-6).all())


def test_distill_streams_and_graphs(hqq):
    z, top, at, lse_t = inputs(64, 8000, 33, torch.bfloat16, torch.int64, 1.0, True, 19)
    ref = hqq.hqq_distill(z, top, at, 1.0, teacher_lse=lse_t, grad=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = hqq.hqq_distill(z, top, at, 1.0, teacher_lse=lse_t, grad=True, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, out))
    graph = torch.cuda.CUDAGraph()
    zin = torch.zeros_like(z)
    with torch.cuda.graph(graph):
        cap = hqq.hqq_distill(zin, top, at, 1.0, teacher_lse=lse_t, grad=True)
    for _ in range(2):
        zin.copy_(z)
        for c in cap:
            c.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, cap))
    E = hqq.hqq_distill(z[:0], top[:0], at[:0], 1.0, grad=True)
    assert E[0].shape == (0,) and E[2].shape == (0, 8000)
