"""Cases of the operators that fine-tune and serve adapters on a quantized
matrix: the linear layer with the low-rank adapters of many requests, its
gradients, and the distillation loss on a teacher's top logits.

``run`` computes each operator in plain torch operations (32 bits, rounded once
at the end) or, with ``own`` set, through weight_only_quantization_b200.

Operators
  adapters  Y[m] = W_hat X[m] + s_a B_a (A_a X[m]) with a = index[m] (no second
            term where index[m] is negative), W_hat = fp16((code - zero) scale).
  backward  dX, dA and dB of that product for a given dY.
  distill   per token w KL(p || softmax(z / T)) against the teacher's top_k
            entries, and its gradient with respect to the logits z.
"""
import math

import torch

own = False

FLOAT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one request generating: one token through an attention projection of the 70B set
        dict(name="adapters_1_token", op="adapters", rows=8192, cols=8192, nbits=3, group=64,
             tokens=1, count=8, rank=16, factors="fp16", pattern="each"),
        # sixteen requests generating, an adapter each, through the gate projection
        dict(name="adapters_16_requests", op="adapters", rows=28672, cols=8192, nbits=3, group=64,
             tokens=16, count=16, rank=16, factors="fp16", pattern="each"),
        # a serving batch of mixed requests, high rank, some without an adapter
        dict(name="adapters_64_mixed", op="adapters", rows=4096, cols=4096, nbits=4, group=64,
             tokens=64, count=32, rank=64, factors="fp16", pattern="mixed"),
        # prompts of a few requests, one after another (ragged; bf16 adapters)
        dict(name="adapters_777_prompts", op="adapters", rows=11008, cols=4096, nbits=2, group=32,
             tokens=777, count=5, rank=24, factors="bf16", pattern="segments"),
        # the low-rank residual of the quantization error on a long prompt: one
        # fp32 pair of factors for every token of the gate projection
        dict(name="adapters_2048_residual", op="adapters", rows=28672, cols=8192, nbits=3,
             group=64, tokens=2048, count=1, rank=16, factors="fp32", pattern="one"),
        # a short sequence through one 7B projection
        dict(name="backward_100_tokens", op="backward", rows=4096, cols=4096, nbits=4, group=64,
             tokens=100, count=1, rank=16, factors="fp16", pattern="one"),
        # sequences of several adapters trained side by side (ragged)
        dict(name="backward_1111_three", op="backward", rows=11008, cols=4096, nbits=4, group=128,
             tokens=1111, count=3, rank=8, factors="fp32", pattern="segments"),
        # one training step's tokens through a 70B projection
        dict(name="backward_2048_tokens", op="backward", rows=8192, cols=8192, nbits=3, group=64,
             tokens=2048, count=1, rank=32, factors="fp32", pattern="one"),
        # a few answer tokens
        dict(name="distill_8_tokens", op="distill", tokens=8, vocab=32000, top_k=32,
             logits="bf16", temperature=1.0, tail=False, keep=1.0),
        # a training step's tokens, a quarter of them prompt (weight 0)
        dict(name="distill_4096_tokens", op="distill", tokens=4096, vocab=32000, top_k=64,
             logits="fp16", temperature=2.0, tail=False, keep=0.75),
        # one added token makes the vocabulary odd; the teacher's normaliser is known
        dict(name="distill_odd_vocabulary", op="distill", tokens=1023, vocab=32001, top_k=20,
             logits="fp32", temperature=1.0, tail=True, keep=0.9),
        # a large vocabulary with many stored entries
        dict(name="distill_large_vocabulary", op="distill", tokens=2048, vocab=131072, top_k=256,
             logits="bf16", temperature=1.5, tail=True, keep=1.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adapters", "backward", "distill"])
    if op == "distill":
        vocab = _log_int(rng, 1000, 131072)
        tokens = _log_int(rng, 1, max(1, min(4096, (2048 * 131072) // vocab)))
        return dict(op=op, tokens=tokens, vocab=vocab, top_k=_log_int(rng, 1, 256),
                    logits=rng.choice(["fp16", "bf16", "fp32"]),
                    temperature=rng.choice([0.5, 1.0, 1.5, 2.0]), tail=rng.random() < 0.5,
                    keep=rng.choice([1.0, 0.75, 0.5]))
    group = rng.choice([16, 32, 64, 128])
    rows = _log_int(rng, 256, 16384)
    if op == "backward" and rng.random() < 0.75:
        rows = -(-rows // 8) * 8
    cols = -(-_log_int(rng, 512, 8192) // group) * group
    tokens = _log_int(rng, 1, 2048) if op == "adapters" else _log_int(rng, 16, 2048)
    pattern = rng.choice(["one", "each", "mixed", "segments"])
    count = 1 if pattern == "one" else _log_int(rng, 2, 32)
    rank = rng.choice([4, 8, 13, 16, 24, 32, 64])
    return dict(op=op, rows=rows, cols=cols, nbits=rng.choice([1, 2, 3, 4, 8]), group=group,
                tokens=tokens, count=count, rank=rank,
                factors=rng.choice(["fp16", "bf16", "fp32"]), pattern=pattern)


def work(case):
    """Bytes and operations of one pass: every input read once, every output
    written once; adapters that some token can have are read."""
    c = case
    if c["op"] == "distill":
        z = FLOAT[c["logits"]].itemsize
        T, V, K = c["tokens"], c["vocab"], c["top_k"]
        kept = T * c["keep"]
        return {"bytes": kept * V * z + T * V * z + kept * K * 12 + T * 12,
                "flops": kept * V * 8}
    M, N, K, r = c["tokens"], c["rows"], c["cols"], c["rank"]
    bits = {1: 1, 2: 2, 3: 3.2, 4: 4, 8: 8}[c["nbits"]]
    used = min(c["count"], M)
    weights = N * K * (bits / 8 + 4 / c["group"])
    factors = used * r * (N + K) * FLOAT[c["factors"]].itemsize
    delta = 2 * M * r * (N + K)
    if c["op"] == "adapters":
        return {"bytes": weights + factors + 2 * M * (N + K) + 4 * M,
                "flops": 2 * M * N * K + delta}
    grads = 4 * c["count"] * r * (N + K)
    return {"bytes": weights + factors + 2 * M * (N + 2 * K) + 4 * M + grads,
            "flops": 2 * M * N * K + 3 * delta}


# ---------------------------------------------------------------- the inputs

def _pack(codes, nbits):
    """Codes (flat, int32) in the library's layout, as bytes."""
    per, step = {1: (8, 1), 2: (4, 2), 3: (10, 3), 4: (2, 4), 8: (1, 8)}[nbits]
    pad = -codes.numel() % per
    c = torch.nn.functional.pad(codes, (0, pad)).view(-1, per)
    shift = torch.arange(per, device=c.device, dtype=torch.int32) * step
    words = (c << shift).sum(1, dtype=torch.int32)
    return words.view(torch.uint8) if nbits == 3 else words.to(torch.uint8)


def _matrix(c, gen, dev):
    """A weight matrix rounded to the nearest of 2^nbits levels per group, as
    packed codes, fp16 scale and zero."""
    N, K, G, L = c["rows"], c["cols"], c["group"], 2 ** c["nbits"] - 1
    packed, scale, zero = [], [], []
    step = max(1, (1 << 26) // K // 10 * 10)      # whole packed words a block: 10 rows fill them
    for n in range(0, N, step):
        w = torch.randn(min(step, N - n), K // G, G, generator=gen, device=dev) * 0.02
        lo, hi = w.amin(2, keepdim=True), w.amax(2, keepdim=True)
        s = ((hi - lo) / L).clamp_min(1e-6)
        z = -lo / s
        codes = torch.round(w / s + z).clamp_(0, L).to(torch.int32)
        packed.append(_pack(codes.view(-1), c["nbits"]))
        scale.append(s.half().view(-1, K // G))
        zero.append(z.half().view(-1, K // G))
    return torch.cat(packed), torch.cat(scale), torch.cat(zero)


def _index(c, gen, dev):
    """The adapter of every token: one for all (None), any for each token, a
    quarter of the tokens without one, or runs of tokens."""
    M, n = c["tokens"], c["count"]
    if c["pattern"] == "one":
        return None
    if c["pattern"] == "segments":
        cuts = torch.sort(torch.randint(0, M + 1, (n - 1,), generator=gen, device=dev)).values
        order = torch.randperm(n, generator=gen, device=dev)
        at = torch.bucketize(torch.arange(M, device=dev), cuts, right=True)
        return order[at].to(torch.int32)
    i = torch.randint(0, n, (M,), generator=gen, device=dev, dtype=torch.int32)
    if c["pattern"] == "mixed":
        i[torch.rand(M, generator=gen, device=dev) < 0.25] = -1
    return i


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    if c["op"] == "distill":
        T, V, K, temp = c["tokens"], c["vocab"], c["top_k"], c["temperature"]
        z = torch.randn(T, V, generator=gen, device=dev) * 2
        z += 6 * (torch.rand(T, V, generator=gen, device=dev) < 2e-3)
        z = z.to(FLOAT[c["logits"]])
        teacher = z.float() + 0.7 * torch.randn(T, V, generator=gen, device=dev)
        top, at = torch.topk(teacher, K, dim=1)
        at[torch.rand(T, K, generator=gen, device=dev) < 0.02] = -1     # unused entries
        lse = torch.logsumexp(teacher / temp, 1) if c["tail"] else None
        weight = (torch.rand(T, generator=gen, device=dev) < c["keep"]).float()
        return dict(c=c, logits=z, top=top.contiguous(), at=at.contiguous(), teacher_lse=lse,
                    weight=weight)
    M, N, K, r, n = c["tokens"], c["rows"], c["cols"], c["rank"], c["count"]
    packed, scale, zero = _matrix(c, gen, dev)
    f = FLOAT[c["factors"]]
    s = dict(c=c, packed=packed, scale=scale, zero=zero,
             X=torch.randn(M, K, generator=gen, device=dev).half(),
             A=(torch.randn(n, r, K, generator=gen, device=dev) / math.sqrt(K)).to(f),
             B=(torch.randn(n, N, r, generator=gen, device=dev) * 0.05).to(f),
             scaling=0.5 + torch.rand(n, generator=gen, device=dev),
             index=_index(c, gen, dev))
    if c["op"] == "backward":
        s["dY"] = (torch.randn(M, N, generator=gen, device=dev) * 0.1).half()
    return s


# ---------------------------------------------------------------- one pass

def _weights(s):
    """W_hat = fp16((code - zero) scale) as fp32, from the packed codes."""
    c = s["c"]
    N, K, b = c["rows"], c["cols"], c["nbits"]
    per, step = {1: (8, 1), 2: (4, 2), 3: (10, 3), 4: (2, 4), 8: (1, 8)}[b]
    words = s["packed"].view(torch.int32) if b == 3 else s["packed"]
    shift = torch.arange(per, device=words.device, dtype=words.dtype) * step
    codes = ((words[:, None] >> shift) & (2 ** b - 1)).view(-1)[:N * K].view(N, -1, c["group"])
    w = (codes.float() - s["zero"].float()[:, :, None]) * s["scale"].float()[:, :, None]
    return w.half().float().view(N, K)


def _share(s):
    """[tokens, count]: the scaling of the token's adapter in its column, else 0."""
    n, M = s["c"]["count"], s["c"]["tokens"]
    if s["index"] is None:
        return s["scaling"].expand(M, 1)
    own_column = s["index"][:, None] == torch.arange(n, device=s["index"].device)
    return own_column.float() * s["scaling"]


def _adapters(s):
    c = s["c"]
    r, n = c["rank"], c["count"]
    X = s["X"].float()
    T = (X @ s["A"].float().view(n * r, -1).T).view(-1, n, r) * _share(s)[:, :, None]
    Y = X @ _weights(s).T + T.view(-1, n * r) @ s["B"].float().transpose(1, 2).reshape(n * r, -1)
    return Y.half()


def _backward(s):
    c = s["c"]
    r, n, K, N = c["rank"], c["count"], c["cols"], c["rows"]
    X, dY, share = s["X"].float(), s["dY"].float(), _share(s)[:, :, None]
    A = s["A"].float().view(n * r, K)
    B = s["B"].float().transpose(1, 2).reshape(n * r, N)
    T = ((X @ A.T).view(-1, n, r) * share).view(-1, n * r)
    P = ((dY @ B.T).view(-1, n, r) * share).view(-1, n * r)
    dX = dY @ _weights(s) + P @ A
    dA = (P.T @ X).view(n, r, K)
    dB = (dY.T @ T).view(N, n, r).transpose(0, 1).contiguous()
    return {"dX": dX.half(), "dA": dA, "dB": dB}


def _distill(s):
    temp = s["c"]["temperature"]
    z = s["logits"].float() / temp
    V = z.shape[1]
    weight = s["weight"]
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    lse = top + torch.log(total)
    valid = (s["at"] >= 0) & (s["at"] < V)
    at = torch.where(valid, s["at"], 0)
    t = torch.where(valid, s["top"].float() / temp, -math.inf)
    if s["teacher_lse"] is None:
        peak = t.amax(1, keepdim=True)
        norm = peak + torch.log(torch.exp(t - peak).sum(1, keepdim=True))
    else:
        norm = s["teacher_lse"][:, None]
    logp = torch.where(valid, t - norm, 0.0)
    p = torch.where(valid, torch.exp(logp), 0.0)
    kept = weight != 0
    terms = torch.where(valid, p * (logp - (z.gather(1, at) - lse)), 0.0)
    loss = torch.where(kept, weight * terms.sum(1), 0.0)
    g = (e / total * p.sum(1, keepdim=True)).scatter_add_(1, at, -p)
    g = torch.where(kept[:, None], g * (weight[:, None] / temp), 0.0)
    return {"loss": loss, "grad": g.to(s["logits"].dtype)}


def run(state):
    s, c = state, state["c"]
    if own:
        import weight_only_quantization_b200 as hqq
        if c["op"] == "distill":
            loss, _, grad = hqq.hqq_distill(s["logits"], s["top"], s["at"], c["temperature"],
                                            teacher_lse=s["teacher_lse"], weight=s["weight"],
                                            grad=True)
            return {"loss": loss, "grad": grad}
        q = hqq.QuantizedMatrix(s["packed"], s["scale"], s["zero"], c["rows"], c["cols"],
                                c["nbits"], c["group"])
        a = hqq.Adapters(s["A"], s["B"], s["scaling"])
        if c["op"] == "adapters":
            return hqq.hqq_linear_adapters(s["X"], q, a, s["index"])
        dX, dA, dB = hqq.hqq_linear_adapters_backward(s["dY"], s["X"], q, a, s["index"])
        return {"dX": dX, "dA": dA, "dB": dB}
    return {"adapters": _adapters, "backward": _backward, "distill": _distill}[c["op"]](s)


# ---------------------------------------------------------------- in 64 bits

def _weights_64(s):
    """The stored matrix from its definition: code i of the flat order, its
    group's zero and scale, one rounding to 32 bits and one to fp16."""
    c = s["c"]
    b, K = c["nbits"], c["cols"]
    out = torch.empty(c["rows"], K, dtype=torch.float64, device=s["packed"].device)
    raw = s["packed"].view(torch.int32) if b == 3 else s["packed"]
    per_word = 10 if b == 3 else 8 // b
    step = max(1, (1 << 25) // K)
    for n in range(0, c["rows"], step):
        m = min(step, c["rows"] - n)
        i = torch.arange(n * K, (n + m) * K, device=out.device)
        word = raw[i // per_word].long()
        code = torch.bitwise_and(word >> (b * (i % per_word)), (1 << b) - 1).double().view(m, K)
        zero = s["zero"][n:n + m].double().repeat_interleave(c["group"], 1)
        scale = s["scale"][n:n + m].double().repeat_interleave(c["group"], 1)
        out[n:n + m] = ((code - zero) * scale).float().half().double()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    if c["op"] == "distill":
        z = s["logits"].double() / c["temperature"]
        valid = (s["at"] >= 0) & (s["at"] < c["vocab"])
        t = (s["top"].double() / c["temperature"]).masked_fill(~valid, -math.inf)
        if s["teacher_lse"] is None:
            logp = torch.log_softmax(t, 1)
        else:
            logp = t - s["teacher_lse"].double()[:, None]
        p = torch.exp(logp)
        logq = torch.log_softmax(z, 1)
        w = s["weight"].double()
        place = s["at"].clamp(0, c["vocab"] - 1)
        kl = torch.where(p > 0, p * (logp - logq.gather(1, place)), 0.0).nan_to_num(0.0).sum(1)
        target = torch.zeros_like(z).scatter_add_(1, place, p.nan_to_num(0.0))
        mass = target.sum(1, keepdim=True)
        grad = (mass * torch.exp(logq) - target) * (w / c["temperature"])[:, None]
        return {"loss": w * kl, "grad": grad}
    W = _weights_64(s)
    X, A, B = s["X"].double(), s["A"].double(), s["B"].double()
    M, n = c["tokens"], c["count"]
    index = s["index"].long() if s["index"] is not None else torch.zeros(M, dtype=torch.long,
                                                                       device=X.device)
    if c["op"] == "adapters":
        Y = X @ W.T
        for a in range(n):
            at = (index == a).nonzero().view(-1)
            Y[at] += s["scaling"][a].double() * ((X[at] @ A[a].T) @ B[a].T)
        return Y
    dY = s["dY"].double()
    dX = dY @ W
    dA, dB = torch.zeros_like(A), torch.zeros_like(B)
    for a in range(n):
        at = (index == a).nonzero().view(-1)
        g = s["scaling"][a].double() * dY[at]
        dX[at] += (g @ B[a]) @ A[a]
        dA[a] = (g @ B[a]).T @ X[at]
        dB[a] = g.T @ (X[at] @ A[a].T)
    return {"dX": dX, "dA": dA, "dB": dB}
