"""The gated delta rule with one decay per head, and the matrix product with an epilogue: what is measured, in
plain torch and through the library.

A layer of the gated delta rule is KDA's with a scalar gate: H_v value heads over H_k key heads (value head h
reads key head h / (H_v / H_k)), a decay alpha per token and value head instead of one per channel, and
projections that carry a bias, an activation or the residual. `run` computes one of the operators, in its plain
form or, with `own`, by the library's calls:

  decode   g = -exp(A_log[h]) softplus(raw_g + dt_bias[h]), alpha = exp(g), beta = sigmoid(raw_beta);
           q^ = scale q / sqrt(|q|^2 + eps), k^ = k / sqrt(|k|^2 + eps);
           S <- alpha S; u = beta (v - S^T k^); S <- S + k^ u^T; o = S^T q^, one token per sequence, the states
           fp32 [K, V] per head in slots of a pool, updated in place.
  spec     the same over requests of T rows each.
  prefill  the same over packed sequences of different lengths, in chunks (cu_seqlens on the GPU).
  matmul   out = act(a w^T + bias) + residual.

Chunks of C rows: with b the running sum of g inside the chunk, D[r, i] = e^(b_r - b_i) and T = (I + A)^-1 for
A[r, i] = beta_r (k^_r . k^_i) D[r, i], i < r:
  U = T diag(beta) (v - e^b (k^ S)),  o = e^b (q^ S) + ((q^ k^^T) * D, i <= r) U,  S <- e^b_C S + (k^ e^(b_C - b))^T U
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HIDDEN = 4096
L2_EPS = 1e-6
CHUNK = 64
MOST_STATES, MOST_ROWS, MOST_TOKENS, MOST_PRODUCTS = 128 * 32, 33494 * 32, 33494, 33494 * HIDDEN * HIDDEN


def listed():
    return [
        # one sequence decoding: the latency of a step
        {"name": "gdn decode one", "op": "decode", "reqs": 1, "tokens": 1, "hk": 16, "hv": 32, "k": 128, "v": 128},
        # the serving decode's 128 sequences: the states' bytes
        {"name": "gdn decode", "op": "decode", "reqs": 128, "tokens": 1, "hk": 16, "hv": 32, "k": 128, "v": 128},
        # a tensor-parallel rank's few heads, many sequences, narrow keys
        {"name": "gdn decode many", "op": "decode", "reqs": 777, "tokens": 1, "hk": 3, "hv": 6, "k": 64, "v": 128},
        # the spec-verify step of 16 requests with 8 rows
        {"name": "gdn spec", "op": "spec", "reqs": 16, "tokens": 8, "hk": 32, "hv": 32, "k": 128, "v": 128},
        # many requests of an odd number of rows, three value heads to a key head
        {"name": "gdn spec odd", "op": "spec", "reqs": 61, "tokens": 5, "hk": 4, "hv": 12, "k": 128, "v": 64},
        # the chunked prefill's eight sequences, about 33,000 tokens
        {"name": "gdn prefill", "op": "prefill", "reqs": 8, "tokens": 5821, "hk": 16, "hv": 32, "k": 128, "v": 128},
        # one long prompt: 32 states, each advanced from end to end
        {"name": "gdn prefill one", "op": "prefill", "reqs": 1, "tokens": 16384, "hk": 32, "hv": 32, "k": 128, "v": 128},
        # many short and odd prompts on a few heads
        {"name": "gdn prefill short", "op": "prefill", "reqs": 257, "tokens": 171, "hk": 4, "hv": 8, "k": 64, "v": 64},
        # the output gate's projection of one decoding sequence: the weights' bytes
        {"name": "matmul one row", "op": "matmul", "m": 1, "n": HIDDEN, "k": HIDDEN, "dtype": "bf16", "out": "bf16", "bias": True, "act": "sigmoid", "residual": False},
        # the gates' and value projections of the serving decode
        {"name": "matmul decode", "op": "matmul", "m": 128, "n": 3 * HIDDEN, "k": HIDDEN, "dtype": "bf16", "out": "bf16", "bias": False, "act": "silu", "residual": False},
        # the output projection of a prefill, added to the residual: the tensor cores' rate
        {"name": "matmul prefill", "op": "matmul", "m": 33494, "n": HIDDEN, "k": HIDDEN, "dtype": "bf16", "out": "bf16", "bias": False, "act": "none", "residual": True},
        # sides that no tile divides, an fp32 residual stream
        {"name": "matmul odd", "op": "matmul", "m": 1000, "n": 1111, "k": 1301, "dtype": "fp16", "out": "fp32", "bias": True, "act": "gelu", "residual": True},
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    op = rng.choice(["decode", "spec", "prefill", "prefill", "matmul", "matmul"])
    if op == "matmul":
        n, k = _log(rng, 32, 4 * HIDDEN), _log(rng, 64, 2 * HIDDEN)
        m = min(_log(rng, 1, 32768), MOST_PRODUCTS // (n * k))
        return {"op": op, "m": m, "n": n, "k": k, "dtype": rng.choice(["bf16", "bf16", "fp16"]), "out": rng.choice(["bf16", "fp16", "fp32"]),
                "bias": rng.random() < 0.5, "act": rng.choice(["none", "none", "relu", "silu", "sigmoid", "gelu", "gelu_tanh"]),
                "residual": rng.random() < 0.5}
    groups = rng.choice([1, 1, 2, 2, 3, 4])
    hk = _log(rng, 1, 32 // groups)
    heads = {"hk": hk, "hv": hk * groups, "k": rng.choice([64, 128, 128]), "v": rng.choice([64, 128, 128])}
    if op == "prefill":
        tokens = _log(rng, 1, 16384)
        reqs = min(_log(rng, 1, 256), max(1, MOST_TOKENS // tokens))
    else:
        tokens = 1 if op == "decode" else rng.randint(2, 16)
        reqs = min(_log(rng, 1, 1024), MOST_STATES // heads["hv"])
        if rng.random() < 0.2:
            heads["k"] = 32
    return {"op": op, "reqs": reqs, "tokens": tokens, **heads}


def _lengths(case):
    """The sequences' lengths: of one sequence the given number, of many between a seventh of and all of it and a
    half more."""
    n, top = case["reqs"], case["tokens"]
    if n == 1 or case["op"] != "prefill":
        return [top] * n
    r = random.Random(1009 * n + top)
    return [r.randint(max(1, top // 7), top + top // 2) for _ in range(n)]


def _rows16(rows, cols, dtype):
    """An [rows, cols] tensor whose rows start on 16-byte boundaries."""
    per = 16 // torch.empty(0, dtype=dtype).element_size()
    return torch.empty(rows, -(-cols // per) * per, dtype=dtype, device="cuda")[:, :cols]


def prepare(case, seed):
    d = "cuda"
    gen = torch.Generator(device=d)
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, device=d, generator=gen)

    s = {"case": case}
    if case["op"] == "matmul":
        m, n, k, dt, out = case["m"], case["n"], case["k"], DTYPES[case["dtype"]], DTYPES[case["out"]]
        s["a"], s["w"], s["out"] = _rows16(m, k, dt), _rows16(n, k, dt), _rows16(m, n, out)
        s["a"].copy_(randn(m, k) * torch.exp(0.3 * randn(m, 1)))   # rows of different size, as after a norm's weight
        s["w"].copy_(randn(n, k) / math.sqrt(k))
        s["bias"] = randn(n).to(dt) if case["bias"] else None
        s["residual"] = None
        if case["residual"]:
            s["residual"] = _rows16(m, n, out)
            s["residual"].copy_(randn(m, n))
        return s
    hk, hv, k, v, reqs = case["hk"], case["hv"], case["k"], case["v"], case["reqs"]
    lens = _lengths(case)
    rows, slots = sum(lens), reqs + reqs // 8 + 1
    s["mixed_qkv"] = randn(rows, 2 * hk * k + hv * v).to(torch.bfloat16)   # after the short convolution
    s["raw_g"], s["raw_beta"] = randn(rows, hv).to(torch.bfloat16), randn(rows, hv).to(torch.bfloat16)
    s["A_log"] = torch.log(1 + 15 * torch.rand(hv, device=d, generator=gen))
    dt = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(hv, device=d, generator=gen))
    s["dt_bias"] = dt + torch.log(-torch.expm1(-dt))   # softplus(dt_bias) from 0.001 to 0.1
    s["pool"] = 0.05 * randn(slots, hv, k, v)
    s["slots"] = torch.randperm(slots, device=d, generator=gen)[:reqs].to(torch.int32)
    cu = torch.zeros(reqs + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(lens), 0)
    s["cu"] = cu.to(d)
    s["out"] = torch.empty(rows, hv * v, dtype=torch.bfloat16, device=d)
    return s


def _doubled(blocks, a, n):
    """The inverses of the unit lower triangular blocks of 2n rows, from those of n rows: [[X, 0], [-Y A X, Y]]."""
    x, y = blocks[:, 0::2], blocks[:, 1::2]
    low = a.view(-1, a.shape[1] // (2 * n), 2 * n, a.shape[2] // (2 * n), 2 * n).diagonal(dim1=1, dim2=3).permute(0, 3, 1, 2)[:, :, n:, :n]
    return torch.cat([torch.cat([x, torch.zeros_like(x)], 3), torch.cat([-(y @ (low @ x)), y], 3)], 2)


def _inverse(a):
    """(I + a)^-1 of strictly lower triangular a [B, C, C], C a power of two."""
    blocks = torch.ones(a.shape[0], a.shape[1], 1, 1, device=a.device, dtype=a.dtype)
    n = 1
    while n < a.shape[1]:
        blocks = _doubled(blocks, a, n)
        n *= 2
    return blocks[:, 0]


def _rule(q, k, v, g, beta, S):
    """The chunked rule over [B, T, .] rows in fp32; returns o [B, T, V] and the state [B, K, V] after the last row."""
    B, T, V = v.shape
    C = 1
    while C < min(T, CHUNK):
        C *= 2
    n = -(-T // C)

    def cut(x):
        return torch.nn.functional.pad(x, (0, 0, 0, n * C - T)).view(B, n, C, -1)

    q, k, v, beta = cut(q), cut(k), cut(v), cut(beta[..., None])
    b = torch.cumsum(cut(g[..., None]), 2)
    far = torch.full((C, C), -torch.inf, device=q.device).triu(1)
    D = torch.exp(b - b.transpose(2, 3) + far)
    A = torch.tril(beta * (k @ k.transpose(2, 3)) * D, -1)
    W = _inverse(A.view(B * n, C, C)).view(B, n, C, C) * beta.transpose(2, 3)
    P = (q @ k.transpose(2, 3)) * D
    e, tail = torch.exp(b), torch.exp(b[:, :, -1:] - b) * k
    outs = []
    for i in range(n):
        u = W[:, i] @ (v[:, i] - e[:, i] * (k[:, i] @ S))
        outs.append(e[:, i] * (q[:, i] @ S) + P[:, i] @ u)
        S = e[:, i, -1:] * S + tail[:, i].transpose(1, 2) @ u
    return torch.cat(outs, 1)[:, :T], S


def _inputs(s, dtype):
    """q^, k^, v [R, T, H_v, .], log-decay and beta [R, T, H_v] in `dtype`, rows past a sequence's end empty, and
    where each of them is in the packed rows."""
    c = s["case"]
    hk, hv, k, v = c["hk"], c["hv"], c["k"], c["v"]
    lens = (s["cu"][1:] - s["cu"][:-1]).long()
    T = max(_lengths(c))
    at = torch.arange(T, device="cuda")
    live = at < lens[:, None]
    row = torch.where(live, s["cu"][:-1, None].long() + at, 0)
    x = s["mixed_qkv"][row].to(dtype)
    R = x.shape[0]
    q = x[..., :hk * k].reshape(R, T, hk, k)
    key = x[..., hk * k:2 * hk * k].reshape(R, T, hk, k)
    q = q * (k ** -0.5 / torch.sqrt(q.square().sum(-1, keepdim=True) + L2_EPS))
    key = key / torch.sqrt(key.square().sum(-1, keepdim=True) + L2_EPS)
    head = torch.arange(hv, device="cuda") // (hv // hk)
    z = s["raw_g"][row].to(dtype) + s["dt_bias"].to(dtype)
    g = -torch.exp(s["A_log"].to(dtype)) * (z.clamp_min(0) + torch.log1p(torch.exp(-z.abs())))
    beta = torch.sigmoid(s["raw_beta"][row].to(dtype))
    mask = live[..., None]
    return (q[:, :, head], key[:, :, head], x[..., 2 * hk * k:].reshape(R, T, hv, v), torch.where(mask, g, 0),
            torch.where(mask, beta, 0)), live, row


def _gdn(s):
    (q, k, v, g, beta), live, row = _inputs(s, torch.float32)
    R, T, H, V = v.shape

    def flat(x):
        return x.transpose(1, 2).reshape(R * H, T, *x.shape[3:])

    slots = s["slots"].long()
    S = s["pool"][slots].view(R * H, -1, V)
    o, S = _rule(flat(q), flat(k), flat(v), flat(g), flat(beta), S)
    s["pool"][slots] = S.view(R, H, -1, V)
    s["out"][row[live]] = o.view(R, H, T, V).transpose(1, 2)[live].reshape(-1, H * V).to(torch.bfloat16)
    return {"out": s["out"], "pool": s["pool"]}


ACTS = {"none": lambda x: x,
        "relu": lambda x: x.clamp_min(0),
        "silu": lambda x: x / (1 + torch.exp(-x)),
        "sigmoid": lambda x: 1 / (1 + torch.exp(-x)),
        "gelu": lambda x: 0.5 * x * (1 + torch.erf(x * math.sqrt(0.5))),
        "gelu_tanh": lambda x: 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))}


def _matmul(s):
    x = s["a"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        x = x + s["bias"].float()
    x = ACTS[s["case"]["act"]](x)
    if s["residual"] is not None:
        x = x + s["residual"].float()
    return s["out"].copy_(x)


def run(state):
    s = state
    c = s["case"]
    if not own:
        return _matmul(s) if c["op"] == "matmul" else _gdn(s)
    from linear_attention_state_recurrent_gb300 import kda
    if c["op"] == "matmul":
        return kda.kda_matmul(s["a"], s["w"], bias=s["bias"], activation=None if c["act"] == "none" else c["act"],
                              residual=s["residual"], out=s["out"])
    args = (s["mixed_qkv"], s["raw_g"], s["raw_beta"], s["A_log"], s["dt_bias"], s["pool"], s["slots"])
    if c["op"] == "decode":
        kda.kda_gdn_decode(*args, num_k_heads=c["hk"], out=s["out"])
    elif c["op"] == "spec":
        kda.kda_gdn_spec_verify(*args, c["tokens"], num_k_heads=c["hk"], out=s["out"])
    else:
        kda.kda_gdn_chunk_prefill(*args, s["cu"], num_k_heads=c["hk"], out=s["out"])
    return {"out": s["out"], "pool": s["pool"]}


def work(case):
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        e = 4 if case["out"] == "fp32" else 2
        return {"bytes": 2 * (m * k + n * k) + m * n * e * (1 + case["residual"]) + 2 * n * case["bias"], "flops": 2 * m * n * k}
    lens, hk, hv, k, v = _lengths(case), case["hk"], case["hv"], case["k"], case["v"]
    rows = sum(lens)
    nbytes = 2 * rows * (2 * hk * k + 2 * hv * v + 2 * hv) + 8 * case["reqs"] * hv * k * v
    if case["op"] != "prefill":   # per token k^T S and q^T S, the decay and the update
        return {"bytes": nbytes, "flops": rows * hv * 7 * k * v}
    # per chunk of c rows: K S, Q S and the state's update, the products inside the chunk (triangles count half) and the inverse
    full, last = sum(n // CHUNK for n in lens), [n % CHUNK for n in lens]
    flops = sum(6 * c * k * v + c * c * (2 * k + 2 * v) + c ** 3 / 3 for c in [CHUNK] * full + last)
    return {"bytes": nbytes, "flops": hv * flops}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "matmul":
        x = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
        for at in range(0, x.shape[0], 4096):
            x[at:at + 4096] = s["a"][at:at + 4096].double() @ s["w"].double().t()
        if s["bias"] is not None:
            x += s["bias"].double()
        x = {"none": lambda t: t, "relu": torch.relu, "silu": lambda t: t * torch.sigmoid(t), "sigmoid": torch.sigmoid,
             "gelu": lambda t: t * torch.special.ndtr(t),
             "gelu_tanh": lambda t: t * torch.sigmoid(math.sqrt(8 / math.pi) * (t + 0.044715 * t ** 3))}[case["act"]](x)
        return x if s["residual"] is None else x + s["residual"].double()
    # token by token, every sequence and head at once; a sequence that has ended keeps its state
    hk, hv, k, v = case["hk"], case["hv"], case["k"], case["v"]
    lens = torch.tensor(_lengths(case), device="cuda")
    first = s["cu"][:-1].long()
    rep = hv // hk
    decay = -torch.exp(s["A_log"].double())
    pool, out = s["pool"].double(), torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    slots = s["slots"].long()
    S = pool[slots]
    for t in range(int(lens.max())):
        on = (lens > t).nonzero()[:, 0] if case["op"] == "prefill" and case["reqs"] > 1 else slice(None)
        row = first[on] + t
        x = s["mixed_qkv"][row].double()
        q, key = x[:, :2 * hk * k].view(-1, 2, hk, k).unbind(1)
        q, key = (y * (y.square().sum(-1, keepdim=True) + L2_EPS).rsqrt() for y in (q, key))
        q, key = (y.repeat_interleave(rep, 1)[:, :, None] for y in (q, key))
        val = x[:, 2 * hk * k:].view(-1, hv, 1, v)
        alpha = torch.exp(decay * torch.nn.functional.softplus(s["raw_g"][row].double() + s["dt_bias"].double(), threshold=50.0))
        beta = torch.special.expit(s["raw_beta"][row].double())
        St = S[on] * alpha[..., None, None]
        St = St + key.transpose(2, 3) @ (beta[..., None, None] * (val - key @ St))
        S[on] = St
        out[row] = (q @ St).view(-1, hv * v) * k ** -0.5
    pool[slots] = S
    return {"out": out, "pool": pool}
