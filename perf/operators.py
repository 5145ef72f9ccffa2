"""The operators around the KDA recurrence of one serving step: what is measured, in plain torch and
through the library.

A KDA layer's step is: the batch's maps (which rows, state slots and cache pages its tokens use), the
residual's addition and RMSNorm with an 8-bit output, the 8-bit projections, the recurrence, and the
8-bit output projection. `run` computes one of the operators, in its plain form or, with `own`, by the
library's calls:

  norm_quant  h = x + residual; y = h / sqrt(mean h^2 + eps) * weight (or y = h without a weight);
              per row and group of 128 columns s = max(max|y|, 448 * 2^-126) / 448 and
              q = e4m3(y / s), round to nearest even. Outputs q, s, h (with a residual), y (if asked).
  matmul      out[m, n] = sum_k a[m, k] sa[m, k / 128] w[n, k] sw[n / 128, k / 128] with e4m3 a and w.
  maps        requests with query lengths q and context lengths c, pages of P tokens: the requests in
              running order (query length 1 first, otherwise as given), cu_seqlens and state slots in
              that order, the pages ceil(c / P) .. ceil((c + q) / P) - 1 of each block-table row taken
              from the top of the free stack in request order, and for each token its position and its
              cache slot page * P + position % P (positions 0 and slots -1 past the last token).
"""
import math
import random

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
TINY = E4M3_MAX * 2.0 ** -126
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HIDDEN = 4096
IN_PROJ = 3 * 4096 + 2 * 4096 + 32   # q | k | v, raw_g, the output gate and raw_beta at H = 32, K = V = 128
MOST_NORM, MOST_MATMUL, MOST_TOKENS = 33494 * HIDDEN, 33494 * HIDDEN * IN_PROJ, 262144


def listed():
    return [
        # one sequence decoding: the latency of a single row
        {"name": "norm one row", "op": "norm_quant", "rows": 1, "cols": HIDDEN, "dtype": "bf16", "residual": True, "norm": True, "y": False},
        # the serving decode's 128 sequences
        {"name": "norm decode", "op": "norm_quant", "rows": 128, "cols": HIDDEN, "dtype": "bf16", "residual": True, "norm": True, "y": False},
        # the chunked prefill's 33,494 tokens
        {"name": "norm prefill", "op": "norm_quant", "rows": 33494, "cols": HIDDEN, "dtype": "bf16", "residual": True, "norm": True, "y": False},
        # the recurrence's outputs on their way to the output projection, no norm, the mixed batch's rows
        {"name": "quant mixed", "op": "norm_quant", "rows": 16480, "cols": HIDDEN, "dtype": "bf16", "residual": False, "norm": False, "y": False},
        # an odd width in fp32 with the unquantised output kept beside the 8-bit one
        {"name": "norm odd fp32", "op": "norm_quant", "rows": 2049, "cols": 5003, "dtype": "fp32", "residual": True, "norm": True, "y": True},
        # the input projection of one decoding sequence: the weights' bytes
        {"name": "matmul one row", "op": "matmul", "m": 1, "n": IN_PROJ, "k": HIDDEN, "out": "bf16"},
        # the input projection of the serving decode
        {"name": "matmul decode", "op": "matmul", "m": 128, "n": IN_PROJ, "k": HIDDEN, "out": "bf16"},
        # the input projection of the chunked prefill: the tensor cores' rate
        {"name": "matmul prefill", "op": "matmul", "m": 33494, "n": IN_PROJ, "k": HIDDEN, "out": "bf16"},
        # the output projection of a short prefill, added to an fp32 residual stream
        {"name": "matmul out fp32", "op": "matmul", "m": 1000, "n": HIDDEN, "k": HIDDEN, "out": "fp32"},
        # sides that no tile divides
        {"name": "matmul odd", "op": "matmul", "m": 77, "n": 1111, "k": 1301, "out": "bf16"},
        # the serving decode's step: every request one token
        {"name": "maps decode", "op": "maps", "reqs": 128, "prefills": 0, "query": 1, "context": 8192, "page": 64, "width": 136},
        # many requests, a quarter of them prefilling, up to 262,144 tokens in the step
        {"name": "maps large", "op": "maps", "reqs": 4096, "prefills": 1024, "query": 253, "context": 32768, "page": 16, "width": 2080},
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    op = rng.choice(["norm_quant", "norm_quant", "matmul", "matmul", "matmul", "maps"])
    if op == "norm_quant":
        cols = _log(rng, 64, 16384)
        rows = min(_log(rng, 1, 32768), MOST_NORM // cols)
        norm = rng.random() < 0.7
        return {"op": op, "rows": rows, "cols": cols, "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                "residual": norm and rng.random() < 0.7, "norm": norm, "y": norm and rng.random() < 0.3}
    if op == "matmul":
        n, k = _log(rng, 32, IN_PROJ), _log(rng, 64, 8192)
        m = min(_log(rng, 1, 32768), MOST_MATMUL // (n * k))
        return {"op": op, "m": m, "n": n, "k": k, "out": rng.choice(["bf16", "bf16", "fp16", "fp32"])}
    reqs = _log(rng, 1, 4096)
    prefills = rng.randint(0, reqs)
    query = _log(rng, 2, 8192)
    if prefills:
        query = max(2, min(query, (MOST_TOKENS - reqs) // prefills))
    context, page = _log(rng, 1, 32768), rng.choice([16, 32, 64, 128])
    return {"op": op, "reqs": reqs, "prefills": prefills, "query": query, "context": context, "page": page,
            "width": -(-(context + query) // page) + rng.randint(0, 8)}


def _tokens(case):
    """The rows that the step's buffers hold: every prefill at its longest."""
    return case["reqs"] - case["prefills"] + case["prefills"] * case["query"]


def _pad(t, cols):
    """The columns padded with zeros to a whole number of groups of 128."""
    return t if cols % 128 == 0 else torch.nn.functional.pad(t, (0, 128 - cols % 128))


def _quantise(y):
    """q [rows, cols] e4m3 and s [rows, groups] fp32 of y [rows, cols] fp32."""
    rows, cols = y.shape
    g = _pad(y, cols).view(rows, -1, 128)
    s = g.abs().amax(-1).clamp_min(TINY) / E4M3_MAX
    q = (g / s[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(rows, -1)[:, :cols], s


def _rows16(rows, cols, dtype, device):
    """An [rows, cols] tensor whose rows start on 16-byte boundaries."""
    per = 16 // torch.empty(0, dtype=dtype).element_size()
    return torch.empty(rows, -(-cols // per) * per, dtype=dtype, device=device)[:, :cols]


def prepare(case, seed):
    d = "cuda"
    gen = torch.Generator(device=d)
    gen.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "norm_quant":
        rows, cols, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]

        def activations():
            """A residual stream: rows of different size, a few columns far larger than the rest."""
            t = torch.randn(rows, cols, device=d, generator=gen)
            t *= torch.exp(0.5 * torch.randn(rows, 1, device=d, generator=gen))
            t[:, :: 509] *= 20.0
            return t.to(dt)

        s["x"] = activations()
        s["residual"] = activations() if case["residual"] else None
        s["weight"] = 1 + 0.2 * torch.randn(cols, device=d, generator=gen) if case["norm"] else None
        s["eps"] = 1e-5
        s["out"] = {"q": _rows16(rows, cols, torch.float8_e4m3fn, d),
                    "scales": torch.empty(-(-cols // 128), rows, device=d).t(),
                    "residual_out": torch.empty_like(s["x"]) if case["residual"] else None,
                    "y": torch.empty_like(s["x"]) if case["y"] else None}
    elif case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        groups, blocks = -(-k // 128), -(-n // 128)
        x = torch.randn(m, k, device=d, generator=gen)
        x *= torch.exp(0.5 * torch.randn(m, 1, device=d, generator=gen))
        x[:, :: 509] *= 20.0
        q, sa = _quantise(x)
        s["a"] = _rows16(m, k, torch.float8_e4m3fn, d)
        s["a"].copy_(q)
        s["a_scales"] = sa.t().contiguous().t()
        del x, q, sa
        w = torch.randn(n, k, device=d, generator=gen) / math.sqrt(k)
        top = _pad(w, k).abs().view(n, groups, 128).amax(-1)
        top = torch.nn.functional.pad(top, (0, 0, 0, blocks * 128 - n)).view(blocks, 128, groups).amax(1)
        sw = top.clamp_min(TINY) / E4M3_MAX
        w = w / sw.repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
        s["w"] = _rows16(n, k, torch.float8_e4m3fn, d)
        s["w"].copy_(w.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn))
        s["w_scales"] = sw
        s["out"] = _rows16(m, n, DTYPES[case["out"]], d)
    else:
        r = np.random.default_rng(seed)
        reqs, page, width, tokens = case["reqs"], case["page"], case["width"], _tokens(case)
        q = np.ones(reqs, np.int64)
        q[r.permutation(reqs)[:case["prefills"]]] = r.integers(max(2, case["query"] // 2), case["query"] + 1, case["prefills"])
        c = r.integers(1, case["context"] + 1, reqs)
        c[(q > 1) & (r.random(reqs) < 0.5)] = 0   # half of the prefills are fresh
        old, new = -(-c // page), np.minimum(-(-(c + q) // page), width)
        pages = r.permutation(int(new.sum()) + 64).astype(np.int32)
        table = np.full((reqs, width), -1, np.int32)
        held = np.arange(width)[None, :] < old[:, None]
        table[held] = pages[:int(held.sum())]
        free = pages[int(held.sum()):]

        def up(a, dt=np.int32):
            return torch.from_numpy(np.ascontiguousarray(a, dt)).to(d)

        s |= {"query_lens": up(q), "context_lens": up(c), "state_slots": up(r.permutation(reqs + 7)[:reqs]),
              "block_table": up(table), "free_pages": up(free), "free_count": up([len(free)]),
              "num_pages": len(pages)}
        s["out"] = {"order": torch.empty(reqs, dtype=torch.int32, device=d), "cu_seqlens": torch.empty(reqs + 1, dtype=torch.int32, device=d),
                    "state_indices": torch.empty(reqs, dtype=torch.int32, device=d), "num_decodes": torch.empty(1, dtype=torch.int32, device=d),
                    "positions": torch.empty(tokens, dtype=torch.int32, device=d), "slot_map": torch.empty(tokens, dtype=torch.int64, device=d),
                    "free_left": torch.empty(1, dtype=torch.int32, device=d)}
    return s


def _norm_quant(s):
    h = s["x"].float()
    out = {}
    if s["residual"] is not None:
        h = h + s["residual"].float()
        out["residual_out"] = h.to(s["x"].dtype)
    y = h
    if s["weight"] is not None:
        y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + s["eps"]) * s["weight"]
    if s["case"]["y"]:
        out["y"] = y.to(s["x"].dtype)
    out["q"], out["scales"] = _quantise(y)
    return out


def _matmul(s):
    (m, k), n = s["a"].shape, s["w"].shape[0]
    a = s["a"].float() * s["a_scales"].repeat_interleave(128, 1)[:, :k]
    w = s["w"].float() * s["w_scales"].repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    return (a @ w.t()).to(DTYPES[s["case"]["out"]])


def _maps(s):
    page, tokens = s["case"]["page"], _tokens(s["case"])
    q, c, table, free = s["query_lens"].long(), s["context_lens"].long(), s["block_table"], s["free_pages"]
    reqs, width = table.shape
    i32 = torch.int32
    order = torch.argsort((q != 1).int(), stable=True)
    cu = torch.nn.functional.pad(torch.cumsum(q[order], 0), (1, 0))
    old = torch.clamp((c + page - 1) // page, max=width)
    new = torch.clamp((c + q + page - 1) // page, max=width)
    end = torch.cumsum(new - old, 0)
    col = torch.arange(width, device=q.device)
    at = s["free_count"].long() - 1 - ((end - new)[:, None] + col)
    take = (col >= old[:, None]) & (col < new[:, None])
    table = torch.where(take, free[at.clamp(0, free.numel() - 1)], table)
    t = torch.arange(tokens, device=q.device)
    seq = torch.searchsorted(cu[1:], t, right=True)
    live = seq < reqs
    seq = seq.clamp(max=reqs - 1)
    r = order[seq]
    pos = c[r] + t - cu[seq]
    slot = table[r, (pos // page).clamp(max=width - 1)].long() * page + pos % page
    return {"order": order.to(i32), "cu_seqlens": cu.to(i32), "state_indices": s["state_slots"][order],
            "num_decodes": (q == 1).sum().to(i32).view(1), "positions": torch.where(live, pos, 0).to(i32),
            "slot_map": torch.where(live, slot, -1), "free_left": (s["free_count"] - end[-1]).to(i32), "block_table": table}


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"norm_quant": _norm_quant, "matmul": _matmul, "maps": _maps}[op](s)
    from linear_attention_state_recurrent_gb300 import kda
    if op == "norm_quant":
        o = s["out"]
        kda.kda_norm_quant(s["x"], s["weight"], s["eps"], residual=s["residual"], residual_out=o["residual_out"],
                           y=o["y"], q=o["q"], scales=o["scales"])
        return {k: v for k, v in o.items() if v is not None}
    if op == "matmul":
        return kda.kda_fp8_matmul(s["a"], s["a_scales"], s["w"], s["w_scales"], out=s["out"])
    o = s["out"]
    kda.kda_batch_maps(s["query_lens"], s["context_lens"], s["state_slots"], s["block_table"], s["free_pages"],
                       s["free_count"], s["case"]["page"], num_pages=s["num_pages"], out=kda.BatchMaps(**o))
    return dict(o, block_table=s["block_table"])


def work(case):
    if case["op"] == "norm_quant":
        e = 4 if case["dtype"] == "fp32" else 2
        n = case["rows"] * case["cols"]
        tensors = 1 + 2 * case["residual"] + case["y"]
        return {"bytes": n * (tensors * e + 1) + case["rows"] * -(-case["cols"] // 128) * 4 + case["norm"] * case["cols"] * 4,
                "flops": n * (3 + 5 * case["norm"] + case["residual"])}
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        g = -(-k // 128)
        return {"bytes": m * k + n * k + 4 * g * (m + -(-n // 128)) + m * n * (4 if case["out"] == "fp32" else 2), "flops": 2 * m * n * k}
    reqs, tokens = case["reqs"], _tokens(case)
    pages = max(1, tokens // case["page"])   # read from the stack, written to the table
    return {"bytes": 28 * reqs + 12 * tokens + 8 * pages, "flops": 0}


def exact(case, seed):
    if case["op"] == "maps":
        return None
    s = prepare(case, seed)
    if case["op"] == "norm_quant":
        rows, cols = s["x"].shape
        h = s["x"].double() if s["residual"] is None else s["x"].double().add_(s["residual"].double())
        out = {"residual_out": h} if case["residual"] else {}
        y = h
        if case["norm"]:
            y = h / (torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / cols + s["eps"]).sqrt() * s["weight"].double()
        if case["y"]:
            out["y"] = y
        scales, q = [], []
        for g in range(0, cols, 128):
            part = y[:, g:g + 128]
            top = torch.maximum(part.amax(1), -part.amin(1)).clamp(min=TINY)
            scales.append(top / E4M3_MAX)
            q.append(part * (E4M3_MAX / top)[:, None])
        return out | {"q": torch.cat(q, 1), "scales": torch.stack(scales, 1)}
    m, n, k = case["m"], case["n"], case["k"]
    out = torch.zeros(m, n, dtype=torch.float64, device="cuda")
    sw = s["w_scales"].double()[torch.arange(n, device="cuda") // 128]
    for g in range(-(-k // 128)):
        at = slice(128 * g, min(k, 128 * g + 128))
        out.addmm_(s["a"][:, at].double() * s["a_scales"][:, g, None].double(), (s["w"][:, at].double() * sw[:, g, None]).t())
    return out
