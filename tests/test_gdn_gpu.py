"""GPU tests of the gated delta rule with one decay per head against its fp64 oracle.

Tolerances, from the arithmetic. Outputs are rounded once to bf16 (half a step is 2^-8 of the value); the products inside
take fp32 values as two bf16 terms: 8 bits of x, 8 bits of the rest, so 2^-17 of the value off at most and 2^-18.7 = 2.3e-6 in the mean. On the path
of a block's state there are six such values (S twice, y, T, U twice): in quadrature 6^(1/2) 2.3e-6 = 5.8e-6 of the state's norm, and
1e-5 with what is left of the errors of the blocks before. Outputs come by the same kind of products: in a row's norm
the rounding of the result (1.1e-3 to 1.7e-3 in the mean) and little else, 2e-3 in all; one value is off by half a step and, where a row is
small beside the terms that cancelled in it, by 1e-2 of the row's mean size. One token's products are fp32 throughout.
With one key for all tokens the sum over i of k^_i u_i is of u of alternating effect, and what counts is not its norm but
the terms': with Y = max |v| + |S_0|, T's rows sum to 2 at most in magnitude (beta (1 + beta + beta (1 - beta) + ..)), so |u_i| <= 2 Y,
and u_i is off by 3 * 2 Y (T, y and the product of their second terms) and 2 Y (its own two terms) times 2^-18.7; over the 64 tokens of
a block, in quadrature: 64^(1/2) * 8 Y 2^-18.7.
"""
import math

import numpy as np
import pytest
import torch

from oracle import gdn as og

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def kda():
    assert torch.cuda.is_available()
    from linear_attention_state_recurrent_gb300 import build
    build.build()
    from linear_attention_state_recurrent_gb300 import kda as k
    return k


def f64(t):
    return t.to(torch.float64).cpu().numpy()


class Case:
    """Inputs of a call, with NaN behind every row and in rows of no sequence."""

    def __init__(self, rows, entries, Hk, Hv, K, V, seed, pad=8, slots=None, spare=4, alike=False, strong=False, dt=True):
        g = torch.Generator().manual_seed(seed)
        randn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.Hk, self.Hv, self.K, self.V = Hk, Hv, K, V
        width = 2 * Hk * K + Hv * V
        self.qkv = torch.full((rows, width + pad), math.nan, dtype=BF16)
        x = randn(rows, width)
        if alike:   # one key for all tokens, and its negative: the largest entries that T can have
            x[:, Hk * K:2 * Hk * K] = x[:1, Hk * K:2 * Hk * K] * torch.where(torch.arange(rows) % 3 == 1, -1.0, 1.0)[:, None]
        self.qkv[:, :width] = x.to(BF16)
        self.rg, self.rb = randn(rows, Hv + 3).to(BF16), (randn(rows, Hv + 1) + (4.0 if alike else 0.0)).to(BF16)
        self.A_log = torch.rand(Hv, generator=g) * 2.77 + (3.0 if strong else -4.0 if alike else 0.0)
        self.dt = -3 + randn(Hv) if dt else None
        n = entries + spare
        self.pool = torch.full((n, Hv * K * V + 4), math.nan)
        self.pool[:, :Hv * K * V] = 0.05 * randn(n, Hv * K * V)
        self.slots = torch.randperm(n, generator=g)[:entries].tolist() if slots is None else slots
        self.width, self.rows = width, rows

    def gpu(self):
        self.d_qkv, self.d_rg, self.d_rb = self.qkv.cuda()[:, :self.width], self.rg.cuda()[:, :self.Hv], self.rb.cuda()[:, :self.Hv]
        self.d_pool = self.pool.cuda()
        self.state = torch.as_strided(self.d_pool, (len(self.pool), self.Hv, self.K, self.V), (self.d_pool.stride(0), self.K * self.V, self.V, 1))
        idx = torch.full((max(1, len(self.slots)), 3), 1 << 30, dtype=torch.int32)
        idx[:len(self.slots), 1] = torch.tensor(self.slots, dtype=torch.int32)
        self.out = torch.full((self.rows, self.Hv * self.V + 4), 7.0, dtype=BF16, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        return (self.d_qkv, self.d_rg, self.d_rb, self.A_log.cuda(), None if self.dt is None else self.dt.cuda(), self.state,
                idx.cuda()[:len(self.slots), 1])

    def check(self, bounds, null_slot=-1, err=0, exact=False, rows=None, alike=False):
        hkv = self.Hv * self.K * self.V
        pool = f64(self.pool[:, :hkv]).reshape(-1, self.Hv, self.K, self.V)
        out, after, flags = og.run(f64(self.qkv[:, :self.width]), f64(self.rg), f64(self.rb), f64(self.A_log),
                                   None if self.dt is None else f64(self.dt), pool, self.slots, bounds, self.Hk, null_slot=null_slot, rows=rows)
        assert self.err.item() == flags == err
        got = f64(self.out)
        assert (got[:, self.Hv * self.V:] == 7.0).all()                       # behind the rows
        free = np.isnan(out[:, 0])
        assert (got[free] == 7.0).all()                                       # rows of no sequence
        g, o = got[~free, :self.Hv * self.V].reshape(-1, self.V), out[~free].reshape(-1, self.V)
        if len(o):
            off = np.linalg.norm(g - o, axis=1) / np.maximum(np.linalg.norm(o, axis=1), 1e-30)
            off = np.where(np.linalg.norm(o, axis=1) == 0, np.linalg.norm(g, axis=1), off)
            total = np.linalg.norm(g - o) / max(np.linalg.norm(o), 1e-30)
            assert total <= 2e-3, total
            rms = np.sqrt((o ** 2).mean(1, keepdims=True))
            assert (np.abs(g - o) <= 2.0 ** -8 * np.abs(o) + (1e-6 if exact else 1e-2) * rms + 1e-30).all()
        p = f64(self.d_pool)
        np.testing.assert_array_equal(p[:, hkv:], f64(self.pool[:, hkv:]))    # behind the slots
        p = p[:, :hkv].reshape(pool.shape)
        worst = 0.0
        for s in range(len(pool)):
            if (after[s] == pool[s]).all():
                np.testing.assert_array_equal(p[s], pool[s])
                continue
            for h in range(self.Hv):
                worst = max(worst, np.linalg.norm(p[s, h] - after[s, h]) / np.linalg.norm(after[s, h]))
        most = 2e-6 if exact else 1e-5
        if alike:
            v = f64(self.qkv[:, 2 * self.Hk * self.K:self.width]).reshape(self.rows, self.Hv, self.V)
            most = 64 ** 0.5 * 8 * 2.0 ** -18.7 * (np.linalg.norm(v, axis=2).max() + np.linalg.norm(pool, axis=(2, 3)).max())
            worst *= max(np.linalg.norm(after[s, h]) for s in range(len(pool)) for h in range(self.Hv))
        assert worst <= most, (worst, most)


HEADS = [(1, 1, 128, 128), (2, 4, 128, 64), (1, 3, 64, 128), (2, 2, 64, 64), (1, 2, 32, 128), (1, 1, 128, 32), (2, 4, 32, 32), (1, 2, 64, 32)]


@pytest.mark.parametrize("Hk, Hv, K, V", HEADS)
@pytest.mark.parametrize("n", [1, 5])
def test_decode(kda, Hk, Hv, K, V, n):
    c = Case(n, n, Hk, Hv, K, V, seed=K + V + n)
    kda.kda_gdn_decode(*c.gpu(), num_k_heads=Hk, out=c.out, err_flags=c.err)
    c.check([(i, i + 1) for i in range(n)], exact=True)


@pytest.mark.parametrize("Hk, Hv, K, V", HEADS)
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 64])
def test_spec_verify(kda, Hk, Hv, K, V, T):
    c = Case(3 * T, 3, Hk, Hv, K, V, seed=T, pad=7 if T == 7 else 8)          # rows off 16-byte boundaries too
    kda.kda_gdn_spec_verify(*c.gpu(), T, num_k_heads=Hk, out=c.out, err_flags=c.err)
    c.check([(r * T, (r + 1) * T) for r in range(3)])


@pytest.mark.parametrize("pad", [7, 8])
@pytest.mark.parametrize("Hk, Hv, K, V", HEADS)
def test_prefill(kda, Hk, Hv, K, V, pad):
    lens = [1, 63, 64, 0, 65, 130, 2, 200]
    cu = np.concatenate([[2], 2 + np.cumsum(lens)]).tolist()
    c = Case(cu[-1] + 3, len(lens), Hk, Hv, K, V, seed=4, pad=pad, dt=V != 64)
    c.qkv[:2] = c.qkv[-3:] = math.nan
    kda.kda_gdn_chunk_prefill(*c.gpu(), torch.tensor(cu, dtype=torch.int32, device="cuda"), num_k_heads=Hk, out=c.out, err_flags=c.err)
    c.check(list(zip(cu, cu[1:])))


@pytest.mark.parametrize("what", ["alike", "strong"])
@pytest.mark.parametrize("K, V", [(128, 128), (64, 64), (32, 32)])
def test_prefill_extremes(kda, what, K, V):
    """The same key again and again with beta near 1 and little decay; and a decay of thousands of nats in a chunk."""
    c = Case(300, 2, 1, 2, K, V, seed=9, **{what: True})
    cu = [0, 170, 300]
    kda.kda_gdn_chunk_prefill(*c.gpu(), torch.tensor(cu, dtype=torch.int32, device="cuda"), num_k_heads=1, out=c.out, err_flags=c.err)
    c.check(list(zip(cu, cu[1:])), alike=what == "alike")


@pytest.mark.parametrize("call", ["decode", "spec", "prefill", "prefill32"])
def test_slots(kda, call):
    T, K = (1 if call == "decode" else 5), (32 if call == "prefill32" else 64)
    c = Case(5 * T, 5, 1, 2, K, 64, seed=8, slots=[2, -1, 0, 9, 4])           # 9 slots: the fourth is past them, 0 is null
    a = c.gpu()
    kw = dict(num_k_heads=1, out=c.out, err_flags=c.err, null_slot=0)
    bounds = [(i * T, i * T + T) for i in range(5)]
    if call == "decode":
        kda.kda_gdn_decode(*a, **kw)
    elif call == "spec":
        kda.kda_gdn_spec_verify(*a, T, **kw)
    else:
        kda.kda_gdn_chunk_prefill(*a, torch.tensor([0, 5, 10, 15, 20, 25], dtype=torch.int32, device="cuda"), **kw)
    c.check(bounds, null_slot=0, err=og.ERR_SLOT_RANGE)


@pytest.mark.parametrize("K", [32, 128])
def test_prefill_lengths_out_of_range(kda, K):
    cu = [0, 70, 60, 60, 400, -5, 20]   # no two ranges share a row
    c = Case(100, 6, 1, 1, K, 64, seed=12)
    kda.kda_gdn_chunk_prefill(*c.gpu(), torch.tensor(cu, dtype=torch.int32, device="cuda"), out=c.out, err_flags=c.err)
    c.check(list(zip(cu, cu[1:])), err=og.ERR_LENGTHS)


@pytest.mark.parametrize("K", [32, 128])
def test_prefill_in_parts_is_prefill(kda, K):
    """A prompt in two calls, the second from the first one's state, then decoded on: the whole by the oracle."""
    c = Case(150, 1, 1, 2, K, 64, seed=13, slots=[3])
    qkv, rg, rb, *rest = c.gpu()
    for r0, r1 in ((0, 77), (77, 149), (149, 150)):
        kw = dict(num_k_heads=1, out=c.out[r0:r1], err_flags=c.err)
        if r1 - r0 == 1:
            kda.kda_gdn_decode(qkv[r0:r1], rg[r0:r1], rb[r0:r1], *rest, **kw)
        else:
            kda.kda_gdn_chunk_prefill(qkv[r0:r1], rg[r0:r1], rb[r0:r1], *rest, torch.tensor([0, r1 - r0], dtype=torch.int32, device="cuda"), **kw)
    c.check([(0, 150)])


@pytest.mark.parametrize("n, Hk, Hv, K, V, top", [(40, 2, 4, 128, 128, 150), (300, 1, 1, 64, 64, 90), (1100, 1, 1, 64, 32, 3)])
def test_prefill_many_sequences(kda, n, Hk, Hv, K, V, top):
    """More chains than multiprocessors; more sequences than are sorted, and than one turn of the chunks' map takes."""
    g = torch.Generator().manual_seed(n)
    cu = [0] + torch.cumsum(torch.randint(0, top, (n,), generator=g), 0).tolist()
    c = Case(cu[-1], n, Hk, Hv, K, V, seed=n)
    args, d_cu = c.gpu(), torch.tensor(cu, dtype=torch.int32, device="cuda")
    kda.kda_gdn_chunk_prefill(*args, d_cu, num_k_heads=Hk, out=c.out, err_flags=c.err)
    c.check(list(zip(cu, cu[1:])))
    # the same bits again, and from a workspace that held something else
    first, out = c.d_pool.clone(), c.out.clone()
    c.d_pool.copy_(c.pool)
    ws = torch.full((kda.kda_gdn_chunk_prefill_workspace_bytes(cu[-1], n, Hv, K, V, Hk),), 255, dtype=torch.uint8, device="cuda")
    kda.kda_gdn_chunk_prefill(*args, d_cu, num_k_heads=Hk, out=c.out, err_flags=c.err, workspace=ws)
    assert torch.equal(first.view(torch.int32), c.d_pool.view(torch.int32)) and torch.equal(out, c.out)


def test_prefill_is_untouched_by_what_lies_around(kda):
    """Infinities and NaN in rows of other sequences, and in the rows behind the last, stay there."""
    lens = [70, 50, 100]
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    c = Case(cu[-1] + 40, 3, 1, 2, 128, 64, seed=21)
    c.qkv[cu[1]:cu[2]] = math.inf
    c.qkv[cu[1] + 7] = math.nan
    c.qkv[cu[3]:] = math.nan
    args, d_cu = c.gpu(), torch.tensor(cu, dtype=torch.int32, device="cuda")
    kda.kda_gdn_chunk_prefill(*args, d_cu, num_k_heads=1, out=c.out, err_flags=c.err)
    spoilt = c.slots[1]
    c.pool[spoilt], c.d_pool[spoilt] = 0.0, 0.0
    keep = c.out[cu[1]:cu[2]].clone()
    c.out[cu[1]:cu[2]] = 7.0
    c.check([(cu[0], cu[1]), (0, 0), (cu[2], cu[3])])
    assert not torch.isfinite(keep[:, :128].float()).any()


@pytest.mark.parametrize("call", ["decode", "spec", "prefill"])
def test_offsets_past_32_bits(kda, call):
    """Slots and rows whose offsets pass 2^31 elements."""
    T = 1 if call == "decode" else 8 if call == "spec" else 70
    n = 2
    c = Case(n * T, n, 1, 1, 64, 64, seed=31, slots=[3, 1], spare=2)
    qkv, rg, rb, A, dt, state, idx = c.gpu()
    pitch = (1 << 31) // (n * T) * 2 + 8 & ~7
    big = torch.empty(n * T * pitch, dtype=BF16, device="cuda").view(n * T, pitch)
    big[:, :c.width] = qkv
    slot = 1 << 30
    pool = torch.empty(4 * slot, dtype=torch.float32, device="cuda").view(4, slot)
    pool[:, :64 * 64] = c.d_pool[:, :64 * 64]
    view = pool.as_strided((4, 1, 64, 64), (slot, 64 * 64, 64, 1))
    wide = big[:, c.width + 8 & ~7:][:, :64]
    kw = dict(out=wide, err_flags=c.err)
    if call == "decode":
        kda.kda_gdn_decode(big[:, :c.width], rg, rb, A, dt, view, idx, **kw)
    elif call == "spec":
        kda.kda_gdn_spec_verify(big[:, :c.width], rg, rb, A, dt, view, idx, T, **kw)
    else:
        kda.kda_gdn_chunk_prefill(big[:, :c.width], rg, rb, A, dt, view, idx, torch.tensor([0, 70, 140], dtype=torch.int32, device="cuda"), **kw)
    c.out[:, :64] = wide
    c.d_pool[:, :64 * 64] = pool[:, :64 * 64]
    c.check([(0, T), (T, 2 * T)])


def test_streams_and_graphs(kda):
    """Every call on another stream with outputs and workspaces of its own, and captured; two graphs with a workspace each."""
    c = Case(3 * 80, 3, 1, 2, 128, 128, seed=41)
    args = c.gpu()
    cu = torch.tensor([0, 80, 160, 240], dtype=torch.int32, device="cuda")
    start = c.d_pool.clone()

    def calls(stream=None, ws=None):
        a, _ = kda.kda_gdn_chunk_prefill(*args, cu, num_k_heads=1, workspace=ws, stream=stream)
        b, _ = kda.kda_gdn_spec_verify(*[t[:24] for t in args[:3]], *args[3:], 8, num_k_heads=1, stream=stream)
        d, _ = kda.kda_gdn_decode(*[t[:3] for t in args[:3]], *args[3:], num_k_heads=1, stream=stream)
        return a, b, d

    want = [t.clone() for t in calls()] + [c.d_pool.clone()]
    s = torch.cuda.Stream()
    c.d_pool.copy_(start)
    s.wait_stream(torch.cuda.current_stream())
    got = calls(s)
    torch.cuda.current_stream().wait_stream(s)
    same = lambda got: all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip([*got, c.d_pool], want))  # noqa: E731
    assert same(got)
    graphs = []
    for _ in range(2):
        ws = torch.empty(kda.kda_gdn_chunk_prefill_workspace_bytes(240, 3, 2, 128, 128, 1), dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = calls(ws=ws)
        graphs.append((g, got, ws))
    for g, got, _ in graphs * 2:
        c.d_pool.copy_(start)
        g.replay()
        assert same(got)


def run(kda, c, call, cu):
    kw = dict(num_k_heads=c.Hk, out=c.out, err_flags=c.err)
    if call == "spec":
        kda.kda_gdn_spec_verify(*c.gpu_args, cu[1], **kw)
    else:
        kda.kda_gdn_chunk_prefill(*c.gpu_args, torch.tensor(cu, dtype=torch.int32, device="cuda"), **kw)


@pytest.mark.parametrize("where", ["key", "value", "gate", "beta"])
@pytest.mark.parametrize("call, K, V, T, at", [("spec", 128, 128, 5, 3), ("spec", 64, 64, 16, 0), ("spec", 128, 32, 20, 17), ("prefill", 32, 64, 40, 9),
                                               ("prefill", 128, 128, 150, 127), ("prefill", 64, 64, 70, 66)])
def test_what_is_not_finite_reaches_no_earlier_token(kda, call, K, V, T, at, where):
    """A row's outputs are finite where the oracle's are, and right; of the chunked form, those of the chunks before."""
    c = Case(2 * T, 2, 1, 2, K, V, seed=31)
    bad = T + at                                                              # in the second sequence
    if where == "key":
        c.qkv[bad, K + 3] = math.nan
    elif where == "value":
        c.qkv[bad, 2 * K + 5], c.qkv[bad, 2 * K + V + 1] = math.inf, math.nan
    elif where == "gate":
        c.rg[bad, 1] = math.nan
    else:
        c.rb[bad, 1] = math.nan
    c.gpu_args = c.gpu()
    run(kda, c, call, [0, T, 2 * T])
    with np.errstate(invalid="ignore"):
        out, after, _ = og.run(f64(c.qkv[:, :c.width]), f64(c.rg), f64(c.rb), f64(c.A_log), f64(c.dt), f64(c.pool[:, :2 * K * V]).reshape(-1, 2, K, V),
                               c.slots, [(0, T), (T, 2 * T)], 1)
    got, state = f64(c.out)[:, :2 * V], f64(c.state)[c.slots[1]]
    np.testing.assert_array_equal(np.isfinite(state), np.isfinite(after[c.slots[1]]))
    seen = np.ones(2 * T, bool)
    if call == "prefill" and K > 32:
        seen[T + at // 64 * 64:bad] = False                                   # its chunk's rows ahead of it
    fine = np.isfinite(out)
    np.testing.assert_array_equal(np.isfinite(got[seen]), fine[seen])
    for h in range(2):
        rows = seen & fine[:, h * V]
        o = np.where(fine, out, 0.0)[rows, h * V:(h + 1) * V]
        rms = np.sqrt((o ** 2).mean(1, keepdims=True))
        g = np.where(fine, got, 0.0)[rows, h * V:(h + 1) * V]
        assert (np.abs(g - o) <= 2.0 ** -8 * np.abs(o) + 1e-2 * rms + 1e-30).all()


@pytest.mark.parametrize("call, K, T", [("spec", 128, 7), ("spec", 64, 16), ("prefill", 32, 50), ("prefill", 128, 150), ("prefill", 64, 90)])
def test_decays_without_end(kda, call, K, T):
    """exp(A_log) past fp32's range, and an infinite raw_g: alpha is 0, and the tokens behind go on as ever."""
    c = Case(2 * T, 2, 1, 3, K, 64, seed=32)
    c.A_log[0] = 100.0
    c.rg[T // 2, 1] = c.rg[T + 2, 2] = math.inf
    c.rg[T - 1, 1] = -math.inf                                                # and one without any
    c.gpu_args = c.gpu()
    run(kda, c, call, [0, T, 2 * T])
    c.check([(0, T), (T, 2 * T)])


@pytest.mark.parametrize("Hk, Hv, K, V", HEADS)
def test_spec_verify_states_to_tf32_pairs(kda, Hk, Hv, K, V):
    """fp32 values enter the products of a few rows as two truncated tf32 terms: six of them on a state's path, each off by 2^-20 at most,
    6^(1/2) 2^-20 = 2.4e-6 of the norm, and fp32 sums of up to 128 terms, 128^(1/2) 2^-24 = 0.7e-6."""
    T = 8
    c = Case(4 * T, 4, Hk, Hv, K, V, seed=41)
    kda.kda_gdn_spec_verify(*c.gpu(), T, num_k_heads=Hk, out=c.out, err_flags=c.err)
    pool = f64(c.pool[:, :Hv * K * V]).reshape(-1, Hv, K, V)
    _, after, _ = og.run(f64(c.qkv[:, :c.width]), f64(c.rg), f64(c.rb), f64(c.A_log), f64(c.dt), pool, c.slots, [(r * T, (r + 1) * T) for r in range(4)], Hk)
    got = f64(c.state)
    for s in c.slots:
        for h in range(Hv):
            assert np.linalg.norm(got[s, h] - after[s, h]) <= 3.1e-6 * np.linalg.norm(after[s, h])


@pytest.mark.parametrize("Hk, Hv, K, lens, slots", [
    (1, 2, 64, [4100], [0]), (1, 2, 64, [4096, 6300, 0, 4200], [3, -1, 2, 0]), (2, 4, 64, [9000, 100], [9, 1]), (1, 1, 128, [4097, 8200], [1, 0]),
    (1, 1, 128, [5000], [-1]), (19, 38, 64, [4200], [2])])
def test_prefill_in_joined_parts(kda, Hk, Hv, K, lens, slots):
    """Few long sequences, whose parts go side by side and are joined; with short ones, no state, a null slot and one past the pool among them.
    A part's end is A S + B: as many products of the same errors on the state's path, and a joined output two terms of 2^-11 of tf32 operands
    beside its rounding of 2^-9 in the mean, below 2e-3 of the norm still."""
    cu = np.concatenate([[3], 3 + np.cumsum(lens)]).tolist()
    rows = max(cu[-1] + 5, 4096 * len(lens))
    c = Case(rows, len(lens), Hk, Hv, K, K, seed=51, slots=slots)
    c.A_log -= 6.0                                                            # little decay: the parts depend on one another
    args = c.gpu()
    kda.kda_gdn_chunk_prefill(*args, torch.tensor(cu, dtype=torch.int32, device="cuda"), num_k_heads=Hk, out=c.out, err_flags=c.err, null_slot=2)
    c.check(list(zip(cu, cu[1:])), null_slot=2, err=og.ERR_SLOT_RANGE if max(slots) >= 4 + len(lens) else 0)


def test_one_graph_cuts_and_leaves_whole(kda):
    """A captured call over one long row range serves lengths that are cut into parts, and such as are not."""
    c = Case(9000, 2, 1, 2, 64, 64, seed=52)
    args, cu = c.gpu(), torch.tensor([0, 9000, 9000], dtype=torch.int32, device="cuda")
    ws = torch.empty(kda.kda_gdn_chunk_prefill_workspace_bytes(9000, 2, 2, 64, 64, num_k_heads=1), dtype=torch.uint8, device="cuda")
    run = lambda: kda.kda_gdn_chunk_prefill(*args, cu, num_k_heads=1, out=c.out, err_flags=c.err, workspace=ws)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for bounds in ([5, 70, 5000], [0, 4096, 4100], [0, 4095, 8191], [0, 0, 9000]):
        c.d_pool.copy_(c.pool)
        c.out.fill_(7.0)
        ws.fill_(255)
        cu.copy_(torch.tensor(bounds, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        c.check(list(zip(bounds, bounds[1:])))


def test_parts_keep_what_is_not_finite(kda):
    """A NaN in the third of the parts reaches no row ahead of its chunk, and every state and row behind it."""
    c = Case(4500, 1, 1, 1, 64, 64, seed=53)
    bad = 2 * 9 * 64 + 70                                                     # eight parts of nine chunks
    c.qkv[bad, 64 + 7] = math.nan
    kda.kda_gdn_chunk_prefill(*c.gpu(), torch.tensor([0, 4500], dtype=torch.int32, device="cuda"), num_k_heads=1, out=c.out, err_flags=c.err)
    got = f64(c.out)[:, :64]
    first = bad // 64 * 64
    assert np.isfinite(got[:first]).all() and not np.isfinite(got[bad:]).any() and not np.isfinite(f64(c.state)[c.slots[0]]).any()
    out, _, _ = og.run(f64(c.qkv[:, :c.width]), f64(c.rg), f64(c.rb), f64(c.A_log), f64(c.dt), f64(c.pool[:, :64 * 64]).reshape(-1, 1, 64, 64), c.slots,
                       [(0, first)], 1)
    o = out[:first]
    assert (np.abs(got[:first] - o) <= 2.0 ** -8 * np.abs(o) + 1e-2 * np.sqrt((o ** 2).mean(1, keepdims=True)) + 1e-30).all()


@pytest.mark.parametrize("scale", [-2.0e5, 1e-12, 0.0])
def test_parts_with_columns_of_any_size(kda, scale):
    """Joined outputs of value columns from 1e-15 to 1e15, and any scale: each column as near as its own size lets it be, and each state.
    Of a state, a column takes the six two-term values of the norm's bound by itself: 1e-5 of it."""
    K = V = 64
    c = Case(4500, 1, 1, 1, K, V, seed=54)
    c.A_log -= 6.0
    size = torch.logspace(-15, 15, V)
    c.qkv[:, 2 * K:c.width] *= size.to(BF16)
    c.pool[:, :K * V] *= size.repeat(K)
    kda.kda_gdn_chunk_prefill(*c.gpu(), torch.tensor([0, 4500], dtype=torch.int32, device="cuda"), num_k_heads=1, scale=scale, out=c.out, err_flags=c.err)
    out, after, _ = og.run(f64(c.qkv[:, :c.width]), f64(c.rg), f64(c.rb), f64(c.A_log), f64(c.dt), f64(c.pool[:, :K * V]).reshape(-1, 1, K, V), c.slots,
                           [(0, 4500)], 1, scale=float(np.float32(scale)))
    got, state = f64(c.out)[:, :V], f64(c.state)[c.slots[0]][0]
    off = np.linalg.norm(got - out, axis=0)
    assert (off <= 2e-3 * np.linalg.norm(out, axis=0)).all(), off / np.linalg.norm(out, axis=0)
    want = after[c.slots[0]][0]
    assert (np.linalg.norm(state - want, axis=0) <= 1e-5 * np.linalg.norm(want, axis=0)).all()
