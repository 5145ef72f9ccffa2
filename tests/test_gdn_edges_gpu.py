"""GPU tests of the gated delta rule's chunked prefill at the edges of its batches, against its fp64 oracle. Tolerances as in
test_gdn_gpu.py: a state within 1e-5 of its norm, an output within its rounding (2^-8 of it) and 1e-2 of its row's mean size, 2e-3 of the norm in all."""
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


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Batch:
    """A prefill's inputs on the GPU: sequences of `lens` rows one after the other."""

    def __init__(self, lens, Hk, Hv, K, V, slots, num_slots, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
        n = self.cu[-1]
        self.Hk, self.K, self.V, self.slots = Hk, K, V, slots
        self.qkv = randn(n, 2 * Hk * K + Hv * V).to(BF16)
        self.rg, self.rb = randn(n, Hv).to(BF16), randn(n, Hv).to(BF16)
        self.A_log, self.dt = torch.rand(Hv, generator=g, device="cuda"), -3 + randn(Hv)   # dt: None for zeros
        self.pool = 0.05 * randn(num_slots, Hv, K, V)
        self.start = self.pool.clone()
        self.out = torch.full((n, Hv * V), 7.0, dtype=BF16, device="cuda")
        self.err = i32([0])

    def run(self, kda, **kw):
        kda.kda_gdn_chunk_prefill(self.qkv, self.rg, self.rb, self.A_log, self.dt, self.pool, i32(self.slots), i32(self.cu), num_k_heads=self.Hk, out=self.out,
                                  err_flags=self.err, **kw)

    def oracle(self, slots, bounds):
        return og.run(*(None if x is None else f64(x) for x in (self.qkv, self.rg, self.rb, self.A_log, self.dt, self.start)), slots, bounds, self.Hk)

    def run_and_check_rows(self, kda, least=1e-30):
        """One sequence: every row by itself, down to `least`, and every head's state."""
        self.run(kda)
        out, after, err = self.oracle(self.slots, [(0, self.cu[1])])
        assert self.err.item() == err == 0
        g, o = (x.reshape(-1, self.V) for x in (f64(self.out), out))
        norms = np.linalg.norm(o, axis=1)
        off = np.linalg.norm(g - o, axis=1)
        seen = norms > least
        assert (off[seen] <= 4e-3 * norms[seen]).all(), (off[seen] / norms[seen]).max()
        assert (off[~seen] <= least).all()
        slot = self.slots[0]
        size = np.linalg.norm(after[slot], axis=(1, 2))
        rel = np.linalg.norm(f64(self.pool)[slot] - after[slot], axis=(1, 2)) / np.maximum(size, least)
        assert rel.max() <= 1e-5, rel.max()

    def check(self, entries):
        """The given sequences' outputs and states; those of their slots alone have changed."""
        assert self.err.item() == 0
        slots, bounds = [self.slots[e] for e in entries], [(self.cu[e], self.cu[e + 1]) for e in entries]
        out, after, _ = self.oracle(slots, bounds)
        rows = np.concatenate([np.arange(*b) for b in bounds])
        g, o = (x[rows].reshape(-1, self.V) for x in (f64(self.out), out))
        assert np.linalg.norm(g - o) <= 2e-3 * np.linalg.norm(o)
        assert (np.abs(g - o) <= 2.0 ** -8 * np.abs(o) + 1e-2 * np.sqrt((o ** 2).mean(1, keepdims=True))).all()
        off = np.linalg.norm(f64(self.pool) - after, axis=(2, 3)) / np.linalg.norm(after, axis=(2, 3))
        assert off.max() <= 1e-5, off.max()
        same = sorted(set(range(len(after))) - set(slots))
        assert torch.equal(self.pool[same], self.start[same])


@pytest.mark.parametrize("K, V", [(64, 64), (128, 32)])
def test_long_runs_of_empty_sequences(kda, K, V):
    """Thousands of entries without rows between the chains of each multiprocessor; every sequence ends inside a chunk and has rows of NaN behind it."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    r = np.random.default_rng(1)
    lens, live = [], []
    for part in range(2):
        for _ in range(sms):
            live.append(len(lens))
            lens += [64 * int(r.integers(2, 5)) + int(r.integers(1, 64)), 70]
        if part == 0:
            lens += [0] * (60 * sms)
    slots = [-1] * len(lens)
    for i, e in enumerate(live):
        slots[e] = i
    b = Batch(lens, 1, 1, K, V, slots, len(live) + 2, seed=K)
    for e in live:
        b.qkv[b.cu[e + 1]:b.cu[e + 2]] = math.nan
    b.run(kda)
    b.check(live)


def test_few_sequences_with_rows_among_many_heads(kda):
    """A step of 256 entries of which 16 have rows, with 64 heads: a hundred chains without rows behind each multiprocessor's own."""
    r = np.random.default_rng(2)
    lens = np.zeros(256, int)
    live = r.permutation(256)[:16].tolist()
    lens[live] = r.integers(65, 128, 16)
    slots = [-1] * 256
    for i, e in enumerate(live):
        slots[e] = i
    b = Batch(lens.tolist(), 2, 64, 64, 32, slots, 17, seed=3)
    b.run(kda)
    b.check(live)


def test_overlapping_ranges_count_no_further_than_the_workspace(kda):
    """Ranges over all rows again and again, 2^31 chunks and more between them: those that the workspace has chunks for are computed, the others count as empty, and
    the lengths' bit says so."""
    rows, n, K, V = 1 << 22, 65600, 64, 32
    b = Batch([rows], 1, 1, K, V, [0], 3, seed=5)
    b.run(kda)
    assert b.err.item() == 0
    want = b.pool[0].clone()
    b.pool.copy_(b.start)
    b.cu = [0, rows] * (n // 2) + [0]
    b.slots = [0, 2, 1] + [2] * (n - 3)
    b.pool[1] = b.pool[0]
    b.run(kda)
    assert b.err.item() == og.ERR_LENGTHS
    assert torch.equal(b.pool[0], want) and torch.equal(b.pool[1], want) and torch.equal(b.pool[2], b.start[2])


@pytest.mark.parametrize("K, Hv, rows", [(64, 1, 4500), (128, 1, 4300), (64, 40, 4200)])
@pytest.mark.parametrize("decay, beta", [(0.03, -30.0), (0.012, -4.0)])
def test_parts_whose_outputs_are_what_is_left_of_the_state(kda, K, Hv, rows, decay, beta):
    """Sequences in joined parts whose values end with the first 500 rows: from there on an output is the transition's row times the part's start, and both shrink, by
    e^-7 to e^-60 within a part. Each row is as near as any: rounded to bf16, 2^-8 of its norm at most (1.7e-3 in the mean), and of terms whose two factors are off by
    half a step of fp16, 2^-11 at most and 2.0e-4 in the mean each, of random signs (little is written, so that the state keeps its rank): 4e-3 in quadrature."""
    b = Batch([rows], 1, Hv, K, K, [1], 3, seed=K + Hv)
    b.A_log.zero_()
    b.dt = None
    b.rg.fill_(math.log(math.expm1(decay)))
    b.rb.fill_(beta)
    b.rb[:500] = 0.0
    b.qkv[500:, 2 * K:] = 0.0
    b.run_and_check_rows(kda)


@pytest.mark.parametrize("size", [2e35, 1e-30])
def test_parts_with_states_near_the_ends_of_fp32(kda, size):
    """Joined outputs where every value is above 2^114, or small: rows as near as any (tolerance as above; little decay, so that the parts depend on one another)."""
    b = Batch([4500], 1, 1, 64, 64, [1], 3, seed=9)
    b.A_log -= 6.0
    b.qkv[:, 128:] *= size
    b.pool *= size
    b.start = b.pool.clone()
    b.run_and_check_rows(kda, least=1e-3 * size)


@pytest.mark.parametrize("K, V, most", [(128, 128, 2.0e-6), (128, 64, 2.0e-6), (64, 64, 2.5e-6)])
def test_states_to_the_products_terms(kda, K, V, most):
    """What is off in a state, of its norm: a bf16 pair is off by 2.3e-6 of a value in the mean. Below T's diagonal its product with Y has three such errors (T's pair, Y's, and the
    second terms' product), and is beta (32 / K)^(1/2) = 0.25 to 0.35 of Z: 1.0e-6 to 1.4e-6. S as the first operand of K S: 2.3e-6 of what is half of Y at most. Sums of 12 steps
    of the products, each cut at 2^-24 of them: 0.5e-6. In quadrature 1.6e-6 to 1.9e-6."""
    b = Batch([700, 65, 640], 1, 2, K, V, [0, 1, 2], 4, seed=K + V)
    b.run(kda)
    _, after, _ = b.oracle(b.slots, list(zip(b.cu, b.cu[1:])))
    got = f64(b.pool)
    for s in b.slots:
        assert np.linalg.norm(got[s] - after[s]) <= most * np.linalg.norm(after[s]), (s, np.linalg.norm(got[s] - after[s]) / np.linalg.norm(after[s]))


@pytest.mark.parametrize("call", ["decode", "spec", "prefill"])
def test_betas_of_zero_and_one(kda, call):
    """raw_beta without bounds: a token that writes nothing at all, and one that replaces what its key reads. Tolerance as at the top."""
    b = Batch([90, 1, 200] if call == "prefill" else [1] * 24 if call == "decode" else [8] * 3, 1, 2, 128, 64, list(range(24 if call == "decode" else 3)), 25, seed=6)
    b.rb[::3], b.rb[1::3] = -math.inf, math.inf
    b.rb[5::7], b.rb[6::7] = -200.0, 200.0
    if call == "prefill":
        b.run(kda)
    else:
        args = (b.qkv, b.rg, b.rb, b.A_log, b.dt, b.pool, i32(b.slots))
        kw = dict(num_k_heads=1, out=b.out, err_flags=b.err)
        kda.kda_gdn_decode(*args, **kw) if call == "decode" else kda.kda_gdn_spec_verify(*args, 8, **kw)
    b.check(range(len(b.slots)))
