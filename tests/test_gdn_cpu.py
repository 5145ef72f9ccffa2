"""The gated delta rule with one decay per head on the host: pins of its fp64 oracle and every refusal of the C ABI and of
the binding. No GPU: each call here fails its checks before anything is launched."""
import ctypes

import numpy as np
import pytest
import torch

from linear_attention_state_recurrent_gb300 import workloads as wl
from oracle import gdn as og
from oracle import kda_oracle as ko


@pytest.fixture(scope="module")
def kda():
    from linear_attention_state_recurrent_gb300 import build
    build.build()
    from linear_attention_state_recurrent_gb300 import kda as k
    return k


# ---- the oracle ---------------------------------------------------------------------------


def test_one_token_by_hand():
    # alpha 1/2, beta 1/2, unit key along the first channel: S = diag(1/2, 1), u = (2 - 1/2, 4) / 2
    S, o = og.step(np.array([[1.0, 0.0], [0.0, 2.0]]), np.array([1.0, 0.0]), np.array([3.0, 0.0]), np.array([2.0, 4.0]), 0.5, 0.5, 2.0, 0.0)
    np.testing.assert_allclose(S, [[0.5 + 0.75, 2.0], [0.0, 1.0]])
    np.testing.assert_allclose(o, [2.5, 4.0])


def test_gate_by_hand():
    alpha, beta = og.gate(np.zeros((1, 2)), np.zeros((1, 2)), np.array([0.0, np.log(2.0)]), np.array([0.0, np.log(np.e - 1)]))
    np.testing.assert_allclose(alpha, [[0.5, np.exp(-2.0)]])      # softplus(0) = ln 2, softplus(ln(e - 1)) = 1
    np.testing.assert_allclose(beta, [[0.5, 0.5]])


@pytest.mark.parametrize("lengths, num_decodes, kind", [([1, 1, 1], 3, "mixed"), ([5, 1, 7], 0, "prefill")])
def test_equals_kda_with_the_same_decay_in_every_channel(lengths, num_decodes, kind):
    w = wl.varlen_case(lengths, 2, 32, 32, seed=3, num_decodes=num_decodes, kind=kind, name="gdn")
    H, K, V = w.H, w.K, w.V
    w.raw_g = np.repeat(np.asarray(w.raw_g)[:, :H * K:K], K, axis=1)         # channel 0's for all channels of its head
    w.dt_bias = np.repeat(np.asarray(w.dt_bias).reshape(H, K)[:, :1], K, axis=1).reshape(-1).astype(np.float32)
    w.lower_bound = None
    r = ko.run(w)
    f = lambda a: (np.asarray(a, np.uint32) << 16).view(np.float32).astype(np.float64)  # noqa: E731
    pool = np.asarray(w.pool)[:, :H * K * V].reshape(-1, H, K, V).astype(np.float64)
    out, after, err = og.run(f(w.mixed_qkv), f(w.raw_g)[:, ::K], f(w.raw_beta), np.float64(w.A_log), np.float64(w.dt_bias[::K]), pool,
                             w.indices(), w.seq_bounds(), H, w.scale, w.eps, w.null_slot)
    assert err == r.err_flags
    np.testing.assert_allclose(out, r.out, rtol=1e-11, atol=1e-13)
    np.testing.assert_allclose(after.reshape(len(pool), -1), r.expected_pool(np.asarray(w.pool))[:, :H * K * V], rtol=1e-11, atol=1e-13)


def test_shared_key_heads_equal_repeated_ones():
    rng = np.random.default_rng(5)
    Hk, Hv, K, V, N = 2, 6, 4, 3, 7
    q, k, v = rng.normal(size=(N, Hk, K)), rng.normal(size=(N, Hk, K)), rng.normal(size=(N, Hv, V))
    g, b, A, dt, pool = rng.normal(size=(N, Hv)), rng.normal(size=(N, Hv)), rng.normal(size=Hv), rng.normal(size=Hv), rng.normal(size=(2, Hv, K, V))
    flat = lambda *x: np.concatenate([y.reshape(N, -1) for y in x], 1)  # noqa: E731
    one = og.run(flat(q, k, v), g, b, A, dt, pool, [1], [(0, N)], Hk)
    two = og.run(flat(q.repeat(3, 1), k.repeat(3, 1), v), g, b, A, dt, pool, [1], [(0, N)], Hv)
    for x, y in zip(one, two):
        np.testing.assert_array_equal(x, y)


def test_slots_and_lengths():
    rng = np.random.default_rng(6)
    pool = rng.normal(size=(3, 1, 2, 2))
    args = (rng.normal(size=(6, 6)), rng.normal(size=(6, 1)), rng.normal(size=(6, 1)), np.zeros(1), None, pool)
    out, after, err = og.run(*args, [0, -1, 3, 1, 2], [(0, 1), (1, 2), (2, 3), (3, 3), (5, 9)], 1, null_slot=0)
    assert err == og.ERR_SLOT_RANGE | og.ERR_LENGTHS
    np.testing.assert_array_equal(after, pool)
    assert np.isfinite(out[:3]).all() and (out[2] == 0).all() and np.isnan(out[3:]).all()


# ---- the C ABI's refusals ------------------------------------------------------------------

FAKE = 1 << 20   # never dereferenced


def call(kda, name, change=None, heads=None, state=None):
    """The call with sound arguments, but for what is changed; the status."""
    H = dict(Hk=2, Hv=4, K=64, V=128, A_log=FAKE, dt_bias=FAKE, scale=0.1, l2_eps=1e-6)
    S = dict(pool=FAKE, num_slots=8, slot_stride=4 * 64 * 128, indices=FAKE, index_stride=1, null_slot=-1)
    A = dict(qkv=FAKE, ld_qkv=768, rg=FAKE, ld_g=4, rb=FAKE, ld_beta=4, n=3, T=4, cu=FAKE, rows=12, ws=FAKE, ws_bytes=1 << 20, out=FAKE, ld_out=512, err=FAKE)
    H.update(heads or {})
    S.update(state or {})
    A.update(change or {})
    hd, st = kda.KdaGdnHeads(**H), kda.KdaState(**S)
    ph = None if heads == {} else ctypes.byref(hd)
    ps = None if state == {} else ctypes.byref(st)
    head = (A["qkv"], A["ld_qkv"], A["rg"], A["ld_g"], A["rb"], A["ld_beta"])
    tail = (ph, ps, A["out"], A["ld_out"], A["err"], None)
    if name == "kda_gdn_decode":
        return kda.lib.kda_gdn_decode(*head, A["n"], *tail)
    if name == "kda_gdn_spec_verify":
        return kda.lib.kda_gdn_spec_verify(*head, A["n"], A["T"], *tail)
    return kda.lib.kda_gdn_chunk_prefill(*head, A["cu"], A["n"], A["rows"], *tail[:2], A["ws"], A["ws_bytes"], *tail[2:])


CALLS = ["kda_gdn_decode", "kda_gdn_spec_verify", "kda_gdn_chunk_prefill"]
BAD = [("heads", {}, 1), ("state", {}, 1),
       ("heads", dict(Hk=0), 1), ("heads", dict(Hk=3), 1), ("heads", dict(Hv=0), 1), ("heads", dict(K=96), 2), ("heads", dict(V=256), 2),
       ("heads", dict(A_log=None), 1), ("heads", dict(A_log=FAKE + 2), 1), ("heads", dict(dt_bias=FAKE + 2), 1),
       ("heads", dict(scale=float("inf")), 1), ("heads", dict(l2_eps=-1e-6), 1), ("heads", dict(l2_eps=float("nan")), 1),
       ("state", dict(pool=None), 1), ("state", dict(pool=FAKE + 8), 1), ("state", dict(indices=None), 1), ("state", dict(indices=FAKE + 2), 1),
       ("state", dict(num_slots=0), 1), ("state", dict(slot_stride=4 * 64 * 128 - 4), 1), ("state", dict(slot_stride=4 * 64 * 128 + 2), 1),
       ("state", dict(index_stride=0), 1), ("state", dict(null_slot=8), 1), ("state", dict(null_slot=-2), 1),
       ("change", dict(qkv=None), 1), ("change", dict(rg=None), 1), ("change", dict(rb=None), 1), ("change", dict(out=None), 1),
       ("change", dict(ld_qkv=767), 1), ("change", dict(ld_g=3), 1), ("change", dict(ld_beta=3), 1), ("change", dict(ld_out=508), 1),
       ("change", dict(ld_out=514), 1), ("change", dict(out=FAKE + 4), 1), ("change", dict(qkv=FAKE + 1), 1), ("change", dict(err=FAKE + 1), 1),
       ("change", dict(n=-1), 1), ("change", dict(n=2 ** 28), 2)]


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("what, bad, status", BAD)
def test_refusals(kda, name, what, bad, status):
    assert call(kda, name, **{what: bad}) == status
    assert kda.last_error()


def test_refusals_of_one_call(kda):
    for T in (0, -1, 65):
        assert call(kda, "kda_gdn_spec_verify", dict(T=T)) == 1
    for change, status in ((dict(cu=None), 1), (dict(cu=FAKE + 2), 1), (dict(rows=-1), 1), (dict(rows=2 ** 31 - 64), 2), 
                           (dict(ws=None), 3), (dict(ws=FAKE + 128), 3), (dict(ws_bytes=0), 3)):
        assert call(kda, "kda_gdn_chunk_prefill", change) == status


def test_workspace_bytes(kda):
    record = 4 * 5120 + (3 * 64 + 4) * 4        # T and W in two terms, blocks on and below the diagonal; the row factors
    n = kda.kda_gdn_chunk_prefill_workspace_bytes(130, 3, 4, 128, 64, num_k_heads=2)
    assert n >= (130 // 64 + 3) * 4 * record and n <= (130 // 64 + 3) * 4 * record + 3 * 256 and n % 16 == 0
    need = kda.kda_gdn_chunk_prefill_workspace_bytes(12, 3, 4, 64, 128, num_k_heads=2)
    assert call(kda, "kda_gdn_chunk_prefill", dict(ws_bytes=need - 1)) == 3
    assert kda.kda_gdn_chunk_prefill_workspace_bytes(130, 3, 4, 32, 64) == 0
    assert kda.kda_gdn_chunk_prefill_workspace_bytes(0, 3, 4, 64, 64) == 0
    for bad in ((-1, 3, 4, 64, 64), (2 ** 31 - 65, 1, 128, 64, 64), (8, -1, 4, 64, 64), (8, 3, 4, 96, 64), (8, 3, 0, 64, 64)):
        with pytest.raises(ValueError):
            kda.kda_gdn_chunk_prefill_workspace_bytes(*bad)


@pytest.mark.parametrize("name", CALLS)
def test_no_sequences_is_nothing_to_do(kda, name):
    assert call(kda, name, dict(n=0)) == 0 and kda.last_error() == ""


# ---- the binding's refusals ----------------------------------------------------------------


def tensors(**change):
    t = dict(mixed_qkv=torch.zeros(4, 768, dtype=torch.bfloat16), raw_g=torch.zeros(4, 4, dtype=torch.bfloat16),
             raw_beta=torch.zeros(4, 4, dtype=torch.bfloat16), A_log=torch.zeros(4), dt_bias=torch.zeros(4),
             initial_state=torch.zeros(8, 4, 64, 128), state_indices=torch.zeros(4, dtype=torch.int32))
    t.update(change)
    return tuple(t.values())


@pytest.mark.parametrize("change, match", [
    (dict(mixed_qkv=None), "mixed_qkv must be a tensor"),
    (dict(mixed_qkv=torch.zeros(4, 768)), "mixed_qkv must be BFloat16"),
    (dict(mixed_qkv=torch.zeros(4, 767, dtype=torch.bfloat16)), "mixed_qkv must have"),
    (dict(mixed_qkv=torch.zeros(768, 4, dtype=torch.bfloat16).t()), "unit inner stride"),
    (dict(initial_state=torch.zeros(8, 4, 64)), "initial_state must be fp32"),
    (dict(initial_state=torch.zeros(8, 4, 64, 128, dtype=torch.float64)), "initial_state must be fp32"),
    (dict(initial_state=torch.zeros(8, 4, 128, 64).transpose(2, 3)), "contiguous"),
    (dict(), "must be on the GPU")])
def test_binding_refusals(kda, change, match):
    with pytest.raises(ValueError, match=match):
        kda.kda_gdn_decode(*tensors(**change), num_k_heads=2)


def test_binding_refuses_counts(kda):
    with pytest.raises(ValueError, match="num_k_heads must divide"):
        kda.kda_gdn_decode(*tensors(), num_k_heads=3)
    with pytest.raises(ValueError, match="num_k_heads must divide"):
        kda.kda_gdn_decode(*tensors(), num_k_heads=0)
    with pytest.raises(ValueError, match="multiple of tokens_per_req"):
        kda.kda_gdn_spec_verify(*tensors(), 3, num_k_heads=2)
    with pytest.raises(ValueError, match="tokens_per_req"):
        kda.kda_gdn_spec_verify(*tensors(), 0, num_k_heads=2)
    with pytest.raises(ValueError, match="cu_seqlens"):
        kda.kda_gdn_chunk_prefill(*tensors(), None)
    with pytest.raises(ValueError, match="cu_seqlens"):
        kda.kda_gdn_chunk_prefill(*tensors(), torch.zeros(2, dtype=torch.int64))


@pytest.mark.parametrize("name", CALLS)
def test_refuses_columns_past_32_bits(kda, name):
    big = dict(ld_qkv=1 << 40, ld_g=1 << 24, ld_beta=1 << 24, ld_out=1 << 32, n=1, rows=1, T=1)
    state = dict(slot_stride=1 << 40)
    assert call(kda, name, big, dict(Hk=1 << 24, Hv=1 << 24), state) == 2
    assert "2^31" in kda.last_error()


def test_workspace_bytes_of_parts(kda):
    """One long sequence is cut into parts (two at 32 heads, eight at 4), whose ends, units and partial outputs follow the records."""
    record = 4 * 5120 + (3 * 64 + 4) * 4
    for rows, H, K, parts in ((16384, 32, 128, 2), (4097, 4, 64, 8), (4095, 4, 64, 1), (8192, 51, 64, 1)):
        more = H * (2 * parts - 1) * (K * K + K) * 4 + rows * (parts - 1) // parts * H * 2 * K * 4 if parts > 1 else 0
        n = kda.kda_gdn_chunk_prefill_workspace_bytes(rows, 1, H, K, K)
        least = (rows // 64 + 1) * (8 + H * record) + more
        assert least <= n <= least + 4 * 256
    assert kda.kda_gdn_chunk_prefill_workspace_bytes(16384, 1, 32, 128, 64) < (16384 // 64 + 1) * (8 + 32 * record) + 4 * 256   # K = V alone
