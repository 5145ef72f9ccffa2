"""The operators around the recurrence on the host: pins of their fp64 oracle and every refusal of
the C ABI and of the binding. No GPU: each call here fails its checks before anything is launched."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import layer_ops as lo


@pytest.fixture(scope="module")
def kda():
    from linear_attention_state_recurrent_gb300 import build
    build.build()
    from linear_attention_state_recurrent_gb300 import kda as k
    return k


# ---- the oracle ---------------------------------------------------------------------------


def test_e4m3_table_matches_torch():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).to(torch.float64).numpy()
    np.testing.assert_array_equal(lo.E4M3_TABLE, t)
    assert lo.e4m3_value(0x7E) == 448.0 and lo.e4m3_value(1) == 2.0 ** -9


def test_norm_quant_by_hand():
    # h = (3, -4): mean square 12.5; the largest of the group becomes 448
    h, y, s, v = lo.norm_quant([[1.0, -5.0]], [[2.0, 1.0]], [1.0, 2.0], 0.0)
    np.testing.assert_allclose(h, [[3, -4]])
    np.testing.assert_allclose(y, [[3 / math.sqrt(12.5), -8 / math.sqrt(12.5)]])
    np.testing.assert_allclose(v, [[168.0, -448.0]])
    np.testing.assert_allclose(s, [[8 / math.sqrt(12.5) / 448]])


def test_norm_quant_groups_and_zero_rows():
    x = np.zeros((2, 300))
    x[1, 0], x[1, 130], x[1, 299] = 1.0, 2.0, -4.0
    _, _, s, v = lo.norm_quant(x, None, None, 0.0)
    assert s.shape == (2, 3) and np.all(s[0] == 2.0 ** -126) and np.all(v[0] == 0)
    np.testing.assert_array_equal(s[1] * 448, [1, 2, 4])
    np.testing.assert_array_equal(v[1, [0, 130, 299]], [448, 448, -448])


def test_fp8_matmul_by_hand():
    a, w = np.ones((1, 129)), np.ones((129, 129))
    out, mag = lo.fp8_matmul(a, [[2.0, 3.0]], w, [[1.0, 10.0], [0.5, 100.0]])
    assert out[0, 0] == 128 * 2 + 30 and out[0, 128] == 128 * 1 + 300
    np.testing.assert_array_equal(out, mag)


def test_batch_maps_by_hand():
    # pages of 4; request 0 prefills 5 tokens, 1 decodes at position 4 (a new page), 2 is idle
    table = np.array([[-1, -1], [9, -1], [7, -1]], np.int32)
    m, err = lo.batch_maps([5, 1, 0], [0, 4, 3], [10, 11, 12], table, [1, 2, 3, 4], 4, 4, 16, 8)
    assert err == 0
    assert m["order"].tolist() == [1, 0, 2] and m["cu_seqlens"].tolist() == [0, 1, 6, 6]
    assert m["state_indices"].tolist() == [11, 10, 12] and m["num_decodes"].tolist() == [1]
    assert m["block_table"].tolist() == [[4, 3], [9, 2], [7, -1]] and m["free_left"].tolist() == [1]
    assert m["positions"].tolist() == [4, 0, 1, 2, 3, 4, 0, 0]
    assert m["slot_map"].tolist() == [8, 16, 17, 18, 19, 12, -1, -1]


# ---- refusals of the C ABI ----------------------------------------------------------------

F = 1 << 20   # never dereferenced: validation fails before any launch


def _norm(kda, **kw):
    a = dict(x=F, ld_x=256, residual=None, ld_residual=0, dtype=0, weight=F, eps=1e-5, N=4, D=256, residual_out=None,
             ld_residual_out=0, y=None, ld_y=0, q=F, ld_q=256, scales=F, sr=1, sg=4, stream=None)
    a.update(kw)
    return kda.lib.kda_norm_quant(*a.values())


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=3), 1), (dict(dtype=-1), 1), (dict(N=-1), 1), (dict(D=0), 1), (dict(D=32769, ld_x=40000, ld_q=40000), 2),
    (dict(N=1 << 31), 2), (dict(x=None), 1), (dict(q=None), 1), (dict(scales=None), 1),
    (dict(residual=F, ld_residual=256), 1), (dict(residual_out=F, ld_residual_out=256), 1),
    (dict(residual=F, ld_residual=255, residual_out=F, ld_residual_out=256), 1),
    (dict(residual=F, ld_residual=256, residual_out=F, ld_residual_out=255), 1),
    (dict(eps=-1.0), 1), (dict(eps=math.inf), 1), (dict(eps=math.nan), 1), (dict(ld_x=255), 1), (dict(ld_q=255), 1),
    (dict(y=F, ld_y=100), 1), (dict(sr=0), 1), (dict(sg=-4), 1), (dict(x=F + 1), 1), (dict(weight=F + 2), 1),
    (dict(x=F + 2, dtype=2), 1), (dict(scales=F + 1), 1)])
def test_norm_quant_refuses(kda, bad, status):
    assert _norm(kda, **bad) == status
    assert kda.last_error()


def test_norm_quant_of_no_rows_is_nothing(kda):
    assert _norm(kda, N=0) == 0 and kda.last_error() == ""


def _matmul(kda, **kw):
    a = dict(a=F, ld_a=128, sa=F, sar=1, sag=8, w=F, ld_w=128, sw=F, swr=1, swg=1, M=8, N=8, K=128, out=F, ld_out=8,
             dtype=0, err=None, stream=None)
    a.update(kw)
    return kda.lib.kda_fp8_matmul(*a.values())


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=3), 1), (dict(M=-1), 1), (dict(N=-1), 1), (dict(K=-1), 1), (dict(M=1 << 31), 1), (dict(N=1 << 31), 1),
    (dict(K=1 << 31, ld_a=1 << 32, ld_w=1 << 32), 1), (dict(a=None), 1), (dict(w=None), 1), (dict(sa=None), 1),
    (dict(sw=None), 1), (dict(out=None), 1), (dict(ld_a=127), 1), (dict(ld_w=0), 1), (dict(ld_out=7), 1),
    (dict(sar=0), 1), (dict(sag=0), 1), (dict(swr=-1), 1), (dict(swg=0), 1), (dict(out=F + 1), 1),
    (dict(out=F + 2, dtype=2), 1), (dict(sa=F + 2), 1), (dict(sw=F + 1), 1), (dict(err=F + 1), 1)])
def test_fp8_matmul_refuses(kda, bad, status):
    assert _matmul(kda, **bad) == status
    assert kda.last_error()


@pytest.mark.parametrize("none", [dict(M=0), dict(N=0, ld_out=0)])
def test_fp8_matmul_of_nothing_is_nothing(kda, none):
    assert _matmul(kda, **none) == 0 and kda.last_error() == ""


def _maps(kda, **kw):
    a = dict(q=F, c=F, slots=F, ss=1, R=4, table=F, ts=8, width=8, free=F, nf=16, fc=F, np=64, page=16, nt=4,
             order=F, cu=F, si=F, nd=F, pos=F, slot_map=F, left=F + 64, err=None, stream=None)
    a.update(kw)
    return kda.lib.kda_batch_maps(*a.values())


@pytest.mark.parametrize("bad,status", [
    (dict(R=-1), 1), (dict(nt=-1), 1), (dict(nf=-1), 1), (dict(np=-1), 1), (dict(width=-1), 1), (dict(R=(1 << 24) + 1), 2),
    (dict(nt=1 << 31), 2), (dict(nf=1 << 31), 1), (dict(np=1 << 31), 1), (dict(page=0), 1), (dict(page=-16), 1),
    (dict(q=None), 1), (dict(c=None), 1), (dict(slots=None), 1), (dict(table=None), 1), (dict(ts=7), 1), (dict(free=None), 1),
    (dict(fc=None), 1), (dict(order=None), 1), (dict(cu=None), 1), (dict(si=None), 1), (dict(nd=None), 1),
    (dict(pos=None), 1), (dict(slot_map=None), 1), (dict(left=None), 1), (dict(ss=0), 1), (dict(left=F), 1),
    (dict(slot_map=F + 4), 1), (dict(q=F + 1), 1), (dict(err=F + 2), 1)])
def test_batch_maps_refuses(kda, bad, status):
    assert _maps(kda, **bad) == status
    assert kda.last_error()


# ---- refusals of the binding --------------------------------------------------------------


def test_norm_quant_binding_refuses(kda):
    x, q = torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(4, 256, dtype=torch.float8_e4m3fn)
    w, s = torch.ones(256), torch.zeros(4, 2)
    for bad in (dict(x=x.double()), dict(x=x[0]), dict(weight=w.bfloat16()), dict(weight=w[:255]), dict(weight=torch.ones(512)[::2]),
                dict(residual=x.float()), dict(residual=x[:3]), dict(residual_out=x), dict(residual=x, residual_out=x[:, :255]),
                dict(q=x), dict(q=q[:2]), dict(q=q.t().contiguous().t()), dict(scales=s[:, :1]), dict(scales=s.double()),
                dict(y=x.float()), dict()):   # the last: all in order but not on the GPU
        a = dict(x=x, weight=w, q=q, scales=s) | bad
        with pytest.raises(ValueError):
            kda.kda_norm_quant(a.pop("x"), a.pop("weight"), **a)


def test_fp8_matmul_binding_refuses(kda):
    e = torch.float8_e4m3fn
    a, w, sa, sw = torch.zeros(4, 256).to(e), torch.zeros(130, 256).to(e), torch.ones(4, 2), torch.ones(2, 2)
    for bad in (dict(a=a[0]), dict(a=a[:, :255]), dict(a=a.float()), dict(w=w.view(torch.uint8)), dict(sa=sa[:3]), dict(sa=sa[:, :1]),
                dict(sw=torch.ones(1, 2)), dict(sw=sw.double()), dict(out=torch.zeros(4, 129)), dict(out=torch.zeros(4, 130).double()),
                dict(out=torch.zeros(130, 4).t()), dict(out_dtype=torch.float64), dict()):
        b = dict(a=a, sa=sa, w=w, sw=sw) | bad
        with pytest.raises(ValueError):
            kda.kda_fp8_matmul(b.pop("a"), b.pop("sa"), b.pop("w"), b.pop("sw"), **b)


def test_batch_maps_binding_refuses(kda):
    def i32(*shape):
        return torch.zeros(*shape, dtype=torch.int32)
    good = dict(query_lens=i32(4), context_lens=i32(4), state_slots=i32(4), block_table=i32(4, 8), free_pages=i32(9),
                free_count=i32(1), page_size=16, num_pages=64, num_tokens=16)
    out = kda.make_batch_maps(4, 16, "cpu")
    for bad in (dict(query_lens=torch.zeros(4)), dict(context_lens=i32(3)), dict(state_slots=i32(2, 2)), dict(state_slots=i32(3)),
                dict(block_table=i32(3, 8)), dict(block_table=i32(8, 4).t()), dict(free_pages=torch.zeros(9)), dict(free_count=i32(0)),
                dict(num_tokens=None), dict(out=out, num_tokens=15), dict(out=out._replace(slot_map=i32(16))),
                dict(out=out._replace(cu_seqlens=i32(4))), dict()):
        with pytest.raises(ValueError):
            kda.kda_batch_maps(**(good | bad))


def test_status_of_a_refusal_reaches_the_caller(kda):
    assert _maps(kda, page=0) == 1
    assert "page_size" in ctypes.cast(kda.lib.kda_last_error(), ctypes.c_char_p).value.decode()


def test_fp8_matmul_refuses_what_one_launch_cannot_cover(kda):
    side = 1 << 30
    assert _matmul(kda, M=side, N=side, ld_out=side) == 2 and "split" in kda.last_error()
    assert _matmul(kda, M=side + 1) == 1
