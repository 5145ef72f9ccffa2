"""The 16-bit product on the host: every refusal of the C ABI and of the binding. No GPU: each call here fails its checks
before anything is launched."""
import pytest
import torch


@pytest.fixture(scope="module")
def kda():
    from linear_attention_state_recurrent_gb300 import build
    build.build()
    from linear_attention_state_recurrent_gb300 import kda as k
    return k


FAKE = 1 << 20   # never dereferenced


def call(kda, **change):
    A = dict(a=FAKE, ld_a=64, w=FAKE, ld_w=64, dtype=0, M=3, N=5, K=64, bias=FAKE, bias_dtype=0, act=0, res=FAKE, ld_res=5, out=FAKE, ld_out=5,
             out_dtype=0, err=FAKE)
    A.update(change)
    return kda.lib.kda_matmul(*A.values(), None)


@pytest.mark.parametrize("change, status", [
    (dict(dtype=2), 1), (dict(dtype=-1), 1), (dict(out_dtype=3), 1), (dict(bias_dtype=1), 1), (dict(dtype=1, bias_dtype=0), 1), (dict(act=-1), 1), (dict(act=6), 1),
    (dict(M=-1), 1), (dict(N=-1), 1), (dict(K=-1), 1), (dict(M=2 ** 30 + 1), 1), (dict(M=2 ** 30, N=2 ** 30, ld_out=2 ** 30, ld_res=2 ** 30), 2),
    (dict(out=None), 1), (dict(a=None), 1), (dict(w=None), 1), (dict(ld_a=63), 1), (dict(ld_w=63), 1), (dict(ld_out=4), 1), (dict(ld_res=4), 1),
    (dict(a=FAKE + 1), 1), (dict(w=FAKE + 1), 1), (dict(out=FAKE + 1), 1), (dict(out=FAKE + 2, out_dtype=2), 1), (dict(res=FAKE + 1), 1), (dict(bias=FAKE + 1), 1),
    (dict(bias=FAKE + 2, bias_dtype=2), 1), (dict(err=FAKE + 2), 1)])
def test_refusals(kda, change, status):
    assert call(kda, **change) == status
    assert kda.last_error()


@pytest.mark.parametrize("change", [dict(M=0), dict(N=0)])
def test_nothing_to_do(kda, change):
    assert call(kda, **change) == 0 and kda.last_error() == ""


def test_plan_refusals(kda):
    import ctypes
    plan = (ctypes.c_int32 * 2)()
    for bad in ((None, 64, None, 64, 0, 5, 64, plan), (None, 64, None, 64, 3, 5, -1, plan), (None, 63, None, 64, 3, 5, 64, plan), (None, 64, None, 64, 3, 5, 64, None)):
        assert kda.lib.kda_matmul_plan(*bad) == 1
    with pytest.raises(ValueError, match="same number of columns"):
        kda.kda_matmul_plan(torch.zeros(2, 3), torch.zeros(2, 4))


BF16 = torch.bfloat16


@pytest.mark.parametrize("a, w, kw, match", [
    (torch.zeros(2, 8), torch.zeros(3, 8), {}, "a must be bf16 or fp16"),
    (torch.zeros(8, dtype=BF16), torch.zeros(3, 8, dtype=BF16), dict(out=torch.zeros(2, 3)), "2-D"),
    (torch.zeros(8, 2, dtype=BF16).t(), torch.zeros(3, 8, dtype=BF16), {}, "unit inner stride"),
    (torch.zeros(2, 8, dtype=BF16), torch.zeros(3, 8, dtype=BF16), dict(activation="tanh"), "activation"),
    (torch.zeros(2, 8, dtype=BF16), torch.zeros(3, 8, dtype=BF16), dict(out_dtype=torch.float64), "out_dtype"),
    (torch.zeros(2, 8, dtype=BF16), torch.zeros(3, 8, dtype=BF16), {}, "must be on the GPU")])
def test_binding_refusals(kda, a, w, kw, match):
    with pytest.raises(ValueError, match=match):
        kda.kda_matmul(a, w, **kw)
