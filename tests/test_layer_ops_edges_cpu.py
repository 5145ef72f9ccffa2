"""Host side of the operators around the recurrence beyond their own refusals: the plan's and the self-test's. No GPU: every call here
fails its checks before anything is launched."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch


@pytest.fixture(scope="module")
def kda():
    from linear_attention_state_recurrent_gb300 import build
    build.build()
    from linear_attention_state_recurrent_gb300 import kda as k
    return k


F = 1 << 20   # never dereferenced: validation fails before any launch


def _selftest(kda, **kw):
    a = dict(a=F, ld_a=128, sa=F, sar=1, sag=8, w=F, ld_w=128, sw=F, swr=1, swg=1, M=8, N=8, K=128, out=F, ld_out=8,
             dtype=0, stalled=0, err=F, stream=None)
    a.update(kw)
    return kda.lib.kda_selftest_fp8_matmul(*a.values())


@pytest.mark.parametrize("bad,word", [(dict(err=None), "err_flags"), (dict(stalled=-1), "stalled"), (dict(stalled=8), "stalled"),
                                      (dict(out=None), "out"), (dict(ld_a=127), "strides"), (dict(dtype=3), "out_dtype")])
def test_fp8_matmul_selftest_refuses(kda, bad, word):
    assert _selftest(kda, **bad) == 1
    assert word in kda.last_error()


def test_fp8_matmul_selftest_of_nothing_is_nothing(kda):
    assert _selftest(kda, M=0) == 0 and kda.last_error() == ""


def test_fp8_matmul_selftest_binding_refuses(kda):
    a, w, out = (torch.zeros(n, 128).to(torch.float8_e4m3fn) for n in (4, 8, 4))
    args = dict(a=a, a_scales=torch.ones(4, 1), w=w, w_scales=torch.ones(1, 1), out=torch.zeros(4, 8), err_flags=None)
    for bad in (dict(a=a[0]), dict(w=w.float()), dict(out=out), dict(stalled=8), dict()):   # the last: not on the GPU
        with pytest.raises(ValueError):
            kda.kda_selftest_fp8_matmul(**(args | bad))


def _plan(kda, **kw):
    a = dict(a=F, ld_a=128, w=F, ld_w=128, M=8, N=8, K=128, plan=(ctypes.c_int32 * 3)())
    a.update(kw)
    return kda.lib.kda_fp8_matmul_plan(*a.values())


@pytest.mark.parametrize("bad", [dict(plan=None), dict(M=0), dict(N=0), dict(K=-1), dict(M=(1 << 30) + 1), dict(ld_a=127), dict(ld_w=0)])
def test_fp8_matmul_plan_refuses(kda, bad):
    assert _plan(kda, **bad) == 1 and kda.last_error()


@pytest.mark.parametrize("off", [dict(a=F + 1), dict(w=F + 8), dict(ld_a=129), dict(ld_w=136), dict(K=0)])
def test_fp8_matmul_plan_of_what_the_tensor_cores_cannot_load(kda, off):
    plan = (ctypes.c_int32 * 3)()
    assert _plan(kda, plan=plan, **off) == 0 and list(plan) == [0, 1, 64]


def test_fp8_matmul_plan_binding(kda):
    e = torch.float8_e4m3fn
    a, w = torch.zeros(4, 129).to(e), torch.zeros(8, 129).to(e)
    assert kda.kda_fp8_matmul_plan(a, w) == (0, 1, 64)
    for bad in ((a[0], w), (a, w[:, :128])):
        with pytest.raises(ValueError):
            kda.kda_fp8_matmul_plan(*bad)


def test_what_a_device_answers_is_asked_again_after_a_failure(kda):
    """With no device to ask, each call gives CUDA's own reason, the second as the first: no failure is kept in place of an
    answer. In a process that sees no GPU, so nothing can be launched."""
    code = f"""
import sys; sys.path.insert(0, {os.path.dirname(os.path.dirname(os.path.abspath(__file__)))!r})
from linear_attention_state_recurrent_gb300 import kda
F = 1 << 20
for i in range(2):
    assert kda.lib.kda_norm_quant(F, 256, None, 0, 0, F, 1e-5, 4, 256, None, 0, None, 0, F, 256, F, 1, 4, None) == 4
    print(kda.last_error())
    assert kda.lib.kda_fp8_matmul(F, 128, F, 1, 8, F, 128, F, 1, 1, 8, 8, 128, F, 8, 0, None, None) == 4
    print(kda.last_error())
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, env=dict(os.environ, CUDA_VISIBLE_DEVICES=""))
    assert r.returncode == 0, r.stderr[-2000:]
    said = [line.split(": ", 1)[1] for line in r.stdout.splitlines()]
    assert len(said) == 4 and len(set(said)) == 1 and "configuration" not in said[0]
