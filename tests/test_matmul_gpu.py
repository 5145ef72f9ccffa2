"""GPU tests of the 16-bit product against 64-bit torch.

Tolerance, from the arithmetic (e is half a step of the output's type, S the sum of the magnitudes of the products): 16-bit products are
exact in fp32; an MMA step adds 16 of them to the sum, each addition off by at most a step (2^-23, a truncating adder) of what is added up:
(K / 16 + 20) 2^-23 S, the 20 for the 16 within a step and a split's join. The activations' slopes are at most 1.13, and their own error is within 64 steps of
2^-24 of the result: e^x for |x| < 20, beyond which the result does not depend on it, takes its argument's rounding 20-fold. Bias and
residual are added in fp32: 2^-23 of the values. One rounding at the end.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def kda():
    assert torch.cuda.is_available()
    from linear_attention_state_recurrent_gb300 import build
    build.build()
    from linear_attention_state_recurrent_gb300 import kda as k
    return k


def rows(m, k, dtype, gen, pad, scale=1.0, skip=0):
    """[m, k] normal values in a buffer whose rows are `pad` elements longer (NaN there), `skip` elements into it."""
    t = torch.full((m * (k + pad) + skip,), math.nan, dtype=dtype, device="cuda")
    t = t[skip:].view(m, k + pad)
    t[:, :k] = (torch.randn(m, k, generator=gen, device="cuda") * scale).to(dtype)
    return t[:, :k]


ACT = {None: lambda x: x, "relu": torch.relu, "silu": lambda x: x * torch.sigmoid(x), "sigmoid": torch.sigmoid,
       "gelu": lambda x: x * torch.special.ndtr(x), "gelu_tanh": lambda x: 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))}


def check(got, a, w, bias=None, act=None, residual=None):
    e = torch.finfo(got.dtype).eps / 2
    K = a.shape[1]
    x = a.double() @ w.double().t()
    S = a.double().abs() @ w.double().abs().t()
    off = (K / 16 + 20) * 2.0 ** -23 * S
    if bias is not None:
        x = x + bias.double()
        off = off + 2.0 ** -23 * x.abs()
    y = ACT[act](x)
    off = 1.13 * off + (64 * 2.0 ** -24 * y.abs() if act not in (None, "relu") else 0.0)
    if residual is not None:
        y = y + residual.double()
        off = off + 2.0 ** -23 * y.abs()
    worst = ((got.double() - y).abs() - off - e * y.abs() - (2.0 ** -24 if got.dtype == FP16 else 0.0))
    assert worst.max().item() <= 0, worst.max().item()


# every arrangement, with sides that its tiles do not divide
SIZES = [(1, 1, 1), (1, 300, 64), (3, 64, 72), (7, 130, 4096), (16, 128, 200), (17, 500, 1000), (32, 129, 64), (33, 256, 136), (64, 1000, 512), (65, 200, 1024), (128, 640, 328),
         (129, 257, 72), (200, 4000, 64), (300, 77, 2048), (513, 1024, 264), (777, 1111, 1304), (2000, 2500, 520)]


@pytest.mark.parametrize("M, N, K", SIZES)
@pytest.mark.parametrize("dtype, out", [(BF16, BF16), (FP16, FP32), (BF16, FP16)])
def test_sizes(kda, M, N, K, dtype, out):
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    a, w = rows(M, K, dtype, g, -K % 8 + 8), rows(N, K, dtype, g, -K % 8, K ** -0.5)
    bias = torch.randn(N, generator=g, device="cuda").to(dtype)
    res = rows(M, N, out, g, -N % 8 + 8)
    o = torch.full((M, N + 8 + -N % 8), 7.0, dtype=out, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert kda.kda_matmul(a, w, bias=bias, activation="silu", residual=res, out=o[:, :N], err_flags=err).data_ptr() == o.data_ptr()
    check(o[:, :N], a, w, bias, "silu", res)
    assert err.item() == 0 and (o[:, N:] == 7.0).all()
    plain = kda.kda_matmul(a, w, out_dtype=out)
    check(plain, a, w)
    assert torch.equal(plain, kda.kda_matmul(a, w, out_dtype=out))            # the same bits again


def test_every_arrangement_is_reached(kda):
    plans = set()
    for M, N, K in SIZES + [(128, 12288, 4096), (1, 4096, 4096), (4096, 4096, 4096)]:
        a, w = torch.empty(M, K + -K % 8, dtype=BF16, device="cuda")[:, :K], torch.empty(N, K + -K % 8, dtype=BF16, device="cuda")[:, :K]
        r, split = kda.kda_matmul_plan(a, w)
        plans.add((r, split > 1))
    assert {r for r, _ in plans} >= {16, 32, 64, 128, 256} and any(s for _, s in plans)
    loose = torch.empty(100, 101, dtype=BF16, device="cuda")
    assert kda.kda_matmul_plan(loose, loose)[0] == 0


@pytest.mark.parametrize("act", list(ACT))
@pytest.mark.parametrize("M, K", [(5, 64), (600, 128)])
def test_activations(kda, act, M, K):
    g = torch.Generator(device="cuda").manual_seed(3)
    a, w = rows(M, K, BF16, g, 0, 4.0), rows(700, K, BF16, g, 0, K ** -0.5)   # values to about +-20
    bias = torch.randn(700, generator=g, device="cuda")
    check(kda.kda_matmul(a, w, bias=bias, activation=act, out_dtype=FP32), a, w, bias, act)


@pytest.mark.parametrize("M, N", [(4, 256), (700, 600)])
@pytest.mark.parametrize("out", [BF16, FP32])
def test_residual_in_place_and_what_has_no_bounds(kda, M, N, out):
    g = torch.Generator(device="cuda").manual_seed(4)
    a, w = rows(M, 96, FP16, g, 0), rows(N, 96, FP16, g, 0, 0.1)
    res = rows(M, N, out, g, 0)
    want = res.clone()
    check(kda.kda_matmul(a, w, residual=res, out=res), a, w, residual=want)
    # infinities and NaN stay where they are; large values on both sides of the activations' range
    a[0] = math.inf
    a[1] = math.nan
    a[2], w[3] = 60000.0, -1.0
    for act in ACT:
        y = kda.kda_matmul(a, w, activation=act, out_dtype=FP32)
        x = ACT[act]((a.float() @ w.float().t()).double())
        assert torch.equal(torch.isnan(y[2:]), torch.isnan(x[2:].float())) and torch.isnan(y[1]).all() and torch.isfinite(y[3:]).all()


@pytest.mark.parametrize("M, N, K", [(1, 40, 33), (5, 130, 1301), (70, 129, 77), (300, 515, 129)])
@pytest.mark.parametrize("skip", [0, 1])
def test_operands_off_16_byte_boundaries(kda, M, N, K, skip):
    g = torch.Generator(device="cuda").manual_seed(5)
    a, w = rows(M, K, BF16, g, 2, 1.0, skip), rows(N, K, BF16, g, 0, K ** -0.5, 1)
    assert kda.kda_matmul_plan(a, w)[0] == 0
    res = rows(M, N, FP32, g, 3)
    check(kda.kda_matmul(a, w, residual=res, activation="gelu", out_dtype=FP32), a, w, None, "gelu", res)


@pytest.mark.parametrize("N, pad, skip", [(600, 1, 0), (600, 0, 1), (601, 0, 0), (603, 5, 0), (520, 8, 0)])
@pytest.mark.parametrize("out", [BF16, FP32])
def test_outputs_off_16_byte_boundaries(kda, N, pad, skip, out):
    g = torch.Generator(device="cuda").manual_seed(6)
    M = 8001
    a, w = rows(M, 512, BF16, g, 0), rows(N, 512, BF16, g, 0, 0.05)
    assert kda.kda_matmul_plan(a, w)[0] == 256
    o, res = rows(M, N, out, g, pad, 1.0, skip), rows(M, N, out, g, 3)
    bias = torch.randn(N, generator=g, device="cuda")
    whole = torch.as_strided(o, (M, N + pad), (N + pad, 1), skip)
    kda.kda_matmul(a, w, bias=bias, residual=res, out=o)
    check(o, a, w, bias, None, res)
    assert torch.isnan(whole[:, N:]).all()                                    # behind the rows


@pytest.mark.parametrize("change, match", [(dict(w=FP16), "w must be BFloat16"), (dict(cols=7), "w must be"), (dict(bias=FP16), "bias must be BFloat16"),
                                           (dict(entries=4), "bias must"), (dict(res=BF16), "residual must be Float"), (dict(out=torch.float64), "out must be bf16")])
def test_refusals(kda, change, match):
    a, w = torch.zeros(2, 8, dtype=BF16, device="cuda"), torch.zeros(3, change.get("cols", 8), dtype=change.get("w", BF16), device="cuda")
    bias = torch.zeros(change.get("entries", 3), dtype=change.get("bias", FP32), device="cuda")
    res = torch.zeros(2, 3, dtype=change.get("res", FP32), device="cuda")
    with pytest.raises(ValueError, match=match):
        kda.kda_matmul(a, w, bias=bias, residual=res, out=torch.zeros(2, 3, dtype=change.get("out", FP32), device="cuda"))


def test_no_inner_axis_and_no_rows(kda):
    bias, res = torch.randn(50, device="cuda"), torch.randn(300, 50, device="cuda")
    a, w = torch.empty(300, 0, dtype=BF16, device="cuda"), torch.empty(50, 0, dtype=BF16, device="cuda")
    y = kda.kda_matmul(a, w, bias=bias, activation="relu", residual=res, out_dtype=FP32)
    assert torch.equal(y, torch.relu(bias) + res)
    assert kda.kda_matmul(torch.empty(0, 8, dtype=BF16, device="cuda"), torch.empty(5, 8, dtype=BF16, device="cuda")).shape == (0, 5)


@pytest.mark.parametrize("M", [4, 300])
def test_offsets_past_32_bits(kda, M):
    """Rows of a and of out whose offsets pass 2^31 elements."""
    pitch = (1 << 31) // M + 4096 & ~7
    g = torch.Generator(device="cuda").manual_seed(7)
    big = torch.empty(M * pitch, dtype=BF16, device="cuda").view(M, pitch)
    a, w = rows(M, 64, BF16, g, 0), rows(300, 64, BF16, g, 0)
    big[:, :64] = a
    o = big[:, 64:364]
    kda.kda_matmul(big[:, :64], w, out=o)
    check(o, a, w)


def test_stream_and_graph(kda):
    g = torch.Generator(device="cuda").manual_seed(8)
    a, w = rows(40, 256, BF16, g, 0), rows(512, 256, BF16, g, 0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o = kda.kda_matmul(a, w, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    check(o, a, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_matmul(a, w, out=o, activation="relu")
    a.copy_(torch.randn(40, 256, generator=g, device="cuda"))
    graph.replay()
    check(o, a, w, None, "relu")
