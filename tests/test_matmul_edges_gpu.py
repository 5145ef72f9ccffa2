"""GPU tests of the 16-bit product's large tiles at the edges of what they write, against 64-bit torch. Tolerances as in test_matmul_gpu.py."""
import pytest
import torch

from tests.test_matmul_gpu import ACT, BF16, FP16, FP32, check, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    assert torch.cuda.is_available()
    from linear_attention_state_recurrent_gb300 import build
    build.build()
    from linear_attention_state_recurrent_gb300 import kda as k
    return k


@pytest.mark.parametrize("N, out", [(320, BF16), (320, FP16), (288, FP32), (352, FP32), (64, BF16), (328, BF16), (300, FP32)])
@pytest.mark.parametrize("act, bias", [(None, False), ("relu", True)])
def test_odd_boxes_of_many_tiles(kda, N, out, act, bias):
    """A short inner axis, so that the epilogue is what a pair waits for; every pair has several tiles of an odd number of boxes, one after the other,
    and neither a residual nor time between their stores. Element by element, several times over."""
    g = torch.Generator(device="cuda").manual_seed(N)
    M, K = 33494, 256 if N > 64 else 64
    a, w = rows(M, K, BF16, g, 0), rows(N, K, BF16, g, 0, K ** -0.5)
    b = torch.randn(N, generator=g, device="cuda") if bias else None
    if N > 64:
        assert kda.kda_matmul_plan(a, w)[0] == 256
    first = None
    for _ in range(5):
        o = torch.full((M, N + -N % 8 + 8), 7.0, dtype=out, device="cuda")
        kda.kda_matmul(a, w, bias=b, activation=act, out=o[:, :N])
        assert (o[:, N:] == 7.0).all()
        if first is None:
            first = o
            check(o[:, :N], a, w, b, act)
        assert torch.equal(o, first)


@pytest.mark.parametrize("N, out, pad", [(320, BF16, 0), (288, FP32, 0), (353, FP16, 7), (329, FP32, 3)])
def test_odd_boxes_with_a_residual_in_place(kda, N, out, pad):
    """The boxes take turns across tiles where residuals come into them too, and where the last columns are stored by rows."""
    g = torch.Generator(device="cuda").manual_seed(N)
    a, w = rows(33494, 256, FP16, g, 0), rows(N, 256, FP16, g, 0, 1 / 16)
    assert kda.kda_matmul_plan(a, w)[0] == 256
    res = rows(33494, N, out, g, pad)
    for _ in range(3):
        o = torch.empty(33494, N + pad, dtype=out, device="cuda")[:, :N]
        o.copy_(res)
        kda.kda_matmul(a, w, residual=o, activation="relu", out=o)
        check(o, a, w, None, "relu", res)


@pytest.mark.parametrize("out_at, res_at", [((0, 0), (3, 0)), ((0, 0), (0, 1)), ((1, 0), (0, 0)), ((0, 1), (5, 1)), ((0, 0), None), ((7, 0), None)])
@pytest.mark.parametrize("M, N, K, out", [(2048, 8192, 16384, BF16), (2048, 8192, 16384, FP32), (8001, 600, 512, FP32), (1500, 1304, 4096, BF16)])
def test_outputs_and_residuals_on_boundaries_of_their_own(kda, M, N, K, out, out_at, res_at):
    """Either off 16-byte boundaries, both or none (how many elements longer than the columns rows are, and where the first begins): where pairs take such outputs as
    well (256 tiles of 256 steps of 270 ns each), and where smaller tiles take them."""
    g = torch.Generator(device="cuda").manual_seed(M)
    a, w = rows(M, K, BF16, g, 0), rows(N, K, BF16, g, 0, K ** -0.5)
    assert kda.kda_matmul_plan(a, w)[0] == 256
    o = rows(M, N, out, g, out_at[0], 1.0, out_at[1])
    res = None if res_at is None else rows(M, N, out, g, res_at[0], 1.0, res_at[1])
    kda.kda_matmul(a, w, residual=res, out=o)
    check(o, a, w, None, None, res)


@pytest.mark.parametrize("act", ["silu", "sigmoid", "gelu_tanh"])
@pytest.mark.parametrize("M", [5, 600])
def test_activations_far_below_zero(kda, act, M):
    """Results down to fp32's smallest normal value, each by itself: act(bias) of an inner axis of zeros, exact. An exponent of up to 90 takes its roundings
    90-fold (2^-24 each; gelu_tanh's has seven, constants and operations, the others' none), e^x and the quotient are off by two steps each, and e^-90 has lost digits: 15 half
    steps more. 7 * 90 + 8 + 15 half steps of 2^-24 at most."""
    x = torch.cat([torch.linspace(-12, 12, 500), torch.linspace(-90, 90, 1000), torch.tensor([-87.0, -87.4, -88.0, -88.6, -10.0, -10.05, 0.0])]).cuda()
    y = ACT[act](x.double()) if act != "gelu_tanh" else x.double() * torch.sigmoid((8 / torch.pi) ** 0.5 * (x.double() + 0.044715 * x.double() ** 3))
    x, y = x[y.abs() >= 2.0 ** -126], y[y.abs() >= 2.0 ** -126]
    a, w = torch.zeros(M, 64, dtype=BF16, device="cuda"), torch.zeros(len(x), 64, dtype=BF16, device="cuda")
    got = kda.kda_matmul(a, w, bias=x, activation=act, out_dtype=FP32).double()
    assert ((got - y).abs() <= 653 * 2.0 ** -24 * y.abs()).all(), ((got - y).abs() / y.abs()).max()
