"""A serving step of a KDA layer (examples/layer_step.py) against the same step with the three operators around
the recurrence written out in torch.

Tolerance: the operators' outputs differ from the plain ones by rounding alone. A projection's bf16 output is
off by at most one step (2^-8 relative, where fp32 sums on either side of a border are rounded apart),
an e4m3 value by at most one (2^-3 relative) where its quotient lies within 2^-16 of a border, which
is one in 2^12 or fewer. If every bf16 value were a step off, the step's output would be off by 2^-8 for each of the
three roundings on its way and twice that through the recurrence's normalisation: 2^-6 bounds the relative L2 error."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    from linear_attention_state_recurrent_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("layer_step", os.path.join(ROOT, "examples", "layer_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


class Plain:
    """The binding with the operators around the recurrence replaced by torch expressions."""

    def __init__(self, kda):
        self.kda = kda

    def __getattr__(self, name):
        return getattr(self.kda, name)

    @staticmethod
    def kda_norm_quant(x, weight=None, eps=1e-5, residual=None):
        h = x.double() if residual is None else x.double() + residual.double()
        y = h if weight is None else h / (h.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()
        n, d = y.shape
        s = y.view(n, d // 128, 128).abs().amax(-1).clamp_min(448 * 2.0 ** -126) / 448
        q = (y.view(n, d // 128, 128) / s[..., None]).clamp(-448, 448).float().to(torch.float8_e4m3fn).view(n, d)
        return q, s.float(), None if residual is None else h.to(x.dtype)

    @staticmethod
    def kda_fp8_matmul(a, a_scales, w, w_scales, out=None, err_flags=None):
        fa = a.double() * a_scales.double().repeat_interleave(128, 1)[:, :a.shape[1]]
        fw = w.double() * w_scales.double().repeat_interleave(128, 0)[:w.shape[0]].repeat_interleave(128, 1)[:, :w.shape[1]]
        y = (fa @ fw.t()).to(torch.bfloat16)
        return y if out is None else out.copy_(y)


@pytest.mark.parametrize("lens", [[1], [1] * 40, [1, 65, 1, 200, 1], [300]])
def test_layer_step_matches_the_plain_operators(example, lens):
    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")
    R, tokens = len(lens), sum(lens)
    layers = [example.KdaLayer(512, 2, 128, R + 2, seed=3) for _ in range(2)]
    layers[1].kda = Plain(layers[1].kda)
    g = torch.Generator().manual_seed(4)
    state = 0.05 * torch.randn(layers[0].state.shape, generator=g).cuda()
    x, residual = torch.randn(2, tokens, 512, generator=g).to(torch.bfloat16).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = torch.full((R, 32), -1, dtype=torch.int32, device="cuda")
    maps = layers[0].maps(i32(lens), i32([0] * R), torch.arange(R + 1, 0, -1, dtype=torch.int32, device="cuda")[:R], table,
                          torch.arange(256, dtype=torch.int32, device="cuda"), i32([256]), tokens, err)
    out = []
    for layer in layers:
        layer.state.copy_(state)
        out.append((*layer.step(x, residual, maps, lens, err), layer.state))
    torch.cuda.synchronize()
    assert err.item() == 0
    assert torch.equal(out[0][1], out[1][1])                       # the residual stream: one rounding of the same sum
    for a, b in zip(out[0], out[1]):
        assert torch.isfinite(a.float()).all()
        rel = ((a.double() - b.double()).norm() / b.double().norm()).item()
        assert rel <= 2.0 ** -6, rel


def test_the_example_runs(example, capsys):
    example.main()
    assert capsys.readouterr().out.count("errors 0") == 3
