"""A serving step of a layer with the gated delta rule (examples/gdn_layer_step.py) against the same step in 64-bit torch and the
fp64 oracle, eager and captured.

Tolerance: every tensor between two steps is rounded to bf16 (half a step: 2^-8 of a value, 2^-8 / 3^(1/2) in the mean), on both sides from
values that differ by little more, so it may be a step (2^-7) off where the sides round apart. On a way through the layer are five
of them (the projections, the recurrence's output, the gated output and the result), in quadrature 5^(1/2) 2^-7 / 3 = 5.8e-3 of the
norm, and twice that through the recurrence's normalisation: 1.2e-2."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import gdn as og

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    from linear_attention_state_recurrent_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("gdn_layer_step", os.path.join(ROOT, "examples", "gdn_layer_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def bf(x):
    return x.to(torch.bfloat16).double()


def plain_step(layer, x, residual, bounds, slots, state):
    """The new residual and state, in fp64 but for the roundings of what lies between the calls."""
    x = x.double()
    silu = lambda t: t * torch.sigmoid(t)  # noqa: E731
    qkv, ab = bf(silu(x @ layer.w_qkv.double().t())), bf(x @ layer.w_ab.double().t())
    gate = bf(torch.sigmoid(x @ layer.w_gate.double().t() + layer.gate_bias.double()))
    n = lambda t: t.double().cpu().numpy()  # noqa: E731
    o, after, err = og.run(n(qkv), n(ab[:, :layer.Hv]), n(ab[:, layer.Hv:2 * layer.Hv]), n(layer.A_log), n(layer.dt_bias), n(state), slots, bounds, layer.Hk)
    assert err == 0
    o = bf(torch.from_numpy(np.nan_to_num(o)).cuda())
    return bf(o * gate) @ layer.w_out.double().t() + residual.double(), torch.from_numpy(after).cuda()


def close(a, b):
    assert torch.isfinite(a.float()).all()
    rel = ((a.double() - b).norm() / b.norm()).item()
    assert rel <= 1.2e-2, rel


@pytest.mark.parametrize("lens", [[1], [1] * 9, [65, 1, 200], [64, 0, 3]])
def test_layer_step(example, lens):
    layer = example.GdnLayer(256, 2, 4, 64, len(lens) + 2, seed=3)
    g = torch.Generator().manual_seed(4)
    layer.state.copy_(0.05 * torch.randn(layer.state.shape, generator=g))
    rows = sum(lens)
    x, residual = torch.randn(2, rows, 256, generator=g).to(torch.bfloat16).cuda()
    slots = list(range(len(lens) + 1, 1, -1))
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    want, after = plain_step(layer, x, residual, list(zip(cu, cu[1:])), slots, layer.state)
    before, start = layer.state.clone(), layer.state.clone()
    index, cu_gpu = torch.tensor(slots, dtype=torch.int32, device="cuda"), torch.tensor(cu, dtype=torch.int32, device="cuda")
    ways = [False] + [True] * (lens == [1] * len(lens))
    for decode in ways:
        layer.state.copy_(start)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        y = layer.step(x, residual, cu_gpu, index, decode=decode, err_flags=err)
        assert err.item() == 0
        close(y, want)
        close(layer.state, after)
        assert torch.equal(layer.state[:2], before[:2])


def test_one_graph_for_other_lengths(example):
    """The captured step, replayed for other lengths and rows, gives what the eager step gives, bit for bit."""
    layer, eager = (example.GdnLayer(256, 1, 2, 128, 6, seed=5) for _ in range(2))
    rows = 200
    x, residual = torch.zeros(2, rows, 256, dtype=torch.bfloat16, device="cuda")
    cu, slots = torch.zeros(5, dtype=torch.int32, device="cuda"), torch.tensor([4, 2, 0, 5], dtype=torch.int32, device="cuda")
    layer.step(x, residual, cu, slots)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.step(x, residual, cu, slots)
    g = torch.Generator().manual_seed(6)
    for lens in ([70, 1, 100, 0], [0, 0, 0, 0], [1, 1, 1, 1], [3, 64, 65, 60]):
        n = sum(lens)
        x.copy_(torch.randn(rows, 256, generator=g))
        residual.copy_(torch.randn(rows, 256, generator=g))
        cu.copy_(torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32))
        graph.replay()
        want = eager.step(x, residual, cu, slots)
        assert torch.equal(y[:n], want[:n]) and torch.equal(layer.state, eager.state)


def test_the_example_runs(example, capsys):
    example.main()
    assert capsys.readouterr().out.count("errors 0") == 3
