"""The example layer of selective scan, end to end: prompts, tokens and gradients through the operators together."""
import importlib.util
import os

import pytest
import torch

from efficient_transformer_gb300 import build as la_build
from efficient_transformer_gb300 import la

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    la_build.build()
    la.load()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "selective_scan.py")
    spec = importlib.util.spec_from_file_location("selective_scan", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("S,G", [(16, 1), (8, 2), (32, 1)])
def test_tokens_continue_prompts(example, S, G):
    # The same operators on the same bfloat16 rows: each side rounds x and z, the convolution, bottleneck, dt, B and C, the
    # scan's rows and the output to bfloat16, half a step (2^-8) each at most: eight on either side, where the products are
    # summed in another order
    assert example.serve(example.SelectiveScan(S=S, G=G)) < 16 * 2.0 ** -8


@pytest.mark.parametrize("S,G", [(16, 1), (8, 4)])
def test_gradients_against_differences(example, S, G):
    """The loss's change along the gradient is the gradient's norm, over steps that bfloat16 resolves."""
    layer = example.SelectiveScan(S=S, G=G)
    g = torch.Generator(device="cuda").manual_seed(4)
    u = torch.randn(2, 300, 256, device="cuda", generator=g).bfloat16()
    out, saved = layer.forward(u, train=True)
    go = torch.randn(*out.shape, device="cuda", generator=g).bfloat16()
    grads = layer.backward(saved, go)
    loss = lambda: float((layer.forward(u)[0].double() * go.double()).sum())  # noqa: E731
    for i, (p, d) in enumerate(zip(layer.params(), grads)):
        assert d.shape == p.shape and bool(torch.isfinite(d.float()).all())
        d = d.float()
        way = d / d.norm() * p.float().norm() * 0.02
        if p is layer.A_log:
            # (a fiftieth of the norm of all the logarithms, on the few that matter most, would be a factor of exp(4): no longer
            # a straight line; they are moved by up to 0.2)
            way = d / d.abs().max() * 0.2
        kept = p.clone()
        p.copy_(kept.float() + way)
        moved = p.float().clone()
        up = loss()
        p.copy_(kept.float() - way)
        moved = moved - p.float()
        down = loss()
        p.copy_(kept)
        want = float((d.double() * moved.double()).sum())
        # second order cancels; the roundings of 600 x 256 outputs and of the rows before them (2^-8 relative at worst, independent)
        # and of the gradients stay below a tenth of a change by a fiftieth along the gradient
        assert abs((up - down) - want) < 0.1 * abs(want), (i, up - down, want)


def test_example_runs(example):
    losses = example.train(example.SelectiveScan(), steps=4)
    assert len(losses) == 4 and all(x == x for x in losses)
    example.main()


def test_a_training_step_captured_beside_an_eager_one(example):
    """Forward and gradients in one graph, replayed, while the tensors of an eager step live: the eager bits."""
    layer = example.SelectiveScan()
    g = torch.Generator(device="cuda").manual_seed(5)
    u = torch.randn(2, 130, 256, device="cuda", generator=g).bfloat16()
    go = torch.randn(2, 130, 256, device="cuda", generator=g).bfloat16()

    def one():
        y, saved = layer.forward(u, train=True)
        return (y,) + layer.backward(saved, go)

    want = one()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        one()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = one()
    for _ in range(2):
        graph.replay()
    la.get_status()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
