"""The example layer, end to end: prompts, tokens and training through the operators together."""
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
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decayed_attention.py")
    spec = importlib.util.spec_from_file_location("decayed_attention", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_tokens_continue_prompts(example):
    # bfloat16 at each of the bottleneck, projection, q and k, scores, x and state, out rows, and output: at most nine
    # half steps (2^-8 each) on either side
    assert example.serve(example.DecayedAttention()) < 18 * 2.0 ** -8


@pytest.mark.parametrize("D", [64, 128])
def test_gradients_against_differences(example, D):
    """The loss's change along the gradient is the gradient's norm: differences of the float32 weights of the norm, and
    of U and V over steps that bfloat16 resolves."""
    layer = example.DecayedAttention(Hq=4, Hkv=2, D=D)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(2, 300, 512, device="cuda", generator=g).bfloat16()
    at = torch.arange(300, device="cuda").expand(2, -1)
    out, saved = layer.forward(x, at)
    go = torch.randn(*out.shape, device="cuda", generator=g).bfloat16()
    grads = layer.backward(saved, go)
    loss = lambda: float((layer.forward(x, at)[0].double() * go.double()).sum())  # noqa: E731
    for i, name in enumerate(("V", "U", "q_weight", "k_weight", "out_weight")):
        p, d = getattr(layer, name), grads[i].float()
        way = d / d.norm() * p.float().norm() * 0.02
        kept = p.clone()
        p.copy_(kept.float() + way)
        moved = p.float().clone()
        up = loss()
        p.copy_(kept.float() - way)
        moved = moved - p.float()
        down = loss()
        p.copy_(kept)
        want = float((d.double() * moved.double()).sum())
        # second order cancels; rounding of 600 x 512 outputs (each 2^-8 relative at worst, independent) and of the
        # gradients stays below a tenth of a change by a fiftieth along the gradient
        assert abs((up - down) - want) < 0.1 * abs(want), (name, up - down, want)


def test_training_lowers_the_loss(example):
    losses = example.train(example.DecayedAttention())
    assert losses[-1] < 0.7 * losses[0], losses
