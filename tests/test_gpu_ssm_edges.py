"""Selective scan and short convolution where something beside the values that are asked for could get into them: channels that
fill no block, sums over several blocks, NaN and infinities, states that grow."""
import pytest
import torch

from efficient_transformer_gb300 import build as la_build
from efficient_transformer_gb300 import la
from test_gpu_ssm import BF, F, FWD, compare, inputs, run_scan, want_scan

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    la_build.build()
    la.load()


# ---- places of a block that hold no channel ----------------------------------------------------------
# (a warp of the gradient has 16, 8, 4 or 2 channels at a time for 8, 16, 32 or 64 states, a block 64, 32, 16 or 16: 24 channels a
# group leave some places empty)

@pytest.mark.parametrize("G", [1, 2])
@pytest.mark.parametrize("S", [8, 16, 32, 64])
def test_steps_offset_by_the_bias(S, G):
    """dt in [2, 3] with a bias of -1.5: every step is positive, every decay below 1; the bias alone, as a step, would be a
    decay of exp(96)."""
    a = inputs(1, 21, 24 * G, S, G, dtype=F, seed=60 + S)
    a["A"] = -torch.linspace(1, 64, S, device="cuda").repeat(24 * G, 1)
    a["dt"], a["dt_bias"] = 2 + a["dt"].sigmoid(), torch.full((24 * G,), -1.5, device="cuda")
    compare(run_scan(a, softplus=False), want_scan(a, softplus=False), F)


@pytest.mark.parametrize("S", [8, 16, 32, 64])
def test_growing_states_of_few_channels(S):
    """A = 3 and steps of softplus(-2): states grow by exp(0.38) a token; the bias alone, as a step, would be a decay of exp(90)."""
    a = inputs(1, 21, 24, S, 1, dtype=F, seed=64 + S)
    a["A"] = torch.full((24, S), 3.0, device="cuda")
    a["dt"], a["dt_bias"] = a["dt"] * 0.5 - 32, torch.full((24,), 30.0, device="cuda")
    compare(run_scan(a), want_scan(a), F)
