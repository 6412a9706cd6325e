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


# ---- growing states of a sequence that is cut into segments -------------------------------------------

@pytest.mark.parametrize("S", [8, 16, 64])
def test_zero_states_stay_zero_where_decays_have_no_value(S):
    """A = 1, steps near 2: a segment's whole decay is past 2^128.  x is zero but for the last tokens, grad_out but for the first
    ones, so that all values are finite: the states, and the gradients through them, are zeros where the segments meet."""
    N = 700
    a = inputs(1, N, 16, S, 1, dtype=F, seed=70 + S, strided=False)
    a["A"] = torch.ones(16, S, device="cuda")
    a["dt"], a["dt_bias"] = 1.8 + 0.4 * a["dt"].sigmoid(), torch.zeros(16, device="cuda")
    a["x"][:, :-8], a["grad_out"][:, 8:] = 0, 0
    del a["initial_state"], a["grad_final_state"]
    compare(run_scan(a, softplus=False), want_scan(a, softplus=False), F)


@pytest.mark.parametrize("S", [8, 16, 64])
def test_small_states_grow_past_a_decay_without_a_value(S):
    """An initial state of 1e-37 and a gradient of the final one of 1e-37 grow by exp(150) within one segment: more than any
    decay that float32 holds, and neither leaves its range."""
    N = 700
    a = inputs(1, N, 16, S, 1, dtype=F, seed=74 + S, strided=False)
    a["A"] = torch.ones(16, S, device="cuda")
    a["dt"], a["dt_bias"] = 1e-3 * a["dt"].sigmoid(), torch.zeros(16, device="cuda")
    a["dt"][:, 320:350] += 5
    a["x"].zero_()
    a["grad_out"].zero_()
    for k in ("initial_state", "grad_final_state"):
        a[k] = (1 + a[k].sigmoid()) * 1e-37
    compare(run_scan(a, softplus=False), want_scan(a, softplus=False), F)


@pytest.mark.parametrize("where", [70, 350, 699])
def test_an_infinite_step_cuts_the_gradient(where):
    """A step of infinity is a decay of 0: the gradients of the tokens before it are those of a sequence that ends there."""
    a = inputs(1, 700, 16, 16, 1, dtype=F, seed=78, strided=False)
    del a["grad_final_state"]
    short = dict(a, lengths=torch.tensor([where], dtype=torch.int32, device="cuda"))
    want = run_scan(short)
    a["dt"][:, where] = float("inf")
    got = run_scan(a)
    for k in ("out", "dx", "ddt", "dz", "dB", "dC"):
        assert bool(got[k][:, :where].isfinite().all()) and torch.equal(got[k][:, :where], want[k][:, :where]), k
    assert torch.equal(got["grad_initial_state"], want["grad_initial_state"])


# ---- rows behind a length in the convolution ----------------------------------------------------------

@pytest.mark.parametrize("W", [2, 3, 4])
def test_infinite_last_row_of_a_padded_sequence(W):
    """Without silu: x of the last token meets the newest tap alone; the rows behind the length add nothing to the others."""
    g = torch.Generator().manual_seed(90 + W)
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    x, w, go = r(2, 40, 16), r(16, W), r(2, 40, 16)
    n = torch.tensor([17, 40], dtype=torch.int32, device="cuda")
    x[0, 16] = 0
    _, want, _ = la.conv_bwd(x, w, go, silu=False, lengths=n)
    x[0, 16] = float("inf")
    dx, got, _ = la.conv_bwd(x, w, go, silu=False, lengths=n)
    assert torch.equal(got[:, :-1], want[:, :-1]) and bool(got[:, -1].isinf().all()) and bool(dx.isfinite().all())


# ---- sums over several blocks of a group's channels ---------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 24, 528, 16, 1), (1, 18, 544, 16, 2), (2, 12, 272, 32, 2), (1, 20, 136, 64, 1), (1, 10, 544, 8, 2),
                                   (2, 9, 256, 64, 1), (1, 300, 288, 16, 1)], ids=lambda s: "x".join(map(str, s)))
def test_several_blocks_of_a_group(shape, dtype):
    a = inputs(*shape, dtype=dtype, seed=sum(shape) + 1)
    compare(run_scan(a), want_scan(a), dtype)


# ---- NaN and infinities --------------------------------------------------------------------------------

# tokens before (e), at (a) and after (l) the NaN that it reaches: the states after it through d x B, the gradients of the
# states before it through the gate, C and the decays
REACH = {
    "x": dict(dx="", ddt="al", dz="al", dB="a", dC="al"),
    "dt": dict(dx="ea", ddt="eal", dz="al", dB="ea", dC="al"),
    "B": dict(dx="a", ddt="al", dz="al", dB="", dC="al"),
    "C": dict(dx="ea", ddt="ea", dz="a", dB="ea", dC=""),
    "z": dict(dx="ea", ddt="ea", dz="a", dB="ea", dC="a"),
    "grad_out": dict(dx="ea", ddt="ea", dz="a", dB="ea", dC="a"),
}


@pytest.mark.parametrize("N,where", [(40, 3), (40, 20), (700, 350)])
@pytest.mark.parametrize("name", list(REACH))
def test_nan_of_a_token_in_the_gradient(name, N, where):
    """A NaN in one token reaches what depends on it by the formula, and nothing else changes by a bit."""
    a = inputs(2, N, 72, 16, 1, dtype=F, seed=80, strided=False)
    want = run_scan(a)
    a[name][1, where, ..., 5] = float("nan")
    got = run_scan(a)
    at = dict(e=slice(0, where), a=slice(where, where + 1), l=slice(where + 1, None))
    for k, tokens in REACH[name].items():
        # channel 5 (of x, dt, z, grad_out) or all (of B and C, in state 5 alone); sums over channels
        where_k = slice(None) if (k in ("dB", "dC")) != (name in ("B", "C")) else slice(5, 6)
        hit = torch.zeros_like(want[k], dtype=torch.bool)
        for t in tokens:
            hit[1, at[t], ..., where_k] = True
        assert torch.equal(torch.isnan(got[k]), hit), k
        assert torch.equal(got[k][~hit], want[k][~hit]), k
