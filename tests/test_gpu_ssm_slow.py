"""Slow channels of the selective scan: states that remember thousands of tokens, where what every decay errs adds up."""
import pytest
import torch

from efficient_transformer_gb300 import build as la_build
from efficient_transformer_gb300 import la

pytestmark = pytest.mark.gpu

N, E, S = 16384, 64, 8


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    la_build.build()
    la.load()


# Step, and the mean error of its decays (csrc/la_ssm.cuh, in round figures).  One that errs by D changes the state by D times the
# share of it that is older.  With terms of one sign these shares are exp(-n step) for n tokens: `memory` in sum, half of it in
# squares.  So the mean error makes mean x memory, and independent ones of 2^-24 a token (of the decay 4e-8, of the state's own
# rounding 3.5e-8 at most, root mean squares) 2^-24 sqrt(memory / 2); twice that, for 64 channels' norm of it is within a
# tenth or so.
@pytest.mark.parametrize("pieces", [1, N // 64], ids=["whole", "pieces"])
@pytest.mark.parametrize("step,mean", [(1e-4, 3e-9), (3e-4, 3e-9), (1e-3, 3e-9), (1e-2, 1e-8), (3e-2, 1e-8), (1e-1, 1e-8)])
def test_states_of_slow_channels(step, mean, pieces):
    """The whole sequence, which the library cuts into segments, and pieces of 64 tokens, whose decays all add up."""
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: 0.5 + torch.rand(*s, device="cuda", generator=g)  # noqa: E731
    dt, x, B, C, A = step * r(1, N, E), r(1, N, E), r(1, N, 1, S), r(1, N, 1, S), -torch.ones(E, S, device="cuda")
    state, n = torch.zeros(1, E, S, device="cuda"), N // pieces
    for i in range(pieces):
        at = slice(i * n, (i + 1) * n)
        la.ssm_fwd(x[:, at].contiguous(), dt[:, at].contiguous(), A, B[:, at].contiguous(), C[:, at].contiguous(),
                   softplus=False, initial_state=state, final_state=state)
    la.get_status()
    # the state in 64 bits: every token's term times the decays after it
    d = dt[0].double()
    after = torch.exp(-(d.sum(0) - d.cumsum(0)))
    want = ((after * d * x[0].double()).T @ B[0, :, 0].double())[None]
    memory = min(1 / step, N / 2)
    assert float((state - want).norm() / want.norm()) < mean * memory + 2 * 2.0 ** -24 * (memory / 2) ** 0.5 + 2.0 ** -23


def test_a_token_has_no_part_in_the_rows_before_it():
    """Not even in their roundings: the tokens after the first 37, and their steps, are others."""
    g = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    x, dt, B, C, A = r(1, 200, E), r(1, 200, E) - 5, r(1, 200, 1, 16), r(1, 200, 1, 16), -torch.exp(r(E, 16))
    want = la.ssm_fwd(x, dt, A, B, C)
    for t in (x, dt, B, C):
        t[:, 37:] = 4 + r(*t[:, 37:].shape)
    got = la.ssm_fwd(x, dt, A, B, C)
    assert torch.equal(got[:, :37], want[:, :37]) and not torch.equal(got[:, 37:], want[:, 37:])


@pytest.mark.parametrize("step,mean", [(1e-4, 3e-9), (1e-3, 3e-9), (1e-2, 2e-8)])
def test_states_of_slow_channels_token_by_token(step, mean):
    """Single tokens, whose decays all have the correction of slow states."""
    n = 4096
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: 0.5 + torch.rand(*s, device="cuda", generator=g)  # noqa: E731
    dt, x, B, C, A = step * r(n, 1, E), r(n, 1, E), r(n, 1, 1, S), r(n, 1, 1, S), -torch.ones(E, S, device="cuda")
    state = torch.zeros(1, E, S, device="cuda")
    for t in range(n):
        at = slice(t, t + 1)
        la.ssm_step(x[at], dt[at], A, B[at], C[at], state, softplus=False)
    la.get_status()
    d = dt[:, 0].double()
    after = torch.exp(-(d.sum(0) - d.cumsum(0)))
    want = ((after * d * x[:, 0].double()).T @ B[:, 0, 0].double())[None]
    memory = min(1 / step, n / 2)
    assert float((state - want).norm() / want.norm()) < mean * memory + 2 * 2.0 ** -24 * (memory / 2) ** 0.5 + 2.0 ** -23
