"""How exact bfloat16 calls of the decayed attention are on the tensor cores.

Rows.  Every term of an output is rounded to bfloat16 once on its way and the output once more; independent roundings of the
same relative size add up to sqrt(2) of what rounding the output alone leaves.  Bound: 1.5 times that (2-norm of a tensor).
States.  float32 inputs' worth: y w in three bfloat16 terms (2^-25), a chunk's and head's sum cut at each of its 8 steps (2^-23
at worst, as its later partial sums are whole and the earlier ones are not: 8 2^-24), sums of these in float32 and
gamma^n from a float32 exponent, (2 |n log gamma| + 2) 2^-24 of a term, where terms of |n log gamma| above 4 hardly
count: (8 + 10 + 1) 2^-24, 1.1e-6."""
import pytest
import torch

import decay_blocks as db
from efficient_transformer_gb300 import build as la_build
from efficient_transformer_gb300 import la
from test_gpu_decay_blocks import draw

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
STATE = 19 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    la_build.build()
    la.load()


def rows_close(got, want, name):
    alone = float((want.to(BF).double() - want).norm() / want.norm())
    err = float((got.double() - want).norm() / want.norm())
    assert err <= 1.5 * alone, (name, err, alone)


# cut and whole sequences, shared heads, every pair of widths
SHAPES = [(2, 8, 4, 1700, 64, 64), (1, 4, 4, 2048, 128, 128), (2, 16, 2, 1300, 128, 128), (1, 12, 4, 1537, 128, 64),
          (1, 12, 4, 1537, 64, 128), (38, 4, 4, 640, 128, 128), (38, 4, 4, 640, 64, 64), (19, 32, 8, 384, 128, 128)]


@pytest.mark.parametrize("scale", [0.125, -3.0])
@pytest.mark.parametrize("ld", [None, 0.0, -1e-3, -0.02])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_rows_and_states(shape, ld, scale):
    q, k, v, go, ld, S0, dS1 = draw(*shape, seed=7, ld=ld)
    S1, dS0 = torch.empty_like(S0), torch.empty_like(S0)
    out = la.decay_fwd(q, k, v, ld, scale=scale, initial_state=S0, final_state=S1)
    grads = la.decay_bwd(q, k, v, go, ld, scale=scale, initial_state=S0, grad_final_state=dS1, grad_initial_state=dS0)
    la.get_status()
    want = db.reference(q, k, v, go, ld, scale, S0, dS1)
    for name, a, b in zip(("out", "dq", "dk", "dv"), (out,) + grads, (want[0], *want[2:5])):
        rows_close(a, b, name)
    for name, a, b in zip(("final_state", "grad_initial_state"), (S1, dS0), (want[1], want[5])):
        for h in range(b.shape[1]):
            assert float((a[:, h] - b[:, h]).norm() / b[:, h].norm()) < STATE, (name, h)


@pytest.mark.parametrize("shape", SHAPES[:5], ids=lambda s: "x".join(map(str, s)))
def test_rows_without_states(shape):
    q, k, v, go, ld, _, _ = draw(*shape, seed=9, ld=-1e-4)
    out, grads = la.decay_fwd(q, k, v, ld), la.decay_bwd(q, k, v, go, ld)
    la.get_status()
    want = db.reference(q, k, v, go, ld)
    for name, a, b in zip(("out", "dq", "dk", "dv"), (out,) + grads, (want[0], *want[2:5])):
        rows_close(a, b, name)


@pytest.mark.parametrize("size", [1e-18, 1e12])
def test_sizes_of_the_inputs(size):
    """The row factors are powers of two: nothing depends on how large the inputs are."""
    q, k, v, go, ld, S0, dS1 = draw(1, 4, 2, 700, 64, 64, seed=3)
    q, S0 = (q.float() * size).to(BF), S0 * size
    out = la.decay_fwd(q, k, v, ld, scale=0.5, initial_state=S0)
    la.get_status()
    want = db.forward(q.double(), k.double(), v.double(), ld, 0.5, S0.double())[0]
    rows_close(out, want, "out")
