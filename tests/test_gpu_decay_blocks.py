"""Rows of the decayed attention and of its gradients against float64, as relative 2-norms of each head's blocks of 128
tokens (decay_blocks: bound and what it finds).  Also: inputs that are broadcast, and states that grow."""
import pytest
import torch

import decay_blocks as db
from efficient_transformer_gb300 import build as la_build
from efficient_transformer_gb300 import la

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    la_build.build()
    la.load()


def draw(B, Hq, Hkv, N, D, Dv, dtype=BF, seed=0, ld=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    mk = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    t = [mk(B, h, N, w).to(dtype) for h, w in ((Hq, D), (Hkv, D), (Hkv, Dv), (Hq, Dv))]
    ld = -torch.exp(torch.linspace(-6.0, 0.7, Hkv, device="cuda")) if ld is None else torch.full((Hkv,), ld, device="cuda")
    return t + [ld, mk(B, Hkv, D, Dv), mk(B, Hkv, D, Dv)]


def compare(q, k, v, go, ld, S0, dS1, states, limit=db.LIMIT):
    out_state = torch.empty(q.shape[0], k.shape[1], q.shape[3], v.shape[3], device="cuda") if states else None
    dS0 = torch.empty_like(out_state) if states else None
    out = la.decay_fwd(q, k, v, ld, scale=0.25, initial_state=S0, final_state=out_state)
    grads = la.decay_bwd(q, k, v, go, ld, scale=0.25, initial_state=S0, grad_final_state=dS1, grad_initial_state=dS0)
    la.get_status()
    want = db.reference(q, k, v, go, ld, 0.25, S0, dS1)
    for name, a, b in zip(("out", "dq", "dk", "dv"), (out,) + grads, (want[0], *want[2:5])):
        assert db.close(a, b, limit), (name, float(db.block_errors(a, b).max()))
    if states:
        for a, b in ((out_state, want[1]), (dS0, want[5])):
            assert b is None or float((a - b).norm() / b.norm()) < 2.0 ** -15


# B, Hq, Hkv, N, D, Dv: cut sequences (few heads) with every pair of widths, shared heads; whole ones (many heads); odd lengths
SHAPES = [(2, 20, 4, 1300, 64, 64), (2, 20, 4, 1300, 128, 128), (1, 12, 4, 1300, 64, 128), (1, 12, 4, 1300, 128, 64),
          (1, 4, 4, 2777, 128, 128), (1, 4, 4, 2777, 64, 64), (1, 8, 1, 2001, 64, 64), (40, 4, 4, 700, 128, 128),
          (40, 4, 4, 700, 64, 64), (26, 18, 6, 385, 64, 128), (26, 18, 6, 385, 128, 64)]


@pytest.mark.parametrize("states", [True, False], ids=["states", "no states"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_blocks(shape, states):
    t = draw(*shape, seed=shape[3])
    if not states:
        t[5] = t[6] = None
    compare(*t, states)


@pytest.mark.parametrize("ld", [0.0, -1e-4, -0.02])
@pytest.mark.parametrize("shape", SHAPES[:4], ids=lambda s: "x".join(map(str, s)))
def test_blocks_of_equal_decays(shape, ld):
    compare(*draw(*shape, seed=1, ld=ld), True)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(2, 4, 2, 300, 64, 64), (1, 4, 2, 200, 128, 64), (1, 4, 2, 1500, 64, 128), (1, 2, 2, 90, 32, 32)],
                         ids=lambda s: "x".join(map(str, s)))
def test_growing_states(shape, dtype):
    """log_decay above 0: gamma up to 1.05, by the same formula."""
    t = draw(*shape, dtype, seed=2)
    t[4] = torch.linspace(0.002, 0.05 if shape[3] <= 300 else 0.01, shape[2], device="cuda")
    compare(*t, True)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
def test_broadcast_inputs(D, dtype):
    """Inputs of stride 0 along the batch, the heads or both, as expand() makes them: the same bits as copies."""
    B, Hq, Hkv, N = 3, 4, 2, 700
    q, k, v, go, ld, S0, dS1 = draw(1, 1, 1, N, D, D, dtype, seed=8)
    ld = torch.tensor([-0.01, -0.3], device="cuda")
    q, go = q.expand(B, Hq, N, D), torch.randn(1, Hq, N, D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(dtype).expand(B, -1, -1, -1)
    k, v = k.expand(B, Hkv, N, D), torch.randn(B, 1, N, D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)).to(dtype).expand(-1, Hkv, -1, -1)
    assert 0 in q.stride() and 0 in k.stride() and 0 in v.stride() and 0 in go.stride()
    got = (la.decay_fwd(q, k, v, ld),) + la.decay_bwd(q, k, v, go, ld)
    q, k, v, go = (t.contiguous() for t in (q, k, v, go))
    want = (la.decay_fwd(q, k, v, ld),) + la.decay_bwd(q, k, v, go, ld)
    la.get_status()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
