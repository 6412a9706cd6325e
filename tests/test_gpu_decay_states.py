"""States that go out, whatever the batch: a state's accuracy does not follow from whether its sequence was cut.

Bound (2-norm of a head's state, relative): as in test_gpu_decay_precision.  One accumulator for whole sequences and two
bfloat16 terms exceeded it: 4e-6 for the terms, 7.4e-5 in all for the gradient of 8 x 128/16 heads, N 4096."""
import pytest
import torch

from efficient_transformer_gb300 import build as la_build
from efficient_transformer_gb300 import la
from test_gpu_decay_precision import STATE as BOUND

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    la_build.build()
    la.load()


def draw(B, Hq, Hkv, N, D, Dv, seed=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(B, h, N, w, device="cuda", generator=g).to(BF) for h, w in ((Hq, D), (Hkv, D), (Hkv, Dv), (Hq, Dv))]


def final(k, v, l, n):
    """The state after n tokens of one head, from zeros, in float64."""
    j = torch.arange(n, device="cuda", dtype=torch.float64)
    return (k[:n].double() * torch.exp(l * (n - 1 - j))[:, None]).T @ v[:n].double()


def error(got, want):
    return float((got - want).norm() / want.norm())


# B, Hq, Hkv, N, D, Dv: many heads, so that sequences stay whole or nearly so; long ones, shared heads, all widths
SHAPES = [(10, 16, 16, 20000, 128, 128), (8, 128, 16, 4096, 128, 128), (4, 40, 40, 16384, 64, 64), (5, 96, 32, 5001, 64, 128),
          (5, 64, 32, 5001, 128, 64), (40, 32, 4, 700, 128, 128), (1, 64, 1, 3000, 64, 64)]


@pytest.mark.parametrize("decay", [0.0, -1e-3])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_long_memories(shape, decay):
    B, Hq, Hkv, N, D, Dv = shape
    r = Hq // Hkv
    q, k, v, go = draw(*shape)
    ld = torch.full((Hkv,), decay, device="cuda")
    S1, dS0 = torch.empty(B, Hkv, D, Dv, device="cuda"), torch.empty(B, Hkv, D, Dv, device="cuda")
    la.decay_fwd(q, k, v, ld, final_state=S1)
    la.decay_bwd(q, k, v, go, ld, grad_initial_state=dS0)
    la.get_status()
    l = float(ld[0])
    j = torch.arange(N, device="cuda", dtype=torch.float64)
    w = torch.exp(l * (j + 1))[:, None]
    for b, h in ((0, 0), (B - 1, Hkv - 1), (B // 2, Hkv // 2)):
        assert error(S1[b, h], final(k[b, h], v[b, h], l, N)) < BOUND
        dS = sum((q[b, h * r + i].double() * w).T @ go[b, h * r + i].double() for i in range(r))
        assert error(dS0[b, h], dS) < BOUND


@pytest.mark.parametrize("D,Dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
def test_uncut_prompts_in_place_with_lengths(D, Dv):
    """A whole prompt's state in place of its starting state, lengths of their own, and what is asked for changing no
    other output: the same rows with a state going out and without."""
    B, Hq, Hkv, N = 38, 8, 4, 4500
    for bwd in (False, True):     # whole sequences, summed in one part (38 x 4 heads, one an SM)
        assert la.decay_workspace_size(B, Hq, Hkv, N, D, BF, bwd, Dv=Dv) == 0
    q, k, v, go = draw(B, Hq, Hkv, N, D, Dv)
    ld = torch.tensor([0.0, -1e-3, -0.05, -1.0], device="cuda")
    n = torch.randint(0, N + 1, (B,), generator=torch.Generator().manual_seed(1)).int()
    n[:6] = torch.tensor([0, 1, 128, 129, N, 4097])
    S0 = torch.randn(B, Hkv, D, Dv, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    S = S0.clone()
    rows = la.decay_fwd(q, k, v, ld, initial_state=S0, lengths=n.cuda())
    out = la.decay_fwd(q, k, v, ld, initial_state=S, final_state=S, lengths=n.cuda())
    dS1, dS0 = S0.flip(0).contiguous(), torch.empty_like(S0)
    grads = la.decay_bwd(q, k, v, go, ld, initial_state=S0, grad_final_state=dS1)
    again = la.decay_bwd(q, k, v, go, ld, initial_state=S0, grad_final_state=dS1, grad_initial_state=dS0)
    la.get_status()
    assert torch.equal(out, rows) and all(torch.equal(a, b) for a, b in zip(grads, again))
    assert torch.equal(S[0], S0[0])
    for b in range(10):
        m = int(n[b])
        for h in range(Hkv):
            l = float(ld[h])
            want = final(k[b, h], v[b, h], l, m) + torch.exp(torch.tensor(l * m, dtype=torch.float64)).cuda() * S0[b, h].double()
            assert error(S[b, h], want) < BOUND or torch.equal(S[b, h].double(), want)
            j = torch.arange(N, device="cuda", dtype=torch.float64)
            w = torch.exp(l * (j + 1))[:, None]
            dS = sum((q[b, 2 * h + i].double() * w).T @ go[b, 2 * h + i].double() for i in range(2))
            dS += torch.exp(torch.tensor(l * N, dtype=torch.float64)).cuda() * dS1[b, h].double()
            assert error(dS0[b, h], dS) < BOUND


@pytest.mark.parametrize("shape", [(64, 32, 8, 512, 128, 128), (32, 8, 8, 1024, 128, 128), (2, 2, 2, 1, 128, 128)],
                         ids=lambda s: "x".join(map(str, s)))
def test_batches_of_prompts_and_their_gradients_captured(shape):
    """The ordinary prefill of a server, whole sequences with states out, into a graph with a caller's workspace."""
    B, Hq, Hkv, N, D, Dv = shape
    q, k, v, go = draw(*shape)
    ld = torch.full((Hkv,), -0.003, device="cuda")
    S1, dS0 = torch.empty(B, Hkv, D, Dv, device="cuda"), torch.empty(B, Hkv, D, Dv, device="cuda")
    out, (dq, dk, dv) = torch.empty_like(q), (torch.empty_like(t) for t in (q, k, v))
    ws = torch.full((max(1, la.decay_workspace_size(B, Hq, Hkv, N, D, BF, True, Dv=Dv)),), 255, dtype=torch.uint8, device="cuda")

    def work():
        la.decay_fwd(q, k, v, ld, final_state=S1, out=out, workspace=ws)
        la.decay_bwd(q, k, v, go, ld, grad_initial_state=dS0, dq=dq, dk=dk, dv=dv, workspace=ws)

    work()
    torch.cuda.synchronize()
    want = [t.clone() for t in (out, S1, dq, dk, dv, dS0)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    for t in (out, S1, dq, dk, dv, dS0):
        t.fill_(float("nan"))
    ws.fill_(255)
    graph.replay()
    la.get_status()
    assert all(torch.equal(a, b) for a, b in zip((out, S1, dq, dk, dv, dS0), want))
    for b, h in ((0, 0), (B - 1, Hkv - 1)):
        assert error(S1[b, h], final(k[b, h], v[b, h], float(ld[h]), N)) < BOUND
