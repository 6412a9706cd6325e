"""GPU parity of the query/key norm with position rotation with the float64 oracle.

Tolerances.  float32 arithmetic: the norm's sum of D squares, rsqrt (2 steps), three products, the
rotation's two and its sine and cosine (angle to 2^-25 turns and 2 steps each): (D / 2 + 24) 2^-24 of the row's largest
turned magnitude covers them; the result is rounded once (2^-8 bfloat16, 2^-24 float32).  Weight
gradients: sums of R rows' terms, each as exact as above, (D / 2 + 24 + rows) 2^-24 of the absolute sum."""
import numpy as np
import pytest
import torch

from efficient_transformer_gb300 import build as la_build
from efficient_transformer_gb300 import la
from oracle import decay as od

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    la_build.build()
    la.load()


def close(got, want, size, D, dtype, extra=0.0, name=""):
    got = got.detach().double().cpu().numpy()
    half = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    tol = half * np.abs(want) + (D / 2 + 24 + extra) * 2.0 ** -24 * size + 1e-37
    assert np.isfinite(got).all()
    bad = np.abs(got - want) / tol
    assert bad.max() <= 1.0, (name, float(bad.max()))


CASES = [
    # B, Hq, Hkv, N, D, rot, axes, interleaved, weights
    (1, 1, 1, 1, 32, 32, 1, False, F), (2, 3, 1, 5, 64, 64, 1, True, None), (3, 8, 2, 17, 128, 128, 3, False, F),
    (1, 5, 5, 33, 128, 32, 2, True, "x"), (2, 7, 1, 64, 64, 48, 3, False, "x"), (1, 4, 4, 700, 32, 16, 1, False, F),
    (65, 9, 3, 1, 128, 96, 4, False, F), (1, 2, 2, 100, 64, 0, 1, False, F), (1, 33, 1, 9, 128, 112, 2, True, F),
]


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[:8])))
@pytest.mark.parametrize("normalize", [True, False])
def test_parity(case, dtype, normalize):
    B, Hq, Hkv, N, D, R, axes, inter, wt = case
    g = torch.Generator().manual_seed(5)
    x = (torch.randn(B, N, Hq + 2 * Hkv, D, generator=g) * 2).to(dtype)
    q, k = x[:, :, :Hq].permute(0, 2, 1, 3), x[:, :, Hq:Hq + Hkv].permute(0, 2, 1, 3)
    gq, gk = (torch.randn(B, H, N, D, generator=g).to(dtype) for H in (Hq, Hkv))
    wt = None if wt is None or not normalize else dtype if wt == "x" else wt
    w = [None, None] if wt is None else [(1 + 0.3 * torch.randn(D, generator=g)).to(wt) for _ in range(2)]
    kw = dict(eps=1e-5, interleaved=inter, normalize=normalize)
    if R:
        # the first token of each sequence far away, on every axis; and negative positions
        pos = torch.randint(-1000, 40000, (axes, B, N), generator=g)
        pos[:, :, 0] = 10 ** 9 + 7
        cut = R // 2 // axes
        kw.update(positions=pos, inv_freq=torch.pow(500000.0, -torch.arange(R // 2, dtype=torch.float64) * 2 / R),
                  sections=[R // 2 - cut * (axes - 1)] + [cut] * (axes - 1))
    dkw = {n: t.cuda() if torch.is_tensor(t) else t for n, t in kw.items()}
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    xd = x.cuda()
    qd, kd = xd[:, :, :Hq].permute(0, 2, 1, 3), xd[:, :, Hq:Hq + Hkv].permute(0, 2, 1, 3)
    got = la.qk_norm_rope_fwd(qd, kd, q_weight=dev(w[0]), k_weight=dev(w[1]), **dkw)
    again = la.qk_norm_rope_bwd(qd, kd, gq.cuda(), gk.cuda(), q_weight=dev(w[0]), k_weight=dev(w[1]), **dkw)
    grads = la.qk_norm_rope_bwd(qd, kd, gq.cuda(), gk.cuda(), q_weight=dev(w[0]), k_weight=dev(w[1]), **dkw)
    la.get_status()
    for a, b in zip(again, grads):
        assert (a is None and b is None) or torch.equal(a, b)
    for i, (src, go) in enumerate(((q, gq), (k, gk))):
        want = od.qk_fwd(src, weight=w[i], **kw)
        close(got[i], want, np.abs(want).max(-1, keepdims=True) * 2, D, dtype, name="fwd")
        dx, dw, dwa = od.qk_bwd(src, go, weight=w[i], **kw)
        r = 1 / np.sqrt((src.double().numpy() ** 2).mean(-1, keepdims=True) + 1e-5) if normalize else 1.0
        xh = np.abs(src.double().numpy() * r).max(-1, keepdims=True)
        u = np.abs(go.double().numpy()).max(-1, keepdims=True) * 2 * (1 if w[i] is None else float(w[i].abs().max()))
        close(grads[i], dx, r * u * (1 + xh * xh), D, dtype, name="dx")
        if w[i] is not None:
            size = (u * xh / float(w[i].abs().max())).sum((0, 1, 2)) + dwa
            close(grads[2 + i], dw, size, D, w[i].dtype, extra=min(B * N * src.shape[1], 4096), name="dw")


def test_broadcast_positions_other_stream_and_graph():
    """Positions shared by the batch (stride 0), on another stream and captured into a graph."""
    B, H, N, D = 3, 4, 50, 64
    g = torch.Generator().manual_seed(9)
    q, k = (torch.randn(B, H, N, D, generator=g).to(BF).cuda() for _ in range(2))
    w = torch.ones(D, device="cuda")
    f = torch.pow(10000.0, -torch.arange(32, dtype=torch.float64) / 32).cuda()
    pos = torch.arange(N, device="cuda")[None, :].expand(B, N)
    want = la.qk_norm_rope_fwd(q, k, q_weight=w, positions=pos.contiguous(), inv_freq=f)
    gwant = la.qk_norm_rope_bwd(q, k, q, k, q_weight=w, positions=pos.contiguous(), inv_freq=f)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = la.qk_norm_rope_fwd(q, k, q_weight=w, positions=pos, inv_freq=f, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = la.qk_norm_rope_fwd(q, k, q_weight=w, positions=pos, inv_freq=f)
        grads = la.qk_norm_rope_bwd(q, k, q, k, q_weight=w, positions=pos, inv_freq=f)
    graph.replay()
    la.get_status()
    assert all(torch.equal(a, b) for a, b in zip(got + grads[:3], want + gwant[:3])) and grads[3] is None


def test_non_finite_row_stays_in_its_row():
    q = torch.randn(1, 2, 8, 64, device="cuda").to(BF)
    k = torch.randn(1, 2, 8, 64, device="cuda").to(BF)
    f = torch.ones(16, dtype=torch.float64, device="cuda")
    pos = torch.arange(8, device="cuda")[None]
    want = la.qk_norm_rope_fwd(q, k, positions=pos, inv_freq=f)
    q2 = q.clone()
    q2[0, 1, 3, 60] = float("inf")
    got = la.qk_norm_rope_fwd(q2, k, positions=pos, inv_freq=f)
    keep = torch.ones(2, 8, dtype=torch.bool)
    keep[1, 3] = False
    assert torch.equal(got[0][0][keep], want[0][0][keep]) and torch.equal(got[1], want[1])
    # without the norm, elements past rot are not met by the rotation's 0 x inf
    got = la.qk_norm_rope_fwd(q2, k, positions=pos, inv_freq=f, normalize=False)
    assert torch.isfinite(got[0][0, 1, 3, :60]).all() and torch.isinf(got[0][0, 1, 3, 60])
