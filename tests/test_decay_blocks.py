"""The blockwise check of decay_blocks on the host: its reference agrees with the oracle, a result rounded as the
kernels round passes it, and mistakes planted in the reference fail it."""
import numpy as np
import pytest
import torch

import decay_blocks as db
from oracle import decay as od

BF = torch.bfloat16


def draw(B, Hq, Hkv, N, D, Dv, seed=0):
    g = torch.Generator().manual_seed(seed)
    mk = lambda h, w: torch.randn(B, h, N, w, generator=g).to(BF).double()  # noqa: E731
    q, k, v, go = mk(Hq, D), mk(Hkv, D), mk(Hkv, Dv), mk(Hq, Dv)
    ld = -torch.exp(torch.linspace(-6.0, 0.7, Hkv))
    return q, k, v, go, ld, torch.randn(B, Hkv, D, Dv, generator=g).double(), torch.randn(B, Hkv, D, Dv, generator=g).double()


def test_reference_is_the_oracle():
    q, k, v, go, ld, S0, dS1 = draw(2, 6, 3, 60, 8, 12)
    n = torch.tensor([60, 17])
    for a, b in zip(db.forward(q, k, v, ld, 0.5, S0, n), od.fwd(q, k, v, ld, 0.5, S0, n)):
        np.testing.assert_allclose(a.numpy(), b, rtol=1e-9, atol=1e-9)
    want = od.fwd(q, k, v, ld, 0.5, S0) + od.bwd(q, k, v, go, ld, 0.5, S0, dS1)
    for a, b in zip(db.reference(q, k, v, go, ld, 0.5, S0, dS1), want):
        np.testing.assert_allclose(a.numpy(), b, rtol=1e-9, atol=1e-9)


SHAPE = (1, 12, 4, 640, 64, 64)     # decays from 0.9975 to 0.13


@pytest.fixture(scope="module")
def case():
    t = draw(*SHAPE, seed=3)
    return t, db.reference(*t[:5], 0.25, *t[5:])


def test_rounded_results_pass(case):
    (q, k, v, go, ld, S0, dS1), want = case
    for x in (want[0], *want[2:5]):
        assert db.close(x.to(BF), x)
    # scores, decayed y and result, each rounded once, chunk by chunk
    g = torch.exp(ld.double())[:, None]
    S, rows, r = S0[0].clone(), [], SHAPE[1] // SHAPE[2]
    i = torch.arange(128).double()
    bf = lambda x: x.to(BF).double()  # noqa: E731
    for t in range(0, SHAPE[3], 128):
        kc, vc, qc = k[0, :, t:t + 128], v[0, :, t:t + 128], q[0, :, t:t + 128].view(SHAPE[2], r, 128, -1)
        w = (g[..., None] ** (i[:, None] - i[None]).clamp(min=0)).tril()
        P = bf(0.25 * torch.einsum("hrid,hjd->hrij", qc, kc) * w[:, None])
        x = 0.25 * qc * (g ** (i + 1))[:, None, :, None]
        rows.append(bf(torch.einsum("hrij,hje->hrie", P, vc) + torch.einsum("hrid,hde->hrie", x, S)))
        S = g[..., None] ** 128 * S + torch.einsum("hjd,hje->hde", bf(kc * (g ** (127 - i))[..., None]), vc)
    assert db.close(torch.cat(rows, 2).reshape(want[0].shape), want[0])


CUT = 384



@pytest.mark.parametrize("mistake", ["carry dropped", "half the carry", "a power of gamma too many", "a power too few",
                                     "a chunk's power too many"])
def test_mistaken_carries_fail(case, mistake):
    """The rows after token 384 from a state that was carried there wrongly; and, in the other direction, the
    gradients before it."""
    (q, k, v, go, ld, S0, dS1), want = case
    g = torch.exp(ld.double())[:, None, None]
    mul = {"carry dropped": 0 * g, "half the carry": 0 * g + 0.5, "a power of gamma too many": g, "a power too few": 1 / g,
           "a chunk's power too many": g ** 128}[mistake]
    S = db.forward(*(x[:, :, :CUT] for x in (q, k, v)), ld, 0.25, S0)[1]
    right, wrong = (db.forward(*(x[:, :, CUT:] for x in (q, k, v)), ld, 0.25, s)[0] for s in (S, S * mul))
    assert db.close(right, want[0][:, :, CUT:], 1e-9)
    assert not db.close(wrong, want[0][:, :, CUT:])
    # the state's gradient at the cut, scaled, and what k and v before it get of it
    dS = db.reference(*(x[:, :, CUT:] for x in (q, k, v, go)), ld, 0.25, S, dS1)[5]
    for d, good in ((dS, True), (dS * mul, False)):
        got = db.reference(*(x[:, :, :CUT] for x in (q, k, v, go)), ld, 0.25, S0, d)
        for name in (3, 4):
            assert db.close(got[name], want[name][:, :, :CUT], 1e-9 if good else db.LIMIT) == good


def test_one_missing_head_of_a_group_fails(case):
    (q, k, v, go, ld, S0, dS1), want = case
    g2 = go.clone()
    g2[:, 3] = 0
    got = db.reference(q, k, v, g2, ld, 0.25, S0, dS1)
    assert not db.close(got[3], want[3]) and not db.close(got[4], want[4])


def test_zero_blocks_have_to_be_zeros():
    x = torch.randn(1, 1, 256, 4)
    x[:, :, 128:] = 0
    y = x.clone()
    assert db.close(y, x)
    y[0, 0, 200, 1] = 1e-6
    assert not db.close(y, x)
