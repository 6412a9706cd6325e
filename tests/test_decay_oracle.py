"""Pins of the decayed attention's oracle that do not come from the oracle: the quadratic form,
autograd of it, differences, splitting a sequence at a state; and of the norm with rotation."""
import numpy as np
import pytest
import torch

from oracle import decay as od


def draw(B, Hq, Hkv, N, D, Dv, seed=0):
    g = np.random.default_rng(seed)
    q, k, v, go = (g.standard_normal(s) for s in ((B, Hq, N, D), (B, Hkv, N, D), (B, Hkv, N, Dv), (B, Hq, N, Dv)))
    ld = -np.exp(g.uniform(-4, 0.5, Hkv))
    return q, k, v, go, ld, g.standard_normal((B, Hkv, D, Dv)), g.standard_normal((B, Hkv, D, Dv))


def quadratic(q, k, v, ld, scale, S0):
    """The definition as one masked matrix product (torch, float64), and the last state."""
    r = q.shape[1] // k.shape[1]
    k, v, S0 = k.repeat_interleave(r, 1), v.repeat_interleave(r, 1), S0.repeat_interleave(r, 1)
    l = ld.repeat_interleave(r)[None, :, None, None]
    i = torch.arange(q.shape[2], dtype=torch.float64)
    ago = i[:, None] - i[None, :]
    W = torch.where(ago >= 0, torch.exp(l * ago.clamp(min=0)), torch.zeros((), dtype=torch.float64))
    out = scale * (((q @ k.transpose(-1, -2)) * W) @ v + torch.exp(l * (i + 1)[:, None]) * (q @ S0))
    left = torch.exp(l * (i[-1] - i)[:, None])
    S1 = torch.exp(l * len(i)) * S0 + (k * left).transpose(-1, -2) @ v
    return out, S1[:, ::r]


@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 1, 1), (2, 4, 2, 9, 3, 5), (1, 6, 2, 17, 4, 2)])
def test_forward_and_gradient_match_the_quadratic_form(shape):
    q, k, v, go, ld, S0, dS1 = draw(*shape)
    t = [torch.from_numpy(x).requires_grad_() for x in (q, k, v, S0)]
    out, S1 = quadratic(t[0], t[1], t[2], torch.from_numpy(ld), 0.7, t[3])
    ((out * torch.from_numpy(go)).sum() + (S1 * torch.from_numpy(dS1)).sum()).backward()
    got = od.fwd(q, k, v, ld, 0.7, S0)
    grads = od.bwd(q, k, v, go, ld, 0.7, S0, dS1)
    for a, b in zip(got + grads, (out, S1, t[0].grad, t[1].grad, t[2].grad, t[3].grad)):
        np.testing.assert_allclose(a, b.detach().numpy(), rtol=1e-11, atol=1e-11)


def test_gradient_matches_differences():
    q, k, v, go, ld, S0, dS1 = draw(1, 2, 1, 5, 2, 3, seed=3)
    grads = od.bwd(q, k, v, go, ld, 1.3, S0, dS1)

    def loss(args):
        out, S1 = od.fwd(args[0], args[1], args[2], ld, 1.3, args[3])
        return (out * go).sum() + (S1 * dS1).sum()

    for n, x in enumerate((q, k, v, S0)):
        for at in np.ndindex(x.shape):
            vals = []
            for h in (1e-5, -1e-5):
                args = [a.copy() for a in (q, k, v, S0)]
                args[n][at] += h
                vals.append(loss(args))
            assert abs((vals[0] - vals[1]) / 2e-5 - grads[n][at]) < 1e-7


def test_a_sequence_may_be_cut_anywhere_and_lengths_end_it():
    q, k, v, _, ld, S0, _ = draw(2, 2, 2, 11, 3, 3, seed=5)
    whole, last = od.fwd(q, k, v, ld, 1.0, S0)
    for cut in (1, 6, 10):
        a, S = od.fwd(q[:, :, :cut], k[:, :, :cut], v[:, :, :cut], ld, 1.0, S0)
        b, S = od.fwd(q[:, :, cut:], k[:, :, cut:], v[:, :, cut:], ld, 1.0, S)
        np.testing.assert_allclose(np.concatenate([a, b], 2), whole, rtol=1e-12)
        np.testing.assert_allclose(S, last, rtol=1e-12)
    k[1, :, 4:] = np.nan
    out, S = od.fwd(q, k, v, ld, 1.0, S0, np.array([0, 4]))
    assert not out[0].any() and not out[1, :, 4:].any() and np.array_equal(S[0], S0[0])
    np.testing.assert_allclose(out[1, :, :4], whole[1, :, :4], rtol=1e-12)


def test_rotation_and_norm_pins():
    g = np.random.default_rng(1)
    x, go, w = g.standard_normal((2, 3, 4, 16)), g.standard_normal((2, 3, 4, 16)), g.standard_normal(16)
    pos = np.array([[[0, 1, 7, 10 ** 12]] * 2, [[3, 2, 1, 0]] * 2])
    f = 10000.0 ** (-np.arange(8) / 8)
    for inter in (False, True):
        kw = dict(weight=w, eps=1e-3, positions=pos, inv_freq=f, sections=[5, 3], interleaved=inter)
        y = od.qk_fwd(x, **kw)
        # a rotation keeps each row's length, and turning back restores the normed row
        xn = od.qk_fwd(x, weight=w, eps=1e-3)
        np.testing.assert_allclose((y ** 2).sum(-1), (xn ** 2).sum(-1), rtol=1e-12)
        dx, dw, _ = od.qk_bwd(x, go, **kw)
        for at in [(0, 0, 0, 0), (1, 2, 3, 15), (0, 1, 2, 9), (1, 0, 1, 4)]:
            vals = []
            for h in (1e-6, -1e-6):
                xx = x.copy()
                xx[at] += h
                vals.append((od.qk_fwd(xx, **kw) * go).sum())
            assert abs((vals[0] - vals[1]) / 2e-6 - dx[at]) < 1e-7
        for e in (0, 7, 12):
            vals = []
            for h in (1e-6, -1e-6):
                ww = w.copy()
                ww[e] += h
                vals.append((od.qk_fwd(x, **dict(kw, weight=ww)) * go).sum())
            assert abs((vals[0] - vals[1]) / 2e-6 - dw[e]) < 1e-7
    # the product of two turned rows depends on the distance alone
    q, k = g.standard_normal((1, 1, 1, 16)), g.standard_normal((1, 1, 1, 16))
    kw = dict(inv_freq=f, normalize=False)
    dots = [(od.qk_fwd(q, positions=np.array([[a]]), **kw) * od.qk_fwd(k, positions=np.array([[a - 5]]), **kw)).sum()
            for a in (5, 6, 1000)]
    np.testing.assert_allclose(dots, dots[0], rtol=1e-11)


def test_oracle_slips_are_caught():
    """Each planted slip in the recurrence breaks the quadratic form."""
    import inspect
    src = inspect.getsource(od)
    slips = [("S[b] = gamma[0] * S[b] + ", "S[b] = S[b] + "), ("A = gam * A\n", "A = A\n"),
             ("dk[:, :, t] = np.einsum(\"bhde,bhe->bhd\", A, v", "dk[:, :, t] = np.einsum(\"bhde,bhe->bhd\", gam * A, v"),
             ("S = gam * S + ", "S = gam * (S + ")]
    q, k, v, go, ld, S0, dS1 = draw(1, 2, 1, 6, 3, 3, seed=9)
    want = od.fwd(q, k, v, ld, 1.0, S0) + od.bwd(q, k, v, go, ld, 1.0, S0, dS1)
    for a, b in slips:
        assert a in src
        bad = src.replace(a, b)
        if "(S + " in b:
            bad = bad.replace(b + "k[:, :, t, :, None] * v[:, :, t, None, :]", b + "k[:, :, t, :, None] * v[:, :, t, None, :])")
        ns = {"__name__": "slip"}
        exec(compile(bad, "slip", "exec"), ns)
        got = ns["fwd"](q, k, v, ld, 1.0, S0) + ns["bwd"](q, k, v, go, ld, 1.0, S0, dS1)
        assert any(np.abs(x - y).max() > 1e-3 for x, y in zip(got, want)), a
