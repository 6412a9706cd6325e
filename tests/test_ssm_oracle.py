"""Pins of oracle/ssm.py: gradients against central differences, the bound of float32 arithmetic against float32 arithmetic,
lengths, and a hand-made case."""
import numpy as np
import pytest

from oracle import ssm


def scan_inputs(seed, B=2, N=5, E=8, S=4, G=2, **flags):
    g = np.random.default_rng(seed)
    r = lambda *s: g.standard_normal(s)  # noqa: E731
    a = dict(x=r(B, N, E), dt=r(B, N, E), A=-np.exp(r(E, S)), B=r(B, N, G, S), C=r(B, N, G, S), skip=r(E), z=r(B, N, E),
             dt_bias=r(E), initial_state=r(B, E, S))
    return {k: v for k, v in a.items() if flags.get(k, True)}, r(B, N, E), r(B, E, S)


NAMES = dict(x="dx", dt="ddt", A="dA", B="dB", C="dC", skip="dskip", z="dz", dt_bias="ddt_bias",
             initial_state="grad_initial_state")


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("lengths", [None, [3, 5], [0, 1]])
def test_scan_gradients_against_differences(softplus, lengths):
    a, g, ds = scan_inputs(0)
    kw = dict(use_softplus=softplus, lengths=lengths)

    def loss(**over):
        f = ssm.scan(**dict(a, **over), **kw)
        return (f["out"].v * g).sum() + (f["final_state"].v * ds).sum()

    res = ssm.scan(**a, **kw, grad_out=g, grad_final_state=ds)
    # a difference of two losses divides by 2e-5 what 64-bit arithmetic loses in them: up to 64 operations on a term's way,
    # 2^-53 each (without softplus some states grow, and their terms are large)
    rounding = 64 * 2.0 ** -53 * (np.abs(res["out"].v * g).sum() + np.abs(res["final_state"].v * ds).sum()) / 1e-5
    rng = np.random.default_rng(1)
    for name, grad in NAMES.items():
        way = rng.standard_normal(a[name].shape)
        diff = (loss(**{name: a[name] + 1e-5 * way}) - loss(**{name: a[name] - 1e-5 * way})) / 2e-5
        assert abs(diff - (res[grad].v * way).sum()) < 1e-6 * (1 + abs(diff)) + rounding, name


@pytest.mark.parametrize("missing", [("z",), ("skip", "dt_bias"), ("initial_state",)])
def test_scan_without_some_inputs(missing):
    a, g, ds = scan_inputs(2, **{m: False for m in missing})
    full, _, _ = scan_inputs(2)
    res = ssm.scan(**a, grad_out=g, grad_final_state=ds)
    for m in missing:
        if m != "initial_state":
            assert res[NAMES[m]] is None
            full[m] = np.full_like(full[m], 1e3) if m == "z" else np.zeros_like(full[m])
        else:
            full[m] = np.zeros_like(full[m])
    want = ssm.scan(**full, grad_out=g / 1e3 if "z" in missing else g, grad_final_state=ds)
    assert np.allclose(res["out"].v * (1e3 if "z" in missing else 1.0), want["out"].v)
    assert np.allclose(res["dA"].v, want["dA"].v)


def test_scan_by_hand():
    # one channel of one state, decays of a half: d = 1, A = -ln 2
    one = np.ones((1, 3, 1))
    res = ssm.scan(one, one, [[-np.log(2.0)]], [[[[1.0]], [[2.0]], [[4.0]]]], np.ones((1, 3, 1, 1)), skip=[0.5], use_softplus=False,
                   initial_state=[[[8.0]]])
    assert np.allclose(res["out"].v[0, :, 0], [5.5, 5.0, 6.75])
    assert np.allclose(res["final_state"].v, 6.25)


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("lengths", [None, [0, 5], [2, 1]])
def test_conv_gradients_against_differences(silu, lengths):
    g = np.random.default_rng(3)
    r = lambda *s: g.standard_normal(s)  # noqa: E731
    B, N, E, W = 2, 5, 3, 4
    a = dict(x=r(B, N, E), weight=r(E, W), bias=r(E), initial_state=r(B, W - 1, E))
    go, ds = r(B, N, E), r(B, W - 1, E)

    def loss(**over):
        f = ssm.conv(**dict(a, **over), silu=silu, lengths=lengths)
        return (f["out"].v * go).sum() + (f["final_state"].v * ds).sum()

    res = ssm.conv(**a, silu=silu, lengths=lengths, grad_out=go, grad_final_state=ds)
    for name, grad in dict(x="dx", weight="dweight", bias="dbias", initial_state="grad_initial_state").items():
        way = r(*a[name].shape)
        diff = (loss(**{name: a[name] + 1e-5 * way}) - loss(**{name: a[name] - 1e-5 * way})) / 2e-5
        assert abs(diff - (res[grad].v * way).sum()) < 1e-6 * (1 + abs(diff)), name


def test_conv_by_hand():
    res = ssm.conv([[[1.0], [2.0], [3.0]]], [[10.0, 1.0]], [0.5], silu=False, initial_state=[[[7.0]]], lengths=[2])
    assert np.allclose(res["out"].v[0, :, 0], [71.5, 12.5, 0.0])
    assert np.allclose(res["final_state"].v, 2.0)


def test_the_bound_holds_for_float32_and_finds_a_mistake():
    a, g, ds = scan_inputs(4, B=1, N=40, E=8, S=8, G=1)
    a = {k: v.astype(np.float32) for k, v in a.items()}
    want = ssm.scan(**a)
    f = np.float32
    h, out = a["initial_state"].copy(), []
    for t in range(40):
        d = np.log1p(np.exp((a["dt"][:, t] + a["dt_bias"]).astype(f))).astype(f)
        h = np.exp(d[..., None] * a["A"]).astype(f) * h + (d * a["x"][:, t])[..., None] * a["B"][:, t]
        y = (h * a["C"][:, t]).sum(-1) + a["skip"] * a["x"][:, t]
        out.append(y * (a["z"][:, t] / (1 + np.exp(-a["z"][:, t]))))
    out = np.stack(out, 1)
    assert out.dtype == f and ssm.distance(out, want["out"], 2.0 ** -23) <= 1
    assert ssm.distance(h, want["final_state"], 2.0 ** -23) <= 1
    h[0, 3, 2] *= 1 + 1e-4
    assert ssm.distance(h, want["final_state"], 2.0 ** -23) > 1
