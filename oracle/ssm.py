"""Float64 CPU oracle of the selective state space scan and of the short causal convolution, token by token, with a
running bound of what float32 arithmetic may lose on the way (test infrastructure; shares no code with the GPU path).

    d = softplus(dt + dt_bias), h_t = exp(d_t A) h_(t-1) + d_t x_t B_t, out_t = (C_t . h_t + skip x_t) z_t sigmoid(z_t)
    out_t = act(bias + sum_j weight_j x_(t - W + 1 + j))

Every number is a pair (v, e): its value in 64 bits, and how far the same operations in float32, each rounded to nearest,
can be from it to first order: e(a b) = |a| e(b) + |b| e(a) + U |a b| and so on, U = 2^-24.  Sums of n terms may be taken in
any order: n U of their absolute terms.  exp, softplus and 1 / x as the GPU has them err by up to 2.5 U, 3 U and 2 U.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24


class Num:
    __slots__ = ("v", "e")
    __array_ufunc__ = None

    def __init__(self, v, e=None):
        self.v = np.asarray(v, np.float64)
        self.e = np.zeros_like(self.v) if e is None else np.asarray(e, np.float64)

    def __add__(self, o):
        o = o if isinstance(o, Num) else Num(o)
        v = self.v + o.v
        return Num(v, self.e + o.e + U * np.abs(v))

    __radd__ = __add__

    def __mul__(self, o):
        o = o if isinstance(o, Num) else Num(o)
        v = self.v * o.v
        return Num(v, np.abs(self.v) * o.e + np.abs(o.v) * self.e + U * np.abs(v))

    __rmul__ = __mul__

    def __sub__(self, o):
        return self + o * -1.0 if isinstance(o, Num) else self + (-o)

    def __getitem__(self, i):
        return Num(self.v[i], self.e[i])

    def sum(self, axis):
        n = int(np.prod([self.v.shape[a] for a in np.atleast_1d(axis)]))
        return Num(self.v.sum(axis), self.e.sum(axis) + n * U * np.abs(self.v).sum(axis))

    def reshape(self, *s):
        return Num(self.v.reshape(*s), self.e.reshape(*s))


def _np(t):
    if t is None:
        return None
    if hasattr(t, "detach"):
        t = t.detach().to("cpu")
        t = t.double().numpy() if t.is_floating_point() else t.numpy()
    return np.asarray(t)


def _num(t):
    return None if t is None else Num(_np(t))


def stack(rows, axis=1):
    return Num(np.stack([r.v for r in rows], axis), np.stack([r.e for r in rows], axis))


def where(c, a, b):
    a, b = (x if isinstance(x, Num) else Num(np.broadcast_to(np.float64(x), np.shape(c))) for x in (a, b))
    return Num(np.where(c, a.v, b.v), np.where(c, a.e, b.e))


def exp(a):
    # (the argument meets log2(e) first: one more rounding of it; results below 2^-126, the smallest normal float32, are
    # flushed to zero: off by at most that)
    v = np.exp(a.v)
    return Num(v, v * (a.e + 2 * U * np.abs(a.v) + 2.5 * U) + 2.0 ** -126)


def sigmoid(a):
    with np.errstate(over="ignore"):
        v = 1.0 / (1.0 + np.exp(-a.v))
    # 1 / (1 + E), E = exp(-a) off by r relative: r E / (1 + E) = r (1 - v), a sum and a reciprocal
    r = a.e + 2 * U * np.abs(a.v) + 2.5 * U
    return Num(v, v * ((1 - v) * r + 3 * U))


def softplus(a):
    v = np.logaddexp(0.0, a.v)
    s = sigmoid(Num(a.v)).v
    # what enters: a, with slope sigmoid; E = exp(-|a|) off by 2.5 U + 2 U |a|; log(1 + E) by 3 U; one sum
    E = np.exp(-np.abs(a.v))
    return Num(v, s * a.e + np.log1p(E) * (2 * U * np.abs(a.v) + 5.5 * U) + U * v)


def _lengths(lengths, B, N):
    return np.full(B, N) if lengths is None else np.clip(_np(lengths).astype(np.int64), 0, N)


def conv(x, weight, bias=None, silu=True, initial_state=None, lengths=None, grad_out=None, grad_final_state=None):
    """dict of out and final_state, and with grad_out of dx, dweight, dbias and grad_initial_state."""
    x, w, bias, g, df = _np(x), _num(weight), _num(bias), _np(grad_out), _np(grad_final_state)
    B, N, E = x.shape
    W = w.v.shape[1]
    n = _lengths(lengths, B, N)
    first = np.zeros((B, W - 1, E)) if initial_state is None else _np(initial_state)
    res = {k: [] for k in ("out", "final_state", "dx", "grad_initial_state")}
    dw, db = Num(np.zeros((E, W))), Num(np.zeros(E))
    for b in range(B):
        rows = np.concatenate([first[b], x[b, :n[b]]])
        out, gp = Num(np.zeros((N, E))), Num(np.zeros((n[b] + 2 * (W - 1), E)))
        for t in range(n[b]):
            v = stack([Num(rows[t + j]) * w[:, j] for j in range(W)], 0).sum(0)
            v = v if bias is None else v + bias
            s = sigmoid(v)
            o = v * s if silu else v
            out.v[t], out.e[t] = o.v, o.e
            if g is not None:
                d = Num(g[b, t])
                if silu:
                    d = d * s * (1.0 + v * Num(1.0 - s.v, s.e + U))
                gp.v[t + W - 1], gp.e[t + W - 1] = d.v, d.e
                db = db + d
                dw = dw + stack([Num(rows[t + j]) * d for j in range(W)], 1)
        res["out"].append(out)
        res["final_state"].append(Num(rows[n[b]:]))
        if g is not None:
            # row p of `rows` (token p - W + 1) meets token t through weight j = p - t
            d = [stack([w[:, j] * gp[p - j + W - 1] for j in range(W)], 0).sum(0) for p in range(n[b] + W - 1)]
            if df is not None:
                for i in range(W - 1):
                    d[n[b] + i] = d[n[b] + i] + Num(df[b, i])
            zero = Num(np.zeros(E))
            res["grad_initial_state"].append(stack(d[:W - 1], 0))
            res["dx"].append(stack(d[W - 1:] + [zero] * (N - n[b]), 0))
    res = {k: stack(v, 0) for k, v in res.items() if v}
    if g is not None:
        res.update(dweight=dw, dbias=db if bias is not None else None)
    return res


def scan(x, dt, A, B, C, skip=None, z=None, dt_bias=None, use_softplus=True, initial_state=None, lengths=None,
         grad_out=None, grad_final_state=None):
    """dict of out and final_state, and with grad_out of dx, ddt, dA, dB, dC, dskip, dz, ddt_bias and
    grad_initial_state (those of missing inputs None)."""
    x, dt, Bm, Cm, z, g = (_num(t) for t in (x, dt, B, C, z, grad_out))
    A, skip, bias = _num(A), _num(skip), _num(dt_bias)
    nB, N, E = x.v.shape
    G, S = Bm.v.shape[2:]
    r = E // G
    n = _lengths(lengths, nB, N)
    h = Num(np.zeros((nB, E, S))) if initial_state is None else _num(initial_state)

    def wide(m, t):
        return Num(np.repeat(m.v[:, t], r, 1), np.repeat(m.e[:, t], r, 1))

    def zeros_past(a, on):
        return Num(np.where(on, a.v, 0.0), np.where(on, a.e, 0.0))

    keep, outs = [], []
    for t in range(N):
        on = (t < n)[:, None]
        xt, v = zeros_past(x[:, t], on), zeros_past(dt[:, t], on)
        v = v if bias is None else v + bias
        d = zeros_past(softplus(v) if use_softplus else v, on)
        zt = None if z is None else zeros_past(z[:, t], on)
        b, c = (Num(np.where(on[..., None], m.v, 0.0)) for m in (wide(Bm, t), wide(Cm, t)))
        a = exp(d[..., None] * A)
        a = where(np.broadcast_to(on[..., None], a.v.shape), a, 1.0)
        u = d * xt
        h0, h = h, a * h + u[..., None] * b
        y = (h * c).sum(2)
        y = y if skip is None else y + skip * xt
        o = y if zt is None else y * (zt * sigmoid(zt))
        outs.append(zeros_past(o, on))
        keep.append((on, xt, v, d, zt, b, c, a, u, h0, h, y))
    res = {"out": stack(outs), "final_state": h}
    if g is None:
        return res
    P = Num(np.zeros((nB, E, S))) if grad_final_state is None else _num(grad_final_state)
    rows = {k: [] for k in ("dx", "ddt", "dB", "dC", "dz")}
    dA, dskip, dbias = [], [], []
    for t in range(N - 1, -1, -1):
        on, xt, v, d, zt, b, c, a, u, h0, h1, y = keep[t]
        gt = zeros_past(g[:, t], on)
        dy = gt
        if zt is not None:
            s = sigmoid(zt)
            rows["dz"].append(zeros_past(gt * y * s * (1.0 + zt * Num(1.0 - s.v, s.e + U)), on))
            dy = gt * (zt * s)
        rows["dC"].append((dy[..., None] * h1).reshape(nB, G, r, S).sum(2))
        gh = P + dy[..., None] * c
        rows["dB"].append((gh * u[..., None]).reshape(nB, G, r, S).sum(2))
        P = a * gh
        q = P * h0
        du = (gh * b).sum(2)
        # (A meets ln 2 and log2(e) on its way)
        qa = (q * A).sum(2)
        dd = Num(qa.v, qa.e + 3 * U * np.abs(qa.v)) + xt * du
        dA.append((q * d[..., None]).sum(0))
        dx = d * du
        if skip is not None:
            dx = dx + skip * dy
            dskip.append((dy * xt).sum(0))
        ddt = zeros_past(dd * sigmoid(v) if use_softplus else dd, on)
        dbias.append(ddt.sum(0))
        rows["dx"].append(zeros_past(dx, on))
        rows["ddt"].append(ddt)
    for k, v in rows.items():
        res[k] = stack(v[::-1]) if v else None
    res.update(dA=stack(dA, 0).sum(0), dskip=stack(dskip, 0).sum(0) if skip is not None else None,
               ddt_bias=stack(dbias, 0).sum(0) if bias is not None else None, grad_initial_state=P)
    return res


def distance(got, want, dtype_eps):
    """The largest |got - want| in units of what it may be: twice the float32 bound (first order doubled), and half a step
    of the output's type (dtype_eps = torch.finfo(type).eps) of the value, and the smallest float32 values."""
    got = _np(got)
    assert got.shape == want.v.shape, (got.shape, want.v.shape)
    assert np.all(np.isfinite(got))
    room = 2 * want.e + dtype_eps / 2 * (np.abs(want.v) + 2 * want.e) + 1e-37
    return float(np.max(np.abs(got - want.v) / room)) if got.size else 0.0
