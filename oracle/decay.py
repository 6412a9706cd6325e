"""Float64 CPU oracle of the decayed linear attention, token by token, and of the query/key norm
with its position rotation (test infrastructure; shares no code with the GPU path).

    S_i = gamma S_{i-1} + k_i v_i^T,   out_i = scale q_i^T S_i,   gamma = exp(log_decay[head])
    A_i = scale q_i g_i^T + gamma A_{i+1}:  dq_i = scale S_i g_i, dk_i = A_i v_i, dv_i = A_i^T k_i

Query head h reads key/value head h // n_rep.  Arrays are [B, H, N, D]; a sequence b has
lengths[b] tokens (None: N); rows past them are not read and come out as zeros.
"""
from __future__ import annotations

import numpy as np


def _np(t):
    if t is None:
        return None
    if hasattr(t, "detach"):
        t = t.detach().to("cpu")
        t = t.double().numpy() if t.is_floating_point() else t.numpy()
    return np.asarray(t)


def _setup(q, k, v, log_decay, initial_state, lengths):
    q, k, v, ld, S0, n = (_np(x) for x in (q, k, v, log_decay, initial_state, lengths))
    B, Hq, N, D = q.shape
    Hkv, Dv = k.shape[1], v.shape[3]
    with np.errstate(over="ignore"):
        gamma = np.exp(ld.astype(np.float64))[None, :, None, None]
    S0 = np.zeros((B, Hkv, D, Dv)) if S0 is None else S0.astype(np.float64)
    n = np.full(B, N) if n is None else np.clip(n.astype(np.int64), 0, N)
    return q.reshape(B, Hkv, Hq // Hkv, N, D), k, v, gamma, S0, n


def fwd(q, k, v, log_decay, scale=1.0, initial_state=None, lengths=None):
    """(out [B, Hq, N, Dv], final state [B, Hkv, D, Dv])."""
    q, k, v, gamma, S, n = _setup(q, k, v, log_decay, initial_state, lengths)
    B, Hkv, r, N, _ = q.shape
    S = S.copy()
    out = np.zeros((B, Hkv, r, N, v.shape[3]))
    for t in range(N):
        for b in np.flatnonzero(t < n):
            S[b] = gamma[0] * S[b] + k[b, :, t, :, None] * v[b, :, t, None, :]
            out[b, :, :, t] = scale * np.einsum("hrd,hde->hre", q[b, :, :, t], S[b])
    return out.reshape(B, Hkv * r, N, -1), S


def bwd(q, k, v, grad_out, log_decay, scale=1.0, initial_state=None, grad_final_state=None):
    """(dq, dk, dv, gradient of the initial state)."""
    q, k, v, gamma, S, _ = _setup(q, k, v, log_decay, initial_state, None)
    B, Hkv, r, N, D = q.shape
    g = _np(grad_out).reshape(B, Hkv, r, N, -1)
    S, gam = S.copy(), gamma
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    for t in range(N):
        S = gam * S + k[:, :, t, :, None] * v[:, :, t, None, :]
        dq[:, :, :, t] = scale * np.einsum("bhre,bhde->bhrd", g[:, :, :, t], S)
    A = np.zeros_like(S) if grad_final_state is None else _np(grad_final_state).astype(np.float64).copy()
    for t in range(N - 1, -1, -1):
        A = A + scale * np.einsum("bhrd,bhre->bhde", q[:, :, :, t], g[:, :, :, t])
        dk[:, :, t] = np.einsum("bhde,bhe->bhd", A, v[:, :, t])
        dv[:, :, t] = np.einsum("bhde,bhd->bhe", A, k[:, :, t])
        A = gam * A
    return dq.reshape(B, Hkv * r, N, D), dk, dv, A


def _angles(positions, inv_freq, sections):
    pos, f = _np(positions), _np(inv_freq).astype(np.float64)
    pos = pos[None] if pos.ndim == 2 else pos
    axis = np.repeat(np.arange(len(pos)), [len(f)] if sections is None else sections)
    # positions times doubles, reduced mod 2 pi in extended precision
    a = pos[axis].astype(np.longdouble) * f.astype(np.longdouble)[:, None, None]
    return np.moveaxis(np.remainder(a, 2 * np.longdouble("3.14159265358979323846264338327950288")), 0, -1).astype(np.float64)


def _rotate(x, angle, interleaved, back=False):
    """x [B, H, N, D], its pairs turned by angle [B, N, pairs] (the other way with `back`)."""
    R = 2 * angle.shape[-1]
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None] * (-1.0 if back else 1.0)
    i, j = (np.arange(0, R, 2), np.arange(1, R, 2)) if interleaved else (np.arange(R // 2), np.arange(R // 2, R))
    y = x.copy()
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., i] * s + x[..., j] * c
    return y


def qk_fwd(x, weight=None, eps=1e-6, positions=None, inv_freq=None, sections=None, interleaved=False, normalize=True):
    """One of q and k."""
    x = _np(x)
    if normalize:
        x = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
        x = x if weight is None else x * _np(weight)
    return x if inv_freq is None else _rotate(x, _angles(positions, inv_freq, sections), interleaved)


def qk_bwd(x, grad, weight=None, eps=1e-6, positions=None, inv_freq=None, sections=None, interleaved=False,
           normalize=True):
    """(gradient of x, gradient of the weight, the sum of the absolute terms of the latter)."""
    x, u = _np(x), _np(grad)
    if inv_freq is not None:
        u = _rotate(u, _angles(positions, inv_freq, sections), interleaved, back=True)
    if not normalize:
        return u, None, None
    r = 1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    xh = x * r
    uw = u if weight is None else u * _np(weight)
    return r * (uw - xh * np.mean(uw * xh, -1, keepdims=True)), (u * xh).sum((0, 1, 2)), np.abs(u * xh).sum((0, 1, 2))
