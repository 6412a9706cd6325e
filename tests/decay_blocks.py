"""The decayed attention in float64 from its quadratic form, with autograd for its gradients, and a measure of how far
rows are off that a lost or misplaced carry cannot hide in: the relative 2-norm of each head's rows in blocks of 128 tokens."""
import torch

# Rounding to bfloat16 leaves 2^-8 of a value at worst and, uniformly spread over a step, 2^-8 / sqrt(3) and the mean of
# a significand's inverse (0.72): 1.6e-3 of it in the mean square.  A row of random terms takes two independent such
# roundings (a score or a decayed y of each term, the result): 2.3e-3 of its norm.  Three times that:
LIMIT = 7e-3


def forward(q, k, v, ld, scale=1.0, S0=None, n=None):
    """(out, final state) of float64 tensors [B, H, N, D]; n: tokens of each sequence."""
    B, Hq, N, D = q.shape
    r = Hq // k.shape[1]
    i = torch.arange(N, device=q.device, dtype=torch.float64)
    n = torch.full((B,), N, device=q.device) if n is None else n.clamp(0, N)
    ok = (i[None] < n[:, None])                                             # [B, N]
    ahead = (i[:, None] - i[None]).clamp(min=0)
    w = torch.exp(ld.double()[:, None, None] * ahead).tril()                # [Hkv, N, N]
    kk, vv = (torch.where(ok[:, None, :, None], t, torch.zeros_like(t)) for t in (k, v))
    qq = torch.where(ok[:, None, :, None], q, torch.zeros_like(q)).view(B, -1, r, N, D)
    P = torch.einsum("bhrid,bhjd->bhrij", qq, kk) * w[:, None]
    out = scale * torch.einsum("bhrij,bhje->bhrie", P, vv)
    left = torch.exp(ld.double()[None, :, None] * (n[:, None, None] - 1 - i).clamp(min=0))     # [B, Hkv, N]
    S1 = torch.einsum("bhjd,bhje->bhde", kk * left[..., None], vv)
    if S0 is not None:
        g = torch.exp(ld.double()[:, None] * (i + 1))                       # [Hkv, N]
        out = out + scale * torch.einsum("bhrid,bhde->bhrie", qq * g[:, None, :, None], S0)
        S1 = S1 + torch.exp(ld.double()[None] * n[:, None])[..., None, None] * S0
    return out.reshape(B, Hq, N, -1), S1


def reference(q, k, v, go, ld, scale=1.0, S0=None, dS1=None):
    """out, final state, dq, dk, dv, gradient of the initial state (None without S0)."""
    t = [x.double().detach().clone().requires_grad_() for x in (q, k, v)] + ([S0.double().clone().requires_grad_()] if S0 is not None else [])
    out, S1 = forward(*t[:3], ld, scale, t[3] if S0 is not None else None)
    loss = (out * go.double()).sum() + (0.0 if dS1 is None else (S1 * dS1.double()).sum())
    grads = torch.autograd.grad(loss, t)
    return [out.detach(), S1.detach(), *grads] + ([None] if S0 is None else [])


def block_errors(got, want, block=128):
    """Relative 2-norm of [B, H, N, W] rows in blocks of tokens: [B, H, blocks]; blocks of zeros have to be zeros.  Blocks are
    whole (the last one is the last 128 tokens): a single row's terms may cancel, so that its roundings, which are relative to
    the terms, are more of it."""
    N = got.shape[2]
    at = [t if t + block <= N else max(N - block, 0) for t in range(0, N, block)]
    cut = [(got[:, :, t:t + block].double(), want[:, :, t:t + block].double()) for t in at]
    e = [((g - w).norm(dim=(2, 3)), w.norm(dim=(2, 3)), g.norm(dim=(2, 3))) for g, w in cut]
    return torch.stack([torch.where(w > 0, d / w.clamp(min=1e-300), torch.where(g > 0, torch.inf, 0.0)) for d, w, g in e], 2)


def close(got, want, limit=LIMIT):
    e = block_errors(got, want)
    return bool(torch.isfinite(got).all()) and float(e.max()) <= limit
