"""A layer of linear attention with decay, as a model trains and serves it, from the library's operators:

    x -> low-rank projection -> q, k, v -> norm of q and k with rotation -> decayed attention -> projection

  forward()   prompts of unequal length in one batch; leaves each sequence's state behind
  step()      the next token of each sequence on a pool of such states, captured into a CUDA graph
  backward()  the gradients, from the operators' own backward passes

    python examples/decayed_attention.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from efficient_transformer_gb300 import la  # noqa: E402


class DecayedAttention:
    def __init__(self, width=512, rank=128, Hq=8, Hkv=2, D=64, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        self.Hq, self.Hkv, self.D = Hq, Hkv, D
        self.V = (rand(rank, width) / width ** 0.5).bfloat16()
        self.U = (rand((Hq + 2 * Hkv) * D, rank) / rank ** 0.5).bfloat16()
        self.q_weight, self.k_weight = torch.ones(D, device="cuda"), torch.ones(D, device="cuda")
        self.out_weight = (rand(width, Hq * D) / (Hq * D) ** 0.5).bfloat16()
        self.inv_freq = 10000.0 ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)
        self.log_decay = torch.log1p(-2.0 ** -torch.linspace(4, 8, Hkv, device="cuda"))   # memories of 16 to 256 tokens

    def _qkv(self, x, positions):
        """q, k (normed and turned) and v: heads of one projection's rows, views that are read where they lie."""
        y = la.lowrank_fwd(x, self.U, self.V).view(*x.shape[:2], -1, self.D).transpose(1, 2)
        q, k, v = y.split([self.Hq, self.Hkv, self.Hkv], 1)
        return (q, k, v) + la.qk_norm_rope_fwd(q, k, **self._rope(positions))

    def _rope(self, positions):
        return dict(q_weight=self.q_weight, k_weight=self.k_weight, positions=positions, inv_freq=self.inv_freq)

    def _project(self, o):
        B, H, N, D = o.shape
        return o.transpose(1, 2).reshape(B, N, H * D) @ self.out_weight.T

    def forward(self, x, positions, state=None, lengths=None):
        """x [B, N, width], positions int64 [B, N]; state [B, Hkv, D, D] float32 holds what came before and is
        brought up to date.  Returns (y, what backward() needs)."""
        q, k, v, qr, kr = self._qkv(x, positions)
        o = la.decay_fwd(qr, kr, v, self.log_decay, scale=self.D ** -0.5, initial_state=state, final_state=state,
                         lengths=lengths)
        return self._project(o), (x, positions, q, k, v, qr, kr, o)

    def step(self, x, positions, pool, slots):
        """One token of each sequence: x [B, 1, width]; sequence b's state is slot slots[b] of the pool."""
        _, _, v, qr, kr = self._qkv(x, positions)
        return self._project(la.decay_step(qr, kr, v, pool, self.log_decay, slots=slots, scale=self.D ** -0.5))

    def backward(self, saved, grad):
        """Gradients of (V, U, q_weight, k_weight, out_weight), for a forward without a state."""
        x, positions, q, k, v, qr, kr, o = saved
        B, N, _ = x.shape
        rows = o.transpose(1, 2).reshape(B * N, -1)
        d_out = grad.reshape(B * N, -1).T @ rows
        go = (grad @ self.out_weight).view(B, N, self.Hq, self.D).transpose(1, 2)
        gq, gk, gv = la.decay_bwd(qr, kr, v, go, self.log_decay, scale=self.D ** -0.5)
        dq, dk, dqw, dkw = la.qk_norm_rope_bwd(q, k, gq, gk, **self._rope(positions))
        dy = torch.cat([dq, dk, gv], 1).transpose(1, 2).reshape(B, N, -1)
        _, dU, dV, _ = la.lowrank_bwd(x, self.U, self.V, dy)
        return dV, dU, dqw, dkw, d_out


def serve(layer, B=3, N=200, tokens=24, width=512):
    """Prompts of unequal length, then token by token; the largest distance of the tokens' rows (relative 2-norm)
    from a prompt that held them all."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(B, N + tokens, width, device="cuda", generator=g).bfloat16()
    lengths = torch.tensor([N - 61 * b for b in range(B)], dtype=torch.int32, device="cuda")
    slots = torch.randperm(B + 2, generator=g, device="cuda")[:B].to(torch.int32)
    pool = torch.zeros(B + 2, layer.Hkv, layer.D, layer.D, device="cuda")
    at = torch.arange(N + tokens, device="cuda").expand(B, -1)
    states = torch.zeros(B, layer.Hkv, layer.D, layer.D, device="cuda")
    layer.forward(x[:, :N].contiguous(), at[:, :N], states, lengths)
    pool[slots.long()] = states

    # the loop's buffers, and one graph of all that a token takes
    token, pos = torch.empty(B, 1, width, dtype=x.dtype, device="cuda"), lengths.long()[:, None].clone()
    pick = torch.arange(B, device="cuda")
    kept, pos0 = pool.clone(), pos.clone()

    def one():
        token.copy_(x[pick, pos[:, 0]][:, None])
        y = layer.step(token, pos, pool, slots)
        pos.add_(1)
        return y

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        one()   # (warm-up; its changes are taken back)
    torch.cuda.current_stream().wait_stream(side)
    pool.copy_(kept)
    pos.copy_(pos0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = one()
    rows = []
    for _ in range(tokens):
        graph.replay()
        rows.append(y.clone())
    rows = torch.cat(rows, 1).float()
    full = layer.forward(x, at)[0].float()
    la.get_status()
    want = torch.stack([full[b, n:n + tokens] for b, n in enumerate(lengths.tolist())])
    return float((rows - want).flatten(1).norm(dim=1).div(want.flatten(1).norm(dim=1)).max())


def train(layer, steps=20, B=2, N=384, width=512, rate=0.05):
    """Gradient steps towards another layer's outputs; the losses."""
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(B, N, width, device="cuda", generator=g).bfloat16()
    at = torch.arange(N, device="cuda").expand(B, -1)
    target = DecayedAttention(width, seed=9).forward(x, at)[0].float()
    params = [layer.V, layer.U, layer.q_weight, layer.k_weight, layer.out_weight]
    master = [p.float() for p in params]
    losses = []
    for _ in range(steps):
        y, saved = layer.forward(x, at)
        err = y.float() - target
        losses.append(float(err.square().mean()))
        for p, m, d in zip(params, master, layer.backward(saved, (err / err.norm()).to(x.dtype))):
            m.sub_(d.float() * (rate * m.norm() / d.float().norm().clamp(min=1e-30)))
            p.copy_(m)
    la.get_status()
    return losses


def main():
    print(f"tokens against the whole prompt: relative difference {serve(DecayedAttention()):.2e}")
    losses = train(DecayedAttention())
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps")


if __name__ == "__main__":
    main()
