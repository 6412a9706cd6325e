"""A layer of selective state space scan, as a model trains and serves it, from the library's operators:

    x -> projection -> (x, z) -> short causal convolution -> low-rank step sizes, B, C -> selective scan gated by z -> projection

  forward()   prompts of unequal length in one batch; leaves each sequence's states behind
  step()      the next token of each sequence on pools of such states, captured into a CUDA graph
  backward()  the gradients, from the operators' own backward passes

    python examples/selective_scan.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from efficient_transformer_gb300 import la  # noqa: E402


class SelectiveScan:
    def __init__(self, width=256, E=512, S=16, G=1, W=4, rank=32, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        self.E, self.S, self.G, self.W, self.rank = E, S, G, W, rank
        self.w_in = (rand(2 * E, width) / width ** 0.5).bfloat16()
        self.conv_w, self.conv_b = (rand(E, W) / W ** 0.5).bfloat16(), (0.1 * rand(E)).bfloat16()
        self.w_bc = (rand(2 * G * S, E) / E ** 0.5).bfloat16()
        self.V = (rand(rank, E) / E ** 0.5).bfloat16()
        self.U = (rand(E, rank) / rank ** 0.5).bfloat16()
        self.A_log = torch.arange(1, S + 1, device="cuda", dtype=torch.float32).log().repeat(E, 1)   # A = -exp(A_log) < 0
        self.skip = torch.ones(E, device="cuda")
        d = torch.exp(torch.linspace(-6.9, -2.3, E, device="cuda"))      # steps of 0.001 to 0.1
        self.dt_bias = d + torch.log(-torch.expm1(-d))
        self.w_out = (rand(width, E) / E ** 0.5).bfloat16()

    @property
    def A(self):
        return -torch.exp(self.A_log)

    def params(self):
        return [self.w_in, self.conv_w, self.conv_b, self.w_bc, self.U, self.V, self.A_log, self.skip, self.dt_bias, self.w_out]

    def states(self, n):
        """Pools of n sequences' states: the convolution's last inputs and the scan's h."""
        return (torch.zeros(n, self.W - 1, self.E, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(n, self.E, self.S, device="cuda"))

    def _scan_inputs(self, x):
        dt = la.lowrank_fwd(x, self.U, self.V)
        bc = x @ self.w_bc.T
        return dt, *(t.unflatten(2, (self.G, self.S)) for t in bc.chunk(2, 2))   # B and C: views into one product

    def _vectors(self, z):
        return dict(skip=self.skip, z=z, dt_bias=self.dt_bias)

    def forward(self, u, states=None, lengths=None, train=False):
        """u [B, N, width]; `states` (of states(B)) hold what came before and are brought up to date.  Returns (y, what
        backward() needs)."""
        xz = u @ self.w_in.T
        x, z = xz.chunk(2, 2)                                             # views: read where they lie
        cs, hs = states if states is not None else (None, None)
        xc = la.conv_fwd(x, self.conv_w, self.conv_b, initial_state=cs, final_state=cs, lengths=lengths)
        dt, B, C = self._scan_inputs(xc)
        kept = None
        if train:
            kept = torch.empty(la.ssm_states_size(u.shape[0], u.shape[1], self.E, self.S), dtype=torch.uint8, device="cuda")
        o = la.ssm_fwd(xc, dt, self.A, B, C, **self._vectors(z), initial_state=hs, final_state=hs, lengths=lengths, states=kept)
        return o @ self.w_out.T, (u, x, z, xc, dt, B, C, o, kept)

    def step(self, u, states, slots):
        """One token of each sequence: u [B, 1, width]; sequence b's states are in slot slots[b] of the pools."""
        x, z = (u @ self.w_in.T).chunk(2, 2)
        xc = la.conv_step(x, states[0], self.conv_w, self.conv_b, slots=slots)
        dt, B, C = self._scan_inputs(xc)
        return la.ssm_step(xc, dt, self.A, B, C, states[1], **self._vectors(z), slots=slots) @ self.w_out.T

    def backward(self, saved, grad):
        """Gradients of params(), for a training forward without states."""
        u, x, z, xc, dt, B, C, o, kept = saved
        flat = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
        d_out = flat(grad).T @ flat(o)
        A = self.A
        dxc, ddt, dA, dB, dC, dskip, dz, dbias = la.ssm_bwd(xc, dt, A, B, C, grad @ self.w_out, **self._vectors(z), states=kept)
        dbc = torch.cat([dB.flatten(2), dC.flatten(2)], 2)
        dx2, dU, dV, _ = la.lowrank_bwd(xc, self.U, self.V, ddt)
        dxc = dxc + dbc @ self.w_bc + dx2
        dx, dw, db = la.conv_bwd(x, self.conv_w, dxc, self.conv_b)
        d_in = flat(torch.cat([dx, dz], 2)).T @ flat(u)
        return d_in, dw, db, flat(dbc).T @ flat(xc), dU, dV, dA * A, dskip, dbias, d_out


def serve(layer, B=3, N=200, tokens=24, width=256):
    """Prompts of unequal length, then token by token; the largest distance of the tokens' rows (relative 2-norm)
    from a prompt that held them all."""
    g = torch.Generator(device="cuda").manual_seed(1)
    u = torch.randn(B, N + tokens, width, device="cuda", generator=g).bfloat16()
    lengths = torch.tensor([N - 61 * b for b in range(B)], dtype=torch.int32, device="cuda")
    slots = torch.randperm(B + 2, generator=g, device="cuda")[:B].to(torch.int32)
    pools, states = layer.states(B + 2), layer.states(B)
    layer.forward(u[:, :N].contiguous(), states, lengths)
    for pool, state in zip(pools, states):
        pool[slots.long()] = state

    # the loop's buffers, and one graph of all that a token takes
    token, pos = torch.empty(B, 1, width, dtype=u.dtype, device="cuda"), lengths.long().clone()
    pick = torch.arange(B, device="cuda")
    kept, pos0 = [p.clone() for p in pools], pos.clone()

    def one():
        token.copy_(u[pick, pos][:, None])
        y = layer.step(token, pools, slots)
        pos.add_(1)
        return y

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        one()   # (warm-up; its changes are taken back)
    torch.cuda.current_stream().wait_stream(side)
    for p, k in zip(pools, kept):
        p.copy_(k)
    pos.copy_(pos0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = one()
    rows = []
    for _ in range(tokens):
        graph.replay()
        rows.append(y.clone())
    rows = torch.cat(rows, 1).float()
    full = layer.forward(u)[0].float()
    la.get_status()
    want = torch.stack([full[b, n:n + tokens] for b, n in enumerate(lengths.tolist())])
    return float((rows - want).flatten(1).norm(dim=1).div(want.flatten(1).norm(dim=1)).max())


def train(layer, steps=10, B=2, N=384, width=256, rate=0.02):
    """Gradient steps towards another layer's outputs; the losses."""
    g = torch.Generator(device="cuda").manual_seed(2)
    u = torch.randn(B, N, width, device="cuda", generator=g).bfloat16()
    target = SelectiveScan(width, seed=9).forward(u)[0].float()
    params = layer.params()
    master = [p.float() for p in params]
    losses = []
    for _ in range(steps):
        y, saved = layer.forward(u, train=True)
        err = y.float() - target
        losses.append(float(err.square().mean()))
        for p, m, d in zip(params, master, layer.backward(saved, (err / err.norm()).to(u.dtype))):
            m.sub_(d.float() * (rate * m.norm() / d.float().norm().clamp(min=1e-30)))
            p.copy_(m)
    la.get_status()
    return losses


def main():
    print(f"tokens against the whole prompt: relative difference {serve(SelectiveScan()):.2e}")
    losses = train(SelectiveScan())
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps")


if __name__ == "__main__":
    main()
