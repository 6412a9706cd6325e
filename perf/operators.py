"""Decayed linear attention and its query/key preparation, as a program uses them.

The operators (state S of one key/value head: D x Dv, float32; decay g = exp(log_decay)):

* ``prompt``: the chunked form, out_i = scale sum_{j <= i} g^(i-j) (q_i . k_j) v_j
  + scale g^(i+1) q_i S_0, and the state after the last token;
* ``train``: its gradient, (dq, dk, dv) and the gradient of the starting state;
* ``step``: the recurrent form for one token, S <- g S + k v^T, out = scale q S, on a pool of
  states addressed by slot;
* ``prepare_qk``: RMS norm of every query and key head, then the rotation of positions with
  one or several axes, in one pass; ``prepare_qk_train``: its gradient with the weights'.

``listed()`` gives the measured cases, ``draw(rng)`` one more of their ranges, ``prepare``
the inputs of a case, ``run`` one pass, ``work`` what a pass cannot do without and ``exact``
the outputs in 64 bits from the definition.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_BASE = 10000.0
_EPS = 1e-6


def _case(op, B, Hq, Hkv, N, D, dtype="bf16", Dv=None, state=False, ragged=False, axes=1, rot=None,
          interleaved=False, weights=True, fused=True, spare=0):
    """A case: `state`: a starting state comes in and the last one goes out; `ragged`: the
    sequences of the batch have lengths of their own; `axes`, `rot`: position axes and rotated
    width; `fused`: inputs are views into one projection [B, N, heads, D]; `spare`: pool slots
    that no sequence of this call uses."""
    return {"op": op, "B": B, "Hq": Hq, "Hkv": Hkv, "N": N, "D": D, "Dv": D if Dv is None else Dv, "dtype": dtype,
            "state": state, "ragged": ragged, "axes": axes, "rot": D if rot is None else rot,
            "interleaved": interleaved, "weights": weights, "fused": fused, "spare": spare}


def listed():
    def named(name, *a, **k):
        return dict(_case(*a, **k), name=name)

    return [
        # the small float32 workload of the attention tests and benchmark: launch latency
        named("prompt_small_f32", "prompt", 1, 2, 2, 256, 32, "f32", state=True, fused=False),
        # the benchmark's 4 x 16-head training shape, as a forward
        named("prompt_b4_h16_n4096_d64", "prompt", 4, 16, 16, 4096, 64),
        # prompts of unequal length in one batch, states going on to the decoder, Dv < D
        named("prompt_ragged_states", "prompt", 7, 12, 4, 1537, 128, Dv=64, state=True, ragged=True),
        # one very long prompt, 32 query heads on 8 key/value heads
        named("prompt_gqa_n65536_d128", "prompt", 1, 32, 8, 65536, 128, state=True),
        # a short ragged float32 training shape with shared heads and a starting state
        named("train_f32_n777", "train", 2, 6, 2, 777, 64, "f32", state=True),
        # the benchmark's 2 x 16-head, N 8192 training shape
        named("train_b2_h16_n8192_d128", "train", 2, 16, 16, 8192, 128),
        # one user, one token: launch latency
        named("step_b1", "step", 1, 16, 16, 1, 128),
        # a full decoding batch on 32 / 8 heads, its slots scattered over a larger pool
        named("step_b192_gqa", "step", 192, 32, 8, 1, 128, spare=61),
        # queries and keys of a decoding batch
        named("qk_decode_b64", "prepare_qk", 64, 32, 8, 1, 128),
        # the long prompt's queries and keys, three position axes (time, height, width)
        named("qk_3axes_n65536", "prepare_qk", 1, 32, 8, 65536, 128, axes=3),
        # gradient at the 4 x 16-head training shape
        named("qk_train_b4_h16_n4096_d64", "prepare_qk_train", 4, 16, 16, 4096, 64),
        # odd length, partial interleaved rotation, float32, two axes (an image's rows and columns)
        named("qk_train_f32_partial", "prepare_qk_train", 3, 5, 5, 1001, 128, "f32", axes=2, rot=64,
              interleaved=True),
    ]


def _limit(op):
    """The largest listed work of an operator: what a drawn case stays below."""
    w = [work(c) for c in listed() if c["op"] == op]
    return max(x["bytes"] for x in w), max(x["flops"] for x in w)


def draw(rng):
    def log_int(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))

    while True:
        op = rng.choice(["prompt", "prompt", "train", "train", "step", "prepare_qk", "prepare_qk_train"])
        Hkv = log_int(1, 16)
        rep = rng.choice([1, 1, 2, 3, 4, 5, 8])
        D = rng.choice([64, 128]) if rng.random() < 0.85 else 32
        Dv = D if rng.random() < 0.7 else rng.choice([64, 128])
        dtype = "bf16" if rng.random() < 0.8 else "f32"
        N = 1 if op == "step" else log_int(1, 65536 if op != "train" else 16384)
        B = log_int(1, 256 if op == "step" else 8)
        c = _case(op, B, Hkv * rep, Hkv, N, D, dtype, Dv=Dv, fused=rng.random() < 0.6)
        if op in ("prompt", "train"):
            c["state"] = rng.random() < 0.5
            c["ragged"] = op == "prompt" and B > 1 and rng.random() < 0.4
        if op == "step":
            c["spare"] = rng.randrange(0, 40)
        if op.startswith("prepare_qk"):
            c["Dv"] = D
            c["rot"] = D if rng.random() < 0.6 else rng.choice([r for r in (16, 32, 64, 96) if r <= D])
            c["axes"] = rng.choice([1, 1, 2, 3])
            c["interleaved"] = rng.random() < 0.4
            c["weights"] = rng.random() < 0.8
        w, (most_b, most_f) = work(c), _limit(op)
        # float32 prompts run on the CUDA cores: kept to a quarter of the long bfloat16 one
        part = 0.25 if dtype == "f32" and op in ("prompt", "train") else 1.0
        if w["bytes"] <= part * most_b and w["flops"] <= part * most_f:
            return c


def _log_decay(H, device, dtype=torch.float32):
    """Decays from 1 - 2^-1 (a few tokens) to 1 - 2^-11 (thousands), evenly in the exponent."""
    x = 1.0 + 10.0 * (torch.arange(H, dtype=torch.float64) + 0.5) / H
    return torch.log1p(-torch.exp2(-x)).to(dtype).to(device)


def _sections(pairs, axes):
    """Pairs of each axis: the first takes what an even split leaves over."""
    each = pairs // axes
    return [pairs - each * (axes - 1)] + [each] * (axes - 1)


def prepare(case, seed):
    """Inputs on the GPU, with the workspace and the state buffers a program keeps."""
    B, Hq, Hkv, N, D, Dv = (case[x] for x in ("B", "Hq", "Hkv", "N", "D", "Dv"))
    dt, dev = _DT[case["dtype"]], torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 7919 + 11)

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(dtype)

    s = {"case": case, "scale": float(D) ** -0.5}
    op = case["op"]
    if op in ("prompt", "train", "step"):
        # q and k come contiguous out of prepare_qk with elements of unit RMS; v is a view into
        # the projection where `fused`
        s["q"], s["k"] = normal(B, Hq, N, D), normal(B, Hkv, N, D)
        s["v"] = normal(B, N, Hkv + 2, Dv)[:, :, 1:1 + Hkv].permute(0, 2, 1, 3) if case["fused"] else normal(B, Hkv, N, Dv)
        s["log_decay"] = _log_decay(Hkv, dev)
    if op == "prompt":
        s["S0"] = normal(B, Hkv, D, Dv, dtype=torch.float32) if case["state"] else None
        s["S1"] = torch.empty(B, Hkv, D, Dv, device=dev) if case["state"] else None
        s["lengths"] = None
        if case["ragged"]:
            n = torch.randint(1, N + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
            n[0] = N
            s["lengths"] = n
    if op == "train":
        s["g"] = normal(B, Hq, N, Dv)
        s["S0"] = normal(B, Hkv, D, Dv, dtype=torch.float32) if case["state"] else None
        s["dS1"] = normal(B, Hkv, D, Dv, scale=0.1, dtype=torch.float32) if case["state"] else None
        s["dS0"] = torch.empty(B, Hkv, D, Dv, device=dev) if case["state"] else None
    if op == "step":
        pool = B + case["spare"]
        s["state"] = normal(pool, Hkv, D, Dv, scale=4.0, dtype=torch.float32)
        s["new_state"] = s["state"].clone()
        s["slots"] = torch.randperm(pool, generator=gen, device=dev)[:B].to(torch.int32)
    if op.startswith("prepare_qk"):
        R, A = case["rot"], case["axes"]
        if case["fused"]:
            qkv = normal(B, N, Hq + 2 * Hkv, D, scale=1.5)
            s["q"] = qkv[:, :, :Hq].permute(0, 2, 1, 3)
            s["k"] = qkv[:, :, Hq:Hq + Hkv].permute(0, 2, 1, 3)
        else:
            s["q"], s["k"] = normal(B, Hq, N, D, scale=1.5), normal(B, Hkv, N, D, scale=1.5)
        s["qw"] = 1.0 + normal(D, scale=0.1, dtype=torch.float32) if case["weights"] else None
        s["kw"] = 1.0 + normal(D, scale=0.1, dtype=torch.float32) if case["weights"] else None
        s["inv_freq"] = torch.pow(_BASE, -torch.arange(R // 2, dtype=torch.float64) * 2 / R).to(dev)
        s["sections"] = _sections(R // 2, A)
        start = torch.randint(0, 30000, (1, B, 1), generator=gen, device=dev)
        n = torch.arange(N, device=dev)
        # one axis: the token's place; more: time, then a raster of 64 columns (rows, columns)
        grid = [n] if A == 1 else [n // 64, n % 64] if A == 2 else [n // 4096, n // 64 % 64, n % 64]
        s["positions"] = (torch.stack(grid)[:, None, :] + start).contiguous()
        if op == "prepare_qk_train":
            s["gq"], s["gk"] = normal(B, Hq, N, D), normal(B, Hkv, N, D)
    if own and op in ("prompt", "train", "prepare_qk_train"):
        from efficient_transformer_gb300 import la
        if op == "prepare_qk_train":
            need = la.qk_norm_rope_workspace_size(B, Hq, Hkv, N, D, dt)
        else:
            need = la.decay_workspace_size(B, Hq, Hkv, N, D, dt, op == "train", Dv=Dv)
        s["ws"] = torch.empty(max(1, need), dtype=torch.uint8, device=dev)
    return s


def run(state):
    """One pass of the case's operator; its outputs."""
    op = state["case"]["op"]
    return (_run_own if own else _run_plain)(op, state)


def _run_own(op, s):
    from efficient_transformer_gb300 import la
    if op == "prompt":
        out = la.decay_fwd(s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"], initial_state=s["S0"],
                           final_state=s["S1"], lengths=s["lengths"], workspace=s["ws"])
        return {"out": out, "final_state": s["S1"]}
    if op == "train":
        dq, dk, dv = la.decay_bwd(s["q"], s["k"], s["v"], s["g"], s["log_decay"], scale=s["scale"],
                                  initial_state=s["S0"], grad_final_state=s["dS1"], grad_initial_state=s["dS0"],
                                  workspace=s["ws"])
        return {"dq": dq, "dk": dk, "dv": dv, "grad_initial_state": s["dS0"]}
    if op == "step":
        # the old states are kept (a rejected draft token falls back to them)
        out = la.decay_step(s["q"], s["k"], s["v"], s["state"], s["log_decay"], slots=s["slots"], scale=s["scale"],
                            state_out=s["new_state"])
        return {"out": out, "state": s["new_state"]}
    rope = dict(q_weight=s["qw"], k_weight=s["kw"], eps=_EPS, positions=s["positions"], inv_freq=s["inv_freq"],
                sections=s["sections"], interleaved=s["case"]["interleaved"])
    if op == "prepare_qk":
        q, k = la.qk_norm_rope_fwd(s["q"], s["k"], **rope)
        return {"q": q, "k": k}
    dq, dk, dqw, dkw = la.qk_norm_rope_bwd(s["q"], s["k"], s["gq"], s["gk"], workspace=s["ws"], **rope)
    return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}


# ---- the plain forms: elementary torch operations in 32 bits --------------------------------

_CHUNK = 128


def _chunked(x, y, z, ld, S, lengths=None):
    """sum_{j <= i} g^(i-j) (x_i . y_j) z_j + g^(i+1) x_i S over [B, Hkv, heads, N, *], chunk by
    chunk, and the state after each sequence's last token.  heads broadcasts between x and y, z."""
    B, N, dev = x.shape[0], x.shape[3], x.device
    l = ld.view(1, -1, 1, 1, 1)
    outs = []
    for c0 in range(0, N, _CHUNK):
        xc, yc, zc = x[..., c0:c0 + _CHUNK, :].float(), y[..., c0:c0 + _CHUNK, :].float(), z[..., c0:c0 + _CHUNK, :].float()
        C = xc.shape[3]
        i = torch.arange(C, device=dev, dtype=torch.float32)
        left = torch.full((B,), C, device=dev) if lengths is None else (lengths - c0).clamp(0, C)
        left = left.view(B, 1, 1, 1, 1).float()
        there = i.view(1, 1, 1, C, 1) < left
        yc, zc = torch.where(there, yc, 0.0), torch.where(there, zc, 0.0)
        ago = i[:, None] - i[None, :]
        weight = torch.where(ago >= 0, torch.exp(l * ago.clamp(min=0)), 0.0)
        o = ((xc @ yc.transpose(-1, -2)) * weight) @ zc + torch.exp(l * (i + 1).view(C, 1)) * (xc @ S)
        outs.append(torch.where(there, o, 0.0))
        after = (left - 1 - i.view(1, 1, 1, C, 1)).clamp(min=0)
        S = torch.exp(l * left) * S + (yc * torch.exp(l * after)).transpose(-1, -2) @ zc
    return torch.cat(outs, 3), S


def _turn(x, s, back=False):
    """Rotate the first `rot` elements of x [B, H, N, D] (float32) by the positions' angles."""
    case = s["case"]
    R = case["rot"]
    axis = torch.repeat_interleave(torch.arange(case["axes"], device=x.device),
                                   torch.tensor(s["sections"], device=x.device))
    angle = s["positions"].double()[axis].permute(1, 2, 0) * s["inv_freq"]
    c, n = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    n = -n if back else n
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if case["interleaved"] else (x[..., :R // 2], x[..., R // 2:R])
    p, q = a * c - b * n, a * n + b * c
    t = torch.stack([p, q], -1).flatten(-2) if case["interleaved"] else torch.cat([p, q], -1)
    return torch.cat([t, x[..., R:]], -1)


def _run_plain(op, s):
    case = s["case"]
    B, Hq, Hkv, N, D, Dv = (case[x] for x in ("B", "Hq", "Hkv", "N", "D", "Dv"))
    r, dt, sc = Hq // Hkv, _DT[case["dtype"]], s["scale"]
    if op in ("prompt", "train"):
        q, k, v = s["q"].view(B, Hkv, r, N, D), s["k"].unsqueeze(2), s["v"].unsqueeze(2)
        S0 = s["S0"].unsqueeze(2) if s["S0"] is not None else torch.zeros(B, Hkv, 1, D, Dv, device=q.device)
    if op == "prompt":
        out, S = _chunked(q, k, v, s["log_decay"], S0, s["lengths"])
        return {"out": (out * sc).reshape(B, Hq, N, Dv).to(dt), "final_state": S.squeeze(2) if case["state"] else None}
    if op == "train":
        g, ld = s["g"].view(B, Hkv, r, N, Dv), s["log_decay"]
        dq, _ = _chunked(g, v, k, ld, S0.transpose(-1, -2))
        # the gradients of k and v run from the last token to the first; what the last state's
        # gradient adds to token j has decayed N - 1 - j times
        fq, fk, fv, fg = (t.flip(3) for t in (q, k, v, g))
        zero = torch.zeros(B, Hkv, 1, D, Dv, device=q.device)
        dv, R = _chunked(fk, fq, fg, ld, zero)
        dk, _ = _chunked(fv, fg, fq, ld, zero.transpose(-1, -2))
        dk, dv = sc * dk.flip(3).sum(2), sc * dv.flip(3).sum(2)
        dS0 = None
        if case["state"]:
            gam = ld.view(1, Hkv, 1, 1)
            after = torch.exp(gam * torch.arange(N - 1, -1, -1, device=q.device, dtype=torch.float32).view(N, 1))
            dk = dk + after * (s["v"].float() @ s["dS1"].transpose(-1, -2))
            dv = dv + after * (s["k"].float() @ s["dS1"])
            dS0 = torch.exp(gam) * sc * R.sum(2) + torch.exp(gam * N) * s["dS1"]
        return {"dq": (sc * dq).reshape(B, Hq, N, D).to(dt), "dk": dk.to(dt), "dv": dv.to(dt), "grad_initial_state": dS0}
    if op == "step":
        at = s["slots"].long()
        q, k, v = s["q"].view(B, Hkv, r, D).float(), s["k"].view(B, Hkv, D).float(), s["v"].reshape(B, Hkv, Dv).float()
        S = s["state"][at] * torch.exp(s["log_decay"]).view(1, Hkv, 1, 1) + k.unsqueeze(-1) * v.unsqueeze(-2)
        new = s["state"].clone()
        new[at] = S
        return {"out": (sc * (q @ S)).view(B, Hq, 1, Dv).to(dt), "state": new}
    if op == "prepare_qk":
        res = {}
        for name, w in (("q", s["qw"]), ("k", s["kw"])):
            x = s[name].float()
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS)
            res[name] = _turn(x if w is None else x * w, s).to(dt)
        return res
    res = {}
    for name, w in (("q", s["qw"]), ("k", s["kw"])):
        x, u = s[name].float(), _turn(s["g" + name].float(), s, back=True)
        rms = torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS)
        xh = x * rms
        uw = u if w is None else u * w
        res["d" + name] = (rms * (uw - xh * (uw * xh).mean(-1, keepdim=True))).to(dt)
        res["d" + name + "_weight"] = None if w is None else (u * xh).sum((0, 1, 2), dtype=torch.float64).float()
    return res


# ---- work and the exact values ---------------------------------------------------------------

def work(case):
    """Inputs read once, outputs written once; the recurrence's products and sums (a state is
    updated once a key/value head and read once a query head and token)."""
    B, Hq, Hkv, N, D, Dv = (case[x] for x in ("B", "Hq", "Hkv", "N", "D", "Dv"))
    e, op = (2 if case["dtype"] == "bf16" else 4), case["op"]
    q, k, v, o, st = B * Hq * N * D, B * Hkv * N * D, B * Hkv * N * Dv, B * Hq * N * Dv, 4 * B * Hkv * D * Dv
    if op == "prompt":
        return {"bytes": e * (q + k + v + o) + (2 * st if case["state"] else 0) + 4 * Hkv,
                "flops": 2 * B * N * D * Dv * (Hq + Hkv)}
    if op == "train":
        return {"bytes": e * (2 * q + 2 * k + 2 * v + o) + (3 * st if case["state"] else 0) + 4 * Hkv,
                "flops": 2 * B * N * D * Dv * (2 * Hq + 3 * Hkv)}
    if op == "step":
        return {"bytes": e * (q + k + v + o) + 2 * st + 4 * B, "flops": 2 * B * D * Dv * (Hq + Hkv)}
    pos = 8 * case["axes"] * B * N
    if op == "prepare_qk":
        return {"bytes": 2 * e * (q + k) + pos, "flops": 8 * (q + k)}
    return {"bytes": 3 * e * (q + k) + pos, "flops": 16 * (q + k)}


def exact(case, seed):
    """The definition token by token in 64 bits."""
    s = prepare(case, seed)
    B, Hq, Hkv, N, D, Dv = (case[x] for x in ("B", "Hq", "Hkv", "N", "D", "Dv"))
    r, op, f8 = Hq // Hkv, case["op"], torch.float64
    if op.startswith("prepare_qk"):
        return _exact_qk(case, s)
    dev, sc = s["q"].device, s["scale"]
    gamma = torch.exp(s["log_decay"].double()).view(1, Hkv, 1, 1)

    def rows(x):  # [N, B, Hkv, heads, width]
        return x.reshape(B, Hkv, -1, N, x.shape[-1]).permute(3, 0, 1, 2, 4).to(f8).contiguous()

    q, k, v = rows(s["q"]), rows(s["k"]), rows(s["v"])
    if op == "step":
        at = s["slots"].long()
        S = s["state"].double()
        S[at] = gamma * S[at] + k[0].transpose(-1, -2) * v[0]
        return {"out": (sc * q[0] @ S[at]).reshape(B, Hq, 1, Dv), "state": S}

    def back(x, heads):
        return x.permute(1, 2, 3, 0, 4).reshape(B, heads, N, x.shape[-1])

    n = torch.full((B,), N, device=dev) if op == "train" or s["lengths"] is None else s["lengths"].long()
    on = (torch.arange(N, device=dev)[:, None] < n[None]).to(f8).view(N, B, 1, 1, 1)
    # past its length a sequence neither decays nor adds
    gam = torch.where(on > 0, gamma[None], torch.ones((), dtype=f8, device=dev))
    k = torch.where(on > 0, k, 0.0)
    v = torch.where(on > 0, v, 0.0)
    S = s["S0"].double() if s["S0"] is not None else torch.zeros(B, Hkv, D, Dv, dtype=f8, device=dev)
    S = S.clone()
    kT = k.transpose(-1, -2).contiguous()
    if op == "prompt":
        out = torch.empty(N, B, Hkv, r, Dv, dtype=f8, device=dev)
        for t in range(N):
            S.mul_(gam[t]).addcmul_(kT[t], v[t])
            torch.matmul(q[t], S, out=out[t])
        return {"out": back(torch.where(on > 0, sc * out, 0.0), Hq), "final_state": S if case["state"] else None}
    g = rows(s["g"])
    dq = torch.empty(N, B, Hkv, r, D, dtype=f8, device=dev)
    dk = torch.empty(N, B, Hkv, 1, D, dtype=f8, device=dev)
    dv = torch.empty(N, B, Hkv, 1, Dv, dtype=f8, device=dev)
    for t in range(N):
        S.mul_(gamma).addcmul_(kT[t], v[t])
        torch.matmul(g[t], S.transpose(-1, -2), out=dq[t])
    # A: the gradient of the state after token t
    A = s["dS1"].double() if s["dS1"] is not None else torch.zeros(B, Hkv, D, Dv, dtype=f8, device=dev)
    A = A.clone()
    qT = (sc * q).transpose(-1, -2).contiguous()
    for t in range(N - 1, -1, -1):
        A.add_(torch.matmul(qT[t], g[t]))
        torch.matmul(v[t], A.transpose(-1, -2), out=dk[t])
        torch.matmul(k[t], A, out=dv[t])
        A.mul_(gamma)
    return {"dq": back(sc * dq, Hq), "dk": back(dk, Hkv), "dv": back(dv, Hkv),
            "grad_initial_state": A if case["state"] else None}


def _exact_qk(case, s):
    """Each pair of elements as one complex number times e^(i angle), norms in 64 bits."""
    R, A = case["rot"], case["axes"]
    angle, first = [], 0
    for a in range(A):
        pairs = s["sections"][a]
        angle.append(s["positions"][a].double()[..., None] * s["inv_freq"][first:first + pairs])
        first += pairs
    spin = torch.polar(torch.ones((), dtype=torch.float64, device=angle[0].device), torch.cat(angle, -1))[:, None]

    def turned(x, spin):
        y = x.clone()
        if case["interleaved"]:
            y[..., :R] = torch.view_as_real(torch.view_as_complex(x[..., :R].unflatten(-1, (R // 2, 2)).contiguous())
                                            * spin).flatten(-2)
        else:
            z = torch.complex(x[..., :R // 2].contiguous(), x[..., R // 2:R].contiguous()) * spin
            y[..., :R // 2], y[..., R // 2:R] = z.real, z.imag
        return y

    res = {}
    for name, w in (("q", s["qw"]), ("k", s["kw"])):
        x = s[name].double()
        wd = torch.ones(case["D"], dtype=torch.float64, device=x.device) if w is None else w.double()
        n2 = x.pow(2).sum(-1, keepdim=True) / case["D"] + _EPS
        if case["op"] == "prepare_qk":
            res[name] = turned(x / n2.sqrt() * wd, spin)
            continue
        u = turned(s["g" + name].double(), spin.conj())
        res["d" + name] = u * wd / n2.sqrt() - x * (u * wd * x).sum(-1, keepdim=True) / (case["D"] * n2 * n2.sqrt())
        res["d" + name + "_weight"] = None if w is None else (u * x / n2.sqrt()).sum((0, 1, 2))
    return res
