"""The selective state space scan and its short causal convolution, as a program uses them.

The operators (x [B, N, E]: N tokens of E channels; a channel has S states; B and C rows shared by
the channels of a group):

* ``conv``: out_t = silu(bias + sum_j weight_j x_(t - W + 1 + j)) for each channel, over prompts, the
  last W - 1 inputs going on to the next call; ``conv_train``: its gradients; ``conv_step``: one token
  of each sequence on a pool of such states addressed by slot;
* ``scan``: d_t = softplus(dt_t + dt_bias), h_t = exp(d_t A) h_(t-1) + d_t x_t B_t,
  out_t = (C_t . h_t + skip x_t) silu(z_t), over prompts, the last h going on; ``scan_train``: a training
  step's forward and gradients; ``scan_step``: one token of each sequence on a pool of h.

``listed()`` gives the measured cases, ``draw(rng)`` one more of their ranges, ``prepare`` the inputs of a
case, ``run`` one pass, ``work`` what a pass cannot do without and ``exact`` the outputs in 64 bits from
the definition.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _case(op, B, N, E, S=16, G=1, W=4, dtype="bf16", state=False, ragged=False, gate=True, extras=True, spare=0):
    """A case.  `state`: a state comes in and the last one goes out (for gradients: theirs as well); `ragged`: the
    sequences of the batch have lengths of their own; `gate`: the scan's output is gated by z (the
    convolution's by itself); `extras`: bias (convolution), or skip and dt_bias (scan); `spare`: pool slots that no
    sequence of this call uses."""
    return {"op": op, "B": B, "N": N, "E": E, "S": S, "G": G, "W": W, "dtype": dtype, "state": state, "ragged": ragged,
            "gate": gate, "extras": extras, "spare": spare}


def listed():
    def named(name, *a, **k):
        return dict(_case(*a, **k), name=name)

    return [
        # prompts of unequal length in one batch, their last inputs going on to the decoder
        named("conv_ragged_states", "conv", 7, 1537, 1024, state=True, ragged=True),
        # one very long prompt
        named("conv_n65536", "conv", 1, 65536, 2048, state=True),
        # a short float32 training shape: three taps, an odd length, channels that fill no tile
        named("conv_train_f32_n777", "conv_train", 2, 777, 200, W=3, dtype="f32", state=True),
        # four training sequences of 4096 tokens at the width of the projection's benchmark
        named("conv_train_b4_n4096", "conv_train", 4, 4096, 4096),
        # one user, one token: launch latency
        named("conv_step_b1", "conv_step", 1, 1, 4096),
        # a full decoding batch, its slots scattered over a larger pool
        named("conv_step_b192", "conv_step", 192, 1, 4096, spare=61),
        # prompts of unequal length with two groups of B and C, states going on to the decoder
        named("scan_ragged_states", "scan", 7, 1537, 1024, G=2, state=True, ragged=True),
        # one very long prompt
        named("scan_n65536", "scan", 1, 65536, 2048, state=True),
        # a short float32 training shape with a starting state, eight states a channel
        named("scan_train_f32_n777", "scan_train", 2, 777, 200, S=8, dtype="f32", state=True),
        # four training sequences of 4096 tokens
        named("scan_train_b4_n4096", "scan_train", 4, 4096, 4096),
        # one user, one token: launch latency
        named("scan_step_b1", "scan_step", 1, 1, 4096),
        # a full decoding batch, its slots scattered over a larger pool
        named("scan_step_b192", "scan_step", 192, 1, 4096, spare=61),
    ]


def _limit(op):
    """The largest listed work of an operator: what a drawn case stays below."""
    w = [work(c) for c in listed() if c["op"] == op]
    return max(x["bytes"] for x in w), max(x["flops"] for x in w)


def draw(rng):
    def log_int(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))

    while True:
        op = rng.choice(["conv", "conv_train", "conv_step", "scan", "scan", "scan_train", "scan_train", "scan_step"])
        step = op.endswith("step")
        G = rng.choice([1, 1, 1, 2, 4])
        # channels of a group in eights, which fill whole tiles or not
        E = G * 8 * log_int(1, 8192 // (8 * G))
        c = _case(op, log_int(1, 256 if step else 8), 1 if step else log_int(1, 65536 if not op.endswith("train") else 16384),
                  E, S=rng.choice([8, 16, 16, 16, 32, 64]), G=G, W=rng.choice([2, 3, 4, 4]),
                  dtype="bf16" if rng.random() < 0.75 else "f32")
        c["state"] = not step and rng.random() < 0.5
        c["ragged"] = not step and c["B"] > 1 and rng.random() < 0.4
        c["gate"], c["extras"] = rng.random() < 0.8, rng.random() < 0.8
        c["spare"] = rng.randrange(0, 40) if step else 0
        w, (most_b, most_f) = work(c), _limit(op)
        # (float32 rows are twice as wide)
        if w["bytes"] <= most_b and w["flops"] <= most_f:
            return c


def prepare(case, seed):
    """Inputs on the GPU, with the workspace and the state buffers a program keeps."""
    B, N, E, S, G, W, op = (case[x] for x in ("B", "N", "E", "S", "G", "W", "op"))
    dt, dev = _DT[case["dtype"]], torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 7919 + 17)

    def normal(*shape, scale=1.0, dtype=dt):
        # (row by row of the first dimension: no float32 copy of the whole beside it)
        t = torch.empty(shape, dtype=dtype, device=dev)
        for row in t if len(shape) > 2 else (t,):
            row.copy_(torch.randn(row.shape, generator=gen, device=dev) * scale)
        return t

    s = {"case": case, "lengths": None}
    if case["ragged"]:
        n = torch.randint(1, N + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
        n[0] = N
        s["lengths"] = n
    if op.startswith("conv"):
        # x is the first half of a projection's rows, whose second half is the scan's gate
        s["x"] = normal(B, N, 2 * E)[:, :, :E]
        s["weight"] = normal(E, W, scale=W ** -0.5)
        s["bias"] = normal(E, scale=0.1) if case["extras"] else None
        hold = lambda *shape, scale=1.0: normal(*shape, W - 1, E, scale=scale)  # noqa: E731
    else:
        x = normal(B, N, E)
        s["x"] = x * torch.sigmoid(x)
        s["dt"] = normal(B, N, E, scale=0.5)
        # B and C are views into one projection whose first columns the step sizes come from
        proj = normal(B, N, 32 + 2 * G * S)
        s["B"] = proj[:, :, 32:32 + G * S].unflatten(2, (G, S))
        s["C"] = proj[:, :, 32 + G * S:].unflatten(2, (G, S))
        s["A"] = -torch.arange(1, S + 1, device=dev, dtype=torch.float32) * torch.exp(0.1 * torch.randn(E, S, generator=gen, device=dev))
        s["z"] = normal(B, N, 2 * E)[:, :, E:] if case["gate"] else None
        s["skip"] = s["dt_bias"] = None
        if case["extras"]:
            s["skip"] = 1.0 + 0.1 * torch.randn(E, generator=gen, device=dev)
            # step sizes from 0.001 to 0.1, evenly in the exponent, through the inverse of softplus
            d = torch.exp(torch.rand(E, generator=gen, device=dev) * math.log(100.0) + math.log(0.001))
            s["dt_bias"] = d + torch.log(-torch.expm1(-d))
        hold = lambda *shape, scale=1.0: normal(*shape, E, S, scale=scale, dtype=torch.float32)  # noqa: E731
    if op.endswith("step"):
        pool = B + case["spare"]
        s["state"] = hold(pool)
        s["new_state"] = s["state"].clone()
        s["slots"] = torch.randperm(pool, generator=gen, device=dev)[:B].to(torch.int32)
        return s
    s["S0"] = hold(B) if case["state"] else None
    s["S1"] = torch.empty_like(s["S0"]) if case["state"] else None
    train = op.endswith("train")
    if train:
        s["g"] = normal(B, N, E)
        s["dS1"] = hold(B, scale=0.1) if case["state"] else None
        s["dS0"] = torch.empty_like(s["S0"]) if case["state"] else None
    if own:
        from efficient_transformer_gb300 import la
        need = 0
        if op == "conv_train":
            need = la.conv_workspace_size(B, N, E, W, dt)
        elif not op.startswith("conv"):
            need = la.ssm_workspace_size(B, N, E, S, G, dt, train)
        s["ws"] = torch.empty(max(1, need), dtype=torch.uint8, device=dev)
        if op == "scan_train":
            s["kept"] = torch.empty(la.ssm_states_size(B, N, E, S), dtype=torch.uint8, device=dev)
    return s


def run(state):
    """One pass of the case's operator; its outputs."""
    return (_run_own if own else _run_plain)(state["case"]["op"], state)


def _run_own(op, s):
    from efficient_transformer_gb300 import la
    gate = s["case"]["gate"]
    if op.startswith("conv"):
        kw = dict(bias=s["bias"], silu=gate)
        if op == "conv_step":
            # the old states are kept (a rejected draft token falls back to them)
            out = la.conv_step(s["x"], s["state"], s["weight"], slots=s["slots"], state_out=s["new_state"], **kw)
            return {"out": out, "state": s["new_state"]}
        kw.update(initial_state=s["S0"], lengths=s["lengths"])
        if op == "conv":
            return {"out": la.conv_fwd(s["x"], s["weight"], final_state=s["S1"], **kw), "final_state": s["S1"]}
        dx, dw, db = la.conv_bwd(s["x"], s["weight"], s["g"], grad_final_state=s["dS1"], grad_initial_state=s["dS0"],
                                 workspace=s["ws"], **kw)
        return {"dx": dx, "dweight": dw, "dbias": db, "grad_initial_state": s["dS0"]}
    a = (s["x"], s["dt"], s["A"], s["B"], s["C"])
    kw = dict(skip=s["skip"], z=s["z"], dt_bias=s["dt_bias"])
    if op == "scan_step":
        out = la.ssm_step(*a, s["state"], slots=s["slots"], state_out=s["new_state"], **kw)
        return {"out": out, "state": s["new_state"]}
    kw.update(initial_state=s["S0"], lengths=s["lengths"], workspace=s["ws"])
    if op == "scan":
        return {"out": la.ssm_fwd(*a, final_state=s["S1"], **kw), "final_state": s["S1"]}
    out = la.ssm_fwd(*a, final_state=s["S1"], states=s["kept"], **kw)
    g = la.ssm_bwd(*a, s["g"], grad_final_state=s["dS1"], grad_initial_state=s["dS0"], states=s["kept"], **kw)
    return dict(zip(("dx", "ddt", "dA", "dB", "dC", "dskip", "dz", "ddt_bias"), g), out=out, final_state=s["S1"],
                grad_initial_state=s["dS0"])


# ---- the plain forms: elementary torch operations in 32 bits --------------------------------

_PART = 512


def _there(s):
    """[B, N, 1]: which tokens are within their sequence's length."""
    B, N = s["case"]["B"], s["case"]["N"]
    n = torch.full((B,), N, device=s["x"].device) if s["lengths"] is None else s["lengths"]
    return (torch.arange(N, device=n.device)[None] < n[:, None])[..., None], n.long()


def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _conv_rows(s, on):
    """The inputs with the W - 1 before the first token in front."""
    B, E, W = (s["case"][x] for x in ("B", "E", "W"))
    x = torch.where(on, s["x"].float(), 0.0)
    first = torch.zeros(B, W - 1, E, device=x.device) if s["S0"] is None else s["S0"].float()
    return torch.cat([first, x], 1)


def _taps(rows, w, bias, N):
    y = sum(w[:, j] * rows[:, j:j + N] for j in range(w.shape[1]))
    return y if bias is None else y + bias.float()


def _plain_conv(op, s):
    case = s["case"]
    B, N, E, W, dt = case["B"], case["N"], case["E"], case["W"], _DT[case["dtype"]]
    w = s["weight"].float()
    if op == "conv_step":
        at = s["slots"].long()
        rows = torch.cat([s["state"][at].float(), s["x"].float()], 1)
        y = _taps(rows, w, s["bias"], 1)
        new = s["state"].clone()
        new[at] = rows[:, 1:].to(dt)
        return {"out": (y * _sigmoid(y) if case["gate"] else y).to(dt), "state": new}
    on, n = _there(s)
    rows = _conv_rows(s, on)
    y = _taps(rows, w, s["bias"], N)
    last = (n[:, None] + torch.arange(W - 1, device=n.device))[..., None].expand(-1, -1, E)
    if op == "conv":
        y = y * _sigmoid(y) if case["gate"] else y
        return {"out": torch.where(on, y, 0.0).to(dt), "final_state": rows.gather(1, last).to(dt) if case["state"] else None}
    g = torch.where(on, s["g"].float(), 0.0)
    if case["gate"]:
        p = _sigmoid(y)
        g = g * p * (1.0 + y * (1.0 - p))
    drows = torch.zeros_like(rows)
    for j in range(W):
        drows[:, j:j + N] += w[:, j] * g
    if case["state"]:
        drows.scatter_add_(1, last, s["dS1"].float())
    dw = torch.stack([(g * rows[:, j:j + N]).sum((0, 1), dtype=torch.float64) for j in range(W)], 1)
    db = g.sum((0, 1), dtype=torch.float64).to(dt) if case["extras"] else None
    # (a state's gradient goes to the rows in front of the first token, whatever the length)
    dx = torch.where(on, drows[:, W - 1:], 0.0)
    return {"dx": dx.to(dt), "dweight": dw.to(dt), "dbias": db,
            "grad_initial_state": drows[:, :W - 1].to(dt) if case["state"] else None}


def _softplus(v):
    return v.clamp(min=0) + torch.log1p(torch.exp(-v.abs()))


def _run_over(a, b):
    """h_t = a_t h_(t-1) + b_t along dimension 1 from h = 0, by doubling; a and b are used up."""
    d = 1
    while d < b.shape[1]:
        b[:, d:] += a[:, d:] * b[:, :-d]
        a[:, d:] = a[:, d:] * a[:, :-d]
        d *= 2
    return b


def _plain_scan(op, s):
    case = s["case"]
    B, N, E, S, G, dt = (case[x] for x in ("B", "N", "E", "S", "G", "dtype"))
    dt, r, dev, train = _DT[dt], E // G, s["x"].device, op == "scan_train"
    A = s["A"]

    def wide(t):     # a group's rows for each of its channels: [.., G, S] -> [.., E, S]
        return t.float().repeat_interleave(r, -2)

    def step_size(v):
        return _softplus(v if s["dt_bias"] is None else v + s["dt_bias"])

    if op == "scan_step":
        at = s["slots"].long()
        x, d = s["x"][:, 0].float(), step_size(s["dt"][:, 0].float())
        h = torch.exp(d[..., None] * A) * s["state"][at] + (d * x)[..., None] * wide(s["B"][:, 0])
        y = (h * wide(s["C"][:, 0])).sum(-1)
        y = y if s["skip"] is None else y + s["skip"] * x
        if s["z"] is not None:
            z = s["z"][:, 0].float()
            y = y * z * _sigmoid(z)
        new = s["state"].clone()
        new[at] = h
        return {"out": y[:, None].to(dt), "state": new}
    on, _ = _there(s)
    h = torch.zeros(B, E, S, device=dev) if s["S0"] is None else s["S0"]
    parts = [slice(t, min(t + _PART, N)) for t in range(0, N, _PART)]
    outs, starts = [], []

    def given(p):
        here = on[:, p]
        x = torch.where(here, s["x"][:, p].float(), 0.0)
        v = s["dt"][:, p].float()
        d = torch.where(here, step_size(v), 0.0)
        b, c = (torch.where(here[..., None], wide(s[k][:, p]), 0.0) for k in ("B", "C"))
        return here, x, v, d, torch.exp(d[..., None] * A), b, c

    def through(p, h0):
        here, x, v, d, a, b, c = given(p)
        u = (d * x)[..., None] * b
        u[:, 0] += a[:, 0] * h0
        return here, x, v, d, a, b, c, _run_over(a.clone(), u)

    def unless(z, here):
        return torch.where(here, z.float(), 0.0)

    for p in parts:
        starts.append(h)
        here, x, v, d, a, b, c, hs = through(p, h)
        y = (hs * c).sum(-1)
        y = y if s["skip"] is None else y + s["skip"] * x
        if s["z"] is not None:
            z = unless(s["z"][:, p], here)
            y = y * z * _sigmoid(z)
        outs.append(torch.where(here, y, 0.0).to(dt))
        h = hs[:, -1].clone()
    res = {"out": torch.cat(outs, 1), "final_state": h if case["state"] else None}
    if not train:
        return res
    rows = {k: [] for k in ("dx", "ddt", "dB", "dC", "dz")}
    f8 = torch.float64
    dA, dskip, dbias = torch.zeros(E, S, dtype=f8, device=dev), torch.zeros(E, dtype=f8, device=dev), torch.zeros(E, dtype=f8, device=dev)
    P = torch.zeros(B, E, S, device=dev) if s["dS1"] is None else s["dS1"]   # of the state after the part
    for p, h0 in zip(reversed(parts), reversed(starts)):
        here, x, v, d, a, b, c, hs = through(p, h0)
        g = unless(s["g"][:, p], here)
        if s["z"] is not None:
            z = unless(s["z"][:, p], here)
            y = (hs * c).sum(-1)
            y = y if s["skip"] is None else y + s["skip"] * x
            sz = _sigmoid(z)
            rows["dz"].append((g * y * sz * (1.0 + z * (1.0 - sz))).to(dt))
            g = g * z * sz
        rows["dC"].append((g[..., None] * hs).unflatten(2, (G, r)).sum(3).to(dt))
        gh = g[..., None] * c
        gh[:, -1] += P
        after = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
        gh = _reverse(after, gh)
        P = a[:, 0] * gh[:, 0]
        before = torch.cat([h0[:, None], hs[:, :-1]], 1)
        q = gh * a * before
        du = (gh * b).sum(-1)
        rows["dB"].append((gh * (d * x)[..., None]).unflatten(2, (G, r)).sum(3).to(dt))
        dd = (q * A).sum(-1) + x * du
        dA += (q * d[..., None]).sum((0, 1), dtype=f8)
        dx = d * du
        if s["skip"] is not None:
            dx = dx + s["skip"] * g
            dskip += (g * x).sum((0, 1), dtype=f8)
        v = v if s["dt_bias"] is None else v + s["dt_bias"]
        ddt = torch.where(here, dd * _sigmoid(v), 0.0)
        dbias += ddt.sum((0, 1), dtype=f8)
        rows["dx"].append(dx.to(dt))
        rows["ddt"].append(ddt.to(dt))
    for k, v in rows.items():
        res[k] = torch.cat(v[::-1], 1) if v else None
    res.update(dA=dA.float(), dskip=dskip.float() if case["extras"] else None,
               ddt_bias=dbias.float() if case["extras"] else None, grad_initial_state=P if case["state"] else None)
    return res


def _reverse(after, c):
    """g_t = c_t + after_t g_(t+1) along dimension 1 (after's last entry meets nothing)."""
    return _run_over(after.flip(1), c.flip(1)).flip(1)


def _run_plain(op, s):
    return (_plain_conv if op.startswith("conv") else _plain_scan)(op, s)


# ---- work and the exact values ---------------------------------------------------------------

def work(case):
    """Inputs read once, outputs written once; the recurrences' products, sums and exponentials for each state and
    token (7: d A, exp, d x B, h, C h; the gradients 17 more)."""
    B, N, E, S, G, W, op = (case[x] for x in ("B", "N", "E", "S", "G", "W", "op"))
    e, rows, some = (2 if case["dtype"] == "bf16" else 4), B * N * E, case["state"]
    if op.startswith("conv"):
        st = e * B * (W - 1) * E
        if op == "conv_train":
            return {"bytes": 3 * e * rows + (3 * st if some else 0) + 2 * e * E * (W + 1), "flops": rows * (6 * W + 10)}
        return {"bytes": 2 * e * rows + (2 * st if some or op == "conv_step" else 0) + e * E * (W + 1), "flops": rows * (2 * W + 4)}
    st, bc, vec = 4 * B * E * S, 2 * B * N * G * S, 4 * E * (S + 2)
    z = 1 if case["gate"] else 0
    if op == "scan_train":
        return {"bytes": e * (rows * (6 + 2 * z) + 2 * bc) + (4 * st if some else 0) + 2 * vec, "flops": rows * (24 * S + 20)}
    return {"bytes": e * (rows * (3 + z) + bc) + (2 * st if some or op == "scan_step" else 0) + vec, "flops": rows * (7 * S + 10)}


def exact(case, seed):
    """The definition token by token in 64 bits."""
    s = prepare(case, seed)
    return (_exact_conv if case["op"].startswith("conv") else _exact_scan)(case, s)


def _exact_conv(case, s):
    B, N, E, W, op, f8 = case["B"], case["N"], case["E"], case["W"], case["op"], torch.float64
    w = s["weight"].double()
    bias = torch.zeros(E, dtype=f8, device=w.device) if s["bias"] is None else s["bias"].double()

    def answer(y):
        return y / (1.0 + torch.exp(-y)) if case["gate"] else y

    if op == "conv_step":
        state, out = s["state"].double(), torch.empty(B, 1, E, dtype=f8, device=w.device)
        for b, at in enumerate(s["slots"].tolist()):
            window = torch.cat([state[at], s["x"][b].double()])
            out[b, 0] = answer(bias + torch.einsum("ew,we->e", w, window))
            state[at] = window[1:]
        return {"out": out, "state": state}
    lengths = [N] * B if s["lengths"] is None else s["lengths"].tolist()
    out = torch.zeros(B, N, E, dtype=f8, device=w.device)
    last = torch.empty(B, W - 1, E, dtype=f8, device=w.device)
    dw, db, dfirst = torch.zeros_like(w), torch.zeros_like(bias), torch.empty_like(last)
    for b, n in enumerate(lengths):
        first = torch.zeros(W - 1, E, dtype=f8, device=w.device) if s["S0"] is None else s["S0"][b].double()
        rows = torch.cat([first, s["x"][b, :n].double()])
        windows = rows.unfold(0, W, 1)                       # [n, E, W]
        y = (windows * w).sum(-1) + bias
        last[b] = rows[n:]
        if op == "conv":
            out[b, :n] = answer(y)
            continue
        g = s["g"][b, :n].double()
        if case["gate"]:
            e = torch.exp(-y)
            g = g * (1.0 + e + y * e) / (1.0 + e) ** 2
        dw += torch.einsum("ne,new->ew", g, windows)
        db += g.sum(0)
        drows = torch.nn.functional.pad(g, (0, 0, W - 1, W - 1)).unfold(0, W, 1).flip(-1).mul(w).sum(-1)
        if case["state"]:
            drows[n:] += s["dS1"][b].double()
        dfirst[b] = drows[:W - 1]
        out[b, :n] = drows[W - 1:]
    if op == "conv":
        return {"out": out, "final_state": last if case["state"] else None}
    return {"dx": out, "dweight": dw, "dbias": db if case["extras"] else None,
            "grad_initial_state": dfirst if case["state"] else None}


def _exact_scan(case, s):
    B, N, E, S, G, op = (case[x] for x in ("B", "N", "E", "S", "G", "op"))
    f8 = torch.float64
    dev, r = s["x"].device, E // G
    A = s["A"].double()
    bias = 0.0 if s["dt_bias"] is None else s["dt_bias"].double()
    skip = torch.zeros(E, dtype=f8, device=dev) if s["skip"] is None else s["skip"].double()
    n = torch.full((B,), N, device=dev) if s["lengths"] is None else s["lengths"].long()

    def token(t):
        """x, the step's argument, B and C for every channel, z; of tokens past a length nothing is used."""
        x, v = s["x"][:, t].double(), s["dt"][:, t].double() + bias
        b, c = (s[k][:, t].double()[:, :, None].expand(B, G, r, S).reshape(B, E, S) for k in ("B", "C"))
        return x, v, torch.logaddexp(v, torch.zeros_like(v)), b, c, None if s["z"] is None else s["z"][:, t].double()

    if op == "scan_step":
        x, v, d, b, c, z = token(0)
        at = s["slots"].long()
        state = s["state"].double()
        h = torch.exp(d[..., None] * A) * state[at] + d[..., None] * b * x[..., None]
        state[at] = h
        y = torch.einsum("bes,bes->be", h, c) + skip * x
        return {"out": (y if z is None else y * z * torch.sigmoid(z))[:, None], "state": state}
    train = op == "scan_train"
    h = torch.zeros(B, E, S, dtype=f8, device=dev) if s["S0"] is None else s["S0"].double()
    out, before = torch.zeros(B, N, E, dtype=f8, device=dev), []
    for t in range(N):
        x, v, d, b, c, z = token(t)
        here = (t < n)[:, None]
        if train:
            before.append(h)
        h = torch.where(here[..., None], torch.exp(d[..., None] * A) * h + (d * x)[..., None] * b, h)
        y = (h * c).sum(-1) + skip * x
        out[:, t] = torch.where(here, y if z is None else y * z * torch.sigmoid(z), 0.0)
    res = {"out": out, "final_state": h if case["state"] else None}
    if not train:
        return res
    P = torch.zeros(B, E, S, dtype=f8, device=dev) if s["dS1"] is None else s["dS1"].double()
    dx, ddt, dz = torch.zeros_like(out), torch.zeros_like(out), torch.zeros_like(out)
    dB, dC = (torch.zeros(B, N, G, S, dtype=f8, device=dev) for _ in range(2))
    dA, dskip = torch.zeros_like(A), torch.zeros_like(skip)
    after = h
    for t in range(N - 1, -1, -1):
        x, v, d, b, c, z = token(t)
        here = (t < n)[:, None]
        h0 = before.pop()
        g = s["g"][:, t].double()
        if z is not None:
            p = torch.sigmoid(z)
            y = (after * c).sum(-1) + skip * x
            dz[:, t] = torch.where(here, g * y * p * (1.0 + z * (1.0 - p)), 0.0)
            g = g * z * p
        g = torch.where(here, g, 0.0)
        x, d = torch.where(here, x, 0.0), torch.where(here, d, 0.0)
        a = torch.exp(d[..., None] * A)
        gh = P + torch.where(here[..., None], g[..., None] * c, 0.0)
        dC[:, t] = (g[..., None] * after).unflatten(1, (G, r)).sum(2)
        dB[:, t] = (gh * (d * x)[..., None]).unflatten(1, (G, r)).sum(2)
        P = a * gh
        q = P * h0
        du = torch.where(here, (gh * b).sum(-1), 0.0)
        dx[:, t] = d * du + skip * g
        ddt[:, t] = torch.where(here, ((q * A).sum(-1) + x * du) * torch.sigmoid(v), 0.0)
        dA += (q * d[..., None]).sum(0)
        dskip += (g * x).sum(0)
        after = h0
    extras = case["extras"]
    res.update(dx=dx, ddt=ddt, dA=dA, dB=dB, dC=dC, dskip=dskip if extras else None, dz=dz if case["gate"] else None,
               ddt_bias=ddt.sum((0, 1)) if extras else None, grad_initial_state=P if case["state"] else None)
    return res
