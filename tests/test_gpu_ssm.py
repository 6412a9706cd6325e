"""Selective scan and short convolution on the GPU against the float64 oracle, whose running bound says how far float32
arithmetic can be off at each element (oracle/ssm.py, `distance`): every output at most twice that, and half a step of its
own type."""
import pytest
import torch

from efficient_transformer_gb300 import build as la_build
from efficient_transformer_gb300 import la
from oracle import ssm

pytestmark = pytest.mark.gpu
F, BF = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    la_build.build()
    la.load()


def inputs(B, N, E, S=16, G=1, dtype=BF, seed=0, strided=True, lengths=None, garbage=float("nan"), slow=0.0):
    """Inputs of a scan on the GPU; past a length the rows hold `garbage`.  `slow`: added to dt_bias (small steps, long
    memories)."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    a = dict(x=r(B, N, E), dt=r(B, N, E) * 0.5, A=-torch.exp(r(E, S)), B=r(B, N, G, S), C=r(B, N, G, S), skip=r(E), z=r(B, N, E),
             dt_bias=r(E) - 2 - slow, initial_state=r(B, E, S), grad_out=r(B, N, E), grad_final_state=r(B, E, S))
    rows = ("x", "dt", "B", "C", "z", "grad_out")
    for k in rows:
        a[k] = a[k].to(dtype)
    if lengths is not None:
        for b, n in enumerate(lengths):
            for k in rows:
                a[k][b, n:] = garbage
        a["lengths"] = torch.tensor(lengths, dtype=torch.int32)
    a = {k: v.cuda() for k, v in a.items()}
    if strided:   # x and z from one projection, B and C from another
        xz = torch.cat([a["x"], a["z"]], 2)
        a["x"], a["z"] = xz[..., :E], xz[..., E:]
        bc = torch.cat([torch.zeros(B, N, 8, device="cuda", dtype=dtype), a["B"].flatten(2), a["C"].flatten(2)], 2)
        a["B"], a["C"] = bc[..., 8:8 + G * S].unflatten(2, (G, S)), bc[..., 8 + G * S:].unflatten(2, (G, S))
    return a


FWD = ("x", "dt", "A", "B", "C")
GRADS = ("dx", "ddt", "dA", "dB", "dC", "dskip", "dz", "ddt_bias")


def clean(a, *names):
    """The oracle's inputs: a length's rows alone are read, but NaN times zero is NaN there."""
    return {n: torch.nan_to_num(a[n].float()) if a[n].is_floating_point() else a[n] for n in names if a.get(n) is not None}


def run_scan(a, softplus=True, states=True, workspace=None):
    """dict like the oracle's from the library's calls."""
    B, N, E = a["x"].shape
    S = a["A"].shape[1]
    kw = dict(softplus=softplus, initial_state=a.get("initial_state"), lengths=a.get("lengths"), skip=a.get("skip"),
              z=a.get("z"), dt_bias=a.get("dt_bias"), workspace=workspace)
    fin, d0 = torch.full((B, E, S), float("nan"), device="cuda"), torch.full((B, E, S), float("nan"), device="cuda")
    kept = torch.full((la.ssm_states_size(B, N, E, S),), 255, dtype=torch.uint8, device="cuda") if states else None
    t = [a[n] for n in FWD]
    out = la.ssm_fwd(*t, final_state=fin, states=kept, **kw)
    res = dict(zip(GRADS, la.ssm_bwd(*t, a["grad_out"], grad_final_state=a.get("grad_final_state"), grad_initial_state=d0,
                                     states=kept, **kw)))
    la.get_status()
    return dict(res, out=out, final_state=fin, grad_initial_state=d0)


def want_scan(a, softplus=True):
    names = FWD + ("skip", "z", "dt_bias", "initial_state", "lengths", "grad_out", "grad_final_state")
    return ssm.scan(**clean(a, *names), use_softplus=softplus)


def compare(got, want, dtype):
    assert set(got) == set(want)
    for k in got:
        assert (got[k] is None) == (want[k] is None), k
        if got[k] is not None:
            eps = torch.finfo(got[k].dtype).eps
            d = ssm.distance(got[k], want[k], eps)
            assert d <= 1, (k, d)


SHAPES = [
    # (B, N, E, S, G): lengths around a tile of 8 and 16 tokens, channels that fill no tile, one channel group of 8
    (1, 1, 8, 16, 1), (2, 2, 16, 8, 1), (1, 7, 24, 16, 1), (2, 8, 32, 16, 2), (1, 9, 40, 32, 1), (3, 15, 16, 64, 1),
    (1, 16, 136, 16, 1), (2, 17, 48, 8, 2), (1, 33, 264, 8, 1), (2, 31, 72, 64, 1), (1, 50, 64, 32, 4), (1, 129, 16, 16, 1),
    # cut into segments
    (1, 400, 16, 16, 1), (2, 777, 8, 8, 1), (1, 515, 24, 64, 1), (1, 640, 16, 32, 2),
]


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_scan_and_gradient(shape, dtype):
    a = inputs(*shape, dtype=dtype, seed=sum(shape))
    compare(run_scan(a), want_scan(a), dtype)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("lengths", [[0, 1, 40], [16, 8, 0], [33, 40, 24], [0, 0, 0], [7, 50, -3]])
def test_lengths(lengths, dtype):
    """Rows past a length hold NaN; lengths outside [0, N] are taken as 0 or N."""
    inside = [min(max(n, 0), 40) for n in lengths]
    a = inputs(3, 40, 24, 16, 1, dtype=dtype, lengths=inside, seed=5)
    a["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    got = run_scan(a)
    compare(got, want_scan(a), dtype)
    for b, n in enumerate(inside):
        for k in ("out", "dx", "ddt", "dz", "dB", "dC"):
            assert not got[k][b, n:].any(), k


def test_lengths_of_segments():
    """Sequences that end before, in and after the cuts of a long batch."""
    a = inputs(4, 900, 8, 16, 1, dtype=F, lengths=[900, 130, 128, 513], garbage=float("inf"), seed=6)
    compare(run_scan(a), want_scan(a), F)


@pytest.mark.parametrize("drop", [("z",), ("skip",), ("dt_bias",), ("initial_state",), ("grad_final_state",),
                                  ("z", "skip", "dt_bias", "initial_state", "grad_final_state")], ids="+".join)
@pytest.mark.parametrize("N", [21, 300])
def test_missing_inputs(drop, N):
    a = inputs(1, N, 16, 16, 1, dtype=F, seed=7)
    a = {k: v for k, v in a.items() if k not in drop}
    compare(run_scan(a), want_scan(a), F)


@pytest.mark.parametrize("N", [21, 300])
def test_without_softplus(N):
    a = inputs(1, N, 16, 16, 1, dtype=F, seed=8)
    a["dt"], a["dt_bias"] = a["dt"].abs(), a["dt_bias"].abs() * 0.1
    compare(run_scan(a, softplus=False), want_scan(a, softplus=False), F)


def test_large_and_small_steps():
    """Steps of 1e-6 (a memory of the whole sequence) to 60 (none at all: exp(d A) is 0)."""
    a = inputs(1, 300, 16, 16, 1, dtype=F, seed=9)
    a["dt_bias"] = torch.linspace(-14, 60, 16, device="cuda")
    compare(run_scan(a), want_scan(a), F)


@pytest.mark.filterwarnings("ignore:overflow:RuntimeWarning", "ignore:invalid:RuntimeWarning")
def test_growing_states():
    a = inputs(1, 40, 8, 8, 1, dtype=F, seed=10)
    a["A"] = -a["A"]
    got, want = run_scan(a), want_scan(a)
    # channels whose states or their gradients pass 2^126 on the way have no float32 values to compare (float32 ends at
    # 2^128; C h and the like are within a factor of 4 of them); dB and dC are sums over such channels too
    large = [abs(want[k].v[0]).max(-1) for k in ("final_state", "grad_initial_state")]
    fits = [e for e in range(8) if max(x[e] for x in large) < 2.0 ** 100]
    assert len(fits) >= 2
    for k in ("out", "final_state", "dx", "ddt", "dz", "grad_initial_state"):
        at = (slice(None), fits) if "state" in k else (slice(None), slice(None), fits)
        assert ssm.distance(got[k][at], want[k][at], torch.finfo(F).eps) <= 1, k
    for k in ("dA", "dskip", "ddt_bias"):
        assert ssm.distance(got[k][fits], want[k][fits], torch.finfo(F).eps) <= 1, k


@pytest.mark.parametrize("N", [40, 700])
def test_the_states_may_be_one_buffer(N):
    a = inputs(2, N, 16, 16, 1, seed=11, lengths=[N, N // 3])
    kw = dict(skip=a["skip"], z=a["z"], dt_bias=a["dt_bias"], lengths=a["lengths"])
    t, fin, both = [a[n] for n in FWD], torch.empty_like(a["initial_state"]), a["initial_state"].clone()
    out = la.ssm_fwd(*t, initial_state=a["initial_state"], final_state=fin, **kw)
    for _ in range(3):
        both.copy_(a["initial_state"])
        again = la.ssm_fwd(*t, initial_state=both, final_state=both, **kw)
        la.get_status()
        assert torch.equal(out, again) and torch.equal(fin, both)


@pytest.mark.parametrize("shape", [(2, 70, 136, 16, 1), (1, 700, 24, 8, 1)])
def test_states_found_again(shape):
    """Without kept states the gradient finds the same ones."""
    a = inputs(*shape, seed=12)
    one, two = run_scan(a, states=True), run_scan(a, states=False)
    for k in one:
        assert torch.equal(one[k], two[k]), k


@pytest.mark.parametrize("shape", [(2, 70, 136, 16, 1), (1, 700, 24, 32, 1)])
def test_workspaces_hold_nothing_that_is_read(shape):
    """Workspaces full of NaN give the same bits, and so does a second run."""
    a = inputs(*shape, seed=13, lengths=[shape[1] - 30] * shape[0])
    B, N, E, S, G = shape
    need = la.ssm_workspace_size(B, N, E, S, G, BF, True)
    want = run_scan(a)
    for fill in (0, 255):
        got = run_scan(a, workspace=torch.full((need,), fill, dtype=torch.uint8, device="cuda"))
        for k in want:
            assert torch.equal(want[k], got[k]), k


def test_broadcast_inputs():
    """Strides of 0: one row of B and C for all tokens, one dt for all sequences."""
    a = inputs(2, 30, 16, 16, 1, dtype=F, seed=14, strided=False)
    for k in ("B", "C"):
        a[k] = a[k][:, :1].expand(-1, 30, -1, -1)
    a["dt"] = a["dt"][:1].expand(2, -1, -1)
    a["grad_out"] = a["grad_out"][:, :1].expand(-1, 30, -1)
    compare(run_scan(a), want_scan(a), F)


@pytest.mark.parametrize("where", [3, 20])
def test_nan_stays_in_its_sequence_and_channel(where):
    """A NaN in x of one token and channel: that channel's later outputs, nothing else."""
    a = inputs(2, 40, 16, 16, 1, dtype=F, seed=15, strided=False)
    kw = dict(skip=a["skip"], z=a["z"], dt_bias=a["dt_bias"])
    want = la.ssm_fwd(*[a[n] for n in FWD], **kw)
    a["x"][1, where, 5] = float("nan")
    got = la.ssm_fwd(*[a[n] for n in FWD], **kw)
    hit = torch.zeros_like(want, dtype=torch.bool)
    hit[1, where:, 5] = True
    assert torch.equal(torch.isnan(got), hit) and torch.equal(got[~hit], want[~hit])


# ---- one token --------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 8, 16, 1), (3, 144, 8, 2), (5, 40, 32, 1), (2, 264, 64, 1), (4, 24, 16, 3)])
def test_scan_step(shape, dtype):
    B, E, S, G = shape
    a = inputs(B, 1, E, S, G, dtype=dtype, seed=20)
    pool = B + 3
    state = torch.randn(pool, E, S, device="cuda")
    slots = torch.randperm(pool, device="cuda")[:B].to(torch.int32)
    a["initial_state"] = state[slots.long()]
    want = ssm.scan(**clean(a, *FWD, "skip", "z", "dt_bias", "initial_state"))
    t = [a[n] for n in FWD]
    kw = dict(skip=a["skip"], z=a["z"], dt_bias=a["dt_bias"], slots=slots)
    new = torch.full_like(state, 7.0)
    out = la.ssm_step(*t, state, state_out=new, **kw)
    kept = state.clone()
    inplace = la.ssm_step(*t, kept, **kw)
    la.get_status()
    compare(dict(out=out, final_state=new[slots.long()]), want, dtype)
    others = torch.ones(pool, dtype=torch.bool, device="cuda")
    others[slots.long()] = False
    assert bool((new[others] == 7).all()) and torch.equal(kept[others], state[others])
    assert torch.equal(inplace, out) and torch.equal(kept[slots.long()], new[slots.long()])


def test_padding_rows_of_a_step():
    a = inputs(4, 1, 16, 16, 1, seed=21)
    state = torch.randn(3, 16, 16, device="cuda")
    slots = torch.tensor([2, -1, 0, 3], dtype=torch.int32, device="cuda")
    kept = state.clone()
    kw = dict(skip=a["skip"], z=a["z"], dt_bias=a["dt_bias"])
    out = la.ssm_step(*[a[n] for n in FWD], kept, slots=slots, **kw)
    alone = state.clone()
    first = la.ssm_step(*[a[n] if n == "A" else a[n][::2] for n in FWD], alone, slots=slots[::2].contiguous(),
                        **dict(kw, z=a["z"][::2]))
    assert not out[1::2].any() and torch.equal(out[::2], first) and torch.equal(kept, alone)
    conv_state, w = torch.randn(3, 3, 16, device="cuda").to(BF), torch.randn(16, 4, device="cuda").to(BF)
    kept = conv_state.clone()
    out = la.conv_step(a["x"], kept, w, slots=slots)
    assert not out[1::2].any() and torch.equal(kept[1], conv_state[1]) and not torch.equal(kept[0], conv_state[0])


@pytest.mark.parametrize("S", [8, 16, 32, 64])
def test_steps_continue_a_prompt(S):
    """A prompt of 20 tokens and 5 single ones: the states and outputs of 25 in one."""
    a = inputs(2, 25, 24, S, 1, dtype=F, seed=22)
    kw = dict(skip=a["skip"], dt_bias=a["dt_bias"])
    part = lambda t, s: t if t.dim() == 2 else t[:, s]  # noqa: E731
    state = a["initial_state"].clone()
    out = [la.ssm_fwd(*[part(a[n], slice(0, 20)) for n in FWD], z=a["z"][:, :20], initial_state=state, final_state=state, **kw)]
    for t in range(20, 25):
        out.append(la.ssm_step(*[part(a[n], slice(t, t + 1)) for n in FWD], state, z=a["z"][:, t:t + 1], **kw))
    want = ssm.scan(**clean(a, *FWD, "skip", "z", "dt_bias", "initial_state"))
    compare(dict(out=torch.cat(out, 1), final_state=state), want, F)


# ---- convolution ------------------------------------------------------------------------------------

def run_conv(x, w, bias, silu, s0, lengths, g, ds1):
    B, N, E = x.shape
    fin, d0 = torch.full_like(s0, float("nan")), torch.full_like(s0, float("nan"))
    out = la.conv_fwd(x, w, bias, silu=silu, initial_state=s0, final_state=fin, lengths=lengths)
    dx, dw, db = la.conv_bwd(x, w, g, bias, silu=silu, initial_state=s0, grad_final_state=ds1, grad_initial_state=d0,
                             lengths=lengths)
    la.get_status()
    return dict(out=out, final_state=fin, dx=dx, dweight=dw, dbias=db, grad_initial_state=d0)


@pytest.mark.parametrize("kind", ["bf16", "f32", "bf16 x f32 weights"])
@pytest.mark.parametrize("silu,bias", [(True, True), (False, True), (True, False)])
@pytest.mark.parametrize("shape", [(1, 1, 8, 4), (2, 2, 16, 4), (1, 3, 24, 3), (2, 9, 40, 2), (3, 64, 136, 4), (1, 200, 520, 3),
                                   (2, 1030, 8, 4)], ids=lambda s: "x".join(map(str, s)))
def test_conv(shape, silu, bias, kind):
    B, N, E, W = shape
    dt, wt = F if kind == "f32" else BF, BF if kind == "bf16" else F
    g = torch.Generator().manual_seed(sum(shape))
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = r(B, N, 2 * E).to(dt).cuda()[..., E:]
    lengths = [max(0, N - 3 * b) for b in range(B)] if B > 1 else None
    go = r(B, N, E).to(dt).cuda()
    if lengths:
        for b, n in enumerate(lengths):
            x[b, n:], go[b, n:] = float("nan"), float("nan")
    w, bs = r(E, W).to(wt).cuda(), r(E).to(wt).cuda() if bias else None
    s0, ds1 = r(B, W - 1, E).to(dt).cuda(), r(B, W - 1, E).to(dt).cuda()
    got = run_conv(x, w, bs, silu, s0, None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda"), go, ds1)
    want = ssm.conv(torch.nan_to_num(x.float()), w, bs, silu, s0, lengths, torch.nan_to_num(go.float()), ds1)
    assert torch.equal(got["final_state"].double().cpu(), torch.from_numpy(want["final_state"].v))
    compare(got, want, dt)
    # without a state: zeros; in one buffer: the same
    none = la.conv_fwd(x, w, bs, silu=silu)
    zero = la.conv_fwd(x, w, bs, silu=silu, initial_state=torch.zeros_like(s0))
    assert torch.equal(none.nan_to_num(), zero.nan_to_num())
    both = s0.clone()
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out = la.conv_fwd(x, w, bs, silu=silu, initial_state=both, final_state=both, lengths=n)
    assert torch.equal(out, got["out"]) and torch.equal(both, got["final_state"])


@pytest.mark.parametrize("lengths", [[0, 1], [2, 3], [5, 40]])
def test_conv_lengths(lengths):
    """Sequences shorter than the window: the final state keeps rows of the initial one."""
    g = torch.Generator().manual_seed(30)
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    x, w, bs, go, s0, ds1 = r(2, 40, 16), r(16, 4), r(16), r(2, 40, 16), r(2, 3, 16), r(2, 3, 16)
    got = run_conv(x, w, bs, True, s0, torch.tensor(lengths, dtype=torch.int32, device="cuda"), go, ds1)
    compare(got, ssm.conv(x, w, bs, True, s0, lengths, go, ds1), F)
    for b, n in enumerate(lengths):
        assert not got["out"][b, n:].any() and not got["dx"][b, n:].any()


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv_step(W, dtype):
    """Token by token through a pool: the rows of a prompt."""
    g = torch.Generator().manual_seed(31 + W)
    r = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()  # noqa: E731
    B, N, E = 3, 6, 40
    x, w, bs, pool = r(B, N, E), r(E, W), r(E), r(5, W - 1, E)
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    want = ssm.conv(x, w, bs, True, pool[slots.long()])
    new = pool.clone()
    out = [la.conv_step(x[:, :1], pool, w, bs, slots=slots, state_out=new)]
    out += [la.conv_step(x[:, t:t + 1], new, w, bs, slots=slots) for t in range(1, N)]
    compare(dict(out=torch.cat(out, 1), final_state=new[slots.long()]), {k: want[k] for k in ("out", "final_state")}, dtype)
    assert torch.equal(new[1], pool[1]) and torch.equal(new[3], pool[3])


# ---- together, graphs, streams ------------------------------------------------------------------------

def test_captured_and_replayed():
    """Forward, gradient and step in CUDA graphs that share a workspace one after the other: the eager bits."""
    a = inputs(1, 700, 24, 16, 1, seed=40)
    B, N, E, S = 1, 700, 24, 16
    ws = torch.empty(la.ssm_workspace_size(B, N, E, S, 1, BF, True), dtype=torch.uint8, device="cuda")
    kept = torch.empty(la.ssm_states_size(B, N, E, S), dtype=torch.uint8, device="cuda")
    w, state = torch.randn(E, 4, device="cuda").to(BF), torch.randn(B, 3, E, device="cuda").to(BF)
    cws = torch.empty(la.conv_workspace_size(B, N, E, 4, BF), dtype=torch.uint8, device="cuda")

    def one():
        kw = dict(skip=a["skip"], z=a["z"], dt_bias=a["dt_bias"], workspace=ws, states=kept)
        x = la.conv_fwd(a["x"], w, initial_state=state)
        t = [x] + [a[n] for n in FWD[1:]]
        out = la.ssm_fwd(*t, **kw)
        grads = la.ssm_bwd(*t, a["grad_out"], **kw)
        return (x, out) + grads + la.conv_bwd(a["x"], w, grads[0], initial_state=state, workspace=cws)[:2]

    want = one()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        one()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = one()
    for _ in range(2):
        for t in got:
            if t is not None:
                t.fill_(float("nan"))
        graph.replay()
        la.get_status()
        for x, y in zip(want, got):
            assert x is None or torch.equal(x, y)


@pytest.mark.parametrize("name", ["ssm_fwd", "ssm_bwd", "conv_bwd"])
def test_memory_is_not_reused_while_the_side_stream_runs(name):
    a = inputs(1, 2500, 64, 16, 1, seed=41, strided=False)
    w = torch.randn(64, 4, device="cuda").to(BF)
    call = {"ssm_fwd": lambda t, **k: (la.ssm_fwd(*t[:2], a["A"], *t[2:4], **k),),
            "ssm_bwd": lambda t, **k: la.ssm_bwd(*t[:2], a["A"], *t[2:5], **k)[:5],
            "conv_bwd": lambda t, **k: la.conv_bwd(t[0], w, t[4], **k)[:2]}[name]
    given = [a[n] for n in ("x", "dt", "B", "C", "grad_out")]
    want = call(given)
    dropped = [t.clone() for t in given]
    here, side = torch.cuda.current_stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)
    got = call(dropped, stream=side)
    del dropped
    sizes = [t.numel() * t.element_size() for t in list(given) + list(want)] + [1 << n for n in range(12, 26, 2)]
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    here.wait_stream(side)
    la.get_status()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    del junk


def test_offsets_past_32_bits():
    """Rows of a [B, N, E] input more than 2^31 elements apart, and a pool of as many states."""
    big = torch.empty((1 << 31) + (1 << 22), dtype=BF, device="cuda")
    E, N = 64, 9
    step = (1 << 31) // (N - 1) // 8 * 8
    x = torch.as_strided(big, (1, N, E), (0, step, 1))
    a = inputs(1, N, E, 16, 1, seed=42, strided=False)
    x.copy_(a["x"])
    w = torch.randn(E, 4, device="cuda").to(BF)
    kw = dict(skip=a["skip"], z=a["z"], dt_bias=a["dt_bias"])
    assert torch.equal(la.ssm_fwd(x, *[a[n] for n in FWD[1:]], **kw), la.ssm_fwd(*[a[n] for n in FWD], **kw))
    for p, q in zip(la.ssm_bwd(x, *[a[n] for n in FWD[1:]], a["grad_out"], **kw), la.ssm_bwd(*[a[n] for n in FWD], a["grad_out"], **kw)):
        assert torch.equal(p, q)
    assert torch.equal(la.conv_fwd(x, w), la.conv_fwd(a["x"], w))
    for p, q in zip(la.conv_bwd(x, w, a["grad_out"])[:2], la.conv_bwd(a["x"], w, a["grad_out"])[:2]):
        assert torch.equal(p, q)
    del big, x
    pool = (1 << 31) // (E * 16) + 5
    state = torch.empty(pool, E, 16, device="cuda")
    state[-2].normal_()
    one = [a[n] if n == "A" else a[n][:, :1] for n in FWD]
    kw["z"] = a["z"][:, :1]
    small = state[-2:-1].clone()
    want = la.ssm_step(*one, small, **kw)
    got = la.ssm_step(*one, state, slots=torch.tensor([pool - 2], dtype=torch.int32, device="cuda"), **kw)
    assert torch.equal(got, want) and torch.equal(state[-2], small[0])


def test_more_sequences_than_a_grid_dimension():
    a = inputs(70000, 1, 8, 8, 1, seed=43)
    got = run_scan(a)
    part = {k: v if k in ("A", "skip", "dt_bias") else v[-3:] for k, v in a.items()}
    want = run_scan(part)
    for k in ("out", "final_state", "dx", "ddt", "dB", "dC", "dz", "grad_initial_state"):
        assert torch.equal(got[k][-3:], want[k]), k
    w = torch.randn(8, 4, device="cuda").to(BF)
    assert torch.equal(la.conv_fwd(a["x"], w)[-3:], la.conv_fwd(a["x"][-3:], w))
