"""GPU parity of the decayed linear attention with the float64 oracle, element by element.

Tolerances.  Let A be the same sum with every input replaced by its absolute value (what rounding
errors are relative to).  float32: each of the D products of a score, the terms of a chunk and the
chunks' carries rounds once, and gamma^n errs by n |log gamma| 2^-24 (below 104 2^-24 wherever the power is
not 0): (D + 128 + 3 chunks + 104) 2^-24 A with chunks of 32 at least.  bfloat16 adds half a step (2^-8)
of the result, and on the tensor cores half a step of A for the operands rounded once: what comes from the
chunk has one such factor (the masked scores), what comes through the state has x, S and, where the state itself is no
output, y as well.  At worst those are three half steps; as they are sums of 64 products or more whose roundings are
independent, one half step holds them wherever the state is an output (three are allowed where not).  A state that is
an output adds up two bfloat16 terms of each y: 2^-16 A."""
import numpy as np
import pytest
import torch

from efficient_transformer_gb300 import build as la_build
from efficient_transformer_gb300 import la
from oracle import decay as od

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    la_build.build()
    la.load()


def f32_part(N, D):
    return (D + 128 + 3 * (N / 32) + 104) * 2.0 ** -24


def check(got, want, A, N, D, tc, name, factors=1):
    got = got.detach().double().cpu().numpy()
    half = 2.0 ** -8 if name in ("out", "dq", "dk", "dv") and check.dtype == torch.bfloat16 else 2.0 ** -24
    tol = half * np.abs(want) + f32_part(N, D) * A + 1e-37
    if tc:
        tol = tol + (factors * 2.0 ** -8 if half > 1e-3 else 0) * A + 2.0 ** -16 * A
    assert np.isfinite(got).all(), name
    bad = np.abs(got - want) / tol
    assert bad.max() <= 1.0, (name, float(bad.max()), np.unravel_index(bad.argmax(), bad.shape))


def draw(B, Hq, Hkv, N, D, Dv, dtype, seed=0, lo=-6.0, hi=0.7):
    g = torch.Generator().manual_seed(seed)
    mk = lambda *s: torch.randn(*s, generator=g).to(dtype)  # noqa: E731
    q, k, v, go = mk(B, Hq, N, D), mk(B, Hkv, N, D), mk(B, Hkv, N, Dv), mk(B, Hq, N, Dv)
    ld = -torch.exp(lo + (hi - lo) * torch.rand(Hkv, generator=g))
    S0, dS1 = torch.randn(B, Hkv, D, Dv, generator=g), torch.randn(B, Hkv, D, Dv, generator=g)
    return q, k, v, go, ld, S0, dS1


def run(shape, dtype, scale=0.25, state=True, lengths=None, seed=0, backward=True):
    B, Hq, Hkv, N, D, Dv = shape
    check.dtype = dtype
    q, k, v, go, ld, S0, dS1 = draw(*shape, dtype, seed)
    if not state:
        S0 = dS1 = None
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    tc = la.decay_kernel_path(B, Hq, Hkv, N, D, dtype, False, Dv=Dv) == la.LA_PATH_TCGEN05
    S1 = torch.full((B, Hkv, D, Dv), float("nan"), device="cuda")
    out = la.decay_fwd(q.cuda(), k.cuda(), v.cuda(), ld.cuda(), scale=scale, initial_state=dev(S0), final_state=S1,
                       lengths=dev(lengths))
    la.get_status()
    want = od.fwd(q, k, v, ld, scale, S0, lengths)
    A = od.fwd(q.abs(), k.abs(), v.abs(), ld, scale, None if S0 is None else S0.abs(), lengths)
    check(out, want[0], A[0], N, D, tc, "out")
    check(S1, want[1], A[1], N, D, tc, "final_state")
    if not backward:
        return
    dS0 = torch.full((B, Hkv, D, Dv), float("nan"), device="cuda")
    args = (q.cuda(), k.cuda(), v.cuda(), go.cuda(), ld.cuda())
    kw = dict(scale=scale, initial_state=dev(S0), grad_final_state=dev(dS1), grad_initial_state=dS0)
    got = la.decay_bwd(*args, **kw)
    first = [t.clone() for t in got + (dS0,)]
    again = la.decay_bwd(*args, **kw)
    la.get_status()
    for a, b in zip(first, again + (dS0,)):
        assert torch.equal(a, b)     # a fixed order of sums
    want = od.bwd(q, k, v, go, ld, scale, S0, dS1)
    A = od.bwd(q.abs(), k.abs(), v.abs(), go.abs(), ld, scale, None if S0 is None else S0.abs(),
               None if dS1 is None else dS1.abs())
    W = max(D, Dv) * (Hq // Hkv)
    for name, a, b, c in zip(("dq", "dk", "dv", "grad_initial_state"), first, want, A):
        check(a, b, c, N, W, tc, name)


BF, F = torch.bfloat16, torch.float32
SHAPES = [
    # B, Hq, Hkv, N, D, Dv: one token, chunk borders and their neighbours, odd lengths, shared heads
    (1, 1, 1, 1, 64, 64), (2, 2, 2, 2, 128, 128), (1, 2, 1, 31, 64, 128), (1, 3, 1, 32, 128, 64), (2, 2, 1, 33, 64, 64),
    (1, 1, 1, 127, 128, 128), (1, 2, 2, 128, 64, 64), (1, 2, 1, 129, 128, 128), (3, 6, 2, 257, 64, 128),
    (1, 5, 1, 300, 128, 64), (1, 8, 1, 200, 64, 64), (1, 2, 2, 513, 128, 128), (2, 4, 4, 640, 64, 64),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_parity(shape, dtype):
    run(shape, dtype)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("D,Dv", [(32, 32), (32, 128), (128, 32), (64, 32)])
def test_narrow_heads(D, Dv, dtype):
    run((1, 4, 2, 150, D, Dv), dtype)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_long_sequence_in_segments(dtype):
    """Few heads and many tokens: the sequence is cut, and the segments' states are joined."""
    shape = (1, 2, 1, 2777, 64, 64)
    assert la.decay_workspace_size(*shape[:5], dtype, True) > 0
    run(shape, dtype)
    run((1, 2, 1, 2560, 128, 128), dtype, state=False, seed=2)


@pytest.mark.parametrize("D,Dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("reps,N", [(1, 1), (1, 257), (3, 130), (2, 640), (1, 1400), (5, 1300)])
def test_no_state_goes_out(reps, N, D, Dv):
    """Without final_state and grad_initial_state: the kernels that round y once.  Given and absent initial states,
    lengths, views of one projection."""
    check.dtype = BF
    Hkv = 2
    q, k, v, go, ld, S0, dS1 = draw(2, reps * Hkv, Hkv, N, D, Dv, BF, seed=N + reps)
    views = [t.transpose(1, 2).contiguous().cuda().transpose(1, 2) for t in (q, k, v, go)]
    n = torch.tensor([N, N // 2], dtype=torch.int32)
    for lengths, state in ((None, S0), (n, None)):
        out = la.decay_fwd(*views[:3], ld.cuda(), scale=0.25, initial_state=None if state is None else state.cuda(),
                           lengths=None if lengths is None else lengths.cuda())
        want, A = od.fwd(q, k, v, ld, 0.25, state, lengths)[0], \
            od.fwd(q.abs(), k.abs(), v.abs(), ld, 0.25, None if state is None else state.abs(), lengths)[0]
        check(out, want, A, N, D, True, "out", factors=3)
    for state, dstate in ((S0, None), (None, dS1)):
        got = la.decay_bwd(*views, ld.cuda(), scale=0.25, initial_state=None if state is None else state.cuda(),
                           grad_final_state=None if dstate is None else dstate.cuda())
        want = od.bwd(q, k, v, go, ld, 0.25, state, dstate)
        A = od.bwd(q.abs(), k.abs(), v.abs(), go.abs(), ld, 0.25, None if state is None else state.abs(),
                   None if dstate is None else dstate.abs())
        for name, a, b, c in zip(("dq", "dk", "dv"), got, want, A):
            check(a, b, c, N, max(D, Dv) * reps, True, name, factors=3)
    la.get_status()


@pytest.mark.parametrize("shape", [(6, 12, 4, 3699, 64, 64), (2, 16, 16, 4000, 128, 128), (2, 32, 4, 8192, 128, 128)],
                         ids=lambda s: "x".join(map(str, s)))
def test_states_of_long_memories(shape):
    """Sums over long memories in cut sequences.  y's two terms leave 2^-17 of each product; the matrix units cut their
    sums at each step of 16 tokens (2^-24 of the sum so far), which the steps within the memory, two a token's head, add
    up over the 512 / Dv accumulators that take turns."""
    B, Hq, Hkv, N, D, Dv = shape
    r, memory = Hq // Hkv, 1000
    assert la.decay_workspace_size(B, Hq, Hkv, N, D, BF, False, Dv=Dv) > 0
    q, k, v, go = (t.cuda() for t in draw(*shape, BF, 13)[:4])
    ld = torch.full((Hkv,), -1.0 / memory, device="cuda")
    S1, dS0 = torch.empty(B, Hkv, D, Dv, device="cuda"), torch.empty(B, Hkv, D, Dv, device="cuda")
    la.decay_fwd(q, k, v, ld, final_state=S1)
    la.decay_bwd(q, k, v, go, ld, grad_initial_state=dS0)
    la.get_status()
    j = torch.arange(N, device="cuda", dtype=torch.float64)
    l = float(ld[0])
    S = (k.double() * torch.exp(l * (N - 1 - j))[:, None]).transpose(2, 3) @ v.double()
    w = (q.double() * torch.exp(l * (j + 1))[:, None]).transpose(2, 3) @ go.double()
    for name, got, want, heads in (("S", S1, S, 1), ("dS", dS0, w.view(B, Hkv, r, D, Dv).sum(2), r)):
        bound = 2.0 ** -17 + 2.0 ** -24 * memory * heads * 2 / 16 / (512 // Dv)
        assert float((got - want).norm() / want.norm()) < bound, name


def test_offsets_past_32_bits():
    """Tensors of more than 2^31 elements, and a slot whose state lies past 2^31 floats."""
    B, H, N, D = 2, 16, 530000, 128
    assert B * H * N * D > 2 ** 31
    part = torch.randn(4, 4001, D, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    x = torch.empty(B, H, N, D, dtype=BF, device="cuda")
    q, k, v = x.fill_(1.0), torch.zeros_like(x), torch.zeros_like(x)
    q[-1, -1, -4001:], k[-1, -1, -4001:], v[-1, -1, -4001:] = part[0], part[1], part[2]
    ld = torch.full((H,), -0.02, device="cuda")
    got = [t[-1:, -1:, -4001:].clone() for t in (la.decay_fwd(q, k, v, ld),)]
    g = torch.zeros_like(x)
    g[-1, -1, -4001:] = part[3]
    got += [t[-1:, -1:, -4001:].clone() for t in la.decay_bwd(q, k, v, g, ld)]
    la.get_status()
    small = [p[None, None].contiguous() for p in part]
    want = (la.decay_fwd(*small[:3], ld[-1:]),) + la.decay_bwd(*small, ld[-1:])
    for a, b in zip(got, want):
        # both are within four half steps of the exact rows, which random signs make of a like size
        assert float((a.float() - b.float()).norm() / b.float().norm()) < 8 * 2.0 ** -8
    del x, q, k, v, g
    pool, Hkv = 16500, 8
    assert (pool - 1) * Hkv * D * D > 2 ** 31
    state = torch.zeros(pool, Hkv, D, D, device="cuda")
    state[-1] = torch.randn(Hkv, D, D, generator=torch.Generator().manual_seed(6)).cuda()
    mine = state[-1:].clone()
    t = [torch.randn(1, Hkv, 1, D, device="cuda") for _ in range(3)]
    out = la.decay_step(*t, state, ld[:Hkv], slots=torch.tensor([pool - 1], dtype=torch.int32, device="cuda"))
    assert torch.equal(out, la.decay_step(*t, mine, ld[:Hkv])) and torch.equal(state[-1:], mine)
    assert not state[:-1].any()


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("N", [50, 1500])
def test_lengths_and_what_lies_past_them(dtype, N):
    shape = (6, 4, 2, N, 64, 128)
    n = torch.tensor([0, 1, N, N + 9, N // 2 + 1, -3], dtype=torch.int32)
    run(shape, dtype, lengths=n, backward=False)
    q, k, v, _, ld, S0, _ = (t.cuda() for t in draw(*shape, dtype, 4))
    want, S1 = [la.decay_fwd(q, k, v, ld, initial_state=S0, lengths=n.cuda(), final_state=(S := torch.empty_like(S0))), S]
    for b, m in enumerate(n.clamp(0, N).tolist()):
        for i, t in enumerate((q, k, v)):
            t[b, :, m:] = (float("nan"), float("inf"), -float("inf"))[i]
    S = S0.clone()     # in place
    out = la.decay_fwd(q, k, v, ld, initial_state=S, final_state=S, lengths=n.cuda())
    la.get_status()
    assert torch.equal(out, want) and torch.equal(S, S1)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_extreme_decays(dtype):
    """No decay, a decay to nothing, one that underflows within a chunk."""
    check.dtype = dtype
    B, Hq, Hkv, N, D = 1, 4, 4, 400, 64
    q, k, v, go, _, S0, dS1 = draw(B, Hq, Hkv, N, D, D, dtype, 7)
    ld = torch.tensor([0.0, -float("inf"), -3.0, -1e-5])
    S1 = torch.empty(B, Hkv, D, D, device="cuda")
    out = la.decay_fwd(q.cuda(), k.cuda(), v.cuda(), ld.cuda(), initial_state=S0.cuda(), final_state=S1)
    dS0 = torch.empty_like(S1)
    grads = la.decay_bwd(q.cuda(), k.cuda(), v.cuda(), go.cuda(), ld.cuda(), initial_state=S0.cuda(),
                         grad_final_state=dS1.cuda(), grad_initial_state=dS0)
    la.get_status()
    tc = la.decay_kernel_path(B, Hq, Hkv, N, D, dtype, False) == la.LA_PATH_TCGEN05
    want = od.fwd(q, k, v, ld, 1.0, S0) + od.bwd(q, k, v, go, ld, 1.0, S0, dS1)
    A = od.fwd(q.abs(), k.abs(), v.abs(), ld, 1.0, S0.abs()) + \
        od.bwd(q.abs(), k.abs(), v.abs(), go.abs(), ld, 1.0, S0.abs(), dS1.abs())
    for name, a, b, c in zip(("out", "final_state", "dq", "dk", "dv", "grad_initial_state"), (out, S1) + grads + (dS0,), want, A):
        check(a, b, c, N, D, tc, name)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_strided_views_other_stream_and_poisoned_workspace(dtype):
    """Views into one projection [B, N, heads, D], on another stream, with workspaces of 0xFF."""
    B, Hq, Hkv, N, D = 2, 4, 2, 1111, 64
    g = torch.Generator().manual_seed(3)
    x = torch.randn(B, N, Hq + 2 * Hkv, D, generator=g).to(dtype).cuda()
    q, k, v = (t.permute(0, 2, 1, 3) for t in (x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]))
    go = torch.randn(B, N, Hq, D, generator=g).to(dtype).cuda().permute(0, 2, 1, 3)
    ld = torch.tensor([-0.01, -0.3]).cuda()
    want = (la.decay_fwd(q.contiguous(), k.contiguous(), v.contiguous(), ld),) + \
        la.decay_bwd(q.contiguous(), k.contiguous(), v.contiguous(), go.contiguous(), ld)
    ws = torch.full((max(1, la.decay_workspace_size(B, Hq, Hkv, N, D, dtype, True)),), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = (la.decay_fwd(q, k, v, ld, workspace=ws, stream=s),)
    got += la.decay_bwd(q, k, v, go, ld, workspace=ws, stream=s)
    s.synchronize()
    la.get_status()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_captured_into_a_graph():
    B, Hq, Hkv, N, D = 1, 2, 2, 1500, 64
    q, k, v, go, ld, S0, dS1 = (t.cuda() for t in draw(B, Hq, Hkv, N, D, D, BF, 11))
    S1, dS0 = torch.empty_like(S0), torch.empty_like(S0)
    ws = torch.empty(la.decay_workspace_size(B, Hq, Hkv, N, D, BF, True), dtype=torch.uint8, device="cuda")
    out, dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)

    def work():
        la.decay_fwd(q, k, v, ld, initial_state=S0, final_state=S1, out=out, workspace=ws)
        la.decay_bwd(q, k, v, go, ld, initial_state=S0, grad_final_state=dS1, grad_initial_state=dS0, dq=dq, dk=dk, dv=dv,
                     workspace=ws)

    work()
    torch.cuda.synchronize()
    want = [t.clone() for t in (out, S1, dq, dk, dv, dS0)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    for t in (out, S1, dq, dk, dv, dS0):
        t.zero_()
    graph.replay()
    la.get_status()
    for a, b in zip((out, S1, dq, dk, dv, dS0), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 32, 32), (3, 6, 2, 64, 128), (5, 11, 1, 128, 64), (2, 40, 2, 128, 128)])
def test_step(shape, dtype):
    """Scattered slots, padding rows, kept old states; strided inputs; the same as a prompt's next token."""
    B, Hq, Hkv, D, Dv = shape
    check.dtype = dtype
    q, k, v, _, ld, _, _ = draw(B, Hq, Hkv, 1, D, Dv, dtype, 21)
    pool = B + 3
    g = torch.Generator().manual_seed(1)
    state = torch.randn(pool, Hkv, D, Dv, generator=g)
    slots = torch.randperm(pool, generator=g)[:B].to(torch.int32)
    if B > 2:
        slots[0], slots[1] = -1, pool
    dev = state.cuda()
    new = torch.full_like(dev, 7.0)
    pad = torch.zeros(B, 2, Hkv, 3 * Dv, dtype=dtype).cuda()
    pad[:, 1, :, Dv:2 * Dv] = v[:, :, 0].cuda()
    vs = pad[:, 1:2, :, Dv:2 * Dv].permute(0, 2, 1, 3)
    out = la.decay_step(q.cuda(), k.cuda(), vs, dev, ld.cuda(), slots=slots.cuda(), scale=0.5, state_out=new)
    assert torch.equal(dev.cpu(), state)
    la.decay_step(q.cuda(), k.cuda(), vs, dev, ld.cuda(), slots=slots.cuda(), scale=0.5)
    la.get_status()
    for b in range(B):
        s = int(slots[b])
        if not 0 <= s < pool:
            assert not out[b].any()
            continue
        one = slice(b, b + 1)
        want = od.fwd(q[one], k[one], v[one], ld, 0.5, state[s:s + 1])
        A = od.fwd(q[one].abs(), k[one].abs(), v[one].abs(), ld, 0.5, state[s:s + 1].abs())
        check(out[one], want[0], A[0], 1, D, False, "out")
        check(new[s:s + 1], want[1], A[1], 1, D, False, "final_state")
        assert torch.equal(new[s], dev[s])
    others = [s for s in range(pool) if s not in slots.tolist()]
    assert (new[others] == 7.0).all() and torch.equal(dev[others].cpu(), state[others])


def test_prompt_then_tokens():
    """A prompt's last state carried on token by token gives the longer prompt's rows."""
    B, Hq, Hkv, N, D = 2, 4, 2, 70, 64
    check.dtype = BF
    q, k, v, _, ld, _, _ = draw(B, Hq, Hkv, N, D, D, BF, 31)
    dev = [t.cuda() for t in (q, k, v)]
    S = torch.empty(B, Hkv, D, D, device="cuda")
    la.decay_fwd(*(t[:, :, :64] for t in dev), ld.cuda(), final_state=S)
    rows = [la.decay_step(*(t[:, :, i:i + 1] for t in dev), S, ld.cuda()) for i in range(64, N)]
    la.get_status()
    want = od.fwd(q, k, v, ld)
    A = od.fwd(q.abs(), k.abs(), v.abs(), ld)
    check(torch.cat(rows, 2), want[0][:, :, 64:], A[0][:, :, 64:], N, D, True, "out")
    check(S, want[1], A[1], N, D, True, "final_state")
