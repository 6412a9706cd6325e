"""Refusals of the selective scan and the short convolution: of the C ABI, on the host before any CUDA call, and of the
binding, with stand-ins."""
import ctypes

import pytest
import torch

from binding_fakes import World, fake
from efficient_transformer_gb300 import build as la_build
from efficient_transformer_gb300 import la

FAKE = 0x10000      # never dereferenced: every call below fails its checks
ODD = 0x10008
F = torch.float32


@pytest.fixture(scope="module")
def lib():
    la_build.build()
    return la.load()


def ref(b, n, h=0):
    return ctypes.pointer(la.LaStrides(b, h, n))


# ---- convolution --------------------------------------------------------------------------------

def conv(lib, **over):
    a = dict(x=FAKE, w=FAKE, bias=FAKE, out=FAKE, s0=None, s1=None, n=None, B=2, N=64, E=128, W=4, dt=la.LA_BF16,
             wdt=la.LA_BF16, silu=1, sx=None, stream=None)
    assert set(over) <= set(a)
    a.update(over)
    return lib.la_conv_fwd(*a.values())


CONV = [(dict(x=None), la.LA_ERR_ARG), (dict(w=None), la.LA_ERR_ARG), (dict(out=None), la.LA_ERR_ARG),
        (dict(B=0), la.LA_ERR_ARG), (dict(N=0), la.LA_ERR_ARG), (dict(N=-4), la.LA_ERR_ARG), (dict(E=0), la.LA_ERR_ARG),
        (dict(dt=7), la.LA_ERR_ARG), (dict(wdt=7), la.LA_ERR_ARG), (dict(dt=la.LA_F32), la.LA_ERR_ARG),
        (dict(N=(1 << 30) + 1), la.LA_ERR_ARG), (dict(B=1 << 30, N=1 << 30), la.LA_ERR_ARG),
        (dict(W=1), la.LA_ERR_UNSUPPORTED), (dict(W=5), la.LA_ERR_UNSUPPORTED), (dict(E=100), la.LA_ERR_UNSUPPORTED),
        (dict(x=ODD), la.LA_ERR_ALIGN), (dict(w=ODD), la.LA_ERR_ALIGN), (dict(bias=ODD), la.LA_ERR_ALIGN),
        (dict(s0=ODD), la.LA_ERR_ALIGN), (dict(s1=ODD), la.LA_ERR_ALIGN), (dict(n=0x10002), la.LA_ERR_ALIGN),
        (dict(sx=ref(-8, 128)), la.LA_ERR_ARG), (dict(sx=ref(8192, 132)), la.LA_ERR_ALIGN),
        (dict(sx=ref(8196, 128)), la.LA_ERR_ALIGN), (dict(E=1 << 20, N=1 << 30, B=1), la.LA_ERR_ARG)]


@pytest.mark.parametrize("i", range(len(CONV)))
def test_conv_rejects(lib, i):
    assert conv(lib, **CONV[i][0]) == CONV[i][1]


def conv_bwd(lib, **over):
    a = dict(x=FAKE, w=FAKE, bias=FAKE, g=FAKE, dx=FAKE, dw=FAKE, db=FAKE, s0=None, ds1=None, ds0=None, n=None, B=2, N=64,
             E=128, W=4, dt=la.LA_BF16, wdt=la.LA_F32, silu=1, sx=None, sg=None, ws=None, nws=0, stream=None)
    assert set(over) <= set(a)
    a.update(over)
    return lib.la_conv_bwd(*a.values())


CONV_BWD = [(dict(g=None), la.LA_ERR_ARG), (dict(dx=None), la.LA_ERR_ARG), (dict(dw=None), la.LA_ERR_ARG),
            (dict(bias=None), la.LA_ERR_ARG), (dict(s0=FAKE, ds0=FAKE), la.LA_ERR_ARG), (dict(ds1=FAKE, ds0=FAKE), la.LA_ERR_ARG),
            (dict(sg=ref(8192, -128)), la.LA_ERR_ARG), (dict(sg=ref(8192, 4)), la.LA_ERR_ALIGN), (dict(ds1=ODD), la.LA_ERR_ALIGN),
            (dict(), la.LA_ERR_WORKSPACE), (dict(ws=FAKE, nws=64), la.LA_ERR_WORKSPACE),
            (dict(ws=FAKE + 16, nws=1 << 30), la.LA_ERR_ALIGN), (dict(W=9), la.LA_ERR_UNSUPPORTED)]


@pytest.mark.parametrize("i", range(len(CONV_BWD)))
def test_conv_bwd_rejects(lib, i):
    assert conv_bwd(lib, **CONV_BWD[i][0]) == CONV_BWD[i][1]


def conv_step(lib, **over):
    a = dict(x=FAKE, w=FAKE, bias=None, out=FAKE, s=FAKE, so=FAKE, slots=None, pool=8, B=8, E=128, W=3, dt=la.LA_F32,
             wdt=la.LA_F32, silu=0, sx=None, stream=None)
    assert set(over) <= set(a)
    a.update(over)
    return lib.la_conv_step(*a.values())


CONV_STEP = [(dict(s=None), la.LA_ERR_ARG), (dict(so=None), la.LA_ERR_ARG), (dict(pool=0), la.LA_ERR_ARG),
             (dict(pool=7), la.LA_ERR_ARG), (dict(B=-1), la.LA_ERR_ARG), (dict(so=ODD), la.LA_ERR_ALIGN),
             (dict(slots=0x10001), la.LA_ERR_ALIGN), (dict(sx=ref(130, 0)), la.LA_ERR_ALIGN)]


@pytest.mark.parametrize("i", range(len(CONV_STEP)))
def test_conv_step_rejects(lib, i):
    assert conv_step(lib, **CONV_STEP[i][0]) == CONV_STEP[i][1]


# ---- scan -----------------------------------------------------------------------------------------

def args(**over):
    a = la.LaSsmArgs(x=FAKE, dt=FAKE, B=FAKE, C=FAKE, z=FAKE, A=FAKE, skip=FAKE, dt_bias=FAKE, batch=2, N=64, E=128, S=16, G=2,
                     dtype=la.LA_BF16, softplus=1)
    for k, v in over.items():
        setattr(a, k, v)
    return a


ARGS = [(dict(x=None), la.LA_ERR_ARG), (dict(dt=None), la.LA_ERR_ARG), (dict(B=None), la.LA_ERR_ARG),
        (dict(C=None), la.LA_ERR_ARG), (dict(A=None), la.LA_ERR_ARG), (dict(batch=0), la.LA_ERR_ARG),
        (dict(N=0), la.LA_ERR_ARG), (dict(E=-8), la.LA_ERR_ARG), (dict(S=0), la.LA_ERR_ARG), (dict(G=0), la.LA_ERR_ARG),
        (dict(G=3), la.LA_ERR_ARG), (dict(dtype=5), la.LA_ERR_ARG), (dict(N=(1 << 30) + 1), la.LA_ERR_ARG),
        (dict(batch=1 << 24, E=1 << 10), la.LA_ERR_ARG), (dict(S=24), la.LA_ERR_UNSUPPORTED), (dict(S=128), la.LA_ERR_UNSUPPORTED),
        (dict(E=24, G=2), la.LA_ERR_UNSUPPORTED), (dict(x=ODD), la.LA_ERR_ALIGN), (dict(z=ODD), la.LA_ERR_ALIGN),
        (dict(A=ODD), la.LA_ERR_ALIGN), (dict(skip=0x10002), la.LA_ERR_ALIGN), (dict(dt_bias=0x10002), la.LA_ERR_ALIGN),
        (dict(initial_state=ODD), la.LA_ERR_ALIGN), (dict(lengths=0x10002), la.LA_ERR_ALIGN),
        (dict(x_strides=ref(8192, -128)), la.LA_ERR_ARG), (dict(dt_strides=ref(8192, 130)), la.LA_ERR_ALIGN),
        (dict(z_strides=ref(8190, 128)), la.LA_ERR_ALIGN), (dict(B_strides=ref(4096, 40, 12)), la.LA_ERR_ALIGN),
        (dict(C_strides=ref(4096, 40, -16)), la.LA_ERR_ARG)]


@pytest.mark.parametrize("i", range(len(ARGS)))
def test_scan_arguments(lib, i):
    a, want = args(**ARGS[i][0]), ARGS[i][1]
    big = 1 << 40
    assert lib.la_ssm_fwd(ctypes.byref(a), FAKE, None, None, 0, FAKE, big, None) == want
    g = la.LaSsmGrads(*[FAKE + 0x1000] * 9)
    assert lib.la_ssm_bwd(ctypes.byref(a), FAKE, None, None, FAKE, big, ctypes.byref(g), FAKE, big, None) == want
    if not any(k.endswith("strides") for k in ARGS[i][0]):
        a.N = 1 if a.N == 64 else a.N
        assert lib.la_ssm_step(ctypes.byref(a), FAKE, FAKE, FAKE, None, 1 << 25, None) == want


def test_scan_rejects(lib):
    a, big = args(), 1 << 40
    assert lib.la_ssm_fwd(None, FAKE, None, None, 0, FAKE, big, None) == la.LA_ERR_ARG
    assert lib.la_ssm_fwd(ctypes.byref(a), None, None, None, 0, FAKE, big, None) == la.LA_ERR_ARG
    assert lib.la_ssm_fwd(ctypes.byref(a), ODD, None, None, 0, FAKE, big, None) == la.LA_ERR_ALIGN
    assert lib.la_ssm_fwd(ctypes.byref(a), FAKE, ODD, None, 0, FAKE, big, None) == la.LA_ERR_ALIGN
    need = lib.la_ssm_states_size(2, 64, 128, 16)
    assert need == 2 * 8 * 128 * 16 * 4
    assert lib.la_ssm_fwd(ctypes.byref(a), FAKE, None, FAKE, need - 1, FAKE, big, None) == la.LA_ERR_WORKSPACE
    long = args(batch=1, N=65536, E=64, G=1)
    ws = lib.la_ssm_workspace_size(1, 65536, 64, 16, 1, la.LA_BF16, 0)
    assert ws > 0
    assert lib.la_ssm_fwd(ctypes.byref(long), FAKE, None, None, 0, FAKE, ws - 1, None) == la.LA_ERR_WORKSPACE
    assert lib.la_ssm_fwd(ctypes.byref(long), FAKE, None, None, 0, None, ws, None) == la.LA_ERR_WORKSPACE
    assert lib.la_ssm_fwd(ctypes.byref(long), FAKE, None, None, 0, FAKE + 16, ws, None) == la.LA_ERR_ALIGN


def test_scan_bwd_rejects(lib):
    names = ("dx", "ddt", "dB", "dC", "dz", "dA", "dskip", "ddt_bias", "grad_initial_state")
    big, need = 1 << 40, lib.la_ssm_states_size(2, 64, 128, 16)

    def call(a=None, g=FAKE, gs=None, ds1=None, states=FAKE, nst=need, ws=FAKE, nws=big, **grads):
        out = la.LaSsmGrads(*[FAKE + 0x1000] * 9)
        for k, v in grads.items():
            setattr(out, k, v)
        return lib.la_ssm_bwd(ctypes.byref(a or args()), g, gs, ds1, states, nst, ctypes.byref(out), ws, nws, None)

    for n in names[:6]:
        assert call(**{n: None}) == la.LA_ERR_ARG
    for n in names[:6] + names[8:]:
        assert call(**{n: ODD}) == la.LA_ERR_ALIGN
    assert call(g=None) == call(states=None) == la.LA_ERR_ARG
    assert call(a=args(z=None)) == call(a=args(skip=None)) == call(a=args(dt_bias=None)) == la.LA_ERR_ARG
    assert call(a=args(initial_state=FAKE + 0x1000)) == call(ds1=FAKE + 0x1000) == la.LA_ERR_ARG
    assert call(gs=ref(8192, 132)) == la.LA_ERR_ALIGN
    assert call(nst=need - 1) == call(ws=None) == call(nws=16) == la.LA_ERR_WORKSPACE
    assert call(ws=FAKE + 128) == la.LA_ERR_ALIGN


def test_scan_step_rejects(lib):
    def call(a, s=FAKE, so=FAKE, slots=None, pool=8, out=FAKE):
        return lib.la_ssm_step(ctypes.byref(a), out, s, so, slots, pool, None)

    one = lambda **k: args(N=1, **k)  # noqa: E731
    assert call(args()) == call(one(), s=None) == call(one(), so=None) == call(one(), out=None) == la.LA_ERR_ARG
    assert call(one(), pool=0) == call(one(), pool=1) == la.LA_ERR_ARG
    assert call(one(initial_state=FAKE)) == call(one(lengths=FAKE)) == la.LA_ERR_ARG
    assert call(one(), so=ODD) == call(one(), slots=0x10001) == la.LA_ERR_ALIGN


def test_sizes(lib):
    dt = la.LA_BF16
    assert lib.la_ssm_workspace_size(1, 64, 128, 24, 1, dt, 0) == lib.la_ssm_states_size(1, 0, 128, 16) == 0
    assert lib.la_conv_workspace_size(1, 64, 12, 4, dt) == 0
    for B, N, E, S, G in ((1, 1, 8, 8, 1), (2, 777, 200, 8, 1), (1, 65536, 2048, 16, 1), (8, 2048, 4096, 64, 4)):
        f, b = (lib.la_ssm_workspace_size(B, N, E, S, G, dt, x) for x in (0, 1))
        assert b >= f >= 0 and b >= 4 * (2 * B * N * G * S + B * E * (S + 2))


def test_sizes_past_the_offsets(lib):
    """Bytes of states that 64 bits do not hold, and grids past 31 bits, are refused, not cut off."""
    dt = la.LA_BF16
    assert lib.la_ssm_states_size(1, 1 << 30, 1 << 24, 64) == 0
    assert lib.la_ssm_workspace_size(1, 1 << 30, 1 << 24, 64, 1, dt, 1) == 0
    assert lib.la_ssm_states_size(1, 1 << 20, 1 << 13, 16) == (1 << 17) * (1 << 13) * 64
    big = (1 << 31) - 8
    assert lib.la_conv_step(FAKE, FAKE, None, FAKE, FAKE, FAKE, None, big, big, big, 4, dt, dt, 1, None, None) == la.LA_ERR_ARG


# ---- binding --------------------------------------------------------------------------------------

def tensors(**over):
    t = dict(x=fake(2, 6, 32), dt=fake(2, 6, 32), A=fake(32, 16, dtype=F), B=fake(2, 6, 2, 16), C=fake(2, 6, 2, 16))
    t.update(over)
    return tuple(t.values())


BAD = [dict(x=fake(2, 32)), dict(x=torch.empty(2, 6, 32)), dict(x=fake(2, 6, 32, dtype=torch.float16)),
       dict(dt=fake(2, 5, 32)), dict(dt=fake(2, 6, 32, dtype=F)), dict(dt=fake(2, 6, 64)[:, :, ::2]), dict(A=fake(32, 16)),
       dict(A=fake(32, 8, dtype=F)), dict(A=fake(16, 32, dtype=F).t()), dict(B=fake(2, 6, 16)), dict(B=fake(2, 6, 1, 16)),
       dict(C=fake(2, 6, 2, 32)), dict(C=None)]


@pytest.mark.parametrize("i", range(len(BAD)))
def test_binding_refuses_inputs(i, monkeypatch):
    w = World(monkeypatch)
    for call in (lambda *a: la.ssm_fwd(*a), lambda *a: la.ssm_bwd(*a, fake(2, 6, 32)),
                 lambda *a: la.ssm_step(*a, fake(4, 32, 16, dtype=F))):
        with pytest.raises((ValueError, TypeError)):
            call(*tensors(**BAD[i]))
    assert not w.lib.calls


def test_binding_refuses(monkeypatch):
    w = World(monkeypatch)
    monkeypatch.setattr(la, "_ssm_need", lambda *a: 512)
    monkeypatch.setattr(la, "ssm_states_size", lambda *a: 512)
    monkeypatch.setattr(la, "_conv_need", lambda *a: 512)
    t, x, wt = tensors(), fake(2, 6, 32), fake(32, 4)
    one = [fake(2, 1, 32), fake(2, 1, 32), fake(32, 16, dtype=F), fake(2, 1, 2, 16), fake(2, 1, 2, 16)]
    pool = fake(4, 32, 16, dtype=F)
    for call in (lambda: la.ssm_fwd(*t, z=fake(2, 6, 16)), lambda: la.ssm_fwd(*t, skip=fake(32)),
                 lambda: la.ssm_fwd(*t, dt_bias=fake(31, dtype=F)), lambda: la.ssm_fwd(*t, lengths=fake(2, dtype=torch.int64)),
                 lambda: la.ssm_fwd(*t, initial_state=fake(2, 16, 32, dtype=F)), lambda: la.ssm_fwd(*t, final_state=fake(2, 32, 16)),
                 lambda: la.ssm_fwd(*t, out=fake(2, 6, 64)[:, :, :32]), lambda: la.ssm_fwd(*t, states=fake(511, dtype=torch.uint8)),
                 lambda: la.ssm_fwd(*t, workspace=fake(511, dtype=torch.uint8)),
                 lambda: la.ssm_bwd(*t, fake(2, 6, 64)), lambda: la.ssm_bwd(*t, x, grad_final_state=fake(2, 32, 16)),
                 lambda: la.ssm_bwd(*t, x, states=fake(100, dtype=F)),
                 lambda: la.ssm_step(*t, pool), lambda: la.ssm_step(*one, fake(4, 32, 8, dtype=F)),
                 lambda: la.ssm_step(*one, pool, slots=fake(3, dtype=torch.int32)),
                 lambda: la.ssm_step(*one, pool, state_out=fake(5, 32, 16, dtype=F)),
                 lambda: la.conv_fwd(x, fake(16, 4)), lambda: la.conv_fwd(x, fake(4, 32).t()),
                 lambda: la.conv_fwd(x, wt, fake(32, dtype=F)), lambda: la.conv_fwd(x, fake(32, 4, dtype=torch.float16)),
                 lambda: la.conv_fwd(x, wt, initial_state=fake(2, 4, 32)), lambda: la.conv_fwd(x, wt, final_state=fake(2, 3, 32, dtype=F)),
                 lambda: la.conv_bwd(x, wt, fake(2, 6, 31)), lambda: la.conv_bwd(x, wt, x, dx=fake(2, 6, 32, dtype=F)),
                 lambda: la.conv_step(x, fake(4, 3, 32), wt), lambda: la.conv_step(one[0], fake(4, 4, 32), wt),
                 lambda: la.conv_step(one[0], fake(4, 3, 32), wt, slots=fake(2, dtype=torch.int64))):
        with pytest.raises((ValueError, TypeError)):
            call()
    assert not w.lib.calls


def calls():
    """name: (function, its tensors, tensors by keyword, number of tensors that it returns)"""
    t, x = tensors(), fake(2, 6, 32)
    one = [fake(2, 1, 32), fake(2, 1, 32), fake(32, 16, dtype=F), fake(2, 1, 2, 16), fake(2, 1, 2, 16), fake(4, 32, 16, dtype=F)]
    vec = lambda: dict(skip=fake(32, dtype=F), dt_bias=fake(32, dtype=F))  # noqa: E731
    state = lambda *names: {n: fake(2, 32, 16, dtype=F) for n in names}  # noqa: E731
    n = lambda: dict(lengths=fake(2, dtype=torch.int32))  # noqa: E731
    rows = lambda *names: {n: fake(2, 3, 32) for n in names}  # noqa: E731
    return {
        "ssm_fwd": (la.ssm_fwd, list(t), dict(vec(), **n(), **state("initial_state", "final_state"), z=fake(2, 6, 32)), 1),
        "ssm_bwd": (la.ssm_bwd, list(tensors()) + [fake(2, 6, 32)],
                    dict(vec(), **n(), **state("initial_state", "grad_final_state", "grad_initial_state"), z=fake(2, 6, 32)), 8),
        "ssm_step": (la.ssm_step, one, dict(vec(), slots=fake(2, dtype=torch.int32), z=fake(2, 1, 32),
                                            state_out=fake(4, 32, 16, dtype=F)), 1),
        "conv_fwd": (la.conv_fwd, [x, fake(32, 4), fake(32)], dict(n(), **rows("initial_state", "final_state")), 1),
        "conv_bwd": (la.conv_bwd, [x, fake(32, 4), fake(2, 6, 32), fake(32)],
                     dict(n(), **rows("initial_state", "grad_final_state", "grad_initial_state")), 3),
        "conv_step": (la.conv_step, [fake(2, 1, 32), fake(4, 3, 32), fake(32, 4), fake(32)],
                      dict(slots=fake(2, dtype=torch.int32), state_out=fake(4, 3, 32)), 1),
    }


NAMES = ["ssm_fwd", "ssm_bwd", "ssm_step", "conv_fwd", "conv_bwd", "conv_step"]


@pytest.fixture
def world(monkeypatch):
    w = World(monkeypatch)
    for name in ("_ssm_need", "ssm_states_size", "_conv_need"):
        monkeypatch.setattr(la, name, lambda *a: 512)
    return w


@pytest.mark.parametrize("name", NAMES)
def test_on_another_stream(name, world):
    """Memory of the side stream; what both streams touch is recorded."""
    from binding_fakes import FakeStream
    side = FakeStream("side")
    f, a, kw, n = calls()[name]
    got = f(*a, **kw, stream=side)
    got = got if isinstance(got, tuple) else (got,)
    assert len(got) == n and world.allocated and {s for _, s in world.allocated} == {"side"}
    for t in got:
        assert set(t.recorded) == {"home", "side"}
    for t in a + list(kw.values()):
        assert "side" in t.recorded
    for t, _ in world.allocated:
        assert any(t is x for x in got) or not hasattr(t, "recorded")
    assert [c[1][-1] for c in world.lib.calls if "size" not in c[0]][-1] == side.cuda_stream


@pytest.mark.parametrize("name", NAMES)
def test_on_the_current_stream(name, world):
    f, a, kw, _ = calls()[name]
    for extra in ({}, dict(stream=world.home)):
        f(*a, **kw, **extra)
    assert not any(hasattr(t, "recorded") for t in a + list(kw.values()) + [t for t, _ in world.allocated])


@pytest.mark.parametrize("name", NAMES)
def test_one_device(name, world):
    f, a, kw, _ = calls()[name]
    f(*a, **kw)
    world.lib.calls.clear()
    for t in a + list(kw.values()):
        t.index = 1
        with pytest.raises((ValueError, TypeError)):
            f(*a, **kw)
        t.index = 0
    world.current_device = 1
    with pytest.raises(ValueError, match="current device"):
        f(*a, **kw)
    assert not world.lib.calls
