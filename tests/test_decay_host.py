"""Refusals of the decayed attention and the query/key norm, on the host before any CUDA call."""
import ctypes

import pytest
import torch

from efficient_transformer_gb300 import build as la_build
from efficient_transformer_gb300 import la

FAKE = ctypes.c_void_p(0x10000)      # never dereferenced: every call below fails its checks
ODD = ctypes.c_void_p(0x10004)


@pytest.fixture(scope="module")
def lib():
    la_build.build()
    return la.load()


def ref(b, h, n):
    return ctypes.pointer(la.LaStrides(b, h, n))


def fwd(lib, **over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, out=FAKE, ld=FAKE, s0=None, s1=None, n=None, B=1, Hq=4, Hkv=2, N=4096, D=64, Dv=64,
             dt=la.LA_BF16, scale=1.0, sq=None, sk=None, sv=None, ws=None, nws=0, stream=None)
    assert set(over) <= set(a)
    a.update(over)
    return lib.la_decay_fwd(*a.values())


FWD = [(dict(q=None), la.LA_ERR_ARG), (dict(out=None), la.LA_ERR_ARG), (dict(ld=None), la.LA_ERR_ARG),
       (dict(B=0), la.LA_ERR_ARG), (dict(N=0), la.LA_ERR_ARG), (dict(Hq=5), la.LA_ERR_ARG), (dict(dt=9), la.LA_ERR_ARG),
       (dict(scale=0.0), la.LA_ERR_ARG), (dict(scale=float("inf")), la.LA_ERR_ARG), (dict(scale=float("nan")), la.LA_ERR_ARG),
       (dict(B=1 << 25, Hq=4), la.LA_ERR_ARG), (dict(sq=ref(-1, 64, 64)), la.LA_ERR_ARG),
       (dict(D=48), la.LA_ERR_UNSUPPORTED), (dict(Dv=256), la.LA_ERR_UNSUPPORTED),
       (dict(k=ODD), la.LA_ERR_ALIGN), (dict(s0=ODD), la.LA_ERR_ALIGN), (dict(s1=ODD), la.LA_ERR_ALIGN),
       (dict(ld=ctypes.c_void_p(0x10002)), la.LA_ERR_ALIGN), (dict(n=ctypes.c_void_p(0x10002)), la.LA_ERR_ALIGN),
       (dict(), la.LA_ERR_WORKSPACE), (dict(ws=FAKE, nws=16), la.LA_ERR_WORKSPACE),
       (dict(ws=ODD, nws=1 << 30), la.LA_ERR_ALIGN)]


@pytest.mark.parametrize("i", range(len(FWD)))
def test_fwd_rejects(lib, i):
    assert fwd(lib, **FWD[i][0]) == FWD[i][1]


def test_bwd_rejects(lib):
    a = [FAKE] * 8 + [None, None, None, 1, 4, 2, 4096, 64, 64, la.LA_BF16, 1.0, None, None, None, None, None, 0, None]
    for i in range(8):
        assert lib.la_decay_bwd(*(a[:i] + [None] + a[i + 1:])) == la.LA_ERR_ARG
    assert lib.la_decay_bwd(*a) == la.LA_ERR_WORKSPACE
    for i in (4, 5, 6, 8, 9, 10):
        assert lib.la_decay_bwd(*(a[:i] + [ODD] + a[i + 1:])) == la.LA_ERR_ALIGN
    for i in (8, 9):     # the initial state's gradient in place of a state that is read
        b = list(a)
        b[i] = b[10] = FAKE
        assert lib.la_decay_bwd(*b) == la.LA_ERR_ARG


def test_a_gradients_workspace_serves_the_forward(lib):
    for B, Hq, Hkv, N, D, Dv in ((1, 2, 2, 256, 32, 32), (2, 4, 2, 1111, 64, 64), (2, 16, 16, 8192, 128, 128), (1, 32, 8, 65536, 128, 64)):
        for dt in (torch.float32, torch.bfloat16):
            f, b = (la.decay_workspace_size(B, Hq, Hkv, N, D, dt, x, Dv=Dv) for x in (False, True))
            assert b >= f >= 0


def step(lib, **over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, out=FAKE, s=FAKE, so=FAKE, ld=FAKE, slots=None, pool=8, B=8, Hq=4, Hkv=2, D=64, Dv=64,
             dt=la.LA_BF16, scale=1.0, sq=None, sk=None, sv=None, stream=None)
    assert set(over) <= set(a)
    a.update(over)
    return lib.la_decay_step(*a.values())


STEP = [(dict(s=None), la.LA_ERR_ARG), (dict(so=None), la.LA_ERR_ARG), (dict(pool=0), la.LA_ERR_ARG),
        (dict(pool=7), la.LA_ERR_ARG), (dict(Hq=3), la.LA_ERR_ARG), (dict(sk=ref(64, -64, 64)), la.LA_ERR_ARG),
        (dict(D=96), la.LA_ERR_UNSUPPORTED), (dict(so=ODD), la.LA_ERR_ALIGN),
        (dict(slots=ctypes.c_void_p(0x10001)), la.LA_ERR_ALIGN)]


@pytest.mark.parametrize("i", range(len(STEP)))
def test_step_rejects(lib, i):
    assert step(lib, **STEP[i][0]) == STEP[i][1]


def args(**over):
    """la_qk_args of a valid call but for `over`."""
    keep = dict(sections=(ctypes.c_int * 2)(20, 12), strides=(ctypes.c_longlong * 3)(64, 64, 1))
    a = la.LaQkArgs(q_weight=0x10000, k_weight=0x10000, weight_dtype=la.LA_F32, eps=1e-6, normalize=1, rot=64, axes=2,
                    sections=keep["sections"], positions=0x10000, pos_strides=keep["strides"], inv_freq=0x10000)
    for n, v in over.items():
        setattr(a, n, v)
    a.keep = keep
    return a


QK = [(dict(eps=-1.0), la.LA_ERR_ARG), (dict(eps=float("nan")), la.LA_ERR_ARG), (dict(weight_dtype=7), la.LA_ERR_ARG),
      (dict(normalize=0), la.LA_ERR_ARG), (dict(rot=-16), la.LA_ERR_ARG), (dict(rot=80), la.LA_ERR_ARG),
      (dict(rot=24), la.LA_ERR_UNSUPPORTED), (dict(positions=None), la.LA_ERR_ARG), (dict(inv_freq=None), la.LA_ERR_ARG),
      (dict(axes=0), la.LA_ERR_ARG), (dict(axes=5), la.LA_ERR_ARG), (dict(sections=None), la.LA_ERR_ARG),
      (dict(sections=(ctypes.c_int * 2)(20, 13)), la.LA_ERR_ARG), (dict(sections=(ctypes.c_int * 2)(40, -8)), la.LA_ERR_ARG),
      (dict(pos_strides=(ctypes.c_longlong * 3)(64, -1, 1)), la.LA_ERR_ARG), (dict(positions=0x10004), la.LA_ERR_ALIGN),
      (dict(q_weight=0x10002), la.LA_ERR_ALIGN)]


@pytest.mark.parametrize("i", range(len(QK)))
def test_qk_args_rejected(lib, i):
    a = args(**QK[i][0])
    assert lib.la_qk_norm_rope_fwd(FAKE, FAKE, FAKE, FAKE, 1, 4, 2, 64, 64, la.LA_BF16, None, None, ctypes.byref(a),
                                   None) == QK[i][1]


def test_qk_rejects(lib):
    a = args()
    base = [FAKE, FAKE, FAKE, FAKE, 1, 4, 2, 64, 64, la.LA_BF16, None, None, ctypes.byref(a), None]

    def call(**over):
        c = list(base)
        for i, v in over.items():
            c[int(i[1:])] = v
        return lib.la_qk_norm_rope_fwd(*c)

    assert call(_0=None) == la.LA_ERR_ARG
    assert call(_12=None) == la.LA_ERR_ARG
    assert call(_5=0) == la.LA_ERR_ARG
    assert call(_8=96) == la.LA_ERR_UNSUPPORTED
    assert call(_2=ODD) == la.LA_ERR_ALIGN
    assert call(_10=ref(4 * 64 * 64, 64 * 64 + 4, 64)) == la.LA_ERR_ALIGN     # rows off 16-byte boundaries
    assert call(_11=ref(-8, 64 * 64, 64)) == la.LA_ERR_ARG
    bwd = [FAKE] * 8 + [1, 4, 2, 64, 64, la.LA_BF16, None, None, None, None, ctypes.byref(a), None, 0, None]
    assert lib.la_qk_norm_rope_bwd(*bwd) == la.LA_ERR_WORKSPACE
    bwd[2] = None
    assert lib.la_qk_norm_rope_bwd(*bwd) == la.LA_ERR_ARG


def test_plans(lib):
    """A workspace only where a sequence is cut, the same for every call of the same sizes."""
    w = la.decay_workspace_size
    assert w(1, 4, 2, 16, 64, torch.bfloat16, False) == 0
    assert w(1, 4, 2, 65536, 64, torch.bfloat16, False) > 0
    assert w(1, 4, 2, 65536, 64, torch.bfloat16, True) >= 2 * 4 * 2 * 64 * 64 * 2
    assert w(1, 5, 2, 65536, 64, torch.bfloat16, False) == 0
    assert w(1, 4, 2, 65536, 64, torch.bfloat16, False, Dv=48) == 0
    assert la.qk_norm_rope_workspace_size(1, 4, 2, 64, 64, torch.bfloat16) > 0
    assert la.decay_kernel_path(1, 4, 2, 65536, 64, torch.float32, False) == la.LA_PATH_SIMT


def test_binding_rejects_before_the_library():
    x = torch.zeros(1, 2, 4, 32)
    with pytest.raises(ValueError, match="CUDA"):
        la.decay_fwd(x, x, x, torch.zeros(2))
    with pytest.raises(ValueError, match="CUDA"):
        la.qk_norm_rope_fwd(x, x)
    with pytest.raises(ValueError, match="positions"):
        la._qk_args(x, None, None, 1e-6, torch.zeros(1, 4, dtype=torch.int32), torch.zeros(16, dtype=torch.float64), None,
                    False, True)
    with pytest.raises(ValueError, match="sections"):
        la._qk_args(x, None, None, 1e-6, torch.zeros(2, 1, 4, dtype=torch.int64), torch.zeros(16, dtype=torch.float64),
                    None, False, True)
    with pytest.raises(TypeError, match="weight"):
        la._qk_args(x, torch.zeros(32, dtype=torch.float16), None, 1e-6, None, None, None, False, True)
