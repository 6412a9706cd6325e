"""The bounded waits of the decayed attention's tensor-core kernels: one that runs out is reported, every role of the
block leaves, and the library stays usable.

The test build of the library (``build(variant="test")``: waits of milliseconds) has a switch that makes warp 4 of
block 0 withhold its first arrival: of the scores' decay in the passes (1), of the decayed y in the sums, which every state that goes out comes from (2).  The MMA
warp's wait for it runs out, and with it, one after the other, the waits of the roles that depend on it.  No
kernel traps or faults: the waits end with an error status."""
import ctypes

import pytest
import torch

from efficient_transformer_gb300 import build as la_build
from efficient_transformer_gb300 import la

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def tlib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    la_build.build()
    la.load()
    lib = la.load(la_build.build(variant="test"))
    lib.la_test_withhold_decay.argtypes = [ctypes.c_int]
    lib.la_test_withhold_decay.restype = ctypes.c_int
    return lib


def status(lib):
    return lib.la_get_status(ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))


# B, Hq, Hkv, N, D, Dv: fewer chunks than stages and more, shared heads, every width
SHAPES = [(1, 2, 2, 100, 64, 64), (2, 4, 1, 1000, 64, 64), (2, 4, 2, 900, 128, 128), (1, 2, 2, 1500, 64, 128),
          (1, 3, 1, 700, 128, 64)]


@pytest.mark.parametrize("bwd", [False, True], ids=["fwd", "bwd"])
@pytest.mark.parametrize("which", [1, 2], ids=["passes", "sums"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_clean(tlib, shape, which, bwd, monkeypatch):
    B, Hq, Hkv, N, D, Dv = shape
    assert la.decay_kernel_path(B, Hq, Hkv, N, D, BF, bwd, Dv=Dv) == la.LA_PATH_TCGEN05
    g = torch.Generator(device="cuda").manual_seed(4)
    q, k, v, go = (torch.randn(B, h, N, w, device="cuda", generator=g).to(BF) for h, w in ((Hq, D), (Hkv, D), (Hkv, Dv), (Hq, Dv)))
    ld = torch.full((Hkv,), -0.02, device="cuda")
    lengths = None if bwd else torch.tensor([N - 7 * b for b in range(B)], dtype=torch.int32, device="cuda")

    def call():
        S = torch.zeros(B, Hkv, D, Dv, device="cuda")
        if bwd:
            return la.decay_bwd(q, k, v, go, ld, grad_initial_state=S) + (S,)
        return la.decay_fwd(q, k, v, ld, final_state=S, lengths=lengths), S

    want = call()
    la.get_status()
    monkeypatch.setattr(la, "load", lambda *a: tlib)
    assert status(tlib) == la.LA_OK
    assert tlib.la_test_withhold_decay(which) == 0
    try:
        call()                                              # enqueued; the kernel runs out later
        assert status(tlib) == la.LA_ERR_TIMEOUT            # reported once ...
    finally:
        assert tlib.la_test_withhold_decay(0) == 0
    assert status(tlib) == la.LA_OK                         # ... and cleared
    got = call()
    assert status(tlib) == la.LA_OK
    for a, b in zip(got, want):
        assert torch.equal(a, b)
