"""Calls on a stream of their own while torch's current one goes on allocating: the side stream is kept busy, so that
its kernels start only after the caller has dropped the inputs and filled as much new memory as the calls use."""
import pytest
import torch

from efficient_transformer_gb300 import build as la_build
from efficient_transformer_gb300 import la

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    la_build.build()
    la.load()


def inputs(*shapes):
    g = torch.Generator().manual_seed(0)
    return [torch.randn(*s, generator=g).to(BF).cuda() for s in shapes]


B, HQ, HKV, N, D = 1, 4, 2, 2500, 64
QKV = [(B, HQ, N, D), (B, HKV, N, D), (B, HKV, N, D)]


def small():
    """The calls' vectors, which the caller keeps."""
    return dict(ld=torch.tensor([-0.02, -0.2], device="cuda"),
                rope=dict(q_weight=torch.ones(D, device="cuda"), k_weight=torch.full((D,), 0.5, device="cuda"),
                          positions=torch.arange(N, device="cuda")[None],
                          inv_freq=torch.ones(8, dtype=torch.float64, device="cuda")))


CALLS = {
    "fwd": (QKV, lambda t, c, **k: (la.fwd(*t, is_causal=True, **k),)),
    "bwd": (QKV + QKV[:1], lambda t, c, **k: la.bwd(*t, is_causal=True, **k)),
    "lowrank_bwd": ([(700, 512), (256, 64), (64, 512), (700, 256)], lambda t, c, **k: la.lowrank_bwd(*t, **k)[:3]),
    "decay_fwd": (QKV, lambda t, c, **k: (la.decay_fwd(*t, c["ld"], **k),)),
    "decay_bwd": (QKV + QKV[:1], lambda t, c, **k: la.decay_bwd(*t, c["ld"], **k)),
    "qk_norm_rope_bwd": (QKV[:2] * 2, lambda t, c, **k: la.qk_norm_rope_bwd(*t, **c["rope"], **k)),
}


@pytest.mark.parametrize("name", CALLS)
def test_memory_is_not_reused_while_the_side_stream_runs(name):
    shapes, call = CALLS[name]
    given, consts = inputs(*shapes), small()
    want = call(given, consts)
    dropped = [t.clone() for t in given]
    here, side = torch.cuda.current_stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)
    got = call(dropped, consts, stream=side)
    del dropped
    # as much memory again as the call had, in blocks of every size that it used
    sizes = [t.numel() * t.element_size() for t in list(given) + list(want)] + [1 << n for n in range(12, 26, 2)]
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    here.wait_stream(side)
    la.get_status()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    del junk
