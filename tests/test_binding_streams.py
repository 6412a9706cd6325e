"""Memory of calls on another stream than torch's current one, on the host with stand-ins (binding_fakes).

torch's allocator reuses a block in the order of the stream that it was allocated on.  So what a call allocates for
itself has to be memory of the stream that its kernels run on, and what both streams touch has to be
recorded on the one that it is not of."""
import pytest
import torch

from binding_fakes import FakeStream, World, fake
from efficient_transformer_gb300 import la

B, HQ, HKV, N, D = 2, 4, 2, 8, 32
F = torch.float32


def qkv(**kw):
    return [fake(B, h, N, D, **kw) for h in (HQ, HKV, HKV)]


def calls():
    """name: (function, its tensors, tensors by keyword, number of tensors that it returns)"""
    q, k, v = qkv()
    go, ld = fake(B, HQ, N, D), fake(HKV, dtype=F)
    S = [fake(B, HKV, D, D, dtype=F) for _ in range(3)]
    rope = dict(positions=fake(B, N, dtype=torch.int64), inv_freq=fake(D // 2, dtype=torch.float64))
    w = dict(q_weight=fake(D, dtype=F), k_weight=fake(D, dtype=F))
    cos = [fake(N, dtype=F) for _ in range(2)]
    x, U, V = fake(8, 32), fake(48, 16), fake(16, 32)
    one = [fake(B, h, 1, D) for h in (HQ, HKV, HKV)]
    return {
        "fwd": (la.fwd, [q, k, v], dict(cos_weight=cos[0], sin_weight=cos[1]), 1),
        "bwd": (la.bwd, [q, k, v, go], {}, 3),
        "lowrank_fwd": (la.lowrank_fwd, [x, U, V, fake(48)], {}, 1),
        "lowrank_bwd": (la.lowrank_bwd, [x, U, V, fake(8, 48), fake(48)], {}, 4),
        "decay_fwd": (la.decay_fwd, [q, k, v, ld], dict(initial_state=S[0], final_state=S[1],
                                                        lengths=fake(B, dtype=torch.int32)), 1),
        "decay_bwd": (la.decay_bwd, [q, k, v, go, ld], dict(initial_state=S[0], grad_final_state=S[1],
                                                            grad_initial_state=S[2]), 3),
        "decay_step": (la.decay_step, one + [fake(5, HKV, D, D, dtype=F), ld], dict(slots=fake(B, dtype=torch.int32)), 1),
        "qk_norm_rope_fwd": (la.qk_norm_rope_fwd, [q, k], dict(w, **rope), 2),
        "qk_norm_rope_bwd": (la.qk_norm_rope_bwd, [q, k, go, k.clone().as_subclass(type(k))], dict(w, **rope), 4),
    }


NAMES = ["fwd", "bwd", "lowrank_fwd", "lowrank_bwd", "decay_fwd", "decay_bwd", "decay_step", "qk_norm_rope_fwd",
         "qk_norm_rope_bwd"]


@pytest.mark.parametrize("name", NAMES)
def test_on_another_stream(name, monkeypatch):
    w, side = World(monkeypatch), FakeStream("side")
    f, args, kw, n = calls()[name]
    got = f(*args, **kw, stream=side)
    got = got if isinstance(got, tuple) else (got,)
    assert len(got) == n and len(w.lib.calls) >= 1
    assert w.allocated and {s for _, s in w.allocated} == {"side"}
    for t in got:
        assert set(t.recorded) == {"home", "side"}
    for t in args + list(kw.values()):
        assert t.recorded == ["side"]
    # scratch: memory of the side stream, which nothing else meets
    for t, _ in w.allocated:
        assert any(t is x for x in got) or not hasattr(t, "recorded")
    assert w.current == [w.home]
    stream = [a for call, a in w.lib.calls if "workspace" not in call][-1][-1]
    assert getattr(stream, "value", stream) in (side.cuda_stream, side.cuda_stream % 2 ** 64)


@pytest.mark.parametrize("name", NAMES)
def test_on_the_current_stream(name, monkeypatch):
    """Nothing to record: one stream orders everything."""
    w = World(monkeypatch)
    f, args, kw, _ = calls()[name]
    for extra in ({}, dict(stream=w.home)):
        f(*args, **kw, **extra)
    assert {s for _, s in w.allocated} == {"home"}
    assert not any(hasattr(t, "recorded") for t in args + list(kw.values()) + [t for t, _ in w.allocated])


def test_buffers_of_the_caller(monkeypatch):
    w, side = World(monkeypatch), FakeStream("side")
    q, k, v = qkv()
    ld, go = fake(HKV, dtype=F), fake(B, HQ, N, D)
    out, ws = fake(B, HQ, N, D), fake(512, dtype=torch.uint8)
    la.decay_fwd(q, k, v, ld, out=out, workspace=ws, stream=side)
    grads = [fake(*t.shape) for t in (q, k, v)]
    la.decay_bwd(q, k, v, go, ld, dq=grads[0], dk=grads[1], dv=grads[2], workspace=ws, stream=side)
    assert not w.allocated
    assert all(set(t.recorded) >= {"side"} for t in [out, ws] + grads)
