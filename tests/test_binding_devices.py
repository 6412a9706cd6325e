"""Calls whose tensors, stream and current device are not of one GPU are refused, on the host with stand-ins
(binding_fakes): the library would launch on the current device with another one's addresses."""
import pytest
import torch

from binding_fakes import FakeStream, World, fake
from efficient_transformer_gb300 import la
from test_binding_streams import B, D, F, HKV, HQ, N, NAMES, calls


@pytest.mark.parametrize("name", NAMES)
def test_one_tensor_on_another_device(name, monkeypatch):
    w = World(monkeypatch)
    f, args, kw, _ = calls()[name]
    f(*args, **kw)
    w.lib.calls.clear()
    # (a first tensor elsewhere: not on the current device)
    for t in args + list(kw.values()):
        t.index = 1
        with pytest.raises((ValueError, TypeError)):
            f(*args, **kw)
        t.index = 0
    assert not w.lib.calls


@pytest.mark.parametrize("name", NAMES)
def test_all_on_another_than_the_current_device(name, monkeypatch):
    w = World(monkeypatch)
    f, args, kw, _ = calls()[name]
    w.current_device = 1
    with pytest.raises(ValueError, match="current device"):
        f(*args, **kw)
    w.current_device = 0
    with pytest.raises(ValueError, match="stream"):
        f(*args, **kw, stream=FakeStream("far", 1))
    assert not w.lib.calls and not w.allocated
    f(*args, **kw, stream=FakeStream("near", 0))


def test_given_buffers_on_another_device(monkeypatch):
    w = World(monkeypatch)
    q, k, v, go, ld = fake(B, HQ, N, D), fake(B, HKV, N, D), fake(B, HKV, N, D), fake(B, HQ, N, D), fake(HKV, dtype=F)
    x, U, V, y = fake(8, 32), fake(48, 16), fake(16, 32), fake(8, 48)
    far, ws = fake(B, HQ, N, D, index=1), fake(4096, dtype=torch.uint8, index=1)
    step = [fake(B, h, 1, D) for h in (HQ, HKV, HKV)] + [fake(5, HKV, D, D, dtype=F), ld]
    for call in (lambda: la.fwd(q, k, v, out=far), lambda: la.fwd(q, k, v, workspace=ws),
                 lambda: la.bwd(q, k, v, go, dq=far), lambda: la.bwd(q, k, v, go, workspace=ws),
                 lambda: la.lowrank_fwd(x, U, V, out=fake(8, 48, index=1)),
                 lambda: la.lowrank_fwd(x, U, V, t_out=fake(8, 16, index=1)),
                 lambda: la.lowrank_bwd(x, U, V, y, workspace=ws), lambda: la.lowrank_bwd(x, U, V, y, t=fake(8, 16, index=1)),
                 lambda: la.decay_fwd(q, k, v, ld, out=far), lambda: la.decay_fwd(q, k, v, ld, workspace=ws),
                 lambda: la.decay_bwd(q, k, v, go, ld, dq=far), lambda: la.decay_bwd(q, k, v, go, ld, workspace=ws),
                 lambda: la.decay_step(*step, state_out=fake(5, HKV, D, D, dtype=F, index=1)),
                 lambda: la.qk_norm_rope_fwd(q, k, q_out=far), lambda: la.qk_norm_rope_bwd(q, k, go, k, dq=far)):
        with pytest.raises(ValueError):
            call()
    assert all("workspace" in name for name, _ in w.lib.calls)
