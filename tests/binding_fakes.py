"""Stand-ins for CUDA tensors, streams and the library, with which the binding runs on the host: what it
allocates is logged with the stream that is current then, and every record_stream."""
import contextlib

import torch

from efficient_transformer_gb300 import la


class FakeStream:
    def __init__(self, name, index=0):
        self.name, self.cuda_stream, self.device = name, hash(name), torch.device("cuda", index)


class FakeCuda(torch.Tensor):
    """A host tensor that says it is on a GPU."""
    index = 0
    is_cuda = property(lambda t: True)
    device = property(lambda t: torch.device("cuda", t.index))

    def get_device(self):
        return self.index

    def record_stream(self, stream):
        self.recorded = getattr(self, "recorded", []) + [stream.name]

    def new_empty(self, shape, **kw):
        return torch.empty(shape, dtype=kw.get("dtype", self.dtype), device=self.device)


def fake(*shape, dtype=torch.bfloat16, index=0):
    t = _host_empty(shape, dtype=dtype).as_subclass(FakeCuda)
    t.index = index
    return t


_host_empty = torch.empty


class FakeLib:
    """Every call succeeds; every workspace takes 512 bytes."""
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 512 if "workspace" in name else 0
        return call


class World:
    def __init__(self, monkeypatch):
        self.lib, self.home, self.allocated, self.current_device = FakeLib(), FakeStream("home"), [], 0
        self.current = [self.home]

        def empty(*shape, dtype=None, device=None):
            shape = shape[0] if len(shape) == 1 and not isinstance(shape[0], int) else shape
            t = fake(*shape, dtype=dtype, index=torch.device(device).index or 0)
            self.allocated.append((t, self.current[-1].name))
            return t

        @contextlib.contextmanager
        def stream(s):
            self.current.append(s)
            yield
            self.current.pop()

        patch = monkeypatch.setattr
        patch(torch, "empty", empty)
        patch(torch, "empty_like", lambda t: empty(t.shape, dtype=t.dtype, device=t.device))
        patch(torch.cuda, "stream", stream)
        patch(torch.cuda, "current_stream", lambda *a: self.current[-1])
        patch(torch.cuda, "current_device", lambda: self.current_device)
        patch(la, "_raw", None)
        patch(la, "load", lambda *a: self.lib)
        for name in ("_decay_need", "_qk_need"):
            patch(la, name, lambda *a: 512)
