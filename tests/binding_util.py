"""A stand-in for the GPU under the Python binding: tensors that say they are CUDA tensors, streams that only have a
name, and a library that records what it is given.  The binding's checks and allocations run on the CPU with it."""
import contextlib
import ctypes

import torch


class FakeStream:
    def __init__(self, cuda_stream, device=0):
        self.cuda_stream, self.device_index = cuda_stream, device


class FakeTensor(torch.Tensor):
    """Host memory under the name of a GPU; `made_on`: the current stream when the binding allocated it."""

    gpu, made_on, recorded, read_on = 0, None, (), None
    world = None  # of the FakeGpu that made it
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.gpu

    def record_stream(self, stream):
        self.recorded += (stream.cuda_stream,)

    def item(self):
        self.read_on = self.world.current.cuda_stream
        return self.world.counts.pop(0)


class FakeLibrary:
    """Every entry point succeeds; calls: (name, arguments)."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, [a.value if isinstance(a, ctypes.c_void_p) else a for a in args]))
            return 4096 if name.endswith("_size") else 0

        return call


class FakeGpu:
    def __init__(self, monkeypatch, eq):
        self.lib, self.current, self.made = FakeLibrary(), FakeStream(7), []
        self.counts = []  # what item() returns
        empty, zeros = torch.empty, torch.zeros

        def allocate(make):
            def fn(*shape, dtype=None, device=None):
                t = make(*shape, dtype=dtype).as_subclass(FakeTensor)
                t.made_on, t.world = self.current.cuda_stream, self
                self.made.append(t)  # kept: no address comes twice
                return t

            return fn

        @contextlib.contextmanager
        def on(stream):
            before, self.current = self.current, stream or self.current
            yield
            self.current = before

        def set_stream(stream):
            self.current = stream

        for where, name, value in ((torch, "empty", allocate(empty)), (torch, "zeros", allocate(zeros)),
                                   (torch.cuda, "stream", on), (torch.cuda, "set_stream", set_stream),
                                   (torch.cuda, "Stream", FakeStream), (torch.cuda, "current_stream", lambda *a: self.current),
                                   (torch.cuda, "current_device", lambda: 0),
                                   (torch._C, "_cuda_getCurrentRawStream", lambda dev: self.current.cuda_stream),
                                   (eq, "load_library", lambda: self.lib)):
            monkeypatch.setattr(where, name, value, raising=False)
        self._zeros = zeros

    def tensor(self, *shape, dtype=torch.float32, gpu=0):
        """A tensor of the caller's."""
        t = self._zeros(shape, dtype=dtype).as_subclass(FakeTensor)
        t.gpu = gpu
        return t

    def given(self, t):
        """Whether a call of the library got the address of t."""
        return any(t.data_ptr() in args for _, args in self.lib.calls)
