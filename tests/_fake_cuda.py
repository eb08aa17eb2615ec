"""CPU stand-ins for CUDA tensors and for the library, to see what the Python
forms hand to the C entries without a GPU."""
import ctypes
import types

import torch


class _Fake(torch.Tensor):
    """A CPU tensor that says it lives on a GPU."""
    index = 0

    @property
    def is_cuda(self):
        return True

    @property
    def device(self):
        return torch.device("cuda", self.index)

    def get_device(self):
        return self.index


class Fake0(_Fake):
    pass


class Fake1(_Fake):
    index = 1


def fake(x, index=0):
    return x.as_subclass((Fake0, Fake1)[index])


def floats_at(address, n):
    """n float32 values of host memory."""
    return list((ctypes.c_float * n).from_address(address))


class StubLibrary:
    """Records every call of a C entry; ``at_call`` may look at the memory."""

    def __init__(self):
        self.calls = []
        self.at_call = None

    def __getattr__(self, name):
        if not name.startswith("vpce_"):
            raise AttributeError(name)
        if name.endswith("_workspace_bytes"):
            return lambda *args: 256

        def entry(*args):
            self.calls.append((name, args))
            if self.at_call is not None:
                self.at_call(name, args)
            return 0

        return entry


def install(monkeypatch, vpce):
    """The stub in the library's place, stream handle 7 on device 0."""
    lib = StubLibrary()
    monkeypatch.setattr(vpce, "_lib", lib)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 7, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(cuda_stream=7))
    return lib
