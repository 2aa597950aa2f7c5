"""Stand-ins for GPU tensors, torch's device and stream functions and the library, for tests of host code without a GPU:
they hold addresses that nothing reads, and record what is asked of them."""
import contextlib
import itertools
from types import SimpleNamespace

import torch

from zero_mixed_precision_amd import _lib


class Tensor:
    """A matrix or vector that says it lies on GPU ``index``."""

    is_cuda = True
    places = itertools.count(0x10000000, 0x1000000)

    def __init__(self, *shape, dtype=torch.bfloat16, index=0, at=None):
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, index
        self.at = next(Tensor.places) if at is None else at
        self.device = torch.device("cuda", index)
        self.recorded = []

    def stride(self):
        return (self.shape[1], 1) if len(self.shape) == 2 else (1,)

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return self.at

    def record_stream(self, stream):
        self.recorded.append(stream)


class Stream:
    cuda_stream = 0x5000


class Torch:
    """Of torch, the types, and a current device and stream that ``cuda.device`` and ``cuda.stream`` change."""

    def __init__(self, current=0):
        self.now = current
        self.cuda = SimpleNamespace(current_device=lambda: self.now, device=self._device, device_count=lambda: 2,
                                    current_stream=lambda *_: Stream(), ExternalStream=lambda handle: ("external", handle))
        for name in ("float16", "bfloat16", "float32", "bool", "uint8"):
            setattr(self, name, getattr(torch, name))

    @contextlib.contextmanager
    def _device(self, index):
        index = index.index if isinstance(index, torch.device) else index
        before, self.now = self.now, index
        try:
            yield
        finally:
            self.now = before


class Library:
    """Every entry point succeeds; ``calls`` has (name, current device, arguments)."""

    def __init__(self, fake):
        self.fake, self.calls = fake, []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, self.fake.now, args))
            return _lib.DS_OK
        return call


def balance(monkeypatch, stream=None, current=0, index=0):
    """An ExpertBalance of 64 experts over stand-ins: (object, torch, library)."""
    from zero_mixed_precision_amd import ExpertBalance

    fake = Torch(current)
    library = Library(fake)
    monkeypatch.setattr(_lib, "lib", library)
    monkeypatch.setattr(_lib, "_raw_stream", lambda i: 0x100 * i)
    op = ExpertBalance.__new__(ExpertBalance)
    op.torch, op.E, op.k, op.coef, op.stream, op._device = fake, 64, 8, 0.01, stream, index
    op.counts, op.value = Tensor(64, dtype=torch.int32, index=index), Tensor(dtype=torch.float32, index=index)
    op._mask_types = (torch.bool, torch.uint8)
    op._at = (1, 2, 3, 4, 5, 1 << 20)
    op._many = True
    return op, fake, library
