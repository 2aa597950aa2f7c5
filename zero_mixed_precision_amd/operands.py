"""What the operators over rows of tokens share: checks of their operands, streams and the GPU that launches go to."""
from __future__ import annotations

from . import _lib
from .multi_tensor import _dtype_of, check_stream


class TokenOperator:
    """An operator with arrays of its own on one GPU, run on ``stream`` (default: torch's current one)."""

    def __init__(self, device, stream):
        import torch

        self.torch, self.stream = torch, stream
        device = torch.device(device)
        if device.type == "cuda" and device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        check_stream(stream, device)
        self.device, self._device, self._many = device, device.index, torch.cuda.device_count() > 1
        self._index_types = (torch.int32, torch.int64)

    def _own(self):
        """The stream that the operator's arrays are made on."""
        from .checkpoint import torch_stream
        return self.torch.cuda.stream(torch_stream(self.stream, self.torch))

    def _here(self, x, what):
        if not x.is_cuda or x.get_device() != self._device:
            raise ValueError(f"{what}: expected a tensor on {self.device}, got one on {x.device}")

    def _rows(self, x, columns, what, rows=None, least=None):
        """(type, address, rows, row stride) of a [rows, columns] matrix whose rows lie any distance apart.  A small call's
        time is the host's: each property of a tensor is asked for once."""
        dt = _dtype_of(x, self.torch, what)
        shape = x.shape
        if not x.is_cuda or x.get_device() != self._device:
            self._here(x, what)
        if len(shape) != 2 or shape[1] != columns or (rows is not None and shape[0] != rows) or \
                (least is not None and shape[0] < least):
            some = rows if rows is not None else "rows" if least is None else f"at least {least}"
            raise ValueError(f"{what}: expected [{some}, {columns}], got {tuple(shape)}")
        n = shape[0]
        if n == 0:
            return dt, None, 0, columns
        stride, inner = x.stride()
        if inner != 1 and columns > 1:
            raise ValueError(f"{what}: the values of a row must be adjacent")
        if n == 1:
            stride = columns
        elif stride < columns:
            raise ValueError(f"{what}: rows overlap")
        return dt, x.data_ptr(), n, stride

    def _indices(self, x, shape, what):
        """(bytes of an index, address, row stride) of int32 or int64 indices."""
        size = x.dtype.itemsize
        if x.dtype not in self._index_types or tuple(x.shape) != shape:
            raise ValueError(f"{what}: expected {shape} int32 or int64 values, got {tuple(x.shape)} of {x.dtype}")
        self._here(x, what)
        columns = shape[1] if len(shape) == 2 else 1
        if shape[0] == 0:
            return size, None, columns
        stride = x.stride()
        if len(shape) == 1:
            if stride[0] != 1 and shape[0] > 1:
                raise ValueError(f"{what}: expected a contiguous tensor")
            return size, x.data_ptr(), 1
        if stride[1] != 1 and columns > 1:
            raise ValueError(f"{what}: the values of a row must be adjacent")
        if shape[0] > 1 and stride[0] < columns:
            raise ValueError(f"{what}: rows overlap")
        return size, x.data_ptr(), columns if shape[0] == 1 else stride[0]

    def _mask(self, mask, tokens):
        if mask is None:
            return None
        if mask.dtype not in (self.torch.bool, self.torch.uint8) or mask.shape != (tokens,):
            raise ValueError(f"mask: expected {tokens} bool or uint8 values")
        self._here(mask, "mask")
        if not mask.is_contiguous():
            raise ValueError("mask: expected a contiguous tensor")
        return mask.data_ptr() if tokens else None

    def _scaler(self, scaler):
        if scaler is None:
            return None
        if not isinstance(scaler, int):
            self._here(scaler, "scaler")
        return _lib._scaler(scaler)

    def _stream(self):
        return _lib._stream_on(self.stream, self._device)

    def _keep(self, *tensors):
        """On a stream of its own: torch does not hand the tensors' memory out again before that stream has used it."""
        from .checkpoint import torch_stream
        there = torch_stream(self.stream, self.torch)
        for x in tensors:
            if x is not None and not isinstance(x, int):
                x.record_stream(there)


def token_count(tokens, most, what="max_tokens"):
    tokens = int(tokens)
    if not 0 <= tokens <= most:
        raise ValueError(f"{what} = {tokens}: 0 to {most} are supported")
    return tokens
