"""ExpertBalance: a mixture-of-experts router's balance loss, counts and gradient.

The auxiliary loss that a training step with experts ("DeepSpeed complete
guide" section 9) adds itself: coef * E * sum_e f_e P_e, with f_e the share of
the (token, choice) pairs that go to expert e and P_e the mean router
probability.  Its gradient carries the device's loss scale, so it joins a
loss-scaled backward pass without a host synchronisation.

    balance = ExpertBalance(num_experts=64, k=8, coef=0.01)
    loss = balance.loss(logits, mask=mask)           # logits: [tokens, experts]
    balance.gradient(logits, dlogits, mask=mask, scaler=step.state)
    logits.backward(dlogits)
"""
from __future__ import annotations

from . import _lib
from .multi_tensor import _dtype_of, check_stream


class ExpertBalance:
    """``loss()`` leaves, on the device: ``value`` (fp32 scalar), ``counts`` (int32 per expert), ``mean_prob`` (fp32 per
    expert) and ``used`` (int32 scalar: rows that counted).  They are overwritten by the next call.

    ``stream``: a stream of its own (default: torch's current one).  The caller orders it after what writes the inputs,
    and what reads the results after it; the inputs may be freed as soon as a call returns."""

    def __init__(self, num_experts: int, k: int, coef: float, device="cuda", stream=None):
        import torch

        self.torch, self.E, self.k, self.coef, self.stream = torch, int(num_experts), int(k), float(coef), stream
        if not 1 <= self.E <= _lib.DS_MAX_EXPERTS or not 1 <= self.k <= min(self.E, _lib.DS_MAX_EXPERT_CHOICES):
            raise ValueError(f"k = {self.k} of {self.E} experts: at most {_lib.DS_MAX_EXPERT_CHOICES} of "
                             f"{_lib.DS_MAX_EXPERTS} are supported")
        from .checkpoint import torch_stream
        with torch.cuda.stream(torch_stream(stream, torch)):
            self.counts = torch.zeros(self.E, dtype=torch.int32, device=device)
            self.mean_prob = torch.zeros(self.E, dtype=torch.float32, device=device)
            self.value = torch.zeros((), dtype=torch.float32, device=device)
            self.used = torch.zeros((), dtype=torch.int32, device=device)
            # enough for any number of tokens (2.1 MB for 512 experts); its count of finished blocks starts at zero
            need = _lib.ds_balance_workspace_bytes(1 << 30, self.E)
            self._ws = torch.zeros((need + 7) // 8, dtype=torch.float64, device=device)
        check_stream(stream, self.counts.device)
        self._device, self._many = self.counts.device.index, torch.cuda.device_count() > 1
        self._mask_types = (torch.bool, torch.uint8)
        self._at = (self.counts.data_ptr(), self.mean_prob.data_ptr(), self.value.data_ptr(), self.used.data_ptr(),
                    self._ws.data_ptr(), self._ws.numel() * 8)

    def _rows(self, x, what):
        """(type, address, tokens, row stride) of a [tokens, experts] matrix.  A small call's time is the host's, half of
        it spent here and in marshalling: each property of a tensor is asked for once."""
        dt = _dtype_of(x, self.torch, what)
        shape = x.shape
        if len(shape) != 2 or shape[1] != self.E:
            raise ValueError(f"{what}: expected [tokens, {self.E}], got {tuple(shape)}")
        if not x.is_cuda or x.get_device() != self._device:
            raise ValueError(f"{what}: expected a tensor on {self.counts.device}, got one on {x.device}")
        T = shape[0]
        if T == 0:
            return dt, None, 0, self.E
        stride, inner = x.stride()
        if inner != 1 and self.E > 1:
            raise ValueError(f"{what}: the experts of a row must be adjacent")
        if T == 1:
            stride = self.E
        elif stride < self.E:
            raise ValueError(f"{what}: rows overlap")
        return dt, x.data_ptr(), T, stride

    def _mask(self, mask, tokens):
        if mask.dtype not in self._mask_types or mask.shape != (tokens,):
            raise ValueError(f"mask: expected {tokens} bool or uint8 values")
        if not mask.is_cuda or mask.get_device() != self._device or not mask.is_contiguous():
            raise ValueError(f"mask: expected a contiguous tensor on {self.counts.device}")
        return mask.data_ptr() if tokens else None

    def _keep(self, *tensors):
        """On a stream of its own: torch does not hand the tensors' memory out again before that stream has used it."""
        from .checkpoint import torch_stream
        there = torch_stream(self.stream, self.torch)
        for x in tensors:
            if x is not None and not isinstance(x, int):
                x.record_stream(there)

    def loss(self, logits, mask=None):
        """Counts and loss of ``logits`` (fp16, bf16 or fp32 [tokens, experts], rows any distance apart); ``mask``:
        bool or uint8 per token, 0 leaves it out.  Returns ``value``."""
        if self._many and self.torch.cuda.current_device() != self._device:     # launches go to the current GPU
            with self.torch.cuda.device(self._device):
                return self.loss(logits, mask)
        dt, z, T, stride = self._rows(logits, "logits")
        counts, mean, value, used, ws, ws_bytes = self._at
        rc = _lib.lib.ds_balance_loss(z, dt, T, self.E, stride, None if mask is None else self._mask(mask, T), self.k,
                                      self.coef, counts, mean, value, used, ws, ws_bytes,
                                      _lib._stream_on(self.stream, self._device))
        if rc:
            _lib._ok(rc, "ds_balance_loss")
        if self.stream is not None:
            self._keep(logits, mask)
        return self.value

    def gradient(self, logits, out, mask=None, scaler=None, accumulate=False):
        """The gradient by ``logits`` of the loss() just taken of them, into ``out`` (their type and shape), times the
        scale of ``scaler`` (a ds_scaler state on the device; None: 1).  accumulate: add to ``out``."""
        if self._many:
            if self.torch.cuda.current_device() != self._device:
                with self.torch.cuda.device(self._device):
                    return self.gradient(logits, out, mask, scaler, accumulate)
            if scaler is not None and not isinstance(scaler, int) and scaler.device != self.counts.device:
                raise ValueError(f"scaler: expected a state on {self.counts.device}, got one on {scaler.device}")
        dt, z, T, stride = self._rows(logits, "logits")
        of, d, rows, gstride = self._rows(out, "out")
        if of != dt or rows != T:
            raise ValueError("out: expected the logits' type and shape")
        rc = _lib.lib.ds_balance_loss_grad(None if scaler is None else _lib._scaler(scaler), z, dt, T, self.E, stride,
                                           None if mask is None else self._mask(mask, T), self.k, self.coef,
                                           self._at[0], self._at[3], d, gstride, accumulate,
                                           _lib._stream_on(self.stream, self._device))
        if rc:
            _lib._ok(rc, "ds_balance_loss_grad")
        if self.stream is not None:
            self._keep(logits, out, mask, scaler)
        return out
