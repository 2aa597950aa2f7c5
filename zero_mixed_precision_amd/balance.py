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
from .multi_tensor import _dtype_of


class ExpertBalance:
    """``loss()`` leaves, on the device: ``value`` (fp32 scalar), ``counts`` (int32 per expert), ``mean_prob`` (fp32 per
    expert) and ``used`` (int32 scalar: rows that counted).  They are overwritten by the next call."""

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
            # enough for any number of tokens (2.1 MB for 512 experts)
            need = _lib.ds_balance_workspace_bytes(1 << 30, self.E)
            self._ws = torch.empty((need + 7) // 8, dtype=torch.float64, device=device)

    def _rows(self, x, what):
        if x.dim() != 2 or x.shape[1] != self.E:
            raise ValueError(f"{what}: expected [tokens, {self.E}], got {tuple(x.shape)}")
        if x.device != self.counts.device:
            raise ValueError(f"{what}: expected a tensor on {self.counts.device}, got one on {x.device}")
        if self.E > 1 and x.shape[0] > 0 and x.stride(1) != 1:
            raise ValueError(f"{what}: the experts of a row must be adjacent")
        stride = x.stride(0) if x.shape[0] > 1 else self.E
        if stride < self.E:
            raise ValueError(f"{what}: rows overlap")
        return stride

    def _mask(self, mask, tokens):
        torch = self.torch
        if mask is None:
            return None
        if mask.dtype not in (torch.bool, torch.uint8) or mask.dim() != 1 or mask.shape[0] != tokens:
            raise ValueError(f"mask: expected {tokens} bool or uint8 values")
        return mask if tokens else None

    def loss(self, logits, mask=None):
        """Counts and loss of ``logits`` (fp16, bf16 or fp32 [tokens, experts], rows any distance apart); ``mask``:
        bool or uint8 per token, 0 leaves it out.  Returns ``value``."""
        torch = self.torch
        stride, T = self._rows(logits, "logits"), logits.shape[0]
        dt = _dtype_of(logits, torch, "logits")
        mask = self._mask(mask, T)
        _lib.ds_balance_loss(logits if T else None, dt, T, self.E, stride, mask, self.k, self.coef, self.counts,
                             self.mean_prob, self.value, self.used, self._ws, stream=self.stream)
        return self.value

    def gradient(self, logits, out, mask=None, scaler=None, accumulate=False):
        """The gradient by ``logits`` of the loss() just taken of them, into ``out`` (their type and shape), times the
        scale of ``scaler`` (a ds_scaler state on the device; None: 1).  accumulate: add to ``out``."""
        torch = self.torch
        stride, gstride, T = self._rows(logits, "logits"), self._rows(out, "out"), logits.shape[0]
        if out.dtype != logits.dtype or out.shape != logits.shape:
            raise ValueError("out: expected the logits' type and shape")
        dt = _dtype_of(logits, torch, "logits")
        mask = self._mask(mask, T)
        _lib.ds_balance_loss_grad(scaler, logits if T else None, dt, T, self.E, stride, mask, self.k, self.coef,
                                  self.counts, self.used, out if T else None, gstride, accumulate, stream=self.stream)
        return out
