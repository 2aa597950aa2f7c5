"""TopLogitDistillation: the loss of a student against a teacher's top logits, with its loss-scaled gradient.

The teacher's k largest logits of each token, with their places, are what a
program keeps of it; the student's logits are whole.  The gradient carries the
device's loss scale ([Guide] section 4.2, dynamic loss scaling), so it joins a
loss-scaled backward pass without a host synchronisation.

    distill = TopLogitDistillation(vocab=32000, k=64, max_tokens=4096, temperature=2.0)
    loss = distill.loss_and_gradient(logits, teacher, index, dlogits, scaler=step.state)
    logits.backward(dlogits)
"""
from __future__ import annotations

from . import _lib
from ._lib import on_its_device
from .operands import TokenOperator, token_count


class TopLogitDistillation(TokenOperator):
    """``loss()`` and ``loss_and_gradient()`` leave, on the device: ``value`` (fp32 scalar: coef times the mean over used
    rows), ``token_loss`` (fp32 [max_tokens], of which the call's tokens are the first: 0 for rows that are not used) and
    ``used`` (int32 scalar: rows that counted).  They are overwritten by the next call; what ``token_loss`` holds behind its
    tokens is of earlier ones.

    ``k``: teacher's entries per row (1..1024; rows may have fewer: a negative place is an absent entry).

    Calls of one object share its workspace and results: one after another, on one stream.

    ``stream``: a stream of its own (default: torch's current one).  The caller orders it after what writes the inputs,
    and what reads the results after it; the inputs may be freed as soon as a call returns."""

    def __init__(self, vocab: int, k: int, max_tokens: int, temperature: float = 1.0, coef: float = 1.0, device="cuda",
                 stream=None):
        self.vocab, self.k, self.temperature, self.coef = int(vocab), int(k), float(temperature), float(coef)
        if not 1 <= self.vocab <= 2 ** 30:
            raise ValueError(f"vocab = {self.vocab}: 1 to 2^30 are supported")
        if not 1 <= self.k <= _lib.DS_MAX_TEACHER_LOGITS:
            raise ValueError(f"k = {self.k}: 1 to {_lib.DS_MAX_TEACHER_LOGITS} are supported")
        if not 2.0 ** -10 <= self.temperature <= 2.0 ** 10:
            raise ValueError(f"temperature = {self.temperature}: 2^-10 to 2^10 are supported")
        self.max_tokens = token_count(max_tokens, 2 ** 30)
        super().__init__(device, stream)
        torch = self.torch
        with self._own():
            self.token_loss = torch.zeros(self.max_tokens, dtype=torch.float32, device=self.device)
            self.value = torch.zeros((), dtype=torch.float32, device=self.device)
            self.used = torch.zeros((), dtype=torch.int32, device=self.device)
            # its count of used rows starts at zero
            need = _lib.ds_distill_workspace_bytes(self.max_tokens)
            self._ws = torch.zeros((need + 7) // 8, dtype=torch.float64, device=self.device)
        self._scratch = (self._ws.data_ptr(), self._ws.numel() * 8)
        self._at = (self.token_loss.data_ptr(), self.value.data_ptr(), self.used.data_ptr())

    def _call(self, logits, teacher, index, out, mask, scaler, accumulate):
        dt, z, T, stride = self._rows(logits, self.vocab, "logits")
        if T > self.max_tokens:
            raise ValueError(f"logits: {T} tokens, at most {self.max_tokens} were asked for")
        tt, t, _, tstride = self._rows(teacher, self.k, "teacher", rows=T)
        size, i, istride = self._indices(index, (T, self.k), "index")
        d, gstride = None, 0
        if out is not None:
            of, d, _, gstride = self._rows(out, self.vocab, "out", rows=T)
            if of != dt:
                raise ValueError(f"out: expected {logits.dtype}, got {out.dtype}")
        rc = _lib.lib.ds_distill_loss(self._scaler(scaler), z, dt, T, self.vocab, stride, t, tt, tstride, i, size, istride,
                                      self.k, self._mask(mask, T), self.temperature, self.coef, *self._at, d, gstride,
                                      bool(accumulate) and T > 0, *self._scratch, self._stream())
        if rc:
            _lib._ok(rc, "ds_distill_loss")
        if self.stream is not None:
            self._keep(logits, teacher, index, out, mask, scaler)
        return self.value

    @on_its_device
    def loss(self, logits, teacher, index, mask=None):
        """``logits``: fp16, bf16 or fp32 [tokens, vocab]; ``teacher``: [tokens, k] of the teacher's logits (any of these
        types), ``index``: int32 or int64 [tokens, k], their places; rows any distance apart.  ``mask``: bool or uint8 per
        token, 0 leaves it out.  Returns ``value``."""
        return self._call(logits, teacher, index, None, mask, None, False)

    @on_its_device
    def loss_and_gradient(self, logits, teacher, index, out, mask=None, scaler=None, accumulate=False):
        """loss(), and its gradient by ``logits`` into ``out`` (their type and shape; may be ``logits`` itself), times the
        scale of ``scaler`` (a ds_scaler state on the device; None: 1).  accumulate: add to ``out``."""
        return self._call(logits, teacher, index, out, mask, scaler, accumulate)
