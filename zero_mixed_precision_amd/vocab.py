"""VocabCrossEntropy: softmax cross entropy over a large vocabulary, from hidden states and the head's weight.

The logits are never kept: the loss goes over the vocabulary once, the gradient
piece by piece.  The gradient carries the device's loss scale ([Guide] section
4.2, dynamic loss scaling), so it joins a loss-scaled backward pass without a
host synchronisation.

    ce = VocabCrossEntropy(vocab=32000, width=4096, max_tokens=4096, dtype=torch.bfloat16)
    loss = ce.loss_and_gradient(hidden, head, targets, dhidden, dhead, scaler=step.state)
    hidden.backward(dhidden)
"""
from __future__ import annotations

from . import _lib
from ._lib import on_its_device
from .operands import TokenOperator, token_count


class VocabCrossEntropy(TokenOperator):
    """``loss()`` and ``loss_and_gradient()`` leave, on the device: ``value`` (fp32 scalar: coef times the mean over used
    rows), ``token_loss`` (fp32 [max_tokens], of which the call's tokens are the first: 0 for rows that are not used) and
    ``used`` (int32 scalar: rows that counted).  They are overwritten by the next call; what ``token_loss`` holds behind its
    tokens is of earlier ones.

    ``dtype``: torch.float16 or torch.bfloat16, of hidden states and weight.  The workspace is allocated here, once.

    Calls of one object share its workspace and results: one after another, on one stream.

    ``stream``: a stream of its own (default: torch's current one).  The caller orders it after what writes the inputs,
    and what reads the results after it; the inputs may be freed as soon as a call returns."""

    def __init__(self, vocab: int, width: int, max_tokens: int, dtype, coef: float = 1.0, device="cuda", stream=None):
        import torch

        self.vocab, self.width, self.coef, self.dtype = int(vocab), int(width), float(coef), dtype
        if dtype not in (torch.float16, torch.bfloat16):
            raise ValueError(f"dtype {dtype} is not float16 or bfloat16")
        if not 1 <= self.vocab <= 2 ** 24 or not 1 <= self.width <= 65536:
            raise ValueError(f"{self.vocab} x {self.width}: a vocabulary of 1 to 2^24 and a width of 1 to 65536 are supported")
        self.max_tokens = token_count(max_tokens, 2 ** 24)
        super().__init__(device, stream)
        with self._own():
            self.token_loss = torch.zeros(self.max_tokens, dtype=torch.float32, device=self.device)
            self.value = torch.zeros((), dtype=torch.float32, device=self.device)
            self.used = torch.zeros((), dtype=torch.int32, device=self.device)
            self._ws_bytes = _lib.ds_vocab_ce_workspace_bytes(self.max_tokens, self.vocab, self.width)
            self._ws = torch.empty(self._ws_bytes, dtype=torch.uint8, device=self.device)
        self._scratch = (self._ws.data_ptr(), self._ws_bytes)
        self._at = (self.token_loss.data_ptr(), self.value.data_ptr(), self.used.data_ptr())

    def _matrix(self, x, what, rows=None):
        dt, at, n, stride = self._rows(x, self.width, what, rows=rows)
        if x.dtype != self.dtype:
            raise ValueError(f"{what}: expected {self.dtype}, got {x.dtype}")
        return dt, at, n, stride

    def _call(self, hidden, weight, targets, dhidden, dweight, mask, scaler, accumulate):
        dt, h, T, hstride = self._matrix(hidden, "hidden")
        if T > self.max_tokens:
            raise ValueError(f"hidden: {T} tokens, at most {self.max_tokens} were asked for")
        _, w, _, wstride = self._matrix(weight, "weight", rows=self.vocab)
        size, y, _ = self._indices(targets, (T,), "targets")
        dh, dhstride, dw, dwstride, dwt = None, 0, None, 0, dt
        if dhidden is not None:
            _, dh, _, dhstride = self._matrix(dhidden, "dhidden", rows=T)
        if dweight is not None:
            dwt, dw, _, dwstride = self._rows(dweight, self.width, "dweight", rows=self.vocab)
            if dwt not in (dt, _lib.DS_FP32):
                raise ValueError(f"dweight: expected {self.dtype} or float32, got {dweight.dtype}")
        rc = _lib.lib.ds_vocab_ce(self._scaler(scaler), h, hstride, w, wstride, dt, y, size, T, self.vocab, self.width,
                                  self._mask(mask, T), self.coef, *self._at, dh, dhstride, dw, dwt, dwstride,
                                  bool(accumulate), *self._scratch, self._stream())
        if rc:
            _lib._ok(rc, "ds_vocab_ce")
        if self.stream is not None:
            self._keep(hidden, weight, targets, dhidden, dweight, mask, scaler)
        return self.value

    @on_its_device
    def loss(self, hidden, weight, targets, mask=None):
        """``hidden``: [tokens, width], ``weight``: [vocab, width], rows any distance apart; ``targets``: int32 or int64
        [tokens], a negative one leaves its row out; ``mask``: bool or uint8 per token, 0 leaves it out.  Returns
        ``value``."""
        return self._call(hidden, weight, targets, None, None, mask, None, False)

    @on_its_device
    def loss_and_gradient(self, hidden, weight, targets, dhidden, dweight, mask=None, scaler=None, accumulate=False):
        """loss(), and its gradients by ``hidden`` into ``dhidden`` (same type) and by ``weight`` into ``dweight`` (same
        type or float32), times the scale of ``scaler`` (a ds_scaler state on the device; None: 1).  Either may be None,
        for a gradient that nobody needs.  accumulate: add to ``dweight``."""
        if dhidden is None and dweight is None:
            raise ValueError("neither dhidden nor dweight is given: loss() takes no gradient")
        if accumulate and dweight is None:
            raise ValueError("accumulate adds to dweight, which is None")
        return self._call(hidden, weight, targets, dhidden, dweight, mask, scaler, accumulate)
