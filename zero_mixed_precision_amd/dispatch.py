"""ExpertDispatch: tokens sorted by expert, moved to the experts and back, and the gradients of both moves.

Beside ExpertBalance in a mixture-of-experts layer ("DeepSpeed complete guide"
section 9): the router's choices become rows in expert order, on which each
expert's products are a contiguous block, and the experts' outputs become the
tokens' weighted sums.

    dispatch = ExpertDispatch(num_experts=64, k=8, max_tokens=4096)
    dispatch.sort(chosen)                                  # [tokens, k]; -1 drops a choice
    dispatch.gather(x, rows)                               # rows[place] = x; expert e: rows offsets[e] .. offsets[e + 1]
    dispatch.combine(outputs, gates, y)                    # y[t] = sum_j gates[t, j] outputs[place[t, j]]
    dispatch.combine_gradient(dy, outputs, gates, doutputs, dgates)
    dispatch.gather_gradient(drows, dx)
"""
from __future__ import annotations

from . import _lib
from ._lib import on_its_device
from .operands import TokenOperator, token_count


class ExpertDispatch(TokenOperator):
    """``sort()`` leaves, on the device: ``offsets`` (int32 [experts + 1]: the rows of expert e start at offsets[e]),
    ``place`` (int32 [max_tokens, k]: the row of each choice, -1 for a dropped one) and ``source`` (int32
    [max_tokens * k]: the choice t * k + j of each row, -1 behind the last one).  The sorted tokens are the first of
    ``place``, their tokens * k choices the first of ``source``; what lies behind is of earlier calls.  They are
    overwritten by the next sort(), and the moves go by them: a layer whose gradient is still to come keeps its own object.
    ``sorts`` counts the calls of sort(); a backward pass hands the count of its forward to ``check_sort()``, which raises
    if another sort() came between.

    Calls of one object go by the same arrays: one after another, on one stream.

    ``stream``: a stream of its own (default: torch's current one).  The caller orders it after what writes the inputs,
    and what reads the results after it; the inputs may be freed as soon as a call returns."""

    sorts = 0

    def __init__(self, num_experts: int, k: int, max_tokens: int, device="cuda", stream=None):
        self.E, self.k = int(num_experts), int(k)
        if not 1 <= self.E <= _lib.DS_MAX_EXPERTS or not 1 <= self.k <= _lib.DS_MAX_EXPERT_CHOICES:
            raise ValueError(f"k = {self.k} of {self.E} experts: at most {_lib.DS_MAX_EXPERT_CHOICES} of "
                             f"{_lib.DS_MAX_EXPERTS} are supported")
        self.max_tokens = token_count(max_tokens, (2 ** 31 - 1) // self.k)
        super().__init__(device, stream)
        torch = self.torch
        with self._own():
            self.offsets = torch.zeros(self.E + 1, dtype=torch.int32, device=self.device)
            self.place = torch.full((self.max_tokens, self.k), -1, dtype=torch.int32, device=self.device)
            self.source = torch.full((self.max_tokens * self.k,), -1, dtype=torch.int32, device=self.device)
            need = _lib.ds_dispatch_workspace_bytes(self.max_tokens, self.E, self.k)
            self._ws = torch.empty((need + 3) // 4, dtype=torch.int32, device=self.device)
        self.tokens = 0                     # of the last sort()
        self._place = self.place.data_ptr()
        self._at = (self.offsets.data_ptr(), self._place, self.source.data_ptr(), self._ws.data_ptr(), self._ws.numel() * 4)

    def _sorted(self, tokens, what):
        if tokens != self.tokens:
            raise ValueError(f"{what}: {tokens} tokens, but sort() had {self.tokens}")

    @on_its_device
    def sort(self, chosen):
        """``chosen``: int32 or int64 [tokens, k], rows any distance apart; a number outside 0..experts-1 drops its
        choice.  Stable: an expert's rows keep the order of their tokens."""
        T = chosen.shape[0] if len(chosen.shape) else -1
        size, at, stride = self._indices(chosen, (T, self.k), "chosen")
        if T > self.max_tokens:
            raise ValueError(f"chosen: {T} tokens, at most {self.max_tokens} were asked for")
        rc = _lib.lib.ds_dispatch_sort(at, size, T, self.E, self.k, stride, *self._at, self._stream())
        if rc:
            _lib._ok(rc, "ds_dispatch_sort")
        self.tokens = T
        self.sorts += 1
        if self.stream is not None:
            self._keep(chosen)
        return self.offsets

    def check_sort(self, sorts):
        """Raises if the last sort() is not the one after which ``sorts`` was read."""
        if sorts != self.sorts:
            raise RuntimeError(f"sorted {self.sorts - sorts} more times since then: the order of these rows is gone (one "
                               "ExpertDispatch for each layer and pass whose gradient is still to come)")

    def _pair(self, tokens_side, sorted_side, names):
        """Both sides of a move: (type, width, address and stride of the tokens' side, address, stride and rows of the
        sorted one)."""
        if len(tokens_side.shape) != 2:
            raise ValueError(f"{names[0]}: expected [tokens, width], got {tuple(tokens_side.shape)}")
        width = tokens_side.shape[1]
        dt, a, T, astride = self._rows(tokens_side, width, names[0])
        self._sorted(T, names[0])
        bt, b, n, bstride = self._rows(sorted_side, width, names[1], least=T * self.k)
        if bt != dt:
            raise ValueError(f"{names[1]}: expected {tokens_side.dtype}, got {sorted_side.dtype}")
        return dt, width, a, astride, b, bstride, n

    @on_its_device
    def gather(self, x, out):
        """out[place[t, j]] = x[t].  ``x``: [tokens, width] in fp16, bf16 or fp32; ``out``: its type, at least tokens * k
        rows; rows behind the last one are left as they are."""
        dt, width, a, astride, b, bstride, n = self._pair(x, out, ("x", "out"))
        rc = _lib.lib.ds_dispatch_gather(a, dt, self.tokens, self.k, width, astride, self._place, b, bstride, n,
                                         self._stream())
        if rc:
            _lib._ok(rc, "ds_dispatch_gather")
        if self.stream is not None:
            self._keep(x, out)
        return out

    @on_its_device
    def gather_gradient(self, dout, dx):
        """dx[t] = sum_j dout[place[t, j]], the gradient of gather() by ``x``."""
        dt, width, a, astride, b, bstride, n = self._pair(dx, dout, ("dx", "dout"))
        rc = _lib.lib.ds_dispatch_gather_grad(b, dt, self.tokens, self.k, width, bstride, n, self._place, a,
                                              astride, self._stream())
        if rc:
            _lib._ok(rc, "ds_dispatch_gather_grad")
        if self.stream is not None:
            self._keep(dout, dx)
        return dx

    @on_its_device
    def combine(self, rows, gates, out):
        """out[t] = sum_j gates[t, j] rows[place[t, j]], summed in fp32 and rounded once (0 for a token without a row).
        ``rows``: at least tokens * k rows; ``gates``: [tokens, k] in fp16, bf16 or fp32, not read for dropped choices."""
        dt, width, a, astride, b, bstride, n = self._pair(out, rows, ("out", "rows"))
        gt, g, _, gstride = self._rows(gates, self.k, "gates", rows=self.tokens)
        rc = _lib.lib.ds_dispatch_combine(b, dt, self.tokens, self.k, width, bstride, n, self._place, g, gt,
                                          gstride, a, astride, self._stream())
        if rc:
            _lib._ok(rc, "ds_dispatch_combine")
        if self.stream is not None:
            self._keep(rows, gates, out)
        return out

    @on_its_device
    def combine_gradient(self, dout, rows, gates, drows, dgates):
        """The gradients of combine(): drows[place[t, j]] = gates[t, j] dout[t] (rows behind the last one are left as they
        are), dgates[t, j] = <dout[t], rows[place[t, j]]> (0 for a dropped choice)."""
        dt, width, a, astride, b, bstride, n = self._pair(dout, rows, ("dout", "rows"))
        dr, d, dn, dstride = self._rows(drows, width, "drows", least=self.tokens * self.k)
        gt, g, _, gstride = self._rows(gates, self.k, "gates", rows=self.tokens)
        dg, e, _, estride = self._rows(dgates, self.k, "dgates", rows=self.tokens)
        if dr != dt:
            raise ValueError(f"drows: expected {dout.dtype}, got {drows.dtype}")
        if dg != gt:
            raise ValueError(f"dgates: expected {gates.dtype}, got {dgates.dtype}")
        rc = _lib.lib.ds_dispatch_combine_grad(a, dt, self.tokens, self.k, width, astride, b, bstride, min(n, dn),
                                               self._place, g, gt, gstride, d, dstride, e, estride,
                                               self._stream())
        if rc:
            _lib._ok(rc, "ds_dispatch_combine_grad")
        if self.stream is not None:
            self._keep(dout, rows, gates, drows, dgates)
        return drows, dgates
