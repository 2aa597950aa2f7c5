"""MultiTensorStep: the optimizer step over a list of tensors.

For parameters that are not one flat partition: mixture-of-experts parameter
groups ("DeepSpeed complete guide" section 9), norms and biases without decay,
fp32 parameters beside 16-bit ones.  One kernel updates all of them with the
arithmetic of the flat step, gated by the same loss scaler.  The Adam states
are held in 32 bits, or in 8 (m in e4m3, v in e5m2, each with an fp32 scale
per 256 elements: 2.03 bytes per element for both states instead of 8).

    step = MultiTensorStep(params, cfg, states="fp8", dither_seed=1)
    step.set_gradients([p.grad for p in params])     # again when a gradient's address changes
    step.step()                                      # check, norm (if clipped), Adam, scaler

A step is one to four kernels (a short list is checked by the kernel that
updates it) and no host synchronisation; it can be captured into a graph.
"""
from __future__ import annotations

import ctypes

from . import _lib
from .config import ZeroMPConfig

ALIGN = _lib.DS_STATE_BLOCK     # elements: where each tensor starts in the flat state arrays


_CODES: dict = {}


def _dtype_of(t, torch, what):
    if not _CODES:
        _CODES.update({torch.float16: _lib.DS_FP16, torch.bfloat16: _lib.DS_BF16, torch.float32: _lib.DS_FP32})
    code = _CODES.get(t.dtype)
    if code is None:
        raise ValueError(f"{what}: dtype {t.dtype} is not float16, bfloat16 or float32")
    return code


def per_tensor(value, default, count, what):
    """A list of ``count`` floats from None (the default), one number, or a sequence of them."""
    if value is None:
        value = default
    if isinstance(value, (int, float)):
        return [float(value)] * count
    value = [float(x) for x in value]
    if len(value) != count:
        raise ValueError(f"{what}: {len(value)} values for {count} tensors")
    return value


def check_stream(stream, device):
    """Refuses a torch stream of another GPU than ``device`` (a raw handle does not say which it belongs to)."""
    there = getattr(stream, "device", None)
    if there is not None and there != device:
        raise ValueError(f"stream: expected one of {device}, got one of {there}")


def check_apart(state, x, what):
    """Refuses a tensor that shares memory with the scaler's state (steps would overwrite the one with the other)."""
    a, b = state.data_ptr(), x.data_ptr()
    if b < a + ctypes.sizeof(_lib.DsScaler) and a < b + x.numel() * x.element_size():
        raise ValueError(f"{what} shares memory with the scaler's state")


class MultiTensorStep:
    """``params``: fp16 or bf16 tensors (the step keeps an fp32 master of each and writes the parameter), or fp32 ones
    (their own master); contiguous, on one GPU, any alignment of their type.

    ``master``, ``m``, ``v`` are flat arrays in which tensor i starts at ``offsets[i]``, a multiple of 256 elements;
    values between tensors are zero and unused.  ``master`` is None if every parameter is fp32.  With states="fp8",
    ``m`` is float8_e4m3fn and ``v`` float8_e5m2, and ``m_scale``, ``v_scale`` hold one scale per 256 elements.
    ``dither_seed`` (8-bit states): None rounds to nearest, a number rounds with the dither of that seed.
    ``cfg``: rate, betas, eps, clipping and accumulation are read at each step; the schedule, the scaler's settings and
    the default decay once, here.
    ``weight_decay`` and ``lr_scale``: one number, or one per tensor (default: the configuration's decay, and 1).
    ``state``: share another step's scaler.  Then check() is called on every step that shares it before update() on
    the first, and only the last has ``end_step``; step() without a check() is for a list that is alone."""

    def __init__(self, params, cfg: ZeroMPConfig, states="fp32", weight_decay=None, lr_scale=None, dither_seed=None,
                 stream=None, state=None, end_step=True):
        import torch

        self.torch, self.cfg, self.stream = torch, cfg, stream
        self.params = list(params)
        count = len(self.params)
        if states not in ("fp32", "fp8"):
            raise ValueError(f"states {states!r} is neither 'fp32' nor 'fp8'")
        if dither_seed is not None and states != "fp8":
            raise ValueError("dither_seed is for states='fp8'")
        self.states, self.end_step = states, bool(end_step)
        self._sdt = _lib.DS_FP8 if states == "fp8" else _lib.DS_FP32
        self._rounding = _lib.DS_ROUND_NEAREST if dither_seed is None else _lib.DS_ROUND_DITHER
        self._seed = 0 if dither_seed is None else int(dither_seed) & (2 ** 64 - 1)
        decay = per_tensor(weight_decay, cfg.weight_decay, count, "weight_decay")
        rates = per_tensor(lr_scale, 1.0, count, "lr_scale")
        wrong = torch.float16 if cfg.bf16 else torch.bfloat16
        for i, p in enumerate(self.params):
            _dtype_of(p, torch, f"parameter {i}")
            if not p.is_contiguous():
                raise ValueError(f"parameter {i}: expected a contiguous tensor")
            if p.dtype == wrong:
                raise ValueError(f"parameter {i}: {p.dtype} in a {'bf16' if cfg.bf16 else 'fp16'} configuration")
            if not p.is_cuda or p.device != self.params[0].device:
                raise ValueError(f"parameter {i}: expected a tensor in the memory of one GPU, got one on {p.device}")
        device = self.params[0].device if count else torch.device("cuda", torch.cuda.current_device())

        check_stream(stream, device)
        # what is called once per step looks at these itself, the rest through on_its_device
        self._device, self._many = device.index, torch.cuda.device_count() > 1
        self.numels = [p.numel() for p in self.params]
        self.offsets, total = [], 0
        for n in self.numels:
            self.offsets.append(total)
            total += (n + ALIGN - 1) // ALIGN * ALIGN
        with torch.cuda.device(device):
            here, there = torch.cuda.current_stream(), self._torch_stream()
        self._shares = state is not None        # a state of its own lies apart from all that the caller has
        if self._shares:
            for i, p in enumerate(self.params):
                check_apart(state, p, f"parameter {i}")
        there.wait_stream(here)                 # the parameters may still be being written
        with torch.cuda.device(device), torch.cuda.stream(there):
            f32 = dict(dtype=torch.float32, device=device)
            copies = any(p.dtype != torch.float32 for p in self.params)
            self.master = torch.zeros(total, **f32) if copies else None
            if states == "fp8":
                self.m = torch.zeros(total, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
                self.v = torch.zeros(total, dtype=torch.uint8, device=device).view(torch.float8_e5m2)
                self.m_scale, self.v_scale = torch.zeros(total // ALIGN, **f32), torch.zeros(total // ALIGN, **f32)
            else:
                self.m, self.v = torch.zeros(total, **f32), torch.zeros(total, **f32)
                self.m_scale = self.v_scale = None
            if self.master is not None:
                for i, p in enumerate(self.params):
                    if p.dtype != torch.float32:
                        self.view(self.master, i).copy_(p.detach().reshape(-1))
            if state is not None and state.device != device:
                raise ValueError(f"state: expected a scaler on {device}, got one on {state.device}")
            self.state = state
            if state is None:
                self.state = torch.zeros(_lib.ds_scaler_size(), dtype=torch.uint8, device=device)
            self._table = torch.zeros(max(_lib.ds_tensor_list_bytes(count), 16), dtype=torch.uint8, device=device)
        if stream is not None:                  # not handed out again while steps on that stream still use them
            for x in (*self.params, *(() if state is None else (state,))):
                x.record_stream(there)
        if state is None:
            with torch.cuda.device(device):
                _lib.ds_state_init(self.state, cfg.init_scale, cfg.min_loss_scale, cfg.loss_scale_window,
                                   cfg.hysteresis, int(cfg.consecutive_hysteresis), int(cfg.dynamic), self.stream)
        self.sched = cfg.lr_schedule()
        self._tensors = (_lib.DsTensor * max(count, 1))()
        for i, p in enumerate(self.params):
            t, at = self._tensors[i], self.offsets[i]
            own = p.dtype == torch.float32
            t.master = p.data_ptr() if own else self.master.data_ptr() + 4 * at
            t.p16 = None if own else p.data_ptr()
            size = 1 if states == "fp8" else 4
            t.m, t.v = self.m.data_ptr() + size * at, self.v.data_ptr() + size * at
            if states == "fp8":
                t.m_scale = self.m_scale.data_ptr() + 4 * (at // ALIGN)
                t.v_scale = self.v_scale.data_ptr() + 4 * (at // ALIGN)
            t.n, t.weight_decay, t.lr_scale = self.numels[i], decay[i], rates[i]
            t.pdt = _dtype_of(p, torch, f"parameter {i}")
        self._grads, self._list, self._list_at = None, None, None
        # what every step passes: this object's own arrays, sized and placed here
        self._state_at = _lib._scaler(self.state)
        self.ws, self._ws_at, self._ws_bytes = None, None, 0
        if cfg.gradient_clipping > 0:
            self._make_workspace()
        self._sched_at = None if self.sched is None else ctypes.byref(self.sched)

    def _torch_stream(self):
        from .checkpoint import torch_stream
        return torch_stream(self.stream, self.torch)

    @_lib.on_its_device
    def _make_workspace(self):
        """Room for the partial sums of squares of the list that set_gradients() writes; no initial contents."""
        torch = self.torch
        shape = _lib.DsTensorList(table=self._table.data_ptr(), tiles=sum((n + 4095) // 4096 for n in self.numels),
                                  elems=sum(self.numels), count=len(self.numels), sdt=self._sdt)
        need = _lib.ds_tensor_list_workspace_bytes(shape)
        with torch.cuda.stream(self._torch_stream()):
            self.ws = torch.empty(max(need // 8, 1), dtype=torch.float64, device=self._table.device)
        self._ws_at, self._ws_bytes = self.ws.data_ptr(), self.ws.numel() * 8

    def _after_steps(self):
        """Torch's current stream goes on after the steps enqueued so far.  (Inside a capture the caller orders a stream
        of the step's own: a wait for one that is not captured would end it.)"""
        if self.stream is not None and not self.torch.cuda.is_current_stream_capturing():
            self.torch.cuda.current_stream().wait_stream(self._torch_stream())

    def _before_steps(self):
        """The steps to come go on after what torch's current stream has been given so far."""
        if self.stream is not None and not self.torch.cuda.is_current_stream_capturing():
            self._torch_stream().wait_stream(self.torch.cuda.current_stream())

    def view(self, flat, i: int):
        """Tensor i as a view of one of the flat arrays."""
        return flat[self.offsets[i]:self.offsets[i] + self.numels[i]]

    @_lib.on_its_device
    def set_gradients(self, grads) -> None:
        """The gradient tensors of the following steps, one per parameter (16-bit in the configuration's format, or
        fp32).  They are read where they lie, so they stay allocated; call it again when one has moved.  On a stream of
        its own the step is ordered after what writes them by the caller."""
        torch = self.torch
        grads = list(grads)
        if len(grads) != len(self.params):
            raise ValueError(f"{len(grads)} gradients for {len(self.params)} parameters")
        wrong = torch.float16 if self.cfg.bf16 else torch.bfloat16
        for i, (g, p) in enumerate(zip(grads, self.params)):
            if g is None or g.numel() != p.numel() or not g.is_contiguous() or g.device != p.device:
                raise ValueError(f"gradient {i}: expected a contiguous tensor of {p.numel()} elements on {p.device}")
            if g.dtype == wrong:
                raise ValueError(f"gradient {i}: {g.dtype} in a {'bf16' if self.cfg.bf16 else 'fp16'} configuration")
            self._tensors[i].gdt = _dtype_of(g, torch, f"gradient {i}")
            self._tensors[i].grad = g.data_ptr() or None
        if self._shares:
            for i, g in enumerate(grads):
                check_apart(self.state, g, f"gradient {i}")
        self._list = None
        tensors = self._tensors if grads else []
        self._list = _lib.ds_tensor_list_write(self._table, tensors, self._sdt, self.stream)
        self._list_at = ctypes.byref(self._list)
        if self.stream is not None:              # not handed out again while steps on that stream still read them
            there = self._torch_stream()
            for g in grads:
                g.record_stream(there)
        self._grads = grads

    def step(self) -> None:
        """One step on the gradients set: overflow check (with the joint norm if clipped), gated Adam, scaler.  Where
        it does not end the step (``end_step``) it comes after check() and is update()."""
        if self._many and self.torch.cuda.current_device() != self._device:
            with self.torch.cuda.device(self._device):
                return self.step()
        if self._list is None:
            raise RuntimeError("set_gradients() before step()")
        c = self.cfg
        if not self.end_step:
            if self._list.checked != self._state_at:
                raise RuntimeError("check() on every step that shares the scaler before this one moves its tensors")
            self.update()
            return
        if c.gradient_clipping > 0 and self._list.checked == self._state_at:
            raise RuntimeError("check() has summed these gradients' squares already: update() is the other half")
        if c.gradient_clipping > 0 and self.ws is None:
            self._make_workspace()
        _lib._ok(_lib.lib.ds_step_list(self._state_at, self._list_at, self._ws_at, self._ws_bytes, c.lr, self._sched_at,
                                       c.betas[0], c.betas[1], c.eps, c.gradient_clipping, c.gradient_accumulation_steps,
                                       self._rounding, self._seed, _lib._stream_on(self.stream, self._device)),
                 "ds_step_list")
        self._list.checked = None

    def check(self) -> None:
        """The first half of step(): the overflow check, with the sum of squares if clipped.  Where several steps share
        a scaler, every check() comes before the first update(), so that all of them see one flag and one norm."""
        if self._many and self.torch.cuda.current_device() != self._device:
            with self.torch.cuda.device(self._device):
                return self.check()
        if self._list is None:
            raise RuntimeError("set_gradients() before check()")
        if self.cfg.gradient_clipping > 0 and self.ws is None:
            self._make_workspace()
        _lib._ok(_lib.lib.ds_check_overflow_list(self._state_at, self._list_at, self._ws_at, self._ws_bytes,
                                                 _lib._stream_on(self.stream, self._device)), "ds_check_overflow_list")
        self._list.checked = self._state_at

    def update(self) -> None:
        """The second half of step(): gated Adam and, with ``end_step``, the scaler."""
        if self._many and self.torch.cuda.current_device() != self._device:
            with self.torch.cuda.device(self._device):
                return self.update()
        if self._list is None:
            raise RuntimeError("set_gradients() before update()")
        c = self.cfg
        _lib._ok(_lib.lib.ds_adam_step_list(self._state_at, self._list_at, c.lr, self._sched_at, c.betas[0], c.betas[1],
                                            c.eps, c.gradient_clipping, c.gradient_accumulation_steps, self._rounding,
                                            self._seed, self.end_step, _lib._stream_on(self.stream, self._device)),
                 "ds_adam_step_list")
        self._list.checked = None

    @property
    @_lib.on_its_device
    def loss_scale(self):
        """The loss scale S as an fp32 scalar on the device (a view of the scaler state: no host synchronisation; torch's
        current stream reads it after the steps enqueued so far)."""
        self._after_steps()
        return self.state[:4].view(self.torch.float32)[0]

    @_lib.on_its_device
    def scaler(self) -> _lib.DsScaler:
        return _lib.ds_state_read(self.state, self.stream)

    @_lib.on_its_device
    def set_applied_steps(self, t: int) -> None:
        """Resume at ``t`` applied steps (the bias corrections, a schedule and the dither go by it)."""
        sc = self.scaler()
        sc.step, sc.iter, sc.skipped = int(t), int(t), 0
        _lib.ds_state_write(self.state, sc, self.stream)

    @_lib.on_its_device
    def moments(self, i: int):
        """(m, v) of tensor i in fp32, after the steps enqueued so far."""
        m, v = self.view(self.m, i), self.view(self.v, i)
        self._after_steps()
        if self.states == "fp32":
            m, v = m.clone(), v.clone()
        else:
            n, blk = self.numels[i], self.offsets[i] // ALIGN
            scale = lambda s: s[blk:blk + (n + ALIGN - 1) // ALIGN].repeat_interleave(ALIGN)[:n]  # noqa: E731
            m, v = m.float() * scale(self.m_scale), v.float() * scale(self.v_scale)
        self._before_steps()
        return m, v

    def _arrays(self):
        out = {"m": self.m, "v": self.v}
        if self.master is not None:
            out["master"] = self.master
        if self.m_scale is not None:
            out.update(m_scale=self.m_scale, v_scale=self.v_scale)
        return out

    @_lib.on_its_device
    def state_dict(self) -> dict:
        """Host copies of the states, masters and scaler (the parameters themselves are the caller's)."""
        sc = self.scaler()                      # synchronises the step's stream
        raw = ctypes.string_at(ctypes.addressof(sc), ctypes.sizeof(sc))
        torch = self.torch
        return {"numels": list(self.numels), "states": self.states,
                "scaler": torch.frombuffer(bytearray(raw), dtype=torch.uint8).clone(),
                **{k: a.detach().cpu() for k, a in self._arrays().items()}}

    @_lib.on_its_device
    def load_state_dict(self, d: dict) -> None:
        """Restore what state_dict() returned; 16-bit parameters are rewritten from their masters."""
        from .checkpoint import validate_scaler

        torch = self.torch
        if list(d["numels"]) != self.numels or d["states"] != self.states:
            raise ValueError("the saved state is of other tensors, or of states in another format")
        arrays = self._arrays()
        for k, a in arrays.items():
            if k not in d or d[k].numel() != a.numel() or d[k].dtype != a.dtype:
                raise ValueError(f"the saved state's {k} does not fit")
        raw = d["scaler"].numpy().tobytes()
        if len(raw) != _lib.ds_scaler_size():
            raise ValueError(f"scaler state of {len(raw)} bytes")
        sc = _lib.DsScaler.from_buffer_copy(raw)
        validate_scaler(sc)
        self._before_steps()                    # parameters and states may still be being read
        with torch.no_grad(), torch.cuda.stream(self._torch_stream()):
            for k, a in arrays.items():
                a.copy_(d[k])
            for i, p in enumerate(self.params):
                if p.dtype != torch.float32:
                    p.copy_(self.view(self.master, i).view(p.shape))
        _lib.ds_state_write(self.state, sc, self.stream)
        self._after_steps()
