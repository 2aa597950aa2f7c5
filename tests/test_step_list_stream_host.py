"""The step over a list on a stream of its own, without a GPU: what torch's current stream reads of it, and writes for it,
is ordered with the steps."""
import ctypes
from types import SimpleNamespace

import pytest
import torch

from zero_mixed_precision_amd import MultiTensorStep, ZeroMPConfig, _lib


class Stream:
    device = None

    def __init__(self, name, log):
        self.name, self.log = name, log

    def wait_stream(self, other):
        self.log.append(f"{self.name} waits for {other.name}")

    def __enter__(self):
        self.log.append(f"on {self.name}")

    def __exit__(self, *_):
        self.log.append("back")


class Array(torch.Tensor):
    """A host tensor whose copies and reads are logged."""
    log: list = []

    @classmethod
    def __torch_function__(cls, func, types, args=(), kwargs=None):
        if func.__name__ in ("clone", "copy_", "float"):
            Array.log.append(func.__name__)
        return super().__torch_function__(func, types, args, kwargs or {})


def make(states, capturing=False, own=True):
    log = Array.log = []
    here, there = Stream("here", log), Stream("there", log)
    fake = SimpleNamespace(float32=torch.float32, no_grad=torch.no_grad, uint8=torch.uint8, frombuffer=torch.frombuffer,
                           cuda=SimpleNamespace(current_stream=lambda *_: here, stream=lambda s: s,
                                                is_current_stream_capturing=lambda: capturing))
    op = MultiTensorStep.__new__(MultiTensorStep)
    op.torch, op.cfg, op.stream, op._device, op._many = fake, ZeroMPConfig(bf16=True), there if own else None, 0, False
    op.states, op.numels, op.offsets = states, [300], [0]
    array = lambda n, t: torch.zeros(n, dtype=t).as_subclass(Array)  # noqa: E731
    op.params = [array(300, torch.bfloat16)]
    op.master, op.m_scale, op.v_scale = array(512, torch.float32), None, None
    op.m, op.v = array(512, torch.float32), array(512, torch.float32)
    if states == "fp8":
        op.m, op.v = array(512, torch.uint8).view(torch.float8_e4m3fn), array(512, torch.uint8).view(torch.float8_e5m2)
        op.m_scale, op.v_scale = array(2, torch.float32), array(2, torch.float32)
    op.state = array(128, torch.uint8)
    return op, log


@pytest.mark.parametrize("states", ["fp32", "fp8"])
def test_moments_are_read_between_steps(states):
    op, log = make(states)
    op.moments(0)
    assert log[0] == "here waits for there" and log[-1] == "there waits for here" and len(log) == 4


def test_the_loss_scale_is_read_after_the_steps():
    op, log = make("fp32")
    op.loss_scale
    assert log == ["here waits for there"]


@pytest.mark.parametrize("states", ["fp32", "fp8"])
def test_a_state_is_loaded_between_what_torch_does_with_the_parameters(states, monkeypatch):
    op, log = make(states)
    sc = _lib.DsScaler(scale=1.0, min_scale=1.0, growth_window=10, hysteresis=1, hysteresis_left=1)
    raw = ctypes.string_at(ctypes.addressof(sc), ctypes.sizeof(sc))
    saved = {"numels": [300], "states": states, "scaler": torch.frombuffer(bytearray(raw), dtype=torch.uint8),
             **{k: a.as_subclass(torch.Tensor).clone() for k, a in op._arrays().items()}}
    log.clear()
    monkeypatch.setattr(_lib, "ds_state_write", lambda *a: log.append("scaler"))
    op.load_state_dict(saved)
    copies = ["copy_"] * (len(op._arrays()) + 1)
    assert [x for x in log if x not in ("on there", "back")] == ["there waits for here", *copies, "scaler",
                                                                 "here waits for there"]


@pytest.mark.parametrize("own,capturing", [(False, False), (True, True)])
def test_nothing_waits_on_one_stream_or_inside_a_capture(own, capturing):
    """Inside a capture the caller orders the streams: a wait for one that is not captured would end it."""
    op, log = make("fp32", capturing, own)
    op.moments(0)
    op.loss_scale
    assert not any("waits" in x for x in log)
