"""Objects whose tensors lie on a GPU that is not torch's current one, without a GPU: every launch is made with theirs
current, on its stream, and the current one is what it was afterwards."""
import ctypes
from types import SimpleNamespace

import pytest
import torch

from tests.stand_in import Library, Stream, Tensor, Torch, balance
from zero_mixed_precision_amd import MultiTensorStep, ZeroMPConfig, _lib


def tensor_step(monkeypatch, current, index, stream=None, end_step=True):
    fake = Torch(current)
    library = Library(fake)
    monkeypatch.setattr(_lib, "lib", library)
    monkeypatch.setattr(_lib, "_raw_stream", lambda i: 0x100 * i)
    monkeypatch.setattr(_lib, "_s", lambda s: 0x100 * fake.now if s is None else s.cuda_stream)
    op = MultiTensorStep.__new__(MultiTensorStep)
    op.torch, op.cfg, op.stream, op._device, op._many = fake, ZeroMPConfig(bf16=True), stream, index, True
    op.params = [Tensor(10, dtype=torch.bfloat16, index=index)]
    op._tensors, op._sdt = (_lib.DsTensor * 1)(), _lib.DS_FP32
    op._table = Tensor(1 << 14, dtype=torch.uint8, index=index)
    op.state, op.ws, op.clip = Tensor(128, dtype=torch.uint8, index=index), None, 0.0
    op._state_at, op._ws_at, op._ws_bytes, op._sched_at, op._rounding, op._seed = 1, None, 0, None, 0, 0
    op.end_step, op._shares = end_step, False
    op._list = _lib.DsTensorList()
    op._list_at, op._grads = ctypes.byref(op._list), None
    return op, fake, library


def where(library):
    """(name, current device, stream) of the calls."""
    return [(name, device, args[-1]) for name, device, args in library.calls]


@pytest.mark.parametrize("current,index", [(0, 1), (1, 0), (1, 1)])
def test_step_over_a_list(current, index, monkeypatch):
    op, fake, library = tensor_step(monkeypatch, current, index)
    op.set_gradients([Tensor(10, dtype=torch.bfloat16, index=index)])
    op.step()
    op.check()
    op.update()
    op.scaler()
    op.set_applied_steps(3)
    names = ["ds_tensor_list_write", "ds_step_list", "ds_check_overflow_list", "ds_adam_step_list", "ds_state_read",
             "ds_state_read", "ds_state_write"]
    assert where(library) == [(name, index, 0x100 * index) for name in names]
    assert fake.now == current


@pytest.mark.parametrize("current,index", [(0, 1), (1, 0), (1, 1)])
def test_balance_loss(current, index, monkeypatch):
    op, fake, library = balance(monkeypatch, current=current, index=index)
    z, out = (Tensor(100, 64, index=index) for _ in range(2))
    mask, state = Tensor(100, dtype=torch.bool, index=index), Tensor(128, dtype=torch.uint8, index=index)
    op.loss(z, mask=mask)
    assert op.gradient(z, out, mask=mask, scaler=state, accumulate=True) is out
    assert where(library) == [(name, index, 0x100 * index) for name in ("ds_balance_loss", "ds_balance_loss_grad")]
    assert library.calls[1][2][0] == state.at and library.calls[1][2][-2] is True
    assert fake.now == current


def test_a_scaler_on_another_gpu_is_refused(monkeypatch):
    op, _, library = balance(monkeypatch, current=1, index=1)
    z = Tensor(100, 64, index=1)
    with pytest.raises(ValueError, match="scaler"):
        op.gradient(z, Tensor(100, 64, index=1), scaler=Tensor(128, dtype=torch.uint8, index=0))
    assert library.calls == []


def test_a_stream_of_another_gpu_is_refused():
    from zero_mixed_precision_amd.multi_tensor import check_stream

    one = SimpleNamespace(device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="stream"):
        check_stream(one, torch.device("cuda", 0))
    for stream in (None, 0x7000, Stream(), one):
        check_stream(stream, torch.device("cuda", 1))
