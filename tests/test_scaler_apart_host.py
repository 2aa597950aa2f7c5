"""A scaler's state that lies inside a tensor of the step, without a GPU: refused before any launch."""
import pytest
import torch

from tests.stand_in import Tensor
from tests.test_other_device_host import tensor_step
from zero_mixed_precision_amd.multi_tensor import check_apart


@pytest.mark.parametrize("off,bad", [(-20, False), (-19, True), (0, True), (127, True), (128, False)])
def test_ranges(off, bad):
    """128 bytes of state and 20 of a tensor."""
    state, x = Tensor(128, dtype=torch.uint8, at=1000), Tensor(10, at=1000 + off)
    if bad:
        with pytest.raises(ValueError, match="gradient 3 shares"):
            check_apart(state, x, "gradient 3")
    else:
        check_apart(state, x, "gradient 3")


def test_gradients(monkeypatch):
    op, _, library = tensor_step(monkeypatch, 0, 0)
    op.state, op._shares = Tensor(128, dtype=torch.uint8, at=0x900000), True
    with pytest.raises(ValueError, match="gradient 0 shares"):
        op.set_gradients([Tensor(10, at=0x900000 + 120)])
    assert library.calls == []
    op.set_gradients([Tensor(10, at=0x900000 + 128)])
    assert [c[0] for c in library.calls] == ["ds_tensor_list_write"]
