"""The balance loss on a stream of its own, without a GPU: what it reads and writes is not handed out again before that
stream has done with it."""
import pytest
import torch

from tests.stand_in import Stream, Tensor, balance


@pytest.mark.parametrize("stream", [Stream(), 0x7000])
def test_what_a_stream_of_its_own_uses_is_recorded_there(stream, monkeypatch):
    op, _, library = balance(monkeypatch, stream)
    want = [("external", stream)] if isinstance(stream, int) else [stream]
    z, out, mask = Tensor(100, 64), Tensor(100, 64), Tensor(100, dtype=torch.bool)
    op.loss(z, mask=mask)
    assert z.recorded == want and mask.recorded == want
    state = Tensor(128, dtype=torch.uint8)
    op.gradient(z, out, mask=mask, scaler=state)
    assert z.recorded == mask.recorded == 2 * want and out.recorded == state.recorded == want
    assert [c[0] for c in library.calls] == ["ds_balance_loss", "ds_balance_loss_grad"]


def test_the_current_stream_needs_no_record(monkeypatch):
    op, _, _ = balance(monkeypatch)
    z, out, mask = Tensor(100, 64), Tensor(100, 64), Tensor(100, dtype=torch.bool)
    op.loss(z, mask=mask)
    op.gradient(z, out, mask=mask)
    assert z.recorded == out.recorded == mask.recorded == []
