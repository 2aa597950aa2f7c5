"""The balance loss on a stream of its own: inputs that the caller lets go of while that stream has yet to read them."""
import pytest
import torch

from tests.test_gpu_balance import logits
from zero_mixed_precision_amd import ExpertBalance

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_inputs_are_not_reused_while_the_stream_has_yet_to_read_them():
    side = torch.cuda.Stream()
    op, plain = ExpertBalance(64, 4, 0.1, stream=side), ExpertBalance(64, 4, 0.1)
    T = 30011
    z = logits(T, 64, "bf16")
    drop = torch.arange(T, device=DEV) % 3 == 0
    want = plain.loss(z, mask=~drop).clone()
    d = plain.gradient(z, torch.empty_like(z), mask=~drop)
    out, mask, copy = torch.empty_like(z), ~drop, z.clone()
    places = {x.data_ptr() for x in (mask, copy)}
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)           # about a tenth of a second
    op.loss(copy, mask=mask)
    op.gradient(copy, out, mask=mask)
    del copy, mask
    again = [torch.zeros(T, dtype=torch.bool, device=DEV), torch.zeros_like(z)]
    assert not side.query(), "the stream was to be busy here"
    assert not places & {x.data_ptr() for x in again}
    torch.cuda.synchronize()
    assert torch.equal(op.value, want) and torch.equal(out, d)
