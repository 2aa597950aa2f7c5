"""The step over a list on a stream of its own: what it uses may be let go of, and read on torch's current stream."""
import pytest
import torch

from zero_mixed_precision_amd import MultiTensorStep, ZeroMPConfig

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def busy(stream):
    """About a tenth of a second of work on ``stream``."""
    stream.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(200_000_000)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_parameters_and_a_shared_scaler_outlive_the_steps_that_use_them(dtype):
    side = torch.cuda.Stream()
    n = 3_000_017
    cfg = ZeroMPConfig(bf16=True, lr=1e-3)
    first = MultiTensorStep([torch.zeros(9, device=DEV)], cfg)
    params = [torch.zeros(n, dtype=dtype, device=DEV)]
    grads = [torch.ones_like(params[0])]
    op = MultiTensorStep(params, cfg, stream=side, state=first.state)
    op.set_gradients(grads)
    places = {params[0].data_ptr(), first.state.data_ptr()}
    busy(side)
    op.check()
    op.update()
    del op, params, first
    again = [torch.empty(n, dtype=dtype, device=DEV), torch.empty(128, dtype=torch.uint8, device=DEV)]
    assert not side.query(), "the stream was to be busy here"
    assert not places & {x.data_ptr() for x in again}
    torch.cuda.synchronize()
