"""The step over a list on a stream of its own: what it uses may be let go of, and read on torch's current stream."""
import pytest
import torch

from zero_mixed_precision_amd import ExpertBalance, MultiTensorStep, ZeroMPConfig

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


@pytest.mark.parametrize("states", ["fp32", "fp8"])
def test_what_the_current_stream_reads_is_after_the_steps(states):
    """Moments, loss scale and a loaded state, while the step's own stream is busy, against a step without one."""
    side = torch.cuda.Stream()
    cfg = ZeroMPConfig(initial_scale_power=10, hysteresis=1, lr=1e-3)
    n = 70_001

    def fresh(stream):
        gen = torch.Generator(device=DEV)
        gen.manual_seed(2)
        params = [(torch.randn(n, generator=gen, device=DEV) * 0.02).half()]
        op = MultiTensorStep(params, cfg, states=states, stream=stream)
        op.set_gradients([torch.randn(n, generator=gen, device=DEV).half()])
        return op

    plain, own = fresh(None), fresh(side)
    busy(side)
    for op in (plain, own):
        op.step()
    m, v = own.moments(0)
    for op in (plain, own):
        op.step()                                # must not reach the moments being read
    assert not side.query(), "the stream was to be busy here"
    again = fresh(None)
    again.step()
    for got, want in zip((m, v), again.moments(0)):
        assert torch.equal(got, want)
    for op in (plain, own):
        op._grads[0][n - 1] = float("inf")
    busy(side)
    own.step()
    assert float(own.loss_scale) == 512.0        # halved by that step
    plain.step()
    saved = again.state_dict()
    busy(side)
    own.load_state_dict(saved)
    got = own.params[0].clone()
    torch.cuda.synchronize()
    assert torch.equal(got, again.params[0]) and torch.equal(own.m.view(torch.uint8), again.m.view(torch.uint8))


def test_a_scaler_inside_a_parameter_is_refused():
    p = torch.zeros(4096, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="parameter 0 shares"):
        MultiTensorStep([p], ZeroMPConfig(bf16=True), state=p.view(torch.uint8)[4096:4224])


def test_leaves_of_autograd_on_a_stream_of_its_own():
    """Parameters and logits that require gradients."""
    side = torch.cuda.Stream()
    p = torch.zeros(100, 8, dtype=torch.bfloat16, device=DEV, requires_grad=True)
    p.grad = torch.ones_like(p)
    op = MultiTensorStep([p], ZeroMPConfig(bf16=True, lr=1e-3), stream=side)
    op.set_gradients([p.grad])
    balance = ExpertBalance(8, 2, 0.1, stream=side)
    side.wait_stream(torch.cuda.current_stream())
    op.step()
    balance.loss(p)
    balance.gradient(p, torch.empty_like(p), scaler=op.state)
    balance.loss(p * 2)
    torch.cuda.synchronize()
    assert int(balance.used) == 100 and op.scaler().step == 1
