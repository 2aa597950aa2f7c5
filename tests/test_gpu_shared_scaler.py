"""Steps over lists that share a scaler: every list is checked before any is updated, and counts once in the norm."""
import pytest
import torch

from tests.test_gpu_step_list import build
from zero_mixed_precision_amd import MultiTensorStep

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def halves(whole, grads, at, **kw):
    """The tensors of ``whole`` as two lists under one scaler."""
    params = [torch.empty_like(p).copy_(p) for p in whole.params]
    first = MultiTensorStep(params[:at], whole.cfg, weight_decay=0.1, end_step=False, **kw)
    second = MultiTensorStep(params[at:], whole.cfg, weight_decay=0.1, state=first.state, **kw)
    first.set_gradients(grads[:at])
    second.set_gradients(grads[at:])
    return first, second, params


@pytest.mark.parametrize("states", ["fp32", "fp8"])
def test_a_list_that_does_not_end_the_step_is_checked_first(states):
    """step() of it, unchecked, would move it before the other list's overflow is known."""
    whole, grads = build([5000, 300], "fp16", "fp16", states, 0.0, 0, dynamic=True)
    first, second, params = halves(whole, grads, 1, states=states)
    old = [p.clone() for p in params]
    grads[1][299] = float("inf")
    with pytest.raises(RuntimeError, match="check"):
        first.step()
    for op in (first, second):
        op.check()
    first.step()
    second.step()
    sc = first.scaler()
    assert sc.skipped == 1 and sc.step == 0 and sc.scale == 128.0
    assert all(torch.equal(p, o) for p, o in zip(params, old))
    with pytest.raises(RuntimeError, match="check"):          # each step anew
        first.step()


@pytest.mark.parametrize("half", ["step", "update"])
@pytest.mark.parametrize("states", ["fp32", "fp8"])
def test_squares_count_once(states, half):
    """check() on both, then step() or update() on the first and update() on the second: the norm of all tensors, as one list of them has it."""
    whole, grads = build([5000, 300, 4096, 9], "bf16", "bf16", states, 0.1, 0)
    first, second, params = halves(whole, grads, 2, states=states)
    for t in (1, 2):
        whole.step()
        for op in (first, second):
            op.check()
        getattr(first, half)()
        second.update()
        a, b = whole.scaler().last_grad_sumsq, first.scaler().last_grad_sumsq
        assert abs(a - b) <= 1e-12 * a and a > 0.01           # fp64 sums of 9405 squares in another order
        assert first.scaler().step == t
        assert all(torch.equal(p, q) for p, q in zip(whole.params, params))


def test_step_after_check_of_one_list():
    """A list that ends its own step: squares that check() has summed are not summed again."""
    one, _ = build([5000, 300], "bf16", "bf16", "fp32", 0.1, 0)
    two, _ = build([5000, 300], "bf16", "bf16", "fp32", 0.1, 0)
    for _ in range(2):
        one.step()
        two.check()
        with pytest.raises(RuntimeError, match="update"):
            two.step()
        two.update()
    torch.cuda.synchronize()
    assert torch.equal(one.state, two.state) and all(torch.equal(p, q) for p, q in zip(one.params, two.params))
