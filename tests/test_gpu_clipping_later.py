"""gradient_clipping turned on, changed and turned off in the configuration of a running step over a list."""
import pytest
import torch

from tests.test_gpu_step_list import LISTS, build, same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("states", ["fp32", "fp8"])
@pytest.mark.parametrize("sizes", ["few", "nine", "hundred", "2049"])
def test_it_counts_from_the_next_step(sizes, states, halves):
    one, _ = build(LISTS[sizes], "bf16", "bf16", states, 0.0, 0)
    two, _ = build(LISTS[sizes], "bf16", "bf16", states, 0.3, 0)     # has room for the squares from the start

    def step(op):
        if halves:
            op.check()
            op.update()
        else:
            op.step()

    for clip in (0.0, 0.3, 0.1, 0.0):
        for op in (one, two):
            op.cfg.gradient_clipping = clip
        for op in (one, two):
            step(op)
        if clip:
            assert one.scaler().last_grad_sumsq > 1.0                # so it clips
            assert one.scaler().last_grad_sumsq == two.scaler().last_grad_sumsq
        for x, y in zip((one.m, one.v, *one.params), (two.m, two.v, *two.params)):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), clip
    one.cfg.gradient_clipping = two.cfg.gradient_clipping = 0.3
    step(one)
    step(two)
    assert same(one, two)
