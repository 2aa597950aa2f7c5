"""ds_step_list, the whole step over a list in one call: the bits of ds_check_overflow_list and ds_adam_step_list, in
every form that it takes by the list's length."""
import pytest
import torch

from zero_mixed_precision_amd import MultiTensorStep, ZeroMPConfig, _lib

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
TILE = 4096
# tiles: 1, 4, 8 (checked by the update), 9, 100 and 300 (a quarter of a tile a block, a whole one), 2048, 2049 (partial
# sums added by the update, or by a kernel of their own)
LISTS = {
    "one": [1],
    "few": [TILE, TILE, 64, 1],
    "eight": [3 * TILE, 0, 2 * TILE + 5, TILE - 1, 77],
    "nine": [8 * TILE, 1],
    "hundred": [TILE + 3 * k for k in range(49)] + [TILE - 1, 3, 0, 257],
    "three hundred": [TILE + 3 * k for k in range(148)] + [4 * TILE],
    "2048": [2000 * TILE, 48 * TILE],
    "2049": [2000 * TILE, 48 * TILE, 3],
}


def build(sizes, copy, grad, states, clip, shift, seed=None, dynamic=False, **kw):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(5)
    half = "fp16" if "fp16" in (copy, grad) else "bf16"
    rate = dict(initial_scale_power=8, hysteresis=1) if dynamic else dict(loss_scale=256.0 if half == "fp16" else 1.0)
    cfg = ZeroMPConfig(bf16=half == "bf16", lr=1e-3, gradient_clipping=clip, **rate)
    sample = lambda n, sigma, t: (torch.randn(n + shift, generator=gen, device=DEV) * sigma).to(t)[shift:]  # noqa: E731
    params = [sample(n, 0.02, TYPES[copy]) for n in sizes]
    grads = [sample(n, 0.5, TYPES[grad]) for n in sizes]
    op = MultiTensorStep(params, cfg, states=states, weight_decay=0.1, dither_seed=seed, **kw)
    op.set_gradients(grads)
    return op, grads


def same(a, b):
    arrays = lambda o: [o.m, o.v, o.state, *o.params, *(x for x in (o.master, o.m_scale, o.v_scale) if x is not None)]  # noqa: E731
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(arrays(a), arrays(b)))


@pytest.mark.parametrize("clip", [0.0, 0.3])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("states,seed", [("fp32", None), ("fp8", None), ("fp8", 3)])
@pytest.mark.parametrize("sizes", list(LISTS))
def test_the_bits_of_the_two_calls(sizes, states, seed, shift, clip):
    for copy, grad in (("bf16", "bf16"), ("fp16", "fp32"), ("fp16", "fp16"), ("fp32", "fp32")):
        one, _ = build(LISTS[sizes], copy, grad, states, clip, shift, seed)
        two, _ = build(LISTS[sizes], copy, grad, states, clip, shift, seed)
        for _ in range(3):
            one.step()
            two.check()
            two.update()
        torch.cuda.synchronize()
        assert same(one, two), (copy, grad)
        assert one.scaler().step == 3


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("states", ["fp32", "fp8"])
@pytest.mark.parametrize("sizes", ["few", "eight", "nine"])
def test_an_overflow_in_any_tile_skips_the_step(sizes, states, value):
    sizes = LISTS[sizes]
    one, g1 = build(sizes, "fp16", "fp16", states, 0.3, 0, dynamic=True)
    two, g2 = build(sizes, "fp16", "fp16", states, 0.3, 0, dynamic=True)
    skipped = 0
    for i, n in enumerate(sizes):
        for at in range(0, n, TILE):
            at = min(n, at + TILE) - 1
            keep = g1[i][at].clone()
            g1[i][at] = g2[i][at] = value
            one.step()
            two.check()
            two.update()
            skipped += 1
            g1[i][at] = g2[i][at] = keep
            assert same(one, two), (i, at)
    assert one.scaler().skipped == skipped and one.scaler().step == 0
    one.step()
    assert one.scaler().step == 1


@pytest.mark.parametrize("sizes", ["few", "nine", "2049"])
def test_what_was_checked_before_counts(sizes):
    """A flag raised and squares summed earlier in the step, by another list."""
    one, _ = build(LISTS[sizes], "bf16", "bf16", "fp32", 0.3, 0)
    two, _ = build(LISTS[sizes], "bf16", "bf16", "fp32", 0.3, 0)
    other, go = build([5000], "bf16", "bf16", "fp32", 0.3, 0)
    for spoiled in (False, True):
        if spoiled:
            go[0][4999] = float("inf")
        for op in (one, two):
            _lib.ds_check_overflow_list(op.state, other._list, other.ws)
        one.step()
        two.check()
        two.update()
        torch.cuda.synchronize()
        assert same(one, two)
    sc = one.scaler()
    assert sc.step == 1 and sc.skipped == 1 and sc.overflow == 0


def test_steps_that_share_a_scaler_clip_by_one_norm():
    """check() on each, then update(): both halves move as one list of all tensors does."""
    sizes = [5000, 300, 4096, 9]
    whole, gw = build(sizes, "bf16", "bf16", "fp32", 0.1, 0)
    cfg = whole.cfg
    params = [torch.empty_like(p).copy_(p) for p in whole.params]
    first = MultiTensorStep(params[:2], cfg, weight_decay=0.1, end_step=False)
    second = MultiTensorStep(params[2:], cfg, weight_decay=0.1, state=first.state)
    first.set_gradients(gw[:2])
    second.set_gradients(gw[2:])
    for _ in range(2):
        whole.step()
        for half in (first, second):
            half.check()
        for half in (first, second):
            half.update()
    torch.cuda.synchronize()
    # fp64 sums of the same squares in another order: below 1e-12 apart, which no rounding to fp32 and bf16 here shows
    a, b = whole.scaler().last_grad_sumsq, first.scaler().last_grad_sumsq
    assert abs(a - b) <= 1e-12 * a and a > 0.01
    for p, q in zip(whole.params, params):
        assert torch.equal(p, q)


def test_graph_replays():
    for sizes in ("few", "nine", "three hundred"):
        eager, _ = build(LISTS[sizes], "bf16", "bf16", "fp8", 0.3, 0, 4)
        caught, _ = build(LISTS[sizes], "bf16", "bf16", "fp8", 0.3, 0, 4)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            caught.step()
        for k in range(4):
            for g, h in zip(eager._grads, caught._grads):
                g.mul_(1.5 if k % 2 else 0.5)
                h.copy_(g)
            torch.cuda.synchronize()
            eager.step()
            graph.replay()
            torch.cuda.synchronize()
            assert same(eager, caught), (sizes, k)


def test_a_scaler_elsewhere_is_refused():
    p = [torch.zeros(10, dtype=torch.bfloat16, device=DEV)]
    cfg = ZeroMPConfig(bf16=True)
    with pytest.raises(ValueError, match="state"):
        MultiTensorStep(p, cfg, state=torch.zeros(_lib.ds_scaler_size(), dtype=torch.uint8))
    with pytest.raises(ValueError, match="state"):
        MultiTensorStep(p, cfg, state=torch.zeros(_lib.ds_scaler_size() - 1, dtype=torch.uint8, device=DEV))
    op = MultiTensorStep(p, cfg)
    for call in (op.step, op.check, op.update):
        with pytest.raises(RuntimeError, match="set_gradients"):
            call()


def test_replaced_gradients_are_not_reused_while_a_step_reads_them():
    """A gradient that set_gradients() has replaced goes back to torch's pool; on a stream of its own a step may still be
    to read it, so its memory must not come back before."""
    side = torch.cuda.Stream()
    n = 3_000_017
    op, grads = build([n], "bf16", "bf16", "fp32", 0.0, 0, stream=side)
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    new = torch.ones_like(grads[0])
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)           # about a tenth of a second
    op.step()
    op.set_gradients([new])
    old = grads.pop()
    at = old.data_ptr()
    del old
    again = torch.empty(n, dtype=torch.bfloat16, device=DEV)
    assert not side.query(), "the stream was to be busy here"
    assert again.data_ptr() != at
    torch.cuda.synchronize()
    assert op.scaler().step == 1
