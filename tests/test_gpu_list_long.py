"""The kernels that long lists take: streams with and without non-temporal hints, four tiles of gradients checked at once,
against 64 bits and against one another."""
import pytest
import torch

from tests.test_gpu_step_list import TYPES, build, same
from tests.test_gpu_tensor_list import HALF, cfg, check_step, make, snapshot
from zero_mixed_precision_amd import MultiTensorStep, _lib

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TILE = 4096
STATES = [("fp32", None), ("fp8", None), ("fp8", 0xFEDCBA9876543210)]


@pytest.mark.parametrize("end_step", [True, False])
@pytest.mark.parametrize("shift", [0, 1, 4])
@pytest.mark.parametrize("copy,grad", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32"), ("fp16", "fp16")])
@pytest.mark.parametrize("states,seed", STATES)
def test_either_kind_of_access(states, seed, copy, grad, shift, end_step, monkeypatch):
    """check() and update() of whole tiles, tails and odd tensors, a block per tile: against 64 bits, and the same bits
    with non-temporal hints and without."""
    sizes = [3 * TILE, TILE + 8, 5, 2 * TILE - 1, 0, TILE]
    scale = 1024.0 if "fp16" in (copy, grad) else 1.0
    ops = []
    for nt in ("1", "0"):
        monkeypatch.setenv("DSZERO_NT", nt)
        op, _, _, _ = make(sizes, copy, grad, states, shift=shift, scale=scale, weight_decay=0.05, dither_seed=seed,
                           gradient_clipping=0.3, end_step=end_step)
        for t in (1, 2):
            before = snapshot(op)
            op.check()
            op.update()
            if not end_step:
                assert op.scaler().step == t - 1         # left to a later call
                _lib.ds_update_loss_scale(op.state)
            check_step(op, before, t, [0.05] * len(sizes), seed=seed)
        ops.append(op)
    assert same(*ops)


@pytest.mark.parametrize("copy,grad", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp32")])
@pytest.mark.parametrize("states,seed", STATES)
def test_past_2_to_24_elements(states, seed, copy, grad, monkeypatch):
    """Where the hints are on by themselves: whole steps give the bits of the other kind."""
    sizes = [(1 << 24) - 3 * TILE, 2 * TILE, 5 * TILE + 9, 33]
    one, _ = build(sizes, copy, grad, states, 0.3, 0, seed)
    two, _ = build(sizes, copy, grad, states, 0.3, 0, seed)
    for _ in range(2):
        monkeypatch.delenv("DSZERO_NT", raising=False)
        one.step()
        monkeypatch.setenv("DSZERO_NT", "0")
        two.step()
    torch.cuda.synchronize()
    assert same(one, two)


@pytest.mark.parametrize("shift", [0, 1, 4])
@pytest.mark.parametrize("grad", ["fp16", "bf16", "fp32"])
def test_squares_of_more_than_2048_tiles(grad, shift):
    """Partial sums of four tiles each: the sum in 64 bits (n roundings at most), and a step clipped by it."""
    sizes = [1500 * TILE, 4 * TILE + 7, 3, 550 * TILE + 100, 0, TILE]
    copy = "bf16" if grad == "fp32" else grad
    scale = 1024.0 if grad == "fp16" else 1.0
    op, _, grads, _ = make(sizes, copy, grad, "fp32", shift=shift, scale=scale, gradient_clipping=0.5)
    before = snapshot(op)
    op.step()
    want = sum(float((g.double() ** 2).sum()) for g in grads)
    got = op.scaler().last_grad_sumsq
    assert abs(got - want) <= 2 * sum(sizes) * 2.0 ** -53 * want
    assert want ** 0.5 / scale > 2 * 0.5                 # so it clips
    check_step(op, before, 1, [0.0] * len(sizes))


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("squares", [False, True])
@pytest.mark.parametrize("grad", ["fp16", "bf16", "fp32"])
def test_an_overflow_anywhere_in_a_group(grad, squares, value):
    """First, middle and last elements of groups of four whole tiles, of the groups at a tensor's end and of its tail."""
    sizes = [1500 * TILE, 600 * TILE + 5, 7]
    half = "fp16" if grad == "fp16" else "bf16"
    params = [torch.zeros(n, dtype=TYPES[half], device=DEV) for n in sizes]
    grads = [torch.ones(n, dtype=TYPES[grad], device=DEV) for n in sizes]
    op = MultiTensorStep(params, cfg(half, gradient_clipping=1.0 if squares else 0.0))
    op.set_gradients(grads)
    places = [(0, at) for tile in (0, 1, 2, 3, 4, 700, 1499) for at in (tile * TILE, tile * TILE + 2049,
                                                                       tile * TILE + TILE - 1)]
    places += [(1, at) for at in (0, 2 * TILE, 4 * TILE - 1, 599 * TILE, 600 * TILE - 1, 600 * TILE, 600 * TILE + 4)]
    for i, at in places + [(2, 0), (2, 6)]:
        grads[i][at] = value
        op.check()
        assert op.scaler().overflow != 0, (i, at)
        grads[i][at] = 1.0
        _lib.ds_state_init(op.state, 1.0, 1.0, 1000, 1, 0, 0)
    op.check()
    sc = op.scaler()
    assert sc.overflow == 0 and sc.grad_sumsq == (float(sum(sizes)) if squares else 0.0)    # ones: exact


@pytest.mark.parametrize("states", ["fp32", "fp8"])
def test_many_tensors_against_64_bits(states):
    """More tensors than two rounds of the table search cover, some of them empty."""
    sizes = [k % 3 for k in range(4500)] + [5000]
    op, _, _, _ = make(sizes, "fp32", "fp32", states)
    before = snapshot(op)
    op.step()
    check_step(op, before, 1, [0.0] * len(sizes))


def test_the_dither_is_unbiased():
    """The mean of the dithered second moments over 2^22 elements against that of 32-bit ones, after 600 steps.  A
    rounding is off by less than a step of its code, 1/4 of the value at most, with a deviation of half of that, and none
    outlasts the value: below sqrt(600) / 8 of the mean for one element, so 0.0015 of it here, of which this allows five.
    A v below the smallest code (1e-9 of its block's top) is one in ten thousand."""
    n, steps = 1 << 22, 600
    gen = torch.Generator(device=DEV)
    means = {}
    for name, kw in (("32", dict(states="fp32")), ("dither", dict(states="fp8", dither_seed=21))):
        op = MultiTensorStep([torch.zeros(n, device=DEV)], cfg(), **kw)
        g = torch.empty(n, device=DEV)
        op.set_gradients([g])
        gen.manual_seed(13)
        for _ in range(steps):
            g.normal_(generator=gen)
            op.step()
        means[name] = float(op.moments(0)[1].double().mean())
    assert abs(means["dither"] / means["32"] - 1) < 0.0075


def test_halves_are_rounded_once():
    """The 16-bit copies of a long list are their masters, rounded."""
    for kind in ("fp16", "bf16"):
        op, _ = build([2049 * TILE + 3], kind, kind, "fp32", 0.0, 0)
        op.step()
        p, master = op.params[0].double(), op.view(op.master, 0).double()
        assert torch.equal(op.params[0], op.view(op.master, 0).to(TYPES[kind]))
        tol = HALF[kind] * master.abs() + (2.0 ** -25 if kind == "fp16" else 0.0)
        assert bool(((p - master).abs() <= tol).all())
