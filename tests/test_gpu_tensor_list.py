"""The optimizer step over a list of tensors on the GPU: against the formulas in 64 bits (list_ref.py), against the flat
step bit for bit, and what it must leave alone."""
import numpy as np
import pytest
import torch

from tests import list_ref as ref
from zero_mixed_precision_amd import MultiTensorStep, ZeroMPConfig, _lib

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}
HP = dict(lr=1e-3, betas=(0.9, 0.999), eps=1e-8)


def cfg(kind="bf16", **kw):
    kw = {**HP, **kw}
    if kind == "fp16":
        return ZeroMPConfig(loss_scale=kw.pop("loss_scale", 1024.0), **kw)
    return ZeroMPConfig(bf16=True, **kw)


def rand(gen, n, sigma, dtype=torch.float32, shift=0):
    """n values at an offset of ``shift`` elements in their storage."""
    x = torch.randn(n + shift, generator=gen, device=DEV) * sigma
    return x.to(dtype)[shift:]


def make(sizes, copy, grad, states, seed=0, shift=0, scale=1.0, **kw):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    kind = "fp16" if "fp16" in (copy, grad) else "bf16"
    c = cfg(kind, **{k: kw.pop(k) for k in list(kw) if k in ("gradient_clipping", "gradient_accumulation_steps",
                                                            "loss_scale", "weight_decay", "betas", "lr", "eps")})
    params = [rand(gen, n, 0.02, TYPES[copy], shift) for n in sizes]
    grads = [rand(gen, n, 1e-2 * scale, TYPES[grad], shift) for n in sizes]
    op = MultiTensorStep(params, c, states=states, **kw)
    op.set_gradients(grads)
    return op, params, grads, gen


def snapshot(op):
    f = lambda t: t.detach().cpu().clone()  # noqa: E731
    out = []
    for i, p in enumerate(op.params):
        d = {"param": f(p), "grad": f(op._grads[i]), "master": f(p if p.dtype == torch.float32 else
                                                                op.view(op.master, i))}
        n, at = op.numels[i], op.offsets[i] // 256
        for k in ("m", "v"):
            a = op.view(getattr(op, k), i)
            d[k] = f(a.view(torch.uint8)) if op.states == "fp8" else f(a)
            if op.states == "fp8":
                d[k + "_scale"] = f(getattr(op, k + "_scale")[at:at + -(-n // 256)])
        out.append(d)
    return out


def norm_factor(before, c, scale, K):
    """1 / (S K) times the clipping coefficient, in 64 bits."""
    inv = 1.0 / (scale * K)
    if c.gradient_clipping:
        sq = sum(float((d["grad"].double() ** 2).sum()) for d in before)
        inv *= min(1.0, c.gradient_clipping / (np.sqrt(sq) * inv + 1e-6))
    return inv


def check_step(op, before, t, decay, rates=None, seed=None):
    """The state after one step that applied, against 64 bits."""
    after, c = snapshot(op), op.cfg
    inv = norm_factor(before, c, op.scaler().scale, c.gradient_accumulation_steps)
    for i, (b, a) in enumerate(zip(before, after)):
        if op.numels[i] == 0:
            continue
        num = lambda x: x.numpy().astype(np.float64)  # noqa: E731
        eight, slack = op.states == "fp8", 0
        if eight:
            n = op.numels[i]
            m = ref.E4M3.decode(b["m"].numpy()) * ref.spread(num(b["m_scale"]), n)
            v = ref.E5M2.decode(b["v"].numpy()) * ref.spread(num(b["v_scale"]), n)
            slack = 1                          # the product with the scale
        else:
            m, v = num(b["m"]), num(b["v"])
        rate = 1.0 if rates is None else rates[i]
        lr = float(np.float32(np.float32(c.lr) * np.float32(rate)))
        got, err = ref.update(num(b["master"]), m, v, num(b["grad"].float()), lr=lr, b1=c.betas[0], b2=c.betas[1],
                              eps=c.eps, wd=decay[i], t=t, inv=inv, slack=slack)
        p = num(a["master"])
        assert np.all(np.abs(p - got["p"]) <= err["p"]), f"tensor {i}: master off by {np.abs(p - got['p']).max()}"
        if a["param"].dtype != torch.float32:
            kind = "bf16" if a["param"].dtype == torch.bfloat16 else "fp16"
            q = num(a["param"].float())
            tol = err["p"] + HALF[kind] * (np.abs(got["p"]) + err["p"]) + (2.0 ** -25 if kind == "fp16" else 0)
            assert np.all(np.abs(q - got["p"]) <= tol), f"tensor {i}: parameter"
        if not eight:
            for k in ("m", "v"):
                assert np.all(np.abs(num(a[k]) - got[k]) <= err[k]), f"tensor {i}: {k}"
            continue
        um, uv = (0.5, 0.5) if seed is None else ref.dither(seed, t, i, op.numels[i])
        ref.check_codes(a["m"].numpy(), num(a["m_scale"]), got["m"], err["m"], um, ref.E4M3, f"tensor {i}: m")
        ref.check_codes(a["v"].numpy(), num(a["v_scale"]), got["v"], err["v"], uv, ref.E5M2, f"tensor {i}: v")


SIZES = {
    "one": [1],
    "blocks": [255, 256, 257, 511, 513],
    "tiles": [4095, 4096, 4097, 12288, 8191],
    "empty": [0, 7, 0, 0, 4100, 0],
    "seventy": [1 + (37 * k) % 300 for k in range(70)],
    "large": [1_000_003, 65_536],
}


@pytest.mark.parametrize("shift", [0, 1, 3])
@pytest.mark.parametrize("states", ["fp32", "fp8"])
@pytest.mark.parametrize("sizes", list(SIZES))
def test_step_against_64_bits(sizes, states, shift):
    """Three steps over every size; arrays at an offset take the element-wise form."""
    sizes = SIZES[sizes]
    op, _, _, gen = make(sizes, "bf16", "bf16", states, shift=shift, weight_decay=0.1)
    for t in (1, 2, 3):
        op.set_gradients([rand(gen, n, 1e-2, torch.bfloat16, shift) for n in sizes])
        before = snapshot(op)
        op.step()
        check_step(op, before, t, [0.1] * len(sizes))
    assert op.scaler().step == 3


@pytest.mark.parametrize("states,seed", [("fp32", None), ("fp8", None), ("fp8", 0xFEDCBA9876543210)])
@pytest.mark.parametrize("copy,grad", [("fp16", "fp16"), ("bf16", "bf16"), ("fp16", "fp32"), ("bf16", "fp32"),
                                       ("fp32", "fp32"), ("fp32", "bf16"), ("fp32", "fp16")])
def test_types(copy, grad, states, seed):
    sizes = [5000, 300, 1, 4096]
    scale = 1024.0 if "fp16" in (copy, grad) else 1.0
    op, _, _, _ = make(sizes, copy, grad, states, scale=scale, weight_decay=0.01, dither_seed=seed)
    for t in (1, 2, 3):
        before = snapshot(op)
        op.step()
        check_step(op, before, t, [0.01] * 4, seed=seed)


@pytest.mark.parametrize("states", ["fp32", "fp8"])
def test_mixed_types_groups_clipping_and_accumulation(states):
    """fp32 and bf16 parameters, fp32 and bf16 gradients, a decay and a rate per tensor, in one list."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(3)
    kinds = [("bf16", "bf16", 9000), ("fp32", "fp32", 4097), ("fp32", "bf16", 77), ("bf16", "fp32", 4096)]
    params = [rand(gen, n, 0.02, TYPES[c]) for c, _, n in kinds]
    grads = [rand(gen, n, 1.0, TYPES[g]) for _, g, n in kinds]
    decay, rates = [0.1, 0.0, 0.5, 0.0], [1.0, 0.25, 3.0, 0.0]
    op = MultiTensorStep(params, cfg(gradient_clipping=0.5, gradient_accumulation_steps=4), states=states,
                         weight_decay=decay, lr_scale=rates)
    op.set_gradients(grads)
    for t in (1, 2):
        before = snapshot(op)
        op.step()
        check_step(op, before, t, decay, rates)
    sq = sum(float((g.double() ** 2).sum()) for g in grads)
    # fp64 sums of n = 17,270 squares, each exact or rounded once
    assert abs(op.scaler().last_grad_sumsq - sq) <= 17270 * 2.0 ** -53 * sq


def test_many_tensors():
    """More tensors than two rounds of the table search cover, some of them empty."""
    sizes = [k % 3 for k in range(4500)] + [5000]
    op, params, grads, _ = make(sizes, "fp32", "fp32", "fp32")
    old = [p.clone() for p in params]
    op.step()
    torch.cuda.synchronize()
    for n, p, o, g in zip(sizes, params, old, grads):
        if n:   # the first step moves each value by lr against its gradient's sign (eps aside)
            moved = (o - p).double()
            want = 1e-3 * g.double() / (g.double().abs() + 1e-8)
            assert float((moved - want).abs().max()) <= 1e-3 * 1e-5 + 4 * ref.E * float(o.abs().max())
    # gradients large against eps / sqrt(1 - beta2) = 3e-7, or the step is short
    assert min(float(g.abs().min()) for g in grads if g.numel()) >= 0


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("copy", ["fp16", "bf16"])
def test_32_bit_states_are_the_flat_step_bit_for_bit(copy, shift):
    sizes = [4096, 5001, 130, 16384, 3]
    scale = 1024.0 if copy == "fp16" else 1.0
    op, params, grads, _ = make(sizes, copy, copy, "fp32", shift=shift, scale=scale, weight_decay=0.05,
                                gradient_clipping=1.0, betas=(0.875, 1 - 2.0 ** -10))   # betas that fp32 holds
    flat = []
    code = {"fp16": _lib.DS_FP16, "bf16": _lib.DS_BF16}[copy]
    for i, (p, g) in enumerate(zip(params, grads)):
        pad = lambda x: torch.cat([x, x.new_zeros(-x.numel() % 8)])  # noqa: E731
        flat.append([pad(op.view(op.master, i)), pad(op.view(op.m, i)), pad(op.view(op.v, i)),
                     pad(p).view(torch.int16), pad(g.clone())])
    st = op.state.clone()
    for _ in range(3):
        # the joint norm as the list's check leaves it, then the flat step on each tensor
        _lib.ds_check_overflow_list(st, op._list, op.ws)
        for n, f in zip(sizes, flat):
            _lib.ds_adam_step(st, *f[:4], code, f[4], code, n, op.cfg.lr, *op.cfg.betas, op.cfg.eps, 0.05, 1.0, 1)
        _lib.ds_update_loss_scale(st)
        op.step()
    torch.cuda.synchronize()
    for i, (n, f) in enumerate(zip(sizes, flat)):
        for mine, k in zip(f[:3], ("master", "m", "v")):
            assert torch.equal(mine[:n], op.view(getattr(op, k), i)), (i, k)
        assert torch.equal(f[3][:n], params[i].view(torch.int16)), i
    assert torch.equal(st, op.state)


@pytest.mark.parametrize("clip", [0.0, 1.0])
@pytest.mark.parametrize("states", ["fp32", "fp8"])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_overflow_changes_nothing_but_the_scaler(states, clip, value):
    sizes = [4096, 3, 8193, 300]
    c = ZeroMPConfig(initial_scale_power=10, hysteresis=1, gradient_clipping=clip, **HP)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    params = [rand(gen, n, 0.02, torch.float16) for n in sizes]
    op = MultiTensorStep(params, c, states=states)
    grads = [rand(gen, n, 1.0, torch.float16) for n in sizes]
    op.set_gradients(grads)
    op.step()
    for i, at in ((0, 4095), (1, 2), (2, 8192), (2, 17), (3, 299)):
        before, scale = snapshot(op), op.scaler().scale
        keep = grads[i][at].clone()
        grads[i][at] = value
        op.step()
        sc = op.scaler()
        assert sc.last_overflow == 1 and sc.scale == max(scale / 2, 1.0) and sc.step == 1
        grads[i][at] = keep
        for b, a in zip(before, snapshot(op)):
            for k in b:
                if k != "grad":
                    assert torch.equal(b[k], a[k]), k
    op.step()
    assert op.scaler().step == 2 and op.scaler().last_overflow == 0


def test_flag_raised_before_and_a_step_of_two_lists():
    """Two lists share a scaler: the first does not advance it, and an overflow in either skips both."""
    c = ZeroMPConfig(initial_scale_power=4, hysteresis=1, **HP)
    gen = torch.Generator(device=DEV)
    a, b = ([rand(gen, 5000, 0.02, torch.float16)] for _ in range(2))
    first = MultiTensorStep(a, c, end_step=False)
    second = MultiTensorStep(b, c, states="fp8", state=first.state)
    ga, gb = ([rand(gen, 5000, 1.0, torch.float16)] for _ in range(2))
    first.set_gradients(ga)
    second.set_gradients(gb)

    def step():
        _lib.ds_check_overflow_list(first.state, first._list)
        _lib.ds_check_overflow_list(first.state, second._list)
        first.step()
        second.step()

    step()
    assert first.scaler().step == 1
    old = a[0].clone(), b[0].clone()
    gb[0][4999] = float("inf")
    step()
    assert first.scaler().step == 1 and torch.equal(a[0], old[0]) and torch.equal(b[0], old[1])


def test_ungated_nan_stays_a_nan_and_to_itself():
    """Without the check a NaN gradient spoils its element only, in 8 bits as in 32."""
    gen = torch.Generator(device=DEV)
    params = [rand(gen, 5000, 0.02)]
    grads = [rand(gen, 5000, 1e-2)]
    op = MultiTensorStep(params, cfg(), states="fp8")
    op.set_gradients(grads)
    grads[0][77] = float("nan")
    _lib.ds_adam_step_list(op.state, op._list, 1e-3, None, 0.9, 0.999, 1e-8, 0.0, 1)
    m, v = op.moments(0)
    for x in (m, v, params[0]):
        bad = torch.isnan(x).cpu()
        assert bad[77] and bad.sum() == 1


def test_extreme_gradients_in_8_bits():
    """Finite gradients whose square overflows fp32, and ones near fp32's smallest, leave finite states."""
    n = 1024
    g = torch.full((n,), 1e-3, device=DEV)
    g[5], g[300], g[301] = 3e38, 1e25, -3e38
    g[512:768] = 1e-37
    g[768:] = 0.0
    op = MultiTensorStep([torch.ones(n, device=DEV)], cfg(), states="fp8")
    op.set_gradients([g])
    for _ in range(5):
        op.step()
        m, v = op.moments(0)
        assert torch.isfinite(m).all() and torch.isfinite(v).all() and torch.isfinite(op.params[0]).all()
        assert (v[:512] > 0).all()              # a second moment that is not zero stays so
        assert (m[768:] == 0).all() and (v[768:] == 0).all()


def test_small_second_moments_do_not_vanish():
    """Beside a large element v keeps the smallest code, so no element gets a step without a denominator."""
    n = 256
    g = torch.full((n,), 1e-6, device=DEV)
    g[0] = 1.0                                  # the others' v is 1e-12 of the block's: far below code 1
    for seed in (None, 5):
        p = torch.zeros(n, device=DEV)
        op = MultiTensorStep([p], cfg(), states="fp8", dither_seed=seed)
        op.set_gradients([g])
        for _ in range(20):
            op.step()
        assert (op.view(op.v, 0).view(torch.uint8) >= 1).all()
        assert float(p.abs().max()) <= 20 * 1e-3 * 1.1


def test_dither_keeps_the_expected_second_moment():
    """The dithered state follows the 32-bit one: each rounding is unbiased, and the EMA is linear, so the mean over 65,536 elements
    differs by noise alone (well below 1 %) and by what the scales' clamps lose."""
    n, steps = 65536, 600
    gen = torch.Generator(device=DEV)
    gen.manual_seed(11)
    sides = {}
    for name, kw in (("32", dict(states="fp32")), ("dither", dict(states="fp8", dither_seed=9))):
        p = torch.zeros(n, device=DEV)
        op = MultiTensorStep([p], cfg(), **kw)
        g = torch.empty(n, device=DEV)
        op.set_gradients([g])
        gen.manual_seed(12)
        for _ in range(steps):
            g.normal_(generator=gen)
            op.step()
        sides[name] = float(op.moments(0)[1].mean())
    assert abs(sides["dither"] / sides["32"] - 1) < 0.04


def test_nearest_holds_what_the_dither_lets_decay():
    """One value of each block keeps the block's top where it is; the others' gradients have stopped.  Their v loses
    0.001 of itself per step, less than half a code (1/16), so nearest keeps every code.  With the dither the mean over
    65,280 values falls as 0.999^300 = 0.741: per value the deviation is below 1/4, so 0.25 / 255 of the mean here."""
    n, steps = 65536, 300
    for seed, want in ((None, 1.0), (5, 0.999 ** steps)):
        p = torch.zeros(n, device=DEV)
        g = torch.ones(n, device=DEV)
        op = MultiTensorStep([p], cfg(), states="fp8", dither_seed=seed)
        op.set_gradients([g])
        op.v.view(torch.uint8).fill_(0x7B)      # every v at the block's top, 1
        op.v_scale.fill_(1 / 57344)
        g.view(-1, 256)[:, 1:] = 0.0
        for _ in range(steps):
            op.step()
        v = op.moments(0)[1].view(-1, 256)
        assert float((v[:, 0] - 1).abs().max()) <= 300 * 12 * ref.E
        assert abs(float(v[:, 1:].mean()) - want) <= 0.01


def test_dither_is_a_function_of_seed_and_step():
    outs = []
    for seed in (1, 1, 2):
        op, _, _, _ = make([70000], "bf16", "bf16", "fp8", dither_seed=seed)
        for _ in range(3):
            op.step()
        outs.append(op.m.view(torch.uint8).cpu())
    assert torch.equal(outs[0], outs[1]) and not torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("states", ["fp32", "fp8"])
def test_results_do_not_depend_on_the_launch(states, monkeypatch):
    """Pinned grids and either kind of access give the same bits."""
    ref_out = None
    for grid, nt in (("0", "-1"), ("1", "0"), ("3", "1"), ("50", "0")):
        monkeypatch.setenv("DSZERO_GRID", grid)
        monkeypatch.setenv("DSZERO_NT", nt)
        op, params, _, _ = make([20000, 5, 4097], "bf16", "bf16", states, gradient_clipping=0.1,
                                dither_seed=4 if states == "fp8" else None)
        for _ in range(2):
            op.step()
        out = [x.view(torch.uint8).cpu() for x in (op.master, op.m, op.v, op.state, *params)]
        ref_out = ref_out or out
        assert all(torch.equal(a, b) for a, b in zip(ref_out, out))


@pytest.mark.parametrize("states", ["fp32", "fp8"])
def test_graph_replays_and_another_stream(states):
    """Replays between eager work give the eager result; so does a step on a stream of its own."""
    def fresh(stream=None):
        return make([9000, 33, 4096], "bf16", "bf16", states, gradient_clipping=0.5, stream=stream,
                    dither_seed=8 if states == "fp8" else None)

    eager, captured = fresh(), fresh()
    side = torch.cuda.Stream()
    other = fresh(side)
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured[0].step()
    for k in range(4):
        for op, _, grads, _ in (eager, captured, other):
            for g in grads:
                g.mul_(0.5 if k % 2 else 2.5)
        torch.cuda.synchronize()
        eager[0].step()
        graph.replay()
        other[0].step()
        torch.cuda.synchronize()
        for o in (captured[0], other[0]):
            for a, b in zip((eager[0].master, eager[0].m, eager[0].v, eager[0].state, *eager[0].params),
                            (o.master, o.m, o.v, o.state, *o.params)):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), k


def test_schedule_and_resume():
    """A schedule moves with the applied steps; a restored state goes on bit for bit."""
    c = ZeroMPConfig(bf16=True, betas=(0.9, 0.999), scheduler="WarmupLR", warmup_min_lr=0.0, warmup_max_lr=1e-2,
                     warmup_num_steps=10)
    gen = torch.Generator(device=DEV)
    p = [rand(gen, 700, 0.02, torch.bfloat16)]
    g = [rand(gen, 700, 1.0, torch.bfloat16)]
    op = MultiTensorStep(p, c, states="fp8", dither_seed=3)
    op.set_gradients(g)
    old = op.master.clone()
    op.step()                                    # lr 0 at the first step
    assert torch.equal(old, op.master)
    for _ in range(4):
        op.step()
    saved = op.state_dict()
    twin = MultiTensorStep([torch.zeros_like(p[0])], c, states="fp8", dither_seed=3)
    twin.load_state_dict(saved)
    twin.set_gradients(g)
    assert torch.equal(twin.params[0], p[0])
    for o in (op, twin):
        o.step()
    for k in ("master", "m", "v", "m_scale", "v_scale", "state"):
        assert torch.equal(getattr(op, k).view(torch.uint8), getattr(twin, k).view(torch.uint8)), k
    with pytest.raises(ValueError):
        MultiTensorStep([torch.zeros(701, device=DEV)], c).load_state_dict(saved)


def test_offsets_past_32_bits():
    """A tensor of more than 2^32 bytes of fp32 and 2^30 elements, checked at both ends and around 2^30."""
    n = (1 << 30) + 4097
    p = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    g = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    op = MultiTensorStep([p], cfg(), states="fp8")
    at = torch.tensor([0, 1 << 28, (1 << 30) - 1, 1 << 30, n - 1], device=DEV)
    g[at] = 1.0
    op.set_gradients([g])
    op.step()
    torch.cuda.synchronize()
    assert torch.equal(torch.nonzero(p).flatten(), at)
    assert torch.allclose(p[at].float(), torch.full((5,), -1e-3, device=DEV), rtol=2 ** -7)
    g[n - 1] = float("inf")
    op.step()
    assert op.scaler().last_overflow == 1


def test_refusals_of_the_class():
    p = torch.zeros(10, dtype=torch.bfloat16, device=DEV)
    op = MultiTensorStep([p], cfg())
    with pytest.raises(RuntimeError, match="set_gradients"):
        op.step()
    for bad in ([], [torch.zeros(9, device=DEV)], [torch.zeros(10)], [torch.zeros(10, 2, device=DEV)[:, 0]], [None],
                [torch.zeros(10, dtype=torch.float16, device=DEV)], [torch.zeros(10, dtype=torch.int32, device=DEV)]):
        with pytest.raises(ValueError):
            op.set_gradients(bad)
    with pytest.raises(_lib.DsError, match="ALIAS"):
        op.set_gradients([p])
    with pytest.raises(RuntimeError, match="set_gradients"):      # a refused list is not used
        op.step()
    with pytest.raises(_lib.DsError, match="ALIAS"):
        MultiTensorStep([p, p], cfg()).set_gradients([torch.zeros_like(p)] * 2)
