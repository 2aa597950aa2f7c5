"""Distillation from a teacher's top logits on the GPU against the formulas in 64 bits, with bounds counted from fp32's half
unit E = 2^-24 and the output type's."""
import math

import pytest
import torch

from zero_mixed_precision_amd import TopLogitDistillation, _lib

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E32 = 2.0 ** -24
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -149}
INF = math.inf


def generator(seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return gen


def soft(x, tau, adds):
    """(log2 of the softmax of x / tau, an absolute bound on it) per row; -infinity stays.  Counted: the difference to the
    maximum, the factor and their product (3 E of the exponent), the sum (`adds` of its terms, their exponents' errors by
    weight, the instruction's 2), its logarithm (4 E of itself or of 1)."""
    a = (x - x.amax(1, keepdim=True)) / tau / math.log(2)
    p = torch.exp2(a)
    total = p.sum(1, keepdim=True)
    size = torch.where(p > 0, a.abs(), 0.0)
    rel = (p * (3 * size * math.log(2) + 2)).sum(1, keepdim=True) / total + adds
    log = torch.log2(total)
    bound = (3 * torch.where(a > -INF, a.abs(), 0.0) + rel / math.log(2) + 4 * log.clamp(min=1) + 2 * (a.abs().clamp(max=1e9) + log)) * E32
    return a - log, bound


def reference(z, teacher, index, mask, tau, coef, scale):
    """Values and bounds in 64 bits; rows that hold NaN, +infinity or a place past the vocabulary are NaN."""
    T, V = z.shape
    z, t = z.double(), teacher.double()
    t = torch.where(index >= 0, t, -INF)
    used = mask & (~(t == -INF)).any(1) & (~(z == -INF)).any(1)
    odd = used & ((~(z < INF)).any(1) | (~(t < INF)).any(1) | (index >= V).any(1))
    fine = used & ~odd
    out = dict(used=used, loss=torch.zeros(T, dtype=torch.float64, device=DEV), d=torch.zeros_like(z))
    out["eloss"], out["ed"] = torch.zeros_like(out["loss"]), torch.zeros_like(z)
    n, k = int(used.sum()), index.shape[1]
    out["n"] = n
    factor = scale * coef * tau / max(n, 1)
    rows = torch.nonzero(fine).flatten()
    if len(rows):
        lp, elp = soft(z[rows], tau, V / 256 + 64)
        lq, elq = soft(t[rows], tau, k / 256 + 64)
        at = index[rows].long().clamp(min=0)
        q = torch.exp2(lq)
        eq = q * (elq * math.log(2) + 2 * E32)
        of, eof = lp.gather(1, at), elp.gather(1, at)
        gap = torch.where(q > 0, lq - of, 0.0)
        term = torch.where(q > 0, q * gap, 0.0)
        eterm = torch.where(q > 0, q * (elq + eof + 2 * E32 * gap.abs()) + eq * gap.abs(), 0.0)
        out["loss"][rows] = tau * tau * math.log(2) * term.sum(1)
        out["eloss"][rows] = tau * tau * math.log(2) * (eterm.sum(1) + (k / 256 + 40) * E32 * term.abs().sum(1))
        p = torch.exp2(lp)
        ep = p * (elp * math.log(2) + 2 * E32)
        d, ed = p, ep
        d = d.scatter_add(1, at, torch.where(index[rows] >= 0, -q, 0.0))
        share = torch.zeros_like(p).scatter_add(1, at, torch.where(index[rows] >= 0, q, 0.0))
        ed = ed + torch.zeros_like(p).scatter_add(1, at, torch.where(index[rows] >= 0, eq, 0.0)) + k * E32 * share
        out["d"][rows] = factor * d
        out["ed"][rows] = factor * (ed + 4 * E32 * d.abs())
    out["loss"][odd] = math.nan
    out["d"][odd] = math.nan
    out["mean"] = coef * out["loss"].sum() / max(n, 1)
    out["emean"] = coef * out["eloss"].sum() / max(n, 1) + 4 * E32 * out["mean"].abs()
    return out


def close(got, want, bound, tiny=True):
    half, tiny = HALF[got.dtype], TINY[got.dtype]
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    tol = bound + half * (want.abs() + bound) + tiny
    bad = ~((got - want).abs() <= tol) & ~torch.isnan(want) & ~(got == want)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, by up to {float((got - want)[bad].abs().max())}"


def state(scale):
    st = torch.zeros(_lib.ds_scaler_size(), dtype=torch.uint8, device=DEV)
    _lib.ds_state_init(st, scale, 1.0, 1000, 1, 0, 0)
    return st


def check(op, z, teacher, index, mask=None, scale=None, out=None, accumulate=False):
    T = z.shape[0]
    base = out.double().clone() if accumulate else None
    r = reference(z, teacher, index, torch.ones(T, dtype=torch.bool, device=DEV) if mask is None else mask != 0,
                  op.temperature, op.coef, scale or 1.0)
    op.loss(z, teacher, index, mask=mask)
    alone = op.token_loss[:T].clone(), op.value.clone()
    out = torch.full_like(z, 7.0) if out is None else out
    op.loss_and_gradient(z, teacher, index, out, mask=mask, scaler=None if scale is None else state(scale),
                         accumulate=accumulate)
    assert int(op.used) == r["n"]
    for a, b in ((alone[0], op.token_loss[:T]), (alone[1], op.value)):       # the same bits with and without the gradient
        assert torch.equal(a.view(torch.int32), b.view(torch.int32))
    close(op.token_loss[:T], r["loss"], r["eloss"])
    close(op.value, r["mean"], r["emean"])
    if accumulate:
        want = torch.where(r["used"][:, None], base + r["d"], base)
        close(out, want, r["ed"] + E32 * want.abs())
        assert torch.equal(out[~r["used"]].double(), base[~r["used"]])
    else:
        close(out, r["d"], r["ed"])
    return r


def inputs(T, V, k, kind, tkind="fp32", seed=0, index=torch.int32, spread=2.0):
    gen = generator(seed)
    z = (torch.randn(T, V, generator=gen, device=DEV) * spread).to(TYPES[kind])
    at = torch.rand(T, V, generator=gen, device=DEV).topk(min(k, V), dim=1).indices if V <= 4096 else \
        torch.arange(k, device=DEV) * (V // k) + torch.randint(V // k, (T, k), generator=gen, device=DEV)
    if k > V:
        at = torch.cat([at, torch.full((T, k - V), -1, device=DEV)], 1)
    t = (torch.randn(T, k, generator=gen, device=DEV) * 3).to(TYPES[tkind])
    return z, t, at.to(index)


SIZES = [(1, 1, 1), (1, 2, 2), (3, 7, 3), (5, 8, 4), (2, 255, 10), (4, 256, 256), (9, 1000, 64), (3, 2047, 5), (2, 2049, 300),
         (5, 8191, 20), (3, 8193, 20), (4, 32000, 64), (2, 32769, 50), (3, 50021, 50), (2, 65543, 1024), (3, 131072, 100),
         (2, 131081, 3), (2, 200003, 700)]


@pytest.mark.parametrize("kind,tkind,index", [("fp16", "fp16", torch.int32), ("bf16", "fp32", torch.int64),
                                              ("fp32", "bf16", torch.int32)])
@pytest.mark.parametrize("T,V,k", SIZES)
def test_against_64_bits(T, V, k, kind, tkind, index):
    z, t, at = inputs(T, V, k, kind, tkind, index=index)
    check(TopLogitDistillation(V, k, T, 1.0), z, t, at)
    check(TopLogitDistillation(V, k, T, 2.5, coef=0.5), z, t, at, scale=1024.0)


@pytest.mark.parametrize("kind", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("T,V,k", [(200, 1000, 16), (77, 5003, 33), (1500, 260, 8), (9, 70001, 100)])
def test_masks_and_lists_of_different_lengths(T, V, k, kind):
    z, t, at = inputs(T, V, k, kind, kind)
    gen = generator(9)
    at = torch.where(torch.rand(T, k, generator=gen, device=DEV) < 0.4, -1, at)
    mask = torch.rand(T, generator=gen, device=DEV) < 0.7
    at[0] = -1                                            # a row without an entry
    t[1] = -INF                                           # or with none above -infinity
    z[2] = -INF                                           # a student whose vocabulary is masked away
    mask[:3] = True
    mask[3] = False
    z[3], t[3] = math.nan, INF                            # what a padded row holds reaches nothing
    op = TopLogitDistillation(V, k, T, 2.0)
    r = check(op, z, t, at, mask=mask, scale=8.0)
    assert not r["used"][:4].any()
    check(op, z, t, at, mask=mask.to(torch.uint8) * 5, out=torch.randn_like(z, dtype=torch.float32).to(z.dtype),
          accumulate=True)
    r = check(op, z, t, at, mask=torch.zeros_like(mask))
    assert r["n"] == 0 and float(op.value) == 0.0


@pytest.mark.parametrize("kind", ["fp16", "bf16", "fp32"])
def test_extreme_logits(kind):
    """Logits at the type's lowest value, -infinity in places, a single one that has it all."""
    low = torch.finfo(TYPES[kind]).min
    V, k = 300, 4
    z, t, at = inputs(8, V, k, kind, kind)
    z[0] = low                                            # nothing but the lowest value: even probabilities
    z[1, 5:] = low
    z[2, ::2] = -INF
    at[2] = torch.tensor([1, 3, 5, 7], device=DEV)
    z[3], z[3, 17] = -INF, 3.0
    at[3] = torch.tensor([17, -1, -1, -1], device=DEV)
    t[4, :3] = -INF                                       # one entry
    t[5] = low                                            # even shares
    z[6] = torch.finfo(TYPES[kind]).max
    t[7, 1] = 200.0
    check(TopLogitDistillation(V, k, 8, 1.0), z, t, at)
    op = TopLogitDistillation(V, k, 1, 1.0)               # a place that the student rules out: an infinite loss
    z, t, at = inputs(1, V, k, kind, kind)
    z[0, int(at[0, 0])] = -INF
    out = torch.empty_like(z)
    assert float(op.loss_and_gradient(z, t, at, out)) == INF
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("kind", ["fp16", "fp32"])
def test_rows_that_are_not_numbers(kind):
    V, k = 5000, 6
    z, t, at = inputs(7, V, k, kind)
    z[0, 4321], z[1, 3], t[2, 1], t[3, 2] = math.nan, INF, math.nan, INF
    at[4, 0] = V
    at[5, 5] = 2 ** 31 - 1
    r = check(TopLogitDistillation(V, k, 7), z, t, at)
    assert r["n"] == 7 and torch.isnan(r["loss"]).tolist() == [True] * 6 + [False]


def test_the_same_place_twice_adds_up():
    V, k = 600, 40
    z, t, at = inputs(6, V, k, "fp32")
    at = torch.randint(0, 9, (6, k), device=DEV, dtype=torch.int32)
    at[5] = 0
    check(TopLogitDistillation(V, k, 6, 1.5), z, t, at)
    check(TopLogitDistillation(V, k, 6, 1.5), z, t, at, out=torch.randn_like(z), accumulate=True)


@pytest.mark.parametrize("kind,V", [("bf16", 1000), ("bf16", 50021), ("fp32", 300), ("fp16", 262147)])
def test_strides_and_in_place(kind, V):
    T, k = 5, 7
    z, t, at = inputs(T, V, k, kind)
    op = TopLogitDistillation(V, k, T, 2.0)
    plain = torch.empty_like(z)
    op.loss_and_gradient(z, t, at, plain)
    first = op.token_loss.clone()

    def apart(x, extra):
        whole = torch.full((x.shape[0], x.shape[1] + extra), 3.0 if x.is_floating_point() else 1, dtype=x.dtype, device=DEV)
        whole[:, 1:1 + x.shape[1]] = x
        return whole, whole[:, 1:1 + x.shape[1]]

    whole, out = apart(torch.zeros_like(z), 5)
    op.loss_and_gradient(apart(z, 3)[1], apart(t, 2)[1], apart(at, 4)[1], out)
    assert torch.equal(out, plain) and torch.equal(op.token_loss, first)
    assert (whole[:, 0] == 3).all() and (whole[:, V + 1:] == 3).all()
    whole, own = apart(z, 4)
    op.loss_and_gradient(own, t, at, own)                 # in the logits' place
    assert torch.equal(own, plain) and (whole[:, V + 1:] == 3).all()


def test_gradient_against_differences():
    """Central differences of the loss in fp32 logits, step h: off by h^2 / 6 of the third derivative (at most 1 / tau^3
    for a softmax, times tau^2) and by the loss's own error over h."""
    T, V, k, tau, h = 2, 50, 5, 1.5, 2.0 ** -6
    z, t, at = inputs(T, V, k, "fp32", spread=1.0)
    op = TopLogitDistillation(V, k, T, tau)
    d = torch.empty_like(z)
    op.loss_and_gradient(z, t, at, d)
    r = reference(z, t, at, torch.ones(T, dtype=torch.bool, device=DEV), tau, 1.0, 1.0)
    bound = h * h / 6 / tau + 2 * float(r["emean"]) / h + 2 * E32 * float(r["mean"]) / h
    for row, v in ((0, 0), (0, int(at[0, 0])), (1, int(at[1, 3])), (1, 49)):
        e = torch.zeros_like(z)
        e[row, v] = h
        up, down = (float(op.loss(z + s * e, t, at)) for s in (1, -1))
        # z +- h is rounded: by half a unit of 8 at most
        assert abs((up - down) / (2 * h) - float(d[row, v])) <= bound + 8 * E32 / h


def test_bits_do_not_depend_on_the_launch_shape(monkeypatch):
    z, t, at = inputs(40, 3001, 30, "bf16")
    op = TopLogitDistillation(3001, 30, 40, 2.0)
    first = torch.empty_like(z)
    op.loss_and_gradient(z, t, at, first)
    loss = op.value.clone()
    for blocks in ("1", "7"):
        monkeypatch.setenv("DSZERO_GRID", blocks)
        again = torch.empty_like(z)
        op.loss_and_gradient(z, t, at, again)
        assert torch.equal(first, again) and torch.equal(loss, op.value)


def test_in_graphs_that_share_a_workspace():
    """Two captured calls of one object, replayed in turn with eager calls between, and new values at the same address."""
    T, V, k = 64, 4000, 16
    z, t, at = inputs(T, V, k, "fp16")
    op = TopLogitDistillation(V, k, T, 1.0)
    out = [torch.empty_like(z) for _ in range(3)]
    mask = torch.ones(T, dtype=torch.bool, device=DEV)
    st = state(256.0)
    op.loss_and_gradient(z, t, at, out[2], mask=mask, scaler=st)
    torch.cuda.synchronize()
    graphs = []
    for n in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[n]):
            op.loss_and_gradient(z, t, at, out[n], mask=mask if n else None, scaler=st)
    for seed in range(1, 4):
        z.copy_(inputs(T, V, k, "fp16", seed=seed)[0])
        mask.copy_(torch.rand(T, generator=generator(seed), device=DEV) < 0.5)
        for n in (0, 1, 1, 0):
            out[n].zero_()
            graphs[n].replay()
            torch.cuda.synchronize()
            got = op.value.clone(), int(op.used)
            op.loss_and_gradient(z, t, at, out[2], mask=mask if n else None, scaler=st)
            assert torch.equal(out[2], out[n]) and torch.equal(got[0], op.value) and got[1] == int(op.used)


def test_sizes_in_turn_and_no_tokens():
    V, k = 1000, 8
    op = TopLogitDistillation(V, k, 300, 1.0)
    for T in (300, 1, 0, 17, 300, 2):
        z, t, at = inputs(max(T, 1), V, k, "bf16", seed=T)
        check(op, z[:T], t[:T], at[:T])
    assert int(op.used) == 2


def test_many_rows():
    """More rows than a grid's blocks hold at once, past 2^31 values."""
    T, V, k = 70001, 32000, 4
    z = torch.zeros(T, V, dtype=torch.bfloat16, device=DEV)
    z[:, 5] = 1.0
    t = torch.zeros(T, k, device=DEV)
    at = torch.tensor([5, 6, 7, 31999], dtype=torch.int32, device=DEV).repeat(T, 1)
    op = TopLogitDistillation(V, k, T, 1.0)
    op.loss_and_gradient(z, t, at, z)
    r = reference(torch.cat([torch.zeros(1, 5, device=DEV), torch.ones(1, 1, device=DEV), torch.zeros(1, V - 6, device=DEV)],
                            1), t[:1], at[:1], torch.ones(1, dtype=torch.bool, device=DEV), 1.0, 1.0, 1.0)
    assert torch.equal(op.token_loss, op.token_loss[:1].expand(T))
    close(op.token_loss[:1], r["loss"], r["eloss"])
    close(z[-1:], r["d"] / T, r["ed"] / T)
    assert torch.equal(z[0], z[-1]) and torch.equal(z[0], z[T // 2])
    del z
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind,T,V,tau", [("bf16", 2, 32000, 1.0), ("fp16", 200, 32000, 2.0), ("fp32", 256, 50021, 1.5),
                                          ("bf16", 64, 200003, 1.0), ("fp16", 257, 3001, 1.0)])
def test_few_rows_in_place_beside_rows_of_nothing(kind, T, V, tau):
    """In the logits' place, rows of nothing but -infinity (the last among them) are not used, however the blocks run: the
    bits of a call that writes elsewhere, and those within the bounds; the workspace serves the calls after it."""
    k = 8
    z, t, at = inputs(T, V, k, kind)
    z[::3] = -INF
    z[-1] = -INF
    z[1:-1:5, :V - 1] = -INF                              # used for their last logit alone, if not for less
    at[1:-1:5] = -1
    at[1:-1:5, 0] = V - 1
    op = TopLogitDistillation(V, k, 600, tau, coef=0.5)
    plain, st = torch.empty_like(z), state(64.0)
    op.loss_and_gradient(z, t, at, plain, scaler=st)
    want = op.value.clone(), op.used.clone(), op.token_loss[:T].clone()
    assert int(op.used) == int((z > -INF).any(1).sum())
    for _ in range(3):
        own = z.clone()
        op.loss_and_gradient(own, t, at, own, scaler=st)
        assert torch.equal(own, plain)
        for a, b in zip((op.value, op.used, op.token_loss[:T]), want):
            assert torch.equal(a, b)
    check(op, z.clone(), t, at, scale=64.0)
    r = check(op, own.copy_(z), t, at, scale=64.0, out=own)
    assert not r["used"][::3].any() and not own[::3].any()
    check(op, *inputs(600, V, k, kind)) if V < 4000 else None


def test_few_rows_in_place_in_a_graph_and_with_more_blocks_than_rows(monkeypatch):
    V, k = 5000, 6
    for T in (1, 5):
        z, t, at = inputs(T, V, k, "bf16")
        if T > 1:
            z[::2] = -INF
        op = TopLogitDistillation(V, k, T, 1.0)
        plain, own = torch.empty_like(z), z.clone()
        op.loss_and_gradient(z, t, at, plain)
        want = op.value.clone(), op.used.clone()
        for blocks in ("1", "7"):
            monkeypatch.setenv("DSZERO_GRID", blocks)
            own.copy_(z)
            op.loss_and_gradient(own, t, at, own)
            assert torch.equal(own, plain) and torch.equal(op.value, want[0]) and torch.equal(op.used, want[1])
        monkeypatch.delenv("DSZERO_GRID")
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            op.loss_and_gradient(own, t, at, own)
        for _ in range(3):
            own.copy_(z)
            op.value.fill_(-1.0)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(own, plain) and torch.equal(op.value, want[0]) and torch.equal(op.used, want[1])
            own.copy_(z)
            op.loss_and_gradient(own, t, at, own)
            assert torch.equal(own, plain) and torch.equal(op.value, want[0])


@pytest.mark.parametrize("kind", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("T,V,k,each", [(5001, 4096, 300, 2), (5001, 4096, 200, 2), (7001, 2100, 700, 3), (3001, 33000, 600, 2)])
def test_long_lists_between_rows_that_are_left_out(T, V, k, each, kind):
    """Blocks that go over several rows, some of them left out between two that are used, with entries in many waves: every
    other place is one of 20, so that most entries share theirs."""
    z, t, at = inputs(T, V, k, kind)
    gen = generator(11)
    at[:, ::2] = torch.randint(0, 20, (T, (k + 1) // 2), generator=gen, device=DEV, dtype=at.dtype)
    mask = (torch.arange(T, device=DEV) % each != 1) & (torch.rand(T, generator=gen, device=DEV) < 0.8)
    op = TopLogitDistillation(V, k, T, 2.0)
    for accumulate in (False, True):
        check(op, z, t, at, mask=mask, scale=256.0, accumulate=accumulate,
              out=torch.randn(T, V, generator=gen, device=DEV).mul_(1e-3).to(z.dtype))


def test_alternating_rows_of_one_block(monkeypatch):
    """One block for all rows, the used ones two apart."""
    monkeypatch.setenv("DSZERO_GRID", "1")
    for T, V, k in ((61, 4096, 300), (61, 9000, 1000), (40, 32000, 700)):
        z, t, at = inputs(T, V, k, "bf16")
        at[:, 1::2] = at[:, :1]
        mask = torch.arange(T, device=DEV) % 2 == 0
        check(TopLogitDistillation(V, k, T, 1.0), z, t, at, mask=mask)
        check(TopLogitDistillation(V, k, T, 1.0), z, t, at, mask=mask, out=torch.ones_like(z), accumulate=True)
