"""Cross entropy over a large vocabulary from hidden states, and its gradients, on the GPU against the formulas in 64 bits,
with bounds counted from fp32's half unit E = 2^-24 and the 16-bit types'."""
import math

import pytest
import torch

from zero_mixed_precision_amd import VocabCrossEntropy, _lib

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E32 = 2.0 ** -24
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -149}


def generator(seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return gen


def reference(x, w, y, mask, coef, scale):
    """Values and bounds in 64 bits.  A logit is off by its length's roundings of the sum of its terms' sizes, a probability
    by that, by its exponent's three roundings, the sum's additions (a tile's in a lane and its joins, 400 at most) and the
    logarithm; dz by its rounding to 16 bits as well; a gradient's value by these, by weight, and by the roundings of its own
    sum."""
    T, V, D = x.shape[0], w.shape[0], w.shape[1]
    half = HALF[x.dtype]
    used = mask & (y >= 0)
    n = int(used.sum())
    x, w = x.double(), w.double()
    x = torch.where(used[:, None], x, 0.0)
    at = torch.where(used, y, 0).long()
    z = x @ w.t()
    ez = (D + 2) * E32 * (x.abs() @ w.abs().t())
    top = z.amax(1, keepdim=True)
    lse = torch.logsumexp(z, 1, keepdim=True)
    p = (z - lse).exp()
    far = (z - top).abs() / math.log(2) + torch.log2((z - top).exp().sum(1, keepdim=True)).clamp(min=1)
    elog = (p * (ez + 3 * far * E32)).sum(1, keepdim=True) + 400 * E32 + 4 * E32 * far.amin(1, keepdim=True)
    loss = torch.where(used, (lse - z.gather(1, at[:, None]))[:, 0], 0.0)
    eloss = (ez.gather(1, at[:, None]) + elog)[:, 0] + 6 * E32 * (lse - top)[:, 0].abs() + \
        4 * E32 * (top - z.gather(1, at[:, None]))[:, 0].abs()
    eloss = torch.where(used, eloss, 0.0)
    factor = scale * coef / max(n, 1)
    dz = p.scatter_add(1, at[:, None], torch.full((T, 1), -1.0, dtype=torch.float64, device=DEV)) * used[:, None]
    edz = (p * (ez + elog + 3 * far * E32 + 4 * E32) + 2 * E32 * dz.abs()) * used[:, None]
    edz = edz + half * (dz.abs() + edz) + 2.0 ** -39           # fp16: half a unit of 2^-24, held times 2^15
    dx, dw = dz @ w * factor, dz.t() @ x * factor
    edx = (edz @ w.abs() + (V + 4) * E32 * (dz.abs() @ w.abs())) * factor + 3 * E32 * dx.abs()
    edw = (edz.t() @ x.abs() + (T + 4) * E32 * (dz.abs().t() @ x.abs())) * factor + 3 * E32 * dw.abs()
    mean = coef * loss.sum() / max(n, 1)
    return dict(n=n, used=used, loss=loss, eloss=eloss, mean=mean,
                emean=coef * eloss.sum() / max(n, 1) + 4 * E32 * mean.abs(), dx=dx, edx=edx * used[:, None], dw=dw, edw=edw)


def close(got, want, bound):
    half, tiny = HALF[got.dtype], TINY[got.dtype]
    got = got.double()
    tol = bound + half * (want.abs() + bound) + tiny
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, by up to {float((got - want).abs().max())}"


def near(got, want):
    """The whole error, relative: what random roundings of dz and of the result leave (a unit of each, divided by sqrt(3),
    together 0.82 half units) with a factor of two."""
    if float(want.norm()):
        assert float((got.double() - want).norm() / want.norm()) <= 2 * 0.82 * HALF[torch.bfloat16 if got.dtype == torch.float32
                                                                                    else got.dtype]


def state(scale):
    st = torch.zeros(_lib.ds_scaler_size(), dtype=torch.uint8, device=DEV)
    _lib.ds_state_init(st, scale, 1.0, 1000, 1, 0, 0)
    return st


def check(op, x, w, y, mask=None, scale=None, dw=None, accumulate=False, dtype=None):
    T = x.shape[0]
    r = reference(x, w, y, torch.ones(T, dtype=torch.bool, device=DEV) if mask is None else mask != 0, op.coef, scale or 1.0)
    op.loss(x, w, y, mask=mask)
    alone = op.token_loss[:T].clone(), op.value.clone()
    dx = torch.full((T, w.shape[1]), 7.0, dtype=x.dtype, device=DEV)
    if dw is None:
        dw = torch.full(w.shape, 7.0, dtype=dtype or w.dtype, device=DEV)
    base = dw.double().clone()
    op.loss_and_gradient(x, w, y, dx, dw, mask=mask, scaler=None if scale is None else state(scale), accumulate=accumulate)
    assert int(op.used) == r["n"]
    for a, b in ((alone[0], op.token_loss[:T]), (alone[1], op.value)):
        assert torch.equal(a, b)
    close(op.token_loss[:T], r["loss"], r["eloss"])
    close(op.value, r["mean"], r["emean"])
    close(dx, r["dx"], r["edx"])
    assert not dx[~r["used"]].any()
    if accumulate:
        close(dw, base + r["dw"], r["edw"] + E32 * (base + r["dw"]).abs())
    else:
        close(dw, r["dw"], r["edw"])
        near(dw, r["dw"])
    near(dx, r["dx"])
    return r


def inputs(T, V, D, kind, seed=0, index=torch.int64):
    gen = generator(seed)
    w = (torch.randn(V, D, generator=gen, device=DEV) * 2 * D ** -0.5).to(TYPES[kind])
    y = torch.randint(V, (T,), generator=gen, device=DEV)
    knows = (torch.rand(T, 1, generator=gen, device=DEV) < 0.5) * 1.0
    x = (torch.randn(T, D, generator=gen, device=DEV) + knows * w[y].float()).to(TYPES[kind])
    return x, w, y.to(index)


SIZES = [(1, 1, 1), (1, 2, 64), (2, 16, 8), (16, 1000, 64), (5, 129, 63), (64, 128, 128), (65, 257, 65), (127, 255, 192),
         (128, 256, 256), (129, 300, 250), (200, 5000, 100), (1, 32000, 512), (33, 10007, 333), (300, 513, 1000),
         (513, 777, 520), (1000, 2000, 40), (2, 70001, 24), (700, 1024, 2048),
         # sums split into parts: over the vocabulary, over the tokens, over both and over pieces
         (3, 20000, 40), (3000, 20, 10), (2500, 9000, 33), (130, 65537, 64), (2049, 300, 16), (4100, 129, 200)]


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("T,V,D", SIZES)
def test_against_64_bits(T, V, D, kind):
    x, w, y = inputs(T, V, D, kind)
    op = VocabCrossEntropy(V, D, T, TYPES[kind])
    check(op, x, w, y)
    check(VocabCrossEntropy(V, D, T + 100, TYPES[kind], coef=0.25), x, w, y.int(), scale=512.0)


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("T,V,D", [(100, 300, 64), (257, 1000, 100), (900, 640, 256)])
def test_rows_that_are_left_out(T, V, D, kind):
    x, w, y = inputs(T, V, D, kind)
    gen = generator(4)
    mask = torch.rand(T, generator=gen, device=DEV) < 0.6
    y = torch.where(torch.rand(T, generator=gen, device=DEV) < 0.2, -100, y)
    x[~mask] = math.nan                                   # padding may hold anything
    x[(y < 0) & mask] = math.inf
    op = VocabCrossEntropy(V, D, T, TYPES[kind])
    r = check(op, x, w, y, mask=mask, scale=64.0)
    assert 0 < r["n"] < T
    check(op, x, w, y, mask=mask.to(torch.uint8) * 3)
    r = check(op, x, w, torch.full_like(y, -1), mask=mask)
    assert r["n"] == 0 and float(op.value) == 0.0
    one = torch.full_like(y, -1)
    one[T // 2] = V - 1
    x[T // 2] = 1.0
    check(op, x, w, one)


@pytest.mark.parametrize("kind,dtype", [("fp16", torch.float32), ("bf16", torch.float32), ("bf16", torch.bfloat16),
                                        ("fp16", torch.float16)])
@pytest.mark.parametrize("T,V,D", [(130, 700, 200), (3000, 20, 10)])
def test_weight_gradients_add_up(T, V, D, kind, dtype):
    op = VocabCrossEntropy(V, D, T, TYPES[kind])
    x, w, y = inputs(T, V, D, kind)
    check(op, x, w, y, dtype=dtype)
    dw = torch.randn(V, D, generator=generator(8), device=DEV).mul_(1e-2).to(dtype)
    for seed in (1, 2):
        x, _, y = inputs(T, V, D, kind, seed=seed)
        check(op, x, w, y, dw=dw, accumulate=True)
    before = dw.clone()
    op.loss_and_gradient(x, w, torch.full_like(y, -1), torch.empty_like(x), dw, accumulate=True)
    assert torch.equal(before, dw)                        # nothing used: nothing added


def test_one_gradient_alone():
    T, V, D = 70, 400, 96
    x, w, y = inputs(T, V, D, "bf16")
    op = VocabCrossEntropy(V, D, T, torch.bfloat16)
    dx, dw, dx2, dw2 = (torch.empty_like(a) for a in (x, w, x, w))
    op.loss_and_gradient(x, w, y, dx, dw)
    op.loss_and_gradient(x, w, y, dx2, None)
    op.loss_and_gradient(x, w, y, None, dw2)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.parametrize("T,V,D", [(40, 500, 64), (40, 500, 128), (150, 300, 100)])
def test_strides(T, V, D):
    """Rows a distance apart, starting off 16 bytes, with NaN between them, give the bits of packed ones."""
    x, w, y = inputs(T, V, D, "bf16")
    op = VocabCrossEntropy(V, D, T, torch.bfloat16)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    op.loss_and_gradient(x, w, y, dx, dw)
    loss = op.token_loss.clone()

    for left, right in ((0, 8), (1, 2), (8, 64)):
        def apart(a, value=math.nan):
            whole = torch.full((a.shape[0], left + a.shape[1] + right), value, dtype=a.dtype, device=DEV)
            whole[:, left:left + a.shape[1]] = a
            return whole, whole[:, left:left + a.shape[1]]

        (hx, ox), (hw, ow) = apart(torch.zeros_like(x), 3.0), apart(torch.zeros_like(w), 3.0)
        op.loss_and_gradient(apart(x)[1], apart(w)[1], y, ox, ow)
        assert torch.equal(ox, dx) and torch.equal(ow, dw) and torch.equal(op.token_loss, loss)
        for h in (hx, hw):
            assert (h[:, :left] == 3).all() and (h[:, left + D:] == 3).all()


def test_targets_past_the_vocabulary_are_nan():
    T, V, D = 20, 300, 64
    x, w, y = inputs(T, V, D, "bf16")
    y[7] = V
    y[9] = 2 ** 40
    op = VocabCrossEntropy(V, D, T, torch.bfloat16)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    assert math.isnan(float(op.loss_and_gradient(x, w, y, dx, dw)))
    bad = torch.zeros(T, dtype=torch.bool, device=DEV)
    bad[7] = bad[9] = True
    assert torch.equal(torch.isnan(op.token_loss), bad) and torch.equal(torch.isnan(dx).any(1), bad)
    assert torch.isnan(dw).all() and int(op.used) == T


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
def test_large_logits(kind):
    """Logits in the thousands: the target has all the probability, or none."""
    T, V, D = 64, 512, 64
    x, w, y = inputs(T, V, D, kind)
    x = (x.float() * 200).to(x.dtype)
    check(VocabCrossEntropy(V, D, T, TYPES[kind]), x, w, y)


def test_pieces_of_the_vocabulary():
    """More tokens than one piece of the whole vocabulary has room for: sums over several pieces, the last one short."""
    T, V, D = 120000, 5003, 64
    x, w, y = inputs(T, V, D, "bf16")
    op = VocabCrossEntropy(V, D, T, torch.bfloat16)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    op.loss_and_gradient(x, w, y, dx, dw)
    assert op._ws_bytes < 2 * T * V + 40 * T * 128
    few = slice(T - 500, T)                               # rows of the gradient, by themselves
    r = reference(x[few], w, y[few], torch.ones(500, dtype=torch.bool, device=DEV), 1.0, 500.0 / T)
    close(op.token_loss[few], r["loss"], r["eloss"])
    close(dx[few], r["dx"], r["edx"])
    want, mean = torch.zeros(V, D, dtype=torch.float64, device=DEV), 0.0
    for lo in range(0, T, 20000):
        r = reference(x[lo:lo + 20000], w, y[lo:lo + 20000], torch.ones(20000, dtype=torch.bool, device=DEV), 1.0, 20000 / T)
        want += r["dw"]
        mean += float(r["mean"]) * 20000 / T
    near(dw, want)
    assert abs(float(op.value) - mean) <= 1e-5 * mean     # 400 + 66 roundings of each row's loss, of size 10 at most


def test_gradient_against_differences():
    """Differences of the loss over steps of h in one value of x or w that 16 bits hold exactly; the second order's error
    is at most the largest |x|, |w| squared times h over the rows' number, for a softmax."""
    T, V, D, h = 4, 40, 16, 2.0 ** -6
    gen = generator(1)
    x = torch.randint(-16, 17, (T, D), generator=gen, device=DEV).div(16).half()       # multiples of 1/16 up to 1
    w = torch.randint(-16, 17, (V, D), generator=gen, device=DEV).div(16).half()
    y = torch.randint(V, (T,), generator=gen, device=DEV)
    op = VocabCrossEntropy(V, D, T, torch.float16)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    op.loss_and_gradient(x, w, y, dx, dw)
    r = reference(x, w, y, torch.ones(T, dtype=torch.bool, device=DEV), 1.0, 1.0)
    for a, d, e, at in ((x, dx, r["edx"], (1, 3)), (x, dx, r["edx"], (3, 15)), (w, dw, r["edw"], (0, 0)),
                        (w, dw, r["edw"], (int(y[2]), 5))):
        moved = []
        for s in (h, -h):
            b = a.clone()
            b[at] += s
            assert float(b[at] - a[at]) == s
            moved.append(float(op.loss(b if a is x else x, b if a is w else w, y)))
        bound = h * h / 6 * 2 + 2 * float(r["emean"]) / h + float(e[at]) + 2.0 ** -11 * abs(float(d[at])) + 2.0 ** -25
        assert abs((moved[0] - moved[1]) / (2 * h) - float(d[at])) <= bound


@pytest.mark.parametrize("V,D,sizes", [(300, 72, (260, 1, 0, 17, 259)), (40000, 24, (9000, 2, 300, 2100))])
def test_sizes_in_turn_and_no_tokens(V, D, sizes):
    op = VocabCrossEntropy(V, D, max(sizes), torch.float16)
    for T in sizes:
        x, w, y = inputs(max(T, 1), V, D, "fp16", seed=T)
        check(op, x[:T], w, y[:T])


def test_bits_do_not_change_and_garbage_in_the_workspace_reaches_nothing():
    T, V, D = 150, 900, 130
    x, w, y = inputs(T, V, D, "bf16")
    op = VocabCrossEntropy(V, D, T, torch.bfloat16)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    op.loss_and_gradient(x, w, y, dx, dw)
    first = [a.clone() for a in (dx, dw, op.token_loss, op.value)]
    for byte in (0, 255, 0x7F):                           # 255 and 0x7F: NaN in every type
        op._ws.fill_(byte)
        op.loss_and_gradient(x, w, y, dx, dw)
        for a, b in zip(first, (dx, dw, op.token_loss, op.value)):
            assert torch.equal(a, b)


def test_in_a_graph_and_on_a_stream():
    T, V, D = 200, 1500, 128
    x, w, y = inputs(T, V, D, "bf16")
    side, st = torch.cuda.Stream(), state(4.0)
    for stream in (None, side):
        op = VocabCrossEntropy(V, D, T, torch.bfloat16, stream=stream)
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            op.loss_and_gradient(x, w, y, dx, dw, scaler=st)
        for seed in (1, 2, 3):
            nx, _, ny = inputs(T, V, D, "bf16", seed=seed)
            x.copy_(nx)
            y.copy_(torch.where(torch.arange(T, device=DEV) % (seed + 1) == 0, -1, ny))
            dx.zero_(), dw.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            got = [a.clone() for a in (dx, dw, op.value, op.used)]
            op.loss_and_gradient(x, w, y, dx, dw, scaler=st)
            torch.cuda.synchronize()
            for a, b in zip(got, (dx, dw, op.value, op.used)):
                assert torch.equal(a, b)


@pytest.mark.parametrize("kind,T,V,D", [("bf16", 2048, 8000, 1024), ("fp16", 1500, 4099, 515), ("bf16", 256, 32000, 2048)])
def test_larger_products(kind, T, V, D):
    x, w, y = inputs(T, V, D, kind)
    check(VocabCrossEntropy(V, D, T, TYPES[kind]), x, w, y, scale=16.0)


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("D", [8, 64, 72, 136, 200])
def test_many_rows_of_few_values(D, kind):
    """The largest tiles, over one to four steps of 64 values."""
    T, V = 4096, 8192
    x, w, y = inputs(T, V, D, kind)
    check(VocabCrossEntropy(V, D, T, TYPES[kind]), x, w, y)


@pytest.mark.parametrize("kind,T,V,D", [("bf16", 2041, 7993, 1024), ("fp16", 2041, 7993, 1003), ("bf16", 3000, 7993, 1024),
                                        ("fp16", 1999, 10007, 2048), ("bf16", 1021, 50021, 1003)])
def test_the_largest_tiles_with_a_short_last_step(kind, T, V, D):
    """Tiles of 256 x 256 for both gradients, over a vocabulary and used tokens that end inside a step of 64; W read in
    place and packed."""
    x, w, y = inputs(T, V, D, kind)
    mask = torch.rand(T, generator=generator(2), device=DEV) < 0.97
    mask[-1] = True
    y[:5] = V - 1                                         # the last step's own columns
    while int(mask.sum()) % 64 == 0:
        mask[int(torch.nonzero(mask)[0])] = False
    check(VocabCrossEntropy(V, D, T, TYPES[kind]), x, w, y, mask=mask, scale=16.0)
    x[~mask] = math.nan
    check(VocabCrossEntropy(V, D, T, TYPES[kind]), x, w, y, mask=mask, dtype=torch.float32)


@pytest.mark.parametrize("kind,T,V,D", [("fp16", 16, 1000, 64), ("bf16", 1021, 50021, 1003), ("fp16", 4096, 32000, 512),
                                        ("bf16", 4096, 8192, 1024)])
def test_a_call_repeats_its_bits(kind, T, V, D):
    """Each of the three sides of tiles, with other work on the GPU between the calls."""
    x, w, y = inputs(T, V, D, kind)
    op = VocabCrossEntropy(V, D, T, TYPES[kind])
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    first = None
    for turn in range(4):
        op.loss_and_gradient(x, w, y, dx, dw)
        got = [a.clone() for a in (dx, dw, op.token_loss, op.value)]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))
        x.float() @ x.float()[:turn + 1].t()
