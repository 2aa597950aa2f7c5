"""The balance loss and its gradient on the GPU against the formulas in 64 bits, with bounds counted from fp32's half
unit E = 2^-24 and the output type's."""
import numpy as np
import pytest
import torch

from zero_mixed_precision_amd import ExpertBalance, _lib

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E32 = 2.0 ** -24
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
TINY = {"fp16": 2.0 ** -25, "bf16": 2.0 ** -134, "fp32": 2.0 ** -148}


def reference(z, mask, k, coef, scale=1.0):
    """Values and error bounds in 64 bits (z: float64 array, mask: bool array)."""
    T, n = z.shape
    nan = np.isnan(z).any(1) | np.isposinf(z).any(1)
    used = mask & ~np.isneginf(z).all(1)
    fine = used & ~nan
    counts = np.zeros(n, np.int64)
    order = np.argsort(-np.where(fine[:, None], z, 0.0), axis=1, kind="stable")[:, :k]
    for t in np.flatnonzero(fine):
        for e in order[t]:
            counts[e] += z[t, e] > -np.inf
    p, rel = np.zeros((T, n)), np.zeros((T, n))
    with np.errstate(invalid="ignore"):
        x = z - np.where(fine, z.max(1, initial=-np.inf), 0.0)[:, None]
        ex = np.exp(x)
        p[fine] = (ex / ex.sum(1, keepdims=True))[fine]
    p[used & nan] = np.nan
    far = np.where(p > 0, np.abs(np.where(np.isfinite(x), x, 0.0)), 0.0)
    # exp of a rounded difference times a rounded constant (3 |x|), the instruction (2); the sum's terms the same by
    # weight, its additions (36 at most); the reciprocal and the product (2)
    rel = (3 * far + 2 + np.nansum(p * (3 * far + 2), axis=1, keepdims=True) + 36 + 2) * E32
    rows = int(used.sum())
    some = max(rows, 1)
    f = counts / (some * k)
    mean = p[used].sum(0) / some if rows else np.zeros(n)
    loss = coef * n * float(f @ mean)
    # a lane adds its rows of the block (32 rows a turn for 8 lanes a row, 512 blocks at most), then 10 more sums
    adds = -(-T // min(512, max(1, -(-T // 16))) // 16) + 12
    emean = (p * rel)[used].sum(0) / some + (adds + 2) * E32 * mean if rows else np.zeros(n)
    factor = scale * coef * n / some if rows else 0.0
    g = f - counts.sum() / (n * some * k)                # as the kernel takes it: less its mean
    dot = np.nansum(p * g, axis=1, keepdims=True)
    d = factor * p * (g - dot)
    edot = np.nansum(p * np.abs(g) * (rel + 40 * E32), axis=1, keepdims=True)
    ed = factor * (p * rel * np.abs(g - dot) + p * (edot + 3 * E32 * (np.abs(g) + np.abs(dot)))) + 4 * E32 * np.abs(d)
    d[~used] = 0.0
    ed[~used] = 0.0
    d[used & nan] = np.nan
    eloss = coef * n * float(f @ emean) + 4 * E32 * abs(loss)
    return dict(counts=counts, used=rows, mean=mean, emean=emean, loss=loss, eloss=eloss, d=d, ed=ed, rows=used)


def check(op, z, kind, mask=None, scaler=None, scale=1.0, out=None, accumulate=False):
    base = out.double().cpu().numpy() if accumulate else 0.0
    out = torch.full_like(z, 7.0) if out is None else out
    value = op.loss(z, mask=mask)
    assert op.gradient(z, out, mask=mask, scaler=scaler, accumulate=accumulate) is out
    m = np.ones(z.shape[0], bool) if mask is None else mask.cpu().numpy() != 0
    r = reference(z.double().cpu().numpy(), m, op.k, float(np.float32(op.coef)), scale)
    assert int(op.used) == r["used"]
    np.testing.assert_array_equal(op.counts.cpu().numpy(), r["counts"])
    mean = op.mean_prob.double().cpu().numpy()
    np.testing.assert_array_equal(np.isnan(mean), np.isnan(r["mean"]))
    ok = ~np.isnan(mean)
    assert np.all(np.abs(mean - r["mean"])[ok] <= r["emean"][ok] + 2.0 ** -149)
    v = float(value)
    assert np.isnan(v) == np.isnan(r["loss"]) and (np.isnan(v) or abs(v - r["loss"]) <= r["eloss"] + 2.0 ** -149)
    d = out.double().cpu().numpy()
    np.testing.assert_array_equal(np.isnan(d), np.isnan(r["d"]))
    with np.errstate(invalid="ignore"):
        want = np.where(r["rows"][:, None], base + r["d"], base)
        tol = r["ed"] + HALF[kind] * (np.abs(want) + r["ed"]) + TINY[kind] + (E32 * np.abs(want) if accumulate else 0)
        bad = ~(np.abs(d - want) <= tol) & ~np.isnan(d)
    assert not bad.any(), f"{bad.sum()} gradients off, by {np.nanmax(np.abs(d - want))}"
    if accumulate:   # rows that are not used are left as they were, bit for bit
        np.testing.assert_array_equal(d[~r["rows"]], base[~r["rows"]])
    return r


def logits(T, n, kind, seed=0, levels=None):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    z = torch.randn(T, n, generator=gen, device=DEV) * 1.5 + torch.randn(n, generator=gen, device=DEV)
    if levels:
        z = (z * levels).round() / levels       # many equal values
    return z.to(TYPES[kind])


@pytest.mark.parametrize("kind", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("T,n,k", [(1, 1, 1), (1, 2, 1), (1, 8, 2), (2, 3, 3), (7, 8, 8), (31, 31, 5), (33, 32, 16),
                                   (100, 33, 1), (65, 60, 4), (257, 64, 8), (130, 65, 9), (1000, 128, 8), (99, 129, 2),
                                   (300, 200, 16), (515, 256, 8), (77, 257, 3), (200, 384, 10), (64, 512, 16),
                                   (20000, 16, 2), (17000, 300, 8)])
def test_against_64_bits(T, n, k, kind):
    z = logits(T, n, kind)
    op = ExpertBalance(n, k, 0.01)
    check(op, z, kind)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    check(op, z, kind, mask=torch.rand(T, generator=gen, device=DEV) < 0.7)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("n,k", [(8, 2), (64, 8), (100, 5), (256, 8), (512, 16)])
def test_ties_go_to_the_lowest_index(n, k, kind):
    check(ExpertBalance(n, k, 1.0), logits(500, n, kind, levels=2), kind)
    r = check(ExpertBalance(n, k, 1.0), torch.zeros(50, n, dtype=TYPES[kind], device=DEV), kind)
    assert list(r["counts"]) == [50] * k + [0] * (n - k)
    # -0 and 0 are equal
    z = torch.zeros(50, n, dtype=TYPES[kind], device=DEV)
    z[:, :k] = -0.0
    check(ExpertBalance(n, k, 1.0), z, kind)


@pytest.mark.parametrize("kind", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("n,k", [(8, 3), (60, 4), (256, 8)])
def test_masked_experts_empty_rows_and_extremes(n, k, kind):
    """-infinity and the type's lowest value in logits; rows with fewer than k experts, with none, and masked ones that
    hold NaN and infinities."""
    z = logits(200, n, kind, seed=4)
    z[:, 1] = float("-inf")
    z[3] = float("-inf")                         # empty
    z[4] = float("-inf")
    z[4, n - 1] = -5.0                           # one expert left
    z[5, 2:] = float("-inf")
    z[6, 3:] = torch.finfo(z.dtype).min
    z[7] = torch.finfo(z.dtype).min
    z[8] = torch.finfo(z.dtype).max
    z[9, 0] = torch.finfo(z.dtype).max           # all probability at one
    mask = torch.ones(200, dtype=torch.uint8, device=DEV)
    mask[10:14] = 0
    z[10], z[11], z[12, 3] = float("nan"), float("inf"), float("-inf")
    r = check(ExpertBalance(n, k, 0.5), z, kind, mask=mask)
    assert r["used"] == 195 and r["counts"][1] == 2      # in rows 7 and 8, where all are equal
    check(ExpertBalance(n, k, 0.5), z, kind, mask=mask.bool())


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_spoiled_row_shows_and_keeps_to_itself(value):
    z = logits(100, 64, "fp32")
    z[40, 17] = value
    z[41] = value
    op = ExpertBalance(64, 4, 0.1)
    r = check(op, z, "fp32")
    assert np.isnan(r["loss"]) and r["used"] == 100 and r["counts"].sum() == 98 * 4


@pytest.mark.parametrize("case", ["no tokens", "all masked", "all empty"])
def test_nothing_used(case):
    op = ExpertBalance(16, 2, 0.1)
    op.loss(logits(50, 16, "bf16"))              # leaves values that must be overwritten
    T = 0 if case == "no tokens" else 33
    z = logits(T, 16, "bf16") if case != "all empty" else torch.full((T, 16), float("-inf"), device=DEV).bfloat16()
    mask = torch.zeros(T, dtype=torch.bool, device=DEV) if case == "all masked" else None
    check(op, z, "bf16", mask=mask)
    assert float(op.value) == 0 and int(op.used) == 0 and float(op.mean_prob.abs().sum()) == 0


@pytest.mark.parametrize("kind", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("n,shift,gap", [(64, 0, 8), (64, 1, 0), (60, 2, 5), (33, 3, 1), (256, 4, 4)])
def test_rows_apart_and_offset(n, shift, gap, kind):
    """Logits and gradients as columns of wider matrices, at any offset; what lies between stays as it is."""
    wide = torch.full((90, n + gap + shift), 3.0, device=DEV).to(TYPES[kind])
    z = wide[:, shift:shift + n]
    z.copy_(logits(90, n, kind))
    room = torch.full((90, n + gap + shift + 3), 9.0, device=DEV).to(TYPES[kind])
    out = room[:, shift:shift + n]
    check(ExpertBalance(n, 3, 0.1), z, kind, out=out)
    assert float(room[:, :shift].float().sum()) == 9.0 * 90 * shift
    assert float(room[:, shift + n:].float().sum()) == 9.0 * 90 * (gap + 3)


@pytest.mark.parametrize("kind", ["fp16", "bf16", "fp32"])
def test_scale_and_accumulation(kind):
    """The device's loss scale multiplies the gradient; accumulation adds it to what is there."""
    st = torch.zeros(_lib.ds_scaler_size(), dtype=torch.uint8, device=DEV)
    _lib.ds_state_init(st, 4096.0, 1.0, 1000, 1)
    z = logits(300, 60, kind)
    mask = torch.ones(300, dtype=torch.uint8, device=DEV)
    mask[::7] = 0
    out = (logits(300, 60, kind, seed=9).float() * 0.01).to(TYPES[kind])
    check(ExpertBalance(60, 4, 0.02), z, kind, mask=mask, scaler=st, scale=4096.0)
    check(ExpertBalance(60, 4, 0.02), z, kind, mask=mask, scaler=st, scale=4096.0, out=out, accumulate=True)


def test_even_counts_have_no_gradient():
    """All experts chosen by every token: f is even and the gradient 0 exactly."""
    z = logits(64, 8, "fp32")
    op = ExpertBalance(8, 8, 1.0)
    op.loss(z)
    assert float(op.gradient(z, torch.empty_like(z)).abs().max()) == 0.0


def test_gradient_against_differences():
    """Central differences of the loss in 64 bits with f held, and of the kernel's own loss along the gradient."""
    z = logits(40, 12, "fp32", seed=2)
    op = ExpertBalance(12, 3, 1.0)
    v0 = float(op.loss(z))
    d = op.gradient(z, torch.empty_like(z)).double().cpu().numpy()
    f = op.counts.double().cpu().numpy() / (40 * 3)
    z64 = z.double().cpu().numpy()

    def loss(x):
        e = np.exp(x - x.max(1, keepdims=True))
        return 12 * float(f @ (e / e.sum(1, keepdims=True)).mean(0))

    assert abs(loss(z64) - v0) <= 1e-6
    h = 1e-5   # truncation h^2 / 6 of third derivatives (below 1) and rounding 1e-16 / h, against values near 1e-3
    for t, e in ((0, 0), (7, 11), (39, 5), (20, 3)):
        up, down = z64.copy(), z64.copy()
        up[t, e] += h
        down[t, e] -= h
        assert abs((loss(up) - loss(down)) / (2 * h) - d[t, e]) <= 1e-9 + 1e-5 * abs(d[t, e])


def test_the_same_bits_again_and_on_another_stream():
    z = logits(5000, 100, "bf16")
    side = torch.cuda.Stream()
    ops = [ExpertBalance(100, 6, 0.1), ExpertBalance(100, 6, 0.1, stream=side)]
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for op in ops:
        d = torch.empty_like(z)
        for _ in range(2):
            op.loss(z)
            op.gradient(z, d)
        torch.cuda.synchronize()
        outs.append((op.value.clone(), op.counts.clone(), op.mean_prob.clone(), d))
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_graph_replays():
    z = logits(3000, 64, "bf16")
    op, eager = ExpertBalance(64, 4, 0.1), ExpertBalance(64, 4, 0.1)
    d, de = torch.empty_like(z), torch.empty_like(z)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op.loss(z)
        op.gradient(z, d)
    for k in range(4):
        z.copy_(logits(3000, 64, "bf16", seed=k))
        torch.cuda.synchronize()
        graph.replay()
        eager.loss(z)
        eager.gradient(z, de)
        torch.cuda.synchronize()
        assert torch.equal(d, de) and torch.equal(op.value, eager.value) and torch.equal(op.counts, eager.counts)


def test_offsets_past_32_bits():
    """More than 2^31 logits: the first and the last rows against a short call of the same rows."""
    T, n = (1 << 23) + 5, 264
    z = torch.zeros(T, n, dtype=torch.bfloat16, device=DEV)
    z[:, 0] = 1.0
    z[-3:] = logits(3, n, "bf16")
    op = ExpertBalance(n, 2, 1.0)
    op.loss(z)
    d = op.gradient(z, torch.empty_like(z))
    want = np.zeros(n, np.int64)
    want[0] = want[1] = T - 3                    # the largest, and of the equal rest the lowest
    for row in torch.topk(z[-3:].float(), 2, dim=1).indices.cpu().tolist():
        for e in row:
            want[e] += 1
    np.testing.assert_array_equal(op.counts.cpu().numpy(), want)
    f = torch.from_numpy(want).to(DEV).double() / (2 * T)
    p = torch.softmax(z[-3:].double(), 1)
    exact = n / T * p * (f - (p * f).sum(1, keepdim=True))
    # fp32 (bounded by 1000 E against the largest term) and the rounding to bf16
    assert float((d[-3:].double() - exact).abs().max()) <= (2.0 ** -8 + 1000 * E32) * float(exact.abs().max())


def test_refusals_of_the_class():
    op = ExpertBalance(8, 2, 0.1)
    z = logits(10, 8, "bf16")
    for bad in (z[:, :7], z.cpu(), z.double(), z.t().contiguous().t(), z[0], z[:1].expand(10, 8)):
        with pytest.raises(ValueError):
            op.loss(bad)
    for bad in (torch.ones(9, dtype=torch.bool, device=DEV), torch.ones(10, device=DEV),
                torch.ones(10, dtype=torch.bool)):
        with pytest.raises(ValueError):
            op.loss(z, mask=bad)
    for out in (z.float(), z[:5], torch.empty_like(z).cpu()):
        with pytest.raises(ValueError):
            op.gradient(z, out)
    with pytest.raises(_lib.DsError, match="ALIAS"):
        op.gradient(z, z)
