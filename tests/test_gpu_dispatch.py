"""Tokens sorted by expert and moved there and back, on the GPU, against the definition: whole numbers equal, values in 64
bits with bounds counted from fp32's half unit E = 2^-24 and the output type's."""
import pytest
import torch

from zero_mixed_precision_amd import ExpertDispatch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E32 = 2.0 ** -24
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -149}


def generator(seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return gen


def order(chosen, E):
    """(offsets, place, source) by the definition, on the host."""
    flat = [int(e) for e in chosen.flatten().tolist()]
    offsets, source, place = [0], [], [-1] * len(flat)
    for e in range(E):
        for p, x in enumerate(flat):
            if x == e:
                place[p] = len(source)
                source.append(p)
        offsets.append(len(source))
    return offsets, place, source + [-1] * (len(flat) - len(source))


def fast_order(chosen, E):
    flat = chosen.reshape(-1).long().cpu()
    valid = (flat >= 0) & (flat < E)
    pairs = torch.nonzero(valid).flatten()
    source = pairs[torch.sort(flat[pairs], stable=True).indices]
    place = torch.full_like(flat, -1)
    place[source] = torch.arange(len(source))
    counts = torch.bincount(flat[pairs], minlength=E)
    return ([0] + counts.cumsum(0).tolist(), place.tolist(),
            source.tolist() + [-1] * (len(flat) - len(source)))


def check_sort(op, chosen):
    T = chosen.shape[0]
    op.sort(chosen)
    want = order(chosen, op.E) if chosen.numel() * op.E < 200000 else fast_order(chosen, op.E)
    assert op.offsets.tolist() == want[0]
    assert op.place[:T].flatten().tolist() == want[1]
    assert op.source[:T * op.k].tolist() == want[2]


def close(got, want, bound):
    """|got - want| within the bound before rounding, half a step of the output's type, and half its smallest number."""
    got, half, tiny = got.double(), HALF[got.dtype], TINY[got.dtype]
    tol = bound + half * (want.abs() + bound) + tiny
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, by up to {float((got - want).abs().max())}"


def check_moves(op, chosen, width, kind, gkind, seed=0, pad=0):
    """All four moves after sort(); ``pad``: values between the rows of every matrix."""
    dtype, gtype, gen = TYPES[kind], TYPES[gkind], generator(seed)
    T, k = chosen.shape
    P = T * k

    def matrix(rows, columns=width, to=dtype):
        whole = torch.randn(rows, columns + pad, generator=gen, device=DEV).to(to)
        return whole, whole[:, :columns]

    x, rows, dout, dsorted = (matrix(n)[1] for n in (T, P, T, P))
    gates = matrix(T, k, gtype)[1]
    op.sort(chosen)
    place = op.place[:T].long()
    there, total = place >= 0, int(op.offsets[-1])
    whole, out = matrix(P)
    was = whole.clone()
    op.gather(x, out)
    source = op.source[:P].long()
    assert torch.equal(out[:total], x[source[:total] // k])
    assert torch.equal(whole[total:], was[total:]) and torch.equal(whole[:, width:], was[:, width:])

    at = place.clamp(min=0)
    r = rows.double()[at] * there[..., None] if P else rows.double().new_zeros(T, k, width)
    g = torch.where(there, gates.double(), 0.0)
    whole, y = matrix(T)
    was = whole.clone()
    op.combine(rows, gates, y)
    terms = g[..., None] * r
    close(y, terms.sum(1), k * E32 * terms.abs().sum(1))
    assert torch.equal(whole[:, width:], was[:, width:])

    whole, drows = matrix(P)
    was = whole.clone()
    dgates = torch.full((T, k), 7.0, dtype=gtype, device=DEV)
    op.combine_gradient(dout, rows, gates, drows, dgates)
    want = g.reshape(-1)[source[:total]][:, None] * dout.double()[source[:total] // k]
    close(drows[:total], want, E32 * want.abs())
    assert torch.equal(whole[total:], was[total:]) and torch.equal(whole[:, width:], was[:, width:])
    terms = dout.double()[:, None] * r
    close(dgates, terms.sum(2), (width + 12) * E32 * terms.abs().sum(2))
    assert not dgates[~there].any()

    dx = matrix(T)[1]
    op.gather_gradient(dsorted, dx)
    terms = dsorted.double()[at] * there[..., None] if P else r
    close(dx, terms.sum(1), k * E32 * terms.abs().sum(1))


def choices(T, k, E, seed=0, dropped=0.0, index=torch.int64):
    gen = generator(seed)
    z = torch.randn(T, E, generator=gen, device=DEV) + torch.randn(E, generator=gen, device=DEV)
    chosen = z.topk(k, dim=1).indices
    if dropped:
        chosen = torch.where(torch.rand(T, k, generator=gen, device=DEV) < dropped, -1, chosen)
    return chosen.to(index)


@pytest.mark.parametrize("index", [torch.int32, torch.int64])
@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 2, 8), (3, 3, 3), (8, 2, 8), (63, 1, 5), (64, 1, 5), (65, 1, 5),
                                   (100, 4, 60), (127, 8, 8), (128, 8, 512), (129, 8, 257), (513, 2, 2), (1000, 16, 100),
                                   (4096, 8, 64), (5000, 3, 511), (40000, 8, 256), (300001, 1, 7)])
def test_sort(T, k, E, index):
    for dropped in (0.0, 0.3):
        check_sort(ExpertDispatch(E, k, T), choices(T, k, E, dropped=dropped, index=index))


@pytest.mark.parametrize("k,most,fewer", [(1, 262145, 262144), (8, 40000, 32768), (2, 600001, 131072)])
def test_sort_of_fewer_tokens_than_asked_for(k, most, fewer):
    """Fewer pairs than the object is made for, in more blocks."""
    op = ExpertDispatch(256, k, most)
    for T in (most, fewer, fewer - 1, 5):
        check_sort(op, choices(T, k, 256, seed=T, dropped=0.1))


def test_sort_of_every_kind_of_choice():
    op = ExpertDispatch(4, 3, 500)
    check_sort(op, torch.full((200, 3), -1, device=DEV))                     # nothing left
    check_sort(op, torch.full((200, 3), 2, device=DEV))                      # the same expert, many times in a row
    check_sort(op, torch.full((200, 3), 4, device=DEV))                      # past the last expert: dropped
    low = torch.tensor([[-2 ** 40, 2 ** 40, 2 ** 32 + 1], [1, -1, 3], [0, 2 ** 31, 0]], device=DEV)
    check_sort(op, low)
    check_sort(op, torch.randint(-2, 6, (500, 3), device=DEV))
    wide = torch.randint(0, 4, (100, 10), device=DEV)
    check_sort(op, wide[:, 2:5])                                             # rows with a distance
    op.sort(torch.empty(0, 3, dtype=torch.int64, device=DEV))
    assert op.offsets.tolist() == [0] * 5


@pytest.mark.parametrize("kind,gkind", [("fp16", "fp16"), ("bf16", "fp32"), ("fp32", "fp32"), ("bf16", "bf16"),
                                        ("fp32", "bf16")])
@pytest.mark.parametrize("T,k,E,width", [(1, 1, 1, 1), (1, 2, 8, 512), (7, 3, 5, 7), (33, 4, 16, 8), (100, 8, 64, 130),
                                         (64, 16, 32, 1001), (257, 2, 3, 520), (30, 5, 12, 4099), (2500, 8, 64, 600),
                                         (3000, 1, 4, 65), (5000, 8, 64, 1001)])
def test_moves(T, k, E, width, kind, gkind):
    op = ExpertDispatch(E, k, T)
    check_moves(op, choices(T, k, E, dropped=0.2), width, kind, gkind)
    check_moves(op, choices(T, k, E, seed=1), width, kind, gkind, seed=2, pad=3)


def test_moves_of_one_object_at_other_sizes():
    op = ExpertDispatch(16, 4, 1000)
    for T, width in ((1000, 64), (1, 300), (500, 9), (0, 16), (999, 2048)):
        chosen = choices(T, 4, 16) if T else torch.empty(0, 4, dtype=torch.int64, device=DEV)
        check_moves(op, chosen, width, "bf16", "fp32")


def test_nothing_of_dropped_choices_is_read():
    """NaN gates and NaN rows behind the last slot reach nothing; a token that lost every choice gets zeros."""
    T, k, E, D = 50, 2, 4, 40
    chosen = choices(T, k, E, dropped=0.5)
    chosen[7] = -1
    op = ExpertDispatch(E, k, T)
    op.sort(chosen)
    total, there = int(op.offsets[-1]), op.place[:T] >= 0
    rows = torch.randn(T * k, D, device=DEV)
    rows[total:] = float("nan")
    gates = torch.where(there, torch.rand(T, k, device=DEV), float("nan"))
    y = op.combine(rows, gates, torch.full((T, D), 5.0, device=DEV))
    assert torch.isfinite(y).all() and not y[7].any()
    drows, dgates = op.combine_gradient(torch.randn(T, D, device=DEV), rows, gates, torch.zeros_like(rows),
                                        torch.full_like(gates, 3.0))
    assert torch.isfinite(drows).all() and torch.isfinite(dgates).all() and not dgates[~there].any()
    dx = op.gather_gradient(rows, torch.full((T, D), 5.0, device=DEV))
    assert torch.isfinite(dx).all() and not dx[7].any()


def test_gradients_against_differences():
    """The moves are linear in x, rows and each gate, so a difference of any size gives the derivative exactly but for
    rounding."""
    T, k, E, D = 12, 3, 5, 24
    chosen = choices(T, k, E, dropped=0.2)
    op = ExpertDispatch(E, k, T)
    op.sort(chosen)
    gen = generator(3)
    x, w = torch.randn(T, D, generator=gen, device=DEV), torch.randn(T * k, D, generator=gen, device=DEV)
    out = lambda x: op.gather(x, torch.zeros(T * k, D, device=DEV)).double()  # noqa: E731
    live = int(op.offsets[-1])
    w[live:] = 0
    dx = op.gather_gradient(w, torch.empty_like(x)).double()
    for t, d in ((0, 0), (5, 13), (11, 23)):
        e = torch.zeros_like(x)
        e[t, d] = 1.0
        diff = ((out(x + e) - out(x - e)) * w.double()).sum() / 2
        # x + 1 and x - 1 are rounded once each, by half a unit of at most 8
        assert abs(float(diff - dx[t, d])) <= 8 * 2 * E32 * float(w.abs().sum(1).max()) * k + k * E32 * float(w.abs().max())
    rows, gates, dy = (torch.randn(*s, generator=gen, device=DEV) for s in ((T * k, D), (T, k), (T, D)))
    comb = lambda r, g: (op.combine(r, g, torch.empty(T, D, device=DEV)).double() * dy.double()).sum()  # noqa: E731
    drows, dgates = op.combine_gradient(dy, rows, gates, torch.zeros_like(rows), torch.empty_like(gates))
    # the sums of a pass: k products a value, each off by k E of its terms' size
    noise = k * E32 * float((dy.abs().double() * comb_abs(op, rows, gates, T, D)).sum())
    for t, j in ((0, 0), (4, 2), (11, 1)):
        e = torch.zeros_like(gates)
        e[t, j] = 4.0
        diff = (comb(rows, gates + e) - comb(rows, gates - e)) / 8
        assert abs(float(diff - dgates[t, j])) <= 2 * noise
    for q, d in ((0, 0), (live - 1, 23)):
        e = torch.zeros_like(rows)
        e[q, d] = 4.0
        diff = (comb(rows + e, gates) - comb(rows - e, gates)) / 8
        assert abs(float(diff - drows[q, d])) <= 2 * noise


def comb_abs(op, rows, gates, T, D):
    """sum_j |gate| |row| of the largest operands above (each moved by up to 4), for the rounding of a pass."""
    return op.combine(rows.abs() + 4, gates.abs() + 4, torch.empty(T, D, device=DEV)).double()


def test_bits_do_not_depend_on_the_launch_shape(monkeypatch):
    T, k, E, D = 3001, 4, 32, 300
    chosen = choices(T, k, E, dropped=0.1)
    gen = generator(5)
    x = torch.randn(T, D, generator=gen, device=DEV).half()
    rows, gates = torch.randn(T * k, D, generator=gen, device=DEV).half(), torch.rand(T, k, generator=gen, device=DEV)

    def once():
        op = ExpertDispatch(E, k, T)
        op.sort(chosen)
        a = op.gather(x, torch.zeros_like(rows))
        y = op.combine(rows, gates, torch.empty_like(x))
        d = op.combine_gradient(x, rows, gates, torch.zeros_like(rows), torch.empty_like(gates))
        return [a, y, *d, op.gather_gradient(rows, torch.empty_like(x)), op.place, op.source]

    first = once()
    for blocks in ("1", "7"):
        monkeypatch.setenv("DSZERO_GRID", blocks)
        for a, b in zip(first, once()):
            assert torch.equal(a, b)


def test_in_a_graph_and_on_a_stream():
    T, k, E, D = 700, 2, 16, 256
    gen = generator(6)
    chosen = choices(T, k, E, seed=1)
    x, gates = torch.randn(T, D, generator=gen, device=DEV).bfloat16(), torch.rand(T, k, generator=gen, device=DEV)
    side = torch.cuda.Stream()
    for stream in (None, side):
        op = ExpertDispatch(E, k, T, stream=stream)
        rows, y = torch.zeros(T * k, D, dtype=x.dtype, device=DEV), torch.empty_like(x)

        def once():
            op.sort(chosen)
            op.gather(x, rows)
            op.combine(rows, gates, y)

        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            once()
        for seed in (2, 3, 4):                                   # other choices at the same address
            chosen.copy_(choices(T, k, E, seed=seed, dropped=0.1))
            y.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            got = y.clone(), op.place.clone()
            once()
            torch.cuda.synchronize()
            assert torch.equal(got[0], y) and torch.equal(got[1], op.place)
            assert op.place[:T].flatten().tolist() == fast_order(chosen, E)[1]


def test_offsets_past_32_bits():
    """Rows whose bytes lie past 2^32 from the first: 3 million of 1024 values in 16 bits."""
    T, k, E, D = 1500000, 2, 3, 1024
    chosen = torch.arange(T * k, device=DEV, dtype=torch.int32).view(T, k) % E
    op = ExpertDispatch(E, k, T)
    op.sort(chosen)
    x = (torch.arange(T, device=DEV) % 251).to(torch.bfloat16)[:, None].repeat(1, D)
    rows = op.gather(x, torch.empty(T * k, D, dtype=torch.bfloat16, device=DEV))
    source = op.source.long()
    want = (source // k % 251).to(torch.bfloat16)
    assert torch.equal(rows[:, 0], want) and torch.equal(rows[:, D - 1], want)
    dx = op.gather_gradient(rows, torch.empty_like(x))           # k equal rows: twice the value, exact in bf16
    assert torch.equal(dx, x * 2)
    del rows, dx, x
    torch.cuda.empty_cache()
