"""The tokens' way to the experts, the distillation loss and the cross entropy without a GPU: what their entry points refuse
before any device work, and what their classes hand to them."""
import ctypes
import math

import pytest
import torch

from tests.stand_in import Library, Stream, Tensor, Torch
from zero_mixed_precision_amd import ExpertDispatch, TopLogitDistillation, VocabCrossEntropy, _lib
from zero_mixed_precision_amd._lib import (DS_BF16, DS_ERR_ALIAS, DS_ERR_ALIGN, DS_ERR_DTYPE, DS_ERR_HPARAM, DS_ERR_NULL,
                                           DS_ERR_SIZE, DS_FP8, DS_FP16, DS_FP32, DS_OK)

L = _lib.lib
fake = pytest.mark.skipif(torch.cuda.device_count() != 0, reason="fake device addresses: CPU-only test")
A, B, C, D, E, F, G, H, I, J, K = (0x100000000 * k for k in range(1, 12))


def caller(name, **defaults):
    def call(**kw):
        assert set(kw) <= set(defaults), kw
        return getattr(L, name)(*{**defaults, **kw}.values())
    return call


sort = caller("ds_dispatch_sort", chosen=A, index_bytes=8, tokens=100, experts=64, k=8, stride=8, offsets=B, place=C,
              source=D, ws=E, nbytes=1 << 20, stream=None)
gather = caller("ds_dispatch_gather", x=A, dt=DS_BF16, tokens=100, k=8, width=64, xs=64, place=B, out=C, os=64, rows=800,
                stream=None)
gather_grad = caller("ds_dispatch_gather_grad", dout=C, dt=DS_BF16, tokens=100, k=8, width=64, os=64, rows=800, place=B,
                     x=A, xs=64, stream=None)
combine = caller("ds_dispatch_combine", out=C, dt=DS_BF16, tokens=100, k=8, width=64, os=64, rows=800, place=B, gates=D,
                 gdt=DS_FP32, gs=8, x=A, xs=64, stream=None)
combine_grad = caller("ds_dispatch_combine_grad", x=A, dt=DS_BF16, tokens=100, k=8, width=64, xs=64, out=C, os=64, rows=800,
                      place=B, gates=D, gdt=DS_FP32, gs=8, drows=E, drs=64, dgates=F, dgs=8, stream=None)
distill = caller("ds_distill_loss", st=A, logits=B, dt=DS_BF16, tokens=100, vocab=1000, zs=1000, teacher=C, tdt=DS_FP32,
                 ts=8, index=D, index_bytes=4, istr=8, k=8, mask=E, tau=2.0, coef=1.0, token_loss=F, loss=G, used=H, grad=I,
                 gs=1000, acc=0, ws=J, nbytes=1 << 20, stream=None)
vocab = caller("ds_vocab_ce", st=A, hidden=B, hs=64, weight=C, ws=64, dt=DS_BF16, targets=D, index_bytes=8, tokens=100,
               vocab=1000, width=64, mask=E, coef=1.0, token_loss=F, loss=G, used=H, dhidden=I, dhs=64, dweight=J,
               dwt=DS_BF16, dws=64, acc=0, work=K, nbytes=1 << 30, stream=None)
HUGE = 1 << 40


@fake
def test_sort_refusals():
    for kw in (dict(tokens=-1), dict(tokens=1 << 28), dict(experts=0), dict(experts=513), dict(k=0), dict(k=17, stride=17),
               dict(stride=7), dict(stride=HUGE), dict(nbytes=4 * 64 - 1)):
        assert sort(**kw) == DS_ERR_SIZE, kw
    for n in (0, 1, 2, 16):
        assert sort(index_bytes=n) == DS_ERR_DTYPE
    for name in ("chosen", "offsets", "place", "source", "ws"):
        assert sort(**{name: None}) == DS_ERR_NULL, name
    for kw in (dict(chosen=A + 4), dict(offsets=B + 2), dict(place=C + 1), dict(source=D + 2), dict(ws=E + 2)):
        assert sort(**kw) == DS_ERR_ALIGN, kw
    for kw in (dict(offsets=A + 8), dict(place=A + 6400 - 4), dict(source=C + 3196), dict(ws=B + 256), dict(place=B)):
        assert sort(**kw) == DS_ERR_ALIAS, kw


@fake
@pytest.mark.parametrize("move", [gather, gather_grad, combine, combine_grad])
def test_move_refusals(move):
    for kw in (dict(tokens=-1), dict(tokens=1 << 28), dict(k=0), dict(k=17), dict(width=0), dict(width=(1 << 24) + 1),
               dict(xs=63), dict(os=63), dict(xs=HUGE), dict(os=HUGE), dict(rows=-1), dict(rows=1 << 31)):
        assert move(**kw) == DS_ERR_SIZE, kw
    for dt in (0, DS_FP8, 9):
        assert move(dt=dt) == DS_ERR_DTYPE
    for name in ("x", "place", "out" if move is not gather_grad else "dout"):
        assert move(**{name: None}) == DS_ERR_NULL, name
    sorted_side = "dout" if move is gather_grad else "out"
    for kw in (dict(x=A + 1), {sorted_side: C + 1}, dict(place=B + 2), {"dt": DS_FP32, sorted_side: C + 2}):
        assert move(**kw) == DS_ERR_ALIGN, kw
    written = {gather: dict(out=A + 2), gather_grad: dict(x=C + 2 * 800 * 64 - 2), combine: dict(x=C),
               combine_grad: dict(drows=C)}[move]
    assert move(**written) == DS_ERR_ALIAS


@fake
def test_gate_refusals():
    for move in (combine, combine_grad):
        assert move(gs=7) == DS_ERR_SIZE and move(gdt=DS_FP8) == DS_ERR_DTYPE and move(gates=None) == DS_ERR_NULL
        assert move(gates=D + 2) == DS_ERR_ALIGN
    assert combine(x=D + 4) == DS_ERR_ALIAS and combine(x=B + 4) == DS_ERR_ALIAS
    for kw in (dict(drs=63), dict(dgs=7)):
        assert combine_grad(**kw) == DS_ERR_SIZE
    for kw in (dict(drows=None), dict(dgates=None)):
        assert combine_grad(**kw) == DS_ERR_NULL
    for kw in (dict(drows=E + 1), dict(dgates=F + 2)):
        assert combine_grad(**kw) == DS_ERR_ALIGN
    for kw in (dict(drows=A), dict(dgates=D), dict(dgates=E), dict(dgates=B + 8)):
        assert combine_grad(**kw) == DS_ERR_ALIAS, kw


@fake
def test_moves_with_nothing_to_do():
    none = dict(tokens=0, rows=0, x=None, place=None)
    assert gather(out=None, **none) == DS_OK and gather_grad(dout=None, **none) == DS_OK
    assert combine(out=None, gates=None, **none) == DS_OK
    assert combine_grad(out=None, gates=None, drows=None, dgates=None, **none) == DS_OK


@fake
def test_distill_refusals():
    for kw in (dict(tokens=-1), dict(tokens=(1 << 30) + 1), dict(vocab=0), dict(vocab=(1 << 30) + 1, zs=HUGE), dict(k=0),
               dict(k=1025, ts=1025, istr=1025), dict(zs=999), dict(ts=7), dict(istr=7), dict(gs=999), dict(zs=HUGE),
               dict(gs=HUGE), dict(nbytes=107)):
        assert distill(**kw) == DS_ERR_SIZE, kw
    for kw in (dict(dt=DS_FP8), dict(tdt=0), dict(index_bytes=2)):
        assert distill(**kw) == DS_ERR_DTYPE, kw
    for tau in (0.0, -1.0, math.nan, math.inf, 2000.0, 1e-4):
        assert distill(tau=tau) == DS_ERR_HPARAM
    for kw in (dict(coef=-1.0), dict(coef=math.nan), dict(coef=math.inf), dict(acc=1, grad=None)):
        assert distill(**kw) == DS_ERR_HPARAM, kw
    for name in ("logits", "teacher", "index", "token_loss", "loss", "used", "ws"):
        assert distill(**{name: None}) == DS_ERR_NULL, name
    for kw in (dict(st=A + 4), dict(logits=B + 1), dict(teacher=C + 2), dict(index=D + 2), dict(token_loss=F + 2),
               dict(loss=G + 1), dict(used=H + 2), dict(grad=I + 1), dict(ws=J + 4), dict(index_bytes=8, index=D + 4)):
        assert distill(**kw) == DS_ERR_ALIGN, kw
    for kw in (dict(grad=B + 2), dict(grad=B, acc=1), dict(grad=B, gs=1001), dict(grad=C), dict(grad=E + 98), dict(ws=G),
               dict(token_loss=B), dict(loss=D), dict(used=G), dict(grad=J + 8), dict(token_loss=A + 64),
               dict(grad=B, teacher=B + 4 * 100), dict(grad=B, st=B + 8)):
        assert distill(**kw) == DS_ERR_ALIAS, kw


@fake
def test_vocab_refusals():
    for kw in (dict(tokens=-1), dict(tokens=(1 << 24) + 1), dict(vocab=0), dict(vocab=(1 << 24) + 1), dict(width=0),
               dict(width=65537, hs=HUGE), dict(hs=63), dict(ws=63), dict(dhs=63), dict(dws=63), dict(ws=HUGE),
               dict(nbytes=_lib.ds_vocab_ce_workspace_bytes(100, 1000, 64) - 1)):
        assert vocab(**kw) == DS_ERR_SIZE, kw
    for kw in (dict(dt=DS_FP32), dict(dt=DS_FP8), dict(index_bytes=1), dict(dwt=DS_FP16), dict(dwt=DS_FP8)):
        assert vocab(**kw) == DS_ERR_DTYPE, kw
    for kw in (dict(coef=-1.0), dict(coef=math.inf), dict(acc=1, dweight=None)):
        assert vocab(**kw) == DS_ERR_HPARAM, kw
    for name in ("hidden", "weight", "targets", "token_loss", "loss", "used", "work"):
        assert vocab(**{name: None}) == DS_ERR_NULL, name
    for kw in (dict(st=A + 4), dict(hidden=B + 1), dict(weight=C + 1), dict(targets=D + 4), dict(token_loss=F + 1),
               dict(loss=G + 2), dict(used=H + 2), dict(dhidden=I + 1), dict(dweight=J + 1), dict(dwt=DS_FP32, dweight=J + 2),
               dict(work=K + 128)):
        assert vocab(**kw) == DS_ERR_ALIGN, kw
    for kw in (dict(dhidden=B), dict(dweight=C + 2), dict(dweight=I + 256), dict(token_loss=D), dict(loss=E), dict(used=G),
               dict(work=C + 256), dict(work=I), dict(dhidden=A + 64)):
        assert vocab(**kw) == DS_ERR_ALIAS, kw


def test_workspace_bytes():
    f = _lib.ds_dispatch_workspace_bytes
    assert f(-1, 8, 2) == 0 and f(8, 0, 2) == 0 and f(8, 513, 2) == 0 and f(8, 8, 17) == 0 and f(1 << 31, 8, 1) == 0
    assert f(0, 8, 2) > 0 and f(1 << 26, 512, 16) == f(1 << 20, 512, 16)
    f = _lib.ds_distill_workspace_bytes
    assert f(-1) == 0 and f((1 << 30) + 1) == 0 and f(100) >= 100 and f(1 << 30) > f(1 << 20)
    f = _lib.ds_vocab_ce_workspace_bytes
    assert f(-1, 8, 8) == 0 and f(8, 0, 8) == 0 and f(8, 8, 0) == 0 and f(8, 8, 65537) == 0 and f(1 << 25, 8, 8) == 0
    assert 0 < f(0, 1, 1) <= f(256, 1, 1) < f(257, 1, 1)
    for V, D in ((1, 1), (500, 64), (32000, 100), (131072, 4096), (1 << 24, 8)):    # what serves many tokens serves fewer
        sizes = [f(t, V, D) for t in (1, 100, 256, 1000, 4096, 5000, 8192, 16000, 40000, 65536, 131072, 131073, 1 << 20)]
        assert sizes == sorted(sizes)
    # a piece's dz, not the vocabulary's, and no more of the weight than that
    assert f(8192, 131072, 4096) < 2 * 8192 * 131072


def test_a_sort_workspace_for_many_tokens_serves_fewer():
    """An object's workspace is that of its largest call; a batch of fewer tokens must not be refused by it."""
    f = _lib.ds_dispatch_workspace_bytes
    for k in (1, 2, 3, 8, 16):
        near = [p // k + d for p in (1024, 1 << 17, 1 << 18, 327680, 1 << 19, 1 << 20, 1 << 24, 1 << 30) for d in range(-2, 3)]
        tokens = sorted({t for t in near + [int(1.07 ** n) for n in range(280)] if t * k < 1 << 31})
        sizes = [f(t, 256, k) for t in tokens]
        assert sizes == sorted(sizes)
        # a row of counts for each block: chunks of 1024 pairs or, past 256 of them, 256 equal ones rounded up to 256
        for t, size in zip(tokens, sizes):
            chunk = -(-max(1024, -(-t * k // 256)) // 256) * 256
            assert size >= 4 * 256 * max(1, -(-t * k // chunk))


def over_stand_ins(monkeypatch, kind, stream=None, current=0, index=0):
    torch_ = Torch(current)
    library = Library(torch_)
    monkeypatch.setattr(_lib, "lib", library)
    monkeypatch.setattr(_lib, "_raw_stream", lambda i: 0x100 * i)
    op = kind.__new__(kind)
    op.torch, op.stream, op._device, op._many, op.device = torch_, stream, index, True, torch.device("cuda", index)
    op.max_tokens, op._scratch, op._at, op.value, op.coef = 100, (9, 64), (1, 2, 3), "value", 1.0
    op._index_types = (torch.int32, torch.int64)
    return op, torch_, library


def dispatch(monkeypatch, **kw):
    op, torch_, library = over_stand_ins(monkeypatch, ExpertDispatch, **kw)
    op.E, op.k, op.tokens = 64, 8, 0
    op.offsets, op._place, op._at = Tensor(100, dtype=torch.int32, index=op._device), 2, (1, 2, 3, 9, 64)
    return op, torch_, library


@pytest.mark.parametrize("stream", [None, Stream(), 0x7000])
@pytest.mark.parametrize("current,index", [(0, 1), (1, 0), (1, 1)])
def test_dispatch_launches_where_its_tensors_are(current, index, stream, monkeypatch):
    op, torch_, library = dispatch(monkeypatch, stream=stream, current=current, index=index)
    t = lambda *s, dtype=torch.bfloat16: Tensor(*s, dtype=dtype, index=index)  # noqa: E731
    chosen, x, y, dy, dx = t(9, 8, dtype=torch.int64), t(9, 32), t(9, 32), t(9, 32), t(9, 32)
    rows, drows, gates, dgates = t(72, 32), t(80, 32), t(9, 8, dtype=torch.float32), t(9, 8, dtype=torch.float32)
    op.sort(chosen)
    op.gather(x, rows)
    op.combine(rows, gates, y)
    op.combine_gradient(dy, rows, gates, drows, dgates)
    op.gather_gradient(drows, dx)
    there = {None: 0x100 * index, 0x7000: 0x7000}.get(stream, 0x5000)
    assert [(c[0], c[1], c[2][-1]) for c in library.calls] == [
        (name, index, there) for name in ("ds_dispatch_sort", "ds_dispatch_gather", "ds_dispatch_combine",
                                          "ds_dispatch_combine_grad", "ds_dispatch_gather_grad")]
    assert torch_.now == current
    want = [] if stream is None else [("external", stream)] if isinstance(stream, int) else [stream]
    for x, n in ((chosen, 1), (x, 1), (y, 1), (rows, 3), (gates, 2), (dgates, 1), (drows, 2), (dx, 1), (dy, 1)):
        assert x.recorded == n * want
    # the sorted side's rows: what both matrices of the gradient have
    assert library.calls[3][2][8] == 72


def test_dispatch_class_refusals(monkeypatch):
    for args in ((0, 1, 5), (513, 1, 5), (8, 0, 5), (8, 17, 5), (8, 2, -1), (8, 2, 1 << 31)):
        with pytest.raises(ValueError):
            ExpertDispatch(*args)
    op, _, library = dispatch(monkeypatch)
    T = lambda *s, dtype=torch.bfloat16, **kw: Tensor(*s, dtype=dtype, **kw)  # noqa: E731
    for chosen in (T(9, 7, dtype=torch.int64), T(9, 8, dtype=torch.float32), T(101, 8, dtype=torch.int32),
                   T(72, dtype=torch.int32), T(9, 8, dtype=torch.int32, index=1)):
        with pytest.raises(ValueError):
            op.sort(chosen)
    op.sort(T(9, 8, dtype=torch.int32))
    g = T(9, 8, dtype=torch.float32)
    bad = [lambda: op.gather(T(8, 32), T(72, 32)), lambda: op.gather(T(9, 32), T(71, 32)),
           lambda: op.gather(T(9, 32), T(72, 31)), lambda: op.gather(T(9, 32), T(72, 32, dtype=torch.float16)),
           lambda: op.gather(T(9, 32, dtype=torch.float64), T(72, 32)), lambda: op.gather(T(9, 32, index=1), T(72, 32)),
           lambda: op.gather(T(9), T(72, 32)), lambda: op.combine(T(72, 32), T(9, 7, dtype=torch.float32), T(9, 32)),
           lambda: op.combine(T(72, 32), T(8, 8, dtype=torch.float32), T(9, 32)),
           lambda: op.combine_gradient(T(9, 32), T(72, 32), g, T(72, 32), T(9, 8)),
           lambda: op.combine_gradient(T(9, 32), T(72, 32), g, T(72, 32, dtype=torch.float32), g),
           lambda: op.combine_gradient(T(9, 32), T(72, 32), g, T(71, 32), g),
           lambda: op.gather_gradient(T(71, 32), T(9, 32))]
    before = len(library.calls)
    for call in bad:
        with pytest.raises(ValueError):
            call()
    assert len(library.calls) == before


@pytest.mark.parametrize("stream", [None, 0x7000])
@pytest.mark.parametrize("current,index", [(0, 1), (1, 1)])
def test_losses_launch_where_their_tensors_are(current, index, stream, monkeypatch):
    t = lambda *s, dtype=torch.bfloat16: Tensor(*s, dtype=dtype, index=index)  # noqa: E731
    there = 0x100 * index if stream is None else stream
    want = [] if stream is None else [("external", stream)]
    mask, state = t(9, dtype=torch.bool), t(128, dtype=torch.uint8)
    op, torch_, library = over_stand_ins(monkeypatch, TopLogitDistillation, stream=stream, current=current, index=index)
    op.vocab, op.k, op.temperature = 500, 4, 2.0
    z, teacher, place, out = t(9, 500), t(9, 4, dtype=torch.float32), t(9, 4, dtype=torch.int32), t(9, 500)
    assert op.loss(z, teacher, place, mask=mask) == "value"
    op.loss_and_gradient(z, teacher, place, out, mask=mask, scaler=state, accumulate=True)
    assert [(c[0], c[1], c[2][-1]) for c in library.calls] == 2 * [("ds_distill_loss", index, there)]
    assert library.calls[0][2][19] is None and library.calls[1][2][19] == out.at and library.calls[1][2][0] == state.at
    assert out.recorded == state.recorded == want and z.recorded == mask.recorded == 2 * want and torch_.now == current

    mask, state = t(9, dtype=torch.bool), t(128, dtype=torch.uint8)
    op, torch_, library = over_stand_ins(monkeypatch, VocabCrossEntropy, stream=stream, current=current, index=index)
    op.vocab, op.width, op.dtype = 500, 32, torch.bfloat16
    x, w, y, dx, dw = t(9, 32), t(500, 32), t(9, dtype=torch.int64), t(9, 32), t(500, 32, dtype=torch.float32)
    assert op.loss(x, w, y, mask=mask) == "value"
    op.loss_and_gradient(x, w, y, dx, dw, mask=mask, scaler=state, accumulate=True)
    assert [(c[0], c[1], c[2][-1]) for c in library.calls] == 2 * [("ds_vocab_ce", index, there)]
    assert library.calls[1][2][16] == dx.at and library.calls[1][2][18:21] == (dw.at, DS_FP32, 32)
    assert dw.recorded == dx.recorded == want and w.recorded == y.recorded == 2 * want and torch_.now == current


def test_loss_class_refusals(monkeypatch):
    for args in ((0, 1, 5), (2 ** 30 + 1, 1, 5), (8, 0, 5), (8, 1025, 5), (8, 2, -1), (8, 2, 5, 0.0), (8, 2, 5, 2000.0)):
        with pytest.raises(ValueError):
            TopLogitDistillation(*args)
    for args in ((0, 8, 5, torch.float16), (8, 0, 5, torch.float16), (8, 65537, 5, torch.float16), (8, 8, 5, torch.float32),
                 (8, 8, 1 << 25, torch.bfloat16), (1 << 25, 8, 5, torch.bfloat16)):
        with pytest.raises(ValueError):
            VocabCrossEntropy(*args)
    T = lambda *s, dtype=torch.bfloat16, **kw: Tensor(*s, dtype=dtype, **kw)  # noqa: E731
    i = lambda *s: T(*s, dtype=torch.int32)  # noqa: E731
    op, _, library = over_stand_ins(monkeypatch, TopLogitDistillation)
    op.vocab, op.k, op.temperature = 500, 4, 2.0
    z, t = T(9, 500), T(9, 4)
    bad = [lambda: op.loss(T(9, 499), t, i(9, 4)), lambda: op.loss(T(101, 500), T(101, 4), i(101, 4)),
           lambda: op.loss(z, T(8, 4), i(9, 4)), lambda: op.loss(z, t, i(9, 3)), lambda: op.loss(z, t, T(9, 4)),
           lambda: op.loss(z, t, i(9, 4), mask=T(8, dtype=torch.bool)), lambda: op.loss(z, t, i(9, 4), mask=i(9)),
           lambda: op.loss(T(9, 500, index=1), t, i(9, 4)),
           lambda: op.loss_and_gradient(z, t, i(9, 4), T(9, 500, dtype=torch.float32)),
           lambda: op.loss_and_gradient(z, t, i(9, 4), T(8, 500)),
           lambda: op.loss_and_gradient(z, t, i(9, 4), T(9, 500), scaler=T(128, dtype=torch.uint8, index=1)),
           lambda: op.loss_and_gradient(z, t, i(9, 4), T(9, 500), scaler=T(100, dtype=torch.uint8))]
    ce, _, also = over_stand_ins(monkeypatch, VocabCrossEntropy)
    ce.vocab, ce.width, ce.dtype = 500, 32, torch.bfloat16
    x, w, y = T(9, 32), T(500, 32), i(9)
    bad += [lambda: ce.loss(T(9, 31), w, y), lambda: ce.loss(T(101, 32), w, i(101)), lambda: ce.loss(x, T(499, 32), y),
            lambda: ce.loss(x, w, i(8)), lambda: ce.loss(x, w, T(9)), lambda: ce.loss(T(9, 32, dtype=torch.float16), w, y),
            lambda: ce.loss(x, T(500, 32, dtype=torch.float16), y), lambda: ce.loss_and_gradient(x, w, y, None, None),
            lambda: ce.loss_and_gradient(x, w, y, T(9, 32), None, accumulate=True),
            lambda: ce.loss_and_gradient(x, w, y, T(9, 32, dtype=torch.float32), None),
            lambda: ce.loss_and_gradient(x, w, y, None, T(500, 32, dtype=torch.float16)),
            lambda: ce.loss_and_gradient(x, w, y, None, T(500, 32, index=1))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    assert library.calls == [] and also.calls == []


def test_rows_that_overlap_or_are_not_adjacent(monkeypatch):
    op, _, library = over_stand_ins(monkeypatch, VocabCrossEntropy)
    op.vocab, op.width, op.dtype = 500, 32, torch.bfloat16
    w, y = Tensor(500, 32), Tensor(9, dtype=torch.int32)
    for stride in ((31, 1), (0, 1), (64, 2)):
        x = Tensor(9, 32)
        x.stride = lambda s=stride: s
        with pytest.raises(ValueError):
            op.loss(x, w, y)
    one = Tensor(1, 32)
    one.stride = lambda: (0, 1)                          # a single row: its distance means nothing
    op.loss(one, w, Tensor(1, dtype=torch.int32))
    assert library.calls[0][2][2] == 32
    y.stride = lambda: (2,)
    with pytest.raises(ValueError):
        op.loss(Tensor(9, 32), w, y)
    assert ctypes.sizeof(ctypes.c_void_p) == 8
