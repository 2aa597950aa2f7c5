"""The balance loss without a GPU: what its entry points refuse before any device work."""
import ctypes

import pytest
import torch

from zero_mixed_precision_amd import ExpertBalance, _lib
from zero_mixed_precision_amd._lib import (DS_BF16, DS_ERR_ALIAS, DS_ERR_ALIGN, DS_ERR_DTYPE, DS_ERR_HPARAM, DS_ERR_NULL,
                                           DS_ERR_SIZE, DS_FP8, DS_FP32, DS_OK)

L = _lib.lib
fake = pytest.mark.skipif(torch.cuda.device_count() != 0, reason="fake device addresses: CPU-only test")
Z, MASK, COUNTS, MEAN, LOSS, USED, WS, D, ST = (0x10000000 * k for k in range(1, 10))
FORWARD = dict(logits=Z, dt=DS_BF16, tokens=100, experts=64, stride=64, mask=MASK, k=8, coef=0.01, counts=COUNTS,
               mean=MEAN, loss=LOSS, used=USED, ws=WS, nbytes=1 << 20, stream=None)
BACKWARD = dict(st=ST, logits=Z, dt=DS_BF16, tokens=100, experts=64, stride=64, mask=MASK, k=8, coef=0.01,
                counts=COUNTS, used=USED, d=D, dstride=64, accumulate=0, stream=None)


def forward(**kw):
    return L.ds_balance_loss(*{**FORWARD, **kw}.values())


def backward(**kw):
    return L.ds_balance_loss_grad(*{**BACKWARD, **kw}.values())


@fake
@pytest.mark.parametrize("call", [forward, backward])
def test_shared_refusals(call):
    for kw in (dict(tokens=-1), dict(tokens=(1 << 30) + 1), dict(experts=0), dict(experts=513, stride=513),
               dict(k=0), dict(k=17), dict(experts=4, k=5), dict(stride=63), dict(stride=(1 << 40) + 1),
               dict(stride=1 << 36)):
        assert call(**kw) == DS_ERR_SIZE, kw
    for dt in (0, DS_FP8, 9):
        assert call(dt=dt) == DS_ERR_DTYPE
    for coef in (-0.1, float("nan"), float("inf")):
        assert call(coef=coef) == DS_ERR_HPARAM
    for kw in (dict(logits=None), dict(counts=None), dict(used=None)):
        assert call(**kw) == DS_ERR_NULL, kw
    for kw in (dict(logits=Z + 1), dict(dt=DS_FP32, logits=Z + 2), dict(counts=COUNTS + 2), dict(used=USED + 2)):
        assert call(**kw) == DS_ERR_ALIGN, kw


@fake
def test_forward_refusals():
    for name in ("mean", "loss", "ws"):
        assert forward(**{name: None}) == DS_ERR_NULL, name
    for kw in (dict(mean=MEAN + 2), dict(loss=LOSS + 1), dict(ws=WS + 4)):
        assert forward(**kw) == DS_ERR_ALIGN, kw
    assert forward(nbytes=_lib.ds_balance_workspace_bytes(100, 64) - 1) == DS_ERR_SIZE
    last = Z + 2 * 6400
    for kw in (dict(counts=last - 4), dict(mean=Z), dict(loss=last - 4), dict(used=Z), dict(ws=Z + 8),
               dict(counts=MASK + 96), dict(mean=COUNTS + 252), dict(loss=COUNTS), dict(used=LOSS), dict(ws=MEAN),
               dict(stride=1 << 20, counts=Z + 2 * 99 * (1 << 20))):
        assert forward(**kw) == DS_ERR_ALIAS, kw


@fake
def test_backward_refusals():
    assert backward(d=None) == DS_ERR_NULL and backward(d=D + 1) == DS_ERR_ALIGN
    assert backward(st=ST + 4) == DS_ERR_ALIGN
    assert backward(dstride=63) == DS_ERR_SIZE and backward(dstride=1 << 36) == DS_ERR_SIZE
    for kw in (dict(d=Z), dict(d=MASK + 96), dict(d=COUNTS), dict(d=USED), dict(d=ST + 64), dict(st=D + 64)):
        assert backward(**kw) == DS_ERR_ALIAS, kw
    assert backward(tokens=0, logits=None, d=None, mask=None) == DS_OK      # nothing to write


def test_workspace_bytes():
    f = _lib.ds_balance_workspace_bytes
    assert f(-1, 8) == 0 and f(8, 0) == 0 and f(8, 513) == 0 and f((1 << 30) + 1, 8) == 0
    sizes = [f(t, 64) for t in (0, 1, 32, 33, 1000, 1 << 20, 1 << 30)]
    assert sizes == sorted(sizes) and sizes[-1] == sizes[-2] and sizes[0] > 0


def test_class_refusals():
    for args in ((0, 1), (513, 1), (8, 0), (8, 9), (64, 17)):
        with pytest.raises(ValueError):
            ExpertBalance(*args, coef=0.1)
    assert ctypes.sizeof(ctypes.c_void_p) == 8
