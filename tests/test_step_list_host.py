"""ds_step_list without a GPU: what it refuses before any device work."""
import ctypes

import pytest
import torch

from zero_mixed_precision_amd import _lib
from zero_mixed_precision_amd._lib import (DS_ERR_ALIAS, DS_ERR_ALIGN, DS_ERR_DTYPE, DS_ERR_HPARAM, DS_ERR_NULL,
                                           DS_ERR_SIZE, DS_FP32, DsTensorList)

# made-up device addresses: refused calls must not reach a kernel, so these run only where no GPU is visible
fake = pytest.mark.skipif(torch.cuda.device_count() != 0, reason="fake device addresses: CPU-only test")
TABLE, ST, WS = 0x700000000, 0x710000000, 0x720000000


@fake
@pytest.mark.parametrize("tiles", [1, 8, 9, 2048, 2049])
def test_refusals(tiles):
    lst = DsTensorList(table=TABLE, tiles=tiles, elems=tiles * 4096, count=1, sdt=DS_FP32)
    need = _lib.ds_tensor_list_workspace_bytes(lst)
    good = dict(st=ST, lst=ctypes.byref(lst), ws=WS, nbytes=need, lr=1e-3, sched=None, b1=0.9, b2=0.999, eps=1e-8,
                clip=1.0, K=1, rounding=0, seed=0, stream=None)

    def step(**kw):
        return _lib.lib.ds_step_list(*{**good, **kw}.values())

    assert step(st=None) == DS_ERR_NULL and step(lst=None) == DS_ERR_NULL
    assert step(st=ST + 4) == DS_ERR_ALIGN and step(ws=WS + 4) == DS_ERR_ALIGN
    assert step(nbytes=need - 1) == DS_ERR_SIZE
    assert step(st=TABLE) == DS_ERR_ALIAS and step(ws=TABLE) == DS_ERR_ALIAS and step(ws=ST + 64) == DS_ERR_ALIAS
    assert step(st=TABLE, ws=None, nbytes=0) == DS_ERR_ALIAS
    for kw in (dict(lr=-1.0), dict(lr=float("nan")), dict(b1=1.0), dict(b2=-0.1), dict(eps=0.0), dict(clip=-1.0),
               dict(K=0), dict(rounding=2), dict(sched=ctypes.byref(_lib.DsLrSchedule.make(9, 0, 1, 1)))):
        assert step(**kw) == DS_ERR_HPARAM, kw
    for kw, want in ((dict(table=None), DS_ERR_NULL), (dict(sdt=0), DS_ERR_DTYPE), (dict(tiles=tiles + 2), DS_ERR_SIZE),
                     (dict(elems=0), DS_ERR_SIZE), (dict(count=-1), DS_ERR_SIZE)):
        bad = DsTensorList(**{**dict(table=TABLE, tiles=tiles, elems=tiles * 4096, count=1, sdt=DS_FP32), **kw})
        assert step(lst=ctypes.byref(bad)) == want, kw
