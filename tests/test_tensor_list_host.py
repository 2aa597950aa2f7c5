"""The step over a list of tensors without a GPU: what the entry points refuse before any device work, the host structs,
and the 8-bit formats of the reference against torch's."""
import ctypes

import numpy as np
import pytest
import torch

from tests import list_ref as ref
from zero_mixed_precision_amd import MultiTensorStep, ZeroMPConfig, _lib
from zero_mixed_precision_amd._lib import (DS_BF16, DS_ERR_ALIAS, DS_ERR_ALIGN, DS_ERR_DTYPE, DS_ERR_HPARAM, DS_ERR_NULL,
                                           DS_ERR_SIZE, DS_FP8, DS_FP16, DS_FP32, DS_OK, DsTensor, DsTensorList)
from zero_mixed_precision_amd.multi_tensor import per_tensor

L = _lib.lib
# made-up device addresses: refused calls must not reach a kernel, so these run only where no GPU is visible
fake = pytest.mark.skipif(torch.cuda.device_count() != 0, reason="fake device addresses: CPU-only test")
TABLE, ST = 0x700000000, 0x710000000
BIG = 1 << 20


def tensor(at=0x10000000, n=1000, **kw):
    """A valid tensor with 32-bit states; keyword arguments replace fields."""
    step = 1 << 24
    d = dict(master=at, p16=at + step, m=at + 2 * step, v=at + 3 * step, m_scale=None, v_scale=None, grad=at + 4 * step,
             n=n, weight_decay=0.0, lr_scale=1.0, pdt=DS_BF16, gdt=DS_BF16)
    d.update(kw)
    return DsTensor(**d)


def tensor8(at=0x10000000, **kw):
    step = 1 << 24
    return tensor(at, **{**dict(m_scale=at + 5 * step, v_scale=at + 6 * step), **kw})


def write(tensors, sdt=DS_FP32, table=TABLE, nbytes=BIG, out=True):
    arr = (DsTensor * max(len(tensors), 1))(*tensors)
    lst = DsTensorList()
    return L.ds_tensor_list_write(ctypes.byref(lst) if out else None, table, nbytes, arr, len(tensors), sdt, None)


def test_structs():
    assert ctypes.sizeof(DsTensor) == 80 and ctypes.sizeof(DsTensorList) == 32
    assert DsTensor.n.offset == 56 and DsTensor.weight_decay.offset == 64 and DsTensor.gdt.offset == 76
    assert DsTensorList.count.offset == 24 and DsTensorList.sdt.offset == 28


def test_table_bytes():
    assert _lib.ds_tensor_list_bytes(0) == 0 and L.ds_tensor_list_bytes(-1) == 0
    for count in (1, 4, 5, 1000):
        assert _lib.ds_tensor_list_bytes(count) == 64 * 128 + -(-4 * count // 16) * 16 + 96 * count


def test_an_empty_list_is_written_without_a_launch():
    lst = DsTensorList(table=1, tiles=2, elems=3, count=4, sdt=5)
    assert L.ds_tensor_list_write(ctypes.byref(lst), None, 0, None, 0, DS_FP32, None) == DS_OK
    assert (lst.table, lst.tiles, lst.elems, lst.count, lst.sdt) == (None, 0, 0, 0, DS_FP32)
    assert _lib.ds_tensor_list_workspace_bytes(lst) == 0


@fake
def test_write_refusals():
    one = [tensor()]
    assert write(one, out=False) == DS_ERR_NULL
    assert write(one, table=None) == DS_ERR_NULL
    assert L.ds_tensor_list_write(ctypes.byref(DsTensorList()), TABLE, BIG, None, 1, DS_FP32, None) == DS_ERR_NULL
    assert L.ds_tensor_list_write(ctypes.byref(DsTensorList()), TABLE, BIG, None, -1, DS_FP32, None) == DS_ERR_SIZE
    assert L.ds_tensor_list_write(ctypes.byref(DsTensorList()), TABLE, 1 << 40, None, (1 << 20) + 1, DS_FP32,
                                  None) == DS_ERR_SIZE
    assert write(one, nbytes=_lib.ds_tensor_list_bytes(1) - 1) == DS_ERR_SIZE
    assert write(one, table=TABLE + 8) == DS_ERR_ALIGN
    for sdt in (0, DS_FP16, DS_BF16, 5):
        assert write(one, sdt=sdt) == DS_ERR_DTYPE
    for n in (-1, (1 << 40) + 1):
        assert write([tensor(n=n)]) == DS_ERR_SIZE
    assert write([tensor(n=1 << 39), tensor(0x90000000, n=(1 << 39) + 1)]) == DS_ERR_SIZE


@fake
@pytest.mark.parametrize("field", ["master", "p16", "m", "v", "grad"])
def test_null_and_misaligned_arrays(field):
    assert write([tensor(**{field: None})]) == DS_ERR_NULL
    assert write([tensor(**{field: getattr(tensor(), field) + 1})]) == DS_ERR_ALIGN
    assert write([tensor(), tensor(0x90000000, **{field: None})]) == DS_ERR_NULL


@fake
def test_type_and_hyperparameter_refusals():
    assert write([tensor(pdt=DS_FP8)]) == DS_ERR_DTYPE and write([tensor(pdt=0)]) == DS_ERR_DTYPE
    assert write([tensor(gdt=DS_FP8)]) == DS_ERR_DTYPE and write([tensor(gdt=9)]) == DS_ERR_DTYPE
    assert write([tensor(pdt=DS_FP32)]) == DS_ERR_HPARAM                    # a copy beside fp32 parameters
    assert write([tensor(m_scale=0x5000000000)]) == DS_ERR_HPARAM           # scales of 32-bit states
    for bad in (-1.0, float("nan"), float("inf")):
        assert write([tensor(weight_decay=bad)]) == DS_ERR_HPARAM
        assert write([tensor(lr_scale=bad)]) == DS_ERR_HPARAM
    for field in ("m_scale", "v_scale"):
        assert write([tensor8(**{field: None})], DS_FP8) == DS_ERR_NULL
        assert write([tensor8(**{field: 0x5000000002})], DS_FP8) == DS_ERR_ALIGN


@fake
def test_alias_refusals():
    a = tensor()
    step = 1 << 24
    for field in ("master", "p16", "m", "v"):
        for other in ("master", "p16", "m", "v", "grad"):
            if field != other:   # the last element of one inside the other
                assert write([tensor(**{field: getattr(a, other) + 1996 // 4 * 4})]) == DS_ERR_ALIAS, (field, other)
    assert write([a, tensor()]) == DS_ERR_ALIAS
    assert write([a, tensor(0x90000000, grad=a.m)]) == DS_ERR_ALIAS
    assert write([tensor(master=TABLE + 16)]) == DS_ERR_ALIAS
    assert write([tensor(grad=TABLE + 16)]) == DS_ERR_ALIAS
    # a long gradient that starts before and reaches into a later tensor's state, past other ranges
    assert write([tensor(n=4), tensor(0x90000000, n=4, grad=0x90000000 + 2 * step + 8)]) == DS_ERR_ALIAS
    assert write([tensor8(m_scale=a.grad)], DS_FP8) == DS_ERR_ALIAS


@fake
def test_step_and_check_refusals():
    lst = DsTensorList(table=TABLE, tiles=1, elems=1000, count=1, sdt=DS_FP32)
    by = ctypes.byref
    hp = (1e-3, None, 0.9, 0.999, 1e-8, 0.0, 1, 0, 0, 1, None)

    def adam(lst_=lst, st=ST, **kw):
        names = ("lr", "sched", "b1", "b2", "eps", "clip", "K", "rounding", "seed", "end", "stream")
        args = dict(zip(names, hp))
        args.update(kw)
        return L.ds_adam_step_list(st, by(lst_) if lst_ is not None else None, *args.values())

    assert adam(None) == DS_ERR_NULL and adam(st=None) == DS_ERR_NULL
    assert adam(st=ST + 4) == DS_ERR_ALIGN and adam(st=TABLE) == DS_ERR_ALIAS
    for kw in (dict(lr=-1.0), dict(lr=float("nan")), dict(b1=1.0), dict(b2=-0.1), dict(eps=0.0), dict(clip=-1.0),
               dict(K=0), dict(rounding=2), dict(sched=by(_lib.DsLrSchedule.make(9, 0, 1, 1)))):
        assert adam(**kw) == DS_ERR_HPARAM, kw
    check = L.ds_check_overflow_list
    assert check(ST, None, None, 0, None) == DS_ERR_NULL and check(None, by(lst), None, 0, None) == DS_ERR_NULL
    assert check(ST + 4, by(lst), None, 0, None) == DS_ERR_ALIGN
    assert check(ST, by(lst), 0x500000004, 1 << 20, None) == DS_ERR_ALIGN
    assert check(ST, by(lst), 0x500000000, 15, None) == DS_ERR_SIZE
    assert check(ST, by(lst), TABLE, 1 << 20, None) == DS_ERR_ALIAS
    assert check(ST, by(lst), ST + 64, 1 << 20, None) == DS_ERR_ALIAS
    for kw in (dict(table=None), dict(count=-1), dict(tiles=5), dict(tiles=0), dict(elems=-1), dict(elems=0),
               dict(elems=(1 << 40) + 1), dict(sdt=0), dict(count=(1 << 20) + 1)):
        bad = DsTensorList(**{**dict(table=TABLE, tiles=1, elems=1000, count=1, sdt=DS_FP32), **kw})
        want = (DS_ERR_NULL if "table" in kw else DS_ERR_DTYPE if "sdt" in kw else DS_ERR_SIZE,)
        assert check(ST, by(bad), None, 0, None) in want and adam(bad) in want, kw
        assert _lib.ds_tensor_list_workspace_bytes(bad) == 0
    empty = DsTensorList(sdt=DS_FP32)
    assert check(ST, by(empty), None, 0, None) == DS_OK and adam(empty, end=0) == DS_OK
    assert _lib.ds_tensor_list_workspace_bytes(lst) == 16


def test_fp8_is_refused_everywhere_else():
    assert L.ds_check_overflow(ST, TABLE, DS_FP8, 0, None) == DS_ERR_DTYPE
    assert L.ds_accumulate(ST, TABLE, DS_FP8, 0, 1, None, None) == DS_ERR_DTYPE


def test_class_refusals_on_host_tensors():
    cfg = ZeroMPConfig(bf16=True)
    for p in (torch.zeros(4), torch.zeros(4, dtype=torch.int32), torch.zeros(4, dtype=torch.float16),
              torch.zeros(4, 4)[:, 0]):
        with pytest.raises(ValueError):
            MultiTensorStep([p], cfg)
    for kw in (dict(states="int8"), dict(dither_seed=1), dict(weight_decay=[0.1, 0.2]), dict(lr_scale=[])):
        with pytest.raises(ValueError):
            MultiTensorStep([torch.zeros(4)], cfg, **kw)
    assert per_tensor(None, 0.5, 2, "x") == [0.5, 0.5] and per_tensor([1, 2], 0, 2, "x") == [1.0, 2.0]


def test_reference_formats_are_torchs():
    codes = np.arange(256, dtype=np.uint8)
    for fmt, kind in ((ref.E4M3, torch.float8_e4m3fn), (ref.E5M2, torch.float8_e5m2)):
        want = torch.from_numpy(codes).view(kind).double().numpy()
        want = np.where(np.isinf(want), np.nan, want)       # the reference holds no infinities
        np.testing.assert_array_equal(fmt.decode(codes), want)
        vals = want[:128][np.isfinite(want[:128])]
        for u in (0.0, 0.5, 1 - 2.0 ** -20):
            np.testing.assert_array_equal(fmt.quantise(vals, u), vals)     # a code's value is kept
        mid = (vals[1:] + vals[:-1]) / 2
        np.testing.assert_array_equal(fmt.quantise(mid, 0.5), vals[1:])
        np.testing.assert_array_equal(fmt.quantise(mid, 0.49), vals[:-1])


def test_reference_dither_is_even():
    """Over the steps an element's dither is spread evenly (deviation of a mean of 4000 uniforms: 0.0046; 5 of them)."""
    um, ur = zip(*(ref.dither(7, t, 3, 600) for t in range(1, 4001)))
    for u in (np.array(um), np.array(ur)):
        assert np.all(np.abs(u.mean(0) - 0.5) < 0.024)
        assert 0 <= u.min() and u.max() < 1
    assert abs(np.corrcoef(np.array(um)[:, 5], np.array(ur)[:, 5])[0, 1]) < 0.1
