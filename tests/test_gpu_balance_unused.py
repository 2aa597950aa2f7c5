"""Rows that are not used have gradient 0, whatever they hold and however large the factor of the others is."""
import pytest
import torch

from tests.test_gpu_balance import logits
from zero_mixed_precision_amd import ExpertBalance, _lib

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("kind", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("n,k", [(8, 2), (60, 4), (256, 8), (300, 3)])
def test_a_factor_past_fp32(n, k, kind):
    """coef E S / T' above fp32's largest value."""
    st = torch.zeros(_lib.ds_scaler_size(), dtype=torch.uint8, device=DEV)
    _lib.ds_state_init(st, 65536.0, 1.0, 1000, 1)
    z = logits(70, n, kind)
    z[1] = float("-inf")
    mask = torch.ones(70, dtype=torch.bool, device=DEV)
    mask[::3] = False
    z[3], z[6] = float("nan"), float("inf")
    op = ExpertBalance(n, k, 3e38)
    op.loss(z, mask=mask)
    d = op.gradient(z, torch.full_like(z, 7.0), mask=mask, scaler=st)
    off = ~mask
    off[1] = True
    assert int((d[off] == 0).sum()) == int(off.sum()) * n
    assert not (d[~off].isfinite() & (d[~off] != 0)).any()
    out = torch.full_like(z, 7.0)
    assert bool((op.gradient(z, out, mask=mask, scaler=st, accumulate=True)[off] == 7).all())
