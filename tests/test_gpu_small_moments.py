"""Second moments below fp32's smallest normal number, with an eps that does not hide them."""
import numpy as np
import pytest
import torch

from tests import list_ref as ref
from tests.test_gpu_tensor_list import check_step, cfg, snapshot
from zero_mixed_precision_amd import MultiTensorStep

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("eps", [1e-30, 1e-18, 1e-15, 1e-12, 1e-8])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("states", ["fp32", "fp8"])
def test_a_subnormal_second_moment_is_a_denominator(states, shift, eps):
    """0.001 g^2 from 2^-126 down to 2^-138, in whole tiles and odd ones, against 64 bits.  Without its root such an
    element would move by lr m / eps.  One element of each block keeps the block's scale in range."""
    n = 4096 + 300
    gen = torch.Generator(device=DEV)
    gen.manual_seed(6)
    grads = torch.exp2(-59.0 + torch.rand(n + shift, generator=gen, device=DEV) * 0.9 -
                       torch.randint(0, 6, (n + shift,), generator=gen, device=DEV)) * torch.where(
                           torch.rand(n + shift, generator=gen, device=DEV) < 0.5, -1.0, 1.0)
    grads = grads[shift:]
    grads[::256] = 1e-3
    params = [(torch.randn(n + shift, generator=gen, device=DEV) * 0.02)[shift:]]
    op = MultiTensorStep(params, cfg(eps=eps), states=states)
    op.set_gradients([grads])
    small = 0.001 * grads.double() ** 2
    assert int((small < 2.0 ** -126).sum()) > 4000 and float(small.min()) > 2.0 ** -141
    before = snapshot(op)
    op.step()
    check_step(op, before, 1, [0.0])
    if eps < 1e-20:      # and as a bound of its own: no element moves further than lr (1 - b1) / sqrt(1 - b2) at t = 1 ...
        moved = np.abs(params[0].double().cpu().numpy() - before[0]["master"].double().numpy())
        # ... over its bias corrections, lr, but for the resolution of a v of 2^-138 in units of 2^-149 and p's own
        assert moved.max() <= 1e-3 * (1 + 2.0 ** -7) + 4 * ref.E
