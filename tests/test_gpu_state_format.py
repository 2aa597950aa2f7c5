"""What the 8-bit states hold at the edges of their format, and how far the parameter may be from 32-bit arithmetic."""
import pytest
import torch

from tests import list_ref as ref
from tests.test_gpu_tensor_list import cfg
from zero_mixed_precision_amd import MultiTensorStep

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def one_step(g, states, dither_seed=None, **kw):
    p = torch.full_like(g, 0.5)
    op = MultiTensorStep([p], cfg(**kw), states=states, dither_seed=dither_seed)
    op.set_gradients([g])
    op.step()
    torch.cuda.synchronize()
    return op, p


@pytest.mark.parametrize("seed", [None, 3])
@pytest.mark.parametrize("n", [256, 700, 4096])
def test_a_block_below_the_smallest_top(n, seed):
    """v = 0.001 g^2 below 2^-110: scale 0; code 1 where v is positive, 0 where it is 0; both stand for 0."""
    g = torch.full((n,), 2.0 ** -52, device=DEV)
    g[::3] = 0.0
    op, _ = one_step(g, "fp8", seed)
    codes = op.view(op.v, 0).view(torch.uint8)
    assert bool((op.v_scale == 0).all()) and codes.tolist() == [0 if i % 3 == 0 else 1 for i in range(n)]
    assert bool((op.moments(0)[1] == 0).all())
    assert float(op.m_scale.min()) > 0                   # m, 0.1 g, is in range
    g.fill_(2.0 ** -120)                                 # 0.1 g below it too
    op, _ = one_step(g, "fp8", seed)
    assert bool((op.m_scale == 0).all()) and bool((op.view(op.m, 0).view(torch.uint8) == 0).all())


@pytest.mark.parametrize("eps", [1e-8, 1e-30])
def test_the_first_step_is_within_a_few_units_of_32_bit_states(eps):
    """From zero states both forms see the same m and v.  Root and reciprocal are within a unit (2 E) each, the forms'
    other roundings of the quotient's parts six (E each) on either side; p's own, of 0.5 and less, two on either side."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(4)
    g = torch.randn(10000, generator=gen, device=DEV) * torch.exp2(torch.randint(-30, 10, (10000,), generator=gen,
                                                                                device=DEV).float())
    (_, p), (_, q) = (one_step(g, states, eps=eps) for states in ("fp8", "fp32"))
    moved = 1e-3                                         # lr: what a first step moves an element by
    assert float((p.double() - q.double()).abs().max()) <= moved * (2 * 2 + 2 * 6) * ref.E + 4 * ref.E * 0.51
