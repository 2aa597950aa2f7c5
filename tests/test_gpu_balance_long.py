"""Mean probabilities and the loss over so many tokens that a block's lanes add up hundreds and thousands of rows.

Each sum's error is bounded without regard to the number of tokens: rounding of a probability (as in test_gpu_balance.py),
64 additions in a lane, 16 rows and a neighbour in a block, then fp64, then two roundings to fp32."""
import numpy as np
import pytest
import torch

from zero_mixed_precision_amd import ExpertBalance

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E32 = 2.0 ** -24
SUMS = 64 + 16 + 1 + 3


def test_equal_rows():
    """2^28 rows alike: every addition of a lane rounds to the same side while its sum is in one binade."""
    row = torch.tensor([0.5, -1.0, 1.25, 0.0, 2.0, -0.75, 1.0, -2.0], dtype=torch.bfloat16, device=DEV)
    T = (1 << 28) + 12345
    z = row.expand(T, 8).contiguous()
    op = ExpertBalance(8, 2, 0.5)
    loss = float(op.loss(z))
    x = row.double().cpu().numpy()
    p = np.exp(x) / np.exp(x).sum()
    bound = (2 * (3 * 4 + 2) + 38 + SUMS) * E32          # logits at most 4 below the largest
    mean = op.mean_prob.double().cpu().numpy()
    assert int(op.used) == T and op.counts.tolist() == [0, 0, T, 0, T, 0, 0, 0]
    assert np.abs(mean / p - 1).max() <= bound, f"{np.abs(mean / p - 1).max() / E32:.0f} E"
    want = 0.5 * 8 * (p[2] + p[4]) / 2
    assert abs(loss / want - 1) <= bound + 4 * E32
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,n,k", [(2 * 64 * 1024 * 32 + 77, 8, 2), (64 * 1024 * 32 + 1, 64, 4), (64 * 1024 * 32, 33, 3),
                                   (3 * 64 * 1024 * 16 + 5, 130, 8), (700_001, 300, 16)])
@pytest.mark.parametrize("masked", [False, True])
def test_random_rows(T, n, k, masked):
    """Some sums of 64 turns and a rest, or none, for each number of lanes a row."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(n)
    z = torch.randn(T, n, generator=gen, device=DEV) + torch.randn(n, generator=gen, device=DEV)
    mask = torch.rand(T, generator=gen, device=DEV) < 0.8 if masked else None
    op = ExpertBalance(n, k, 0.5)
    loss = float(op.loss(z, mask=mask))
    mean, counts, far = torch.zeros(n, dtype=torch.float64, device=DEV), torch.zeros(n, dtype=torch.int64, device=DEV), 0.0
    for at in range(0, T, 1 << 20):
        x = z[at:at + (1 << 20)]
        rows = slice(None) if mask is None else mask[at:at + (1 << 20)]
        x = x[rows]
        if len(x) == 0:
            continue
        p = torch.softmax(x.double(), 1)
        mean += p.sum(0)
        far = max(far, float((x.amax(1) - x.amin(1)).max()))
        counts += torch.bincount(torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k].reshape(-1), minlength=n)
    used = T if mask is None else int(mask.sum())
    mean = (mean / used).cpu().numpy()
    assert int(op.used) == used and op.counts.tolist() == counts.tolist()
    bound = (2 * (3 * far + 2) + 38 + SUMS) * E32
    assert np.abs(op.mean_prob.double().cpu().numpy() / mean - 1).max() <= bound
    want = 0.5 * n * float(counts.double().cpu().numpy() / (k * used) @ mean)
    assert abs(loss / want - 1) <= bound + 4 * E32
    del z, x, p
    torch.cuda.empty_cache()
