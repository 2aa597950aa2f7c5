"""One workspace through calls of different sizes: one block, some that meet in one kernel, many with a second one."""
import pytest
import torch

from tests.test_gpu_balance import check, logits
from zero_mixed_precision_amd import ExpertBalance

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,k", [(1, 1), (8, 2), (33, 4), (64, 8), (64, 16), (65, 4), (130, 8), (300, 3)])
def test_sizes_in_turn(n, k):
    """32 tokens a block up to 128 experts: 4096 tokens are 128 blocks, 4097 are 129."""
    op = ExpertBalance(n, k, 0.1)
    for T in (33, 4096, 1, 4097, 0, 64, 9000, 1000, 33):
        check(op, logits(T, n, "bf16", seed=T), "bf16")
        torch.cuda.synchronize()
        assert int(op._ws.view(torch.int32)[64]) == 0       # the count of finished blocks, behind 32 parts of the loss


def test_replays_between_calls_of_other_sizes():
    small, large = logits(500, 64, "bf16"), logits(4096, 64, "bf16", seed=1)
    op, eager = ExpertBalance(64, 8, 0.1), ExpertBalance(64, 8, 0.1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op.loss(large)
    for seed in range(4):
        large.copy_(logits(4096, 64, "bf16", seed=seed))
        op.loss(small)
        torch.cuda.synchronize()
        graph.replay()
        eager.loss(large)
        torch.cuda.synchronize()
        for a, b in ((op.value, eager.value), (op.counts, eager.counts), (op.mean_prob, eager.mean_prob),
                     (op.used, eager.used)):
            assert torch.equal(a, b)
