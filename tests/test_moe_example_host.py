"""The mixture-of-experts example's steps of the backward pass without a GPU: over an ExpertDispatch whose moves are torch's."""
import importlib.util
import os

import pytest
import torch

from tests.stand_in import Library, Tensor, Torch
from zero_mixed_precision_amd import ExpertDispatch, _lib


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_training.py")
    spec = importlib.util.spec_from_file_location("moe_training", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


class Plain(ExpertDispatch):
    """Every choice is there; rows in the order of a stable sort."""

    def __init__(self, k):
        self.k = k

    def sort(self, chosen):
        order = torch.sort(chosen.flatten(), stable=True).indices
        self.place = torch.empty_like(order)
        self.place[order] = torch.arange(len(order))
        self.sorts += 1

    def gather(self, x, out):
        out[self.place] = x.repeat_interleave(self.k, 0)
        return out

    def gather_gradient(self, dout, dx):
        return dx.copy_(dout[self.place].view(-1, self.k, dout.shape[1]).sum(1))

    def combine(self, rows, gates, out):
        return out.copy_((rows[self.place].view(-1, self.k, rows.shape[1]) * gates[..., None]).sum(1))

    def combine_gradient(self, dout, rows, gates, drows, dgates):
        drows[self.place] = (dout[:, None] * gates[..., None]).flatten(0, 1)
        dgates.copy_((rows[self.place].view(-1, self.k, rows.shape[1]) * dout[:, None]).sum(2))
        return drows, dgates


def test_a_backward_pass_after_another_sort_is_refused():
    ex, gen = example(), torch.Generator().manual_seed(1)
    T, k, D = 12, 2, 5
    dispatch = Plain(k)

    def forward(seed):
        x = torch.randn(T, D, generator=gen, requires_grad=True)
        gates = torch.rand(T, k, generator=gen, requires_grad=True)
        dispatch.sort(torch.randint(4, (T, k), generator=torch.Generator().manual_seed(seed)))
        rows = ex.Gather.apply(x, dispatch)
        return x, gates, rows, ex.Combine.apply(rows * 3, gates, dispatch)

    x, gates, _, y = forward(1)
    y.sum().backward()                                    # y = 3 x times the sum of the gates
    assert torch.allclose(x.grad, 3 * gates.sum(1, keepdim=True).expand(T, D))
    assert torch.allclose(gates.grad, 3 * x.sum(1, keepdim=True).expand(T, k), atol=1e-5)
    x, gates, rows, y = forward(1)
    forward(2)
    for out in (y, rows):
        with pytest.raises(RuntimeError, match="sorted 1 more time"):
            out.sum().backward(retain_graph=True)
    assert x.grad is None and gates.grad is None


def test_sorts_are_counted(monkeypatch):
    fake = Torch()
    monkeypatch.setattr(_lib, "lib", Library(fake))
    monkeypatch.setattr(_lib, "_raw_stream", lambda i: 0x100)
    op = ExpertDispatch.__new__(ExpertDispatch)
    op.torch, op.stream, op._device, op._many, op.device = fake, None, 0, False, torch.device("cuda", 0)
    op.E, op.k, op.tokens, op.max_tokens, op.offsets = 64, 8, 0, 100, None
    op._at, op._index_types = (1, 2, 3, 9, 64), (torch.int32, torch.int64)
    before = op.sorts
    op.check_sort(before)
    op.sort(Tensor(9, 8, dtype=torch.int32))
    op.check_sort(before + 1)
    with pytest.raises(RuntimeError):
        op.check_sort(before)
    with pytest.raises(ValueError):
        op.sort(Tensor(101, 8, dtype=torch.int32))
    op.check_sort(before + 1)                             # a refused call sorts nothing
    assert ExpertDispatch.sorts == 0
