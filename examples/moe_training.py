"""A small mixture-of-experts layer trained in mixed precision with the step over a list of tensors.

    python examples/moe_training.py [--steps 200] [--states fp8|fp32] [--half fp16|bf16]

One layer routes each token to k of E experts and learns a random teacher.  PyTorch runs the router's and the experts'
products forward and backward; the framework does the rest on the device (the host reads where each expert's rows start, so
that PyTorch can take them):

  * ExpertDispatch: the tokens' rows in expert order, the experts' outputs weighted and summed for each token, and the
    gradients of both moves, as steps of the backward pass;
  * ExpertBalance: counts per expert, the balance loss, and its loss-scaled gradient by the router's logits, which joins
    the backward pass;
  * MultiTensorStep: overflow check and joint norm over all parameters' gradients, AdamW with states in 8 bits (or 32),
    the loss scaler.  The experts' biases take no decay.
"""
import argparse

import torch

from zero_mixed_precision_amd import ExpertBalance, ExpertDispatch, MultiTensorStep, ZeroMPConfig


class Gather(torch.autograd.Function):
    """Tokens' rows [T, D] in expert order [T * k, D]."""

    @staticmethod
    def forward(ctx, x, dispatch):
        ctx.dispatch, ctx.sorts = dispatch, dispatch.sorts
        return dispatch.gather(x, x.new_zeros(x.shape[0] * dispatch.k, x.shape[1]))

    @staticmethod
    def backward(ctx, drows):
        ctx.dispatch.check_sort(ctx.sorts)
        dx = drows.new_empty(drows.shape[0] // ctx.dispatch.k, drows.shape[1])
        return ctx.dispatch.gather_gradient(drows.contiguous(), dx), None


class Combine(torch.autograd.Function):
    """The experts' rows [T * k, D], weighted and summed for each token [T, D]."""

    @staticmethod
    def forward(ctx, rows, gates, dispatch):
        ctx.dispatch, ctx.sorts = dispatch, dispatch.sorts
        ctx.save_for_backward(rows, gates)
        return dispatch.combine(rows, gates, rows.new_empty(gates.shape[0], rows.shape[1]))

    @staticmethod
    def backward(ctx, dy):
        ctx.dispatch.check_sort(ctx.sorts)
        rows, gates = ctx.saved_tensors
        return *ctx.dispatch.combine_gradient(dy.contiguous(), rows, gates, torch.zeros_like(rows),
                                              torch.empty_like(gates)), None


class MoELayer:
    """x [T, D] -> sum over the k chosen experts of gate * expert(x); parameters are 16-bit leaf tensors."""

    def __init__(self, width, hidden, experts, k, half, gen, device, tokens):
        def leaf(*shape, sigma):
            w = torch.randn(*shape, generator=gen, device=device) * sigma
            return w.to(half).requires_grad_()

        self.k = k
        self.dispatch = ExpertDispatch(experts, k, tokens, device=device)
        self.router = leaf(experts, width, sigma=0.02)
        self.up = [leaf(hidden, width, sigma=width ** -0.5) for _ in range(experts)]
        self.up_bias = [leaf(hidden, sigma=0.0) for _ in range(experts)]
        self.down = [leaf(width, hidden, sigma=hidden ** -0.5) for _ in range(experts)]

    def parameters(self):
        return [self.router, *self.up, *self.up_bias, *self.down]

    def __call__(self, x):
        logits = x @ self.router.t()
        gates, chosen = torch.softmax(logits.float(), 1).topk(self.k, dim=1)
        gates = (gates / gates.sum(1, keepdim=True)).to(x.dtype)
        starts = self.dispatch.sort(chosen).tolist()
        rows = Gather.apply(x, self.dispatch)
        parts = [torch.nn.functional.silu(rows[lo:hi] @ up.t() + bias) @ down.t()
                 for lo, hi, up, bias, down in zip(starts, starts[1:], self.up, self.up_bias, self.down)]
        out = Combine.apply(torch.cat(parts), gates, self.dispatch)
        return out, logits


def train(steps=200, states="fp8", half="fp16", tokens=512, width=64, hidden=128, experts=8, k=2, seed=0, report=None):
    """Returns the losses (a list of floats, read once at the end), the last counts per expert and the optimizer step."""
    device = torch.device("cuda:0")
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    dtype = torch.float16 if half == "fp16" else torch.bfloat16
    layer = MoELayer(width, hidden, experts, k, dtype, gen, device, tokens)
    teacher = torch.randn(width, width, generator=gen, device=device) * width ** -0.5
    params = layer.parameters()
    cfg = ZeroMPConfig(bf16=half == "bf16", initial_scale_power=12, loss_scale_window=100, lr=2e-3, weight_decay=0.01,
                       gradient_clipping=1.0)
    step = MultiTensorStep(params, cfg, states=states, dither_seed=seed if states == "fp8" else None,
                           weight_decay=[0.0 if p.dim() == 1 else 0.01 for p in params])
    balance = ExpertBalance(experts, k, coef=0.1)
    for p in params:
        p.grad = torch.zeros_like(p)            # gradients keep their addresses: one table for the whole run
    step.set_gradients([p.grad for p in params])
    losses = []
    for n in range(steps):
        x = torch.randn(tokens, width, generator=gen, device=device)
        target = torch.tanh(x @ teacher)
        y, logits = layer(x.to(dtype))
        loss = (y.float() - target).square().mean()
        aux = balance.loss(logits.detach())
        dlogits = balance.gradient(logits.detach(), torch.empty_like(logits), scaler=step.state)
        torch.autograd.backward([loss * step.loss_scale, logits], [None, dlogits])
        step.step()
        torch._foreach_zero_([p.grad for p in params])
        losses.append((loss + aux).detach())
        if report and (n + 1) % 50 == 0:
            report(f"step {n + 1}: loss {float(losses[-1]):.4f}, balance {float(aux):.4f}, counts "
                   f"{balance.counts.tolist()}, scale {step.scaler().scale:g}")
    return torch.stack(losses).tolist(), balance.counts.tolist(), step


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--states", choices=("fp8", "fp32"), default="fp8")
    ap.add_argument("--half", choices=("fp16", "bf16"), default="fp16")
    a = ap.parse_args()
    train(a.steps, a.states, a.half, report=lambda s: print(s, flush=True))
