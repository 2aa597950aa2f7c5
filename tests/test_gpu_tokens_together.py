"""The operators of a training step with experts together: router and balance loss, tokens to the experts and back, cross
entropy over the vocabulary, distillation of the same hidden states, all gradients under one loss scale, and the step over
the parameters.  Gradients against torch's own in fp64 from the same 16-bit parameters."""
import importlib.util
import os

import pytest
import torch

from zero_mixed_precision_amd import (ExpertBalance, ExpertDispatch, MultiTensorStep, TopLogitDistillation,
                                      VocabCrossEntropy, ZeroMPConfig)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
T, D, E, K, V, N = 384, 96, 8, 2, 1200, 12           # tokens, width, experts, choices, vocabulary, teacher's entries
COEF, TAU = 0.05, 2.0


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_training.py")
    spec = importlib.util.spec_from_file_location("moe_training", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def data(dtype, seed=0):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def leaf(*shape, sigma):
        return (torch.randn(*shape, generator=gen, device=DEV) * sigma).to(dtype)

    params = [leaf(E, D, sigma=0.3), *[leaf(D, D, sigma=D ** -0.5) for _ in range(E)], leaf(V, D, sigma=D ** -0.5)]
    x = leaf(T, D, sigma=1.0)
    targets = torch.randint(V, (T,), generator=gen, device=DEV)
    mask = torch.rand(T, generator=gen, device=DEV) < 0.85
    teacher = torch.randn(T, N, generator=gen, device=DEV) * 2
    index = torch.rand(T, V, generator=gen, device=DEV).topk(N, dim=1).indices
    return params, x, targets, mask, teacher, index


def reference(params, x, targets, mask, teacher, index, chosen):
    """All losses and the gradients of their sum in fp64, with the router's choices given (they have no gradient)."""
    leaves = [p.double().requires_grad_() for p in params]
    router, experts, head = leaves[0], leaves[1:-1], leaves[-1]
    x = x.double()
    z = x @ router.t()
    p = torch.softmax(z, 1)
    gates = p.gather(1, chosen)
    gates = gates / gates.sum(1, keepdim=True)
    each = torch.stack([x @ w.t() for w in experts], 1)          # [T, E, D]
    h = x + (gates[..., None] * each.gather(1, chosen[..., None].expand(-1, -1, D))).sum(1)
    f = torch.bincount(chosen[mask].flatten(), minlength=E).double() / (int(mask.sum()) * K)
    balance = COEF * E * (f * p[mask].mean(0)).sum()
    logits = h @ head.t()
    ce = torch.nn.functional.cross_entropy(logits[mask], targets[mask])
    q = torch.softmax(teacher.double() / TAU, 1)
    log_p = torch.log_softmax(logits / TAU, 1).gather(1, index)
    kl = (q * (q.log() - log_p)).sum(1)[mask].mean() * TAU ** 2
    grads = torch.autograd.grad(balance + ce + kl, leaves)
    return [float(v.detach()) for v in (balance, ce, kl)], grads


@pytest.mark.parametrize("dtype,scale", [(torch.float16, 256.0), (torch.bfloat16, 1.0)])
def test_one_step(dtype, scale):
    params, x, targets, mask, teacher, index = data(dtype)
    leaves = [p.clone().requires_grad_() for p in params]
    router, experts, head = leaves[0], leaves[1:-1], leaves[-1]
    cfg = ZeroMPConfig(bf16=dtype == torch.bfloat16, loss_scale=scale, lr=1e-3)
    step = MultiTensorStep([p.data for p in leaves], cfg)
    ex = example()
    balance, dispatch = ExpertBalance(E, K, COEF), ExpertDispatch(E, K, T)
    ce = VocabCrossEntropy(V, D, T, dtype)
    distill = TopLogitDistillation(V, N, T, temperature=TAU)

    z = x @ router.t()
    gates, chosen = torch.softmax(z.float(), 1).topk(K, dim=1)
    gates = gates / gates.sum(1, keepdim=True)
    starts = dispatch.sort(chosen).tolist()
    rows = ex.Gather.apply(x, dispatch)
    out = torch.cat([rows[lo:hi] @ w.t() for lo, hi, w in zip(starts, starts[1:], experts)])
    h = x + ex.Combine.apply(out, gates, dispatch)
    logits = h @ head.t()
    dz, dh, dhead = (torch.empty_like(a) for a in (z, h, head))
    losses = [balance.loss(z.detach(), mask=mask).clone()]
    balance.gradient(z.detach(), dz, mask=mask, scaler=step.state)
    losses.append(ce.loss_and_gradient(h.detach(), head.detach(), targets, dh, dhead, mask=mask, scaler=step.state))
    dlogits = logits.detach().clone()                            # the gradient in the logits' place
    losses.append(distill.loss_and_gradient(dlogits, teacher, index, dlogits, mask=mask, scaler=step.state))
    torch.autograd.backward([z, h, logits], [dz, dh, dlogits])
    head.grad += dhead
    step.set_gradients([p.grad for p in leaves])
    before = [p.detach().clone() for p in leaves]
    step.step()

    want, grads = reference(params, x, targets, mask, teacher, index, chosen)
    half = torch.finfo(dtype).eps / 2
    # a loss goes through four values rounded to 16 bits one after another (expert's output, combined row, hidden state,
    # for the distillation the logits), a gradient through their like on the way back as well, each off by half a step of
    # its own at most; these are sums of many, whose roundings do not add up in one direction: whole norms, 8 half steps
    for got, w in zip(losses, want):
        assert abs(float(got) - w) <= 8 * half * max(1.0, abs(w))
    for p, g in zip(leaves, grads):
        assert float((p.grad.double() / scale - g).norm() / g.norm()) <= 8 * half
    assert int(ce.used) == int(distill.used) == int(balance.used) == int(mask.sum())
    assert step.scaler().step == 1 and step.scaler().overflow == 0
    assert all(not torch.equal(a, p.detach()) for a, p in zip(before, leaves))


def test_an_overflow_of_any_loss_skips_the_step():
    """A row with an infinite logit: its gradient is not finite, the step changes nothing and the scale falls."""
    params, x, targets, mask, _, _ = data(torch.float16)
    head = params[-1]
    cfg = ZeroMPConfig(initial_scale_power=8, hysteresis=1, lr=1e-3)
    dhead = torch.empty_like(head)
    step = MultiTensorStep([head], cfg)
    step.set_gradients([dhead])
    ce = VocabCrossEntropy(V, D, T, torch.float16)
    x[3] = float("inf")
    mask[3] = True
    before = head.clone()
    ce.loss_and_gradient(x, head, targets, None, dhead, mask=mask, scaler=step.state)
    step.step()
    sc = step.scaler()
    assert torch.equal(head, before) and sc.step == 0 and sc.skipped == 1 and sc.scale == 128.0
    mask[3] = False                                              # left out, it reaches nothing
    ce.loss_and_gradient(x, head, targets, None, dhead, mask=mask, scaler=step.state)
    step.step()
    assert step.scaler().step == 1 and not torch.equal(head, before)


def test_the_example_and_its_layers_gradients():
    ex = example()
    losses, counts, step = ex.train(steps=5, tokens=128)
    assert len(losses) == 5 and sum(counts) == 128 * 2 and step.scaler().iter == 5
    gen = torch.Generator(device=DEV)
    gen.manual_seed(3)
    layer = ex.MoELayer(32, 48, 4, 2, torch.bfloat16, gen, DEV, 100)
    x = torch.randn(100, 32, generator=gen, device=DEV).bfloat16().requires_grad_()
    dy = torch.randn(100, 32, generator=gen, device=DEV).bfloat16()
    y, logits = layer(x)
    y.backward(dy)
    leaves = [p.detach().double().requires_grad_() for p in (x, *layer.parameters())]
    xd, router, rest = leaves[0], leaves[1], leaves[2:]
    up, bias, down = rest[:4], rest[4:8], rest[8:]
    chosen = torch.softmax(logits.detach().float(), 1).topk(2, dim=1).indices
    g = torch.softmax(xd @ router.t(), 1).gather(1, chosen)
    g = g / g.sum(1, keepdim=True)
    each = torch.stack([torch.nn.functional.silu(xd @ u.t() + b) @ d.t() for u, b, d in zip(up, bias, down)], 1)
    want = (g[..., None] * each.gather(1, chosen[..., None].expand(-1, -1, 32))).sum(1)
    grads = torch.autograd.grad((want * dy.double()).sum(), leaves)
    # whole norms: some eight values rounded to 16 bits on the way there and back
    assert float((y.detach().double() - want).norm() / want.norm()) <= 8 * 2.0 ** -8
    for p, w in zip((x, *layer.parameters()), grads):
        assert float((p.grad.double() - w).norm() / w.norm()) <= 8 * 2.0 ** -8


def test_the_binding_gives_the_classes_results():
    """The entry points under their C names, with strided tensors, against the classes."""
    from zero_mixed_precision_amd import _lib

    params, x, targets, mask, teacher, index = data(torch.bfloat16)
    head, bf, f32 = params[-1], _lib.DS_BF16, _lib.DS_FP32
    ce = VocabCrossEntropy(V, D, T, torch.bfloat16, coef=0.5)
    dx, dhead = torch.empty_like(x), torch.empty_like(head)
    ce.loss_and_gradient(x, head, targets, dx, dhead, mask=mask)
    token_loss, loss, used = (torch.empty(n, dtype=d, device=DEV) for n, d in ((T, torch.float32), (1, torch.float32),
                                                                              (1, torch.int32)))
    ws = torch.empty(_lib.ds_vocab_ce_workspace_bytes(T, V, D), dtype=torch.uint8, device=DEV)
    wide, dx2, dhead2 = torch.cat([x, x], 1)[:, :D], torch.empty_like(x), torch.empty_like(head)
    _lib.ds_vocab_ce(None, wide, 2 * D, head, D, bf, targets, 8, T, V, D, mask, 0.5, token_loss, loss, used, dx2, D, dhead2, bf,
                     D, False, ws)
    assert torch.equal(dx, dx2) and torch.equal(dhead, dhead2) and torch.equal(loss[0], ce.value)

    logits = x @ head.t()
    distill = TopLogitDistillation(V, N, T, temperature=TAU)
    d, d2 = torch.empty_like(logits), torch.empty_like(logits)
    distill.loss_and_gradient(logits, teacher, index, d, mask=mask)
    ws = torch.zeros((_lib.ds_distill_workspace_bytes(T) + 7) // 8, dtype=torch.float64, device=DEV)
    _lib.ds_distill_loss(None, logits, bf, T, V, V, teacher, f32, N, index, 8, N, N, mask, TAU, 1.0, token_loss, loss, used, d2,
                         V, False, ws)
    assert torch.equal(d, d2) and torch.equal(loss[0], distill.value)

    chosen = index[:, :K] % E
    op = ExpertDispatch(E, K, T)
    offsets = op.sort(chosen)
    rows, y, gates = torch.zeros(T * K, D, dtype=x.dtype, device=DEV), torch.empty_like(x), torch.rand(T, K, device=DEV)
    op.gather(x, rows)
    op.combine(rows, gates, y)
    drows, dgates = op.combine_gradient(x, rows, gates, torch.zeros_like(rows), torch.empty_like(gates))
    dx = op.gather_gradient(rows, torch.empty_like(x))
    ints = lambda n: torch.empty(n, dtype=torch.int32, device=DEV)  # noqa: E731
    o2, place, source, ws = ints(E + 1), ints(T * K), ints(T * K), ints(_lib.ds_dispatch_workspace_bytes(T, E, K) // 4)
    r2, y2, dr2, dg2, dx2 = (torch.zeros_like(a) for a in (rows, y, drows, dgates, dx))
    strided = index[:, :K] % E
    wide = torch.cat([strided, strided], 1)
    _lib.ds_dispatch_sort(wide[:, :K], 8, T, E, K, 2 * K, o2, place, source, ws)
    _lib.ds_dispatch_gather(x, bf, T, K, D, D, place, r2, D, T * K)
    _lib.ds_dispatch_combine(r2, bf, T, K, D, D, T * K, place, gates, f32, K, y2, D)
    _lib.ds_dispatch_combine_grad(x, bf, T, K, D, D, r2, D, T * K, place, gates, f32, K, dr2, D, dg2, K)
    _lib.ds_dispatch_gather_grad(r2, bf, T, K, D, D, T * K, place, dx2, D)
    for a, b in ((offsets, o2), (op.place.view(-1), place), (op.source, source), (rows, r2), (y, y2), (drows, dr2),
                 (dgates, dg2), (dx, dx2)):
        assert torch.equal(a, b)
    for bad in (lambda: _lib.ds_dispatch_gather(x.cpu(), bf, T, K, D, D, place, r2, D, T * K),
                lambda: _lib.ds_dispatch_sort(wide[:, :K], 8, T, E, K, K, o2, place, source, ws),
                lambda: _lib.ds_distill_loss(None, logits, bf, T, V + 1, V + 1, teacher, f32, N, index, 8, N, N, mask, TAU, 1.0,
                                             token_loss, loss, used, None, 0, False, ws),
                lambda: _lib.ds_vocab_ce(None, x, D, head, D, bf, targets.int(), 8, T, V, D, mask, 0.5, token_loss, loss, used,
                                         dx2, D, None, bf, 0, False, ws)):
        with pytest.raises(ValueError):
            bad()
