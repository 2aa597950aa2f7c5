"""Cases of the optimizer step over a list of tensors and of the experts' balance loss, for timing and for comparison.

Each case is one pass that a training program makes: a whole optimizer step (overflow check, the gradient's norm where it
is clipped, AdamW with states in 32 or in 8 bits, the scaler) or the balance loss of a router with its gradient.  ``run``
has two forms.  With ``own`` false it is elementary torch operations; with ``own`` true it is the framework's call.

The tensors of a step are views of flat storage, each starting on a multiple of 256 elements; the values between them are
zero and stay zero.
"""
import math

import torch

own = False

ALIGN = 256                      # elements: where a tensor starts, and the block that shares a scale in 8 bits
LR, BETA1, BETA2, EPS, DECAY = 1e-4, 0.9, 0.999, 1e-8, 0.1
COEF = 0.01
SEED = 0x1234567887654321        # of the dither of 8-bit states
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
# one transformer layer of the repository's ragged layout: q, k, v, o; gate, up, down; two norms
LAYER = "16777216*4,45088768*3,4096*2"
LAYERS4 = "16777216*16,45088768*12,4096*8"
M32 = 0xFFFFFFFF
GOLD, ROOT2, ROOT3 = 0x9E3779B9, 0x6A09E667, 0xBB67AE85


def _step(name, states, sizes, grad, copy, clip=0.0, dither=False):
    return {"name": name, "kind": "step", "states": states, "sizes": sizes, "grad": grad, "copy": copy, "clip": clip,
            "dither": dither}


def _balance(name, tokens, experts, k, logits, masked=False):
    return {"name": name, "kind": "balance", "tokens": tokens, "experts": experts, "k": k, "logits": logits,
            "masked": masked}


def listed():
    return [
        # two norms, a scalar and a short bias: what counts is the latency of the calls
        _step("step32 few small", "fp32", "4096*2,64,1", "bf16", "bf16"),
        # the norms of 32 layers and odd leftovers beside a flat partition, clipped, loss-scaled fp16
        _step("step32 many odd", "fp32", "4096*65,1000003,65537*3,333,7", "fp16", "fp16", clip=1.0),
        # one layer in bf16
        _step("step32 layer", "fp32", LAYER, "bf16", "bf16"),
        # four layers, fp16, clipped
        _step("step32 4 layers", "fp32", LAYERS4, "fp16", "fp16", clip=1.0),
        # the same range with states in 8 bits
        _step("step8 few small", "fp8", "4096*2,64,1", "bf16", "bf16"),
        # parameters kept in fp32 alone, with gradients summed in fp32
        _step("step8 many odd", "fp8", "4096*65,1000003,65537*3,333,7", "fp32", "fp32", clip=1.0, dither=True),
        _step("step8 layer", "fp8", LAYER, "bf16", "bf16", dither=True),
        _step("step8 4 layers", "fp8", LAYERS4, "bf16", "bf16", clip=1.0, dither=True),
        # one token over a few experts
        _balance("balance 1 token", 1, 8, 2, "bf16"),
        # a micro-batch of 4096 tokens, part of it padding, loss-scaled fp16
        _balance("balance 4096 x 64", 4096, 64, 8, "fp16", masked=True),
        # odd sizes, router in fp32
        _balance("balance odd fp32", 10007, 60, 4, "fp32", masked=True),
        # a long batch over many experts
        _balance("balance 131072 x 256", 131072, 256, 8, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.4:      # fewer chosen than there are: with all of them chosen the gradient is zero
        tokens, experts = _log_int(rng, 1, 131072), _log_int(rng, 2, 256)
        c = _balance("", tokens, experts, rng.randint(1, min(8, experts - 1)), rng.choice(["fp16", "bf16", "fp32"]),
                     rng.random() < 0.5)
    else:
        total, count = _log_int(rng, 1, 400_000_000), _log_int(rng, 1, 200)
        weights = [math.exp(rng.uniform(0, 8)) for _ in range(count)]
        sizes = [max(1, int(total * w / sum(weights))) for w in weights]
        copy = rng.choice(["fp16", "bf16", "fp32"])
        grad = rng.choice([copy, "fp32"])
        states = rng.choice(["fp32", "fp8"])
        c = _step("", states, ",".join(map(str, sizes)), grad, copy, rng.choice([0.0, 1.0]),
                  states == "fp8" and rng.random() < 0.5)
    del c["name"]
    return c


def _sizes(case):
    out = []
    for part in case["sizes"].split(","):
        n, _, times = part.partition("*")
        out += [int(n)] * int(times or 1)
    return out


def _offsets(sizes):
    offs, at = [], 0
    for n in sizes:
        offs.append(at)
        at += -(-n // ALIGN) * ALIGN
    return offs, at


def _scale(kind):
    return 65536.0 if kind == "fp16" else 1.0    # fp16 gradients carry a loss scale, the others none


def work(case):
    if case["kind"] == "step":
        n = sum(_sizes(case))
        g = 4 if case["grad"] == "fp32" else 2
        p = 8 if case["copy"] == "fp32" else 10
        s = 16 if case["states"] == "fp32" else 4 + 16 / 256
        return {"bytes": n * (g + p + s), "flops": n * (18 if case["states"] == "fp32" else 40)}
    n, b = case["tokens"] * case["experts"], 4 if case["logits"] == "fp32" else 2
    mask = case["tokens"] if case["masked"] else 0
    return {"bytes": 2 * n * b + mask + 8 * case["experts"], "flops": n * (12 + case["k"])}


# ---- inputs ----------------------------------------------------------------------------------------------------------


def _prepare_step(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    sizes = _sizes(case)
    offs, total = _offsets(sizes)
    t = 100                                             # steps applied before this one
    dtype = TYPES[case["copy"]]
    real = torch.zeros(total, dtype=torch.bool, device=dev)
    for o, n in zip(offs, sizes):
        real[o:o + n] = True

    def normal(sigma):
        return torch.randn(total, generator=gen, device=dev).mul_(sigma).mul_(real)

    scale = _scale(case["grad"])
    master = normal(0.02)
    grad = normal(1e-3 * scale).to(TYPES[case["grad"]])
    m = normal(3e-4)
    v = normal(1e-3).square_().mul_(1 - BETA2 ** t).add_(1e-12).mul_(real)
    s = {"case": case, "sizes": sizes, "offs": offs, "t": t, "scale": scale, "grad": grad, "master": master,
         "params": master if dtype == torch.float32 else master.to(dtype)}
    del real
    if case["states"] == "fp32":
        s["m"], s["v"] = m, v
    else:                                               # held in 8 bits with a scale for each 256
        for key, x, most, kind in (("m", m, 448, torch.float8_e4m3fn), ("v", v, 57344, torch.float8_e5m2)):
            x = x.view(-1, ALIGN)
            sc = x.abs().amax(1) / most
            s[key + "_scale"] = sc
            s[key] = (x / torch.where(sc > 0, sc, 1)[:, None]).clamp_(-most, most).to(kind).view(-1)
    few = [n >= 65536 for n in sizes]                   # norms and biases do not decay
    s["decay"] = [DECAY if big else 0.0 for big in few]
    s["applied"] = torch.tensor(float(t), dtype=torch.float64, device=dev)
    if own:
        s["op"] = _own_step(s)
    return s


def _own_step(s):
    """The framework's handle over the same tensors, as a program makes it once before its training loop."""
    import zero_mixed_precision_amd as z

    c = s["case"]
    cfg = z.ZeroMPConfig(bf16="fp16" not in (c["grad"], c["copy"]), loss_scale=s["scale"], lr=LR,
                         betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY, gradient_clipping=c["clip"])
    views = lambda flat: [flat[o:o + n] for o, n in zip(s["offs"], s["sizes"])]  # noqa: E731
    op = z.MultiTensorStep(views(s["params"]), cfg, states=c["states"], weight_decay=s["decay"],
                           dither_seed=SEED if c["dither"] else None)
    if op.master is not None:
        op.master.copy_(s["master"])
        s["master"] = op.master
    for key in ("m", "v") + (("m_scale", "v_scale") if c["states"] == "fp8" else ()):
        getattr(op, key).copy_(s[key])
        s[key] = getattr(op, key)
    op.set_gradients(views(s["grad"]))
    op.set_applied_steps(s["t"])
    return op


def _prepare_balance(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    T, E = case["tokens"], case["experts"]
    # a router in training: some experts are liked better than others
    z = torch.randn(T, E, generator=gen, device=dev) + 0.5 * torch.randn(E, generator=gen, device=dev)
    mask = None
    if case["masked"]:
        mask = (torch.rand(T, generator=gen, device=dev) < 0.9).to(torch.uint8)
    s = {"case": case, "logits": z.to(TYPES[case["logits"]]), "mask": mask, "scale": _scale(case["logits"])}
    if own:
        import zero_mixed_precision_amd as z_amd
        from zero_mixed_precision_amd import _lib

        s["op"] = z_amd.ExpertBalance(E, case["k"], COEF)
        s["scaler"] = None
        if s["scale"] != 1.0:
            s["scaler"] = torch.zeros(_lib.ds_scaler_size(), dtype=torch.uint8, device=dev)
            _lib.ds_state_init(s["scaler"], s["scale"], 1.0, 1000, 1, 0, 0)
        s["dlogits"] = torch.empty_like(s["logits"])
    return s


def prepare(case, seed):
    return (_prepare_step if case["kind"] == "step" else _prepare_balance)(case, seed)


# ---- plain forms -----------------------------------------------------------------------------------------------------


def _mix(x):
    x = x ^ (x >> 16)
    x = (x * ROOT2) & M32
    x = x ^ (x >> 15)
    x = (x * ROOT3) & M32
    return x ^ (x >> 16)


def _places(s):
    """The tensor that each block of 256 belongs to, and the block's number in it."""
    start = torch.tensor([o // ALIGN for o in s["offs"]], device=s["grad"].device)
    block = torch.arange(s["grad"].numel() // ALIGN, device=start.device)
    tensor = torch.searchsorted(start, block, right=True) - 1
    return tensor, block - start[tensor]


def _dither(s, t, tensor, block):
    """The dither of m's codes (20 bits) and of v's (21), by block and element (half a step each without dither)."""
    if not s["case"]["dither"]:
        return 1 << 19, 1 << 20
    dev = s["grad"].device
    key = torch.full((), SEED >> 32, dtype=torch.int64, device=dev)
    key = _mix(_mix(key) ^ (SEED & M32))
    key = _mix((key + t.long() * GOLD) & M32)
    key = _mix((key + tensor * GOLD) & M32)
    key = _mix((key + block * GOLD) & M32)[:, None]
    lane = torch.arange(ALIGN, device=dev) * GOLD
    return (((key + lane) & M32) >> 12).int(), (((_mix(key ^ ROOT3) + lane) & M32) >> 11).int()


def _encode(x, u, most, low, bits, kind, keep):
    """x by blocks of 256 as 8-bit floats of ``kind`` (largest value ``most``, smallest normal one ``low``, a step every
    2^bits of an fp32 bit pattern) and scales; keep: a positive value never becomes zero."""
    top = x.abs().amax(1)
    ok = top >= 2.0 ** -110
    a = (x.abs() * torch.where(ok, most / top, 0)[:, None]).clamp_(max=most)
    small = a < low                                     # in the binade above, whose steps are as wide
    zero = (127 + round(math.log2(low))) << 23 - bits
    code = (torch.where(small, a + low, a).view(torch.int32) + u) >> bits
    code = code - torch.where(small, zero, zero - (1 << 23 - bits))
    if keep:
        code = torch.where(x > 0, code.clamp(min=1), code)
    code = code + torch.where(x < 0, 128, 0)
    return code.to(torch.uint8).view(kind).view(-1), torch.where(ok, top * (1 / most), 0)


def _plain_step(s):
    c = s["case"]
    g = s["grad"].float()
    fine = torch.isfinite(g).all()
    inv = torch.full((), 1 / s["scale"], dtype=torch.float32, device=g.device)
    if c["clip"]:
        norm = g.double().square().sum().sqrt() * inv.double()
        inv = (inv.double() * (c["clip"] / (norm + 1e-6)).clamp(max=1)).float()
    t = s["applied"] + 1
    size = (LR / (1 - BETA1 ** t)).float()
    root = (1 / (1 - BETA2 ** t).sqrt()).float()
    eight = c["states"] == "fp8"
    if eight:
        m = (s["m"].float().view(-1, ALIGN) * s["m_scale"][:, None]).view(-1)
        v = (s["v"].float().view(-1, ALIGN) * s["v_scale"][:, None]).view(-1)
    else:
        m, v = s["m"], s["v"]
    g = g * inv
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g.square()
    tensor, block = _places(s)
    shrink = torch.tensor([LR * d for d in s["decay"]], device=g.device)[tensor]
    p = s["master"]
    p = (p.view(-1, ALIGN) - shrink[:, None] * p.view(-1, ALIGN)).view(-1)
    p = p - size * (m / (v.sqrt() * root + EPS))
    if eight:
        um, uv = _dither(s, t, tensor, block)
        mc, ms = _encode(m.view(-1, ALIGN), um, 448, 2.0 ** -6, 20, torch.float8_e4m3fn, False)
        vc, vs = _encode(v.view(-1, ALIGN), uv, 57344, 2.0 ** -14, 21, torch.float8_e5m2, True)
        new = {"m": mc.view(torch.uint8), "m_scale": ms, "v": vc.view(torch.uint8), "v_scale": vs}
    else:
        new = {"m": m, "v": v}
    for key, x in {**new, "master": p}.items():         # a step whose gradient is not finite changes nothing
        old = s[key].view(x.dtype)
        old.copy_(torch.where(fine, x, old))
    if s["params"] is not s["master"]:
        s["params"].copy_(s["master"])
    s["applied"] = s["applied"] + fine


def _plain_balance(s):
    c = s["case"]
    z = s["logits"].float()
    T, E, k = c["tokens"], c["experts"], c["k"]
    valid = torch.ones(T, dtype=torch.bool, device=z.device) if s["mask"] is None else s["mask"] != 0
    top = z.amax(1)
    valid = valid & (top > -math.inf)
    used = valid.sum()
    e = torch.exp(z - top[:, None])
    p = torch.where(valid[:, None], e / e.sum(1, keepdim=True), 0)
    column = torch.arange(E, device=z.device)
    left, chosen = z, torch.zeros(T, E, dtype=torch.bool, device=z.device)
    for _ in range(k):                                  # the largest left, the lowest index among equals
        best = left.amax(1, keepdim=True)
        first = torch.where(left == best, column, E).amin(1, keepdim=True)
        hit = (column == first) & (best > -math.inf)
        chosen = chosen | hit
        left = torch.where(hit, -math.inf, left)
    counts = (chosen & valid[:, None]).sum(0)
    some = used.clamp(min=1).double()
    f = (counts / (k * some)).float()
    mean = (p.double().sum(0) / some).float()
    loss = COEF * E * (f * mean).sum()
    factor = (s["scale"] * COEF * E / some).float()
    d = factor * p * (f - (p * f).sum(1, keepdim=True))
    return {"loss": loss, "counts": counts.int(), "mean": mean, "used": used.int(), "dlogits": d.to(s["logits"].dtype)}


def run(s):
    c = s["case"]
    if c["kind"] == "balance":
        if not own:
            return _plain_balance(s)
        op = s["op"]
        op.loss(s["logits"], mask=s["mask"])
        op.gradient(s["logits"], s["dlogits"], mask=s["mask"], scaler=s["scaler"])
        return {"loss": op.value, "counts": op.counts, "mean": op.mean_prob, "used": op.used, "dlogits": s["dlogits"]}
    if own:
        s["op"].step()
    else:
        _plain_step(s)
    keys = ["params", "m", "v"] + (["master"] if s["params"] is not s["master"] else [])
    return {k: s[k] for k in keys + (["m_scale", "v_scale"] if c["states"] == "fp8" else [])}


# ---- the definition, in 64 bits --------------------------------------------------------------------------------------


def _hash32(x):
    x ^= x >> 16
    x = x * ROOT2 % 2 ** 32
    x ^= x >> 15
    x = x * ROOT3 % 2 ** 32
    return x ^ x >> 16


def _exact_codes(x, u, most, exponent, mantissa, keep):
    """Codes' values and scales of x (float64, blocks of 256), from the definition: floor(a / ulp + u) steps of ulp."""
    top = x.abs().max(dim=1, keepdim=True).values
    a = torch.nan_to_num(x.abs() / top * most, nan=0.0)
    ulp = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** exponent))) - mantissa)
    q = (torch.floor(a / ulp + u) * ulp).clamp(max=most)
    if keep:
        q = torch.maximum(q, (x > 0) * 2.0 ** (exponent - mantissa))
    return (q * torch.sign(x)).reshape(-1), (top / most).reshape(-1)


def _exact_step(case, seed):
    s = _prepare_step(case, seed)
    c, t = case, s["t"] + 1
    g = s["grad"]
    norm2 = sum(float(x.double().pow(2).sum()) for x in g.split(1 << 26))
    norm = math.sqrt(norm2) / s["scale"]
    factor = (min(1.0, c["clip"] / (norm + 1e-6)) if c["clip"] else 1.0) / s["scale"]
    eight = c["states"] == "fp8"
    out = {"params": torch.zeros(g.numel(), dtype=torch.float64, device=g.device)}
    for key in ("m", "v"):
        out[key] = torch.zeros_like(out["params"])
        if eight:
            out[key + "_scale"] = torch.zeros(g.numel() // ALIGN, dtype=torch.float64, device=g.device)
    lane = torch.arange(ALIGN, device=g.device) * GOLD
    for j, (o, n, wd) in enumerate(zip(s["offs"], s["sizes"], s["decay"])):
        whole = -(-n // ALIGN) * ALIGN
        for lo in range(0, whole, 1 << 26):             # parts of a tensor: whole blocks
            at = slice(o + lo, o + min(whole, lo + (1 << 26)))
            blk = slice(at.start // ALIGN, at.stop // ALIGN)
            x = g[at].double() * factor
            m, v = s["m"][at].double(), s["v"][at].double()
            if eight:
                m = (m.view(-1, ALIGN) * s["m_scale"][blk].double()[:, None]).view(-1)
                v = (v.view(-1, ALIGN) * s["v_scale"][blk].double()[:, None]).view(-1)
            m = BETA1 * m + (1 - BETA1) * x
            v = BETA2 * v + (1 - BETA2) * x * x
            p = s["master"][at].double() * (1 - LR * wd)
            out["params"][at] = p - LR / (1 - BETA1 ** t) * m / (torch.sqrt(v) / math.sqrt(1 - BETA2 ** t) + EPS)
            if not eight:
                out["m"][at], out["v"][at] = m, v
                continue
            um = uv = 0.5
            if c["dither"]:
                key = _hash32(_hash32(_hash32(_hash32(SEED >> 32) ^ SEED % 2 ** 32) + t * GOLD & M32) + j * GOLD & M32)
                key = _mix((key + torch.arange(lo // ALIGN, lo // ALIGN + blk.stop - blk.start, device=g.device) * GOLD)
                           % 2 ** 32)[:, None]
                um = torch.floor((key + lane) % 2 ** 32 / 4096.0) / 2.0 ** 20
                uv = torch.floor((_mix(key ^ ROOT3) + lane) % 2 ** 32 / 2048.0) / 2.0 ** 21
            out["m"][at], out["m_scale"][blk] = _exact_codes(m.view(-1, ALIGN), um, 448, -6, 3, False)
            out["v"][at], out["v_scale"][blk] = _exact_codes(v.view(-1, ALIGN), uv, 57344, -14, 2, True)
    if c["copy"] != "fp32":
        out["master"] = out["params"]
    return out


def _exact_balance(case, seed):
    s = _prepare_balance(case, seed)
    T, E, k = case["tokens"], case["experts"], case["k"]
    z = s["logits"].double()
    rows = torch.ones(T, dtype=torch.bool, device=z.device) if s["mask"] is None else s["mask"] > 0
    n = int(rows.sum())
    order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]
    counts = torch.bincount(order[rows].reshape(-1), minlength=E)
    p = torch.softmax(z, dim=1) * rows[:, None]
    f = counts.double() / max(1, n * k)
    mean = p.sum(0) / max(1, n)
    d = p * (f - (p @ f)[:, None]) * (s["scale"] * COEF * E / max(1, n))
    return {"loss": COEF * E * (f @ mean), "counts": counts.int(), "mean": mean, "used": n, "dlogits": d}


def exact(case, seed):
    return (_exact_step if case["kind"] == "step" else _exact_balance)(case, seed)
