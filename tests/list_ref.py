"""The step over a list of tensors in 64 bits, from its formulas, with bounds on what fp32 arithmetic may differ by.

E = 2^-24 is half a unit of fp32: each of its operations is off by at most E relative to its result."""
import numpy as np

E = 2.0 ** -24
BLOCK = 256
M32 = 2 ** 32 - 1


def mix(x):
    x = np.asarray(x, dtype=np.uint64)
    x = x ^ (x >> np.uint64(16))
    x = (x * np.uint64(0x6A09E667)) & np.uint64(M32)
    x = x ^ (x >> np.uint64(15))
    x = (x * np.uint64(0xBB67AE85)) & np.uint64(M32)
    return x ^ (x >> np.uint64(16))


def dither(seed, t, tensor, n):
    """(u of m, u of v) in [0, 1) for the n elements of a tensor."""
    gold = np.uint64(0x9E3779B9)
    m = np.uint64(M32)
    k = mix(mix(seed >> 32) ^ np.uint64(seed & M32))
    k = mix((k + np.uint64(t) * gold) & m)
    k = mix((k + np.uint64(tensor) * gold) & m)
    i = np.arange(n, dtype=np.uint64)
    k = mix((k + (i // np.uint64(BLOCK)) * gold) & m)
    lane = (i % np.uint64(BLOCK)) * gold
    um = ((k + lane) & m) >> np.uint64(12)
    uv = ((mix(k ^ np.uint64(0xBB67AE85)) + lane) & m) >> np.uint64(11)
    return um.astype(np.float64) / 2 ** 20, uv.astype(np.float64) / 2 ** 21


class Format:
    """An 8-bit float: sign, exponent (smallest normal 2^low), ``man`` bits of mantissa, largest value ``most``."""

    def __init__(self, man, low, most):
        self.man, self.low, self.most = man, low, most
        self.tiny = 2.0 ** (low - man)          # the smallest positive value

    def decode(self, codes):
        """The values of codes (uint8); what lies above the largest is NaN here."""
        c = np.asarray(codes, dtype=np.uint8).astype(np.int64)
        exp, man = (c & 127) >> self.man, c & (2 ** self.man - 1)
        mag = np.where(exp == 0, man * self.tiny, (2 ** self.man + man) * np.exp2(exp - 1.0) * self.tiny)
        mag = np.where(mag > self.most, np.nan, mag)
        return np.where(c >= 128, -mag, mag)

    def quantise(self, a, u):
        """floor(a / ulp + u) steps of ulp, at most the largest value (a >= 0)."""
        a = np.clip(a, 0.0, self.most)
        ulp = np.exp2(np.floor(np.log2(np.maximum(a, 2.0 ** self.low))) - self.man)
        return np.minimum(np.floor(a / ulp + u) * ulp, self.most)


E4M3, E5M2 = Format(3, -6, 448.0), Format(2, -14, 57344.0)


def by_block(x, fill=0.0):
    """x as [blocks, 256], padded."""
    out = np.full((-(-x.size // BLOCK), BLOCK), fill)
    out.reshape(-1)[:x.size] = x
    return out


def spread(scale, n):
    return np.repeat(scale, BLOCK)[:n]


def update(master, m, v, grad, *, lr, b1, b2, eps, wd, t, inv, slack=0):
    """Adam in 64 bits; returns {"p", "m", "v"} and the bounds of their fp32 errors.  ``slack``: relative errors (in E)
    that v already comes with, and m's as many of its size."""
    master, m, v, grad = (np.asarray(x, np.float64) for x in (master, m, v, grad))
    f = lambda x: float(np.float32(x))  # noqa: E731
    eps, lr, wd = f(eps), f(lr), f(wd)
    g = grad * inv
    size = np.abs(b1 * m) + np.abs((1 - b1) * g)
    m1 = b1 * m + (1 - b1) * g
    v1 = b2 * v + (1 - b2) * g * g
    step, root = lr / (1 - b1 ** t), 1 / np.sqrt(1 - b2 ** t)
    den = np.sqrt(v1) * root + eps
    p = master - lr * wd * master
    p1 = p - step * m1 / den
    # m: g * inv (inv itself rounded, 2), 1 - beta rounded, the product and the sum: 5 + slack of the parts' size
    em = (5 + slack) * E * size + 2.0 ** -149
    # v: g twice (2 * 2), square, 1 - beta, product, sum: 8 + slack relative (all terms positive); tiny ones absolute
    ev = (10 + slack) * E * v1 + 2.0 ** -147
    # p: m's error over the denominator; the denominator is off by half of v's error and 5 roundings; quotient,
    # step size and product 4; the decay and the two subtractions 4 of |p|
    ratio = step * np.abs(m1) / den
    # sqrt(v1) may itself be off by sqrt(2^-147) where v1 is as small as that
    edge = np.sqrt(ev) if np.any(v1 < 2.0 ** -120) else 0.0
    ep = step * em / den + ratio * (((10 + slack) / 2 + 10) * E + np.where(v1 < 2.0 ** -120, edge * root / den, 0.0))
    ep = ep + 4 * E * (np.abs(master) + np.abs(p1) + ratio)
    return {"p": p1, "m": m1, "v": v1}, {"p": ep, "m": em, "v": ev}


def code_bounds(x, ex, u, fmt):
    """Lowest and highest values that the codes of |x| may have given x's error bound, and the scale with its bound."""
    n = x.size
    ax, eb = by_block(np.abs(x)), by_block(ex)
    top = np.minimum(ax.max(1), 2.0 ** 126)
    etop = eb.max(1) + 2 * E * top
    scale = top / fmt.most
    ok = top >= 2.0 ** -110
    safe = np.where(ok, top, 1.0)
    a = np.abs(x) * spread(np.where(ok, fmt.most / safe, 0.0), n)
    ea = ex * spread(np.where(ok, fmt.most / safe, 0.0), n) + a * (spread(np.where(ok, etop / safe, 0.0), n) + 4 * E)
    ea = ea + fmt.tiny * 2.0 ** -20              # a is held to 2^-20 (m) or 2^-21 (v) of a subnormal code
    return fmt.quantise(a - ea, u), fmt.quantise(a + ea, u), scale, etop / fmt.most + 2 * E * scale


def check_codes(codes, scale, x, ex, u, fmt, what):
    """Codes (uint8) and scales of the stored state x."""
    lo, hi, want, bound = code_bounds(x, ex, u, fmt)
    want = np.where(want * fmt.most < 2.0 ** -110, 0.0, want)
    assert np.all(np.abs(scale - want) <= bound), f"{what}: scale off by {np.max(np.abs(scale - want))}"
    got = fmt.decode(codes)
    if fmt is E5M2:                              # v: never negative, never 0 where it is positive
        lo, hi = (np.where(x > 0, np.maximum(q, fmt.tiny), q) for q in (lo, hi))
        assert np.all(got >= 0), what
    else:
        sure = np.abs(x) > ex
        assert np.all((np.sign(got) == np.sign(x))[sure & (got != 0)]), f"{what}: sign"
    bad = ~((np.abs(got) >= lo) & (np.abs(got) <= hi))
    assert not bad.any(), f"{what}: {bad.sum()} codes outside, first {np.flatnonzero(bad)[:4]}"
