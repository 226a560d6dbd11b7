"""The step over a list of tensors, restated in 64 bits with numpy: the grad
norm, AdamW, and the 8-bit moments' encoding, straight from their formulas.

The library computes in fp32; this module also gives the first-order bounds
of its rounding errors (U is half an ulp of 1 in fp32), which the tests use
as tolerances: an 8-bit code is right when it is the code of some moment
within that bound of the exact one.
"""

import numpy as np

BLOCK = 256
U = 2.0**-24


# ------------------------------------------------------------- the encoding --

def exponent(x):
    """floor(log2 x) of positive finite x (fp32 subnormals: -127, as their fp32 exponent field reads)."""
    return np.maximum(np.frexp(x)[1] - 1, -127)


def rows(x, fill=0.0):
    """x in rows of a block, the last filled up."""
    x = np.asarray(x)
    n = -(-len(x) // BLOCK) * BLOCK
    out = np.full(n, fill, dtype=x.dtype)
    out[: len(x)] = x
    return out.reshape(-1, BLOCK)


def per_element(scale, n):
    return np.repeat(np.asarray(scale).astype(np.int64), BLOCK)[:n]


def scale_of(top, mantissa, width, least):
    """A block's scale byte from its largest magnitude: the exponent, one more above `mantissa`, less `width`."""
    top = np.asarray(top, np.float64)
    ok = np.isfinite(top)
    t = np.where(ok & (top > 0), top, 1.0)
    e = exponent(t) + 127
    e = np.where(t > mantissa * 2.0 ** (e - 127), e + 1, e)
    e = np.where(ok & (top > 0), e, 0)
    return np.where(ok & (e < 255), np.maximum(e - width, least), 255)


def m_scale(m):
    return scale_of(np.abs(rows(m)).max(1), 1.75, 8, 8)


def v_scale(v):
    r = rows(v)
    top = np.where((r < 0).any(1), np.nan, r.max(1))
    return scale_of(top, 1.875, 31, 0)


def e4m3_values():
    c = np.arange(128)
    e, f = c >> 3, c & 7
    val = np.where(e > 0, (1 + f / 8.0) * 2.0 ** (e - 7.0), f / 8.0 * 2.0**-6)
    val[127] = np.nan
    return val


E4M3 = e4m3_values()


def m_values(codes, scale):
    """What exp_avg codes stand for."""
    codes = np.asarray(codes).astype(np.int64)
    s = per_element(scale, len(codes))
    mag = E4M3[codes & 127]
    out = np.where(codes >= 128, -mag, mag) * 2.0 ** (s - 127.0)
    return np.where(s == 255, np.nan, out)


def v_values(codes, scale):
    """What exp_avg_sq codes stand for."""
    codes = np.asarray(codes).astype(np.int64)
    s = per_element(scale, len(codes))
    e, f = (codes >> 3) + s, codes & 7
    out = np.where(e > 0, (1 + f / 8.0) * 2.0 ** (e - 127.0), f / 8.0 * 2.0**-126)
    return np.where(s == 255, np.nan, np.where(codes == 0, 0.0, out))


def m_rounded(m, scale):
    """The representable value nearest to each m (ties to the even code) under the given scales."""
    m = np.asarray(m, np.float64)
    s = per_element(scale, len(m))
    x = np.abs(m) * 2.0 ** (127.0 - s)
    hi = np.searchsorted(E4M3[:127], x, side="left").clip(0, 126)
    lo = np.maximum(hi - 1, 0)
    mid = (E4M3[lo] + E4M3[hi]) / 2
    pick = np.where(x > mid, hi, np.where(x < mid, lo, np.where(lo % 2 == 0, lo, hi)))
    pick = np.where(x == E4M3[hi], hi, pick)
    out = np.copysign(E4M3[pick] * 2.0 ** (s - 127.0), m)
    return np.where(s == 255, np.nan, out)


def v_rounded(v, scale, up):
    """v between its two neighbouring values: the upper one where the distance from the lower, as a fraction of
    theirs, plus `up` reaches 1; never below the smallest value for v > 0."""
    v = np.asarray(v, np.float64)
    s = per_element(scale, len(v))
    pos = v > 0
    t = np.where(pos, v, 1.0)
    step = 2.0 ** (np.maximum(exponent(t), -126) - 3.0)
    q = np.floor(t / step + up) * step
    e1 = s + 0.0
    least = np.where(e1 > 0, 1.125 * 2.0 ** (e1 - 127), 0.125 * 2.0**-126)
    return np.where(s == 255, np.nan, np.where(pos, np.maximum(q, least), 0.0))


def rounding_fraction(n, tensor, step, seed, first=0):
    """The 16 pseudo-random bits of elements first.. of a tensor, as fractions."""
    i = np.arange(first, first + n, dtype=np.uint64)
    x = ((i >> np.uint64(1)) * np.uint64(0x9E3779B9) + np.uint64((seed + tensor * 0x510E527F + step * 0x6A09E667) % 2**32))
    x &= np.uint64(0xFFFFFFFF)
    for mul in (0xBB67AE85, 0xA54FF53B):
        p = x * np.uint64(mul)
        x = (p ^ (p >> np.uint64(32))) & np.uint64(0xFFFFFFFF)
    r = np.where(i & np.uint64(1), x >> np.uint64(16), x & np.uint64(0xFFFF))
    return r.astype(np.float64) / 65536.0


# ----------------------------------------------------------------- the step --

def grad_norm(grads, inv_scale, max_norm):
    """(norm, coefficient, found, zeros) of a list of grads (float arrays)."""
    g = np.concatenate([np.asarray(x, np.float64).ravel() * inv_scale for x in grads] or [np.zeros(0)])
    found = not np.isfinite(g).all()
    norm = np.sqrt(np.sum(g * g))
    coef = 1.0
    if max_norm > 0 and max_norm / (norm + 1e-6) < 1:
        coef = max_norm / (norm + 1e-6)
    return (np.nan if found else norm), coef, found, int((g == 0).sum())


def adamw(w, g, m, v, hp, step, inv_scale=1.0, coef=1.0, wd_mult=1.0):
    """(w', m', v') and the bounds of the fp32 result's rounding errors of each.

    The bounds count roundings of half an ulp, relative to each term: m' has
    the scaled grad (2), the constants (1 each), the products (1 each) and the
    sum (1): 5 on |b1 m| + |(1-b1) g|.  v' has the grad squared (4), a
    constant (1), the products (2), the sum (1): 8.  The denominator has half
    of v's (4), the root, the division, its constant, the sum and eps (5): 9;
    the update adds 3 more; the weight's decay 2 and the final subtraction 1."""
    w, g, m, v = (np.asarray(x, np.float64) for x in (w, g, m, v))
    b1, b2 = hp["beta1"], hp["beta2"]
    g = g * inv_scale * coef
    mb = np.abs(b1 * m) + np.abs((1 - b1) * g)
    m1 = b1 * m + (1 - b1) * g
    v1 = b2 * v + (1 - b2) * g * g
    size = hp["lr"] / (1 - b1**step)
    denom = np.sqrt(v1 / (1 - b2**step)) + hp["eps"]
    w1 = w * (1 - hp["lr"] * hp["weight_decay"] * wd_mult) - size * m1 / denom
    slack = 1.01 * U
    tiny = 2.0**-149  # subnormal results: an absolute half unit per operation
    return (w1, m1, v1), (slack * (3 * np.abs(w) + 18 * size * mb / denom) + 4 * tiny, slack * 5 * mb + 4 * tiny,
                          slack * 8 * v1 + 4 * tiny)
