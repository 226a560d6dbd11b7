"""The 8-bit matrices, their products, the RMS norm and dropout, restated in
64 bits with numpy straight from their formulas, with the first-order bounds
of the library's fp32 rounding errors (U is half an ulp of 1 in fp32) that
the tests use as tolerances.
"""

import numpy as np

from . import tensors as T

BLOCK = 128
U = T.U
EPS = {"f32": 2.0**-24, "bf16": 2.0**-8, "f16": 2.0**-11}  # half a step, relative
# From here on nearest rounding gives infinity: half a step past the largest value, (2 - 2^-11) 2^15 of fp16's 11 bits,
# (2 - 2^-8) 2^127 of bf16's 8, (2 - 2^-24) 2^127 of fp32's 24.
OVER = {"f32": (2 - 2.0**-24) * 2.0**127, "bf16": (2 - 2.0**-8) * 2.0**127, "f16": (2 - 2.0**-11) * 2.0**15}
TINY = {"f32": 2.0**-150, "bf16": 2.0**-134, "f16": 2.0**-25}  # half of the smallest value


# ------------------------------------------------------------- the encoding --

def blocks_of(cols):
    return -(-cols // BLOCK)


def scale_size(rows, cols):
    return -(-rows // 128) * -(-blocks_of(cols) // 4) * 512


def scale_places(rows, cols):
    """Place of the byte of each row and block."""
    groups = -(-blocks_of(cols) // 4)
    r, b = np.arange(rows)[:, None], np.arange(blocks_of(cols))[None]
    return ((r // 128) * groups + b // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4


def tops(x, square=False):
    """The largest magnitude of each row and block (of each square, for all of its rows); NaN where one is."""
    rows, cols = x.shape
    full = np.zeros((rows, blocks_of(cols) * BLOCK))
    full[:, :cols] = np.abs(x)
    top = full.reshape(rows, -1, BLOCK).max(2)
    if square:
        for r in range(0, rows, BLOCK):
            top[r:r + BLOCK] = top[r:r + BLOCK].max(0)
    return top


def scales(x, square=False):
    """The scale byte of each row and block."""
    return T.scale_of(tops(np.asarray(x, np.float64), square), 1.75, 8, 8)


def per_column(scale, cols):
    return np.repeat(np.asarray(scale).astype(np.int64), BLOCK, axis=1)[:, :cols]


def rounded(x, scale):
    """The values that x's codes stand for under these scale bytes."""
    x = np.asarray(x, np.float64)
    s = per_column(scale, x.shape[1])
    bad = s == 255
    unit = 2.0 ** (np.where(bad, 127, s) - 127.0)
    v = np.where(bad, 0.0, x) / unit
    e = np.maximum(np.frexp(v)[1] - 4, -9)
    q = np.clip(np.rint(v / 2.0**e) * 2.0**e, -448, 448) * unit
    return np.where(bad, np.nan, q)


def values(codes, scale):
    """What codes stand for."""
    codes = np.asarray(codes).astype(np.int64)
    s = per_column(scale, codes.shape[1])
    mag = T.E4M3[codes & 127]
    return np.where(s == 255, np.nan, np.where(codes >= 128, -mag, mag) * 2.0 ** (s - 127.0))


# ----------------------------------------------------------------- products --

def product(a, b):
    """a b^T of two matrices' values, and its fp32 rounding's bound: a product passes at most 32 additions in its step
    along k, one per step, and those that join parts of k, each off by at most one last place (2 U)."""
    k = a.shape[1]
    return a @ b.T, 2 * U * (32 + k / 32 + 8) * (np.abs(a) @ np.abs(b).T)


# ------------------------------------------------------------------ dropout --

def threshold(p):
    return int(np.rint(p * 65536))


def random16(numbers, seed, site, t):
    """The 16-bit numbers of elements `numbers` (int64)."""
    i = np.asarray(numbers).astype(np.uint64)
    low, high = (i >> np.uint64(1)) & np.uint64(0xFFFFFFFF), i >> np.uint64(33)
    x = low * np.uint64(0x9E3779B9) + high * np.uint64(0x3C6EF372) \
        + np.uint64((seed + site * 0x510E527F + t * 0x6A09E667) % 2**32)
    x &= np.uint64(0xFFFFFFFF)
    for c in (0xBB67AE85, 0xA54FF53B):
        x = x * np.uint64(c)
        x = (x ^ (x >> np.uint64(32))) & np.uint64(0xFFFFFFFF)
    return np.where(i & np.uint64(1), x >> np.uint64(16), x & np.uint64(0xFFFF)).astype(np.int64)


def dropout(x, drop, numbers=None):
    """(dropout of x, its fp32 rounding's bound); drop: dict of p, seed, site, t, or None."""
    x = np.asarray(x, np.float64)
    if not drop or threshold(drop["p"]) == 0:
        return x, np.zeros_like(x)
    n = np.arange(x.size) if numbers is None else numbers
    r = random16(n, drop["seed"], drop["site"], drop["t"]).reshape(x.shape)
    y = np.where(r < threshold(drop["p"]), 0.0, x) * (65536 / (65536 - threshold(drop["p"])))
    return y, 2 * U * np.abs(y) + TINY["f32"]


# --------------------------------------------------------------------- norm --

# Additions that a row's term passes: 32 of a thread, 5 of a warp, 16 of the warps.
ROW_DEPTH = 53


def norm_input(x, residual, drop):
    """(h before its rounding, the bound of fp32's)."""
    h, d = dropout(x, drop)
    if residual is not None:
        h = h + residual
        d = d + U * np.abs(h)
    return h, d


def norm(h, gain, eps):
    """(rstd, its bound), (y, its bound) of stored h, before y's own rounding."""
    m = (h * h).mean(1) + eps
    rstd = 1 / np.sqrt(m)
    # the sum's error halves in the root; the mean, eps as fp32, its addition, and the root with its refinement
    drstd = rstd * U * (ROW_DEPTH / 2 + 8)
    y = h * rstd[:, None] * gain
    dy = np.abs(y) * U * (ROW_DEPTH / 2 + 8 + 3) + TINY["f32"]
    return (rstd, drstd), (y, dy)


def norm_backward(dy, h, gain, rstd, dres):
    """((dh, bound), (dgain, bound)) before roundings to the outputs' type."""
    n = h.shape[1]
    hat, g = h * rstd[:, None], dy * gain
    mean = (g * hat).mean(1, keepdims=True)
    dmean = U * (ROW_DEPTH + 6) * np.abs(g * hat).mean(1, keepdims=True)
    inner = g - hat * mean
    dh = rstd[:, None] * inner
    bound = rstd[:, None] * (3 * U * np.abs(g) + np.abs(hat) * (dmean + 4 * U * np.abs(mean)) + 2 * U * np.abs(inner))
    if dres is not None:
        dh = dh + dres
        bound = bound + U * np.abs(dh)
    dgain = (dy * hat).sum(0)
    return (dh, bound + TINY["f32"]), (dgain, U * (len(h) + 12) * np.abs(dy * hat).sum(0) + TINY["f32"] * n)


def near(got, want, bound, dtype):
    """Which of the outputs of this type are right: within the bound of fp32's errors and half a step."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    with np.errstate(invalid="ignore"):
        tol = bound + (np.abs(want) + bound) * EPS[dtype] + TINY[dtype]
        close = (np.abs(got - want) <= tol) & (np.abs(want) - bound < OVER[dtype])
        over = np.isinf(got) & (np.sign(got) == np.sign(want)) & (np.abs(want) + bound >= OVER[dtype])
        return close | over | (np.isnan(got) & np.isnan(want)) | (got == want)
