"""Plain 64-bit forms of the operators on 8-bit floating-point blocks and of the row permutations, in numpy.

Written from the definitions in include/moe_mi355x.h and independent of the library.  Every form returns what the
library should give before its last rounding and a bound on how far it may be from that.
"""

import numpy as np

B, TOP = 128, 448.0
U32 = 2.0 ** -24   # half a step of fp32, relative
HALF_STEP = {"f32": U32, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
FLOOR = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}   # half a step below the normal range


def e4m3(v):
    """The nearest E4M3 values, ties to even (|v| <= 448)."""
    a = np.abs(np.asarray(v, np.float64))
    step = 2.0 ** (np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    return np.sign(v) * np.rint(a / step) * step


def quotients(x):
    """448 x / amax by blocks of 128 columns of x [R, K] in fp64 (0 for blocks of zeros), and the scales."""
    v = np.asarray(x, np.float64).reshape(len(x), -1, B)
    top = np.abs(v).max(2, keepdims=True)
    return np.divide(TOP * v, top, out=np.zeros_like(v), where=top > 0).reshape(len(x), -1), (top / TOP)[:, :, 0]


def exact_codes(r, *shape):
    """Codes whose products are multiples of 1/4 up to 9: the matrix units' alignment loses nothing of them."""
    return r.choice(np.array([0, 0.5, 1, 1.5, 2, 3, -0.5, -1, -1.5, -2, -3]), size=shape)


def scales_of(r, *shape):
    return np.exp(0.7 * r.normal(size=shape)).astype(np.float32)


def product(a, sa, w, sw, off, aligned):
    """y [R, N] of rows a [R, K] with scales sa [R, K/128] and weights w [E, N, K] with scales sw [E, N/128 up, K/128],
    and a bound on the error before the rounding of y.

    fp32 steps: the two scales are multiplied, a block's sum is exact or rounded once for each of its two MFMAs, it is
    scaled and added to the running sum, or the running sum is brought to the block's scale by a factor that carries
    three roundings and one of its own: less than 8 roundings of each partial sum per block, and 8 parts are added.
    aligned: codes from exact_codes on both sides, whose block sums are exact.  Else each of a block's 128 products is
    off by at most itself or 2^-13 of the largest one, whichever is less.
    """
    R, K = a.shape
    E, N, _ = w.shape
    y, bound = np.zeros((R, N)), np.zeros((R, N))
    sw = sw.astype(np.float64)[:, np.arange(N) // B]
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        if off[e + 1] == off[e]:
            continue
        size = np.zeros((int(off[e + 1] - off[e]), N))
        for b in range(K // B):
            c = slice(b * B, b * B + B)
            f = sa[r, b:b + 1].astype(np.float64) * sw[e, :, b]
            y[r] += f * (a[r, c] @ w[e, :, c].T)
            mag = np.abs(a[r, c]) @ np.abs(w[e, :, c]).T
            size += np.abs(f) * mag
            if not aligned:
                largest = np.abs(a[r, c]).max(1)[:, None] * np.abs(w[e, :, c]).max(1)
                bound[r] += np.abs(f) * np.minimum(mag, B * 2.0 ** -13 * largest)
        bound[r] += (8 * (K // B) + 16) * U32 * size
    return y, bound


def ffn(x, sx, gate, up, down, off, aligned):
    """y [R, H] of the SwiGLU FFN and a bound.  gate, up, down: (codes, scales); x, gate and up `aligned` as above.

    silu turns a relative error of g into at most (1 + |g|) times it; exponential, sum, reciprocal and products add
    less than ten roundings.  Where h's error crosses a boundary of its code's rounding, or moves its block's maximum,
    the code may be the neighbour: the bound adds each possible change times its weight.
    """
    g, dg = product(x, sx, *gate, off, aligned)
    u, du = product(x, sx, *up, off, aligned)
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-g))
        h = g * s * u
        # |silu'| <= 1.1
        d = 1.1 * dg * np.abs(u) + np.abs(g * s) * du + 1.1 * dg * du + (10 + 2 * np.abs(g)) * U32 * np.abs(h)
    size = np.abs(h).reshape(len(h), h.shape[1] // B, B)
    dd = d.reshape(size.shape)
    top = size.max(2, keepdims=True)
    lo, hi = (size - dd).max(2, keepdims=True).clip(min=0), (size + dd).max(2, keepdims=True)
    q = e4m3(np.divide(TOP * size, top, out=np.zeros_like(size), where=top > 0))
    with np.errstate(divide="ignore", invalid="ignore"):
        least = np.where(hi > 0, TOP * (size - dd).clip(min=0) / hi, 0.0)
        most = np.where(lo > 0, np.minimum(TOP * (size + dd) / lo, TOP), TOP)
    moved = np.maximum(q - e4m3(least * (1 - 4 * U32)), e4m3(np.minimum(most * (1 + 4 * U32), TOP)) - q)
    hs = (top / TOP)[:, :, 0]
    # value of a code: its scale moves by (hi - lo) / 2 at most, relative to it
    shift = np.divide(np.maximum(hi - top, top - lo), top, out=np.zeros_like(top), where=top > 0) + 2 * U32
    codes = (np.sign(h).reshape(size.shape) * q).reshape(h.shape)
    y, bound = product(codes, hs, *down, off, False)
    wide = np.abs(down[0]) * np.abs(down[1]).astype(np.float64)[:, np.arange(down[0].shape[1]) // B][:, :, np.arange(h.shape[1]) // B]
    slack = ((moved * (1 + shift) + q * shift) * hs[:, :, None]).reshape(h.shape)
    for e in range(len(wide)):
        r = slice(int(off[e]), int(off[e + 1]))
        bound[r] += slack[r] @ wide[e].T
    return y, bound


def rounded(want, bound, dt):
    """The bound with the rounding to a type on top."""
    return bound + HALF_STEP[dt] * (np.abs(want) + bound) + FLOOR[dt]
