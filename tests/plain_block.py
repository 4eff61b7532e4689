"""Plain 64-bit forms of routing with a balance bias, the int8 products and the block norms, in numpy.

Written from the definitions in include/moe_mi355x.h and independent of the library.
"""

import numpy as np

U32 = 2.0 ** -24   # half a step of fp32, relative
U16 = 2.0 ** -11   # of fp16
UB16 = 2.0 ** -8   # of bf16
HALF_STEP = {"f32": U32, "f16": U16, "bf16": UB16}


def route_biased(logits, bias, k, kpt=None, score="sigmoid", renorm=True, scale=1.0, G=1, keep=1, topn=1):
    """ids [T, k], gates [T, k] (fp64), one token and one expert at a time."""
    T, E = logits.shape
    big = float(np.finfo(np.float32).max)
    ids, gates = np.full((T, k), -1, np.int64), np.zeros((T, k))
    for t in range(T):
        kt = k if kpt is None else int(kpt[t])
        if not 1 <= kt <= k:
            continue
        l = np.clip(logits[t].astype(np.float64), -big, big)
        here = (bias > -np.inf) & ~np.isnan(logits[t]) & ~np.isnan(bias)
        s = np.zeros(E)
        with np.errstate(over="ignore"):
            if score == "sigmoid":
                s[here] = 1.0 / (1.0 + np.exp(-l[here]))
            elif here.any():
                e = np.exp(l[here] - l[here].max())
                s[here] = e / e.sum()
        key = {e: s[e] + float(bias[e]) for e in range(E) if here[e]}
        if G > 1:
            n = E // G
            totals = []
            for g in range(G):
                mine = sorted((key[e] for e in range(g * n, (g + 1) * n) if e in key), reverse=True)[:max(topn, 1)]
                if mine:
                    totals.append((-sum(mine), g))
            kept = {g for _, g in sorted(totals)[:keep]}
            key = {e: v for e, v in key.items() if e // n in kept}
        chosen = [e for _, e in sorted((-v, e) for e, v in key.items())[:kt]]
        w = np.array([s[e] for e in chosen])
        if renorm and len(w):
            w = w / w.sum() if w.sum() > 0 else np.zeros(len(w))
        ids[t, :len(chosen)] = chosen
        gates[t, :len(chosen)] = w * scale
    return ids, gates


def quotients(x):
    """127 x / amax of each row in fp64 (0 for rows of zeros), and the rows' scales."""
    x = x.astype(np.float64)
    top = np.abs(x).max(1, keepdims=True)
    return np.divide(127 * x, top, out=np.zeros_like(x), where=top > 0), (top / 127)[:, 0]


def codes(x):
    q, s = quotients(x)
    return np.rint(q), s


def grouped(a, w, offsets):
    """rows of a [R, K] times w[e].T for each row's expert, in fp64 (rows behind the last group: 0)."""
    out = np.zeros((a.shape[0], w.shape[1]))
    for e in range(w.shape[0]):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        out[r] = a[r].astype(np.float64) @ w[e].astype(np.float64).T
    return out


def expert_of_row(offsets, rows):
    e = np.searchsorted(np.asarray(offsets), np.arange(rows), side="right") - 1
    return np.minimum(e, len(offsets) - 2)


def ffn_int8(xc, xs, offsets, gate, up, down):
    """y [R, H] and how far the library may be from it before the rounding of y.

    gate, up, down: (codes, scales).  u = 2^-24.  The library's gate and up values carry three roundings each
    (int32 to fp32, the product of the scales, their product); silu turns a relative error d of g into at most
    (1 + |g|) d, and its own exponential, sum, reciprocal and products add less than ten roundings.  So h is
    off by at most (16 + 4 |g|) u, relative.  Where that crosses a rounding boundary of fp16, h and through it
    its code (or, by the row's maximum, every code of the row) may be the neighbour: the bound adds each
    possible change of a code times its weight.
    """
    e = expert_of_row(offsets, len(xc))
    g = grouped(xc, gate[0], offsets) * xs[:, None] * gate[1].astype(np.float64)[e]
    u = grouped(xc, up[0], offsets) * xs[:, None] * up[1].astype(np.float64)[e]
    with np.errstate(over="ignore"):
        h = g / (1 + np.exp(-g)) * u
    d = (16 + 4 * np.abs(g)) * U32
    low, mid, high = (np.clip(h * f, -65504, 65504).astype(np.float16).astype(np.float64)
                      for f in (1 - d, 1.0, 1 + d))
    top = [np.abs(v).max(1, keepdims=True) for v in (low, mid, high)]
    c, s = codes(mid)

    def rounded(v, t):
        return np.rint(np.divide(127 * v, t, out=np.zeros_like(v), where=t > 0))

    ends = [rounded(v, t) for v in (low, high) for t in top]
    moved = np.max([np.abs(x - c) for x in ends], axis=0)
    sd = down[1].astype(np.float64)[e]
    y = grouped(c, down[0], offsets) * s[:, None] * sd
    absdown = np.abs(down[0].astype(np.int16))
    slack = grouped(moved, absdown, offsets) * s[:, None] * sd
    # the scale of a row whose maximum may move, and the fp32 steps: the scale, the int32 sum, two products, and
    # up to eight partial sums
    shift = np.divide(np.abs(np.stack(top) - top[1]).max(0), top[1], out=np.zeros_like(top[1]), where=top[1] > 0)
    total = grouped(np.abs(c), absdown, offsets) * s[:, None] * sd
    return y, slack + total * (shift + 12 * U32)


def rms_norm(x, weight, eps):
    x = x.astype(np.float64)
    n = x / np.sqrt((x * x).mean(1, keepdims=True) + eps)
    return n if weight is None else n * weight.astype(np.float64)


def combine_norm(y, rows, gates, shared, weight, eps, gate, residual, scale):
    """out [T, H] and how far the library may be from it before the rounding of out.

    u = 2^-24: y of a token is a chain of at most k + 1 rounded sums, off by (k + 2) u of the sum A of its terms'
    magnitudes.  The sum of squares is one of at most 128 rounded steps per thread and a tree of 16, so
    its root is off by less than 80 u plus what y's own error moves it by (at most its norm over y's); each
    further factor and the last sum add one rounding.
    """
    T, k = rows.shape
    H = y.shape[1]
    v, a = np.zeros((T, H)), np.zeros((T, H))
    for j in range(k):
        live = rows[:, j] >= 0
        term = gates[live, j:j + 1].astype(np.float64) * y[rows[live, j]].astype(np.float64)
        v[live] += term
        a[live] += np.abs(term)
    if shared is not None:
        v += shared.astype(np.float64)
        a += np.abs(shared.astype(np.float64))
    err = (k + 2) * U32 * a
    n = v
    if weight is not None:
        root = np.sqrt((v * v).mean(1, keepdims=True) + eps)
        w = weight.astype(np.float64)
        n = v / root * w
        err = err / root * np.abs(w) + np.abs(n) * (84 * U32 + np.sqrt((err * err).mean(1, keepdims=True)) / root)
    if gate is not None:
        g = gate.astype(np.float64)
        n, err = n * g, err * np.abs(g) + U32 * np.abs(n * g)
    r = 0.0 if residual is None else scale * residual.astype(np.float64)
    return n + r, err + 2 * U32 * (np.abs(n) + np.abs(r))
