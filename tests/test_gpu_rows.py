"""Rows to expert order and the gradients of dispatch and combine, against 64-bit forms and against differences.

Tolerances: an output of one product or copy is off by half a step of its type.  fp32 sums of n terms in any order are
off by at most n half steps of the sum of the terms' magnitudes; the kernels add a thread's at most H / 16 terms, six
steps of a wavefront and eight wavefronts, or a token's k slots.
"""

import numpy as np
import pytest
import torch

from expert_serving_amd import abi

import plain_fp8 as P
from gpu_util import dev, say
from test_gpu_fp8 import DT, FP8, np64, on

pytestmark = pytest.mark.gpu

NAMES = {abi.MOE_F32: "f32", abi.MOE_F16: "f16", abi.MOE_BF16: "bf16"}


def shape_of(T, H, k):
    act = abi.MOE_BF16 if H % 64 == 0 else abi.MOE_F32
    return abi.make_shape(num_tokens=T, hidden=H, num_experts=max(16, k), intermediate=64, top_k=k, act_dtype=act)


def slots(r, T, k, dropped, extra=0):
    """row_of_slot [T, k]: kept slots take distinct rows of 0 .. T k + extra - 1, dropped ones -1."""
    rows = r.permutation(T * k + extra)[:T * k].astype(np.int32).reshape(T, k)
    rows[r.random((T, k)) < dropped] = -1
    return rows


CASES = [
    # tokens, H, k, share of dropped slots, rows more than slots
    (1, 128, 1, 0.0, 0), (1, 7168, 8, 0.0, 0), (3, 64, 2, 0.0, 1), (17, 640, 3, 0.3, 4), (5, 256, 16, 0.5, 0),
    (33, 4096, 2, 0.1, 0), (4, 512, 5, 1.0, 3), (301, 192, 9, 0.05, 0), (2, 14336, 4, 0.0, 0), (64, 2048, 8, 0.2, 2),
]
ODD = [(7, 8, 2, 0.0, 0), (13, 40, 3, 0.3, 1), (6, 1000, 4, 0.2, 0)]   # (H no multiple of 64)


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,H,k,dropped,extra", CASES + ODD)
def test_dispatch_rows(T, H, k, dropped, extra, dt, weighted):
    say(f"dispatch rows {T} x {H} k={k} {dt} {weighted}")
    r = np.random.default_rng(T + H + k)
    n = T * k + extra
    ros, g = slots(r, T, k, dropped, extra), r.normal(size=(T, k)).astype(np.float32)
    x = on(r.normal(size=(T, H)), DT[dt][0])
    out = torch.full((n, H), -7.0, device=dev(), dtype=x.dtype)
    abi.moe_dispatch_rows(shape_of(T, H, k), DT[dt][1], x, on(ros), on(g) if weighted else None, n, out)
    want = np.full((n, H), -7.0)
    x64 = np64(x)
    for t in range(T):
        for j in range(k):
            if ros[t, j] >= 0:
                want[ros[t, j]] = x64[t] * (float(g[t, j]) if weighted else 1.0)
    if not weighted:
        assert np.array_equal(np64(out), want)
    else:
        # one product in fp32, then the type's rounding
        assert np.all(np.abs(np64(out) - want) <= P.rounded(want, P.U32 * np.abs(want), dt))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,H,k,dropped,extra", [c for c in CASES if c[1] % 128 == 0])
def test_dispatch_rows_fp8(T, H, k, dropped, extra, dt):
    """Codes and scales are those of quantize_fp8, at the slots' rows."""
    r = np.random.default_rng(T + H + k)
    n = T * k + extra
    ros = slots(r, T, k, dropped, extra)
    x = on(r.normal(size=(T, H)) * np.exp(r.normal(size=(T, 1))), DT[dt][0])
    codes = torch.full((n, H), 0x55, device=dev(), dtype=torch.uint8)
    scales = torch.full((n, H // 128), -7.0, device=dev())
    abi.moe_dispatch_rows_fp8(shape_of(T, H, k), DT[dt][1], x, on(ros), n, codes, scales)
    c, s = abi.quantize_fp8(x)
    c = c.view(torch.uint8).cpu().numpy()
    want_c, want_s = np.full((n, H), 0x55, np.uint8), np.full((n, H // 128), -7.0)
    for t in range(T):
        for j in range(k):
            if ros[t, j] >= 0:
                want_c[ros[t, j]], want_s[ros[t, j]] = c[t], np64(s)[t]
    assert np.array_equal(codes.cpu().numpy(), want_c) and np.array_equal(np64(scales), want_s)


def backward(T, H, k, dt, dp, ros, n, g, x, want_x=True, want_w=True):
    dx = torch.full((T, H), -7.0, device=dev(), dtype=DT[dt][0]) if want_x else None
    dw = torch.full((T, k), -7.0, device=dev()) if want_w else None
    abi.moe_dispatch_rows_backward(shape_of(T, H, k), DT[dt][1], dp, ros, n, g, x, dx, dw)
    return dx, dw


@pytest.mark.parametrize("mode", ["plain", "weighted", "with weights", "weights alone"])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,H,k,dropped,extra", CASES + ODD)
def test_dispatch_rows_backward(T, H, k, dropped, extra, dt, mode):
    say(f"dispatch rows backward {T} x {H} k={k} {dt} {mode}")
    r = np.random.default_rng(T + H + k)
    n = T * k + extra
    ros, g = slots(r, T, k, dropped, extra), r.normal(size=(T, k)).astype(np.float32)
    x, dp = on(r.normal(size=(T, H)), DT[dt][0]), on(r.normal(size=(n, H)), DT[dt][0])
    unnamed = np.setdiff1d(np.arange(n), ros)
    dp[on(unnamed)] = float("nan")                  # rows that no slot names are not used
    weighted, grads = mode != "plain", mode in ("with weights", "weights alone")
    dx, dw = backward(T, H, k, dt, dp, on(ros), n, on(g) if weighted else None, x if grads else None,
                      mode != "weights alone", grads)
    p, x64 = np64(dp), np64(x)
    want, size = np.zeros((T, H)), np.zeros((T, H))
    want_w, size_w = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            if ros[t, j] >= 0:
                term = p[ros[t, j]] * (float(g[t, j]) if weighted else 1.0)
                want[t] += term
                size[t] += np.abs(term)
                want_w[t, j] = p[ros[t, j]] @ x64[t]
                size_w[t, j] = np.abs(p[ros[t, j]]) @ np.abs(x64[t])
    if dx is not None:
        assert np.all(np.abs(np64(dx) - want) <= P.rounded(want, (k + 1) * P.U32 * size, dt))
    if dw is not None:
        assert np.all(np.abs(np64(dw) - want_w) <= (H / 16 + 16) * P.U32 * size_w)


@pytest.mark.parametrize("mode", ["both", "rows", "gates", "in place"])
@pytest.mark.parametrize("ydt,odt", [("bf16", "f32"), ("f32", "f32"), ("f16", "bf16"), ("bf16", "bf16"), ("f32", "f16")])
@pytest.mark.parametrize("T,H,k,dropped,extra", CASES + ODD)
def test_combine_backward(T, H, k, dropped, extra, ydt, odt, mode):
    say(f"combine backward {T} x {H} k={k} {ydt} {odt} {mode}")
    r = np.random.default_rng(T + H + k)
    n = T * k + extra
    ros, g = slots(r, T, k, dropped, extra), r.random((T, k)).astype(np.float32)
    y, do = on(r.normal(size=(n, H)), DT[ydt][0]), on(r.normal(size=(T, H)), DT[odt][0])
    y64, o64 = np64(y), np64(do)
    dy = {"gates": None, "in place": y}.get(mode, torch.full((n, H), -7.0, device=dev(), dtype=y.dtype))
    dg = None if mode == "rows" else torch.full((T, k), -7.0, device=dev())
    abi.moe_combine_backward(shape_of(T, H, k), DT[odt][1], do, DT[ydt][1], None if mode == "rows" else y, on(ros),
                             on(g), n, dy, dg)
    want = y64.copy() if mode == "in place" else np.full((n, H), -7.0)
    bound, want_g, size_g = np.zeros((n, H)), np.zeros((T, k)), np.zeros((T, k))
    named = np.zeros(n, bool)
    for t in range(T):
        for j in range(k):
            q = ros[t, j]
            if q >= 0:
                named[q] = True
                want[q] = o64[t] * float(g[t, j])
                bound[q] = P.U32 * np.abs(want[q])
                want_g[t, j], size_g[t, j] = y64[q] @ o64[t], np.abs(y64[q]) @ np.abs(o64[t])
    if dy is not None:
        got = np64(dy)
        assert np.all(np.abs(got - want)[named] <= P.rounded(want, bound, ydt)[named])
        assert np.array_equal(got[~named], want[~named])
    if dg is not None:
        assert np.all(np.abs(np64(dg) - want_g) <= (H / 16 + 16) * P.U32 * size_g)


def test_rows_outside_the_buffer_count_as_none():
    """Entries at or beyond num_rows, and any negative one, name no row: nothing is read or written there."""
    T, H, k, n = 9, 256, 4, 20
    r = np.random.default_rng(0)
    ros = slots(r, T, k, 0.0)
    big = ros.copy()
    big[ros >= n] = np.resize(np.array([n, 2 ** 31 - 1, -2, -2 ** 31, 1 << 20], np.int32), (ros >= n).sum())
    none = np.where(ros < n, ros, -1).astype(np.int32)
    x, g = on(r.normal(size=(T, H)), torch.bfloat16), on(r.random((T, k)).astype(np.float32))
    rows = on(r.normal(size=(n, H)), torch.bfloat16)
    s, b = shape_of(T, H, k), abi.MOE_BF16
    for m in (big, none):
        m = on(m)
        outs = [torch.zeros(n, H, device=dev(), dtype=torch.bfloat16), torch.zeros(n, H, device=dev(), dtype=torch.uint8),
                torch.zeros(n, H // 128, device=dev()), torch.zeros(T, H, device=dev(), dtype=torch.bfloat16),
                torch.full((T, k), -7.0, device=dev()), torch.zeros(n, H, device=dev(), dtype=torch.bfloat16),
                torch.full((T, k), -7.0, device=dev())]
        abi.moe_dispatch_rows(s, b, x, m, g, n, outs[0])
        abi.moe_dispatch_rows_fp8(s, b, x, m, n, outs[1], outs[2])
        abi.moe_dispatch_rows_backward(s, b, rows, m, n, g, x, outs[3], outs[4])
        abi.moe_combine_backward(s, b, x, b, rows, m, g, n, outs[5], outs[6])
        if m.equal(on(big)):
            first = outs
    assert all(torch.equal(a, c) for a, c in zip(first, outs))
    assert (outs[4][on(none) < 0] == 0).all() and (outs[6][on(none) < 0] == 0).all()


def test_no_rows_at_all():
    T, H, k = 5, 256, 2
    s, b = shape_of(T, H, k), abi.MOE_BF16
    ros, g = torch.full((T, k), 3, dtype=torch.int32, device=dev()), torch.ones(T, k, device=dev())
    x, one = torch.ones(T, H, device=dev(), dtype=torch.bfloat16), torch.ones(1, H, device=dev(), dtype=torch.bfloat16)
    dx, dw = torch.ones_like(x), torch.ones_like(g)
    abi.moe_dispatch_rows(s, b, x, ros, g, 0, one)
    abi.moe_dispatch_rows_backward(s, b, one, ros, 0, g, x, dx, dw)
    assert (one == 1).all() and (dx == 0).all() and (dw == 0).all()
    abi.moe_combine_backward(s, b, x, b, one, ros, g, 0, one, dw.fill_(1))
    assert (one == 1).all() and (dw == 0).all()


def test_gradients_against_differences():
    """<out, weighting> as a function of x, weights, y and gates, against differences of the forward calls: every
    function is linear in each argument, so a difference is exact up to the forward's roundings (fp32)."""
    T, H, k = 6, 64, 3
    r = np.random.default_rng(5)
    n = T * k
    ros = on(slots(r, T, k, 0.2))
    s = abi.make_shape(num_tokens=T, hidden=H, num_experts=16, intermediate=64, top_k=k)
    f = lambda *sh: on(r.normal(size=sh).astype(np.float32))  # noqa: E731
    x, w, weight = f(T, H), f(T, k), f(n, H)
    named = torch.zeros(n, dtype=torch.bool, device=dev())
    named[ros[ros >= 0].long()] = True

    def sorted_sum(x, w):
        out = torch.zeros(n, H, device=dev())
        abi.moe_dispatch_rows(s, abi.MOE_F32, x, ros, w, n, out)
        return float((out.double() * weight.double())[named].sum())

    dx, dw = backward(T, H, k, "f32", weight, ros, n, w, x)
    y, out_weight = f(n, H), f(T, H)

    def combined(y, g):
        out = torch.zeros(T, H, device=dev())
        abi.moe_combine(s, y, ros, g, None, out)
        return float((out.double() * out_weight.double()).sum())

    dy, dg = torch.zeros(n, H, device=dev()), torch.zeros(T, k, device=dev())
    abi.moe_combine_backward(s, abi.MOE_F32, out_weight, abi.MOE_F32, y, ros, w, n, dy, dg)
    for fun, args, grads in ((sorted_sum, (x, w), (dx, dw)), (combined, (y, w), (dy, dg))):
        base = fun(*args)
        for i in (0, 1):
            step = torch.randn_like(args[i])
            moved = list(args)
            moved[i] = args[i] + step
            step = (moved[i].double() - args[i].double())
            d = fun(*moved) - base
            want = float((grads[i].double() * step).sum())
            # fp32 roundings of some thousand terms of size up to about 10 on either side
            assert abs(d - want) <= 1e-6 * 6000 and abs(want) > 1e-2, (fun, i, d, want)


def test_rows_past_32_bit_offsets():
    """2.2e9 elements in the permuted rows: the last row is reached and no other."""
    T, H, k = 16640, 8192, 16
    n = T * k
    s, b = shape_of(T, H, k), abi.MOE_BF16
    ros = torch.arange(n, dtype=torch.int32, device=dev()).view(T, k)
    g = torch.ones(T, k, device=dev())
    g[-1, -1] = 0.5
    x = torch.ones(T, H, device=dev(), dtype=torch.bfloat16)
    x[-1] = 2.0
    out = torch.zeros(n, H, device=dev(), dtype=torch.bfloat16)
    abi.moe_dispatch_rows(s, b, x, ros, g, n, out)
    assert (out[:-k] == 1).all() and (out[-k:-1] == 2).all() and (out[-1] == 1).all()
    dx, dw = torch.zeros_like(x), torch.zeros_like(g)
    abi.moe_dispatch_rows_backward(s, b, out, ros, n, g, x, dx, dw)
    assert (dx[:-1] == k).all() and (dx[-1] == 2 * (k - 1) + 0.5).all()
    assert (dw[:-1] == H).all() and (dw[-1, :-1] == 4 * H).all() and dw[-1, -1] == 2 * H
    abi.moe_combine_backward(s, b, x, b, out, ros, g, n, out, dw)
    assert (out[:-k] == 1).all() and (out[-k:-1] == 2).all() and (out[-1] == 1).all() and (dw[:-1] == H).all()
    codes = out.view(torch.uint8).view(-1)[:n * H].view(n, H)
    scales = torch.zeros(n, H // 128, device=dev())
    abi.moe_dispatch_rows_fp8(s, b, x, ros, n, codes, scales)
    assert (codes == 0x7E).all() and torch.allclose(scales[-1], scales[0] * 2)
