"""The norm in front of the layer and the end of the block against plain 64-bit forms.

moe_norm's tolerance, u = 2^-24: a thread adds at most 64 squares one after another, and a tree of at most 22
steps joins the threads; the sum is off by at most 88 u, its root by 44 u; the root, the quotient and the two
products add five: 50 u of the value, and the output's own rounding.
"""

import numpy as np
import pytest
import torch

from expert_serving_amd import abi

import plain_block as P
from gpu_util import dev, say

pytestmark = pytest.mark.gpu

DT = {"f32": (torch.float32, abi.MOE_F32), "f16": (torch.float16, abi.MOE_F16), "bf16": (torch.bfloat16, abi.MOE_BF16)}


def np64(t):
    return t.detach().cpu().double().numpy()


def randn(seed, *shape, dtype=torch.float32):
    g = torch.Generator(device=dev())
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device=dev()).to(dtype)


@pytest.mark.parametrize("src,out", [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("rows,cols,codes", [(1, 64, False), (3, 128, True), (5, 832, False), (61, 4096, True),
                                             (7, 7168, True), (2, 16384, True), (2, 33024, True), (1, 70016, False)])
def test_norm(rows, cols, codes, src, out):
    say(f"norm {rows} x {cols} {src} -> {out} codes {codes}")
    x = (randn(cols, rows, cols) * torch.exp(2 * randn(cols + 1, rows, 1))).to(DT[src][0])
    x[-1, ::3] = 0
    w = 1 + 0.2 * randn(cols + 2, cols)
    o = torch.full((rows, cols), -7.0, device=dev(), dtype=DT[out][0])
    c = torch.empty(rows, cols, dtype=torch.int8, device=dev()) if codes else None
    s = torch.empty(rows, device=dev()) if codes else None
    abi.moe_norm(rows, cols, DT[src][1], x, w, 1e-6, DT[out][1], o, c, s)
    want = P.rms_norm(np64(x), np64(w), 1e-6)
    tol = (50 * P.U32 + P.HALF_STEP[out]) * np.abs(want) + 1e-44
    assert np.all(np.abs(np64(o) - want) <= tol)
    if codes:
        q, sc = P.quotients(want)
        # the row's factor cancels in a quotient: x w, 127 (x w), the maximum and the quotient are rounded
        assert np.all(np.abs(c.cpu().numpy() - q) <= 0.5 + 127 * 4 * P.U32)
        assert np.all(np.abs(np64(s) - sc) <= 52 * P.U32 * sc)
        c2, s2 = torch.empty_like(c), torch.empty_like(s)
        abi.moe_norm(rows, cols, DT[src][1], x, w, 1e-6, DT[out][1], None, c2, s2)   # codes alone: the same ones
        assert torch.equal(c, c2) and torch.equal(s, s2)


def test_norm_of_zero_rows_and_without_weight():
    x = torch.zeros(3, 256, device=dev())
    x[1] = randn(1, 256)
    o, c, s = torch.empty_like(x), torch.empty(3, 256, dtype=torch.int8, device=dev()), torch.empty(3, device=dev())
    abi.moe_norm(3, 256, abi.MOE_F32, x, None, 1e-12, abi.MOE_F32, o, c, s)
    want = P.rms_norm(np64(x), None, 1e-12)
    assert np.all(np.abs(np64(o) - want) <= 51 * P.U32 * np.abs(want))
    assert (c[0] == 0).all() and s[0] == 0 and (o[0] == 0).all()


def test_norm_in_place():
    for dt in ("f32", "bf16"):
        x = randn(4, 9, 4096, dtype=DT[dt][0])
        o = torch.empty_like(x)
        abi.moe_norm(9, 4096, DT[dt][1], x, None, 1e-6, DT[dt][1], o, None, None)
        abi.moe_norm(9, 4096, DT[dt][1], x, None, 1e-6, DT[dt][1], x, None, None)
        assert torch.equal(x, o)


# ---- the end of the block --------------------------------------------------------------------------------------

def gate_of(kind, T, H):
    if kind is None:
        return None
    name, dt = kind
    t = DT[dt][0]
    if name == "channel":
        return randn(7, 1, H, dtype=t)
    if name == "token":
        return randn(7, T, 1, dtype=t)
    if name == "both":
        return randn(7, T, H, dtype=t)
    if name == "odd":       # rows that start anywhere
        return randn(7, T, H + 3, dtype=t)[:, 1:1 + H]
    return randn(7, T, H + 8, dtype=t)[:, :H]   # "wide": aligned rows, further apart


END_CASES = [
    # T, H, k, y, stream, shared, gate, post norm, residual scale, share of dropped slots
    (1, 64, 1, "f16", "bf16", False, None, True, 1.0, 0.0),
    (5, 4096, 2, "f16", "bf16", True, ("channel", "bf16"), True, 0.5, 0.3),
    (33, 7168, 8, "f16", "bf16", True, ("both", "bf16"), True, 1.0, 0.1),
    (7, 2048, 3, "bf16", "f32", False, ("both", "f32"), True, -2.0, 0.6),
    (4, 512, 16, "f32", "f32", True, ("token", "f32"), True, 1.0, 0.5),
    (3, 132, 4, "f32", "f32", True, ("odd", "f32"), True, 1.0, 0.2),
    (6, 832, 5, "f16", "f32", False, ("odd", "bf16"), False, 0.25, 0.2),
    (6, 1024, 2, "bf16", "bf16", False, ("wide", "bf16"), True, 0.0, 0.0),
    (3, 33024, 2, "f16", "bf16", True, ("token", "bf16"), True, 1.0, 0.4),
    (2, 16640, 9, "f32", "bf16", False, ("channel", "f32"), True, 1.0, 0.0),
    (300, 256, 2, "f32", "bf16", False, None, False, 1.0, 1.0),
]


@pytest.mark.parametrize("case", END_CASES, ids=lambda c: "-".join(str(v) for v in c[:5]))
def test_combine_norm(case):
    T, H, k, y, stream, sh, gk, normed, scale, gone = case
    say(f"combine_norm {case}")
    act = abi.MOE_BF16 if H % 64 == 0 else abi.MOE_F32
    shape = abi.make_shape(num_tokens=T, hidden=H, num_experts=16, intermediate=64, top_k=k, act_dtype=act)
    yp = randn(1, T * k, H, dtype=DT[y][0])
    r = np.random.default_rng(T + H)
    rows = r.permutation(T * k).reshape(T, k).astype(np.int32)
    rows[r.random((T, k)) < gone] = -1
    for i in range(T * k):                          # rows nothing points at are not read
        if i not in set(rows.reshape(-1).tolist()) and T * k < 200:
            yp[i] = float("nan")
    g = torch.rand(T, k, device=dev()) + 0.01
    shared = randn(2, T, H, dtype=DT[y][0]) if sh else None
    w = 1 + 0.2 * randn(3, H) if normed else None
    res = randn(4, T, H, dtype=DT[stream][0])
    gate = gate_of(gk, T, H)
    b = abi.make_block(post_norm=w, eps=1e-5, gate=gate, residual_scale=scale, stream_dtype=DT[stream][1])
    out = torch.full((T, H), -7.0, device=dev(), dtype=DT[stream][0])
    ros = torch.from_numpy(rows).to(dev())
    abi.moe_combine_norm(shape, b, DT[y][1], yp, ros, g, shared, res if scale else None, out)
    want, err = P.combine_norm(np.nan_to_num(np64(yp)), rows, np64(g), None if shared is None else np64(shared),
                               None if w is None else np64(w), 1e-5, None if gate is None else np64(gate),
                               np64(res), scale)
    tol = err + P.HALF_STEP[stream] * np.abs(want) + 1e-44
    assert np.all(np.abs(np64(out) - want) <= tol), np.max(np.abs(np64(out) - want) / tol)
    if scale:                                       # the residual's own buffer may take the result
        abi.moe_combine_norm(shape, b, DT[y][1], yp, ros, g, shared, res, res)
        assert torch.equal(res, out)


def test_end_is_moe_combine_without_norm_gate_and_residual():
    T, H, k = 37, 1024, 4
    shape = abi.make_shape(num_tokens=T, hidden=H, num_experts=8, intermediate=64, top_k=k)
    y, g, sh = randn(1, T * k, H), torch.rand(T, k, device=dev()), randn(2, T, H)
    rows = torch.randperm(T * k, device=dev(), dtype=torch.int32).view(T, k)
    a, b = torch.empty(T, H, device=dev()), torch.empty(T, H, device=dev())
    abi.moe_combine(shape, y, rows, g, sh, a)
    abi.moe_combine_norm(shape, abi.make_block(residual_scale=0.0, stream_dtype=abi.MOE_F32), abi.MOE_F32, y, rows, g,
                         sh, None, b)
    assert torch.equal(a, b)


def test_residual_scale_of_zero_reads_no_residual():
    """A residual scale of 0 does not read the residual: infinities there do not reach the output."""
    T, H, k = 3, 256, 1
    shape = abi.make_shape(num_tokens=T, hidden=H, num_experts=8, intermediate=64, top_k=k)
    rows = torch.arange(T, device=dev(), dtype=torch.int32).view(T, k)
    out = torch.empty(T, H, device=dev())
    res = torch.full((T, H), float("inf"), device=dev())
    abi.moe_combine_norm(shape, abi.make_block(residual_scale=0.0, stream_dtype=abi.MOE_F32), abi.MOE_F32,
                         randn(1, T, H), rows, torch.ones(T, k, device=dev()), None, res, out)
    assert torch.isfinite(out).all()


def test_more_rows_than_one_axis_of_a_launch_holds():
    """Blocks of a row each, with 2^32 threads and more."""
    rows = 70_000_000
    x = torch.ones(rows, 128, device=dev(), dtype=torch.bfloat16)
    x[-1] = torch.linspace(-3, 3, 128, device=dev()).to(torch.bfloat16)
    codes, scales = abi.quantize_int8(x)
    assert np.array_equal(codes[-1].cpu().numpy(), P.codes(np64(x[-1:]))[0][0])
    assert bool((codes[:-1:65_521] == 127).all()) and int(codes[-2].sum()) == 127 * 128
    assert float(scales[-2]) == np.float32(1) / np.float32(127)
    del codes, scales
    want = P.rms_norm(np64(x[-1:]), None, 1e-5)
    abi.moe_norm(rows, 128, abi.MOE_BF16, x, None, 1e-5, abi.MOE_BF16, x, None, None)
    assert np.all(np.abs(np64(x[-1:]) - want) <= (P.UB16 + 50 * P.U32) * np.abs(want))
    assert bool((x[:-1:65_521] == 1).all()) and bool((x[-2] == 1).all())
    del x
    T, H = 17_000_000, 64
    shape = abi.make_shape(num_tokens=T, hidden=H, num_experts=1, intermediate=64, top_k=1)
    y = torch.ones(T, H, device=dev(), dtype=torch.bfloat16)
    ros, g = torch.arange(T, device=dev(), dtype=torch.int32).view(T, 1), torch.ones(T, 1, device=dev())
    g[-1], g[-2] = 3.0, 2.0
    res = torch.ones(T, H, device=dev(), dtype=torch.bfloat16)
    abi.moe_combine_norm(shape, abi.make_block(residual_scale=1.0, stream_dtype=abi.MOE_BF16), abi.MOE_BF16, y, ros, g,
                         None, res, res)
    assert bool((res[-1] == 4).all()) and bool((res[-2] == 3).all()) and bool((res[:-2:4_099] == 2).all())
