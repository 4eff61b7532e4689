"""NaN, infinities and values just outside fp16's range in the int8 operators, on every plan of the products: what is
not a number stays visible as one, and the same values set the same flags whatever the batch."""

import pytest
import torch

from expert_serving_amd import abi

import plain_block as P
from gpu_util import dev, f32, say
from test_gpu_block import Block, tiny
from test_gpu_int8 import DT, offsets_of, on, run_ffn
from test_gpu_int8_large import codes, draw_ffn, gen

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
H_RANGE, Y_RANGE = abi.MOE_FLAG_H_RANGE, abi.MOE_FLAG_Y_RANGE

PLANS = {
    # H, I, rows per expert, top_k
    "stream, rows quantised on the way": (128, 256, [3, 0, 5, 2], 1),
    "stream, wide blocks": (4096, 512, [1] * 8, 8),
    "stream, few long rows": (512, 2048, [4, 6, 0, 0], 1),
    "stream": (512, 256, [40, 0, 7, 33], 2),
    "32-row tiles": (7168, 640, [15, 33, 1, 0, 20, 40, 9, 17, 30, 5, 6, 12, 18, 11, 16, 7], 2),
    "split gate and up": (7168, 2048, [1] * 8, 8),
    "32-row tiles, split down": (4096, 14336, [14, 20, 9, 3, 0, 11, 1, 6], 2),
    "large tiles": (384, 640, [300, 1, 66, 130, 0, 3], 4),
    "large tiles, split down": (2048, 14336, [300, 129, 63, 20, 0, 0, 0, 0], 2),
}


def plan(name):
    H, I, counts, k = PLANS[name]
    return H, I, len(counts), offsets_of(counts), k


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("name", PLANS)
def test_a_nan_row_scale_stays_in_its_row(name, dt):
    say(f"nan rows: {name} {dt}")
    H, I, E, off, k = plan(name)
    rows, g = int(off[-1]), gen(H + I)
    x, xs = codes(g, rows, H), (1 + torch.rand(rows, generator=g, device=dev())) / 73
    w = abi.int8_ffn(*draw_ffn(H, I, E, H + I))
    bad = sorted({0, rows // 2, rows - 1})
    want, flags = run_ffn(x, xs, on(off), w, H, I, E, rows // k, k, dt)
    assert flags == 0 and torch.isfinite(want).all()
    xs[bad] = NAN
    y, flags = run_ffn(x, xs, on(off), w, H, I, E, rows // k, k, dt)
    assert torch.isnan(y[bad]).all()
    rest = [r for r in range(rows) if r not in bad]
    assert torch.equal(y[rest], want[rest])
    assert flags == (H_RANGE | Y_RANGE if dt == "f16" else H_RANGE)


@pytest.mark.parametrize("which", ["gate", "up"])
@pytest.mark.parametrize("name", PLANS)
def test_a_nan_weight_scale_reaches_its_expert_only(name, which):
    """One channel of one expert's gate or up scales: a NaN in every h row of that expert."""
    H, I, E, off, k = plan(name)
    rows, g = int(off[-1]), gen(H + I)
    x, xs = codes(g, rows, H), (1 + torch.rand(rows, generator=g, device=dev())) / 73
    parts = draw_ffn(H, I, E, H + I)
    want, _ = run_ffn(x, xs, on(off), abi.int8_ffn(*parts), H, I, E, rows // k, k, "f32")
    parts[which == "up"][1][0, I - 3] = NAN
    y, flags = run_ffn(x, xs, on(off), abi.int8_ffn(*parts), H, I, E, rows // k, k, "f32")
    n = int(off[1])
    assert torch.isnan(y[:n]).all() and torch.equal(y[n:], want[n:]) and flags == H_RANGE


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", [(5, 128), (5, 2048), (5, 7168), (3, 14336), (2, 40960), (2, 131072),
                                       (16385, 1024), (16385, 2048)])
def test_quantised_rows_that_are_not_finite(rows, cols, dt):
    """Their scale is not finite either (NaN for a NaN); the other rows are those of a tensor without them."""
    g = gen(cols)
    x = torch.randn(rows, cols, generator=g, device=dev()).to(DT[dt][0])
    c0, s0 = abi.quantize_int8(x)
    for at, v in ((0, NAN), (cols - 1, NAN), (cols // 2 + 1, INF), (5, -INF)):
        bad = x.clone()
        bad[1, at] = v
        c, s = abi.quantize_int8(bad)
        keep = [r for r in range(min(rows, 5)) if r != 1] + [rows - 1] * (rows > 5)
        assert torch.isnan(s[1]) if v != v else torch.isinf(s[1])
        assert torch.equal(c[keep], c0[keep]) and torch.equal(s[keep], s0[keep])


@pytest.mark.parametrize("stream", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [128, 2048, 7168, 131072])
def test_norm_codes_of_what_is_not_finite(cols, stream):
    g = gen(cols + 1)
    x = torch.randn(3, cols, generator=g, device=dev()).to(DT[stream][0])
    weight = 1 + 0.1 * torch.randn(cols, generator=g, device=dev())

    def norm(x, weight):
        c, s = torch.empty(3, cols, dtype=torch.int8, device=dev()), f32(3)
        abi.moe_norm(3, cols, DT[stream][1], x, weight, 1e-6, abi.MOE_BF16, None, c, s)
        return c, s

    c0, s0 = norm(x, weight)
    for v in (NAN, INF, -INF):
        bad = x.clone()
        bad[1, 77] = v
        c, s = norm(bad, weight)
        assert torch.isnan(s[1]) and torch.equal(c[::2], c0[::2]) and torch.equal(s[::2], s0[::2])
    weight[cols - 5] = NAN
    assert torch.isnan(norm(x, weight)[1]).all()


@pytest.mark.parametrize("norms", [True, False])
@pytest.mark.parametrize("tokens", [1, 9, 60, 300])
def test_a_nan_token_of_the_int8_block(tokens, norms):
    """Its routing finds no expert; its shared expert has to answer NaN, and no other token notices."""
    b = Block(tiny(tokens=tokens, top_k=4, k_choices=None, capacity_factor=0.0, shared_inter=384), seed=31, norms=norms,
              scale=0.0)
    outs = []
    for value in (None, NAN):
        if value is not None:
            b.x[tokens // 2, 3] = value
        out, ws = torch.empty(b.T, b.H, dtype=torch.bfloat16, device=dev()), b.workspace(True)
        b.run(True, out, ws)
        torch.cuda.synchronize()
        outs.append((out, abi.moe_read_device_flags(ws)))
    (want, f0), (out, f1) = outs
    keep = [t for t in range(tokens) if t != tokens // 2]
    assert torch.isnan(out[tokens // 2]).all() and torch.equal(out[keep], want[keep])
    assert f0 == 0 and f1 & H_RANGE


def line(name, gate, up):
    """Every h is silu(gate) * up in row 0, and of 2^-8 times smaller gates and ups in the others: row codes 1, weight
    codes 1 in the first column and 0 elsewhere, so that the int32 sums are 1."""
    H, I, E, off, k = plan(name)
    rows = int(off[-1])
    x = torch.ones(rows, H, dtype=torch.int8, device=dev())
    xs = torch.full((rows,), 2.0 ** -8, device=dev())
    xs[0] = 1.0
    first = torch.zeros(E, I, H, dtype=torch.int8, device=dev())
    first[:, :, 0] = 1
    down = torch.ones(E, H, I, dtype=torch.int8, device=dev())
    of = lambda v, n: torch.full((E, n), v, device=dev())  # noqa: E731
    w = abi.int8_ffn((first, of(gate, I)), (first, of(up, I)), (down, of(2.0 ** -16, H)))
    y, flags = run_ffn(x, xs, on(off), w, H, I, E, rows // k, k, "f32")
    return y, flags, 127.0 * I * 2.0 ** -16 / 127   # y of a row of equal h is h times the last


@pytest.mark.parametrize("name", PLANS)
def test_h_between_the_largest_fp16_value_and_its_rounding(name):
    """fp32 values above 65504 that round to it are out of range on every plan; 65504 itself is not.  silu(256) is 256,
    so h is one rounding of 256 times the up value (exact for these), y four more of fp32 and up to eight parts."""
    for up, flag in ((255.875, 0), (65510.0 / 256, H_RANGE), (65519.0 / 256, H_RANGE), (65520.0 / 256, H_RANGE),
                     (1024.0, H_RANGE)):
        for sign in (1.0, -1.0):
            y, flags, f = line(name, 256.0, sign * up)
            assert flags == flag, (up, sign)
            want = sign * 65504.0 * f
            assert torch.all((y[0] - want).abs() <= 12 * P.U32 * abs(want)), (up, sign)


@pytest.mark.parametrize("name", PLANS)
def test_h_of_gates_near_the_largest_float(name):
    """silu of a huge gate is the gate, and of a huge negative one zero: clamped and flagged, not a NaN."""
    for gate, up, h, flag in ((3.0e38, 1.0, 65504.0, H_RANGE), (3.0e38, -1.0, -65504.0, H_RANGE),
                              (-3.0e38, 1.0, 0.0, 0), (1.0e38, 1.0, 65504.0, H_RANGE)):
        y, flags, f = line(name, gate, up)
        assert flags == flag, (gate, up)
        assert torch.all((y[0] - h * f).abs() <= 12 * P.U32 * abs(h) * f), (gate, up)
