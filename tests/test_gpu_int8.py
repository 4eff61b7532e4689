"""The int8 operators against plain 64-bit forms.  Each tolerance counts the roundings of the fp32 steps
(2^-24 each, relative) and of the output's type; see plain_block.py for the FFN's."""

import numpy as np
import pytest
import torch

from expert_serving_amd import abi

import plain_block as P
from gpu_util import dev, i32, say

pytestmark = pytest.mark.gpu

DT = {"f32": (torch.float32, abi.MOE_F32), "f16": (torch.float16, abi.MOE_F16), "bf16": (torch.bfloat16, abi.MOE_BF16)}


def np64(t):
    return t.detach().cpu().double().numpy()


def offsets_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def on(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(dev())
    return t if dtype is None else t.to(dtype)


def weights(r, E, N, K):
    w = np.clip(np.rint(r.normal(size=(E, N, K)) * 32), -127, 127).astype(np.int8)
    return w, ((1 + 0.3 * r.random((E, N))) / (32 * K ** 0.5)).astype(np.float32)


# ---- quantisation --------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 128), (3, 512), (17, 640), (5, 2048), (2, 7168), (2, 14336), (2, 40960),
                                       (1, 131072)])
def test_quantize(dt, rows, cols):
    say(f"quantize {dt} {rows} x {cols}")
    r = np.random.default_rng(cols + rows)
    x = on(r.normal(size=(rows, cols)) * np.exp(3 * r.normal(size=(rows, 1))), DT[dt][0])
    x[0, 7] = x[0].abs().max() * 2                 # ties: half of the maximum is 63.5 steps
    x[0, 9], x[0, 64], x[0, 100] = x[0, 7] / 2, -x[0, 7] / 2, 0.0
    codes, scales = abi.quantize_int8(x)
    q, s = P.quotients(np64(x))
    c = codes.cpu().numpy()
    if dt == "f32":   # 127 v and the quotient are rounded once each
        assert np.all(np.abs(c - q) <= 0.5 + 127 * 2 * P.U32)
    else:             # 127 v is exact and no other quotient is within 9e-7 of a tie
        assert np.array_equal(c, np.rint(q))
    assert c[0, 9] == 64 and c[0, 64] == -64 and c[0, 7] == 127
    assert np.all(np.abs(scales.cpu().numpy() - s) <= P.U32 * s)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_quantize_zero_tiny_and_huge_rows(dt):
    x = torch.zeros(6, 256, device=dev(), dtype=DT[dt][0])
    ramp = torch.linspace(-1, 1, 256, device=dev())
    for i, f in enumerate([0.0, 1.0, 1e-37, 3e-39, 2e38, 3e30]):
        x[i] = (ramp * f).to(x.dtype)
    codes, scales = abi.quantize_int8(x)
    q, s = P.quotients(np64(x))
    assert np.all(np.abs(codes.cpu().numpy() - q) <= 0.5 + 127 * 2 * P.U32)
    assert (codes[0] == 0).all() and scales[0] == 0
    # (scales below fp32's normal range are multiples of 2^-149)
    assert np.all(np.abs(scales.cpu().double().numpy() - s) <= P.U32 * s + 2.0 ** -150)


@pytest.mark.parametrize("dt,cols", [("f16", 1024), ("bf16", 1408), ("f32", 896), ("f16", 2048)])
def test_quantize_many_short_rows(dt, cols):
    """16384 rows and more of up to 256 16-byte granules take a wavefront each."""
    g = torch.Generator(device=dev())
    g.manual_seed(cols)
    x = (torch.randn(16385, cols, generator=g, device=dev()) * 3).to(DT[dt][0])
    codes, scales = abi.quantize_int8(x)
    top = x.double().abs().amax(1, keepdim=True)
    q = 127 * x.double() / top
    assert torch.all((codes.double() - q).abs() <= 0.5 + (127 * 2 * P.U32 if dt == "f32" else 0))
    assert torch.all((scales.double() - top[:, 0] / 127).abs() <= P.U32 * top[:, 0] / 127)


def test_quantize_past_32_bit_offsets():
    rows, cols = 270000, 8192                      # 2.2e9 values
    x = torch.empty(rows, cols, device=dev(), dtype=torch.bfloat16)
    x.fill_(1.0)
    x[-1] = torch.linspace(-3, 3, cols, device=dev()).to(torch.bfloat16)
    codes, scales = abi.quantize_int8(x)
    assert np.array_equal(codes[-1].cpu().numpy(), P.codes(np64(x[-1:]))[0][0])
    assert (codes[-2] == 127).all() and (codes[0] == 127).all() and abs(float(scales[-1]) - 3 / 127) < 1e-8


# ---- the product ---------------------------------------------------------------------------------------------

def product(a, sa, offsets, w, sw, dt, fill=-7.0):
    rows, K = a.shape
    E, N, _ = w.shape
    y = torch.full((rows, N), fill, device=dev(), dtype=DT[dt][0])
    ws = torch.empty(abi.moe_workspace_size_gemm_int8(rows, N, K, E), dtype=torch.uint8, device=dev())
    abi.moe_grouped_gemm_int8(rows, N, K, E, a, sa, offsets, w, sw, DT[dt][1], y, ws)
    torch.cuda.synchronize()
    return y, abi.moe_read_device_flags(ws)


GEMM_CASES = [
    # rows per expert, N, K, rows behind the last group
    ([1], 16, 128, 0), ([0], 64, 256, 3), ([7], 304, 384, 0), ([17], 4096, 2048, 0), ([33], 272, 14336, 2),
    ([1, 0, 5, 0], 144, 512, 0), ([64] * 3, 256, 256, 0), ([200, 0, 31, 1], 528, 640, 9), ([130], 1040, 896, 5),
    ([256, 257, 3, 64, 65, 33], 256, 384, 0), ([700], 512, 1024, 0), ([0, 0, 0], 128, 128, 4),
    ([3] * 40 + [0] * 20, 96, 256, 1), ([2100], 160, 256, 0),
    # column tiles x big row tiles just over a few rounds of the compute units: the last row tiles become small ones,
    # one of them of a short row tile
    ([256 * 32, 200], 2048, 128, 3), ([150, 256 * 20 + 130, 256 * 12 + 80], 2048, 128, 0), ([256 * 17], 4096, 128, 0),
]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("counts,N,K,extra", GEMM_CASES)
def test_grouped_gemm(counts, N, K, extra, dt):
    say(f"int8 gemm {counts[:6]} N={N} K={K} +{extra} {dt}")
    r = np.random.default_rng(N + K)
    off = offsets_of(counts)
    rows, E, live = int(off[-1]) + extra, len(counts), int(off[-1])
    a = np.clip(np.rint(r.normal(size=(rows, K)) * 40), -127, 127).astype(np.int8)
    sa = np.exp(r.normal(size=rows)).astype(np.float32)
    sa[live:] = np.nan                              # rows behind the last group are not read
    w, sw = weights(r, E, N, K)
    y, flags = product(on(a), on(sa), on(off), on(w), on(sw), dt)
    e = P.expert_of_row(off, rows)
    f = np.where(np.isnan(sa), 0, sa).astype(np.float64)[:, None] * sw.astype(np.float64)[e]
    want = P.grouped(a, w, off) * f
    # int32 to fp32, the scales' product, their product: 3 roundings of each part; up to 8 parts are added
    slack = 11 * P.U32 * P.grouped(np.abs(a.astype(np.int16)), np.abs(w.astype(np.int16)), off) * f
    tol = slack + (0 if dt == "f32" else P.HALF_STEP[dt] * (np.abs(want) + slack) + 2.0 ** -25)
    got = np64(y)
    assert np.all(np.abs(got - want)[:live] <= tol[:live])
    assert (got[live:] == -7.0).all() and flags == 0


def test_all_rows_without_offsets():
    r = np.random.default_rng(1)
    for rows in (1, 31, 70, 200, 2100):
        a = r.integers(-127, 128, (rows, 256)).astype(np.int8)
        w, sw = weights(r, 1, 80, 256)
        sa = np.ones(rows, np.float32)
        one, _ = product(on(a), on(sa), None, on(w), on(sw), "f32")
        two, _ = product(on(a), on(sa), on(np.array([0, rows], np.int32)), on(w), on(sw), "f32")
        want = (a.astype(np.float64) @ w[0].astype(np.float64).T) * sw.astype(np.float64)
        slack = 3 * P.U32 * (np.abs(a.astype(np.int16)).astype(np.float64) @ np.abs(w[0].astype(np.int16)).T) * sw
        assert np.all(np.abs(np64(one) - want) <= slack * 4) and np.all(np.abs(np64(two) - want) <= slack * 4)


def test_largest_sums_stay_exact():
    """All codes 127 over the longest K: the int32 sum is 127 * 127 * 131072."""
    K = 131072
    a = torch.full((3, K), 127, dtype=torch.int8, device=dev())
    w = torch.full((1, 32, K), 127, dtype=torch.int8, device=dev())
    w[0, 1] = -127
    one = torch.ones(3, device=dev())
    y, _ = product(a, one, None, w, torch.ones(1, 32, device=dev()), "f32")
    want = 127.0 * 127.0 * K
    assert torch.all((y[:, 0] - want).abs() <= want * 8 * P.U32) and torch.all((y[:, 1] + want).abs() <= want * 8 * P.U32)


def test_fp16_range_is_flagged():
    a = torch.full((2, 128), 127, dtype=torch.int8, device=dev())
    w = torch.full((1, 16, 128), 127, dtype=torch.int8, device=dev())
    y, flags = product(a, torch.tensor([1.0, 1e-6], device=dev()), None, w, torch.ones(1, 16, device=dev()), "f16")
    assert flags == abi.MOE_FLAG_Y_RANGE and torch.isinf(y[0]).all() and torch.isfinite(y[1]).all()


def test_weights_past_32_bit_offsets():
    E, N, K = 40, 8192, 8192                       # 2.7e9 codes
    w = torch.ones(E, N, K, dtype=torch.int8, device=dev())
    w[-1, -1] = 2
    a = torch.ones(3, K, dtype=torch.int8, device=dev())
    off = torch.zeros(E + 1, dtype=torch.int32, device=dev())
    off[-1] = 3
    y, _ = product(a, torch.ones(3, device=dev()), off, w, torch.ones(E, N, device=dev()), "f32")
    assert (y[:, :-1] == K).all() and (y[:, -1] == 2 * K).all()


# ---- the FFN -------------------------------------------------------------------------------------------------

FFN_CASES = [
    # H, I, rows per expert, top_k (rows a multiple of it), rows left over
    (128, 128, [1], 1, 0), (256, 384, [0, 3, 0, 2], 1, 2), (512, 256, [40, 0, 7, 33], 2, 0),
    (384, 640, [300, 1, 66, 130, 0, 3], 4, 4), (256, 128, [257, 64, 65], 2, 0), (128, 256, [2, 1] * 8, 8, 0),
    (1024, 2048, [2, 0, 0, 0, 0, 0, 0, 0], 2, 0), (256, 512, [0, 0], 1, 1), (128, 3200, [90, 70], 1, 0),
]


def run_ffn(x, xs, off, w, H, I, E, tokens, k, dt, fill=-7.0):
    s = abi.make_shape(num_tokens=tokens, hidden=H, num_experts=E, intermediate=I, top_k=k)
    y = torch.full((tokens * k, H), fill, device=dev(), dtype=DT[dt][0])
    ws = torch.empty(abi.moe_workspace_size_int8(s), dtype=torch.uint8, device=dev())
    abi.moe_grouped_ffn_int8(s, x, xs, off, w, DT[dt][1], y, ws)
    torch.cuda.synchronize()
    return y, abi.moe_read_device_flags(ws)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("H,I,counts,k,extra", FFN_CASES)
def test_grouped_ffn(H, I, counts, k, extra, dt):
    say(f"int8 ffn H={H} I={I} {counts} k={k} +{extra} {dt}")
    r = np.random.default_rng(H + I)
    E = max(len(counts), k)
    counts = counts + [0] * (E - len(counts))
    off = offsets_of(counts)
    live, rows = int(off[-1]), int(off[-1]) + extra
    assert rows % k == 0
    x = np.clip(np.rint(r.normal(size=(rows, H)) * 32), -127, 127).astype(np.int8)
    xs = ((1 + r.random(rows)) / 32).astype(np.float32)
    xs[live:] = np.nan
    g, u, d = weights(r, E, I, H), weights(r, E, I, H), weights(r, E, H, I)
    w = abi.int8_ffn(*((on(c), on(s)) for c, s in (g, u, d)))
    y, flags = run_ffn(on(x), on(xs), on(off), w, H, I, E, rows // k, k, dt)
    want, slack = P.ffn_int8(x, np.where(np.isnan(xs), 0, xs).astype(np.float64), off, g, u, d)
    tol = slack + (0 if dt == "f32" else P.HALF_STEP[dt] * (np.abs(want) + slack) + 2.0 ** -25)
    got = np64(y)
    say(f"  largest error {np.abs(got - want)[:live].max() if live else 0:.2e}, "
        f"largest share of its bound {(np.abs(got - want) / np.maximum(tol, 1e-300))[:live].max() if live else 0:.2f}")
    assert np.all(np.abs(got - want)[:live] <= tol[:live])
    assert (got[live:] == -7.0).all() and flags == 0


def test_ffn_range_of_h():
    """h outside fp16 is clamped and flagged, the rows without such a value are not touched by it."""
    H = I = 128
    x = torch.full((2, H), 127, dtype=torch.int8, device=dev())
    w1 = torch.full((1, I, H), 127, dtype=torch.int8, device=dev())
    s = torch.ones(1, I, device=dev())
    w = abi.int8_ffn((w1, s), (w1, s), (w1, s * 1e-6))
    off = torch.tensor([0, 2], dtype=torch.int32, device=dev())
    y, flags = run_ffn(x, torch.tensor([1.0, 1e-6], device=dev()), off, w, H, I, 1, 2, 1, "f32")
    assert flags == abi.MOE_FLAG_H_RANGE
    want = 65504.0 * 127 * I * 1e-6                # every h is 65504: code 127, scale 65504 / 127
    assert torch.all((y[0] - want).abs() <= 4 * P.U32 * want) and torch.isfinite(y).all()


def test_ffn_of_large_gates():
    """Gates far on either side of 0: silu goes to 0 or to the gate, without a NaN."""
    H = I = 128
    x = torch.full((1, H), 127, dtype=torch.int8, device=dev())
    w1 = torch.ones(1, I, H, dtype=torch.int8, device=dev())
    w1[0, ::2] = -1                                # gate -127 * 128 * s and 127 * 128 * s
    up = torch.ones(1, I, H, dtype=torch.int8, device=dev())
    off = torch.tensor([0, 1], dtype=torch.int32, device=dev())
    for s in (1.0, 1e-2, 6e-3, 1e-4):
        w = abi.int8_ffn((w1, torch.full((1, I), s, device=dev())), (up, torch.full((1, I), 1e-4, device=dev())),
                         (w1, torch.full((1, H), 1e-3, device=dev())))
        y, _ = run_ffn(x, torch.ones(1, device=dev()), off, w, H, I, 1, 1, 1, "f32")
        want, slack = P.ffn_int8(np64(x), np.ones(1), np.array([0, 1]), *((t.cpu().numpy(), sc.cpu().numpy())
                                 for t, sc in (w["gate"], w["up"], w["down"])))
        assert np.all(np.abs(np64(y) - want) <= slack), s


def test_helpers_on_a_given_stream_own_their_memory():
    """Memory freed while the current stream still has work on it is not handed to a call on another stream."""
    side = torch.cuda.Stream()
    x = torch.randn(2048, 4096, device=dev()).to(torch.bfloat16)
    busy = torch.empty(1 << 30, dtype=torch.uint8, device=dev())
    makers = (lambda st: abi.quantize_int8(x, stream=st), lambda st: abi.quantize_mxfp8(x, stream=st),
              lambda st: (abi.to_f16_weights(x, stream=st),))
    for make in makers:
        want = [t.clone() for t in make(None)]
        torch.cuda.synchronize()
        for _ in range(40):                            # some milliseconds of work before the last use
            busy.fill_(1)
        late = [torch.empty_like(t) for t in want]
        for t in late:
            t.zero_()
        del late, t
        got = make(side.cuda_stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
        got = make(torch.cuda.default_stream().cuda_stream)   # (0)
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
