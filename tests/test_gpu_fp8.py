"""The operators on 8-bit floating-point blocks of 128 against plain 64-bit forms (plain_fp8.py has the bounds)."""

import numpy as np
import pytest
import torch

from expert_serving_amd import abi

import plain_fp8 as P
from gpu_util import dev, say

pytestmark = pytest.mark.gpu

DT = {"f32": (torch.float32, abi.MOE_F32), "f16": (torch.float16, abi.MOE_F16), "bf16": (torch.bfloat16, abi.MOE_BF16)}
FP8 = torch.float8_e4m3fn


def np64(t):
    return t.detach().float().cpu().double().numpy() if t.dtype == FP8 else t.detach().cpu().double().numpy()


def offsets_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def on(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(dev())
    return t if dtype is None else t.to(dtype)


def codes8(a):
    return on(a.astype(np.float32)).to(FP8)


# ---- quantisation --------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 128), (3, 512), (17, 640), (5, 2048), (2, 7168), (300, 384), (1, 131072)])
def test_quantize(dt, rows, cols):
    say(f"quantize fp8 {dt} {rows} x {cols}")
    r = np.random.default_rng(cols + rows)
    x = on(r.normal(size=(rows, cols)) * np.exp(2 * r.normal(size=(rows, 1))), DT[dt][0])
    x[0, 7], x[0, 9], x[0, 11] = 7.0, 7.0 * 17 / 448, -7.0 * 19 / 448   # (in fp16 and bf16: near) ties of codes
    x[-1, -128:] = 0
    x[-1, -1] = 0.25
    codes, scales = abi.quantize_fp8(x)
    q, s = P.quotients(np64(x))
    c = np64(codes)
    if dt == "f32":   # 448 v and the quotient may be off in their last bit: either neighbour where that decides
        near = np.minimum(np.abs(c - P.e4m3(q * (1 - 4 * P.U32))), np.abs(c - P.e4m3(np.clip(q * (1 + 4 * P.U32), -448, 448))))
        assert np.all(near == 0)
    else:             # 448 v is exact, and a quotient that is no tie is further from one than fp32 rounds
        assert np.array_equal(c, P.e4m3(q))
    assert c[-1, -1] == 448 and (c[-1, -128:-1] == 0).all()
    assert np.all(np.abs(np64(scales) - s) <= P.U32 * s)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_quantize_zero_tiny_and_huge_blocks(dt):
    x = torch.zeros(6, 256, device=dev(), dtype=DT[dt][0])
    ramp = torch.linspace(-1, 1, 256, device=dev())
    for i, f in enumerate([0.0, 1.0, 1e-37, 3e-39, 2e38, 3e30]):
        x[i] = (ramp * f).to(x.dtype)
    codes, scales = abi.quantize_fp8(x)
    q, s = P.quotients(np64(x))
    c = np64(codes)
    assert np.all((c == P.e4m3(q * (1 - 4 * P.U32))) | (c == P.e4m3(np.clip(q * (1 + 4 * P.U32), -448, 448))))
    assert (c[0] == 0).all() and (scales[0] == 0).all()
    # (scales below fp32's normal range are multiples of 2^-149)
    assert np.all(np.abs(np64(scales) - s) <= P.U32 * s + 2.0 ** -150)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("E,N,K", [(1, 128, 128), (3, 144, 256), (2, 16, 384), (1, 400, 640)])
def test_quantize_weights(dt, E, N, K):
    r = np.random.default_rng(N + K)
    w = on(r.normal(size=(E, N, K)), DT[dt][0])
    codes, scales = abi.quantize_fp8_weights(w)
    v, c, s = np64(w), np64(codes), np64(scales)
    assert s.shape == (E, -(-N // 128), K // 128)
    for e in range(E):
        for n in range(0, N, 128):
            for k in range(0, K, 128):
                part = v[e, n:n + 128, k:k + 128]
                top = np.abs(part).max()
                assert abs(s[e, n // 128, k // 128] - top / 448) <= P.U32 * top / 448
                got, q = c[e, n:n + 128, k:k + 128], 448 * part / top
                assert np.all((got == P.e4m3(q * (1 - 4 * P.U32))) | (got == P.e4m3(np.clip(q * (1 + 4 * P.U32), -448, 448))))


def test_quantize_past_32_bit_offsets():
    rows, cols = 270000, 8192                      # 2.2e9 values
    x = torch.empty(rows, cols, device=dev(), dtype=torch.bfloat16)
    x.fill_(1.0)
    x[-1] = torch.linspace(-3, 3, cols, device=dev()).to(torch.bfloat16)
    codes, scales = abi.quantize_fp8(x)
    q, s = P.quotients(np64(x[-1:]))
    assert np.array_equal(np64(codes[-1:]), P.e4m3(q)) and np.all(np.abs(np64(scales[-1:]) - s) <= P.U32 * s)
    assert (codes[-2].float() == 448).all() and (codes[0].float() == 448).all()


# ---- the product ---------------------------------------------------------------------------------------------

def product(a, sa, offsets, w, sw, dt, fill=-7.0):
    rows, K = a.shape
    E, N, _ = w.shape
    y = torch.full((rows, N), fill, device=dev(), dtype=DT[dt][0])
    ws = torch.empty(abi.moe_workspace_size_gemm_fp8(rows, N, K, E), dtype=torch.uint8, device=dev())
    ws.fill_(0xA5)
    abi.moe_grouped_gemm_fp8(rows, N, K, E, a, sa, offsets, w, sw, DT[dt][1], y, ws)
    torch.cuda.synchronize()
    return y, abi.moe_read_device_flags(ws)


GEMM_CASES = [
    # rows per expert, N, K, rows behind the last group
    ([1], 16, 128, 0), ([0], 64, 256, 3), ([7], 304, 384, 0), ([17], 4096, 2048, 0), ([33], 272, 14336, 2),
    ([1, 0, 5, 0], 144, 512, 0), ([64] * 3, 256, 256, 0), ([200, 0, 31, 1], 528, 640, 9), ([130], 1040, 896, 5),
    ([256, 257, 3, 64, 65, 33], 256, 384, 0), ([700], 512, 1024, 0), ([0, 0, 0], 128, 128, 4),
    ([3] * 40 + [0] * 20, 96, 256, 1), ([2100], 160, 256, 0), ([150, 130, 193, 129, 255], 400, 1152, 0),
    # column tiles x big row tiles just over a few rounds of the compute units: the last row tiles become small ones,
    # one of them of a short row tile
    ([256 * 32, 200], 2048, 128, 3), ([256 * 17], 4096, 128, 0),
]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("counts,N,K,extra", GEMM_CASES)
def test_grouped_gemm(counts, N, K, extra, dt):
    say(f"fp8 gemm {counts[:6]} N={N} K={K} +{extra} {dt}")
    r = np.random.default_rng(N + K)
    off = offsets_of(counts)
    rows, E, live = int(off[-1]) + extra, len(counts), int(off[-1])
    a, sa = P.exact_codes(r, rows, K), P.scales_of(r, rows, K // 128)
    sa[live:] = np.nan                              # rows behind the last group are not read
    w, sw = P.exact_codes(r, E, N, K), P.scales_of(r, E, -(-N // 128), K // 128) / 16
    y, flags = product(codes8(a), on(sa), on(off), codes8(w), on(sw), dt)
    want, bound = P.product(a[:live], sa[:live], w, sw, off, True)
    tol = P.rounded(want, bound, dt)
    got = np64(y)
    say(f"  largest share of the bound {(np.abs(got[:live] - want) / tol).max() if live else 0:.2f}")
    assert np.all(np.abs(got[:live] - want) <= tol)
    assert (got[live:] == -7.0).all() and flags == 0


@pytest.mark.parametrize("counts,N,K", [([5, 40], 272, 1024), ([300, 77], 256, 512), ([16], 64, 4096)])
def test_products_of_all_codes(counts, N, K):
    """Codes over the whole range of E4M3, subnormals among them: the matrix units' alignment is in the bound, and
    the error over all outputs stays where it was measured to be (1.4e-5 of the norm for normal data)."""
    r = np.random.default_rng(K)
    off = offsets_of(counts)
    rows, E = int(off[-1]), len(counts)
    a = P.e4m3(np.clip(r.normal(size=(rows, K)) * np.exp(1.5 * r.normal(size=(rows, K))) * 8, -448, 448))
    w = P.e4m3(np.clip(r.normal(size=(E, N, K)) * 100, -448, 448))
    sa, sw = P.scales_of(r, rows, K // 128), P.scales_of(r, E, -(-N // 128), K // 128) / 4096
    y, _ = product(codes8(a), on(sa), on(off), codes8(w), on(sw), "f16")
    want, bound = P.product(a, sa, w, sw, off, False)
    got = np64(y)
    assert np.all(np.abs(got - want) <= P.rounded(want, bound, "f16"))
    assert np.linalg.norm(got - want) <= (2.0 ** -11 + 1e-4) * np.linalg.norm(want)


def test_all_rows_without_offsets():
    r = np.random.default_rng(1)
    w, sw = P.exact_codes(r, 1, 80, 256), P.scales_of(r, 1, 1, 2)
    for rows in (1, 31, 70, 200, 2100):
        a, sa = P.exact_codes(r, rows, 256), P.scales_of(r, rows, 2)
        one, _ = product(codes8(a), on(sa), None, codes8(w), on(sw), "bf16")
        two, _ = product(codes8(a), on(sa), on(np.array([0, rows], np.int32)), codes8(w), on(sw), "bf16")
        want, bound = P.product(a, sa, w, sw, [0, rows], True)
        tol = P.rounded(want, bound, "bf16")
        assert np.all(np.abs(np64(one) - want) <= tol) and np.all(np.abs(np64(two) - want) <= tol)


@pytest.mark.parametrize("rows", [3, 40, 300])
def test_scales_far_apart(rows):
    """Scales of neighbouring blocks up to 2^200 apart, subnormal and zero ones among them."""
    r = np.random.default_rng(rows)
    K, N = 1280, 160
    a, w = P.exact_codes(r, rows, K), P.exact_codes(r, 1, N, K)
    sa = np.ldexp(1 + r.random((rows, K // 128)), r.integers(-120, -20, (rows, K // 128))).astype(np.float32)
    sa[:, 3] = 0.0
    sa[:, 5] = np.ldexp(r.integers(1, 1000, rows).astype(np.float64), -149).astype(np.float32)
    sa[0] = np.ldexp(1.5, np.linspace(-126, -40, K // 128).astype(int)).astype(np.float32)
    sa[1] = sa[0, ::-1]
    sw = np.ldexp(1 + r.random((1, 2, K // 128)), r.integers(0, 20, (1, 2, K // 128))).astype(np.float32)
    sw[0, 1] = np.ldexp(1.25, np.linspace(60, -20, K // 128).astype(int)).astype(np.float32)
    y, _ = product(codes8(a), on(sa), None, codes8(w), on(sw), "bf16")
    want, bound = P.product(a, sa, w, sw, [0, rows], True)
    # a scale below 2^-126 may count as any up to that: 128 products of up to 9
    low = 128 * 9 * 2.0 ** -126 * sw[0, np.arange(N) // 128].astype(np.float64)[:, [3, 5]].sum(1)
    assert np.all(np.abs(np64(y) - want) <= P.rounded(want, bound + low, "bf16"))


def test_fp16_range_is_flagged():
    a = torch.full((2, 128), 64.0, device=dev()).to(FP8)
    w = torch.full((1, 16, 128), 64.0, device=dev()).to(FP8)
    y, flags = product(a, torch.tensor([[1.0], [1e-6]], device=dev()), None, w, torch.ones(1, 1, 1, device=dev()), "f16")
    assert flags == abi.MOE_FLAG_Y_RANGE and torch.isinf(y[0]).all() and torch.isfinite(y[1]).all()
    y, flags = product(a, torch.tensor([[1.0], [1e-6]], device=dev()), None, w, torch.ones(1, 1, 1, device=dev()), "bf16")
    assert flags == 0 and (y[0] == 64 * 64 * 128).all()


def test_weights_past_32_bit_offsets():
    E, N, K = 40, 8192, 8192                       # 2.7e9 codes
    w = torch.ones(E, N, K, dtype=torch.bfloat16, device=dev()).to(FP8)
    w[-1, -1] = torch.full((K,), 2.0, device=dev()).to(FP8)
    a = torch.ones(3, K, device=dev()).to(FP8)
    off = torch.zeros(E + 1, dtype=torch.int32, device=dev())
    off[-1] = 3
    y, _ = product(a, torch.ones(3, K // 128, device=dev()), off, w, torch.ones(E, N // 128, K // 128, device=dev()), "bf16")
    assert (y[:, :-1] == K).all() and (y[:, -1] == 2 * K).all()


def test_rows_past_32_bit_offsets():
    rows, N, K = 300000, 64, 8192                  # 2.5e9 codes
    a = torch.ones(rows, K, dtype=torch.bfloat16, device=dev()).to(FP8)
    a[-1] = torch.full((K,), 0.5, device=dev()).to(FP8)
    w = torch.ones(1, N, K, device=dev()).to(FP8)
    y, _ = product(a, torch.ones(rows, K // 128, device=dev()), None, w, torch.ones(1, 1, K // 128, device=dev()), "bf16")
    assert (y[:-1] == K).all() and (y[-1] == K / 2).all()


def test_gradient_of_the_rows_is_the_product_with_transposed_weights():
    r = np.random.default_rng(3)
    E, N, K, off = 3, 256, 384, offsets_of([20, 0, 70])
    w = on(r.normal(size=(E, N, K)), torch.bfloat16)
    codes, scales = abi.quantize_fp8_weights(w)
    dy = on(r.normal(size=(90, N)), torch.bfloat16)
    dc, ds = abi.quantize_fp8(dy)
    turned = codes.view(torch.uint8).transpose(1, 2).contiguous().view(FP8)
    dx, _ = product(dc, ds, on(off), turned, scales.transpose(1, 2).contiguous(), "bf16")
    full = np64(codes) * np64(scales)[:, np.arange(N) // 128][:, :, np.arange(K) // 128]
    g = np64(dc) * np64(ds)[:, np.arange(N) // 128]
    want = np.concatenate([g[:20] @ full[0], g[20:] @ full[2]])
    _, bound = P.product(np64(dc), np64(ds), np64(turned), np64(scales.transpose(1, 2)), off, False)
    assert np.all(np.abs(np64(dx) - want) <= P.rounded(want, bound, "bf16"))


# ---- the FFN -------------------------------------------------------------------------------------------------

FFN_CASES = [
    # H, I, rows per expert, top_k (rows a multiple of it), rows left over
    (128, 128, [1], 1, 0), (256, 384, [0, 3, 0, 2], 1, 2), (512, 256, [40, 0, 7, 33], 2, 0),
    (384, 640, [300, 1, 66, 130, 0, 3], 4, 4), (256, 128, [257, 64, 65], 2, 0), (128, 256, [2, 1] * 8, 8, 0),
    (1024, 2048, [2, 0, 0, 0, 0, 0, 0, 0], 2, 0), (256, 512, [0, 0], 1, 1), (128, 3200, [90, 70], 1, 0),
    (640, 896, [193, 255, 129], 1, 3),
]


def draw_ffn(r, H, I, E):
    g = P.exact_codes(r, E, I, H), P.scales_of(r, E, I // 128, H // 128) / (4 * H ** 0.5)
    u = P.exact_codes(r, E, I, H), P.scales_of(r, E, I // 128, H // 128) / (4 * H ** 0.5)
    d = P.exact_codes(r, E, H, I), P.scales_of(r, E, H // 128, I // 128) / (4 * I ** 0.5)
    return g, u, d


def run_ffn(x, xs, off, w, H, I, E, tokens, k, dt, fill=-7.0):
    s = abi.make_shape(num_tokens=tokens, hidden=H, num_experts=E, intermediate=I, top_k=k)
    y = torch.full((tokens * k, H), fill, device=dev(), dtype=DT[dt][0])
    ws = torch.empty(abi.moe_workspace_size_fp8(s), dtype=torch.uint8, device=dev())
    ws.fill_(0xA5)
    abi.moe_grouped_ffn_fp8(s, x, xs, off, w, DT[dt][1], y, ws)
    torch.cuda.synchronize()
    return y, abi.moe_read_device_flags(ws)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("H,I,counts,k,extra", FFN_CASES)
def test_grouped_ffn(H, I, counts, k, extra, dt):
    say(f"fp8 ffn H={H} I={I} {counts} k={k} +{extra} {dt}")
    r = np.random.default_rng(H + I)
    E = max(len(counts), k)
    counts = counts + [0] * (E - len(counts))
    off = offsets_of(counts)
    live, rows = int(off[-1]), int(off[-1]) + extra
    assert rows % k == 0
    x, xs = P.exact_codes(r, rows, H), P.scales_of(r, rows, H // 128)
    xs[live:] = np.nan
    g, u, d = draw_ffn(r, H, I, E)
    w = abi.fp8_ffn(*((codes8(c), on(s)) for c, s in (g, u, d)))
    y, flags = run_ffn(codes8(x), on(xs), on(off), w, H, I, E, rows // k, k, dt)
    want, bound = P.ffn(x[:live], xs[:live], g, u, d, off, True)
    tol = P.rounded(want, bound, dt)
    got = np64(y)
    say(f"  largest error {np.abs(got[:live] - want).max() if live else 0:.2e} of {np.abs(want).max() if live else 0:.2e}, "
        f"largest share of its bound {(np.abs(got[:live] - want) / tol).max() if live else 0:.2f}")
    assert np.all(np.abs(got[:live] - want) <= tol)
    assert (got[live:] == -7.0).all() and flags == 0


def test_ffn_of_large_gates():
    """Gates far on either side of 0: silu goes to 0 or to the gate, without a NaN."""
    H = I = 128
    x = codes8(np.full((1, H), 1.0))
    gate = np.ones((1, I, H))
    gate[0, ::2] = -1
    off = np.array([0, 1])
    for s in (1.0, 1e-2, 6e-3, 1e-4, 1e4):
        parts = [(gate, np.full((1, 1, 1), s, np.float32)), (np.ones((1, I, H)), np.full((1, 1, 1), 1e-4, np.float32)),
                 (gate, np.full((1, 1, 1), 1e-3, np.float32))]
        w = abi.fp8_ffn(*((codes8(c), on(v)) for c, v in parts))
        y, flags = run_ffn(x, torch.ones(1, 1, device=dev()), on(off.astype(np.int32)), w, H, I, 1, 1, 1, "bf16")
        want, bound = P.ffn(np.ones((1, H)), np.ones((1, 1)), *parts, off, True)
        assert flags == 0 and np.all(np.abs(np64(y) - want) <= P.rounded(want, bound, "bf16")), s
