"""The operators on 8-bit floating-point blocks as they are used: one after the other around a routed batch, captured
and replayed, on streams of their own, at sizes that fill the compute units several times, and on values that are not
finite."""

import numpy as np
import pytest
import torch

from expert_serving_amd import abi

import plain_fp8 as P
from gpu_util import dev, say
from test_gpu_fp8 import DT, FP8, codes8, draw_ffn, np64, offsets_of, on, product, run_ffn

pytestmark = pytest.mark.gpu


BARE = abi.make_block(residual_scale=0.0, stream_dtype=abi.MOE_F32)   # the combination alone, in fp32


# ---- a batch routed, sorted, run, brought back, and its gradients ----------------------------------------------

def routed(T, H, I, E, k, seed):
    """A batch with its routing: the permutation that moe_dispatch leaves."""
    r = np.random.default_rng(seed)
    s = abi.make_shape(num_tokens=T, hidden=H, num_experts=E, intermediate=I, top_k=k)
    x = on(r.normal(size=(T, H)), torch.bfloat16)
    router = on(r.normal(size=(E, H)) / H ** 0.5, torch.bfloat16)
    i32 = lambda *sh: torch.full(sh, -1, dtype=torch.int32, device=dev())  # noqa: E731
    ids, gates, cnt, off, ros, token_of, dropped = i32(T, k), torch.zeros(T, k, device=dev()), i32(E), i32(E + 1), \
        i32(T, k), i32(T * k), i32(1)
    perm = torch.zeros(T * k, H, dtype=torch.bfloat16, device=dev())
    ws = torch.empty(abi.moe_workspace_size(s), dtype=torch.uint8, device=dev())
    abi.moe_route_topk(s, x, router, None, None, None, None, ids, gates, ws)
    abi.moe_dispatch(s, x, ids, cnt, off, ros, token_of, dropped, perm, ws)
    return r, s, x, gates, off, ros, perm


SIZES = [(1, 256, 128, 8, 2), (5, 384, 256, 4, 3), (70, 256, 384, 8, 2), (600, 512, 256, 6, 4)]


@pytest.mark.parametrize("T,H,I,E,k", SIZES)
def test_layer_of_single_calls(T, H, I, E, k):
    """Router, sort as codes, FFN, combination: against the 64-bit forms of the same codes."""
    say(f"fp8 layer {T} x {H}, {E} experts of {I}, top {k}")
    r, s, x, gates, off, ros, perm = routed(T, H, I, E, k, T)
    n = T * k
    codes = torch.empty(n, H, dtype=torch.uint8, device=dev()).view(FP8)
    scales = torch.empty(n, H // 128, device=dev())
    abi.moe_dispatch_rows_fp8(s, abi.MOE_BF16, x, ros, n, codes, scales)
    again, ascales = abi.quantize_fp8(perm)         # the rows that moe_dispatch copied
    assert torch.equal(codes.view(torch.uint8), again.view(torch.uint8)) and torch.equal(scales, ascales)
    copied = torch.zeros_like(perm)
    abi.moe_dispatch_rows(s, abi.MOE_BF16, x, ros, None, n, copied)
    assert torch.equal(copied, perm)
    parts = [abi.quantize_fp8_weights(on(r.normal(size=sh) / sh[2] ** 0.5, torch.bfloat16))
             for sh in ((E, I, H), (E, I, H), (E, H, I))]
    y, flags = run_ffn(codes, scales, off, abi.fp8_ffn(*parts), H, I, E, T, k, "bf16")
    o = off.cpu().numpy()
    want, bound = P.ffn(np64(codes), np64(scales), *((np64(c), np64(v)) for c, v in parts), o, False)
    tol = P.rounded(want, bound, "bf16")
    assert flags == 0 and o[-1] == n and np.all(np.abs(np64(y) - want) <= tol)
    out = torch.zeros(T, H, device=dev())
    abi.moe_combine_norm(s, BARE, abi.MOE_BF16, y, ros, gates, None, None, out)
    g, m, ro = np64(gates), np64(y), ros.cpu().numpy()
    full = (g[:, :, None] * m[ro]).sum(1)
    size = (np.abs(g)[:, :, None] * np.abs(m[ro])).sum(1)
    assert np.all(np.abs(np64(out) - full) <= (k + 1) * P.U32 * size)


@pytest.mark.parametrize("T,H,I,E,k", SIZES)
def test_gradients_of_single_calls(T, H, I, E, k):
    """Combination backwards, the down product's gradient as a product with the transposed codes, and the sort
    backwards: against the 64-bit chain of the same codes."""
    r, s, x, gates, off, ros, perm = routed(T, H, I, E, k, T + 1)
    n, o, ro = T * k, off.cpu().numpy(), ros.cpu().numpy()
    y, d_out = on(r.normal(size=(n, H)), torch.bfloat16), on(r.normal(size=(T, H)), torch.float32)
    d_y, d_gates = torch.zeros(n, H, device=dev(), dtype=torch.bfloat16), torch.zeros(T, k, device=dev())
    abi.moe_combine_backward(s, abi.MOE_F32, d_out, abi.MOE_BF16, y, ros, gates, n, d_y, d_gates)
    full = np.zeros((n, H))
    full[ro.reshape(-1)] = (np64(gates)[:, :, None] * np64(d_out)[:, None]).reshape(n, H)
    assert np.all(np.abs(np64(d_y) - full) <= P.rounded(full, P.U32 * np.abs(full), "bf16"))
    dots = (np64(y)[ro] * np64(d_out)[:, None]).sum(2)
    size = np.abs(np64(y)[ro] * np64(d_out)[:, None]).sum(2)
    assert np.all(np.abs(np64(d_gates) - dots) <= (H / 16 + 16) * P.U32 * size)
    w, ws = abi.quantize_fp8_weights(on(r.normal(size=(E, H, H)) / H ** 0.5, torch.bfloat16))
    turned, tscales = w.view(torch.uint8).transpose(1, 2).contiguous().view(FP8), ws.transpose(1, 2).contiguous()
    dc, ds = abi.quantize_fp8(d_y)
    d_perm, _ = product(dc, ds, off, turned, tscales, "bf16")
    want, bound = P.product(np64(dc), np64(ds), np64(turned), np64(tscales), o, False)
    assert np.all(np.abs(np64(d_perm) - want) <= P.rounded(want, bound, "bf16"))
    d_x = torch.zeros(T, H, device=dev(), dtype=torch.bfloat16)
    abi.moe_dispatch_rows_backward(s, abi.MOE_BF16, d_perm, ros, n, None, None, d_x, None)
    rows = np64(d_perm)[ro]
    assert np.all(np.abs(np64(d_x) - rows.sum(1)) <= P.rounded(rows.sum(1), (k + 1) * P.U32 * np.abs(rows).sum(1), "bf16"))


# ---- captured, and on streams of their own -----------------------------------------------------------------------

class Chain:
    """Sort as codes, FFN, combination and its gradient with buffers of their own."""

    def __init__(self, T, H, I, E, k, seed):
        r, self.s, self.x, self.gates, self.off, self.ros, _ = routed(T, H, I, E, k, seed)
        n = self.n = T * k
        self.parts = [abi.quantize_fp8_weights(on(r.normal(size=sh) / sh[2] ** 0.5, torch.bfloat16))
                      for sh in ((E, I, H), (E, I, H), (E, H, I))]
        self.w = abi.fp8_ffn(*self.parts)
        self.codes = torch.zeros(n, H, dtype=torch.uint8, device=dev())
        self.scales = torch.zeros(n, H // 128, device=dev())
        self.y = torch.zeros(n, H, dtype=torch.bfloat16, device=dev())
        self.out, self.dx = torch.zeros(T, H, device=dev()), torch.zeros(T, H, dtype=torch.bfloat16, device=dev())
        self.dy, self.dg = torch.zeros_like(self.y), torch.zeros(T, k, device=dev())
        self.ws = torch.empty(abi.moe_workspace_size_fp8(self.s), dtype=torch.uint8, device=dev())

    def run(self, stream=None):
        s, n, b = self.s, self.n, abi.MOE_BF16
        abi.moe_dispatch_rows_fp8(s, b, self.x, self.ros, n, self.codes, self.scales, stream)
        abi.moe_grouped_ffn_fp8(s, self.codes, self.scales, self.off, self.w, b, self.y, self.ws, stream)
        abi.moe_combine_norm(s, BARE, b, self.y, self.ros, self.gates, None, None, self.out, stream)
        abi.moe_combine_backward(s, abi.MOE_F32, self.out, b, self.y, self.ros, self.gates, n, self.dy, self.dg, stream)
        abi.moe_dispatch_rows_backward(s, b, self.dy, self.ros, n, None, None, self.dx, None, stream)

    def outputs(self):
        return [t.clone() for t in (self.codes, self.scales, self.y, self.out, self.dy, self.dg, self.dx)]

    def clear(self):
        for t in (self.codes, self.scales, self.y, self.out, self.dy, self.dg, self.dx):
            t.zero_()


@pytest.mark.parametrize("T,H,I,E,k", [(1, 256, 128, 8, 2), (40, 1024, 512, 4, 2), (600, 512, 384, 6, 4), (2048, 256, 2048, 8, 2)])
def test_captured_and_replayed(T, H, I, E, k):
    """Two graphs of the same chain, each with its workspace and buffers: every replay gives the eager result bit for
    bit, with eager calls between and new inputs in the captured buffers."""
    say(f"fp8 chain in a graph {T} x {H}, {E} experts of {I}")
    chains = [Chain(T, H, I, E, k, 3), Chain(T, H, I, E, k, 4)]
    graphs = []
    for c in chains:
        c.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        graphs.append(g)
    eager = Chain(T, H, I, E, k, 5)
    for turn in range(3):
        for i, (c, g) in enumerate(zip(chains, graphs)):
            c.x.copy_(torch.roll(c.x, 1 + turn, 0) * (1 + turn))
            c.clear()
            c.run()
            want = c.outputs()
            c.clear()
            eager.run()
            g.replay()
            eager.run()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(c.outputs(), want)), (turn, i)


@pytest.mark.parametrize("T,H,I,E,k", [(3, 256, 256, 8, 2), (300, 512, 384, 4, 2), (2048, 256, 2048, 8, 2)])
def test_two_streams_at_once(T, H, I, E, k):
    chains = [Chain(T, H, I, E, k, 6), Chain(T, H, I, E, k, 7)]
    want = []
    for c in chains:
        c.run()
        torch.cuda.synchronize()
        want.append(c.outputs())
        c.clear()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in chains]
    for _ in range(5):
        for c, st in zip(chains, streams):
            c.run(st.cuda_stream)
    torch.cuda.synchronize()
    for c, w in zip(chains, want):
        assert all(torch.equal(a, b) for a, b in zip(c.outputs(), w))


# ---- many tiles ------------------------------------------------------------------------------------------------

MANY = [
    # rows per expert, N, K: more tiles than compute units, of every height, and a last round that is cut
    ([2048 + 17 * i for i in range(4)], 2560, 384), ([300, 5000, 1, 0, 700, 64, 129, 256], 1536, 256),
    ([256 * 48 + 100], 4096, 128), ([256 * 17], 4112, 1664), ([300, 2000, 1, 0, 700, 64, 129, 256], 4112, 1664),
    ([190, 130, 70, 250] * 16, 1040, 1664), ([90, 200, 40, 300] * 16, 1040, 128), ([256 * 9 + 3], 8192, 128), ([64] * 128, 768, 256), ([1] * 200 + [3000], 512, 256),
]


@pytest.mark.parametrize("counts,N,K", MANY)
def test_many_tiles(counts, N, K):
    say(f"fp8 gemm of many tiles {counts[:5]} N={N} K={K}")
    r = np.random.default_rng(N + K)
    off = offsets_of(counts)
    rows, E = int(off[-1]), len(counts)
    a, sa = P.exact_codes(r, rows, K), P.scales_of(r, rows, K // 128)
    w, sw = P.exact_codes(r, E, N, K), P.scales_of(r, E, -(-N // 128), K // 128) / 16
    y, flags = product(codes8(a), on(sa), on(off), codes8(w), on(sw), "bf16")
    want, bound = P.product(a, sa, w, sw, off, True)
    assert flags == 0 and np.all(np.abs(np64(y) - want) <= P.rounded(want, bound, "bf16"))
    again, _ = product(codes8(a), on(sa), on(off), codes8(w), on(sw), "bf16")
    assert torch.equal(y, again)                    # (whatever the blocks' order)


@pytest.mark.parametrize("counts,H,I", [([700, 0, 2500, 300, 1, 130, 900, 64], 512, 1280), ([280] * 24, 384, 640)])
def test_ffn_of_many_tiles(counts, H, I):
    r = np.random.default_rng(H)
    E, off = len(counts), offsets_of(counts)
    rows = int(off[-1])
    x, xs = P.exact_codes(r, rows, H), P.scales_of(r, rows, H // 128)
    parts = draw_ffn(r, H, I, E)
    w = abi.fp8_ffn(*((codes8(c), on(s)) for c, s in parts))
    y, flags = run_ffn(codes8(x), on(xs), on(off), w, H, I, E, rows, 1, "bf16")
    want, bound = P.ffn(x, xs, *parts, off, True)
    assert flags == 0 and np.all(np.abs(np64(y) - want) <= P.rounded(want, bound, "bf16"))
    again, _ = run_ffn(codes8(x), on(xs), on(off), w, H, I, E, rows, 1, "bf16")
    assert torch.equal(y, again)


# 128 x 128 tiles and larger ones of every height, rows and columns that end inside a tile, and K from fewer stages than
# are under way to more than share a load of scales
TILES = [([200, 0, 31, 1, 300, 129], 1040), ([700], 1168), ([256, 257, 3, 64, 65, 33, 190, 130], 4112), ([450, 260], 5136)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("K", [128, 256, 384, 1152, 2304])
@pytest.mark.parametrize("counts,N", TILES)
def test_tiles(counts, N, K, dt):
    say(f"fp8 tiles {counts} N={N} K={K} {dt}")
    r = np.random.default_rng(N + K)
    off = offsets_of(counts)
    live, E = int(off[-1]), len(counts)
    rows = live + 5
    a, sa = P.exact_codes(r, rows, K), P.scales_of(r, rows, K // 128)
    sa[live:] = np.nan
    w, sw = P.exact_codes(r, E, N, K), P.scales_of(r, E, -(-N // 128), K // 128) / 64
    y, flags = product(codes8(a), on(sa), on(off), codes8(w), on(sw), dt)
    want, bound = P.product(a[:live], sa[:live], w, sw, off, True)
    got = np64(y)
    assert flags == 0 and np.all(np.abs(got[:live] - want) <= P.rounded(want, bound, dt))
    assert (got[live:] == -7.0).all()


@pytest.mark.parametrize("rows,N,K", [(700, 1152, 1280), (2600, 2560, 1280), (4500, 2560, 1664)])
def test_tiles_of_all_codes_and_scales_far_apart(rows, N, K):
    r = np.random.default_rng(rows)
    a = P.e4m3(np.clip(r.normal(size=(rows, K)) * np.exp(1.5 * r.normal(size=(rows, K))) * 8, -448, 448))
    w = P.e4m3(np.clip(r.normal(size=(1, N, K)) * 100, -448, 448))
    sa = np.ldexp(1 + r.random((rows, K // 128)), r.integers(-120, -20, (rows, K // 128))).astype(np.float32)
    sa[:, 3] = 0.0
    sw = np.ldexp(1 + r.random((1, N // 128, K // 128)), r.integers(0, 20, (1, N // 128, K // 128))).astype(np.float32)
    y, _ = product(codes8(a), on(sa), None, codes8(w), on(sw), "bf16")
    want, bound = P.product(a, sa, w, sw, [0, rows], False)
    # the scale of 0 may count as any up to 2^-126
    low = 128 * 448.0 ** 2 * 2.0 ** -126 * sw[0, np.arange(N) // 128, 3].astype(np.float64)
    assert np.all(np.abs(np64(y) - want) <= P.rounded(want, bound + low, "bf16"))


# ---- values that are not finite --------------------------------------------------------------------------------

# rows of one expert, N (or I), K: streams of 16 and of 32 rows and of more of them, 128 x 128 tiles, large tiles
PLANS = [(3, 128, 256), (29, 128, 1280), (300, 256, 256), (700, 1152, 256), (5000, 2560, 256),
         (5000, 2560, 1664)]


@pytest.mark.parametrize("rows,N,K", PLANS)
def test_products_of_values_that_are_not_finite(rows, N, K):
    """A row whose scale is not finite or that has a NaN code is NaN, a column of such a weight block too, and no
    other value changes."""
    r = np.random.default_rng(rows)
    a, sa = codes8(P.exact_codes(r, rows, K)), on(P.scales_of(r, rows, K // 128))
    w, sw = codes8(P.exact_codes(r, 1, N, K)), on(P.scales_of(r, 1, N // 128, K // 128))
    base, flags = product(a, sa, None, w, sw, "bf16")
    assert flags == 0 and torch.isfinite(base).all()
    sa[0, 1], sa[rows - 1, 0] = float("inf"), float("nan")
    a.view(torch.uint8)[rows // 2, K - 1] = 0x7F
    y, _ = product(a, sa, None, w, sw, "bf16")
    bad = torch.zeros(rows, dtype=torch.bool, device=dev())
    bad[[0, rows // 2, rows - 1]] = True
    assert torch.isnan(y[bad]).all() and torch.equal(y[~bad], base[~bad])
    _, flags = product(a, sa, None, w, sw, "f16")
    assert flags == abi.MOE_FLAG_Y_RANGE
    if N > 128:
        sw[0, 1, 0] = float("inf")
        y, _ = product(a, sa, None, w, sw, "bf16")
        assert torch.isnan(y[:, 128:256]).all() and torch.equal(y[~bad][:, :128], base[~bad][:, :128])
        assert torch.equal(y[~bad][:, 256:], base[~bad][:, 256:])


@pytest.mark.parametrize("rows,I,H", [(3, 128, 256), (9, 4096, 128), (29, 128, 1280), (300, 256, 256), (700, 640, 256),
                                      (5000, 1280, 256), (3000, 256, 3328)])
def test_ffn_of_values_that_are_not_finite(rows, I, H):
    """An h that is not finite, of a NaN scale or of an overflow, sets the flag and makes its own row NaN alone."""
    r = np.random.default_rng(rows)
    x, xs = codes8(P.exact_codes(r, rows, H)), on(P.scales_of(r, rows, H // 128))
    parts = draw_ffn(r, H, I, 1)
    w = abi.fp8_ffn(*((codes8(c), on(s)) for c, s in parts))
    off = on(np.array([0, rows], np.int32))
    base, flags = run_ffn(x, xs, off, w, H, I, 1, rows, 1, "bf16")
    assert flags == 0 and torch.isfinite(base).all()
    for row, scale in ((0, float("nan")), (rows - 1, 1e30)):   # 1e30: gate times up passes fp32's range
        moved = xs.clone()
        moved[row] = scale
        y, flags = run_ffn(x, moved, off, w, H, I, 1, rows, 1, "bf16")
        bad = torch.zeros(rows, dtype=torch.bool, device=dev())
        bad[row] = True
        assert flags & abi.MOE_FLAG_H_RANGE and torch.isnan(y[bad]).all() and torch.equal(y[~bad], base[~bad]), (row, flags)


@pytest.mark.parametrize("rows", [3, 29, 300, 1500])
def test_ffn_of_scales_far_apart(rows):
    """Row scales of 2^100 and 2^-100 against gate and up scales that bring them back: no step in between leaves the
    range of fp32."""
    r = np.random.default_rng(rows)
    H = I = 256
    x, xs = P.exact_codes(r, rows, H), P.scales_of(r, rows, H // 128)
    g, u, d = draw_ffn(r, H, I, 1)
    lift = np.ldexp(1.0, np.array([118, -100]))     # of the two blocks of H
    xs = (xs * lift).astype(np.float32)
    g, u = ((c, (s / lift).astype(np.float32)) for c, s in (g, u))
    parts = (g, u, d)
    w = abi.fp8_ffn(*((codes8(c), on(s)) for c, s in parts))
    y, flags = run_ffn(codes8(x), on(xs), on(np.array([0, rows], np.int32)), w, H, I, 1, rows, 1, "bf16")
    want, bound = P.ffn(x, xs, *parts, [0, rows], True)
    assert flags == 0 and np.all(np.abs(np64(y) - want) <= P.rounded(want, bound, "bf16"))


@pytest.mark.parametrize("rows,H,I", [(8, 2048, 768), (2, 4096, 1280), (24, 1024, 512)])
def test_few_rows_take_the_codes_of_the_formula(rows, H, I):
    """Normal data: an h off by some 1e-5, as sums on the 8-bit units are, changes a code here and there, each half a
    step of its value, which shows in so few rows.  fp32 sums, off by less than 1e-6, change one in some 1e5 of them:
    none of these, and the error stays the rounding of y (2^-11 at most) and of the second sums (1.4e-5)."""
    r = np.random.default_rng(H)
    x, xs = abi.quantize_fp8(on(r.normal(size=(rows, H)), torch.bfloat16))
    parts = [abi.quantize_fp8_weights(on(r.normal(size=sh) / sh[2] ** 0.5, torch.bfloat16))
             for sh in ((1, I, H), (1, I, H), (1, H, I))]
    y, _ = run_ffn(x, xs, on(np.array([0, rows], np.int32)), abi.fp8_ffn(*parts), H, I, 1, rows, 1, "f16")
    want, _ = P.ffn(np64(x), np64(xs), *((np64(c), np64(v)) for c, v in parts), [0, rows], True)
    off = np.linalg.norm(np64(y) - want) / np.linalg.norm(want)
    say(f"  error {off:.2e}")
    assert off <= 2.0 ** -11 + 1e-4
