"""The int8 operators on weights too large to be streamed by every row tile: 32-row tiles through LDS, the split
products and their sums, the large tiles with a split.  The plain forms run in fp64 on the device, an expert at a
time; the bounds are those of the small cases (plain_block.py derives them)."""

import numpy as np
import pytest
import torch

from expert_serving_amd import abi

import plain_block as P
from gpu_util import dev, f32, rms, say
from test_gpu_block import Block, np64, tiny
from test_gpu_int8 import DT, offsets_of, on, product, run_ffn

pytestmark = pytest.mark.gpu


def codes(g, *shape):
    return torch.randint(-127, 128, shape, generator=g, device=dev(), dtype=torch.int8)


def scales(g, n, K):
    return (1 + 0.3 * torch.rand(n, generator=g, device=dev())) / (73 * K ** 0.5)


def gen(seed):
    g = torch.Generator(device=dev())
    g.manual_seed(seed)
    return g


def mm(a, w):
    """a @ w.T in fp64, exact for codes"""
    return a.double() @ w.double().T.contiguous()


def within(got, want, slack, dt):
    tol = slack + (0 if dt == "f32" else P.HALF_STEP[dt] * (want.abs() + slack) + 2.0 ** -25)
    err = (got.double() - want).abs()
    say(f"  largest share of its bound {float((err / tol.clamp_min(1e-300)).max()):.2f}")
    return bool((err <= tol).all())


PRODUCTS = [
    # rows per expert, N, K, rows behind the last group
    ([20, 40], 28672, 8192, 2),                         # few rows on large tiles
    ([10, 15, 0, 3], 16384, 4096, 2),                   # 32-row tiles, two parts
    ([10, 15, 0, 3], 28688, 4096, 2),                   # 32-row tiles, enough of them: no parts
    ([3] * 50 + [7] * 14, 2048, 256, 1),                # many experts of few rows
    ([1, 0, 1, 2, 0, 0, 1, 0], 4096, 14336, 0),         # fewer rows than experts: eight parts
    ([25] * 6 + [50, 0], 16384, 4096, 3),               # 16 to 64 rows an expert
    ([33, 0, 1, 30, 16, 17, 32, 31], 12304, 4224, 0),   # the same, ragged
    ([300], 4096, 14336, 1),                            # large tiles, three parts
    ([129, 64, 65, 255, 256, 1, 0, 3], 2064, 8192, 5),  # large tiles of every height, two parts
]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("counts,N,K,extra", PRODUCTS)
def test_grouped_gemm(counts, N, K, extra, dt):
    say(f"int8 gemm {counts} N={N} K={K} +{extra} {dt}")
    g = gen(N + K)
    off = offsets_of(counts)
    live, rows, E = int(off[-1]), int(off[-1]) + extra, len(counts)
    a, sa = codes(g, rows, K), torch.randn(rows, generator=g, device=dev()).exp()
    sa[live:] = float("nan")
    w, sw = codes(g, E, N, K), scales(g, (E, N), K)
    y, flags = product(a, sa, on(off), w, sw, dt)
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        if counts[e]:
            f = sa[r, None].double() * sw[e].double()
            slack = 11 * P.U32 * mm(a[r].double().abs(), w[e].double().abs()) * f
            assert within(y[r], mm(a[r], w[e]) * f, slack, dt), e
    assert (y[live:] == -7.0).all() and flags == 0


def ffn64(xc, xs, gate, up, down):
    """plain_block.ffn_int8 for one expert's rows, on the device"""
    g = mm(xc, gate[0]) * xs[:, None].double() * gate[1].double()
    u = mm(xc, up[0]) * xs[:, None].double() * up[1].double()
    h = g / (1 + torch.exp(-g)) * u
    d = (16 + 4 * g.abs()) * P.U32
    low, mid, high = ((h * f).clamp(-65504, 65504).half().double() for f in (1 - d, torch.ones_like(d), 1 + d))
    top = [v.abs().amax(1, keepdim=True) for v in (low, mid, high)]

    def rounded(v, t):
        return torch.where(t > 0, 127 * v / t, torch.zeros_like(v)).round()

    c, s = rounded(mid, top[1]), top[1] / 127
    moved = torch.stack([(rounded(v, t) - c).abs() for v in (low, high) for t in top]).amax(0)
    f = s * down[1].double()
    y = mm(c, down[0]) * f
    absdown = down[0].double().abs()
    slack = mm(moved, absdown) * f
    shift = torch.where(top[1] > 0, torch.maximum((top[0] - top[1]).abs(), (top[2] - top[1]).abs()) / top[1],
                        torch.zeros_like(s))
    return y, slack + mm(c.abs(), absdown) * f * (shift + 12 * P.U32)


FFNS = [
    # H, I, rows per expert, top_k, rows left over
    (7168, 2048, [1] * 8, 8, 0),                        # one token: split gate/up of 32-row tiles, two-part down
    (4096, 14336, [1, 0, 3, 0, 2, 0, 0, 0], 1, 1),      # a few tokens: eight-part down
    (4096, 14336, [14, 20, 9, 33, 0, 31, 1, 20], 2, 0),  # 16 to 64 rows an expert
    (2048, 4224, [60, 1, 33, 64, 32, 0, 90, 50], 2, 4),
    (4096, 14336, [14, 20, 9, 3, 0, 11, 1, 6], 2, 0),    # 32-row tiles, two parts in the down projection
    (7168, 640, [15, 33, 1, 0, 20, 40, 9, 17, 30, 5, 6, 12, 18, 11, 16, 7], 2, 6),  # the same, no parts
    (512, 2048, [4, 1, 7, 0] * 16, 4, 8),                # many experts of few rows
    (2048, 14336, [300, 129, 63, 20, 0, 0, 0, 0], 2, 0),  # large tiles, three parts
]


def draw_ffn(H, I, E, seed):
    g = gen(seed)
    return tuple((codes(g, E, n, k), scales(g, (E, n), k)) for n, k in ((I, H), (I, H), (H, I)))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("H,I,counts,k,extra", FFNS)
def test_grouped_ffn(H, I, counts, k, extra, dt):
    say(f"int8 ffn H={H} I={I} {counts} k={k} +{extra} {dt}")
    E, off, g = len(counts), offsets_of(counts), gen(H + I + 1)
    live, rows = int(off[-1]), int(off[-1]) + extra
    assert rows % k == 0
    x, xs = codes(g, rows, H), (1 + torch.rand(rows, generator=g, device=dev())) / 73
    xs[live:] = float("nan")
    w = draw_ffn(H, I, E, H + I)
    y, flags = run_ffn(x, xs, on(off), abi.int8_ffn(*w), H, I, E, rows // k, k, dt)
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        if counts[e]:
            want, slack = ffn64(x[r], xs[r], *((c[e], s[e]) for c, s in w))
            assert within(y[r], want, slack, dt), e
    assert (y[live:] == -7.0).all() and flags == 0


@pytest.mark.parametrize("H,I,tokens,E,k", [(7168, 2048, 1, 8, 8), (4096, 14336, 40, 4, 1), (2048, 14336, 300, 2, 1)])
def test_ranges_are_flagged(H, I, tokens, E, k):
    """h outside fp16 is clamped and flagged, and so is y; rows without such a value are untouched by it."""
    rows = tokens * k
    x = torch.full((rows, H), 127, dtype=torch.int8, device=dev())
    xs = torch.full((rows,), 1e-6, device=dev())
    xs[0] = 1.0
    w1 = torch.full((E, I, H), 127, dtype=torch.int8, device=dev())
    w2 = torch.full((E, H, I), 127, dtype=torch.int8, device=dev())
    one = torch.ones(E, I, device=dev())
    off = torch.tensor([rows * i // E for i in range(E + 1)], dtype=torch.int32, device=dev())
    for scale, dt, flag in ((1e-6, "f32", abi.MOE_FLAG_H_RANGE),
                            (1.0, "f16", abi.MOE_FLAG_H_RANGE | abi.MOE_FLAG_Y_RANGE)):
        w = abi.int8_ffn((w1, one), (w1, one), (w2, torch.full((E, H), scale, device=dev())))
        y, flags = run_ffn(x, xs, off, w, H, I, E, tokens, k, dt)
        assert flags == flag
        want = 65504.0 * 127 * I * scale               # every h of row 0 is 65504: code 127, scale 65504 / 127
        if dt == "f32":
            assert torch.all((y[0] - want).abs() <= 12 * P.U32 * want) and torch.isfinite(y).all()
        else:
            assert torch.isinf(y[0]).all()


BLOCKS = {
    "one_token": tiny(tokens=1, top_k=8, k_choices=None, capacity_factor=0.0, shared_inter=0).replace(
        hidden=7168, inter=2048, experts=8),
    "shared_split": tiny(tokens=100, top_k=2, k_choices=None, capacity_factor=0.0, shared_inter=2048).replace(hidden=2048),
    "shared_wide": tiny(tokens=100, top_k=2, k_choices=None, capacity_factor=0.0, shared_inter=8448).replace(hidden=1024),
    "shared_large": tiny(tokens=40, top_k=2, k_choices=None, capacity_factor=0.0, shared_inter=16384).replace(hidden=2048),
    "large_split": tiny(tokens=150, top_k=2, k_choices=None, capacity_factor=0.0, shared_inter=256).replace(
        hidden=1024, inter=14336, experts=4),
    "lds_few": tiny(tokens=20, top_k=2, k_choices=None, capacity_factor=0.0).replace(
        hidden=2048, inter=14336, experts=4),
    "lds_split": tiny(tokens=40, top_k=2, k_choices=None, capacity_factor=0.0).replace(
        hidden=2048, inter=14336, experts=4),
}


@pytest.mark.parametrize("name", BLOCKS)
def test_int8_block(name):
    """The layer's tolerance, 2e-2 of the rms; and the same bits on every replay of a captured call."""
    say(f"int8 block {name}")
    b = Block(BLOCKS[name], stream="f32", seed=21)
    out, d, ws = f32((b.T, b.H)), b.debug(), b.workspace(True)
    b.run(True, out, ws, d)
    torch.cuda.synchronize()
    tokens = np.arange(min(b.T, 24))
    want = b.plain(True, d, tokens)
    err = np.abs(np64(out)[tokens] - want)
    say(f"  max err / rms {err.max() / rms(want):.2e}")
    assert err.max() <= 2e-2 * rms(want)
    assert abi.moe_read_device_flags(ws) == 0
    again = torch.empty_like(out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.run(True, again, ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.run(True, again, ws)
    for _ in range(3):
        again.fill_(float("nan"))
        ws.fill_(0x5A)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(again, out)


@pytest.mark.parametrize("offsets", [False, True])
def test_rows_and_outputs_past_32_bit_offsets(offsets):
    """More than 2^31 codes of rows, and more than 2^31 outputs."""
    for rows, N, K in ((600_001, 16, 4096), (300_001, 8192, 128)):
        a = torch.ones(rows, K, dtype=torch.int8, device=dev())
        a[-1], a[-2] = 3, 2
        w = torch.ones(1, N, K, dtype=torch.int8, device=dev())
        w[0, -1] = -1
        off = torch.tensor([0, rows], dtype=torch.int32, device=dev()) if offsets else None
        y, flags = product(a, torch.ones(rows, device=dev()), off, w, torch.ones(1, N, device=dev()), "bf16")
        for r, f in ((0, 1), (rows // 2, 1), (rows - 3, 1), (rows - 2, 2), (rows - 1, 3)):
            assert bool((y[r, :-1] == f * K).all()) and float(y[r, -1]) == -f * K, (rows, r)
        assert flags == 0
        del a, w, y


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,N,K,parts", [(60, 28672, 8192, 2), (64, 4096, 14336, 3), (100, 4096, 14336, 3),
                                            (300, 4096, 14336, 3), (700, 1040, 14336, 3), (2100, 512, 16384, 4)])
def test_split_products_of_all_rows(rows, N, K, parts, dt):
    """Without offsets: K in parts, for each height of the row tiles, and the sum of the parts."""
    say(f"int8 gemm of all rows {rows} x {N} x {K} {dt}")
    assert abi.moe_workspace_size_gemm_int8(rows, N, K, 1) >= parts * rows * N * 4
    g = gen(rows + N)
    a, sa = codes(g, rows, K), torch.randn(rows, generator=g, device=dev()).exp()
    w, sw = codes(g, 1, N, K), scales(g, (1, N), K)
    y, flags = product(a, sa, None, w, sw, dt)
    f = sa[:, None].double() * sw[0].double()
    slack = 11 * P.U32 * mm(a.double().abs(), w[0].double().abs()) * f
    assert within(y, mm(a, w[0]) * f, slack, dt) and flags == 0
    if dt == "f16":
        big = sa.clone()
        big[rows // 2] = 1e9
        y2, flags = product(a, big, None, w, sw, dt)
        keep = [r for r in range(rows) if r != rows // 2]
        assert flags == abi.MOE_FLAG_Y_RANGE and torch.equal(y2[keep], y[keep])
