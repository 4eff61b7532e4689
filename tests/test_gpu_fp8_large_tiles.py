"""The 256 x 256 tiles of the products on 8-bit floating-point blocks at sizes that stay on them whatever K is: more of
them than four on a compute unit at a short K, than 9 / 8 of the units up to K = 2048 and than 5 / 8 beyond.  Rows of an
expert repeat a few drawn ones, so that the 64-bit forms stay small."""

import numpy as np
import pytest
import torch

from expert_serving_amd import abi

import plain_fp8 as P
import test_gpu_fp8_run as R
from gpu_util import dev, say
from test_gpu_fp8 import codes8, draw_ffn, offsets_of, on, product, run_ffn
from test_gpu_fp8_ranges import spread

pytestmark = pytest.mark.gpu


def inside(y, want, tol, ref):
    """Largest share of its bound that an output's error takes, row i of y against row ref[i] of want."""
    top = 0.0
    want, tol, ref = on(want), on(tol), on(ref)
    for i in range(0, len(ref), 1024):
        at = ref[i:i + 1024]
        share = float(((y[i:i + 1024].double() - want[at]).abs() / tol[at]).max())
        assert share == share                       # (a NaN)
        top = max(top, share)
    return top


# rows per expert, column tiles at K up to 512 and beyond: tiles of every height, none cut; and a last round of the
# compute units that is cut, in quarters with all, with some and with none of their rows
SHAPES = [([256 * 12 + 7, 200, 130, 64, 1, 0, 300], 16400, 8208), ([256 * 16 + 100], 16384, 5120),
          ([256 * 16 + 1], 16368, 5104)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("K", [128, 256, 384, 1152, 2304])
@pytest.mark.parametrize("counts,short,long", SHAPES)
def test_products(counts, short, long, K, dt):
    N = short if K <= 512 else long
    say(f"fp8 large tiles {counts} N={N} K={K} {dt}")
    r = np.random.default_rng(N + K)
    E, D = len(counts), 24
    at, ref, roff = spread(counts, D)
    a, sa = P.exact_codes(r, D, K), P.scales_of(r, D, K // 128)
    w, sw = P.exact_codes(r, E, N, K), P.scales_of(r, E, -(-N // 128), K // 128) / 64
    live, extra = len(at), 5
    rows = np.concatenate([at, np.zeros(extra, int)])
    scales = sa[rows]
    scales[live:] = np.nan
    args = codes8(a[rows]), on(scales), on(offsets_of(counts)), codes8(w), on(sw), dt
    y, flags = product(*args)
    want, bound = P.product(np.tile(a, (E, 1)), np.tile(sa, (E, 1)), w, sw, roff, True)
    share = inside(y[:live], want, P.rounded(want, bound, dt), ref)
    say(f"  largest share of the bound {share:.2f}")
    assert flags == 0 and share <= 1 and (y[live:] == -7.0).all()
    again, _ = product(*args)
    assert torch.equal(y, again)                    # (whatever the blocks' order)


# rows per expert, H, I: both products on large tiles of one schedule, with a cut last round
FFNS = [([300, 2000, 1, 0, 700, 64, 129, 256], 4224, 2304), ([256 * 129 + 1], 512, 2304), ([256 * 40, 256 * 24 + 70], 1024, 2176)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("counts,H,I", FFNS)
def test_ffns(counts, H, I, dt):
    say(f"fp8 ffn on large tiles {counts} H={H} I={I} {dt}")
    r = np.random.default_rng(H + I)
    E, D = len(counts), 16
    at, ref, roff = spread(counts, D)
    x, xs = P.exact_codes(r, D, H), P.scales_of(r, D, H // 128)
    live, extra = len(at), 3
    rows = np.concatenate([at, np.zeros(extra, int)])
    scales = xs[rows]
    scales[live:] = np.nan
    parts = draw_ffn(r, H, I, E)
    w = abi.fp8_ffn(*((codes8(c), on(s)) for c, s in parts))
    args = codes8(x[rows]), on(scales), on(offsets_of(counts)), w, H, I, E, live + extra, 1, dt
    y, flags = run_ffn(*args)
    want, bound = P.ffn(np.tile(x, (E, 1)), np.tile(xs, (E, 1)), *parts, roff, True)
    share = inside(y[:live], want, P.rounded(want, bound, dt), ref)
    say(f"  largest share of the bound {share:.2f}")
    assert flags == 0 and share <= 1 and (y[live:] == -7.0).all()
    again, _ = run_ffn(*args)
    assert torch.equal(y, again)


def test_captured_and_replayed():
    R.test_captured_and_replayed(3300, 2560, 2304, 2, 2)


def test_two_streams_at_once():
    R.test_two_streams_at_once(3300, 2560, 2304, 2, 2)


def test_products_of_values_that_are_not_finite():
    R.test_products_of_values_that_are_not_finite(5000, 2560, 2304)


def test_ffn_of_values_that_are_not_finite():
    R.test_ffn_of_values_that_are_not_finite(7000, 2304, 2560)


def test_all_codes_and_scales_far_apart():
    R.test_tiles_of_all_codes_and_scales_far_apart(4500, 2560, 2304)
