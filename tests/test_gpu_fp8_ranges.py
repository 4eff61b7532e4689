"""The products and the FFN on 8-bit floating-point blocks at the ends of their ranges and on every plan, against the
64-bit forms (plain_fp8.py has the bounds)."""

import numpy as np
import pytest
import torch

from expert_serving_amd import abi

import plain_fp8 as P
from gpu_util import say
from test_gpu_fp8 import codes8, draw_ffn, np64, offsets_of, on, run_ffn

pytestmark = pytest.mark.gpu


def spread(counts, distinct):
    """Rows of many experts drawn from few: of every expert row i holds row i % distinct, so that the 64-bit form is
    taken of `distinct` rows per expert.  (row of the drawn ones, row of the 64-bit form) for each row, its offsets."""
    at = np.concatenate([np.arange(c) % distinct for c in counts]) if sum(counts) else np.zeros(0, int)
    return at, at + distinct * np.repeat(np.arange(len(counts)), counts), distinct * np.arange(len(counts) + 1)


# rows per expert, H, I: a stream whose second product quantises h, streams with a launch for it, 128 x 128 tiles for
# the second product, large tiles
LIFTED = [([3], 256, 128), ([9], 128, 4096), ([29], 256, 1280), ([700], 256, 640), ([300] * 8, 4224, 2304)]


@pytest.mark.parametrize("counts,H,I", LIFTED)
def test_ffn_of_h_near_the_end_of_fp32(counts, H, I):
    """Finite h up to 3e38: the codes of blocks whose maximum is above 2^126, the reciprocal of which is no normal
    number, are those of any other block."""
    say(f"fp8 ffn of large h {counts[:3]} H={H} I={I}")
    r = np.random.default_rng(H + I)
    E, D = len(counts), min(16, max(counts))
    at, ref, roff = spread(counts, D)
    x, xs = P.exact_codes(r, D, H), (1 + r.random((D, H // 128))).astype(np.float32)
    rx, rxs = np.tile(x, (E, 1)), np.tile(xs, (E, 1))
    g, u, d = draw_ffn(r, H, I, E)
    u, d = (u[0], (u[1] * 1e36).astype(np.float32)), (d[0], (d[1] * 1e-34).astype(np.float32))

    def h_of(u):
        ga, _ = P.product(rx, rxs, *g, roff, True)
        return np.abs(ga / (1 + np.exp(-ga)) * P.product(rx, rxs, *u, roff, True)[0])

    u = (u[0], (u[1] * (3e38 / h_of(u).max())).astype(np.float32))
    tops = h_of(u).reshape(len(rx), -1, 128).max(2)
    assert tops.max() < 3.3e38 and (tops > 2.0 ** 126).sum() >= 2
    w = abi.fp8_ffn(*((codes8(c), on(s)) for c, s in (g, u, d)))
    rows = len(at)
    y, flags = run_ffn(codes8(x[at]), on(xs[at]), on(offsets_of(counts)), w, H, I, E, rows, 1, "bf16")
    want, bound = P.ffn(rx, rxs, g, u, d, roff, True)
    share = (np.abs(np64(y) - want[ref]) / P.rounded(want, bound, "bf16")[ref]).max()
    say(f"  {(tops > 2.0 ** 126).sum()} of {tops.size} blocks above 2^126, largest share of the bound {share:.2f}")
    assert flags == 0 and share <= 1
