"""Row calls on shapes of any layer: H that the layer's own type would not take, and buffers without rows."""

import numpy as np
import pytest
import torch

from expert_serving_amd import abi

import test_gpu_rows as G
from gpu_util import dev, say
from test_gpu_fp8 import DT, on

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,H,k,dropped,extra", G.ODD)
def test_columns_that_a_bf16_layer_does_not_take(T, H, k, dropped, extra, dt):
    """The same bits as on a shape of an fp32 layer, against which the forms are tested."""
    say(f"rows {T} x {H} k={k} {dt} on a bf16 shape")
    r = np.random.default_rng(T + H + k)
    n, b = T * k + extra, DT[dt][1]
    ros, g = on(G.slots(r, T, k, dropped, extra)), on(r.normal(size=(T, k)).astype(np.float32))
    x, rows = on(r.normal(size=(T, H)), DT[dt][0]), on(r.normal(size=(n, H)), DT[dt][0])
    results = []
    for act in (abi.MOE_F32, abi.MOE_BF16):
        s = abi.make_shape(num_tokens=T, hidden=H, num_experts=max(16, k), intermediate=64, top_k=k, act_dtype=act)
        z = lambda *sh: torch.full(sh, -7.0, device=dev(), dtype=x.dtype)  # noqa: E731
        f = lambda: torch.full((T, k), -7.0, device=dev())  # noqa: E731
        out, dx, dw, dy, dg = z(n, H), z(T, H), f(), z(n, H), f()
        abi.moe_dispatch_rows(s, b, x, ros, g, n, out)
        abi.moe_dispatch_rows_backward(s, b, rows, ros, n, g, x, dx, dw)
        abi.moe_combine_backward(s, b, x, b, rows, ros, g, n, dy, dg)
        results.append((out, dx, dw, dy, dg))
    assert all(torch.equal(p, q) for p, q in zip(*results))


def test_tensors_without_rows():
    """A batch whose tokens all go elsewhere: the permuted tensors are empty ones."""
    T, H, k, b = 5, 256, 2, abi.MOE_BF16
    s = abi.make_shape(num_tokens=T, hidden=H, num_experts=16, intermediate=64, top_k=k)
    ros, g = torch.full((T, k), -1, dtype=torch.int32, device=dev()), torch.ones(T, k, device=dev())
    x = torch.ones(T, H, device=dev(), dtype=torch.bfloat16)
    none, scales = torch.empty(0, H, device=dev(), dtype=torch.bfloat16), torch.empty(0, H // 128, device=dev())
    codes = torch.empty(0, H, device=dev(), dtype=torch.uint8)
    abi.moe_dispatch_rows(s, b, x, ros, g, 0, none)
    abi.moe_dispatch_rows_fp8(s, b, x, ros, 0, codes, scales)
    dx, dw, dg = torch.ones_like(x), torch.ones_like(g), torch.ones_like(g)
    abi.moe_dispatch_rows_backward(s, b, none, ros, 0, g, x, dx, dw)
    abi.moe_combine_backward(s, b, x, b, none, ros, g, 0, none, dg)
    abi.moe_combine_backward(s, b, x, b, none, ros, g, 0, none, None)
    assert (dx == 0).all() and (dw == 0).all() and (dg == 0).all()
    c, v = abi.quantize_fp8(none)
    assert c.shape == (0, H) and v.shape == (0, H // 128)
