"""What the entry points on 8-bit floating-point blocks, the row permutations and their gradients refuse, and what they
accept without work: host checks only, no kernel is launched and no pointer read."""

import ctypes

import pytest

import workloads as W
from expert_serving_amd import abi

P = 0x10000        # aligned, never read
ODD = 0x10004      # 4-byte aligned only
BAD = 0x10002      # 2-byte aligned only
INV, UNS, WSP = abi.MOE_ERR_INVALID_ARG, abi.MOE_ERR_UNSUPPORTED, abi.MOE_ERR_WORKSPACE
F32, BF16, F16 = abi.MOE_F32, abi.MOE_BF16, abi.MOE_F16


def shape(**kw):
    return abi.make_shape(W.CONFIGS["mixtral_decode"], **kw)


def ffn(**kw):
    f = dict.fromkeys(("gate", "gate_scales", "up", "up_scales", "down", "down_scales"), P)
    f.update(kw)
    return abi.MoeFp8Ffn(**f)


@pytest.mark.parametrize("args,status", [
    ((-1, 128, BF16, P, P, P), INV), ((4, 0, BF16, P, P, P), INV), ((4, 128, 3, P, P, P), INV),
    ((4, 64, BF16, P, P, P), UNS), ((4, 130, F32, P, P, P), UNS),
    ((4, 128, BF16, None, P, P), INV), ((4, 128, BF16, ODD, P, P), INV), ((4, 128, BF16, P, ODD, P), INV),
    ((4, 128, BF16, P, P, BAD), INV), ((4, 128, BF16, P, None, P), INV), ((0, 128, F16, P, P, P), 0),
])
def test_quantize_refusals(args, status):
    assert abi.lib().moe_quantize_fp8(*args, None) == status


@pytest.mark.parametrize("args,status", [
    ((0, 128, 128, BF16, P, P, P), INV), ((1, 0, 128, BF16, P, P, P), INV), ((1, 128, 128, 5, P, P, P), INV),
    ((1, 24, 128, BF16, P, P, P), UNS), ((1, 128, 192, BF16, P, P, P), UNS), ((513, 128, 128, BF16, P, P, P), UNS),
    ((1, 1 << 17, 1 << 15, BF16, P, P, P), UNS), ((1, 16 << 20, 128, BF16, P, P, P), UNS),
    ((1, 128, 128, BF16, ODD, P, P), INV), ((1, 128, 128, BF16, P, None, P), INV), ((1, 128, 128, F32, P, P, BAD), INV),
])
def test_quantize_weights_refusals(args, status):
    assert abi.lib().moe_quantize_fp8_weights(*args, None) == status


@pytest.mark.parametrize("dims,status", [
    ((-1, 64, 128, 1), INV), ((4, 0, 128, 1), INV), ((4, 64, 0, 1), INV), ((4, 64, 128, 0), INV),
    ((4, 64, 128, 513), UNS), ((4, 24, 128, 1), UNS), ((4, 64, 192, 1), UNS), ((4, 64, 262144, 1), 0),
    ((4, 16384, 131072, 1), UNS), ((4, 1 << 23, 128, 512), UNS), ((0, 64, 128, 1), 0),
    ((1 << 30, 64, 128, 1), UNS),
])
def test_gemm_dimensions(dims, status):
    n = ctypes.c_size_t(0)
    assert abi.lib().moe_workspace_size_gemm_fp8(*dims, ctypes.byref(n)) == status
    assert abi.lib().moe_workspace_size_gemm_fp8(4, 64, 128, 1, None) == INV


def test_gemm_refusals():
    L = abi.lib()
    ws = abi.moe_workspace_size_gemm_fp8(64, 256, 512, 4)

    def call(rows=64, n=256, k=512, E=4, a=P, sa=P, off=P, b=P, sb=P, dt=BF16, y=P, wsp=P, size=ws):
        return L.moe_grouped_gemm_fp8(rows, n, k, E, a, sa, off, b, sb, dt, y, wsp, size, None)

    assert call(a=None) == INV and call(a=ODD) == INV and call(sa=None) == INV and call(sa=BAD) == INV
    assert call(off=None) == INV and call(off=BAD) == INV   # several experts need their offsets
    assert call(b=ODD) == INV and call(sb=None) == INV and call(sb=BAD) == INV
    assert call(y=ODD) == INV and call(wsp=None) == INV and call(wsp=ODD) == INV
    assert call(dt=3) == INV and call(dt=-1) == INV
    assert call(dt=F32) == UNS                              # the matrix units' sums do not carry 24 bits
    assert call(size=ws - 1) == WSP
    assert call(rows=0) == 0
    assert call(rows=0, E=1, off=None) == 0


@pytest.mark.parametrize("bad,status", [
    (dict(hidden=4160), UNS), (dict(intermediate=14400), UNS), (dict(act_dtype=F32), UNS), (dict(down_dtype=F16), UNS),
    (dict(num_tokens=-1), INV), (dict(top_k=9), INV), (dict(num_experts=513), UNS),
])
def test_fp8_shapes(bad, status):
    n = ctypes.c_size_t(0)
    s = shape(**bad)
    assert abi.lib().moe_workspace_size_fp8(ctypes.byref(s), ctypes.byref(n)) == status


def test_ffn_refusals():
    L, s = abi.lib(), shape()
    ws = abi.moe_workspace_size_fp8(s)

    def call(s=s, x=P, xs=P, off=P, w=ffn(), dt=F16, y=P, wsp=P, n=ws):
        return L.moe_grouped_ffn_fp8(ctypes.byref(s), x, xs, off, ctypes.byref(w) if w else None, dt, y, wsp, n, None)

    assert call(x=None) == INV and call(x=ODD) == INV and call(xs=BAD) == INV and call(off=None) == INV
    assert call(w=None) == INV
    for name in ("gate", "up", "down"):
        assert call(w=ffn(**{name: None})) == INV and call(w=ffn(**{name: ODD})) == INV, name
        assert call(w=ffn(**{name + "_scales": None})) == INV and call(w=ffn(**{name + "_scales": BAD})) == INV, name
    assert call(dt=7) == INV and call(dt=F32) == UNS and call(y=ODD) == INV and call(wsp=ODD) == INV
    assert call(n=ws - 1) == WSP
    assert call(s=shape(num_tokens=0)) == 0


def test_dispatch_rows_refusals():
    L = abi.lib()

    def call(s=shape(), dt=BF16, x=P, ros=P, w=None, n=128, out=P):
        return L.moe_dispatch_rows(ctypes.byref(s), dt, x, ros, w, n, out, None)

    assert call(dt=3) == INV and call(dt=-1) == INV and call(n=-1) == INV
    assert call(x=None) == INV and call(x=ODD) == INV and call(ros=None) == INV and call(ros=BAD) == INV
    assert call(w=BAD) == INV and call(out=None) == INV and call(out=ODD) == INV
    odd = shape(act_dtype=F32, hidden=12)
    assert call(s=odd) == UNS and call(s=odd, dt=F16) == UNS and call(s=odd, dt=F32, n=0) == 0
    assert call(s=shape(num_tokens=0)) == 0 and call(n=0) == 0
    assert L.moe_dispatch_rows(None, BF16, P, P, None, 4, P, None) == INV


def test_dispatch_rows_fp8_refusals():
    L = abi.lib()

    def call(s=shape(), dt=BF16, x=P, ros=P, n=128, codes=P, scales=P):
        return L.moe_dispatch_rows_fp8(ctypes.byref(s), dt, x, ros, n, codes, scales, None)

    assert call(dt=3) == INV and call(n=-1) == INV and call(x=ODD) == INV and call(ros=BAD) == INV
    assert call(codes=ODD) == INV and call(codes=None) == INV and call(scales=None) == INV and call(scales=BAD) == INV
    assert call(s=shape(hidden=192)) == UNS
    assert call(s=shape(num_tokens=0)) == 0 and call(n=0) == 0


def test_dispatch_rows_backward_refusals():
    L = abi.lib()

    def call(s=shape(), dt=BF16, dp=P, ros=P, n=128, w=P, x=P, dx=P, dw=P):
        return L.moe_dispatch_rows_backward(ctypes.byref(s), dt, dp, ros, n, w, x, dx, dw, None)

    assert call(dt=3) == INV and call(n=-1) == INV and call(dp=None) == INV and call(dp=ODD) == INV
    assert call(ros=None) == INV and call(w=BAD) == INV and call(dx=ODD) == INV and call(dw=BAD) == INV
    assert call(dx=None, dw=None) == INV
    assert call(w=None) == INV                              # no weights, no gradient of them
    assert call(x=None) == INV and call(x=ODD) == INV       # the weights' gradient reads x
    assert call(s=shape(act_dtype=F32, hidden=12)) == UNS
    zero = shape(num_tokens=0)
    assert call(s=zero) == 0 and call(s=zero, w=None, x=None, dw=None) == 0 and call(s=zero, dx=None) == 0


def test_combine_backward_refusals():
    L = abi.lib()

    def call(s=shape(), odt=F32, do=P, ydt=BF16, y=P, ros=P, g=P, n=128, dy=P, dg=P):
        return L.moe_combine_backward(ctypes.byref(s), odt, do, ydt, y, ros, g, n, dy, dg, None)

    assert call(odt=3) == INV and call(ydt=-1) == INV and call(n=-1) == INV
    assert call(do=None) == INV and call(do=ODD) == INV and call(ros=None) == INV and call(g=None) == INV
    assert call(g=BAD) == INV and call(dy=ODD) == INV and call(dg=BAD) == INV and call(dy=None, dg=None) == INV
    assert call(y=None) == INV and call(y=ODD) == INV       # the gates' gradient reads y
    odd = shape(act_dtype=F32, hidden=12)
    assert call(s=odd) == UNS and call(s=odd, ydt=F32, odt=F16) == UNS
    zero = shape(num_tokens=0)
    assert call(s=zero) == 0 and call(s=zero, y=None, dg=None) == 0 and call(s=zero, dy=None) == 0


def test_helpers_refuse_strided_tensors_on_a_stream():
    import torch
    t = torch.zeros(4, 256)[:, ::2]
    for f in (abi.quantize_fp8, abi.quantize_fp8_weights):
        with pytest.raises(ValueError):
            f(t, stream=1)
