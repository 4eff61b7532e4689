"""What the routing with a balance bias, the int8 and the block entry points refuse, and what they accept without
work: host checks only, no kernel is launched and no pointer read."""

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
    return abi.MoeInt8Ffn(**f)


def block(**kw):
    b = abi.make_block(stream_dtype=BF16)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


def test_route_biased_refusals():
    L, s = abi.lib(), shape()
    ws = abi.moe_workspace_size(s)

    def call(s=s, x=None, w=None, sel=P, logits=P, lo=None, kpt=None, ids=P, gates=P, wsp=P, n=ws):
        return L.moe_route_biased(ctypes.byref(s), x, w, None, sel, logits, lo, kpt, ids, gates, wsp, n, None)

    assert call(sel=None) == INV
    assert call(sel=BAD) == INV
    assert call(ids=None) == INV and call(gates=None) == INV and call(wsp=None) == INV and call(wsp=ODD) == INV
    assert call(logits=None) == INV                       # neither logits nor x and a router
    assert call(logits=None, x=P) == INV
    assert call(logits=BAD) == INV and call(lo=ODD) == INV and call(kpt=BAD) == INV
    assert call(n=ws - 1) == WSP
    assert call(s=shape(top_k=0)) == INV
    assert call(s=shape(num_experts=513)) == UNS
    assert call(s=shape(num_groups=8, topk_groups=1, top_k=2)) == INV
    zero = shape(num_tokens=0)
    assert call(s=zero) == 0


@pytest.mark.parametrize("args,status", [
    ((-1, 128, BF16, P, P, P), INV), ((4, 0, BF16, P, P, P), INV), ((4, 128, 3, P, P, P), INV),
    ((4, 64, BF16, P, P, P), UNS), ((4, 130, F32, P, P, P), UNS),
    ((4, 128, BF16, None, P, P), INV), ((4, 128, BF16, ODD, P, P), INV), ((4, 128, BF16, P, ODD, P), INV),
    ((4, 128, BF16, P, P, BAD), INV), ((4, 128, BF16, P, None, P), INV), ((0, 128, F16, P, P, P), 0),
])
def test_quantize_refusals(args, status):
    assert abi.lib().moe_quantize_int8(*args, None) == status


@pytest.mark.parametrize("dims,status", [
    ((-1, 64, 128, 1), INV), ((4, 0, 128, 1), INV), ((4, 64, 0, 1), INV), ((4, 64, 128, 0), INV),
    ((4, 64, 128, 513), UNS), ((4, 24, 128, 1), UNS), ((4, 64, 192, 1), UNS), ((4, 64, 131200, 1), UNS),
    ((4, 16384, 131072, 1), UNS), ((4, 1 << 23, 128, 512), UNS), ((4, 16, 131072, 1), 0),
])
def test_gemm_dimensions(dims, status):
    n = ctypes.c_size_t(0)
    assert abi.lib().moe_workspace_size_gemm_int8(*dims, ctypes.byref(n)) == status
    assert abi.lib().moe_workspace_size_gemm_int8(4, 64, 128, 1, None) == INV


def test_gemm_refusals():
    L = abi.lib()
    ws = abi.moe_workspace_size_gemm_int8(64, 256, 512, 4)

    def call(rows=64, n=256, k=512, E=4, a=P, sa=P, off=P, b=P, sb=P, dt=F32, y=P, wsp=P, size=ws):
        return L.moe_grouped_gemm_int8(rows, n, k, E, a, sa, off, b, sb, dt, y, wsp, size, None)

    assert call(a=None) == INV and call(a=ODD) == INV and call(sa=None) == INV and call(sa=BAD) == INV
    assert call(off=None) == INV                            # several experts need their offsets
    assert call(b=ODD) == INV and call(sb=ODD) == INV and call(y=ODD) == INV and call(wsp=None) == INV
    assert call(dt=3) == INV and call(dt=-1) == INV
    assert call(size=ws - 1) == WSP
    assert call(rows=0) == 0
    assert call(rows=0, E=1, off=None) == 0


@pytest.mark.parametrize("bad,status", [
    (dict(hidden=4160), UNS), (dict(intermediate=14400), UNS), (dict(shared_intermediate=64), UNS),
    (dict(act_dtype=F32), UNS), (dict(down_dtype=F16), UNS), (dict(intermediate=131200), UNS),
    (dict(num_tokens=-1), INV), (dict(top_k=9), INV),
])
def test_int8_shapes(bad, status):
    n = ctypes.c_size_t(0)
    s = shape(**bad)
    assert abi.lib().moe_workspace_size_int8(ctypes.byref(s), ctypes.byref(n)) == status


def test_ffn_int8_refusals():
    L, s = abi.lib(), shape()
    ws = abi.moe_workspace_size_int8(s)

    def call(s=s, x=P, xs=P, off=P, w=ffn(), dt=F16, y=P, wsp=P, n=ws):
        return L.moe_grouped_ffn_int8(ctypes.byref(s), x, xs, off, ctypes.byref(w) if w else None, dt, y, wsp, n,
                                      None)

    assert call(x=None) == INV and call(x=ODD) == INV and call(xs=BAD) == INV and call(off=None) == INV
    assert call(w=None) == INV
    for name in ("gate", "gate_scales", "up", "up_scales", "down", "down_scales"):
        assert call(w=ffn(**{name: None})) == INV, name
        assert call(w=ffn(**{name: ODD})) == INV, name
    assert call(dt=7) == INV and call(y=ODD) == INV and call(wsp=ODD) == INV
    assert call(n=ws - 1) == WSP
    assert call(s=shape(num_tokens=0)) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INV), (dict(cols=0), INV), (dict(src=F16), INV), (dict(odt=F16), INV),
    (dict(eps=0.0), INV), (dict(eps=-1e-6), INV), (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV),
    (dict(out=None), INV), (dict(codes=P), INV), (dict(scales=P), INV),
    (dict(cols=96), UNS), (dict(cols=96, src=F32, odt=F32, rows=0), 0), (dict(cols=6, src=F32, odt=F32), UNS),
    (dict(cols=192, codes=P, scales=P), UNS), (dict(x=None), INV), (dict(x=ODD), INV), (dict(w=ODD), INV),
    (dict(out=ODD), INV), (dict(codes=ODD, scales=P), INV), (dict(codes=P, scales=BAD), INV),
    (dict(x=P, out=P, src=F32), INV), (dict(rows=0, out=P), 0),
])
def test_norm_refusals(kw, status):
    a = dict(rows=4, cols=128, src=BF16, x=P, w=None, eps=1e-6, odt=BF16, out=2 * P, codes=None, scales=None)
    a.update(kw)
    assert abi.lib().moe_norm(a["rows"], a["cols"], a["src"], a["x"], a["w"], a["eps"], a["odt"], a["out"],
                              a["codes"], a["scales"], None) == status


BLOCK_ERRORS = [
    (dict(eps=0.0), INV), (dict(eps=float("nan")), INV), (dict(residual_scale=float("inf")), INV),
    (dict(stream_dtype=F16), INV), (dict(post_norm=ODD), INV),
    (dict(gate=P, gate_dtype=F16), INV), (dict(gate=BAD, gate_dtype=F32), INV), (dict(gate=P + 1, gate_dtype=BF16), INV),
    (dict(gate=P, gate_row_stride=-1), INV), (dict(gate=P, gate_col_stride=2), INV),
]


@pytest.mark.parametrize("bad,status", BLOCK_ERRORS)
def test_combine_norm_refuses_the_block(bad, status):
    s, b = shape(num_tokens=4), block(**bad)
    assert abi.lib().moe_combine_norm(ctypes.byref(s), ctypes.byref(b), F16, P, P, P, None, P, P, None) == status


def test_combine_norm_refusals():
    L, s = abi.lib(), shape(num_tokens=4)

    def call(s=s, b=block(), dt=F16, y=P, rows=P, g=P, sh=None, res=P, out=P):
        return L.moe_combine_norm(ctypes.byref(s), ctypes.byref(b) if b else None, dt, y, rows, g, sh, res, out, None)

    assert call(b=None) == INV and call(dt=5) == INV
    assert call(y=None) == INV and call(y=ODD) == INV and call(rows=None) == INV and call(g=BAD) == INV
    assert call(sh=ODD) == INV and call(res=ODD) == INV and call(out=None) == INV and call(out=ODD) == INV
    assert call(res=None) == INV                             # a residual scale without a residual
    assert call(s=abi.make_shape(num_tokens=4, hidden=132, num_experts=4, intermediate=64, act_dtype=F32)) == UNS
    assert call(s=shape(num_tokens=0), b=block(residual_scale=0.0), res=None) == 0


def test_block_refusals():
    L, s = abi.lib(), shape()
    ws = abi.moe_workspace_size_block(s)
    wsi = abi.moe_workspace_size_int8(s)

    def call(s=s, b=block(), x=P, wr=P, w=(P, P, P, None, None, None), out=P, wsp=P, n=ws):
        return L.moe_block_forward(ctypes.byref(s), ctypes.byref(b) if b else None, x, wr, None, None, *w, out, None,
                                   wsp, n, None)

    def call8(s=s, b=block(), x=P, wr=P, w=ffn(), sh=None, out=P, wsp=P, n=wsi):
        return L.moe_block_forward_int8(ctypes.byref(s), ctypes.byref(b) if b else None, x, wr, None, None,
                                        ctypes.byref(w) if w else None, ctypes.byref(sh) if sh else None, out, None,
                                        wsp, n, None)

    for f, size in ((call, ws), (call8, wsi)):
        assert f(b=None) == INV and f(x=None) == INV and f(wr=ODD) == INV and f(out=ODD) == INV and f(wsp=None) == INV
        assert f(n=size - 1) == WSP
        assert f(b=block(select_bias=BAD)) == INV and f(b=block(pre_norm=ODD)) == INV
        assert f(b=block(stream_dtype=F32)) == UNS           # the layer cannot take an fp32 stream without a norm
        for bad, status in BLOCK_ERRORS:
            assert f(b=block(**bad)) == status, bad
        assert f(s=shape(num_tokens=0)) == 0
    assert call(w=(P, None, P, None, None, None)) == INV
    assert call(s=shape(shared_intermediate=128), n=1 << 40) == INV   # its weights are missing
    assert call8(w=None) == INV and call8(w=ffn(up=None)) == INV
    assert call8(s=shape(shared_intermediate=128), n=1 << 40) == INV
    f32 = abi.make_shape(num_tokens=4, hidden=132, num_experts=4, intermediate=64, act_dtype=F32)
    assert call(s=f32, b=block(pre_norm=P), n=1 << 40) == UNS         # bf16 rows of 132 are not 16-byte aligned
    n = ctypes.c_size_t(0)
    assert L.moe_workspace_size_block(ctypes.byref(shape(top_k=0)), ctypes.byref(n)) == INV
    assert L.moe_workspace_size_block(ctypes.byref(s), None) == INV
    assert L.moe_workspace_size_int8(ctypes.byref(s), None) == INV


def test_gate_strides_of_the_binding():
    import torch
    T, H = 5, 64
    assert [(b.gate_row_stride, b.gate_col_stride, b.gate_dtype) for b in (
        abi.make_block(gate=torch.zeros(H)), abi.make_block(gate=torch.zeros(1, H)),
        abi.make_block(gate=torch.zeros(T, 1, dtype=torch.bfloat16)), abi.make_block(gate=torch.zeros(T, H)),
        abi.make_block(gate=torch.zeros(T, 2 * H)[:, 3:3 + H]), abi.make_block(gate=torch.zeros(1, 1)))
    ] == [(0, 1, F32), (0, 1, F32), (1, 0, BF16), (H, 1, F32), (2 * H, 1, F32), (0, 0, F32)]
    with pytest.raises(ValueError):
        abi.make_block(gate=torch.zeros(T, 2 * H)[:, ::2])
    with pytest.raises(KeyError):
        abi.make_block(gate=torch.zeros(H, dtype=torch.float16))
    for dims in ((), (1, T, H)):
        with pytest.raises(ValueError):
            abi.make_block(gate=torch.zeros(dims))


def test_strided_tensors_are_not_quantised_on_another_stream():
    import torch
    with pytest.raises(ValueError):
        abi.quantize_int8(torch.zeros(128, 128).t(), stream=1)


@pytest.mark.parametrize("dims,tokens,taken", [
    ((64,), 5, True), ((1, 64), 5, True), ((5, 1), 5, True), ((5, 64), 5, True), ((1, 1), 5, True), ((1,), 5, True),
    ((9, 64), 5, True), ((9, 1), 5, True), ((5, 1), 0, True), ((0, 64), 0, True),   # rows of a padded batch
    ((32,), 5, False), ((1, 65), 5, False), ((5, 128), 5, False), ((4, 1), 5, False), ((2, 64), 5, False),
    ((0, 1), 5, False), ((5, 0), 5, False), ((64, 5), 5, False),
])
def test_gates_that_do_not_fit_the_call_are_refused(dims, tokens, taken):
    """Before the library sees them: their strides would be walked past the end of the tensor.  (What fits reaches the
    library, which finds that the other arguments are missing.)"""
    import torch
    s = abi.make_shape(num_tokens=tokens, hidden=64, num_experts=4, intermediate=64)
    b = abi.make_block(gate=torch.zeros(dims))
    calls = (lambda: abi.moe_combine_norm(s, b, F16, None, None, None, None, None, None, stream=1),
             lambda: abi.moe_block_forward(s, b, *[None] * 11, None, None, 0, stream=1),
             lambda: abi.moe_block_forward_int8(s, b, *[None] * 7, None, None, 0, stream=1))
    for f in calls:
        with pytest.raises(abi.MoeError if taken else ValueError):
            f()
    if 0 not in dims:
        b.gate, b.gate_row_stride = None, 0                  # (the struct is the caller's)
        with pytest.raises(abi.MoeError):
            calls[0]()
