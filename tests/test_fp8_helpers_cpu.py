"""What the helpers around the calls on 8-bit floating-point blocks refuse before any call."""

import pytest
import torch

from expert_serving_amd import abi


@pytest.mark.parametrize("shape", [(256,), (2, 3, 128, 256), (1, 1, 1, 128, 128)])
def test_weights_are_matrices(shape):
    """A tensor of other dimensions than [N, K] and [E, N, K] is refused rather than quantised in part."""
    with pytest.raises(ValueError, match="N, K"):
        abi.quantize_fp8_weights(torch.ones(shape))


@pytest.mark.parametrize("f", [abi.quantize_fp8, abi.quantize_fp8_weights, abi.quantize_int8, abi.quantize_mxfp8,
                               lambda t: abi.to_f16_weights(t.bfloat16())])
def test_host_tensors_are_refused(f):
    """A kernel that read one would fault."""
    with pytest.raises(ValueError, match="GPU"):
        f(torch.ones(128, 128))


def test_helpers_run_on_their_tensors_device():
    """Not on the current device, whose stream knows nothing of the other's work."""
    at = abi._tensors_on(None, torch.device("cuda", 1))
    assert isinstance(at, torch.cuda.device) and at.idx == 1


P = 0x10000   # aligned, never read


@pytest.mark.parametrize("fields", [dict(act_dtype=abi.MOE_BF16), dict(act_dtype=abi.MOE_F32), dict(act_dtype=7),
                                    dict(num_experts=0), dict(intermediate=0, score=9, out_dtype=5, num_groups=0)])
def test_row_calls_take_tokens_columns_and_slots_from_their_shape(fields):
    """H is a multiple of 8, or of 4 where every row is fp32, whatever the layer's types and weights are."""
    L = abi.lib()

    def calls(hidden, dt, out, top_k=2, T=5):
        s = abi.make_shape(**dict(dict(num_tokens=T, hidden=hidden, num_experts=8, intermediate=64, top_k=top_k), **fields))
        got = {L.moe_dispatch_rows(s, dt, P, P, P, 0, P, None)}
        s.num_tokens = 0 if T > 0 else T           # (the gradients write without rows too)
        return got | {L.moe_dispatch_rows_backward(s, dt, P, P, 0, P, P, P, P, None),
                      L.moe_combine_backward(s, out, P, dt, P, P, P, 0, P, P, None)}

    for hidden in (8, 40, 1000, 192):
        for dt in (abi.MOE_F32, abi.MOE_BF16, abi.MOE_F16):
            assert calls(hidden, dt, abi.MOE_F32) == {0}, (hidden, dt)
    assert calls(12, abi.MOE_F32, abi.MOE_F32) == {0}
    assert calls(12, abi.MOE_BF16, abi.MOE_BF16) == {abi.MOE_ERR_UNSUPPORTED}
    assert calls(8, abi.MOE_F32, abi.MOE_F32, top_k=16) == {0}
    assert calls(8, abi.MOE_F32, abi.MOE_F32, top_k=17) == {abi.MOE_ERR_UNSUPPORTED}
    assert calls(8, abi.MOE_F32, abi.MOE_F32, top_k=0) == {abi.MOE_ERR_INVALID_ARG}
    assert calls(0, abi.MOE_F32, abi.MOE_F32) == {abi.MOE_ERR_INVALID_ARG}
    assert calls(8, abi.MOE_F32, abi.MOE_F32, T=-1) == {abi.MOE_ERR_INVALID_ARG}
    s = abi.make_shape(**dict(dict(num_tokens=3, hidden=192, num_experts=8, intermediate=64, top_k=2), **fields))
    assert L.moe_dispatch_rows_fp8(s, abi.MOE_BF16, P, P, 0, P, P, None) == abi.MOE_ERR_UNSUPPORTED
    s.hidden = 384
    assert L.moe_dispatch_rows_fp8(s, abi.MOE_BF16, P, P, 0, P, P, None) == 0


def test_row_calls_refuse_more_elements_than_an_int_counts():
    s = abi.make_shape(num_tokens=1 << 20, hidden=1 << 11, num_experts=8, intermediate=64, top_k=2)
    assert abi.lib().moe_dispatch_rows(s, abi.MOE_BF16, P, P, P, 0, P, None) == abi.MOE_ERR_UNSUPPORTED
    s.hidden, s.num_tokens, s.top_k = 8, 1 << 27, 16
    assert abi.lib().moe_dispatch_rows(s, abi.MOE_BF16, P, P, P, 0, P, None) == abi.MOE_ERR_UNSUPPORTED


def test_buffers_without_rows_may_be_null():
    """As those of torch tensors without elements are."""
    L = abi.lib()
    s = abi.make_shape(num_tokens=0, hidden=256, num_experts=8, intermediate=128, top_k=2)
    some = abi.make_shape(num_tokens=3, hidden=256, num_experts=8, intermediate=128, top_k=2)
    b, inv = abi.MOE_BF16, abi.MOE_ERR_INVALID_ARG
    assert L.moe_quantize_fp8(0, 128, b, None, None, None, None) == 0
    n = abi.moe_workspace_size_gemm_fp8(0, 64, 128, 4)
    assert L.moe_grouped_gemm_fp8(0, 64, 128, 4, None, None, P, P, P, b, None, P, n, None) == 0
    assert L.moe_grouped_gemm_fp8(0, 64, 128, 4, None, None, None, P, P, b, None, P, n, None) == inv
    w = abi.MoeFp8Ffn(P, P, P, P, P, P)
    assert L.moe_grouped_ffn_fp8(s, None, None, P, w, b, None, P, abi.moe_workspace_size_fp8(s), None) == 0
    for rows in (0, 5):
        assert L.moe_dispatch_rows(s, b, None, None, None, rows, None, None) == 0
        assert L.moe_dispatch_rows_fp8(s, b, None, None, rows, None, None, None) == 0
        assert L.moe_dispatch_rows_backward(s, b, None, None, rows, None, None, None, None, None) == 0
        assert L.moe_combine_backward(s, b, None, b, None, None, None, rows, None, None, None) == 0
    assert L.moe_dispatch_rows(some, b, P, P, None, 0, None, None) == 0
    assert L.moe_dispatch_rows_fp8(some, b, P, P, 0, None, None, None) == 0
    assert L.moe_combine_backward(some, b, P, b, None, P, P, 0, None, None, None) == 0
    assert L.moe_dispatch_rows(some, b, P, P, None, 1, None, None) == inv
    assert L.moe_dispatch_rows_fp8(some, b, P, P, 1, P, None, None) == inv
    assert L.moe_dispatch_rows_backward(some, b, None, P, 1, None, None, P, None, None) == inv
    assert L.moe_dispatch_rows_backward(some, b, P, P, 0, None, None, None, None, None) == inv
    assert L.moe_combine_backward(some, b, P, b, None, P, P, 1, None, P, None) == inv
    assert L.moe_combine_backward(some, b, P, b, P, P, P, 1, None, None, None) == inv
