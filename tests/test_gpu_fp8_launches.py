"""What the products on 8-bit floating-point blocks launch: the blocks of the kernels in a captured call."""

import ctypes

import pytest
import torch

from expert_serving_amd import abi

from gpu_util import dev, say

pytestmark = pytest.mark.gpu


class KernelNode(ctypes.Structure):
    """hipKernelNodeParams"""
    _fields_ = [("block", ctypes.c_uint * 3), ("extra", ctypes.c_void_p), ("func", ctypes.c_void_p),
                ("grid", ctypes.c_uint * 3), ("params", ctypes.c_void_p), ("shared", ctypes.c_uint)]


def grids(call):
    """Blocks of every kernel that a call enqueues, which is captured and not run."""
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        call()
    hip, graph, n = abi.lib(), ctypes.c_void_p(g.raw_cuda_graph()), ctypes.c_size_t(0)
    assert hip.hipGraphGetNodes(graph, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert hip.hipGraphGetNodes(graph, nodes, ctypes.byref(n)) == 0
    out = []
    for node in nodes:
        kind, k = ctypes.c_int(-1), KernelNode()
        assert hip.hipGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0 and kind.value == 0
        assert hip.hipGraphKernelNodeGetParams(ctypes.c_void_p(node), ctypes.byref(k)) == 0
        out.append(k.grid[0] * k.grid[1] * k.grid[2])
    return out


def most(rows, E, N, stream=False):
    """128 x 128 tiles that the rows of E experts can make, in eighths of equal size; of a stream, which is one launch
    without a list of tiles, tiles of 32 rows x 32 columns at least."""
    if stream:
        return (rows // 32 + min(rows, E)) * -(-N // 32)
    return -(-(rows // 256 + min(rows, E)) * 2 * -(-N // 128) // 8) * 8


@pytest.mark.parametrize("rows,E,N,K", [(1024, 1, 4096, 4096), (2000, 1, 4096, 4096), (600, 8, 4096, 14336),
                                        (5525, 15, 2688, 384), (8192, 8, 4096, 1024), (300, 64, 1024, 128)])
def test_blocks_of_a_product(rows, E, N, K):
    """A list of tiles and a product: no more blocks than there can be tiles, or the 256 that stay and draw theirs."""
    z = lambda *sh: torch.zeros(*sh, dtype=torch.uint8, device=dev())  # noqa: E731
    f = lambda *sh: torch.zeros(*sh, device=dev())  # noqa: E731
    a, sa, b, sb = z(rows, K), f(rows, K // 128), z(E, N, K), f(E, -(-N // 128), K // 128)
    off, y = torch.zeros(E + 1, dtype=torch.int32, device=dev()), torch.zeros(rows, N, dtype=torch.bfloat16, device=dev())
    ws = z(abi.moe_workspace_size_gemm_fp8(rows, N, K, E))
    got = grids(lambda: abi.moe_grouped_gemm_fp8(rows, N, K, E, a, sa, off, b, sb, abi.MOE_BF16, y, ws))
    bound = most(rows, E, N, len(got) == 1)
    say(f"fp8 gemm {rows} rows, {E} experts, {N} x {K}: blocks {got}, tiles {bound} at most")
    assert max(got) <= max(256, bound)


@pytest.mark.parametrize("rows,E,H,I", [(700, 1, 256, 640), (900, 4, 1024, 768)])
def test_blocks_of_an_ffn(rows, E, H, I):
    z = lambda *sh: torch.zeros(*sh, dtype=torch.uint8, device=dev())  # noqa: E731
    f = lambda *sh: torch.zeros(*sh, device=dev())  # noqa: E731
    x, xs, off = z(rows, H), f(rows, H // 128), torch.zeros(E + 1, dtype=torch.int32, device=dev())
    w = abi.fp8_ffn(*((z(E, n, k), f(E, n // 128, k // 128)) for n, k in ((I, H), (I, H), (H, I))))
    s = abi.make_shape(num_tokens=rows, hidden=H, num_experts=E, intermediate=I, top_k=1)
    y, ws = torch.zeros(rows, H, dtype=torch.bfloat16, device=dev()), z(abi.moe_workspace_size_fp8(s))
    got = grids(lambda: abi.moe_grouped_ffn_fp8(s, x, xs, off, w, abi.MOE_BF16, y, ws))
    say(f"fp8 ffn {rows} rows, {E} experts, {H} x {I}: blocks {got}, tiles {most(rows, E, H)} at most")
    assert max(got) <= max(256, most(rows, E, H))
