"""The pair kernel's grid, read from a captured graph: dx and dW sharing a
launch get a CTA pair for every tile of either while there are SMs."""
import ctypes as C

import pytest
import torch

pytestmark = pytest.mark.gpu

capi = pytest.importorskip("routed_nvfp4_expert_b200.capi")

BF16 = torch.bfloat16
PAIR_THREADS = 384


class _KernelNode(C.Structure):
    _fields_ = [("func", C.c_void_p), ("grid", C.c_uint * 3), ("block", C.c_uint * 3), ("smem", C.c_uint),
                ("params", C.c_void_p), ("extra", C.c_void_p), ("kern", C.c_void_p), ("ctx", C.c_void_p)]


def _launches(call):
    """(CTAs, threads) of every kernel that the call launches."""
    cu = C.CDLL("libcuda.so.1")
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    raw, n = C.c_void_p(graph.raw_cuda_graph()), C.c_size_t(0)
    assert cu.cuGraphGetNodes(raw, None, C.byref(n)) == 0
    nodes = (C.c_void_p * n.value)()
    assert cu.cuGraphGetNodes(raw, nodes, C.byref(n)) == 0
    out = []
    for node in nodes:
        kind, p = C.c_int(-1), _KernelNode()
        assert cu.cuGraphNodeGetType(C.c_void_p(node), C.byref(kind)) == 0
        if kind.value == 0:
            assert cu.cuGraphKernelNodeGetParams_v2(C.c_void_p(node), C.byref(p)) == 0
            out.append((p.grid[0] * p.grid[1] * p.grid[2], p.block[0]))
    return out


# tiles of dx [T, K] and dW [N, K]: 256 x 128, 256 x 128, 256 x 256, 256 x 128, 256 x 256
@pytest.mark.parametrize("T,K,N,tiles", [(1024, 1024, 1024, 32 + 32), (777, 1000, 515, 32 + 24), (1500, 1500, 1500, 36 + 36),
                                         (8720, 64, 8704, 35 + 34), (4096, 1024, 4096, 64 + 64)])
def test_a_pair_for_every_tile(T, K, N, tiles):
    x, w, dy = (torch.zeros(*s, dtype=BF16, device="cuda") for s in ((T, K), (N, K), (T, N)))
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ws = capi.alloc_linear_backward_workspace(dy, x, w)
    pairs = [ctas for ctas, threads in _launches(lambda: capi.linear_bf16_backward(dy, x, w, ws, dx=dx, dw=dw))
             if threads == PAIR_THREADS]
    assert pairs == [2 * min(74, tiles)]
