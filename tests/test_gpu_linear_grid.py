"""The pair kernel's grid, read from a captured graph: dx and dW sharing a
launch get a CTA pair for every tile of either while there are SMs."""
import pytest
import torch

from graph_launches import launches

pytestmark = pytest.mark.gpu

capi = pytest.importorskip("routed_nvfp4_expert_b200.capi")

BF16 = torch.bfloat16
PAIR_THREADS = 384


# tiles of dx [T, K] and dW [N, K]: 256 x 128, 256 x 128, 256 x 256, 256 x 128, 256 x 256
@pytest.mark.parametrize("T,K,N,tiles", [(1024, 1024, 1024, 32 + 32), (777, 1000, 515, 32 + 24), (1500, 1500, 1500, 36 + 36),
                                         (8720, 64, 8704, 35 + 34), (4096, 1024, 4096, 64 + 64)])
def test_a_pair_for_every_tile(T, K, N, tiles):
    x, w, dy = (torch.zeros(*s, dtype=BF16, device="cuda") for s in ((T, K), (N, K), (T, N)))
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ws = capi.alloc_linear_backward_workspace(dy, x, w)
    pairs = [ctas for ctas, threads in launches(lambda: capi.linear_bf16_backward(dy, x, w, ws, dx=dx, dw=dw))
             if threads == PAIR_THREADS]
    assert pairs == [2 * min(74, tiles)]
