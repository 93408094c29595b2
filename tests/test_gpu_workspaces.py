"""One workspace of the largest batch for batches of other lengths."""
import pytest
import torch

pytestmark = pytest.mark.gpu

capi = pytest.importorskip("routed_nvfp4_expert_b200.capi")

BF16 = torch.bfloat16


def test_linear_backward():
    K, N = 72, 1024
    g = torch.Generator().manual_seed(0)
    x, w = torch.randn(4160, K, generator=g).to(BF16).cuda(), torch.randn(N, K, generator=g).to(BF16).cuda()
    dy, z = (torch.randn(4160, N, generator=g).to(BF16).cuda() for _ in range(2))
    big = capi.alloc_linear_backward_workspace(dy, x, w)
    for T in (4160, 4097, 4096, 777, 1):
        got = []
        for ws in (big, capi.alloc_linear_backward_workspace(dy[:T], x[:T], w)):
            dx, dw, db = torch.empty_like(x[:T]), torch.empty_like(w), torch.empty(N, device="cuda")
            ws.fill_(0xFF)
            capi.linear_bf16_backward(dy[:T], x[:T], w, ws, z=z[:T], act="silu", dx=dx, dw=dw, db=db)
            capi.moe_read_device_status(ws)
            got.append((dx, dw, db))
        assert all(torch.equal(a, b) for a, b in zip(*got))


def test_balance():
    E, k = 288, 8
    cfg = capi.SiteConfig(256, 128, 0, E, 0, E, k, 2.5, 7.0)
    g = torch.Generator().manual_seed(1)
    logits = torch.randn(2369, E, generator=g).cuda()
    ids = torch.randint(0, E, (2369, k), generator=g, dtype=torch.int32).cuda()
    big = capi.alloc_balance_workspace(cfg, 2369)
    for T in (2369, 2368, 300, 7):
        got = []
        for ws in (big, capi.alloc_balance_workspace(cfg, T)):
            counts, mean = torch.empty(1, E, dtype=torch.int32, device="cuda"), torch.empty(1, E, device="cuda")
            loss = torch.empty(1, device="cuda")
            ws.fill_(0xFF)
            capi.moe_balance_loss(cfg, logits[:T], ids[:T], 0.1, counts, mean, loss, ws)
            got.append((counts, mean, loss))
        assert all(torch.equal(a, b) for a, b in zip(*got))
        assert int(got[0][0].sum()) == T * k
