"""Calls without tokens: what they write, and what they accept."""
import pytest
import torch

pytestmark = pytest.mark.gpu

capi = pytest.importorskip("routed_nvfp4_expert_b200.capi")

BF16 = torch.bfloat16


def _operands(T=0, K=64, N=32):
    return (torch.ones(T, K, dtype=BF16, device="cuda"), torch.ones(N, K, dtype=BF16, device="cuda"),
            torch.ones(T, N, dtype=BF16, device="cuda"))


def test_the_status_word_is_cleared():
    """A fresh workspace holds anything; the status read after the call is the call's."""
    x, w, y = _operands()
    ws = capi.alloc_linear_workspace(x, w).fill_(0xFF)
    capi.linear_bf16(x, w, y, ws)
    capi.moe_read_device_status(ws)
    db = torch.full((32,), 5.0, device="cuda")
    ws = capi.alloc_linear_backward_workspace(y, x, w).fill_(0xFF)
    capi.linear_bf16_backward(y, x, w, ws, db=db)
    capi.moe_read_device_status(ws)
    assert not db.any()


def test_the_gradient_of_no_tokens_alone():
    """An empty dx, or empty routing-weight gradients, as the only gradient wanted: their pointers may be NULL."""
    x, w, y = _operands()
    ws = capi.alloc_linear_backward_workspace(y, x, w)
    dx = torch.empty_like(x)
    capi.linear_bf16_backward(y, x, w, ws, dx=dx)
    cfg = capi.SiteConfig(256, 128, 0, 16, 0, 16, 2, 2.5, 7.0)
    logits, ids = torch.empty(0, 16, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda")
    capi.moe_router_backward(cfg, logits, ids, torch.empty_like(logits), d_weights=torch.empty(0, 2, device="cuda"))
    # no sequences: an empty d_loss
    logits, ids = torch.zeros(4, 16, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    out = torch.full_like(logits, 3.0)
    capi.moe_router_backward(cfg, logits, ids, out, counts=torch.empty(0, 16, dtype=torch.int32, device="cuda"),
                             d_loss=torch.empty(0, device="cuda"), seq_offsets=torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert (out == 3.0).all()


def test_dw_of_a_wide_pitch_is_cleared():
    """Rows 2^31 bytes and more apart."""
    x, w, y = _operands(N=2)
    pitch = (1 << 30) + 8
    buf = torch.full((pitch + 64,), 7.0, dtype=BF16, device="cuda")
    dw = torch.as_strided(buf, (2, 64), (pitch, 1))
    capi.linear_bf16_backward(y, x, w, capi.alloc_linear_backward_workspace(y, x, w), dw=dw)
    assert not dw.any() and float(buf[64]) == 7.0 and float(buf[pitch - 1]) == 7.0
