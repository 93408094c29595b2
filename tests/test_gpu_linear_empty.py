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
