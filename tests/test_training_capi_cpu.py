"""Refusals and sizes of the balance and linear entry points, before any launch."""
import ctypes as C

import pytest
import torch

from routed_nvfp4_expert_b200 import capi

P = [0x10000 * (i + 1) for i in range(12)]     # pointers that are never followed: every call here is refused or a no-op
WS = 0x4000000


def _cfg(**kw):
    base = dict(hidden=256, intermediate=128, shared_intermediate=0, num_experts=16, local_begin=0, local_end=16,
                top_k=4, routed_scaling_factor=2.5, swiglu_limit=7.0)
    base.update(kw)
    return capi.SiteConfig(**base).c()


def _err():
    return capi.lib().moe_last_error().decode()


def test_balance_sizes_and_refusals():
    lib, cfg = capi.lib(), _cfg()
    size = lib.moe_balance_workspace_size
    assert size(C.byref(cfg), 0, 1) == size(C.byref(cfg), 64, 100) == 256
    need = size(C.byref(cfg), 10000, 3)
    assert need >= (148 - 8 + 3) * 16 * 8
    assert size(C.byref(cfg), -1, 1) == 0 and size(C.byref(cfg), 4, -1) == 0
    bad = _cfg(top_k=17)
    assert size(C.byref(bad), 4, 1) == 0

    def call(T=10000, off=P[2], n=3, coef=0.1, logits=P[0], ids=P[1], counts=P[3], mean=P[4], loss=P[5], ws=WS, nb=need):
        return lib.moe_balance_loss(C.byref(cfg), logits, ids, T, off, n, coef, counts, mean, loss, ws, nb, None)

    for kw, code, frag in [
        (dict(T=-1), 1, "T="), (dict(n=-1), 1, "num_seqs"), (dict(off=None), 1, "num_seqs"), (dict(off=P[2] + 4), 1, "seq_offsets"),
        (dict(n=1 << 21), 2, "num_seqs"), (dict(coef=float("nan")), 1, "coef"), (dict(coef=float("inf")), 1, "coef"),
        (dict(logits=None), 1, "logits"), (dict(ids=P[1] + 8), 1, "ids"), (dict(counts=None), 1, "counts"),
        (dict(mean=P[4] + 1), 1, "mean_scores"), (dict(loss=None), 1, "loss"), (dict(ws=None), 3, "workspace"),
        (dict(ws=WS + 16), 3, "workspace"), (dict(nb=need - 1), 3, "workspace"),
    ]:
        assert call(**kw) == code and frag in _err(), kw
    assert lib.moe_balance_loss(C.byref(cfg), None, None, 0, P[2], 0, 0.1, None, None, None, None, 0, None) == 0


def test_router_backward_refusals():
    lib, cfg = capi.lib(), _cfg()

    def call(T=8, dw=P[2], off=None, n=1, coef=0.1, counts=P[3], dl=P[4], out=P[5], logits=P[0], ids=P[1]):
        return lib.moe_router_backward(C.byref(cfg), logits, ids, T, dw, off, n, coef, counts, dl, out, None)

    for kw, frag in [(dict(dw=None, counts=None, dl=None), "both NULL"), (dict(counts=None), "go together"),
                     (dict(dl=None), "go together"), (dict(out=None), "d_logits"), (dict(logits=P[0] + 4), "logits"),
                     (dict(ids=None), "ids"), (dict(n=2), "num_seqs"), (dict(T=-3), "T="), (dict(dw=P[2] + 2), "d_weights"),
                     (dict(coef=float("nan")), "coef")]:
        assert call(**kw) == 1 and frag in _err(), kw
    assert call(T=0) == 0


def test_linear_sizes_and_refusals():
    lib = capi.lib()
    size, bsize = lib.linear_workspace_size, lib.linear_backward_workspace_size
    assert size(4, 64, 32, 64, 64) == 256
    assert size(4, 63, 32, 63, 64) == 256 + 512                    # x copied to rows of 64
    assert size(1, 63, 32, 63, 64) == 256                          # one row needs none
    assert size(4, 63, 32, 64, 63) == 256 + 32 * 64 * 2
    assert bsize(4, 64, 30, 64, 64) >= 256 + 4 * 32 * 2 + 30 * 4
    for a in [(-1, 64, 32, 64, 64), (4, 0, 32, 64, 64), (4, 64, 0, 64, 64), (4, 64, 32, 63, 64), (4, 64, 32, 64, 63),
              (1 << 24, 64, 32, 64, 64), (4, 64, 32, 1 << 40, 64)]:
        assert size(*a) == 0 and bsize(*a) == 0, a

    def fwd(act=1, x=P[0], ldx=64, T=4, K=64, w=P[1], ldw=64, N=32, b=P[2], r=P[3], ldr=32, z=P[4], ldz=32, y=P[5],
            ldy=32, ws=WS, nb=256):
        return lib.linear_bf16(act, x, ldx, T, K, w, ldw, N, b, r, ldr, z, ldz, y, ldy, ws, nb, None)

    for kw, code, frag in [
        (dict(act=5), 1, "activation"), (dict(act=-1), 1, "activation"), (dict(T=-1), 1, "T="), (dict(K=0), 1, "K="),
        (dict(x=None), 1, "x"), (dict(x=P[0] + 2), 1, "x"), (dict(w=None), 1, "w"), (dict(y=None), 1, "y"),
        (dict(b=P[2] + 4), 1, "bias"), (dict(r=P[3] + 4), 1, "residual"), (dict(z=P[4] + 4), 1, "z_out"),
        (dict(ldx=63), 1, "ldx"), (dict(ldw=10), 1, "ldw"), (dict(ldr=31), 1, "ldr"), (dict(ldz=0), 1, "ldz"),
        (dict(ldy=31), 1, "ldy"), (dict(ldy=1 << 39), 2, "ldy"), (dict(ws=None), 3, "workspace"),
        (dict(ws=WS + 64), 3, "workspace"), (dict(nb=255), 3, "workspace"), (dict(ldx=65), 3, "workspace"),
    ]:
        assert fwd(**kw) == code and frag in _err(), kw
    assert fwd(T=0, x=None, ws=None, nb=0) == 0

    need = bsize(4, 64, 32, 64, 64)

    def bwd(act=1, dy=P[0], lddy=32, z=P[1], ldz=32, x=P[2], ldx=64, T=4, K=64, w=P[3], ldw=64, N=32, dx=P[4], lddx=64,
            dw=P[5], lddw=64, db=P[6], ws=WS, nb=need):
        return lib.linear_bf16_backward(act, dy, lddy, z, ldz, x, ldx, T, K, w, ldw, N, dx, lddx, dw, lddw, db, ws, nb, None)

    for kw, code, frag in [
        (dict(dx=None, dw=None, db=None), 1, "all NULL"), (dict(dy=None), 1, "dy"), (dict(z=None), 1, "z"),
        (dict(x=None), 1, "x"), (dict(w=None), 1, "w"), (dict(lddy=3), 1, "lddy"), (dict(ldz=3), 1, "ldz"),
        (dict(lddx=63), 1, "lddx"), (dict(lddw=63), 1, "lddw"), (dict(db=P[6] + 4), 1, "db"), (dict(dx=P[4] + 8), 1, "dx"),
        (dict(nb=need - 1), 3, "workspace"), (dict(ws=None), 3, "workspace"), (dict(act=9), 1, "activation"),
    ]:
        assert bwd(**kw) == code and frag in _err(), kw
    assert bwd(T=0, dw=None, db=None, dy=None, ws=None, nb=0) == 0


def test_the_binding_checks_its_tensors():
    cfg = capi.SiteConfig(256, 128, 0, 16, 0, 16, 4, 2.5, 7.0)
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(32, 64, dtype=torch.bfloat16)
    y, ws = torch.zeros(4, 32, dtype=torch.bfloat16), torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        capi.linear_bf16(x, w, y, ws)
    with pytest.raises(ValueError, match="bfloat16"):
        capi.linear_bf16(x.float(), w, y, ws)
    with pytest.raises(ValueError, match="logits"):
        capi.moe_balance_loss(cfg, torch.zeros(4, 15), torch.zeros(4, 4, dtype=torch.int32), 0.1,
                              torch.zeros(1, 16, dtype=torch.int32), torch.zeros(1, 16), torch.zeros(1), ws)
    with pytest.raises(ValueError, match="activation"):
        capi._activation("swish")
