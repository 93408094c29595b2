"""Which form a short batch of many sequences takes: a CTA per sequence where a
sequence's rows times experts are few, else rows shared over the grid."""
import pytest
import torch

from graph_launches import launches

pytestmark = pytest.mark.gpu

capi = pytest.importorskip("routed_nvfp4_expert_b200.capi")


@pytest.mark.parametrize("T,E,B,by_sequence", [
    (512, 8, 8, True), (512, 288, 8, True), (513, 288, 64, False), (512, 288, 7, False), (2048, 8, 64, False),
    (512, 1024, 64, False), (144, 1024, 8, True), (144, 1024, 7, False), (145, 1024, 64, False), (128, 288, 1, True),
    (129, 288, 1, False), (36, 1024, 1, True), (128, 1024, 1, False), (128, 1024, 8, True),
])
def test_form(T, E, B, by_sequence):
    k = 4
    cfg = capi.SiteConfig(256, 128, 0, E, 0, E, k, 2.5, 7.0)
    g = torch.Generator().manual_seed(T + E)
    logits = torch.randn(T, E, generator=g).cuda()
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32).cuda()
    off = torch.tensor([T * i // B for i in range(B + 1)], dtype=torch.int32, device="cuda")
    counts, mean = torch.empty(B, E, dtype=torch.int32, device="cuda"), torch.empty(B, E, device="cuda")
    loss, ws = torch.empty(B, device="cuda"), capi.alloc_balance_workspace(cfg, T, B)

    def call():
        capi.moe_balance_loss(cfg, logits, ids, 0.1, counts, mean, loss, ws, seq_offsets=off)

    assert len(launches(call)) == (1 if by_sequence else 2)
    call()
    share = logits.double().sigmoid()
    share = share / share.sum(1, keepdim=True)
    for b in range(B):
        lo, hi = int(off[b]), int(off[b + 1])
        # n positive terms and a row's sum of E, each rounded to fp32 at every step, scores within 16 half steps
        assert ((mean[b].double() - share[lo:hi].mean(0)).abs() <= (hi - lo + 2 * E + 64) * 2.0 ** -24 * share[lo:hi].mean(0)).all()
        assert torch.equal(counts[b].long(), torch.bincount(ids[lo:hi].reshape(-1).long(), minlength=E))
