"""The bounded-wait failure path of the FP4 pair GEMM, made to happen without a
fault through moe_set_wait_limit: the call reports a timeout, ends, and the same
call with the default limit gives the bits that it gave before."""
import pytest
import torch

from helpers import site_inputs, workload
from test_gpu_prefill import _prefill

pytestmark = pytest.mark.gpu

capi = pytest.importorskip("routed_nvfp4_expert_b200.capi")


@pytest.mark.parametrize("limit", [0, 300, 2000, 20000])
@pytest.mark.parametrize("T", [300, 1500])
def test_waits_that_run_out(T, limit):
    wl = workload("tiny_t4", T)
    cfg, site, y, ws, v = _prefill(wl, site_inputs(wl))
    P = capi.moe_padded_rows(cfg, T)
    view = capi.view_tensor
    xq, xsf = view(v.xq_codes, (P, wl.H // 2), torch.uint8), view(v.xq_sf, (P * wl.H // 16,), torch.uint8)
    hq, hsf = view(v.hq_codes, (P, wl.I // 2), torch.uint8), view(v.hq_sf, (P * wl.I // 16,), torch.uint8)
    xts, hts = view(v.xq_scale, (P,), torch.float32), view(v.hq_scale, (P,), torch.float32)
    wts = view(v.weights, (T * wl.k,), torch.float32)
    ws2 = capi.alloc_workspace(cfg, T, capi.PATH_PREFILL).zero_()
    h, r = torch.zeros((P, wl.I), dtype=torch.bfloat16, device="cuda"), torch.zeros((P, wl.H), device="cuda")
    calls = [(lambda: capi.nvfp4_grouped_gemm(cfg, capi.PROJ_GATE_UP, xq, xsf, xts, T, v.plan, wts, site, h, ws2), h),
             (lambda: capi.nvfp4_grouped_gemm(cfg, capi.PROJ_DOWN, hq, hsf, hts, T, v.plan, wts, site, r, ws2), r)]
    for call, out in calls:
        call()
        capi.moe_read_device_status(ws2)
        want = out.clone()
        for _ in range(4):
            capi.moe_set_wait_limit(limit)
            try:
                call()
                try:
                    capi.moe_read_device_status(ws2)
                    assert limit > 0 and torch.equal(out, want)
                except capi.MoEError as e:
                    assert e.status == 5             # MOE_ERR_DEVICE_TIMEOUT
            finally:
                capi.moe_set_wait_limit(-1)
            call()
            capi.moe_read_device_status(ws2)
            assert torch.equal(out, want)
