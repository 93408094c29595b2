"""Refusals of calls without tokens or sequences: a gradient whose tensor is
empty may have a NULL pointer."""
import ctypes as C

from routed_nvfp4_expert_b200 import capi


def test_nothing_to_differentiate_is_no_error():
    lib = capi.lib()
    cfg = capi.SiteConfig(256, 128, 0, 16, 0, 16, 4, 2.5, 7.0).c()
    off, coef = 0x10000, 0.1                               # never followed: every call here is a no-op or refused

    def router(T, n, dw=None, counts=None, dl=None):
        return lib.moe_router_backward(C.byref(cfg), 0x20000, 0x30000, T, dw, off, n, coef, counts, dl, 0x40000, None)

    assert router(0, 1) == 0 and router(4, 0) == 0 and router(0, 0) == 0
    assert router(4, 1) == 1 and "both NULL" in lib.moe_last_error().decode()
    assert router(0, 1, dl=0x50000) == 1 and "go together" in lib.moe_last_error().decode()

    def linear(T):
        return lib.linear_bf16_backward(0, None, 32, None, 0, None, 64, T, 64, 0x20000, 64, 32, None, 0, None, 0, None,
                                        None, 0, None)

    assert linear(0) == 0
    assert linear(4) == 1 and "all NULL" in lib.moe_last_error().decode()
