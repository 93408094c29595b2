"""A workspace allocated for the largest batch serves every smaller one: the
sizes never decrease with the number of tokens, features or sequences."""
import ctypes as C

import pytest

from routed_nvfp4_expert_b200 import capi

TOKENS = sorted(set(range(0, 5000)) | {t + d for t in range(4096, 140000, 2048) for d in range(-2, 35)})


def _never_decreases(sizes):
    last = 0
    for at, n in sizes:
        assert n >= max(last, 1), at
        last = n


@pytest.mark.parametrize("E,k", [(8, 2), (288, 8), (1024, 16)])
def test_balance(E, k):
    cfg = capi.SiteConfig(256, 128, 0, E, 0, E, k, 2.5, 7.0).c()
    size = capi.lib().moe_balance_workspace_size
    for B in (1, 7, 300):
        _never_decreases((T, size(C.byref(cfg), T, B)) for T in TOKENS)
    for T in (1, 128, 129, 2048, 2369, 50000):
        _never_decreases((B, size(C.byref(cfg), T, B)) for B in range(0, 3000, 7))


@pytest.mark.parametrize("K,N,ldx,ldw", [(64, 1024, 64, 64), (256, 12288, 256, 256), (1003, 515, 1003, 1003), (1, 1, 1, 1),
                                         (640, 4691, 648, 643)])
def test_linear(K, N, ldx, ldw):
    lib = capi.lib()
    for size in (lib.linear_workspace_size, lib.linear_backward_workspace_size):
        _never_decreases((T, size(T, K, N, ldx, ldw)) for T in TOKENS)
        for T in (1, 33, 4097, 20000):
            _never_decreases((n, size(T, K, n, ldx, ldw)) for n in range(1, 13000, 37))
