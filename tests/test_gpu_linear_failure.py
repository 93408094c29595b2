"""The bounded-wait failure path of the BF16 linear layer, made to happen
without a fault: with a zero limit the first wait for a copy still in flight
runs out. The kernel must report MOE_ERR_DEVICE_TIMEOUT in its status word,
wait with the default limit for what it has in flight, return, and leave the
device usable: the same call with the default limit gives the bits it gave
before."""
import pytest
import torch

pytestmark = pytest.mark.gpu

capi = pytest.importorskip("routed_nvfp4_expert_b200.capi")

BF16 = torch.bfloat16


def _fails_and_recovers(call, ws, outs):
    call()
    capi.moe_read_device_status(ws)
    want = [t.clone() for t in outs]
    for _ in range(3):
        capi.moe_set_wait_limit(0)
        try:
            call()
            with pytest.raises(capi.MoEError) as e:
                capi.moe_read_device_status(ws)
            assert e.value.status == 5           # MOE_ERR_DEVICE_TIMEOUT
        finally:
            capi.moe_set_wait_limit(-1)
        call()
        capi.moe_read_device_status(ws)
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def _rand(g, *shape):
    return torch.randn(*shape, generator=g).to(BF16).cuda()


# parts sent between the CTAs of a cluster (up to 32 columns) or read from it; no cluster
@pytest.mark.parametrize("T,K,N", [(1, 4096, 4096), (16, 8192, 1000), (128, 4096, 4096), (200, 2048, 300), (1, 64, 40000)])
def test_few_tokens(T, K, N):
    g = torch.Generator().manual_seed(T)
    x, w = _rand(g, T, K), _rand(g, N, K)
    y = torch.empty(T, N, dtype=BF16, device="cuda")
    ws = capi.alloc_linear_workspace(x, w)
    _fails_and_recovers(lambda: capi.linear_bf16(x, w, y, ws, act="silu"), ws, [y])


def test_few_tokens_backward():
    T, K, N = 200, 2048, 300
    g = torch.Generator().manual_seed(3)
    x, w, dy, z = _rand(g, T, K), _rand(g, N, K), _rand(g, T, N), _rand(g, T, N)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(N, device="cuda")
    ws = capi.alloc_linear_backward_workspace(dy, x, w)
    _fails_and_recovers(lambda: capi.linear_bf16_backward(dy, x, w, ws, z=z, act="gelu", dx=dx, dw=dw, db=db), ws,
                        [dx, dw, db])


@pytest.mark.parametrize("T,K,N", [(2049, 4096, 1280), (600, 64, 6000), (4096, 12288, 700), (900, 130, 4097)])
def test_many_tokens(T, K, N):
    g = torch.Generator().manual_seed(T)
    x, w, r = _rand(g, T, K), _rand(g, N, K), _rand(g, T, N)
    y, z = torch.empty(T, N, dtype=BF16, device="cuda"), torch.empty(T, N, dtype=BF16, device="cuda")
    ws = capi.alloc_linear_workspace(x, w)
    _fails_and_recovers(lambda: capi.linear_bf16(x, w, y, ws, act="gelu", residual=r, z=z), ws, [y, z])


@pytest.mark.parametrize("T,K,N,act", [(777, 1000, 515, "silu"), (2048, 1024, 2048, "none"), (64, 4096, 1024, "gelu")])
def test_many_tokens_backward(T, K, N, act):
    g = torch.Generator().manual_seed(T)
    x, w, dy, z = _rand(g, T, K), _rand(g, N, K), _rand(g, T, N), _rand(g, T, N)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ws = capi.alloc_linear_backward_workspace(dy, x, w)
    _fails_and_recovers(lambda: capi.linear_bf16_backward(dy, x, w, ws, z=z if act != "none" else None, act=act, dx=dx,
                                                          dw=dw), ws, [dx, dw])


@pytest.mark.parametrize("limit", [300, 2000, 20000])
def test_waits_that_run_out_somewhere(limit):
    """Limits near the copies' latency (ns): the producers and the issuer of a
    pair stop at different steps, in some runs or in all. Whatever the status,
    the calls end and the next one is right."""
    T, K, N = 2049, 4096, 1280
    g = torch.Generator().manual_seed(limit)
    x, w = _rand(g, T, K), _rand(g, N, K)
    y = torch.empty(T, N, dtype=BF16, device="cuda")
    ws = capi.alloc_linear_workspace(x, w)
    capi.linear_bf16(x, w, y, ws)
    want = y.clone()
    for _ in range(5):
        capi.moe_set_wait_limit(limit)
        try:
            capi.linear_bf16(x, w, y, ws)
            try:
                capi.moe_read_device_status(ws)
                assert torch.equal(y, want)
            except capi.MoEError as e:
                assert e.status == 5
        finally:
            capi.moe_set_wait_limit(-1)
        capi.linear_bf16(x, w, y, ws)
        capi.moe_read_device_status(ws)
        assert torch.equal(y, want)
