"""The activations' tails: values and slopes relative to themselves.

Tolerances: z is exact (products of two bf16 numbers, no sum). The activation
and its slope are evaluated within 2^-13 of themselves where the slope has no
zero near (z <= -3), and the result is rounded to bf16 once (2^-8); db of one
token is the unrounded slope times dy."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

capi = pytest.importorskip("routed_nvfp4_expert_b200.capi")

BF16, F64 = torch.bfloat16, torch.float64
LOWEST = {"gelu": -12.5, "gelu_tanh": -9.5, "silu": -80.0}


def _cdf(act, z):
    """y / z and its derivative."""
    if act == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)), torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        s = torch.sigmoid(c * (z + 0.044715 * z ** 3))
        return s, s * torch.sigmoid(-c * (z + 0.044715 * z ** 3)) * c * (1 + 3 * 0.044715 * z * z)
    return torch.sigmoid(z), torch.sigmoid(z) * torch.sigmoid(-z)


def _operands(act, T, N):
    x = torch.linspace(1.0, 2.0, T).to(BF16).cuda()[:, None]
    w = torch.linspace(LOWEST[act] / 2, -0.25, N).to(BF16).cuda()[:, None]
    return x, w


@pytest.mark.parametrize("act", LOWEST)
@pytest.mark.parametrize("T,N", [(3, 1000), (1500, 2000)])
def test_values_in_the_tail(act, T, N):
    x, w = _operands(act, T, N)
    y = torch.empty(T, N, dtype=BF16, device="cuda")
    capi.linear_bf16(x, w, y, capi.alloc_linear_workspace(x, w), act=act)
    z = x.to(F64) @ w.to(F64).T
    ref = z * _cdf(act, z)[0]
    assert float(ref.abs().min()) > 0
    err = ((y.to(F64) - ref) / ref).abs()
    assert float(err.max()) <= 2.0 ** -8 + 2.0 ** -13, (float(err.max()), float(z.reshape(-1)[err.argmax()]))


@pytest.mark.parametrize("act", LOWEST)
def test_slopes_in_the_tail(act):
    N = 3000
    z = torch.linspace(LOWEST[act], -3.0, N).to(BF16).cuda()[None]
    x, w = torch.ones(1, 8, dtype=BF16, device="cuda"), torch.ones(N, 8, dtype=BF16, device="cuda")
    dy = torch.full((1, N), 0.5, dtype=BF16, device="cuda")
    db = torch.empty(N, device="cuda")
    capi.linear_bf16_backward(dy, x, w, capi.alloc_linear_backward_workspace(dy, x, w), z=z, act=act, db=db)
    Z = z[0].to(F64)
    value, slope = _cdf(act, Z)
    ref = 0.5 * (value + Z * slope)
    assert float(((db.to(F64) - ref) / ref).abs().max()) <= 2.0 ** -13


@pytest.mark.parametrize("act", ["relu", *LOWEST])
def test_far_out(act):
    """Finite z of any size: the value is z or 0 and the slope 1 or 0, never NaN."""
    far = torch.tensor([1e3, 1e6, 1e10, 1e19, 1e20, 1e30, 3e38]).to(BF16)
    z = torch.cat([far, -far]).cuda()[None]
    N = z.shape[1]
    x, w = torch.ones(1, 8, dtype=BF16, device="cuda"), torch.ones(N, 8, dtype=BF16, device="cuda")
    db = torch.empty(N, device="cuda")
    capi.linear_bf16_backward(torch.ones_like(z), x, w, capi.alloc_linear_backward_workspace(z, x, w), z=z, act=act, db=db)
    want = torch.cat([torch.ones(len(far)), torch.zeros(len(far))]).cuda()
    assert torch.equal(db, want), db
    x, w = torch.ones(1, 1, dtype=BF16, device="cuda"), z.T.contiguous()
    y = torch.empty(1, N, dtype=BF16, device="cuda")
    capi.linear_bf16(x, w, y, capi.alloc_linear_workspace(x, w), act=act)
    assert torch.equal(y, torch.where(z > 0, z, torch.zeros_like(z))), y
