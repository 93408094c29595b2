"""The BF16 linear layer with its fused epilogue and its gradients
(linear_bf16, linear_bf16_backward) against plain formulas in 64 bits.

Tolerances. Products of bf16 are exact in fp32; the tensor core's accumulation
may truncate: each of the n / 16 steps and of the few joins is off by at most
2^-22 of the sum of magnitudes, which gives ACC(n) = (n / 16 + 16) 2^-22. The
activation and its slope (bounded by 1.13) are evaluated in fp32 to a few
steps: 2^-20 of |z| + 1. A result rounded to bf16 moves by at most 2^-8 of
itself. dz enters its products rounded to bf16 (2^-8 of each element)."""
import math
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

capi = pytest.importorskip("routed_nvfp4_expert_b200.capi")

BF16, F64 = torch.bfloat16, torch.float64
HALF = 2.0 ** -8
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def _acc(n):
    return (n / 16 + 16) * 2.0 ** -22


def _act(name, z):
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z * torch.sigmoid(z) if name == "silu" else z


def _slope(name, z):
    if name == "none":
        return torch.ones_like(z)
    zz = z.clone().requires_grad_()
    (g,) = torch.autograd.grad(_act(name, zz).sum(), zz)
    return g


def _rand(g, *shape, scale=1.0, pitch=0):
    """bf16 rows in a buffer of the given pitch, whose other columns hold a marker."""
    t = torch.full((shape[0], max(pitch, shape[1])), 77.0, dtype=BF16, device="cuda")
    v = t[:, :shape[1]]
    v.copy_((torch.randn(*shape, generator=g) * scale).to(BF16))
    return v


def _tail_untouched(v, rows, cols):
    full = torch.as_strided(v, (rows, v.stride(0)), (v.stride(0), 1), v.storage_offset())
    return bool((full[:, cols:] == 77.0).all())


def _forward_case(T, K, N, act, bias, residual, keep, pitches, seed=0):
    g = torch.Generator().manual_seed(seed + T + 7 * K + 13 * N)
    px, pw, po = (0 if pitches is None else pitches[i] for i in range(3))
    x, w = _rand(g, T, K, pitch=px and K + px), _rand(g, N, K, scale=K ** -0.5, pitch=pw and K + pw)
    b = (torch.randn(N, generator=g)).to(BF16).cuda() if bias else None
    r = _rand(g, T, N, pitch=po and N + po) if residual else None
    y, z = _rand(g, T, N, pitch=po and N + po), (_rand(g, T, N, pitch=po and N + po) if keep else None)
    return x, w, b, r, y, z


def _check_forward(x, w, b, r, y, z, act):
    (T, K), N = x.shape, w.shape[0]
    X, W = x.to(F64), w.to(F64)
    Z, A = X @ W.T, X.abs() @ W.abs().T
    if b is not None:
        Z, A = Z + b.to(F64), A + b.to(F64).abs()
    Y = _act(act, Z)
    off = 1.2 * _acc(K) * A + 2.0 ** -20 * (Z.abs() + 1e-6)
    if r is not None:
        Y = Y + r.to(F64)
        off = off + 2.0 ** -22 * r.to(F64).abs()
    d = (y.to(F64) - Y).abs()
    assert (d <= HALF * Y.abs() + 1.01 * off).all(), float((d - HALF * Y.abs()).max())
    if z is not None:
        assert ((z.to(F64) - Z).abs() <= HALF * Z.abs() + 1.01 * off).all()


SHAPES = [
    # T, K, N, act, bias, residual, keep z, extra pitch of (x, w, outputs)
    (1, 64, 128, "none", True, True, False, None),
    (1, 4096, 1024, "silu", True, False, True, None),
    (1, 1, 1, "relu", True, True, True, None),
    (2, 1003, 517, "gelu", True, True, True, None),
    (3, 7, 130, "gelu_tanh", False, False, False, (1, 1, 1)),
    (16, 4096, 4096, "none", False, True, False, (8, 16, 8)),
    (17, 520, 200, "gelu", True, False, True, (3, 0, 5)),
    (33, 100, 1000, "silu", True, True, False, (0, 5, 0)),
    (64, 256, 300, "relu", True, True, True, None),
    (65, 64, 64, "gelu", False, False, False, None),
    (130, 1003, 1537, "gelu", True, True, True, None),
    (200, 2048, 512, "silu", True, True, False, None),
    (256, 512, 4096, "gelu_tanh", True, False, True, None),
    (257, 72, 1000, "relu", True, True, False, (8, 8, 4)),
    (511, 1024, 2048, "none", True, True, False, None),
    (1000, 640, 1111, "gelu", True, True, True, None),
    (2049, 4096, 1280, "silu", True, True, True, None),
    (5000, 64, 129, "none", False, True, False, None),
    (4096, 1024, 4096, "gelu", True, False, True, (16, 8, 24)),
    # long reductions, a padded pitch under an odd length
    (600, 12288, 1024, "gelu", True, True, True, None),
    (1300, 6000, 1101, "silu", True, True, True, (0, 0, 3)),
    (300, 4096, 6000, "none", False, True, False, None),
]


@pytest.mark.parametrize("T,K,N,act,bias,residual,keep,pitches", SHAPES)
def test_forward_matches_the_formula(T, K, N, act, bias, residual, keep, pitches):
    x, w, b, r, y, z = _forward_case(T, K, N, act, bias, residual, keep, pitches)
    ws = capi.alloc_linear_workspace(x, w)
    ws.fill_(0xFF)                                   # its contents need no initialisation
    capi.linear_bf16(x, w, y, ws, bias=b, residual=r, act=act, z=z)
    capi.moe_read_device_status(ws)
    _check_forward(x, w, b, r, y, z, act)
    assert _tail_untouched(y, T, N) and (z is None or _tail_untouched(z, T, N))


@pytest.mark.parametrize("act", ACTS)
def test_every_activation_both_ways(act):
    T, K, N = 70, 136, 264
    x, w, b, r, y, z = _forward_case(T, K, N, act, True, True, True, None, seed=3)
    x.mul_(4)                                        # pre-activations out into the tails
    ws = capi.alloc_linear_workspace(x, w)
    capi.linear_bf16(x, w, y, ws, bias=b, residual=r, act=act, z=z)
    _check_forward(x, w, b, r, y, z, act)
    _check_backward(T, K, N, act, x, w, z, torch.Generator().manual_seed(1))


@pytest.mark.parametrize("T,N", [(5, 100), (300, 257), (1500, 1024)])
def test_residual_in_place(T, N):
    x, w, b, r, y, _ = _forward_case(T, 256, N, "silu", True, True, False, None)
    ws = capi.alloc_linear_workspace(x, w)
    capi.linear_bf16(x, w, y, ws, bias=b, residual=r, act="silu")
    capi.linear_bf16(x, w, r, ws, bias=b, residual=r, act="silu")
    assert torch.equal(r, y)


@pytest.mark.parametrize("T", [4, 600])
def test_infinities_and_nan_stay_in_their_rows_and_columns(T):
    K, N = 96, 144
    x, w, b, _, y, _ = _forward_case(T, K, N, "none", True, False, False, None)
    x[1, 5] = float("nan")
    x[2, 95] = float("inf")
    w[7, 0] = float("nan")
    ws = capi.alloc_linear_workspace(x, w)
    capi.linear_bf16(x, w, y, ws, bias=b)
    bad = torch.zeros(T, N, dtype=torch.bool, device="cuda")
    bad[1], bad[:, 7] = True, True
    assert torch.isnan(y[bad]).all()
    inf = torch.isinf(y)
    assert bool((inf[2] | bad[2]).all())
    bad[2] = True
    assert torch.isfinite(y[~bad]).all()


def _check_backward(T, K, N, act, x, w, z, g, want=("dx", "dw", "db"), pitches=None):
    p = pitches or (0, 0, 0)
    dy = _rand(g, T, N, scale=0.1, pitch=p[0] and N + p[0])
    dx = _rand(g, T, K, pitch=p[1] and K + p[1]) if "dx" in want else None
    dw = _rand(g, N, K, pitch=p[2] and K + p[2]) if "dw" in want else None
    db = torch.full((N,), float("nan"), device="cuda") if "db" in want else None
    ws = capi.alloc_linear_backward_workspace(dy, x, w)
    ws.fill_(0xFF)
    capi.linear_bf16_backward(dy, x, w, ws, z=z if act != "none" else None, act=act, dx=dx, dw=dw, db=db)
    capi.moe_read_device_status(ws)
    X, W, G = x.to(F64), w.to(F64), dy.to(F64)
    dz, e = G, torch.zeros_like(G)                   # e: the slope's evaluation in fp32
    if act != "none":
        Z = z.to(F64)
        dz, e = G * _slope(act, Z), 2.0 ** -20 * G.abs() * (1 + Z.abs())
    for got, a, b, ea, n in ((dx, dz, W, e, N), (dw, dz.T, X, e.T, T)):
        if got is None:
            continue
        ref = a @ b
        rounded = 0.0 if act == "none" else HALF     # dy itself is the operand without an activation
        tol = HALF * ref.abs() + 1.01 * ((rounded + _acc(n)) * (a.abs() @ b.abs()) + ea @ b.abs()) + 1e-30
        assert ((got.to(F64) - ref).abs() <= tol).all(), float(((got.to(F64) - ref).abs() - tol).max())
    if db is not None:
        tol = 1.01 * ((T + 8) * 2.0 ** -24 * dz.abs().sum(0) + e.sum(0)) + 1e-30
        assert ((db.to(F64) - dz.sum(0)).abs() <= tol).all()
    for v, rows in ((dx, T), (dw, N)):
        assert v is None or _tail_untouched(v, rows, K)
    return dy, dx, dw, db


@pytest.mark.parametrize("T,K,N,act,want,pitches", [
    (1, 64, 128, "none", ("dx", "dw", "db"), None),
    (1, 1, 1, "relu", ("dx", "dw", "db"), None),
    (2, 515, 1003, "gelu", ("dx", "dw", "db"), None),
    (3, 130, 7, "silu", ("dx", "dw", "db"), (1, 3, 5)),
    (40, 4096, 512, "none", ("dx",), None),
    (64, 256, 512, "relu", ("dx", "dw", "db"), None),
    (65, 200, 1000, "gelu_tanh", ("dw",), (0, 0, 8)),
    (100, 96, 33, "none", ("dx", "dw", "db"), None),
    (129, 1000, 777, "silu", ("db",), None),
    (200, 72, 136, "gelu", ("dx", "db"), (8, 8, 0)),
    (300, 512, 260, "none", ("dw", "db"), None),
    (777, 1000, 515, "silu", ("dx", "dw", "db"), None),
    (2048, 1024, 1536, "gelu", ("dx", "dw", "db"), None),
    (1025, 2048, 512, "none", ("dx", "dw", "db"), (16, 8, 8)),
    (6000, 64, 128, "relu", ("dx", "dw", "db"), None),
    (2500, 2000, 1100, "gelu", ("dx", "dw", "db"), None),
    (1200, 4100, 2000, "none", ("dx", "dw"), None),
    (1300, 2050, 4500, "silu", ("dx",), (3, 5, 0)),
])
def test_backward_matches_the_formula(T, K, N, act, want, pitches):
    g = torch.Generator().manual_seed(T + K + N)
    x, w = _rand(g, T, K), _rand(g, N, K, scale=K ** -0.5)
    z = _rand(g, T, N, scale=1.5)
    _check_backward(T, K, N, act, x, w, z, g, want, pitches)


def _poisoned(t, pitch):
    """The same rows at this pitch, NaN between them; the buffer ends with the last row's last element."""
    rows, cols = t.shape
    buf = torch.full(((rows - 1) * pitch + cols,), float("nan"), dtype=BF16, device="cuda")
    v = torch.as_strided(buf, (rows, cols), (pitch, 1))
    v.copy_(t)
    return v


@pytest.mark.parametrize("extra", range(8))
@pytest.mark.parametrize("T,K,N", [(45, 203, 331), (1400, 264, 1090)])
def test_rows_on_every_element_boundary(T, K, N, extra):
    """Pitches of every residue mod 8, which put rows on every 2-byte offset of
    a 16-byte piece, through the copies, the dz pass and the epilogues of both
    kernels; nothing between the rows enters a result or is written."""
    g = torch.Generator().manual_seed(T + extra)
    x = _poisoned(_rand(g, T, K), K + extra)
    w = _poisoned(_rand(g, N, K, scale=K ** -0.5), K + (extra + 3) % 8)
    b = torch.randn(N, generator=g).to(BF16).cuda()
    r = _poisoned(_rand(g, T, N), N + (extra + 5) % 8)
    y, zo = _rand(g, T, N, pitch=N + 1 + extra), _rand(g, T, N, pitch=N + 1 + (extra + 2) % 8)
    ws = capi.alloc_linear_workspace(x, w)
    ws.fill_(0xFF)
    capi.linear_bf16(x, w, y, ws, bias=b, residual=r, act="gelu", z=zo)
    capi.moe_read_device_status(ws)
    _check_forward(x, w, b, r, y, zo, "gelu")
    assert _tail_untouched(y, T, N) and _tail_untouched(zo, T, N)
    z = _poisoned(_rand(g, T, N), N + (extra + 1) % 8)
    _check_backward(T, K, N, "silu", x, w, z, g, pitches=(1 + extra, 1 + (extra + 2) % 8, 1 + (extra + 5) % 8))


@pytest.mark.parametrize("T,K,N,act", [
    (1, 1472, 5760, "silu"), (1, 544, 5936, "none"), (16, 842, 5409, "gelu_tanh"), (275, 326, 2036, "none"),
    (275, 328, 11040, "gelu"), (9706, 1344, 128, "relu"), (2, 4627, 2091, "silu"), (48, 1632, 2048, "gelu"),
])
def test_reductions_of_very_different_lengths(T, K, N, act):
    """Few tokens or few features: dx and dW in launches of their own or sharing
    one, and db joined by few CTAs."""
    g = torch.Generator().manual_seed(T + K + N)
    x, w = _rand(g, T, K), _rand(g, N, K, scale=K ** -0.5)
    _check_backward(T, K, N, act, x, w, _rand(g, T, N, scale=1.5), g)


@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_gradients_match_differences(act):
    """Directional differences of sum(dy * y) in 64 bits, through the forward's own kept z."""
    T, K, N = 24, 40, 56
    g = torch.Generator().manual_seed(9)
    x, w, b = _rand(g, T, K), _rand(g, N, K, scale=K ** -0.5), torch.randn(N, generator=g).to(BF16).cuda()
    y, z = torch.empty(T, N, dtype=BF16, device="cuda"), torch.empty(T, N, dtype=BF16, device="cuda")
    ws = capi.alloc_linear_workspace(x, w)
    capi.linear_bf16(x, w, y, ws, bias=b, act=act, z=z)
    dy, dx, dw, db = _check_backward(T, K, N, act, x, w, z, g)
    G = dy.to(F64)

    def f(X, W, B):
        return float((G * _act(act, X @ W.T + B)).sum())

    X, W, B = x.to(F64), w.to(F64), b.to(F64)
    # z was rounded (2^-8 of itself, slope's derivative at most 1.1), dz and the results too (2^-8 each)
    e = G.abs() * (2 * HALF * 1.13 + 1.1 * HALF * z.to(F64).abs()) + 1e-6
    h = 1e-4
    for i, (got, mag) in enumerate(((dx, e @ W.abs()), (dw, e.T @ X.abs()), (db, e.sum(0)))):
        v = torch.randn(got.shape, generator=torch.Generator().manual_seed(i), dtype=F64).cuda()
        hi, lo = [X, W, B], [X, W, B]
        hi[i], lo[i] = hi[i] + h * v, lo[i] - h * v
        diff = (f(*hi) - f(*lo)) / (2 * h)
        assert abs(float((got.to(F64) * v).sum()) - diff) <= float((v.abs() * mag).sum()) + 1e-6


def test_no_tokens():
    x, w = torch.empty(0, 64, dtype=BF16, device="cuda"), torch.ones(32, 64, dtype=BF16, device="cuda")
    y = torch.empty(0, 32, dtype=BF16, device="cuda")
    ws = capi.alloc_linear_workspace(x, w)
    capi.linear_bf16(x, w, y, ws)
    buf = torch.full((32, 72), 77.0, dtype=BF16, device="cuda")
    db = torch.full((32,), 5.0, device="cuda")
    capi.linear_bf16_backward(y, x, w, ws, dw=buf[:, :64], db=db)
    assert not buf[:, :64].any() and not db.any() and bool((buf[:, 64:] == 77.0).all())


@pytest.mark.parametrize("T,K,N", [(6, 512, 640), (700, 515, 333), (2049, 1032, 4096)])
def test_repeats_graphs_and_streams(T, K, N):
    g = torch.Generator().manual_seed(4)
    data = [(_rand(g, T, K), _rand(g, T, N, scale=0.1)) for _ in range(2)]
    w, b = _rand(g, N, K, scale=K ** -0.5), torch.randn(N, generator=g).to(BF16).cuda()

    def buffers():
        e = lambda *s: torch.empty(*s, dtype=BF16, device="cuda")  # noqa: E731
        return dict(y=e(T, N), z=e(T, N), dx=e(T, K), dw=e(N, K), db=torch.empty(N, device="cuda"),
                    ws=capi.alloc_linear_workspace(data[0][0], w),
                    wsb=capi.alloc_linear_backward_workspace(data[0][1], data[0][0], w))

    def call(x, dy, o):
        capi.linear_bf16(x, w, o["y"], o["ws"], bias=b, act="gelu", z=o["z"])
        capi.linear_bf16_backward(dy, x, w, o["wsb"], z=o["z"], act="gelu", dx=o["dx"], dw=o["dw"], db=o["db"])

    want = []
    for x, dy in data:
        want.append(buffers())
        call(x, dy, want[-1])
    torch.cuda.synchronize()
    outs = ("y", "z", "dx", "dw", "db")
    side = torch.cuda.Stream()
    o = buffers()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(*data[0], o)
    side.synchronize()
    assert all(torch.equal(o[n], want[0][n]) for n in outs)
    x, dy = data[0][0].clone(), data[0][1].clone()
    o = buffers()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(x, dy, o)
    for n in (1, 0, 1):
        x.copy_(data[n][0])
        dy.copy_(data[n][1])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o[k], want[n][k]) for k in outs)


def test_offsets_past_32_bits():
    """Outputs and operands of more than 2^31 elements: the last rows and columns."""
    T, K, N = 36000, 64, 60000
    g = torch.Generator(device="cuda").manual_seed(2)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=BF16)  # noqa: E731
    x, w, b = rn(T, K), rn(N, K) / 8, rn(N)
    y, z = torch.empty(T, N, dtype=BF16, device="cuda"), torch.empty(T, N, dtype=BF16, device="cuda")
    ws = capi.alloc_linear_workspace(x, w)
    capi.linear_bf16(x, w, y, ws, bias=b, act="silu", z=z)
    for rows in (slice(0, 3), slice(T - 200, T)):
        _check_forward(x[rows], w, b, None, y[rows], z[rows], "silu")
    dy = y                                           # any values of its size
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(N, device="cuda")
    ws = capi.alloc_linear_backward_workspace(dy, x, w)
    capi.linear_bf16_backward(dy, x, w, ws, z=z, act="silu", dx=dx, dw=dw, db=db)
    capi.moe_read_device_status(ws)
    rows, cols = slice(T - 100, T), slice(N - 100, N)
    G, Z = dy[rows].to(F64), z[rows].to(F64)
    dz, e = G * _slope("silu", Z), 2.0 ** -20 * G.abs() * (1 + Z.abs())
    W = w.to(F64).abs()
    tol = HALF * (dz @ w.to(F64)).abs() + 1.01 * ((HALF + _acc(N)) * (dz.abs() @ W) + e @ W)
    assert ((dx[rows].to(F64) - dz @ w.to(F64)).abs() <= tol).all()
    G, Z, X = dy[:, cols].to(F64), z[:, cols].to(F64), x.to(F64)
    dz, e = G * _slope("silu", Z), 2.0 ** -20 * G.abs() * (1 + Z.abs())
    tol = HALF * (dz.T @ X).abs() + 1.01 * ((HALF + _acc(T)) * (dz.abs().T @ X.abs()) + e.T @ X.abs())
    assert ((dw[cols].to(F64) - dz.T @ X).abs() <= tol).all()
    assert ((db[cols].to(F64) - dz.sum(0)).abs() <= 1.01 * ((T + 8) * 2.0 ** -24 * dz.abs().sum(0) + e.sum(0))).all()


def test_the_first_calls_of_a_process_may_be_captured():
    code = """
import torch
from routed_nvfp4_expert_b200 import capi
BF = torch.bfloat16
x, w, b = torch.randn(300, 250).to(BF).cuda(), torch.randn(400, 250).to(BF).cuda(), torch.randn(400).to(BF).cuda()
y, z, dx, dw = (torch.empty(*s, dtype=BF, device="cuda") for s in ((300, 400), (300, 400), (300, 250), (400, 250)))
db = torch.empty(400, device="cuda")
cfg = capi.SiteConfig(256, 128, 0, 500, 0, 500, 4, 2.5, 7.0)
logits, ids = torch.randn(300, 500, device="cuda"), torch.randint(0, 500, (300, 4), device="cuda", dtype=torch.int32)
counts, mean, loss = torch.empty(1, 500, dtype=torch.int32, device="cuda"), torch.empty(1, 500, device="cuda"), torch.empty(1, device="cuda")
d_logits, one = torch.empty(300, 500, device="cuda"), torch.ones(1, device="cuda")
ws, wsb, wsl = capi.alloc_linear_workspace(x, w), capi.alloc_linear_backward_workspace(y, x, w), capi.alloc_balance_workspace(cfg, 300)
def calls():
    capi.linear_bf16(x, w, y, ws, bias=b, act="gelu", z=z)
    capi.linear_bf16_backward(y, x, w, wsb, z=z, act="gelu", dx=dx, dw=dw, db=db)
    capi.moe_balance_loss(cfg, logits, ids, 0.1, counts, mean, loss, wsl)
    capi.moe_router_backward(cfg, logits, ids, d_logits, coef=0.1, counts=counts, d_loss=one)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    calls()
g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (y, z, dx, dw, db, counts, mean, loss, d_logits)]
calls()
torch.cuda.synchronize()
assert all(torch.equal(a, t) for a, t in zip(got, (y, z, dx, dw, db, counts, mean, loss, d_logits)))
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_two_calls_at_once_with_workspaces_of_their_own():
    g = torch.Generator().manual_seed(6)
    jobs = []
    for T, K, N in ((300, 1001, 400), (20, 4096, 2048)):
        x, w = _rand(g, T, K), _rand(g, N, K, scale=K ** -0.5)
        jobs.append((x, w, torch.empty(T, N, dtype=BF16, device="cuda"), capi.alloc_linear_workspace(x, w),
                     torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for x, w, y, ws, st in jobs:
            capi.linear_bf16(x, w, y, ws, act="silu", stream=st)
    torch.cuda.synchronize()
    for x, w, y, ws, _ in jobs:
        capi.moe_read_device_status(ws)
        _check_forward(x, w, None, None, y, None, "silu")


def test_two_large_calls_at_once():
    """Two launches that each fill the GPU, competing for the SMs."""
    g = torch.Generator().manual_seed(8)
    jobs = []
    for T, K, N in ((2049, 4096, 1280), (700, 8192, 4000)):
        x, w = _rand(g, T, K), _rand(g, N, K, scale=K ** -0.5)
        y = [torch.empty(T, N, dtype=BF16, device="cuda") for _ in range(2)]
        ws = capi.alloc_linear_workspace(x, w)
        capi.linear_bf16(x, w, y[0], ws, act="silu")
        jobs.append((x, w, y, ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(30):
        for x, w, y, ws, st in jobs:
            capi.linear_bf16(x, w, y[1], ws, act="silu", stream=st)
    torch.cuda.synchronize()
    for x, w, y, ws, _ in jobs:
        capi.moe_read_device_status(ws)
        assert torch.equal(y[0], y[1])
        _check_forward(x, w, None, None, y[1], None, "silu")


def test_a_training_block_with_the_router():
    """The operators as a training step runs them: up projection, down projection
    closing the residual, router, balance loss; then back to the first weight."""
    T, H, I, E, k, coef = 150, 256, 512, 16, 4, 0.05
    cfg = capi.SiteConfig(H, 128, 0, E, 0, E, k, 2.5, 7.0)
    g = torch.Generator().manual_seed(11)
    x, w1, w2 = _rand(g, T, H), _rand(g, I, H, scale=H ** -0.5), _rand(g, H, I, scale=I ** -0.5)
    b1 = torch.randn(I, generator=g).mul(0.1).to(BF16).cuda()
    wr, bias = (torch.randn(E, H, generator=g) / 16).cuda(), torch.zeros(E, device="cuda")
    e = lambda *s, **o: torch.empty(*s, device="cuda", **o)  # noqa: E731
    a, z1, h = e(T, I, dtype=BF16), e(T, I, dtype=BF16), e(T, H, dtype=BF16)
    ws = [capi.alloc_linear_workspace(x, w1), capi.alloc_linear_workspace(a, w2)]
    capi.linear_bf16(x, w1, a, ws[0], bias=b1, act="gelu", z=z1)
    capi.linear_bf16(a, w2, h, ws[1], residual=x)
    logits, ids, wts = e(T, E), e(T, k, dtype=torch.int32), e(T, k)
    capi.moe_router_topk(cfg, h, wr, bias, logits, ids, wts)
    off = torch.tensor([0, 40, T], dtype=torch.int32, device="cuda")
    counts, mean, loss = e(2, E, dtype=torch.int32), e(2, E), e(2)
    capi.moe_balance_loss(cfg, logits, ids, coef, counts, mean, loss, capi.alloc_balance_workspace(cfg, T, 2), off)
    d_wts, d_loss, d_logits = torch.randn(T, k, generator=g).mul(0.01).cuda(), torch.ones(2, device="cuda"), e(T, E)
    capi.moe_router_backward(cfg, logits, ids, d_logits, d_weights=d_wts, coef=coef, counts=counts, d_loss=d_loss,
                             seq_offsets=off)
    dh = (d_logits @ wr).to(BF16)
    da, dw2, dx, dw1, db1 = e(T, I, dtype=BF16), e(H, I, dtype=BF16), e(T, H, dtype=BF16), e(I, H, dtype=BF16), e(I)
    capi.linear_bf16_backward(dh, a, w2, capi.alloc_linear_backward_workspace(dh, a, w2), dx=da, dw=dw2)
    capi.linear_bf16_backward(da, x, w1, capi.alloc_linear_backward_workspace(da, x, w1), z=z1, act="gelu", dx=dx,
                              dw=dw1, db=db1)
    # the same in 64 bits by automatic differentiation
    P = [t.to(F64).requires_grad_() for t in (x, w1, b1, w2)]
    H1 = _act("gelu", P[0] @ P[1].T + P[2]) @ P[3].T + P[0]
    s = torch.sigmoid(H1 @ wr.to(F64).T)
    total = torch.zeros((), dtype=F64, device="cuda")
    for q in range(2):
        lo, hi = int(off[q]), int(off[q + 1])
        f = counts[q].to(F64) * E / (k * (hi - lo))
        total = total + coef * (f * (s[lo:hi] / s[lo:hi].sum(1, keepdim=True)).mean(0)).sum()
    chosen = s.gather(1, ids.long())
    total = total + (2.5 * chosen / chosen.sum(1, keepdim=True) * d_wts.to(F64)).sum()
    want = torch.autograd.grad(total, P)
    dx = dx.to(F64) + dh.to(F64)                     # the residual's gradient is dh itself
    # eight bf16 roundings on the way (a, z1, h, dh, da, dz, the results), each at most 2^-8 of its tensor
    for got, ref in ((dx, want[0]), (dw1, want[1]), (db1, want[2]), (dw2, want[3])):
        assert float((got.to(F64) - ref).norm() / ref.norm()) <= 8 * HALF
    total = total.detach()
    chosen = chosen.detach()
    assert abs(float(loss.sum()) - float((total - (2.5 * chosen / chosen.sum(1, keepdim=True) * d_wts.to(F64)).sum()))) \
        <= 8 * HALF * float(loss.sum())
