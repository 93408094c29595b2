"""The router's balance loss and the logits' gradient (moe_balance_loss,
moe_router_backward) against plain formulas in 64 bits.

Tolerances, in fp32 half steps u = 2^-24: a score is off by at most 16 u
relative (exponential, reciprocal, product), a row's sum by E u more, a sum of
n positive rows by n u more; every term of mean_scores and loss is positive, so
these are relative bounds. In the gradient, f - mean and v - m subtract, so the
bound is relative to the sum of the magnitudes."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

capi = pytest.importorskip("routed_nvfp4_expert_b200.capi")

U = 2.0 ** -24
RSF = 2.5


def _cfg(E, k):
    return capi.SiteConfig(256, 128, 0, E, 0, E, k, RSF, 7.0)


def _inputs(T, E, k, seed, dropped=False, twice=False):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(T, E, generator=g) * 2
    ids = torch.rand(T, E, generator=g).topk(k, dim=1).indices.to(torch.int32) if T else torch.zeros(0, k, dtype=torch.int32)
    if dropped and T:
        ids[torch.rand(T, k, generator=g) < 0.2] = -1
        ids[0] = E                      # a token whose assignments are all out of range
    if twice and k > 1:
        ids[:, 1] = ids[:, 0]           # the same expert in two slots
    return logits, ids


def _reference(logits, ids, off, E, k, coef, counts=None, d_loss=None, d_weights=None):
    """Counts, mean scores, losses; with gradients' inputs also d_logits and the
    magnitudes its bound is relative to."""
    l = logits.double()
    s, rest = torch.sigmoid(l), torch.sigmoid(-l)
    S = s.sum(1, keepdim=True)
    share = torch.where(S > 0, s / S, torch.zeros_like(s))
    B = len(off) - 1
    cnt = torch.zeros(B, E, dtype=torch.int64)
    mean, loss = torch.zeros(B, E, dtype=torch.float64), torch.zeros(B, dtype=torch.float64)
    grad, mag = torch.zeros_like(l), torch.zeros_like(l)
    for b in range(B):
        lo, hi = off[b], off[b + 1]
        if hi <= lo:
            continue
        n = hi - lo
        ok = ids[lo:hi][(ids[lo:hi] >= 0) & (ids[lo:hi] < E)].long()
        cnt[b] = torch.bincount(ok, minlength=E)
        mean[b] = share[lo:hi].sum(0) / n
        f = (cnt[b] if counts is None else counts[b]).double() * E / (k * n)
        loss[b] = coef * (f * mean[b]).sum()
        if d_loss is not None:
            c = d_loss[b].double() * coef / n
            m = (share[lo:hi] * f).sum(1, keepdim=True)
            w = torch.where(S[lo:hi] > 0, c / S[lo:hi], torch.zeros_like(S[lo:hi])) * s[lo:hi] * rest[lo:hi]
            grad[lo:hi] += w * (f - m)
            mag[lo:hi] += w.abs() * (f + m)
        if d_weights is not None:
            for t in range(lo, hi):
                slots = [(int(e), float(v)) for e, v in zip(ids[t], d_weights[t]) if 0 <= e < E]
                C = sum(float(s[t, e]) for e, _ in slots)
                if C == 0:
                    continue
                m = sum(v * float(s[t, e]) for e, v in slots) / C
                ma = sum(abs(v) * float(s[t, e]) for e, v in slots) / C
                for e, v in slots:
                    ds = float(s[t, e] * rest[t, e])
                    grad[t, e] += RSF / C * (v - m) * ds
                    mag[t, e] += RSF / C * (abs(v) + ma) * ds
    return cnt, mean, loss, grad, mag


def _run(T, E, k, off, coef, logits, ids, stream=None):
    B = len(off) - 1 if off is not None else 1
    cfg = _cfg(E, k)
    counts = torch.full((B, E), -7, dtype=torch.int32, device="cuda")
    mean = torch.full((B, E), float("nan"), device="cuda")
    loss = torch.full((B,), float("nan"), device="cuda")
    ws = capi.alloc_balance_workspace(cfg, T, B)
    o = None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")
    capi.moe_balance_loss(cfg, logits.cuda(), ids.cuda(), coef, counts, mean, loss, ws, seq_offsets=o, stream=stream)
    return counts, mean, loss


CASES = [
    # T, E, k, offsets (None: one sequence), dropped, the same expert twice
    (1, 8, 1, None, False, False),
    (1, 16, 16, None, False, False),
    (7, 3, 2, [0, 0, 3, 3, 7, 7], False, False),
    (33, 31, 4, [2, 9, 30], True, False),
    (64, 288, 8, None, False, True),
    (256, 100, 5, [0, 255, 256], True, False),
    (257, 288, 8, [0, 257], False, False),
    (300, 1024, 16, [0, 1, 2, 150, 299], True, True),
    # expert counts that end inside a row's last vectors, at each number of lanes per row
    (20, 33, 3, None, False, False),
    (50, 40, 4, [0, 20, 50], False, True),
    (2100, 112, 12, [0, 700, 2090], True, True),
    (1900, 10, 3, None, False, True),
    (90, 330, 5, [0, 40, 90], False, False),
    (70, 650, 16, None, True, False),
    (3000, 322, 4, [0, 1000, 2999], False, False),
    (2500, 129, 4, None, False, False),
    (5000, 64, 6, [0, 34, 34, 35, 4000, 4990], True, False),
    (9001, 384, 8, None, False, False),
]
GRAD_CASES = [c for c in CASES if c[0] <= 3000]


@pytest.mark.parametrize("T,E,k,off,dropped,twice", CASES)
def test_balance_matches_the_formula(T, E, k, off, dropped, twice):
    logits, ids = _inputs(T, E, k, T + E, dropped, twice)
    ref_off = [0, T] if off is None else off
    cnt, mean, loss, _, _ = _reference(logits, ids, ref_off, E, k, 0.01)
    counts, got_mean, got_loss = (v.cpu() for v in _run(T, E, k, off, 0.01, logits, ids))
    assert torch.equal(counts.long(), cnt)
    n = max(b - a for a, b in zip(ref_off, ref_off[1:]))
    tol = (n + 2 * E + 64) * U
    assert ((got_mean.double() - mean).abs() <= tol * mean).all()
    assert ((got_loss.double() - loss).abs() <= tol * loss).all()


@pytest.mark.parametrize("terms", ["both", "weights", "loss"])
@pytest.mark.parametrize("T,E,k,off,dropped,twice", GRAD_CASES)
def test_router_backward_matches_the_formula(T, E, k, off, dropped, twice, terms):
    logits, ids = _inputs(T, E, k, T * 3 + E, dropped, twice)
    ref_off = [0, T] if off is None else off
    B = len(ref_off) - 1
    g = torch.Generator().manual_seed(T)
    d_loss = torch.randn(B, generator=g) if terms != "weights" else None
    # of the balance term's size, so that neither hides the other
    d_weights = torch.randn(T, k, generator=g) * 1e-3 if terms != "loss" else None
    cnt, _, _, grad, mag = _reference(logits, ids, ref_off, E, k, 0.5, None, d_loss, d_weights)
    cfg = _cfg(E, k)
    keep = torch.randn(T, E, generator=g)
    out = keep.cuda()
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    capi.moe_router_backward(cfg, logits.cuda(), ids.cuda(), out, d_weights=cu(d_weights), coef=0.5,
                             counts=cnt.to(torch.int32).cuda() if d_loss is not None else None, d_loss=cu(d_loss),
                             seq_offsets=None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda"))
    out = out.cpu()
    inside = torch.zeros(T, dtype=torch.bool)
    inside[ref_off[0]:ref_off[-1]] = True
    assert torch.equal(out[~inside], keep[~inside])         # rows of no sequence are left as they were
    d = (out.double() - grad)[inside].abs()
    assert (d <= (E + 64) * 2 * U * mag[inside] + 1e-40).all(), float((d / (mag[inside] + 1e-40)).max() / U)


def test_gradient_matches_differences_of_the_loss():
    T, E, k, off, coef = 40, 24, 4, [0, 13, 40], 0.3
    logits, ids = _inputs(T, E, k, 5)
    g = torch.Generator().manual_seed(1)
    d_loss, d_w = torch.randn(2, generator=g), torch.randn(T, k, generator=g) * 1e-2
    cnt, *_ = _reference(logits, ids, off, E, k, coef)

    def objective(l):
        _, _, loss, _, _ = _reference(l, ids, off, E, k, coef, counts=cnt)
        s = torch.sigmoid(l.double())
        chosen = s.gather(1, ids.long())
        w = RSF * chosen / chosen.sum(1, keepdim=True)
        return float((loss * d_loss.double()).sum() + (w * d_w.double()).sum())

    out = torch.empty(T, E, device="cuda")
    capi.moe_router_backward(_cfg(E, k), logits.cuda(), ids.cuda(), out, d_weights=d_w.cuda(), coef=coef,
                             counts=cnt.to(torch.int32).cuda(), d_loss=d_loss.cuda(),
                             seq_offsets=torch.tensor(off, dtype=torch.int32, device="cuda"))
    out = out.cpu().double()
    for seed in range(3):
        v = torch.randn(T, E, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)
        h = 1e-5
        diff = (objective(logits.double() + h * v) - objective(logits.double() - h * v)) / (2 * h)
        # differences: third derivatives times h^2 and 1e-16 / h; gradient: fp32
        assert abs(float((out * v).sum()) - diff) <= 1e-8 + 1e-5 * float((out * v).abs().sum())


def test_extreme_logits():
    """-inf, very low and very high logits, and a row of zero scores: no NaN where
    the formula has a value; a NaN stays in its own sequence (row for the gradient)."""
    E, k = 40, 4
    logits, ids = _inputs(6, E, k, 3)
    logits[0] = float("-inf")                       # every score 0
    logits[1, ::2] = float("-inf")
    logits[2] = 80.0
    logits[3] = -80.0
    logits[4, 0] = float("inf")
    off = [0, 5, 6]
    d_loss, d_w = torch.ones(2), torch.full((6, k), 1e-3)
    cnt, mean, loss, grad, mag = _reference(logits, ids, off, E, k, 0.1, None, d_loss, d_w)
    counts, got_mean, got_loss = (v.cpu() for v in _run(6, E, k, off, 0.1, logits, ids))
    assert ((got_mean.double() - mean).abs() <= (2 * E + 64) * U * mean + 1e-40).all()
    out = torch.empty(6, E, device="cuda")
    args = dict(d_weights=d_w.cuda(), coef=0.1, counts=cnt.to(torch.int32).cuda(), d_loss=d_loss.cuda(),
                seq_offsets=torch.tensor(off, dtype=torch.int32, device="cuda"))
    capi.moe_router_backward(_cfg(E, k), logits.cuda(), ids.cuda(), out, **args)
    assert ((out.cpu().double() - grad).abs() <= (E + 64) * 2 * U * mag + 1e-38).all()
    logits[5, 7] = float("nan")
    counts, got_mean, got_loss = (v.cpu() for v in _run(6, E, k, off, 0.1, logits, ids))
    assert torch.isnan(got_loss).tolist() == [False, True] and not torch.isnan(got_mean[0]).any()
    capi.moe_router_backward(_cfg(E, k), logits.cuda(), ids.cuda(), out, **args)
    assert not torch.isnan(out[:5]).any() and torch.isnan(out[5]).all()


def test_offsets_past_32_bits():
    """More than 2^31 logits: the last sequence's results and gradients."""
    T, E, k, last = 7_500_000, 288, 2, 60
    g = torch.Generator(device="cuda").manual_seed(1)
    logits = torch.randn(T, E, device="cuda", generator=g)
    ids = torch.randint(0, E, (T, k), device="cuda", generator=g, dtype=torch.int32)
    cfg, off = _cfg(E, k), torch.tensor([0, T - last, T], dtype=torch.int32, device="cuda")
    counts, mean = torch.empty(2, E, dtype=torch.int32, device="cuda"), torch.empty(2, E, device="cuda")
    loss, out = torch.empty(2, device="cuda"), torch.empty(T, E, device="cuda")
    ws = capi.alloc_balance_workspace(cfg, T, 2)
    capi.moe_balance_loss(cfg, logits, ids, 0.1, counts, mean, loss, ws, seq_offsets=off)
    assert int(counts[0].sum()) == (T - last) * k
    assert abs(float(mean[0].double().sum()) - 1) <= (T / 148 / 16 + 148 + 2 * E + 64) * U    # the sums' longest chain
    d_loss, d_w = torch.ones(2, device="cuda"), torch.randn(T, k, device="cuda", generator=g) * 1e-3
    capi.moe_router_backward(cfg, logits, ids, out, d_weights=d_w, coef=0.1, counts=counts, d_loss=d_loss, seq_offsets=off)
    tail = slice(T - last, T)
    cnt, m, l, grad, mag = _reference(logits[tail].cpu(), ids[tail].cpu(), [0, last], E, k, 0.1, None, d_loss[:1].cpu(),
                                      d_w[tail].cpu())
    assert torch.equal(counts[1:].cpu().long(), cnt)
    assert ((mean[1:].cpu().double() - m).abs() <= (last + 2 * E + 64) * U * m).all()
    assert ((out[tail].cpu().double() - grad).abs() <= (E + 64) * 2 * U * mag + 1e-40).all()


def test_no_tokens_and_no_sequences():
    counts, mean, loss = _run(0, 16, 2, None, 1.0, torch.zeros(0, 16), torch.zeros(0, 2, dtype=torch.int32))
    assert not counts.any() and not mean.any() and not loss.any()
    counts, mean, loss = _run(600, 16, 2, [5, 5, 5], 1.0, *_inputs(600, 16, 2, 0))
    assert not counts.any() and not mean.any() and not loss.any()


def test_wrong_offsets_stay_in_bounds():
    """Offsets outside [0, T] are read as its ends; descending ones give no result
    worth having, and no access outside the rows."""
    T, E, k = 700, 32, 4
    logits, ids = _inputs(T, E, k, 1)
    a = _run(T, E, k, [-5, 300, T + 1000], 0.1, logits, ids)
    b = _run(T, E, k, [0, 300, T], 0.1, logits, ids)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    _run(T, E, k, [600, 20, 650, 0], 0.1, logits, ids)
    torch.cuda.synchronize()


@pytest.mark.parametrize("T", [200, 6000])
def test_repeats_graphs_and_streams(T):
    """Equal bits from repeated calls, from another stream and from a replayed graph on new inputs."""
    E, k = 96, 8
    off = torch.tensor([0, T // 3, T], dtype=torch.int32, device="cuda")
    data = [tuple(v.cuda() for v in _inputs(T, E, k, s)) for s in (1, 2)]
    cfg = _cfg(E, k)
    d_loss = torch.ones(2, device="cuda")

    def call(logits, ids, bufs):
        counts, mean, loss, ws, grad = bufs
        capi.moe_balance_loss(cfg, logits, ids, 0.1, counts, mean, loss, ws, seq_offsets=off)
        capi.moe_router_backward(cfg, logits, ids, grad, coef=0.1, counts=counts, d_loss=d_loss, seq_offsets=off)

    def buffers():
        return (torch.empty(2, E, dtype=torch.int32, device="cuda"), torch.empty(2, E, device="cuda"),
                torch.empty(2, device="cuda"), capi.alloc_balance_workspace(cfg, T, 2), torch.empty(T, E, device="cuda"))

    want = []
    for logits, ids in data:
        bufs = buffers()
        call(logits, ids, bufs)
        want.append(bufs)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    bufs = buffers()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(*data[0], bufs)
    side.synchronize()
    for i in (0, 1, 2, 4):
        assert torch.equal(bufs[i], want[0][i])
    logits, ids = data[0][0].clone(), data[0][1].clone()
    bufs = buffers()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(logits, ids, bufs)
    for n in (1, 0, 1):
        logits.copy_(data[n][0])
        ids.copy_(data[n][1])
        graph.replay()
        torch.cuda.synchronize()
        for i in (0, 1, 2, 4):
            assert torch.equal(bufs[i], want[n][i])


def test_after_the_router():
    """As a training step calls it: the router's own logits and ids."""
    T, H, E, k = 37, 256, 16, 4
    cfg = capi.SiteConfig(H, 128, 0, E, 0, E, k, RSF, 7.0)
    g = torch.Generator().manual_seed(0)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    wr = (torch.randn(E, H, generator=g) / 16).cuda()
    bias = torch.randn(E, generator=g).mul(0.1).cuda()
    logits, ids = torch.empty(T, E, device="cuda"), torch.empty(T, k, dtype=torch.int32, device="cuda")
    weights = torch.empty(T, k, device="cuda")
    capi.moe_router_topk(cfg, x, wr, bias, logits, ids, weights)
    counts, mean, loss = _run(T, E, k, None, 0.01, logits, ids)
    cnt, m, l, _, _ = _reference(logits.cpu(), ids.cpu(), [0, T], E, k, 0.01)
    assert torch.equal(counts.cpu().long(), cnt) and int(counts.sum()) == T * k
    assert np.allclose(loss.cpu().numpy(), l.numpy(), rtol=(T + 2 * E + 64) * U, atol=0)


@pytest.mark.parametrize("E", [16, 64, 288, 384])
@pytest.mark.parametrize("T", [700, 5000])
def test_rows_of_a_neighbour_never_enter_a_sequence(E, T):
    """Sequences that end inside a group of rows worked on together: NaN rows of
    one, before the first and behind the last leave the others' results as they
    are, to the bit."""
    k = 4
    cfg = capi.SiteConfig(4096, 1024, 1024, E, 0, E, k, 2.5, 7.0)
    g = torch.Generator().manual_seed(E + T)
    logits = torch.randn(T, E, generator=g).cuda()
    ids = torch.randint(0, E, (T, k), generator=g).to(torch.int32).cuda()
    off = [3, 3 + T // 5, 5 + T // 5, 6 + T // 5, T // 2 + 1, T - 9]
    B = len(off) - 1
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")

    def call(x):
        counts = torch.full((B, E), -1, dtype=torch.int32, device="cuda")
        mean, loss = torch.full((B, E), 7.0, device="cuda"), torch.full((B,), 7.0, device="cuda")
        ws = capi.alloc_balance_workspace(cfg, T, B)
        ws.fill_(0xFF)
        capi.moe_balance_loss(cfg, x, ids, 0.01, counts, mean, loss, ws, seq_offsets=offsets)
        return counts, mean, loss

    bad = logits.clone()
    bad[:off[0]] = float("nan")
    bad[off[-1]:] = float("nan")
    bad[off[1]:off[2]] = float("nan")
    want, got = call(logits), call(bad)
    assert torch.equal(got[0], want[0])
    for b in range(B):
        if b == 1:
            assert got[1][b].isnan().all() and got[2][b].isnan()
        else:
            assert torch.equal(got[1][b], want[1][b]) and torch.equal(got[2][b], want[2][b])
    share = logits.double().sigmoid()
    share = share / share.sum(1, keepdim=True)
    for b in range(B):
        # sums of at most T terms of one sign in fp32, each within 2^-20 of its value
        ref = share[off[b]:off[b + 1]].mean(0)
        assert ((want[1][b].double() - ref).abs() <= (2.0 ** -20 + T * 2.0 ** -24) * ref).all()
