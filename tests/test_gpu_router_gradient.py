"""Which weights moe_router_backward differentiates where assignments are
dropped, and its range: rows of very low scores, large and small gradients.

Tolerances, in fp32 half steps u = 2^-24: the exponent l log2 e of a score is
rounded twice (the constant, the product), which moves the score by up to
1.25 |l| u; exponential, reciprocal and sum add 16 u. A term of the gradient
holds up to four such factors beside sums of E terms and is bounded relative to
the magnitudes that it adds or subtracts."""
import pytest
import torch

pytestmark = pytest.mark.gpu

capi = pytest.importorskip("routed_nvfp4_expert_b200.capi")

U = 2.0 ** -24
RSF = 2.5


def _cfg(E, k):
    return capi.SiteConfig(256, 128, 0, E, 0, E, k, RSF, 7.0)


def _weight_gradient(logits, ids, v):
    """d logits of sum v_j rsf s_j / C over the slots with an id in [0, E), and the magnitudes that it adds up."""
    E = logits.shape[1]
    s, rest = torch.sigmoid(logits.double()), torch.sigmoid(-logits.double())
    ok = (ids >= 0) & (ids < E)
    at = torch.where(ok, ids, 0).long()
    p = torch.where(ok, s.gather(1, at), 0.0)
    C = p.sum(1, keepdim=True)
    p = torch.where(C > 0, p / C, 0.0)
    v = torch.where(ok, v.double(), 0.0)
    slope = RSF * p * rest.gather(1, at)
    grad = torch.zeros_like(s).scatter_add(1, at, slope * (v - (v * p).sum(1, keepdim=True)))
    mag = torch.zeros_like(s).scatter_add(1, at, slope * (v.abs() + (v.abs() * p).sum(1, keepdim=True)))
    return grad, mag


def _loss_gradient(logits, counts, k, coef, d_loss):
    """d logits of the balance loss of one sequence of all rows."""
    T, E = logits.shape
    s, rest = torch.sigmoid(logits.double()), torch.sigmoid(-logits.double())
    p = s / s.sum(1, keepdim=True)
    f = counts.double() * E / (k * T)
    m = (p * f).sum(1, keepdim=True)
    w = p * rest * (float(d_loss) * coef / T)
    return w * (f - m), w.abs() * (f + m)


def _tol(E, logits):
    return (E + 64 + 8 * 1.25 * float(logits.abs().max())) * 2 * U


def _call(logits, ids, k, **kw):
    out = torch.full(logits.shape, float("nan"), device="cuda")
    cu = {n: t.cuda() if torch.is_tensor(t) else t for n, t in kw.items()}
    capi.moe_router_backward(_cfg(logits.shape[1], k), logits.cuda(), ids.cuda(), out, **cu)
    return out.cpu().double()


@pytest.mark.parametrize("T,E,k", [(5, 16, 2), (300, 96, 8), (2600, 288, 8), (40, 700, 16)])
def test_assignments_dropped_after_the_weights_were_normalised(T, E, k):
    """The router's ids unchanged with d_weights 0 where an assignment was
    dropped: the gradient of moe_router_topk's weights, in which the dropped
    experts' scores stay; the counts may leave the drops out."""
    H = 256
    g = torch.Generator().manual_seed(T + E)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    wr, bias = (torch.randn(E, H, generator=g) / 16).cuda(), torch.randn(E, generator=g).mul(0.1).cuda()
    logits, weights = torch.empty(T, E, device="cuda"), torch.empty(T, k, device="cuda")
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    capi.moe_router_topk(_cfg(E, k), x, wr, bias, logits, ids, weights)
    keep = torch.rand(T, k, generator=g) < 0.7
    keep[0] = False
    keep[1, 1:] = False                                    # a single kept weight still depends on the others' scores
    keep[1, 0] = True
    v = torch.randn(T, k, generator=g) * keep
    logits, ids = logits.cpu(), ids.cpu()

    marked = torch.where(keep, ids, -1)
    cfg = _cfg(E, k)
    counts = torch.empty(1, E, dtype=torch.int32, device="cuda")
    mean, loss = torch.empty(1, E, device="cuda"), torch.empty(1, device="cuda")
    capi.moe_balance_loss(cfg, logits.cuda(), marked.cuda(), 0.5, counts, mean, loss, capi.alloc_balance_workspace(cfg, T))
    counts = counts.cpu()
    assert torch.equal(counts[0].long(), torch.bincount(ids[keep].long(), minlength=E))
    out = _call(logits, ids, k, d_weights=v, coef=0.5, counts=counts, d_loss=torch.tensor([0.7]))
    grad, mag = _weight_gradient(logits, ids, v)
    bal, bal_mag = _loss_gradient(logits, counts, k, 0.5, 0.7)
    assert ((out - grad - bal).abs() <= _tol(E, logits) * (mag + bal_mag) + 1e-40).all()
    assert float(grad[1].abs().max()) > 1e-4               # v - m does not vanish for the single kept slot

    # the weights' part against differences of the weights in use
    only = _call(logits, ids, k, d_weights=v)

    def objective(l):
        s = torch.sigmoid(l).gather(1, ids.long())
        return float((RSF * s / s.sum(1, keepdim=True) * v.double()).sum())

    d = torch.randn(T, E, generator=g, dtype=torch.float64)
    h = 1e-5
    diff = (objective(logits.double() + h * d) - objective(logits.double() - h * d)) / (2 * h)
    # differences: third derivatives times h^2 and 1e-16 / h; gradient: fp32
    assert abs(float((only * d).sum()) - diff) <= 1e-8 + 1e-5 * float((only * d).abs().sum())


@pytest.mark.parametrize("T,E,k", [(300, 96, 8), (2600, 288, 5)])
def test_assignments_left_out_before_the_weights_are_normalised(T, E, k):
    """An id outside [0, E): the gradient of weights normalised over the others."""
    g = torch.Generator().manual_seed(T)
    logits = torch.randn(T, E, generator=g)
    ids = torch.rand(T, E, generator=g).topk(k, dim=1).indices.to(torch.int32)
    keep = torch.rand(T, k, generator=g) < 0.6
    keep[0], keep[1, 1:] = False, False
    v = torch.randn(T, k, generator=g)
    marked = torch.where(keep, ids, torch.tensor(-1, dtype=torch.int32))
    out = _call(logits, marked, k, d_weights=v)
    l = logits.double().requires_grad_()
    s = torch.sigmoid(l).gather(1, ids.long()) * keep
    C = s.sum(1, keepdim=True)
    (want,) = torch.autograd.grad((RSF * s / torch.where(C > 0, C, 1.0) * v.double()).sum(), l)
    _, mag = _weight_gradient(logits, marked, v)
    assert ((out - want).abs() <= _tol(E, logits) * mag + 1e-40).all()
    assert not out[0].any()


@pytest.mark.parametrize("T,E,k", [(64, 40, 4), (3000, 96, 8), (50, 288, 8), (9, 700, 16)])
@pytest.mark.parametrize("scale", [1e-8, 1.0, 1e5])
def test_rows_of_very_low_scores(T, E, k, scale):
    """Logits down to where a score just exceeds 2^-126 (l > -87.3), with small
    and loss-scaled upstream gradients: no intermediate leaves the range, and
    nothing is lost where the gradient itself is an ordinary number."""
    g = torch.Generator().manual_seed(E)
    logits = -75.0 - 12.2 * torch.rand(T, E, generator=g)
    logits[1] = -87.0                                      # all equal: v - m alone decides
    logits[2, : E // 2] = 3.0                              # ordinary scores beside the lowest
    ids = torch.rand(T, E, generator=g).topk(k, dim=1).indices.to(torch.int32)
    v = torch.randn(T, k, generator=g) * scale
    counts = torch.bincount(ids.reshape(-1).long(), minlength=E).to(torch.int32)[None]
    d_loss = torch.tensor([scale])
    grad, mag = _weight_gradient(logits, ids, v)
    bal, bal_mag = _loss_gradient(logits, counts, k, 0.5, d_loss)
    tol = _tol(E, logits)
    assert tol < 3e-4
    out = _call(logits, ids, k, d_weights=v)
    assert ((out - grad).abs() <= tol * mag + 1e-40).all()
    out = _call(logits, ids, k, counts=counts, coef=0.5, d_loss=d_loss)
    assert ((out - bal).abs() <= tol * bal_mag + 1e-40).all()
    out = _call(logits, ids, k, d_weights=v, counts=counts, coef=0.5, d_loss=d_loss)
    assert ((out - grad - bal).abs() <= tol * (mag + bal_mag) + 1e-40).all()


def test_a_large_scaling_factor_at_the_lowest_scores():
    """rsf / C beyond the range while every weight is rsf / k: slots of equal
    upstream gradients have a gradient of 0 up to rounding, not NaN or infinity."""
    T, E, k, rsf = 6, 32, 4, 1000.0
    logits = torch.full((T, E), -87.2)
    ids = torch.arange(k, dtype=torch.int32).repeat(T, 1)
    cfg = capi.SiteConfig(256, 128, 0, E, 0, E, k, rsf, 7.0)
    out = torch.empty(T, E, device="cuda")
    v = torch.ones(T, k)
    v[T // 2:, 0] = 3.0
    capi.moe_router_backward(cfg, logits.cuda(), ids.cuda(), out, d_weights=v.cuda())
    out = out.cpu().double()
    # with equal scores, m = sum(v s) (1 / C) is off by its three sums, the products, the reciprocal and the last
    # product: 8 u of |v| = 1, and a weight is rsf / 4
    assert (out[:T // 2].abs() <= rsf / 4 * 8 * U).all()
    # m = 1.5
    want = rsf / 4 * (v.double() - v.double().mean(1, keepdim=True))
    assert ((out[:, :k] - want).abs() <= 1e-5 * rsf).all() and not out[:, k:].any()


@pytest.mark.parametrize("E,k", [(40, 4), (288, 8)])
def test_a_very_small_loss_gradient(E, k):
    """The balance loss's factor is scaled inside; a gradient of 1e-28 keeps its accuracy."""
    T = 64
    g = torch.Generator().manual_seed(E)
    logits = torch.randn(T, E, generator=g)
    ids = torch.rand(T, E, generator=g).topk(k, dim=1).indices.to(torch.int32)
    counts = torch.bincount(ids.reshape(-1).long(), minlength=E).to(torch.int32)[None]
    d_loss = torch.tensor([1e-28])
    bal, mag = _loss_gradient(logits, counts, k, 0.5, d_loss)
    out = _call(logits, ids, k, counts=counts, coef=0.5, d_loss=d_loss)
    assert ((out - bal).abs() <= _tol(E, logits) * mag + 1e-40).all()
