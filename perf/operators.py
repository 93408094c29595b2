"""Cases of the training-side operators that stand beside the router and the dense layers:

  balance      moe_balance_loss       per-expert counts, mean normalised scores and the balance loss of each sequence
  router_bwd   moe_router_backward    gradient of the logits from the routing weights and from the balance loss
  linear       linear_bf16            y = act(x W^T + b) + residual
  linear_bwd   linear_bf16_backward   dx, dW, db from dy and the pre-activation z

`run` computes a case in plain torch operations, or with `own` set through the library's entry points.
"""
import math

import torch

own = False

BF16 = torch.bfloat16
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


# ------------------------------------------------------------------ cases

def _linear(name, T, K, N, act, bias=True, residual=False, keep_z=False):
    return dict(name=name, op="linear", T=T, K=K, N=N, act=act, bias=bias, residual=residual, keep_z=keep_z)


def _linear_bwd(name, T, K, N, act, bias=True):
    return dict(name=name, op="linear_bwd", T=T, K=K, N=N, act=act, bias=bias)


def listed():
    return [
        # one decoded token through a square projection that closes a residual branch
        _linear("linear_t1", 1, 4096, 4096, "none", residual=True),
        # a decode batch through a dense layer's up projection
        _linear("linear_t32", 32, 4096, 12288, "silu"),
        # a short prompt at ragged sizes: rows that are not 16-byte aligned
        _linear("linear_ragged", 333, 1003, 1537, "gelu", residual=True),
        # a prompt through a dense layer's down projection and residual
        _linear("linear_t4096", 4096, 12288, 4096, "none", residual=True),
        # a training micro-batch: up projection that keeps its pre-activation
        _linear("linear_t16384", 16384, 4096, 12288, "gelu", keep_z=True),
        # gradients at the smallest site's sizes
        _linear_bwd("linear_bwd_t64", 64, 256, 512, "relu"),
        # gradients at ragged sizes
        _linear_bwd("linear_bwd_ragged", 777, 1000, 515, "silu"),
        # gradients of a dense layer's up projection over one prompt-sized micro-batch
        _linear_bwd("linear_bwd_t4096", 4096, 4096, 12288, "gelu"),
        # the balance of one decode batch
        dict(name="balance_t64", op="balance", T=64, E=288, k=8, seqs=1, pad=0, dropped=False),
        # a packed training batch of ragged sequences with padding behind the last, some assignments dropped
        dict(name="balance_packed", op="balance", T=131072, E=288, k=8, seqs=48, pad=1000, dropped=True),
        # one prompt-sized micro-batch
        dict(name="router_bwd_t4096", op="router_bwd", T=4096, E=288, k=8, seqs=1, pad=0, dropped=False),
        # a packed training batch
        dict(name="router_bwd_packed", op="router_bwd", T=65536, E=288, k=8, seqs=37, pad=500, dropped=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("linear", "linear_bwd", "balance", "router_bwd"))
    if op in ("linear", "linear_bwd"):
        most = 16384 * 4096 * 12288 // (2 if op == "linear_bwd" else 1)
        while True:
            K, N = _log_int(rng, 64, 12288), _log_int(rng, 64, 12288)
            if rng.random() < 0.5:
                K, N = max(64, K // 64 * 64), max(64, N // 64 * 64)
            T = _log_int(rng, 1, 16384)
            if T * K * N <= most:
                break
        c = dict(op=op, T=T, K=K, N=N, act=rng.choice(ACTS), bias=rng.random() < 0.7)
        if op == "linear":
            c.update(residual=rng.random() < 0.5, keep_z=rng.random() < 0.3)
        return c
    T = _log_int(rng, 1, 131072 if op == "balance" else 65536)
    E = rng.choice((8, 16, 64, 100, 160, 256, 288, 384))
    return dict(op=op, T=T, E=E, k=rng.randint(1, 8), seqs=rng.randint(1, max(1, min(64, T // 2))),
                pad=rng.randint(0, T // 8), dropped=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs

COEF = 1e-2      # weight of the balance loss
RSF = 2.5        # routed scaling factor


def _offsets(case, gen):
    """seqs + 1 ascending offsets into T - pad rows; some sequences may be empty."""
    n = case["T"] - case["pad"]
    cuts = torch.randint(0, n + 1, (case["seqs"] - 1,), generator=gen)
    return torch.cat([torch.zeros(1, dtype=torch.int64), cuts.sort().values, torch.tensor([n])]).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s, scale=1.0: (torch.randn(*s, device="cuda", generator=g) * scale)  # noqa: E731
    op, T = case["op"], case["T"]
    s = dict(case=case)
    if op in ("linear", "linear_bwd"):
        K, N = case["K"], case["N"]
        s["x"] = rn(T, K).to(BF16)
        s["w"] = rn(N, K, scale=K ** -0.5).to(BF16)
        if op == "linear":
            s["bias"] = rn(N, scale=0.5).to(BF16) if case["bias"] else None
            s["residual"] = rn(T, N).to(BF16) if case["residual"] else None
            s["y"] = torch.empty(T, N, dtype=BF16, device="cuda")
            s["z_out"] = torch.empty(T, N, dtype=BF16, device="cuda") if case["keep_z"] else None
        else:
            s["dy"] = rn(T, N, scale=2.0 ** -6).to(BF16)
            s["z"] = rn(T, N).to(BF16) if case["act"] != "none" else None
            s["dx"] = torch.empty(T, K, dtype=BF16, device="cuda")
            s["dw"] = torch.empty(N, K, dtype=BF16, device="cuda")
            s["db"] = torch.empty(N, dtype=torch.float32, device="cuda") if case["bias"] else None
        return s
    E, k = case["E"], case["k"]
    host = torch.Generator().manual_seed(seed)
    logits = rn(T, E) + rn(E, scale=0.5)                  # some experts are favoured
    ids = (logits.sigmoid() + rn(E, scale=0.1)).topk(k, dim=1).indices.to(torch.int32)
    if case["dropped"]:                                   # assignments dropped for capacity are marked -1
        ids = torch.where(torch.rand(T, k, device="cuda", generator=g) < 0.03, torch.full_like(ids, -1), ids)
    s["logits"], s["ids"] = logits, ids.contiguous()
    s["seq_offsets"] = _offsets(case, host).cuda()
    B = case["seqs"]
    if op == "balance":
        s["counts"] = torch.empty(B, E, dtype=torch.int32, device="cuda")
        s["mean_scores"] = torch.empty(B, E, device="cuda")
        s["loss"] = torch.empty(B, device="cuda")
    else:
        s["counts"] = _counts(ids, s["seq_offsets"], T, E)
        # objective: mean over the sequences and tokens
        s["d_loss"] = (1.0 + rn(B, scale=0.1)) / B
        s["d_weights"] = rn(T, k, scale=1e-3 / T)
        s["d_logits"] = rn(T, E, scale=1e-5 / T)          # rows behind the last sequence stay as they are
    return s


# ------------------------------------------------------------------ plain forms

def _act(act, z):
    if act == "none":
        return z
    if act == "relu":
        return z * (z > 0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z / (1.0 + torch.exp(-z))


def _act_grad(act, z):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * z * z)
    s = 1.0 / (1.0 + torch.exp(-z))
    return s * (1.0 + z * (1.0 - s))


def _sequence_of(seq_offsets, T):
    """Sequence of every row, and whether the row belongs to one."""
    row = torch.arange(T, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(seq_offsets[1:].contiguous(), row, right=True)
    inside = (row >= seq_offsets[0]) & (row < seq_offsets[-1])
    return seq.clamp(max=seq_offsets.numel() - 2), inside


def _counts(ids, seq_offsets, T, E):
    B = seq_offsets.numel() - 1
    seq, inside = _sequence_of(seq_offsets, T)
    valid = (ids >= 0) & (ids < E) & inside[:, None]
    at = torch.where(valid, seq[:, None] * E + ids, B * E)       # the rest goes to a place of its own
    flat = torch.zeros(B * E + 1, dtype=torch.int32, device="cuda")
    flat.index_add_(0, at.reshape(-1).long(), torch.ones(at.numel(), dtype=torch.int32, device="cuda"))
    return flat[:-1].view(B, E)


def _plain_linear(s):
    c = s["case"]
    z = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act(c["act"], z)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    out = {"y": y.to(BF16)}
    if c["keep_z"]:
        out["z"] = z.to(BF16)
    return out


def _plain_linear_bwd(s):
    c = s["case"]
    dz = s["dy"].float()
    if c["act"] != "none":
        dz = dz * _act_grad(c["act"], s["z"].float())
    out = {"dx": (dz @ s["w"].float()).to(BF16), "dw": (dz.t() @ s["x"].float()).to(BF16)}
    if s["db"] is not None:
        out["db"] = dz.sum(0)
    return out


def _plain_balance(s):
    T, E = s["logits"].shape
    k, off = s["ids"].shape[1], s["seq_offsets"]
    row = torch.arange(T, device="cuda")
    member = ((row >= off[:-1, None]) & (row < off[1:, None])).float()          # [B, T]
    score = 1.0 / (1.0 + torch.exp(-s["logits"]))
    share = score / score.sum(1, keepdim=True)
    length = (off[1:] - off[:-1]).float().clamp(min=1.0)[:, None]
    mean = member @ share / length
    counts = _counts(s["ids"], off, T, E)
    loss = COEF * (counts.float() * (E / k) / length * mean).sum(1)
    return {"counts": counts, "mean_scores": mean, "loss": loss}


def _plain_router_bwd(s):
    logits, ids, off = s["logits"], s["ids"], s["seq_offsets"]
    T, E = logits.shape
    k = ids.shape[1]
    seq, inside = _sequence_of(off, T)
    length = (off[1:] - off[:-1]).float().clamp(min=1.0)
    score, rest = 1.0 / (1.0 + torch.exp(-logits)), 1.0 / (1.0 + torch.exp(logits))   # s and 1 - s
    total = score.sum(1, keepdim=True)
    load = (s["counts"].float() * (E / k) / length[:, None])[seq]                      # f of the row's sequence
    mean_load = (load * score).sum(1, keepdim=True) / total
    d_score = (s["d_loss"] * COEF / length)[seq][:, None] * (load - mean_load) / total
    # the routing weights: w_j = RSF s_j / sum_chosen s
    valid = (ids >= 0) & (ids < E)
    at = torch.where(valid, ids, 0).long()
    chosen = torch.where(valid, score.gather(1, at), 0.0)
    chosen_total = chosen.sum(1, keepdim=True)
    scale = torch.where(chosen_total > 0, RSF / chosen_total, 0.0)
    dw = torch.where(valid, s["d_weights"], 0.0)
    mean_dw = (dw * chosen).sum(1, keepdim=True) * scale / RSF
    d_score = d_score.scatter_add(1, at, torch.where(valid, scale * (dw - mean_dw), 0.0))
    return torch.where(inside[:, None], d_score * score * rest, s["d_logits"])


# ------------------------------------------------------------------ the library's calls

def _site_config(c):
    from routed_nvfp4_expert_b200 import capi
    return capi.SiteConfig(4096, 1024, 1024, c["E"], 0, c["E"], c["k"], RSF, 7.0)


def _own(s):
    from routed_nvfp4_expert_b200 import capi
    c = s["case"]
    op = c["op"]
    if op == "linear":
        if "ws" not in s:                                 # a program keeps one for its sizes
            s["ws"] = capi.alloc_linear_workspace(s["x"], s["w"])
        capi.linear_bf16(s["x"], s["w"], s["y"], s["ws"], bias=s["bias"], residual=s["residual"], act=c["act"],
                         z=s["z_out"])
        return {"y": s["y"], "z": s["z_out"]} if c["keep_z"] else {"y": s["y"]}
    if op == "linear_bwd":
        if "ws" not in s:
            s["ws"] = capi.alloc_linear_backward_workspace(s["dy"], s["x"], s["w"])
        capi.linear_bf16_backward(s["dy"], s["x"], s["w"], s["ws"], z=s["z"], act=c["act"], dx=s["dx"], dw=s["dw"],
                                  db=s["db"])
        out = {"dx": s["dx"], "dw": s["dw"]}
        if s["db"] is not None:
            out["db"] = s["db"]
        return out
    if "cfg" not in s:
        s["cfg"] = _site_config(c)
    if op == "balance":
        if "ws" not in s:
            s["ws"] = capi.alloc_balance_workspace(s["cfg"], c["T"], c["seqs"])
        capi.moe_balance_loss(s["cfg"], s["logits"], s["ids"], COEF, s["counts"], s["mean_scores"], s["loss"],
                              s["ws"], seq_offsets=s["seq_offsets"])
        return {"counts": s["counts"], "mean_scores": s["mean_scores"], "loss": s["loss"]}
    capi.moe_router_backward(s["cfg"], s["logits"], s["ids"], s["d_logits"], d_weights=s["d_weights"], coef=COEF,
                             counts=s["counts"], d_loss=s["d_loss"], seq_offsets=s["seq_offsets"])
    return s["d_logits"]


_PLAIN = {"linear": _plain_linear, "linear_bwd": _plain_linear_bwd, "balance": _plain_balance,
          "router_bwd": _plain_router_bwd}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ work

def work(case):
    T = case["T"]
    if case["op"] == "linear":
        K, N = case["K"], case["N"]
        sides = 1 + case["residual"] + case["keep_z"]
        return {"bytes": 2 * (T * K + N * K + sides * T * N + case["bias"] * N), "flops": 2 * T * K * N}
    if case["op"] == "linear_bwd":
        K, N = case["K"], case["N"]
        ins = T * N * (1 + (case["act"] != "none")) + T * K + N * K
        return {"bytes": 2 * (ins + T * K + N * K) + 4 * N * case["bias"], "flops": 4 * T * K * N}
    E, k, B = case["E"], case["k"], case["seqs"]
    rows = T - case["pad"]
    if case["op"] == "balance":
        return {"bytes": 4 * (rows * (E + k) + 2 * B * E + 2 * B + 1), "flops": 8 * rows * E}
    return {"bytes": 4 * (rows * (2 * E + 2 * k) + B * E + 2 * B + 1), "flops": 16 * rows * E}


# ------------------------------------------------------------------ 64 bits

def _act64(act, z):
    if act == "none":
        return z.clone()
    if act == "relu":
        return torch.maximum(z, torch.zeros_like(z))
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":            # (1 + tanh u) / 2 = sigmoid(2 u)
        return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    return z * torch.sigmoid(z)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        z = torch.zeros(1, case["N"], dtype=torch.float64, device="cuda") if s["bias"] is None else s["bias"].double()[None]
        z = torch.addmm(z, s["x"].double(), s["w"].double().T)
        y = _act64(case["act"], z)
        if s["residual"] is not None:
            y += s["residual"].double()
        return {"y": y, "z": z} if case["keep_z"] else {"y": y}
    if op == "linear_bwd":
        dz = s["dy"].double()
        if case["act"] != "none":
            z = s["z"].double().requires_grad_()
            (dz,) = torch.autograd.grad(_act64(case["act"], z), z, dz)
        out = {"dx": torch.mm(dz, s["w"].double()), "dw": torch.mm(dz.T, s["x"].double())}
        if s["db"] is not None:
            out["db"] = torch.mv(dz.T, torch.ones(case["T"], dtype=torch.float64, device="cuda"))
        return out
    T, E, k = case["T"], case["E"], case["k"]
    off = s["seq_offsets"].tolist()
    logits = s["logits"].double().requires_grad_()
    score = torch.sigmoid(logits)
    share = score / score.sum(1, keepdim=True)
    counts, means, losses = [], [], []
    for b in range(case["seqs"]):
        lo, hi = off[b], off[b + 1]
        ids = s["ids"][lo:hi]
        c = torch.bincount(ids[ids >= 0].reshape(-1), minlength=E)
        n = max(1, hi - lo)
        mean = share[lo:hi].sum(0) / n
        counts.append(c)
        means.append(mean)
        losses.append(COEF * torch.dot(c.double() * (E / (k * n)), mean))
    if op == "balance":
        return {"counts": torch.stack(counts).to(torch.int32), "mean_scores": torch.stack(means).detach(),
                "loss": torch.stack(losses).detach()}
    rows = off[-1]
    valid = (s["ids"] >= 0)[:rows]
    picked = torch.take_along_dim(score[:rows], s["ids"][:rows].long().clamp(min=0), 1) * valid
    total = picked.sum(1, keepdim=True)
    weights = RSF * picked / torch.where(total > 0, total, torch.ones_like(total))
    objective = torch.dot(torch.stack(losses), s["d_loss"].double()) + (weights * s["d_weights"][:rows].double()).sum()
    (grad,) = torch.autograd.grad(objective, logits)
    grad[rows:] = s["d_logits"][rows:].double()
    return grad
