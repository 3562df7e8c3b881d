"""What the losses of the output head are measured on.

Four operators on the hidden rows x [T, D] and the head's weights w [V, D], each
in its plain form (elementary torch operations, fp32) and as the package's call.
z[t, v] = x[t] . w[v] are the logits, which the package's calls never keep:

  loss        cross entropy: lse[t] - z[t, target[t]], with lse (head_loss)
  loss_bwd    its gradient to x and w, from upstream gradients of loss and lse
              (head_loss_bwd)
  distill     from a teacher's k top logits per token, at a temperature: the
              divergence of softmax(z / temperature) from the teacher's softmax
              over those k (head_distill)
  distill_bwd its gradient to x and w (head_distill_bwd)

Tokens without a target (-100), or without a teacher's entry (-1), do not count.
"""
import math

import torch

own = False


def listed():
    return [
        # the log-probability of one decoded token
        dict(name="loss one token", op="loss", T=1, D=2048, V=32768, pad=0.0),
        # a few candidates' tokens scored together, a vocabulary of odd size
        dict(name="loss few tokens", op="loss", T=50, D=4096, V=100003, pad=0.0),
        # a short tuning batch, half of it prompts without targets, odd sizes
        dict(name="loss odd", op="loss", T=1333, D=2064, V=50001, pad=0.5),
        # a training batch over a large vocabulary
        dict(name="loss training", op="loss", T=8192, D=4096, V=131072, pad=0.0),
        # the gradient of a short micro-batch
        dict(name="loss_bwd short", op="loss_bwd", T=96, D=2048, V=32768, pad=0.0, dlse=False),
        # a tuning batch with a z loss, odd sizes
        dict(name="loss_bwd odd", op="loss_bwd", T=1333, D=2064, V=50001, pad=0.5, dlse=True),
        # the training batch
        dict(name="loss_bwd training", op="loss_bwd", T=8192, D=4096, V=131072, pad=0.0, dlse=False),
        # a short sequence against eight entries of a teacher
        dict(name="distill short", op="distill", T=64, D=2048, V=32768, k=8, pad=0.0, temperature=1.0, type="fp32"),
        # a training batch against a teacher's 64 stored entries, in 16 bits
        dict(name="distill training", op="distill", T=8192, D=2048, V=131072, k=64, pad=0.1, temperature=2.0, type="bf16"),
        # an odd batch's gradient
        dict(name="distill_bwd odd", op="distill_bwd", T=777, D=1416, V=50001, k=20, pad=0.1, temperature=1.0, type="fp32"),
        # the training batch's
        dict(name="distill_bwd training", op="distill_bwd", T=8192, D=2048, V=131072, k=64, pad=0.1, temperature=2.0, type="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["loss", "loss_bwd", "distill", "distill_bwd"])
    while True:
        T, D, V = _log(rng, 1, 16384), 8 * _log(rng, 16, 1024), _log(rng, 512, 200000)
        if T * V <= 2 ** 30 and V * D <= 2 ** 29 and T * V * D <= 2 ** 41:
            break
    case = dict(op=op, T=T, D=D, V=V, pad=rng.choice([0.0, 0.1, 0.5]))
    if op == "loss_bwd":
        case["dlse"] = rng.random() < 0.5
    if op in ("distill", "distill_bwd"):
        case.update(k=_log(rng, 1, 128 if V > 20000 else 20), temperature=rng.choice([1.0, 2.0, 0.7]), type=rng.choice(["fp32", "bf16"]))
    return case


# ------------------------------------------------------------------ inputs --

def _counting(case):
    """Tokens that count: every sequence of 512 begins with its prompt."""
    at = torch.arange(case["T"], device="cuda") % 512
    return at >= int(case["pad"] * min(512, case["T"]))


def _teacher_entries(case, g):
    """k distinct tokens per row, the frequent ones (low numbers) more often, in
    an order of their own for each row, and descending logits; some rows have
    fewer entries, as where a teacher's small tail was cut off."""
    T, V, k = case["T"], case["V"], case["k"]
    edges = torch.maximum((V * (torch.arange(k + 1, device="cuda", dtype=torch.float64) / k) ** 2).long(), torch.arange(k + 1, device="cuda"))
    u = torch.rand(T, k, device="cuda", generator=g)
    index = torch.minimum(edges[:-1] + (u * (edges[1:] - edges[:-1])).long(), edges[1:] - 1)
    index = index.gather(1, torch.rand(T, k, device="cuda", generator=g).argsort(1))
    logits = (2.5 * torch.randn(T, k, device="cuda", generator=g) + 8.0).sort(1, descending=True).values
    kept = torch.where(torch.rand(T, 1, device="cuda", generator=g) < 0.2, 1 + (torch.rand(T, 1, device="cuda", generator=g) * k).long(), k)
    index[torch.arange(k, device="cuda") >= kept] = -1
    index[~_counting(case)] = -1
    return logits.to(torch.float32 if case["type"] == "fp32" else torch.bfloat16), index.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T, D, V = case["T"], case["D"], case["V"]
    w = (0.05 * torch.randn(V, D, device="cuda", generator=g)).to(torch.bfloat16)
    s = dict(op=case["op"], w=w)
    if case["op"].startswith("loss"):
        likely = (V * torch.rand(T, device="cuda", generator=g) ** 3).long().clamp_max(V - 1)
        s["targets"] = torch.where(_counting(case), likely, -100).to(torch.int32)
        n = max(1, int((s["targets"] >= 0).sum()))
    else:
        s["teacher"], s["index"] = _teacher_entries(case, g)
        s["temperature"] = case["temperature"]
        likely = s["index"][:, 0].long().clamp_min(0)
        n = max(1, int((s["index"][:, 0] >= 0).sum()))
    # logits of standard deviation 1.5, the likely token's up to log V + 4 above
    # them, as a model between its first steps and its last has them
    lift = torch.rand(T, 1, device="cuda", generator=g) * (math.log(V) + 4.0)
    x = torch.randn(T, D, device="cuda", generator=g) * (1.5 / (0.05 * math.sqrt(D))) + w[likely].float() * (lift / (0.0025 * D))
    s["x"] = x.to(torch.bfloat16)
    if case["op"].endswith("_bwd"):
        # what the forward returned, and the gradient of the tokens' mean
        s["dloss"] = torch.full((T,), 1.0 / n, device="cuda")
        z = torch.matmul(s["x"].float(), w.float().t())
        if case["op"] == "loss_bwd":
            s["lse"] = torch.logsumexp(z, 1)
            s["dlse"] = 2e-4 / n * s["lse"] if case["dlse"] else None
            s["lse"][s["targets"] < 0] = 0.0
        else:
            s["lse"] = torch.logsumexp(z / case["temperature"], 1)
            s["logits"] = z.gather(1, s["index"].long().clamp_min(0))
            s["logits"][s["index"] < 0] = 0.0
            s["lse"][(s["index"] < 0).all(1)] = 0.0
    return s


# ------------------------------------------------------------- plain forms --

def _logits(s):
    return torch.matmul(s["x"].float(), s["w"].float().t())


def _log_sum_exp(z):
    top = z.amax(1, keepdim=True)
    return (top + (z - top).exp().sum(1, keepdim=True).log()).squeeze(1)


def _loss(s):
    z = _logits(s)
    counts = s["targets"] >= 0
    zero = torch.zeros((), device=z.device)
    lse = torch.where(counts, _log_sum_exp(z), zero)
    logit = torch.where(counts, z.gather(1, s["targets"].long().clamp_min(0)[:, None]).squeeze(1), zero)
    return lse - logit, lse, logit


def _gradients(s, dz):
    return torch.matmul(dz, s["w"].float()).to(torch.bfloat16), torch.matmul(dz.t(), s["x"].float()).to(torch.bfloat16)


def _loss_bwd(s):
    counts = s["targets"] >= 0
    p = (_logits(s) - s["lse"][:, None]).exp()
    up = s["dloss"] if s["dlse"] is None else s["dloss"] + s["dlse"]
    dz = p * up[:, None]
    at = s["targets"].long().clamp_min(0)[:, None]
    dz.scatter_add_(1, at, -s["dloss"][:, None])
    return _gradients(s, torch.where(counts[:, None], dz, torch.zeros((), device=dz.device)))


def _teacher(s):
    """The teacher's probabilities, their logarithms (0 where there is no entry), and the rows that count."""
    there = s["index"] >= 0
    t = torch.where(there, s["teacher"].float() / s["temperature"], torch.full((), -math.inf, device="cuda"))
    counts = there.any(1)
    lse = torch.where(counts, _log_sum_exp(t), torch.zeros((), device="cuda"))
    log_q = torch.where(there, t - lse[:, None], torch.zeros((), device="cuda"))
    return torch.where(there, log_q.exp(), torch.zeros((), device="cuda")), log_q, counts


def _distill(s):
    q, log_q, counts = _teacher(s)
    z = _logits(s)
    zero = torch.zeros((), device=z.device)
    lse = torch.where(counts, _log_sum_exp(z / s["temperature"]), zero)
    logits = torch.where(s["index"] >= 0, z.gather(1, s["index"].long().clamp_min(0)), zero)
    return (q * (log_q + lse[:, None] - logits / s["temperature"])).sum(1), lse, logits


def _distill_bwd(s):
    q, _, counts = _teacher(s)
    up = (s["dloss"] / s["temperature"])[:, None]
    dz = (_logits(s) / s["temperature"] - s["lse"][:, None]).exp() * up
    dz.scatter_add_(1, s["index"].long().clamp_min(0), -q * up)
    return _gradients(s, torch.where(counts[:, None], dz, torch.zeros((), device=dz.device)))


def run(s):
    op = s["op"]
    if own:
        import moe_grouped_gemm_bf16_amd as mg
        if op == "loss":
            r = mg.head_loss(s["x"], s["w"], s["targets"])
            return r.loss, r.lse, r.logit
        if op == "loss_bwd":
            return mg.head_loss_bwd(s["x"], s["w"], s["targets"], s["lse"], s["dloss"], dlse=s["dlse"])
        if op == "distill":
            r = mg.head_distill(s["x"], s["w"], s["teacher"], s["index"], temperature=s["temperature"])
            return r.loss, r.lse, r.logits
        return mg.head_distill_bwd(s["x"], s["w"], s["teacher"], s["index"], s["lse"], s["logits"], s["dloss"], temperature=s["temperature"])
    return {"loss": _loss, "loss_bwd": _loss_bwd, "distill": _distill, "distill_bwd": _distill_bwd}[op](s)


# -------------------------------------------------------------------- work --

def work(case):
    T, D, V = case["T"], case["D"], case["V"]
    skip = int(case["pad"] * min(512, T))
    n = sum(max(0, min(512, T - b) - skip) for b in range(0, T, 512))   # tokens that count
    read = 2 * n * D + 2 * V * D
    entries = 4 * T if case["op"].startswith("loss") else T * case["k"] * (8 if case["type"] == "fp32" else 6)
    if case["op"].endswith("_bwd"):
        # logits, gradient to x, gradient to w; lse, dloss and the entries' logits come in
        more = (12 if case["dlse"] else 8) * T if case["op"] == "loss_bwd" else 8 * T + 4 * T * case["k"]
        return {"bytes": read + entries + more + 2 * T * D + 2 * V * D, "flops": 6.0 * n * D * V}
    out = 12 * T if case["op"] == "loss" else 8 * T + 4 * T * case["k"]
    return {"bytes": read + entries + out, "flops": 2.0 * n * D * V}


# ------------------------------------------------------------------- exact --

def exact(case, seed):
    """From the definitions, in 64 bits, over pieces of the tokens."""
    s = prepare(case, seed)
    T = case["T"]
    f64 = torch.float64
    W = s["w"].to(f64)
    step = max(1, 2 ** 29 // case["V"])
    backward = case["op"].endswith("_bwd")
    tau = s.get("temperature", 1.0)
    parts, dW = [], torch.zeros_like(W) if backward else None
    for b in range(0, T, step):
        X = s["x"][b:b + step].to(f64)
        z = X @ W.T
        rows = torch.arange(len(X), device="cuda")
        # target distribution over the entries (index [n, j], weight [n, j])
        if case["op"].startswith("loss"):
            at = s["targets"][b:b + step].long()[:, None]
            q = (at >= 0).to(f64)
        else:
            at = s["index"][b:b + step].long()
            t = (s["teacher"][b:b + step].to(f64) / tau).masked_fill(at < 0, -1e300)
            q = torch.softmax(t, 1) * (at >= 0)
        live = (at >= 0).any(1)
        if backward:
            lse = s["lse"][b:b + step].to(f64)
            up = s["dloss"][b:b + step].to(f64) / tau
            dense = up if s.get("dlse") is None else up + s["dlse"][b:b + step].to(f64)
            dz = torch.exp(z / tau - lse[:, None]) * (dense * live)[:, None]
            r = rows[:, None].expand_as(at)[at >= 0]
            dz.index_put_((r, at[at >= 0]), -(q * up[:, None])[at >= 0], accumulate=True)
            dW += dz.T @ X
            parts.append((dz @ W,))
        else:
            lse = torch.logsumexp(z / tau, 1) * live
            zk = torch.where(at >= 0, z[rows[:, None], at.clamp_min(0)], torch.zeros((), dtype=f64, device="cuda"))
            loss = (torch.xlogy(q, q) + q * (lse[:, None] - zk / tau)).sum(1)
            parts.append((loss, lse, zk[:, 0] if case["op"] == "loss" else zk))
        del z
    whole = tuple(torch.cat(p) for p in zip(*parts))
    return whole + (dW,) if backward else whole
