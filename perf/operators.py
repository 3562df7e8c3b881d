"""What the MoE layer's routing and 8-bit operators are measured on.

Six operators, each in its plain form (elementary torch operations, fp32 or
wider) and as the package's call:

  fwd        y[i] = x[i] W[e]^T on E4M3 codes, one fp32 scale per row and 128
             columns of x, one per 128 x 128 block of W (moe fwd_fp8)
  dgrad      dx[i] = dy[i] W[e] on the same weights (dgrad_fp8)
  quantize   bf16 or fp32 values to such codes and scales: rows, rows gathered
             by index, silu(g) u of a gate-up product, or weights
             (fp8_quantize, fp8_quantize_swiglu, fp8_quantize_weights)
  route      logits to top-k experts and weights, the row order of the grouped
             products, per-expert counts, balance and z losses (moe_route)
  route_bwd  gradient of the weights and of both losses to the logits
             (moe_route_bwd)
  combine_bwd  gradient of the weighted combine of routed rows to the rows and
             to the weights (moe_combine_bwd)
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
AMAX_MIN = 2.0 ** -100


def listed():
    return [
        # one decoded token of a top-8 layer: eight experts with one row each
        dict(name="fwd one token", op="fwd", E=64, M=8, N=768, K=2048, rows="few"),
        # a prefill or training batch through the gate-up weights
        dict(name="fwd training", op="fwd", E=32, M=32768, N=4096, K=2048, rows="router"),
        # the uniform eight-group shape of the package's benchmark
        dict(name="dgrad uniform", op="dgrad", E=8, M=32768, N=768, K=2048, rows="even"),
        # a skewed split with empty experts, widths that end inside a tile
        dict(name="dgrad skewed", op="dgrad", E=16, M=5003, N=1408, K=2064, rows="zipf"),
        # a decoded batch's activations
        dict(name="quantize few rows", op="quantize", form="rows", M=64, K=2048, T=64, type="bf16"),
        # the SwiGLU between two 8-bit products of a training batch
        dict(name="quantize swiglu", op="quantize", form="swiglu", M=32768, K=2048, T=0, type="bf16"),
        # one decoding step's router
        dict(name="route decode", op="route", T=16, E=128, k=8, type="fp32", normalize=True, pad=0.0, off=0),
        # a training batch, padded at its end, two experts switched off
        dict(name="route training", op="route", T=65536, E=256, k=8, type="fp32", normalize=True, pad=0.03, off=2),
        # a short odd batch with 16-bit logits
        dict(name="route_bwd odd", op="route_bwd", T=1333, E=60, k=4, type="bf16", normalize=False, pad=0.1, off=0),
        # the training batch
        dict(name="route_bwd training", op="route_bwd", T=65536, E=256, k=8, type="fp32", normalize=True, pad=0.03, off=2),
        # a small batch with a third of the rows on other ranks
        dict(name="combine_bwd small", op="combine_bwd", T=100, D=2048, k=8, weights=True, absent=0.3),
        # a training batch's output combine
        dict(name="combine_bwd training", op="combine_bwd", T=8192, D=2048, k=8, weights=True, absent=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "dgrad", "quantize", "route", "route_bwd", "combine_bwd"])
    if op in ("fwd", "dgrad"):
        while True:
            E = _log(rng, 2, 128)
            M = _log(rng, 1, 32768)
            N = 16 * _log(rng, 4, 256)
            K = 16 * _log(rng, 4, 448)
            if E * N * K <= 2 ** 28 and M * N * K <= 2 ** 38:
                break
        return dict(op=op, E=E, M=M, N=N, K=K, rows=rng.choice(["router", "zipf", "even", "few"]))
    if op == "quantize":
        form = rng.choice(["rows", "gather", "swiglu", "weights"])
        K = 16 * _log(rng, 4, 448)
        M = _log(rng, 1, min(32768, 2 ** 26 // K))
        if form == "weights":
            return dict(op=op, form=form, M=_log(rng, 1, 32), K=K, T=16 * _log(rng, 1, 128), type=rng.choice(["bf16", "fp32"]))
        T = max(1, M // rng.choice([1, 2, 8])) if form == "gather" else M
        return dict(op=op, form=form, M=M, K=K, T=T, type="bf16" if form == "swiglu" else rng.choice(["bf16", "fp32"]))
    if op in ("route", "route_bwd"):
        E = _log(rng, 4, 512)
        return dict(op=op, T=_log(rng, 1, min(65536, 2 ** 24 // E)), E=E, k=rng.randint(1, min(E // 2, 10)), type=rng.choice(["fp32", "bf16"]),
                    normalize=rng.random() < 0.5, pad=rng.choice([0.0, 0.2]), off=rng.choice([0, 0, 1]))
    k = rng.randint(1, 10)
    D = 8 * _log(rng, 8, 896)
    return dict(op=op, T=_log(rng, 1, min(16384, 2 ** 27 // (D * k))), D=D, k=k, weights=rng.random() < 0.8, absent=rng.choice([0.0, 0.3]))


# ------------------------------------------------------------------ inputs --

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _sizes(case, seed):
    """Rows per expert: `even`, as a router with learned preferences deals them,
    `zipf` with empty experts, or `few` experts of one or a few rows."""
    E, M = case["E"], case["M"]
    r = np.random.RandomState(seed % (1 << 31))
    if case["rows"] == "even":
        n = np.full(E, M // E)
        n[: M - n.sum()] += 1
    elif case["rows"] == "few":
        n = np.bincount(r.permutation(E)[np.arange(M) % min(E, max(8, E // 4))], minlength=E)
    else:
        w = np.exp(0.3 * r.randn(E)) if case["rows"] == "router" else r.permutation(np.arange(1, E + 1) ** -1.2 * (np.arange(E) < max(1, E - E // 8)))
        n = np.bincount(r.choice(E, M, p=w / w.sum()), minlength=E)
    return [int(v) for v in n]


def _offsets(sizes):
    return torch.tensor(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32), device="cuda")


def _activations(g, M, K):
    """Rows of differing size with a few columns that stand out."""
    x = torch.randn(M, K, device="cuda", generator=g)
    x *= torch.exp(0.5 * torch.randn(M, 1, device="cuda", generator=g)) * torch.exp(0.7 * torch.randn(K, device="cuda", generator=g))
    return x


def _scales(amax):
    """A block's scale and its inverse, each one correctly rounded division
    (a Python number as an operand would be turned into a product)."""
    amax = amax.clamp_min(AMAX_MIN)
    top = torch.full_like(amax, E4M3_MAX)
    return amax / top, top / amax


def _row_codes(x):
    """fp32 [M, K] -> (E4M3 values [M, K], scales fp32 [ceil(K/128), M])."""
    M, K = x.shape
    nb = -(-K // 128)
    blocks = torch.nn.functional.pad(x, (0, nb * 128 - K)).view(M, nb, 128)
    scale, inv = _scales(blocks.abs().amax(2))
    q = (blocks * inv[:, :, None]).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(M, nb * 128)[:, :K].contiguous().view(torch.float8_e4m3fn), scale.t().contiguous()


def _weight_codes(w):
    """fp32 [E, N, K] -> (E4M3 values, scales fp32 [E, ceil(N/128), ceil(K/128)])."""
    E, N, K = w.shape
    nn, nk = -(-N // 128), -(-K // 128)
    b = torch.nn.functional.pad(w, (0, nk * 128 - K, 0, nn * 128 - N)).view(E, nn, 128, nk, 128)
    scale, inv = _scales(b.abs().amax((2, 4)))
    q = (b * inv[:, :, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(E, nn * 128, nk * 128)
    return q[:, :N, :K].contiguous().view(torch.float8_e4m3fn), scale


def _product_inputs(case, seed):
    E, M, N, K = (case[c] for c in "EMNK")
    g = _gen(seed)
    q, s = _row_codes(_activations(g, M, K if case["op"] == "fwd" else N))
    w8 = torch.empty(E, N, K, dtype=torch.uint8, device="cuda")
    ws = torch.empty(E, -(-N // 128), -(-K // 128), device="cuda")
    step = max(1, 2 ** 26 // (N * K))
    for e in range(0, E, step):
        c, ws[e:e + step] = _weight_codes(torch.randn(min(step, E - e), N, K, device="cuda", generator=g) * K ** -0.5)
        w8[e:e + step] = c.view(torch.uint8)
    sizes = _sizes(case, seed)
    return dict(q=q.view(torch.uint8), s=s, w8=w8, ws=ws, sizes=sizes, offsets=_offsets(sizes))


def _quantize_inputs(case, seed):
    g = _gen(seed)
    M, K, T = case["M"], case["K"], case["T"]
    t = torch.float32 if case["type"] == "fp32" else torch.bfloat16
    if case["form"] == "weights":
        return dict(x=(torch.randn(M, T, K, device="cuda", generator=g) * K ** -0.5).to(t))
    if case["form"] == "swiglu":
        return dict(x=_activations(g, M, 2 * K).to(t))
    x = _activations(g, T, K)
    x[torch.rand(T, device="cuda", generator=g) < 0.02] = 0.0      # padding tokens
    s = dict(x=x.to(t))
    if case["form"] == "gather":
        s["gather"] = torch.randint(0, T, (M,), device="cuda", generator=g, dtype=torch.int32)
    return s


def _router_inputs(case, seed):
    T, E = case["T"], case["E"]
    g = _gen(seed)
    logits = 1.5 * torch.randn(T, E, device="cuda", generator=g) + 0.5 * torch.randn(E, device="cuda", generator=g)
    logits = logits.to(torch.float32 if case["type"] == "fp32" else torch.bfloat16)
    if case["off"]:
        logits[:, torch.randperm(E, device="cuda", generator=g)[:case["off"]]] = -math.inf
    mask = None
    if case["pad"]:
        mask = torch.ones(T, dtype=torch.bool, device="cuda")
        mask[T - int(case["pad"] * T):] = False
    return dict(logits=logits, mask=mask)


def prepare(case, seed):
    op = case["op"]
    if op in ("fwd", "dgrad"):
        s = _product_inputs(case, seed)
    elif op == "quantize":
        s = _quantize_inputs(case, seed)
    elif op == "route":
        s = _router_inputs(case, seed)
    elif op == "route_bwd":
        s = _router_inputs(case, seed)
        s["case"] = case
        # what the forward left
        w, experts, lse, counts, _, tokens = _gate(s)[:6]
        g = _gen(seed + 1)
        s.update(weights=w, experts=experts, lse=lse, counts=counts, tokens=tokens,
                 dweights=torch.randn(case["T"], case["k"], device="cuda", generator=g) / case["T"],
                 dloss=torch.tensor([1e-2, 1e-3], device="cuda"))
    else:
        g = _gen(seed)
        T, D, k = case["T"], case["D"], case["k"]
        M = T * k
        order = torch.randperm(M, device="cuda", generator=g)
        token_rows = order.to(torch.int32).view(T, k)
        if case["absent"]:
            token_rows = torch.where(torch.rand(T, k, device="cuda", generator=g) < case["absent"], -1, token_rows)
        s = dict(dout=torch.randn(T, D, device="cuda", generator=g).bfloat16(), rows=torch.randn(M, D, device="cuda", generator=g).bfloat16(),
                 token_rows=token_rows.contiguous(), weights=torch.softmax(torch.randn(T, k, device="cuda", generator=g), 1) if case["weights"] else None,
                 # (the spare row takes what the plain form writes for absent rows)
                 drows=torch.zeros(M + 1, D, dtype=torch.bfloat16, device="cuda"))
    s["case"] = case
    return s


# -------------------------------------------------------------- plain forms --

def _plain_product(s):
    """One product per expert on the dequantised operands."""
    case, forward = s["case"], s["case"]["op"] == "fwd"
    N, K = case["N"], case["K"]
    x = s["q"].view(torch.float8_e4m3fn).float()
    x *= s["s"].t().repeat_interleave(128, 1)[:, :x.shape[1]]
    out = torch.empty(case["M"], N if forward else K, dtype=torch.bfloat16, device="cuda")
    at = 0
    for e, n in enumerate(s["sizes"]):
        if n == 0:
            continue
        w = s["w8"][e].view(torch.float8_e4m3fn).float()
        w *= s["ws"][e].repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
        out[at:at + n] = (x[at:at + n] @ (w.t() if forward else w)).bfloat16()
        at += n
    return out


def _plain_quantize(s):
    case = s["case"]
    if case["form"] == "weights":
        return list(_weight_codes(s["x"].float()))
    if case["form"] == "swiglu":
        g, u = s["x"].float().chunk(2, 1)
        return list(_row_codes(g / (1 + torch.exp(-g)) * u))
    return list(_row_codes((s["x"][s["gather"].long()] if case["form"] == "gather" else s["x"]).float()))


def _gate(s):
    """weights, experts, lse, counts, prob_sum, tokens, z_sum, probabilities."""
    case = s["case"]
    T, E, k = case["T"], case["E"], case["k"]
    l = s["logits"].float()
    live = torch.isfinite(l).any(1) if s["mask"] is None else s["mask"] & torch.isfinite(l).any(1)
    l = torch.where(live[:, None], l, -math.inf)
    top, experts = torch.sort(l, dim=1, descending=True, stable=True)
    top, experts = top[:, :k], experts[:, :k].to(torch.int32)
    high = torch.where(live, top[:, 0], 0.0)
    ex = torch.exp(l - high[:, None])
    total = ex.sum(1)
    p = ex / torch.where(live, total, 1.0)[:, None]
    lse = torch.where(live, high + torch.log(total), 0.0)
    chosen = torch.isfinite(top)
    experts = torch.where(chosen, experts, -1)
    w = torch.exp(top - high[:, None])
    w = w / torch.where(live, w.sum(1) if case["normalize"] else total, 1.0)[:, None]
    counts = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    counts = counts.index_add_(0, torch.where(chosen, experts, E).view(-1), torch.ones(T * k, dtype=torch.int32, device="cuda"))[:E]
    return w, experts, lse, counts, p.double().sum(0).float(), live.sum().to(torch.int32).view(1), lse.double().square().sum(), p


def _plain_route(s):
    case = s["case"]
    T, E, k = case["T"], case["E"], case["k"]
    w, experts, lse, counts, psum, tokens, zsum, _ = _gate(s)
    n = tokens.double().clamp_min(1)
    balance = E * (counts.double() * psum.double()).sum() / counts.double().sum().clamp_min(1) / n
    loss = torch.stack([balance.view(()), (zsum / n).view(())]).float()
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), counts.cumsum(0)]).to(torch.int32)
    flat = experts.view(-1).long()
    key, order = torch.sort(torch.where(flat < 0, E, flat), stable=True)
    gather = torch.where(key < E, order // k, -1).to(torch.int32)
    rows = torch.empty_like(order)
    rows[order] = torch.arange(T * k, device="cuda")
    return [w, experts, lse, counts, psum, tokens, loss, offsets, gather, torch.where(flat < 0, -1, rows).to(torch.int32).view(T, k)]


def _plain_route_bwd(s):
    case = s["case"]
    E = case["E"]
    live = s["experts"][:, :1] >= 0
    l = s["logits"].float()
    p = torch.where(live, torch.exp(l - s["lse"][:, None]), 0.0)
    n = s["tokens"].float()
    c = s["counts"].float() * (E / s["counts"].sum() / n * s["dloss"][0])
    d = p * (c - (p * c).sum(1, keepdim=True) + 2 * s["dloss"][1] / n * s["lse"][:, None])
    at = s["experts"].long().clamp_min(0)
    dw = torch.where(s["experts"] >= 0, s["dweights"], 0.0)
    dot = (dw * s["weights"]).sum(1, keepdim=True)
    if case["normalize"]:
        d.scatter_add_(1, at, s["weights"] * (dw - dot))
    else:
        d -= p * dot
        d.scatter_add_(1, at, s["weights"] * dw)
    return d.to(s["logits"].dtype)


def _plain_combine_bwd(s):
    case = s["case"]
    T, k, D = case["T"], case["k"], case["D"]
    flat = s["token_rows"].view(-1).long()
    w = s["weights"].view(-1) if s["weights"] is not None else torch.ones(T * k, device="cuda")
    dout = s["dout"].float()
    s["drows"][torch.where(flat < 0, T * k, flat)] = (w.view(T, k, 1) * dout[:, None]).bfloat16().view(T * k, D)
    drows = s["drows"][:T * k]
    if s["weights"] is None:
        return [drows]
    dot = (s["rows"][flat.clamp_min(0)].float().view(T, k, D) * dout[:, None]).sum(2)
    return [drows, torch.where(s["token_rows"] >= 0, dot, 0.0)]


# --------------------------------------------------------------- the calls --

def _own(s):
    import moe_grouped_gemm_bf16_amd as mg
    case = s["case"]
    op = case["op"]
    if op == "fwd":
        return mg.fwd_fp8(s["q"], s["s"], s["w8"], s["ws"], s["offsets"])
    if op == "dgrad":
        return mg.dgrad_fp8(s["q"], s["s"], s["w8"], s["ws"], s["offsets"])
    if op == "quantize":
        if case["form"] == "weights":
            q, scale = mg.fp8_quantize_weights(s["x"])
        elif case["form"] == "swiglu":
            q, scale = mg.fp8_quantize_swiglu(s["x"])
        else:
            q, scale = mg.fp8_quantize(s["x"], gather=s.get("gather"))
        return [q.view(torch.float8_e4m3fn), scale]
    if op == "route":
        r = mg.moe_route(s["logits"], case["k"], normalize=case["normalize"], mask=s["mask"])
        return [r.weights, r.experts, r.lse, r.counts, r.prob_sum, r.tokens, r.loss, r.offsets, r.gather, r.token_rows]
    if op == "route_bwd":
        return mg.moe_route_bwd(s["logits"], s["weights"], s["experts"], s["lse"], s["counts"], s["tokens"], dweights=s["dweights"],
                                dloss=s["dloss"], normalize=case["normalize"])
    drows, dweights = mg.moe_combine_bwd(s["dout"], s["rows"], s["token_rows"], s["weights"], drows=s["drows"][:-1])
    return [drows] if dweights is None else [drows, dweights]


def run(s):
    if own:
        return _own(s)
    op = s["case"]["op"]
    if op in ("fwd", "dgrad"):
        return _plain_product(s)
    return {"quantize": _plain_quantize, "route": _plain_route, "route_bwd": _plain_route_bwd, "combine_bwd": _plain_combine_bwd}[op](s)


def work(case):
    op = case["op"]
    if op in ("fwd", "dgrad"):
        E, M, N, K = (case[c] for c in "EMNK")
        # experts with rows: the others' weights are not needed
        if case["rows"] in ("even", "few"):
            live = min(E, M) if case["rows"] == "even" else min(M, E, max(8, E // 4))
        else:
            share = np.full(E, 1.0 / E) if case["rows"] == "router" else np.arange(1, E + 1) ** -1.2 * (np.arange(E) < max(1, E - E // 8))
            live = float((1 - (1 - share / share.sum()) ** M).sum())
        nn, nk = -(-N // 128), -(-K // 128)
        inner, outer = (K, N) if op == "fwd" else (N, K)
        return {"bytes": live * (N * K + 4 * nn * nk) + M * inner + 4 * M * -(-inner // 128) + 2 * M * outer + 4 * (E + 1), "flops": 2 * M * N * K}
    if op == "quantize":
        M, K, T = case["M"], case["K"], case["T"]
        size = 4 if case["type"] == "fp32" else 2
        if case["form"] == "weights":
            return {"bytes": M * T * K * (size + 1) + 4 * M * -(-T // 128) * -(-K // 128), "flops": 2 * M * T * K}
        read = M * 2 * K * size if case["form"] == "swiglu" else min(M, T) * K * size
        return {"bytes": read + M * K + 4 * M * -(-K // 128) + (4 * M if case["form"] == "gather" else 0), "flops": (8 if case["form"] == "swiglu" else 2) * M * K}
    if op in ("route", "route_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        size = 4 if case["type"] == "fp32" else 2
        if op == "route":
            return {"bytes": T * E * size + T * (4 * k * 4 + 4) + (T if case["pad"] else 0) + 12 * E, "flops": T * E * (4 + k)}
        return {"bytes": 2 * T * E * size + T * (3 * 4 * k + 4) + 4 * E, "flops": 8 * T * E}
    T, D, k = case["T"], case["D"], case["k"]
    live = T * k * (1 - case["absent"])
    return {"bytes": 2 * T * D + live * D * (4 if case["weights"] else 2) + T * k * (12 if case["weights"] else 4), "flops": live * D * (3 if case["weights"] else 1)}


# ------------------------------------------------- the definitions, 64 bits --

def _decode(codes):
    """E4M3 codes (uint8) to float64, by their bit fields."""
    c = np.arange(256)
    m, e = c & 7, (c >> 3) & 15
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v[(c & 127) == 127] = np.nan
    return torch.tensor(np.where(c >= 128, -v, v), device="cuda")[codes.int()]


def _encode(v):
    """float64 to the nearest E4M3 value (ties to an even mantissa)."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_product(s):
    case = s["case"]
    forward = case["op"] == "fwd"
    M, N, K = case["M"], case["N"], case["K"]
    inner = K if forward else N
    col = torch.arange(inner, device="cuda") // 128
    out = torch.empty(M, N if forward else K, dtype=torch.float64, device="cuda")
    bounds = s["offsets"].tolist()
    n_block, k_block = torch.arange(N, device="cuda") // 128, torch.arange(K, device="cuda") // 128
    for e in range(case["E"]):
        lo, hi = bounds[e], bounds[e + 1]
        if lo == hi:
            continue
        x = _decode(s["q"][lo:hi]) * s["s"].double()[col, lo:hi].t()
        w = _decode(s["w8"][e]) * s["ws"][e].double()[n_block][:, k_block]
        out[lo:hi] = torch.mm(x, w.t().contiguous() if forward else w)
    return out


def _exact_blocks(v, group):
    """Codes' values and scales of v [..., n, K], one scale per 128 columns and `group` rows."""
    *lead, n, K = v.shape
    row, col = torch.arange(n, device="cuda") // group, torch.arange(K, device="cuda") // 128
    amax = torch.zeros(*lead, int(row[-1]) + 1, int(col[-1]) + 1, dtype=torch.float64, device="cuda")
    for b in range(int(col[-1]) + 1):
        part = v[..., 128 * b:128 * b + 128].abs().amax(-1)
        if group == 1:
            amax[..., b] = part
        else:
            amax[..., b] = torch.nn.functional.pad(part, (0, -n % group)).view(*lead, -1, group).amax(-1)
    amax = amax.clamp_min(AMAX_MIN)
    # a scale and its inverse are fp32 numbers by definition, their product with a value too
    inv = (E4M3_MAX / amax).float()
    full = inv if group == 1 else inv[..., row, :]
    return _encode((v.float() * full[..., col]).double()), amax / E4M3_MAX


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("fwd", "dgrad"):
        return _exact_product(s)
    if op == "quantize":
        x = s["x"].double()
        if case["form"] == "weights":
            return list(_exact_blocks(x, 128))
        if case["form"] == "swiglu":
            g, u = x[:, :case["K"]], x[:, case["K"]:]
            x = g * torch.sigmoid(g) * u
        elif case["form"] == "gather":
            x = x[s["gather"].long()]
        q, scale = _exact_blocks(x, 1)
        return [q, scale.t().contiguous()]
    if op == "combine_bwd":
        T, D, k = case["T"], case["D"], case["k"]
        dout, drows = s["dout"].double(), torch.zeros(T * k, D, dtype=torch.float64, device="cuda")
        dweights = torch.zeros(T, k, dtype=torch.float64, device="cuda")
        for j in range(k):
            t = torch.nonzero(s["token_rows"][:, j] >= 0).view(-1)
            r = s["token_rows"][t, j].long()
            drows[r] = dout[t] * (s["weights"][t, j].double()[:, None] if case["weights"] else 1.0)
            dweights[t, j] = (s["rows"][r].double() * dout[t]).sum(1)
        return [drows, dweights] if case["weights"] else [drows]
    l = s["logits"].double()
    T, E = l.shape
    live = torch.isfinite(l).any(1)
    if s["mask"] is not None:
        live &= s["mask"]
    p = torch.zeros_like(l)
    p[live] = torch.softmax(l[live], 1)
    lse = torch.zeros(T, dtype=torch.float64, device="cuda")
    lse[live] = torch.logsumexp(l[live], 1)
    n = max(1, int(live.sum()))
    if op == "route_bwd":
        experts, got = s["experts"].long(), s["experts"] >= 0
    else:
        experts = torch.argsort(-torch.where(live[:, None], l, -math.inf), dim=1, stable=True)[:, :case["k"]]
        got = live[:, None] & torch.isfinite(torch.gather(l, 1, experts))
    w = torch.where(got, torch.gather(p, 1, experts.clamp_min(0)), 0.0)
    total = w.sum(1, keepdim=True).clamp_min(1e-300)
    if case["normalize"]:
        w = w / total
    counts = torch.bincount(experts[got], minlength=E).double()
    share = counts / counts.sum().clamp_min(1)
    if op == "route":
        loss = torch.stack([E * (share * p.sum(0) / n).sum(), lse.square().sum() / n])
        return [w, None, lse, None, p.sum(0), None, loss, None, None, None]
    # gradient with respect to the probabilities, then through the softmax
    dw = torch.where(got, s["dweights"].double(), 0.0)
    if case["normalize"]:
        dw = (dw - (dw * w).sum(1, keepdim=True)) / total
    dp = (E * share / n * s["dloss"].double()[0]).expand(T, E).clone()
    dp.scatter_add_(1, experts.clamp_min(0), torch.where(got, dw, 0.0))
    return p * (dp - (p * dp).sum(1, keepdim=True) + 2 * lse[:, None] / n * s["dloss"].double()[1])
