"""Plain 64-bit references of the block-scaled fp8 operators and of the router
(test infrastructure; NumPy only, no code of the library)."""
import numpy as np

TOP = 448.0
FLOOR = 2.0 ** -100
BLOCK = 128


def e4m3_values():
    """The 256 codes' values by their bit fields (bias 7; S.1111.111 is NaN)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v = np.where(c >= 128, -v, v)
    v[(c & 127) == 127] = np.nan
    return v


def encode(v):
    """float64 values (|v| <= 448 (1 + 2^-20)) to E4M3 codes, to nearest even."""
    v = np.asarray(v, np.float64)
    a = np.abs(v)
    with np.errstate(divide="ignore", invalid="ignore"):
        step = np.exp2(np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
        q = np.minimum(np.rint(a / step) * step, TOP)            # rint: half to even
    table = e4m3_values()[:127]
    code = np.searchsorted(table, np.where(np.isnan(q), 0, q)).astype(np.uint8)
    code = np.where(np.isnan(q), 127, code).astype(np.uint8)
    return (code | (np.signbit(v).astype(np.uint8) << 7)).astype(np.uint8)


def quantize(x, group):
    """fp32 values [n, K] to (codes, scales [ceil(n/group), ceil(K/128)]): one
    scale per `group` rows and 128 columns, in the operator's fp32 arithmetic."""
    x = np.asarray(x, np.float32)
    n, K = x.shape
    nr, nb = -(-n // group), -(-K // BLOCK)
    codes = np.zeros((n, K), np.uint8)
    scales = np.zeros((nr, nb), np.float32)
    for r in range(nr):
        for b in range(nb):
            blk = x[r * group:(r + 1) * group, b * BLOCK:(b + 1) * BLOCK]
            a = np.float32(max(np.nanmax(np.abs(blk)) if not np.isnan(blk).all() else 0.0, FLOOR))
            with np.errstate(invalid="ignore"):
                scales[r, b] = a / np.float32(TOP)
                inv = np.float32(TOP) / a
                codes[r * group:(r + 1) * group, b * BLOCK:(b + 1) * BLOCK] = encode((blk * inv).astype(np.float64))
    return codes, scales


def dequant_rows(codes, scales):
    """codes [M, K], scales [ceil(K/128), M] -> float64 [M, K]."""
    K = codes.shape[1]
    return e4m3_values()[codes] * np.repeat(scales.astype(np.float64).T, BLOCK, 1)[:, :K]


def dequant_weights(codes, scales):
    """codes [E, N, K], scales [E, ceil(N/128), ceil(K/128)] -> float64."""
    _, N, K = codes.shape
    s = np.repeat(np.repeat(scales.astype(np.float64), BLOCK, 1)[:, :N], BLOCK, 2)[:, :, :K]
    return e4m3_values()[codes] * s


def product(q, w, off, dgrad):
    """Rows q [M, R] and weights w [E, N, K] (float64) -> (sums, sums of magnitudes)."""
    E, N, K = w.shape
    P = K if dgrad else N
    out, mag = np.zeros((q.shape[0], P)), np.zeros((q.shape[0], P))
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        m = w[e] if dgrad else w[e].T
        out[lo:hi] = q[lo:hi] @ m
        mag[lo:hi] = np.abs(q[lo:hi]) @ np.abs(m)
    return out, mag


def route(logits, k, normalize, mask=None, first=0, local=None):
    """Every output of the router, float64 and int64."""
    l = np.array(logits, np.float64)
    T, E = l.shape
    local = E - first if local is None else local
    l = np.where(np.isnan(l), -np.inf, np.minimum(l, np.finfo(np.float32).max))
    live = (l > -np.inf).any(1)
    if mask is not None:
        live &= np.asarray(mask).astype(bool)
    l[~live] = -np.inf
    top = np.where(live, l.max(1, initial=-np.inf), 0.0)
    with np.errstate(divide="ignore"):
        ex = np.exp(l - top[:, None])
        s = ex.sum(1)
        lse = np.where(live, top + np.log(np.where(live, s, 1.0)), 0.0)
    p = ex / np.where(live, s, 1.0)[:, None]
    order = np.argsort(-l, axis=1, kind="stable")[:, :k]
    got = np.take_along_axis(l, order, 1) > -np.inf
    experts = np.where(got, order, -1)
    w = np.where(got, np.take_along_axis(p, order, 1), 0.0)
    if normalize:
        # (from the exponentials: a sum of probabilities could underflow)
        we = np.where(got, np.take_along_axis(ex, order, 1), 0.0)
        w = we / np.where(live, we.sum(1), 1.0)[:, None]
    counts = np.bincount(experts[got], minlength=E)
    n = int(live.sum())
    psum = p.sum(0)
    balance = E * (counts / max(1, counts.sum()) * psum / max(1, n)).sum()
    z = (lse ** 2).sum() / max(1, n)
    off = np.concatenate([[0], np.cumsum(counts[first:first + local])])
    flat = experts.reshape(-1)
    here = (flat >= first) & (flat < first + local)
    idx = np.nonzero(here)[0]
    rows_order = idx[np.argsort(flat[idx], kind="stable")]
    gather = np.full(T * k, -1, np.int64)
    gather[:len(rows_order)] = rows_order // k
    token_rows = np.full(T * k, -1, np.int64)
    token_rows[rows_order] = np.arange(len(rows_order))
    return dict(weights=w, experts=experts, lse=lse, counts=counts, prob_sum=psum, tokens=np.array([n]), loss=np.array([balance, z]),
                offsets=off, gather=gather, token_rows=token_rows.reshape(T, k), p=p, live=live)


def route_loss(logits, r, dw, dloss, normalize):
    """The scalar whose gradient moe_route_bwd computes: <weights, dw> + dloss .
    (balance, z), with the choice of experts and the counts of `r` held fixed."""
    l = np.array(logits, np.float64)
    E = l.shape[1]
    total = 0.0
    n, c = max(1, int(r["tokens"][0])), r["counts"] / max(1, r["counts"].sum())
    for t in np.nonzero(r["live"])[0]:
        m = l[t].max()
        p = np.exp(l[t] - m)
        lse = m + np.log(p.sum())
        p = p / p.sum()
        got = r["experts"][t] >= 0
        w = p[r["experts"][t][got]]
        if normalize:
            w = w / w.sum()
        total += (w * dw[t][got]).sum() if dw is not None else 0.0
        total += dloss[0] * E * (c * p).sum() / n + dloss[1] * lse ** 2 / n
    return total


def route_bwd(r, dw, dloss, normalize):
    """Gradient (float64) and the sum of the magnitudes that it adds up."""
    p, n = r["p"], max(1, int(r["tokens"][0]))
    T, E = p.shape
    g = dloss[0] * E * r["counts"] / max(1, r["counts"].sum()) / n
    zc = 2 * dloss[1] / n * r["lse"][:, None]
    got = r["experts"] >= 0
    d = np.where(got, dw, 0.0) if dw is not None else np.zeros(r["weights"].shape)
    dot = (d * r["weights"]).sum(1, keepdims=True)
    adot = (np.abs(d) * r["weights"]).sum(1, keepdims=True)
    pg = (p * g).sum(1, keepdims=True)
    out = p * (g - pg + zc - (0 if normalize else dot))
    mag = p * (np.abs(g) + (p * np.abs(g)).sum(1, keepdims=True) + np.abs(zc) + (0 if normalize else adot))
    for t in range(T):
        for j in np.nonzero(got[t])[0]:
            e = r["experts"][t, j]
            out[t, e] += r["weights"][t, j] * (d[t, j] - (dot[t, 0] if normalize else 0.0))
            mag[t, e] += r["weights"][t, j] * (abs(d[t, j]) + (adot[t, 0] if normalize else 0.0))
    out[~r["live"]] = 0.0
    return out, mag
