"""The output head's losses and gradients in 64 bits (torch, on any device),
and how far results in 32 and 16 bits may be from them.

Bounds, with u = 2^-24 (half a step of fp32) and h = 2^-8 (half a step of bf16,
relative to the value):
  z      a sum of D products in fp32: (D + 2) u sum_d |x w|
  c z log2(e) - reference: the factor is rounded three times (temperature, its
         inverse, the product), the fma and the reference once each, at values
         up to A = max |c z| log2(e): 16 A u in all, with the joining of parts
  lse    c times z's bound, 16 A u, u per addition of a chain of at most
         100 + V / 1024, 4 u of itself
  q      exponentials of c t and their sum: (16 + 8 max |c t| + k) u relative
  dz     a p with p's relative error (lse is an input: c z's bound and 16 A u,
         4 |lse| u), b q with q's, and h of itself
  dx, dw sums of dz's errors against |w|, |x|; one u per term of the fp32 sum;
         h of the result
"""
import torch

U, H = 2.0 ** -24, 2.0 ** -8
LOG2E = 1.4426950408889634


def entries(targets=None, teacher=None, index=None, temperature=1.0):
    """(index [T, k] with -1 for none, q [T, k], max |c t| per token)."""
    if targets is not None:
        at = targets.long()[:, None].clamp_min(-1)
        return at, (at >= 0).double(), torch.zeros(len(at), dtype=torch.float64, device=at.device)
    t = teacher.double()
    t = torch.where(t.isnan(), -torch.inf, t).clamp_max(torch.finfo(torch.float32).max)
    at = torch.where((index < 0) | (t == -torch.inf), -1, index.long())
    t = torch.where(at < 0, -torch.inf, t / temperature)
    live = (at >= 0).any(1, keepdim=True)
    top = torch.where(live, t.amax(1, keepdim=True), 0.0)
    q = torch.where(at >= 0, (t - top).exp(), 0.0)
    q = q / q.sum(1, keepdim=True).clamp_min(1e-300)
    # differences from the largest: those whose q does not vanish count
    size = torch.where(q > 1e-30, (t - top).abs(), 0.0).amax(1)
    return at, q, size


def forward(x, w, at, q, size, temperature=1.0, first=0):
    """(loss, lse, logits, tolerances of the three)."""
    X, W, c = x.double(), w.double(), 1.0 / temperature
    D, V, k = X.shape[1], W.shape[0], at.shape[1]
    z = X @ W.T
    ze = ((D + 2) * U) * (X.abs() @ W.abs().T).amax(1)
    live = (at >= 0).any(1)
    A = (c * LOG2E) * z.abs().amax(1)
    lse = torch.where(live, torch.logsumexp(c * z, 1), 0.0)
    lse_tol = c * ze + U * (16 * A + 100 + V / 1024 + 4 * lse.abs())
    here = (at >= first) & (at < first + V)
    zk = torch.where(here, z.gather(1, (at - first).clamp(0, V - 1)), 0.0)
    term = torch.where(q > 0, q.clamp_min(1e-300).log() + lse[:, None] - c * zk, 0.0)
    loss = (q * term).sum(1)
    rq = U * (16 + 8 * size + k)
    loss_tol = lse_tol + c * ze + rq * (1 + 2 * (q * term.abs()).sum(1)) + U * (4 * lse.abs() + 8 * A)
    return loss, lse, zk, loss_tol, lse_tol, ze[:, None].expand_as(zk)


def backward(x, w, at, q, size, lse, up, dense=None, temperature=1.0, first=0, step=H):
    """(dx, dw, tolerances of both): up is dloss, dense the weight of the
    probabilities where it is not dloss, step dz's rounding: h, or h h where it is
    the sum of two values (the second is h of dz at most, and rounded to h of it)."""
    X, W, c = x.double(), w.double(), 1.0 / temperature
    T, D = X.shape
    V, k = W.shape[0], at.shape[1]
    z = X @ W.T
    ze = ((D + 2) * U) * (X.abs() @ W.abs().T)
    live = (at >= 0).any(1)
    b = torch.where(live, up.double() * c, 0.0)
    a = b if dense is None else torch.where(live, dense.double() * c, 0.0)
    lse = lse.double()
    P = torch.where(live[:, None], a[:, None] * (c * z - lse[:, None]).exp(), 0.0)
    A = (c * LOG2E) * z.abs().amax(1) + lse.abs()
    here = (at >= first) & (at < first + V)
    S = torch.zeros(T, V, dtype=torch.float64, device=x.device)
    rows = torch.arange(T, device=x.device)[:, None].expand_as(at)[here]
    S.index_put_((rows, (at - first)[here]), (b[:, None] * q)[here], accumulate=True)
    dz = P - S
    rq = (U * (24 + 8 * size + 2 * k))[:, None]
    dze = P.abs() * (c * ze + U * (16 * A + 16)[:, None]) + S.abs() * rq
    dze = dze + step * (dz.abs() + dze) + 1e-37
    dx, dw = dz @ W, dz.T @ X
    m = dz.abs() + dze
    dx_tol = dze @ W.abs() + ((V + 72) * U) * (m @ W.abs())
    dw_tol = dze.T @ X.abs() + ((T + 8) * U) * (m.T @ X.abs())
    return dx, dw, dx_tol + H * (dx.abs() + dx_tol) + 1e-37, dw_tol + H * (dw.abs() + dw_tol) + 1e-37
