"""One MoE layer from its router logits to every gradient, the calls together
as a layer uses them, against torch autograd in fp32 on the CPU.

Forward: moe_route -> fp8_quantize gathered by the route -> fwd_fp8 (gate-up)
-> fp8_quantize_swiglu -> fwd_fp8 (down) -> moe_combine.  Backward:
moe_combine_bwd -> fp8_quantize -> dgrad_fp8 (down; the SwiGLU gradient is test
glue) -> fp8_quantize -> dgrad_fp8 (gate-up) -> moe_combine, kgemm_wgrad on the
bf16 rows, and moe_route_bwd with the balance and z losses.  The reference
differentiates the same layer on the dequantised weights.  What is between
them: E4M3 roundings (2^-4 half steps, normally distributed rounding error of
about 2.6% per operand) of x, h, dy and dgu, so about 4% per product and 8%
after two of them; the bound of 0.12 in Frobenius norm is far below what a
wrong expert, scale or row order gives (order 1).
"""
import pytest
import torch

import moe_grouped_gemm_bf16_amd as mg

pytestmark = pytest.mark.gpu


def _dequant(w8, ws):
    E, N, K = w8.shape
    s = ws.repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    return w8.view(torch.float8_e4m3fn).float() * s


@pytest.mark.parametrize("T", [24, 500])
def test_layer_forward_and_backward(T):
    print("[case] fp8 layer", T, flush=True)
    torch.manual_seed(1)
    D, I, E, k = 256, 144, 8, 2
    x = torch.randn(T, D).bfloat16()
    logits = torch.randn(T, E)
    mask = torch.ones(T, dtype=torch.bool)
    mask[-3:] = False
    w13, w2 = torch.randn(E, 2 * I, D) * D ** -0.5, torch.randn(E, D, I) * I ** -0.5
    dout = torch.randn(T, D).bfloat16()
    dloss = torch.tensor([0.5, 0.05])

    # ---- the library
    xd, ld, doutd = x.cuda(), logits.cuda(), dout.cuda()
    w13q, w13s = mg.fp8_quantize_weights(w13.cuda())
    w2q, w2s = mg.fp8_quantize_weights(w2.cuda())
    r = mg.moe_route(ld, k, mask=mask.cuda())
    rows = int(r.offsets[-1])
    x8, xs = mg.fp8_quantize(xd, gather=r.gather, offsets=r.offsets)
    M = r.gather.numel()
    gu = mg.fwd_fp8(x8, xs, w13q, w13s, r.offsets, out=torch.zeros(M, 2 * I, dtype=torch.bfloat16, device="cuda"))
    h8, hs = mg.fp8_quantize_swiglu(gu, offsets=r.offsets)
    y_rows = mg.fwd_fp8(h8, hs, w2q, w2s, r.offsets, out=torch.zeros(M, D, dtype=torch.bfloat16, device="cuda"))
    y = mg.moe_combine(y_rows, r.token_rows, r.weights)
    dy_rows, dweights = mg.moe_combine_bwd(doutd, y_rows, r.token_rows, r.weights)
    dy8, dys = mg.fp8_quantize(dy_rows, offsets=r.offsets)
    dh = mg.dgrad_fp8(dy8, dys, w2q, w2s, r.offsets, out=torch.zeros(M, I, dtype=torch.bfloat16, device="cuda")).float()
    g, u = gu.float().chunk(2, 1)
    s = torch.sigmoid(g)
    dgu = torch.cat([dh * u * s * (1 + g * (1 - s)), dh * g * s], 1).bfloat16()
    h = (g * s * u).bfloat16()
    dgu8, dgus = mg.fp8_quantize(dgu, offsets=r.offsets)
    dx_rows = mg.dgrad_fp8(dgu8, dgus, w13q, w13s, r.offsets)
    dx = mg.moe_combine(dx_rows, r.token_rows)
    x_rows = xd[r.gather.clamp_min(0).long()].contiguous()
    dw13 = mg.wgrad(dgu, x_rows, r.offsets, E)
    dw2 = mg.wgrad(dy_rows, h, r.offsets, E)
    dlogits = mg.moe_route_bwd(ld, r.weights, r.experts, r.lse, r.counts, r.tokens, dweights, dloss.cuda())
    torch.cuda.synchronize()

    # ---- the reference
    xr, lr = x.float().requires_grad_(True), logits.clone().requires_grad_(True)
    w13r = _dequant(w13q.cpu(), w13s.cpu()).requires_grad_(True)
    w2r = _dequant(w2q.cpu(), w2s.cpu()).requires_grad_(True)
    p = torch.softmax(lr, 1) * mask[:, None]
    top, experts = torch.sort(p.detach(), dim=1, descending=True, stable=True)
    experts = experts[:, :k]
    w = torch.gather(p, 1, experts)
    w = w / w.sum(1, keepdim=True).clamp_min(1e-30)
    yr = torch.zeros(T, D)
    live = [t for t in range(T) if mask[t]]
    counts = torch.zeros(E)
    for e in range(E):
        tok, slot = torch.nonzero((experts == e) & mask[:, None], as_tuple=True)
        counts[e] = len(tok)
        if len(tok) == 0:
            continue
        a = xr[tok] @ w13r[e].t()
        ye = (torch.nn.functional.silu(a[:, :I]) * a[:, I:]) @ w2r[e].t()
        yr = yr.index_add(0, tok, ye * w[tok, slot][:, None])
    n = len(live)
    balance = E * (counts / counts.sum() * p.sum(0) / n).sum()
    z = (torch.logsumexp(lr, 1)[:n] ** 2).sum() / n
    ((yr * dout.float()).sum() + dloss[0] * balance + dloss[1] * z).backward()

    assert rows == n * k and torch.equal(r.counts.cpu(), counts.int())
    assert abs(float(r.loss[0]) - float(balance.detach())) < 1e-5 and abs(float(r.loss[1]) - float(z.detach())) < 1e-4
    for name, got, want in (("y", y, yr.detach()), ("dx", dx, xr.grad), ("dw13", dw13, w13r.grad), ("dw2", dw2, w2r.grad),
                            ("dlogits", dlogits, lr.grad)):
        rel = float((got.cpu().double() - want.double()).norm() / want.double().norm())
        print(f"[case] {name}: relative Frobenius {rel:.3e}", flush=True)
        assert rel < 0.12, name
    assert (y[-3:] == 0).all() and (dx[-3:] == 0).all() and (dlogits[-3:] == 0).all()


def test_routed_rows_feed_the_bf16_calls():
    """The route's offsets, gather and token_rows in the fused bf16 forward:
    the layer's output equals the plain one on the same bf16 rows."""
    print("[case] route into fwd_swiglu", flush=True)
    torch.manual_seed(3)
    T, D, I, E, k = 300, 128, 64, 6, 3
    x = torch.randn(T, D).bfloat16()
    w13, w2 = (torch.randn(E, 2 * I, D) * D ** -0.5).bfloat16(), (torch.randn(E, D, I) * I ** -0.5).bfloat16()
    r = mg.moe_route(torch.randn(T, E, device="cuda"), k, normalize=False)
    h = mg.fwd_swiglu(x.cuda(), w13.cuda(), r.offsets, gather=r.gather)
    y = mg.moe_combine(mg.fwd(h, w2.cuda(), r.offsets), r.token_rows, r.weights).cpu().double()
    want = torch.zeros(T, D, dtype=torch.float64)
    ex, w = r.experts.cpu(), r.weights.cpu().double()
    for t in range(T):
        for j in range(k):
            e = int(ex[t, j])
            a = w13[e].double() @ x[t].double()
            want[t] += w[t, j] * (w2[e].double() @ (torch.nn.functional.silu(a[:I]) * a[I:]))
    # bf16 roundings of h, the rows and the output, 2^-8 each at most
    assert float((y - want).norm() / want.norm()) < 3 * 2.0 ** -8
