"""The output head's cross entropy and distillation and their gradients on the
GPU, against tests/head_ref.py (64 bits; its bounds are the tolerances here)."""
import math

import pytest
import torch

import head_ref as ref
import moe_grouped_gemm_bf16_amd as mg

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _say(*a):
    print("[case]", *a, flush=True)


def _near(name, got, want, tol):
    assert got.shape == want.shape, name
    off = (got.double() - want).abs()
    bad = ~(off <= tol)
    assert not bad.any(), (name, int(bad.sum()), float((off / tol)[bad].max()), bad.nonzero()[:4].tolist())


def _inputs(T, V, D, seed, spread=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = (0.1 * torch.randn(V, D, device=DEV, generator=g)).bfloat16()
    x = (torch.randn(T, D, device=DEV, generator=g) * (15.0 * spread / math.sqrt(D))).bfloat16()
    return g, x, w


def _targets(g, T, V, ignored):
    t = torch.randint(0, V, (T,), device=DEV, generator=g, dtype=torch.int32)
    t[torch.rand(T, device=DEV, generator=g) < ignored] = -100
    return t


def _loss_case(T, V, D, ignored=0.0, z_loss=False, seed=0, uniform=True):
    _say("loss", T, V, D, ignored, z_loss)
    g, x, w = _inputs(T, V, D, seed)
    t = _targets(g, T, V, ignored)
    r = mg.head_loss(x, w, t)
    e = ref.entries(targets=t)
    loss, lse, logit, tl, ts, tz = ref.forward(x, w, *e)
    _near("lse", r.lse, lse, ts)
    _near("logit", r.logit, logit[:, 0], tz[:, 0])
    _near("loss", r.loss, loss, tl)
    dloss = torch.full((T,), 1.0 / max(1, T), device=DEV) if uniform else torch.randn(T, device=DEV, generator=g)
    dlse = 0.01 * r.lse if z_loss else None
    dx, dw = mg.head_loss_bwd(x, w, t, r.lse, dloss, dlse=dlse)
    wx, ww, tx, tw = ref.backward(x, w, *e, r.lse, dloss, None if dlse is None else dloss.double() + dlse.double())
    _near("dx", dx, wx, tx)
    _near("dw", dw, ww, tw)
    return x, w, t, r, dx, dw


SHAPES = [(1, 1, 8), (1, 300, 64), (2, 5, 72), (63, 127, 136), (64, 128, 128), (65, 129, 520), (130, 257, 64), (257, 1000, 72),
          (300, 4097, 40), (700, 2049, 264), (1, 20001, 2048), (17, 5000, 1032)]


@pytest.mark.parametrize("i", range(len(SHAPES)))
@pytest.mark.parametrize("ignored", [0.0, 0.4])
def test_loss(i, ignored):
    _loss_case(*SHAPES[i], ignored=ignored, z_loss=i % 2 == 1, seed=i, uniform=i % 3 != 0)


# whole tiles of 256 x 256 and of 256 x 128, edges in every direction
@pytest.mark.parametrize("T,V,D", [(2048, 8192, 64), (2100, 8500, 72), (4096, 4100, 192), (1111, 16411, 320), (3000, 33000, 8)])
def test_loss_in_large_tiles(T, V, D):
    _loss_case(T, V, D, ignored=0.1, z_loss=True, seed=T, uniform=False)


def test_loss_in_pieces_of_the_vocabulary():
    # 65600 tokens: pieces of 4096 entries, the last one short
    _loss_case(65600, 4500, 16, ignored=0.02, seed=5)


def test_no_token_counts_and_one_token_counts():
    T, V, D = 300, 700, 72
    g, x, w = _inputs(T, V, D, 1)
    t = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    r = mg.head_loss(x, w, t)
    dx, dw = mg.head_loss_bwd(x, w, t, r.lse, torch.ones(T, device=DEV))
    for v in (*r, dx, dw):
        assert (v == 0).all()
    t[299] = V - 1
    r = mg.head_loss(x, w, t)
    e = ref.entries(targets=t)
    loss, lse, logit, tl, ts, tz = ref.forward(x, w, *e)
    _near("loss", r.loss, loss, tl)
    up = torch.ones(T, device=DEV)
    dx, dw = mg.head_loss_bwd(x, w, t, r.lse, up)
    wx, ww, tx, tw = ref.backward(x, w, *e, r.lse, up)
    _near("dx", dx, wx, tx)
    _near("dw", dw, ww, tw)
    assert (dx[:299] == 0).all()


def test_empty_batch():
    _, x, w = _inputs(4, 100, 64, 1)
    t = torch.empty(0, dtype=torch.int32, device=DEV)
    r = mg.head_loss(x[:0], w, t)
    assert all(v.numel() == 0 for v in r)
    dw = torch.full_like(w, 7.0)
    dx, dw2 = mg.head_loss_bwd(x[:0], w, t, r.lse, r.loss, dw=dw)
    assert dx.shape == (0, 64) and dw2 is dw and (dw == 0).all()


def test_confident_and_hopeless_tokens():
    """Targets far above and far below the rest: losses near 0 and of hundreds,
    probabilities that vanish, weights of very different size."""
    T, V, D = 200, 1500, 64
    g, x, w = _inputs(T, V, D, 3, spread=20.0)
    t = _targets(g, T, V, 0.0)
    z = x.double() @ w.double().T
    t[:100] = z[:100].argmax(1).int()
    t[100:] = z[100:].argmin(1).int()
    r = mg.head_loss(x, w, t)
    e = ref.entries(targets=t)
    loss, lse, logit, tl, ts, tz = ref.forward(x, w, *e)
    _near("loss", r.loss, loss, tl)
    for up in (torch.full((T,), 1e-30, device=DEV), torch.logspace(-20, 3, T, device=DEV), torch.zeros(T, device=DEV)):
        dx, dw = mg.head_loss_bwd(x, w, t, r.lse, up)
        wx, ww, tx, tw = ref.backward(x, w, *e, r.lse, up)
        _near("dx", dx, wx, tx)
        _near("dw", dw, ww, tw)


def test_a_row_that_is_not_finite_stays_alone():
    T, V, D = 300, 600, 72
    g, x, w = _inputs(T, V, D, 4)
    t = _targets(g, T, V, 0.0)
    clean = mg.head_loss(x, w, t)
    cx, _ = mg.head_loss_bwd(x, w, t, clean.lse, torch.ones(T, device=DEV))
    y = x.clone()
    y[17, 3], y[255, 0], y[299, 5] = math.nan, math.inf, -math.inf
    r = mg.head_loss(y, w, t)
    dx, _ = mg.head_loss_bwd(y, w, t, r.lse, torch.ones(T, device=DEV))
    odd = torch.zeros(T, dtype=torch.bool, device=DEV)
    odd[[17, 255, 299]] = True
    assert not r.loss[odd].isfinite().any() and not dx[odd].isfinite().any()
    assert torch.equal(r.loss[~odd], clean.loss[~odd]) and torch.equal(dx[~odd], cx[~odd])


def test_rows_that_do_not_count_may_hold_anything():
    T, V, D = 300, 600, 72
    g, x, w = _inputs(T, V, D, 6)
    t = _targets(g, T, V, 0.3)
    want = mg.head_loss(x, w, t)
    up = torch.ones(T, device=DEV)
    wx, ww = mg.head_loss_bwd(x, w, t, want.lse, up)
    x[t < 0] = math.nan
    up[t < 0] = math.nan
    r = mg.head_loss(x, w, t)
    dx, dw = mg.head_loss_bwd(x, w, t, r.lse, up)
    for a, b in zip((*want, wx, ww), (*r, dx, dw)):
        assert torch.equal(a, b)


def test_bitwise_reproducible():
    x, w, t, r, dx, dw = _loss_case(1500, 9000, 136, ignored=0.2, seed=9)
    for _ in range(3):
        s = mg.head_loss(x, w, t)
        ex, ew = mg.head_loss_bwd(x, w, t, r.lse, torch.full((1500,), 1.0 / 1500, device=DEV))
        assert all(torch.equal(a, b) for a, b in zip((*r, dx, dw), (*s, ex, ew)))


def _teacher(g, T, V, k, dtype, missing=0.1):
    index = torch.rand(T, V, device=DEV, generator=g).argsort(1)[:, :k].int()
    teacher = (3.0 * torch.randn(T, k, device=DEV, generator=g) + 5.0).to(dtype)
    index[torch.rand(T, k, device=DEV, generator=g) < missing] = -1
    index[torch.rand(T, device=DEV, generator=g) < missing] = -1
    return teacher, index


def _distill_check(x, w, teacher, index, tau, up=None):
    T = len(x)
    r = mg.head_distill(x, w, teacher, index, temperature=tau)
    e = ref.entries(teacher=teacher, index=index, temperature=tau)
    loss, lse, zk, tl, ts, tz = ref.forward(x, w, *e, temperature=tau)
    _near("lse", r.lse, lse, ts)
    _near("logits", r.logits, zk, tz)
    _near("loss", r.loss, loss, tl)
    up = torch.full((T,), 0.3 / T, device=DEV) if up is None else up
    dx, dw = mg.head_distill_bwd(x, w, teacher, index, r.lse, r.logits, up, temperature=tau)
    wx, ww, tx, tw = ref.backward(x, w, *e, r.lse, up, temperature=tau)
    _near("dx", dx, wx, tx)
    _near("dw", dw, ww, tw)
    return r, dx, dw


KSHAPES = [(1, 8, 8, 1), (1, 3000, 520, 65), (3, 70, 72, 64), (66, 129, 64, 7), (130, 600, 136, 256), (257, 1000, 72, 63), (700, 2500, 264, 20),
           (2100, 8300, 64, 5)]


@pytest.mark.parametrize("i", range(len(KSHAPES)))
@pytest.mark.parametrize("dtype,tau", [(torch.float32, 1.0), (torch.bfloat16, 2.0), (torch.float32, 0.7)])
def test_distill(i, dtype, tau):
    T, V, D, k = KSHAPES[i]
    _say("distill", T, V, D, k, dtype, tau)
    g, x, w = _inputs(T, V, D, 20 + i)
    teacher, index = _teacher(g, T, V, k, dtype)
    _distill_check(x, w, teacher, index, tau, torch.randn(T, device=DEV, generator=g) if i % 2 else None)


def test_distill_in_pieces_of_the_vocabulary():
    T, V, D, k = 65600, 4500, 16, 3
    g, x, w = _inputs(T, V, D, 31)
    index = torch.randint(0, V // 3, (T, k), device=DEV, generator=g, dtype=torch.int32) * 3
    index += torch.arange(k, device=DEV, dtype=torch.int32)          # distinct, over both pieces
    _distill_check(x, w, torch.randn(T, k, device=DEV, generator=g), index, 1.0)


def test_entries_that_are_not_there():
    T, V, D, k = 70, 500, 64, 6
    g, x, w = _inputs(T, V, D, 32)
    teacher, index = _teacher(g, T, V, k, torch.float32, 0.0)
    teacher[0, 2], teacher[1, 0], teacher[2], teacher[3, 1] = -math.inf, math.nan, -math.inf, math.inf
    index[4], teacher[5, :5], index[6, 1:] = -1, torch.finfo(torch.float32).min, -7
    r, dx, _ = _distill_check(x, w, teacher, index, 1.0)
    for t in (2, 4):
        assert r.loss[t] == 0 and r.lse[t] == 0 and (dx[t] == 0).all()
    assert (r.logits[index < 0] == 0).all()


def test_the_same_entry_twice():
    T, V, D, k = 70, 500, 64, 130
    g, x, w = _inputs(T, V, D, 33)
    index = torch.randint(0, 40, (T, k), device=DEV, generator=g, dtype=torch.int32)
    _distill_check(x, w, torch.randn(T, k, device=DEV, generator=g), index, 1.0)


def test_one_entry_is_a_target():
    """k = 1 at temperature 1 is the cross entropy: the same bits."""
    T, V, D = 300, 900, 136
    g, x, w = _inputs(T, V, D, 34)
    t = _targets(g, T, V, 0.2)
    a = mg.head_loss(x, w, t)
    b = mg.head_distill(x, w, torch.randn(T, 1, device=DEV, generator=g), t[:, None].contiguous())
    assert torch.equal(a.lse, b.lse)
    up = torch.full((T,), 1.0 / T, device=DEV)
    ax, aw = mg.head_loss_bwd(x, w, t, a.lse, up)
    bx, bw = mg.head_distill_bwd(x, w, torch.zeros(T, 1, device=DEV), t[:, None].contiguous(), b.lse, b.logits, up)
    # the target's logit is summed in another order: its p may round to the neighbour
    for u, v in ((ax, bx), (aw, bw)):
        assert (u.double() - v.double()).norm() <= 2.0 ** -7 * u.double().norm()


@pytest.mark.parametrize("cut", [1, 500, 1023])
def test_vocabulary_in_two_parts(cut):
    """Two ranks' parts, joined as they would be."""
    T, V, D, k = 150, 1024, 72, 9
    g, x, w = _inputs(T, V, D, 35)
    t = _targets(g, T, V, 0.2)
    parts = [(w[:cut].contiguous(), 0), (w[cut:].contiguous(), cut)]
    rs = [mg.head_loss(x, p, t, first=f) for p, f in parts]
    e = ref.entries(targets=t)
    loss, lse, logit, tl, ts, tz = ref.forward(x, w, *e)
    counts = t >= 0
    joined = torch.where(counts, torch.logaddexp(rs[0].lse, rs[1].lse), 0.0)
    _near("lse", joined, lse, 2 * ts)
    _near("loss", joined - (rs[0].logit + rs[1].logit), loss, 3 * tl)
    up = torch.full((T,), 1.0 / T, device=DEV)
    for p, f in parts:
        dx, dw = mg.head_loss_bwd(x, p, t, joined, up, first=f)
        wx, ww, tx, tw = ref.backward(x, p, *e, joined, up, first=f)
        _near("dx", dx, wx, tx)
        _near("dw", dw, ww, tw)
    teacher, index = _teacher(g, T, V, k, torch.float32)
    rs = [mg.head_distill(x, p, teacher, index, temperature=1.5, first=f) for p, f in parts]
    counts = (index >= 0).any(1)
    joined = torch.where(counts, torch.logaddexp(rs[0].lse, rs[1].lse), 0.0)
    logits = rs[0].logits + rs[1].logits
    e = ref.entries(teacher=teacher, index=index, temperature=1.5)
    for p, f in parts:
        dx, dw = mg.head_distill_bwd(x, p, teacher, index, joined, logits, up, temperature=1.5, first=f)
        wx, ww, tx, tw = ref.backward(x, p, *e, joined, up, temperature=1.5, first=f)
        _near("dx", dx, wx, tx)
        _near("dw", dw, ww, tw)


def test_one_gradient_alone_and_callers_buffers():
    T, V, D = 150, 700, 72
    g, x, w = _inputs(T, V, D, 36)
    t = _targets(g, T, V, 0.2)
    r = mg.head_loss(x, w, t)
    up = torch.ones(T, device=DEV)
    dx, dw = mg.head_loss_bwd(x, w, t, r.lse, up)
    only, none = mg.head_loss_bwd(x, w, t, r.lse, up, need_dw=False)
    assert none is None and torch.equal(only, dx)
    none, only = mg.head_loss_bwd(x, w, t, r.lse, up, need_dx=False)
    assert none is None and torch.equal(only, dw)
    assert mg.head_loss_bwd(x, w, t, r.lse, up, need_dx=False, need_dw=False) == (None, None)
    # buffers that are parts of larger ones: what lies around them stays
    bx, bw = torch.full((T + 2, D), 3.0, device=DEV).bfloat16(), torch.full((V + 2, D), 3.0, device=DEV).bfloat16()
    ox, ow = mg.head_loss_bwd(x, w, t, r.lse, up, dx=bx[1:-1], dw=bw[1:-1])
    assert torch.equal(ox, dx) and torch.equal(ow, dw) and ox.data_ptr() == bx[1:].data_ptr()
    for b in (bx, bw):
        assert (b[0] == 3).all() and (b[-1] == 3).all()
    teacher, index = _teacher(g, T, V, 4, torch.float32)
    d = mg.head_distill(x, w, teacher, index)
    dx, dw = mg.head_distill_bwd(x, w, teacher, index, d.lse, d.logits, up)
    assert torch.equal(mg.head_distill_bwd(x, w, teacher, index, d.lse, d.logits, up, need_dw=False)[0], dx)
    assert torch.equal(mg.head_distill_bwd(x, w, teacher, index, d.lse, d.logits, up, need_dx=False)[1], dw)


def test_two_streams_at_once():
    cases = [_inputs(700, 5000, 136, 40 + i) for i in range(2)]
    ts = [_targets(g, 700, 5000, 0.1) for g, _, _ in cases]
    up = torch.full((700,), 1.0 / 700, device=DEV)

    def step(i):
        _, x, w = cases[i]
        r = mg.head_loss(x, w, ts[i])
        return (*r, *mg.head_loss_bwd(x, w, ts[i], r.lse, up))

    want = [step(i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((i, step(i)))
    torch.cuda.synchronize()
    for i, r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want[i]))


def test_captured_and_replayed():
    """One graph of both losses and their gradients, inputs changed in place
    between replays, eager work of the same kind between them."""
    T, V, D, k = 300, 3000, 136, 5
    g, x, w = _inputs(T, V, D, 50)
    t = _targets(g, T, V, 0.2)
    teacher, index = _teacher(g, T, V, k, torch.bfloat16)
    up = torch.full((T,), 1.0 / T, device=DEV)

    def step():
        r = mg.head_loss(x, w, t)
        d = mg.head_distill(x, w, teacher, index, temperature=2.0)
        return (*r, *mg.head_loss_bwd(x, w, t, r.lse, up), *d,
                *mg.head_distill_bwd(x, w, teacher, index, d.lse, d.logits, up, temperature=2.0))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        x.copy_(torch.randn(T, D, device=DEV, generator=g))
        t.copy_(_targets(g, T, V, 0.3 * i))                # other tokens count, other numbers of them
        index.copy_(_teacher(g, T, V, k, torch.bfloat16, 0.1 * i)[1])
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


def test_weights_past_32_bits():
    """w of more than 2^32 bytes: the first, middle and last entries."""
    T, V, D = 5, 300001, 8192
    x = torch.randn(T, D, device=DEV).bfloat16() * 0.1
    w = torch.empty(V, D, dtype=torch.bfloat16, device=DEV)
    for b in range(0, V, 50000):
        w[b:b + 50000].normal_(std=0.1)
    t = torch.tensor([0, V - 1, V // 2, -1, 262145], dtype=torch.int32, device=DEV)
    r = mg.head_loss(x, w, t)
    z = torch.cat([x.double() @ w[b:b + 20000].double().T for b in range(0, V, 20000)], 1)
    live = t >= 0
    # (per token: (D + 2) u sum |x w|, at most 1.5 D 0.08^2 u here, plus the sums')
    tol = 2.0 ** -24 * (8200 * D * 0.02 + 400)
    assert ((r.lse - torch.where(live, torch.logsumexp(z, 1), 0.0)).abs() <= tol).all()
    assert ((r.logit - torch.where(live, z.gather(1, t.long().clamp_min(0)[:, None])[:, 0], 0.0)).abs() <= tol).all()
    dx, dw = mg.head_loss_bwd(x, w, t, r.lse, torch.ones(T, device=DEV))
    dz = torch.where(live[:, None], (z - r.lse.double()[:, None]).exp(), 0.0)
    dz[torch.arange(T, device=DEV)[live], t.long()[live]] -= 1
    want = sum(dz[:, b:b + 20000] @ w[b:b + 20000].double() for b in range(0, V, 20000))
    assert (dx.double() - want).norm() <= 2.0 ** -7 * want.norm() and (dx[3] == 0).all()
    for v in (0, V - 1, V // 2, 262145, 7, 200000):
        want = dz[:, v] @ x.double()
        assert (dw[v].double() - want).norm() <= 2.0 ** -7 * want.norm(), v


def test_hidden_rows_past_32_bits():
    T, V, D = 2100000, 9, 1032
    x = torch.empty(T, D, dtype=torch.bfloat16, device=DEV)
    for b in range(0, T, 300000):
        x[b:b + 300000].normal_(std=0.3)
    w = torch.randn(V, D, device=DEV).bfloat16() * 0.1
    t = torch.randint(0, V, (T,), device=DEV, dtype=torch.int32)
    t[12345] = -1
    r = mg.head_loss(x, w, t)
    dx, dw = mg.head_loss_bwd(x, w, t, r.lse, torch.full((T,), 1.0 / T, device=DEV))
    want_w = torch.zeros(V, D, dtype=torch.float64, device=DEV)
    for b in range(0, T, 100000):
        s = slice(b, b + 100000)
        e = ref.entries(targets=t[s])
        loss, lse, _, tl, ts, _ = ref.forward(x[s], w, *e)
        _near("loss", r.loss[s], loss, tl)
        wx, ww, tx, _ = ref.backward(x[s], w, *e, r.lse[s], torch.full((len(lse),), 1.0 / T, device=DEV))
        _near("dx", dx[s], wx, tx)
        want_w += ww
    # fp32 sums of 2.1 million terms in a chain: their rounding errors, as
    # independent, are sqrt(T) u of a term's size against sqrt(T) for the sum
    assert (dw.double() - want_w).norm() <= 2.0 ** -6 * want_w.norm()


def test_through_a_layer_and_both_losses():
    """An expert layer, then cross entropy and distillation on one head, their
    gradients added and taken back through the layer: against torch autograd in
    fp64 on the CPU."""
    T, D, V, E, k = 200, 136, 1100, 3, 8
    g = torch.Generator().manual_seed(60)
    h = torch.randn(T, D, generator=g).bfloat16()
    we = (torch.randn(E, D, D, generator=g) / math.sqrt(D)).bfloat16()
    w = (0.2 * torch.randn(V, D, generator=g)).bfloat16()
    offsets = torch.tensor([0, 80, 80, T], dtype=torch.int32)
    t = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    t[::7] = -100
    teacher = torch.randn(T, k, generator=g) * 2
    index = torch.rand(T, V, generator=g).argsort(1)[:, :k].int()
    n, alpha, tau = int((t >= 0).sum()), 0.3, 2.0

    c = [v.to(DEV) for v in (h, we, w, offsets, t, teacher, index)]
    x = mg.fwd(c[0], c[1], c[3])
    a = mg.head_loss(x, c[2], c[4])
    b = mg.head_distill(x, c[2], c[5], c[6], temperature=tau)
    loss = (1 - alpha) * a.loss.sum() / n + alpha * tau * tau * b.loss.sum() / T
    ax, aw = mg.head_loss_bwd(x, c[2], c[4], a.lse, torch.full((T,), (1 - alpha) / n, device=DEV))
    bx, bw = mg.head_distill_bwd(x, c[2], c[5], c[6], b.lse, b.logits, torch.full((T,), alpha * tau * tau / T, device=DEV), temperature=tau)
    dx, dw = ax + bx, aw.float() + bw.float()
    dh, dwe = mg.dgrad(dx, c[1], c[3]), mg.wgrad(dx, c[0], c[3])

    leaves = [v.double().requires_grad_() for v in (h, we, w)]
    y = torch.cat([leaves[0][:80] @ leaves[1][0].T, leaves[0][80:] @ leaves[1][2].T])
    xr = y + (x.cpu().double() - y).detach()               # the layer's output as it was rounded
    z = xr @ leaves[2].T
    ce = torch.nn.functional.cross_entropy(z, t.long(), ignore_index=-100)
    q = torch.softmax(teacher.double() / tau, 1)
    kd = (q * (q.log() - torch.log_softmax(z / tau, 1).gather(1, index.long()))).sum(1).mean()
    want = (1 - alpha) * ce + alpha * tau * tau * kd
    want.backward()
    assert abs(float(loss) - float(want.detach())) <= 1e-5 * abs(float(want.detach()))
    # dz, dx of each loss, their sum and the product's result: five roundings of at most 2^-8
    for name, got, leaf in (("h", dh, leaves[0]), ("we", dwe, leaves[1]), ("w", dw, leaves[2])):
        off = (got.cpu().double() - leaf.grad).norm() / leaf.grad.norm()
        assert off <= 5 * 2.0 ** -8, (name, float(off))


# the weights' gradient in parts over the tokens; the last sizes that go in 64 x
# 64 tiles and the first that do not; large and small tiles in one product; few
# tokens, whose tiles take fewer rows of w than they have
@pytest.mark.parametrize("T,V,D", [(6000, 700, 200), (3971, 1798, 352), (20000, 130, 72), (64, 16384, 72), (65, 8192, 1544), (65, 16384, 1544),
                                   (65, 16640, 1544), (1333, 50001, 72), (2050, 3333, 1544), (129, 300, 64), (128, 300, 72),
                                   (100, 20011, 1000), (128, 65721, 512), (200, 33333, 264), (256, 66000, 1544), (257, 66000, 72), (127, 70001, 8), (127, 70001, 520)])
def test_loss_by_every_cut(T, V, D):
    _loss_case(T, V, D, ignored=0.05, z_loss=True, seed=V, uniform=False)


@pytest.mark.parametrize("T,V,D", [(200, 1500, 64), (1500, 9000, 136)])
@pytest.mark.parametrize("tau", [None, 1.0, 1e-6])
def test_logits_of_any_size(T, V, D, tau):
    """Rows of x from 1e-3 to 1e30: the losses stay finite and near, and where
    one entry has all the probability the gradient is the difference of two rows
    of w."""
    g, x, w = _inputs(T, V, D, 70)
    x = (x.float() * torch.logspace(-3, 30, T, device=DEV)[:, None]).bfloat16()
    z = x.double() @ w.double().T
    best = z.argmax(1).int()
    t = torch.where(torch.arange(T, device=DEV) % 2 == 0, best, _targets(g, T, V, 0.0))
    up = torch.randn(T, device=DEV, generator=g)
    if tau is None:
        r, e, c = mg.head_loss(x, w, t), ref.entries(targets=t), 1.0
        dx, dw = mg.head_loss_bwd(x, w, t, r.lse, up)
    else:
        index, teacher, c = t[:, None].contiguous(), torch.zeros(T, 1, device=DEV), 1.0 / tau
        r = mg.head_distill(x, w, teacher, index, temperature=tau)
        e = ref.entries(teacher=teacher, index=index, temperature=tau)
        dx, dw = mg.head_distill_bwd(x, w, teacher, index, r.lse, r.logits, up, temperature=tau)
    loss, lse, _, tl, ts, _ = ref.forward(x, w, *e, temperature=1.0 / c)
    _near("lse", r.lse, lse, ts)
    _near("loss", r.loss, loss, tl)
    assert dx.isfinite().all() and dw.isfinite().all()
    top = z.topk(2, 1).values
    alone = c * (top[:, 0] - top[:, 1]) > 1e-3 * c * top[:, 0].abs() + 100.0
    assert alone.sum() > T / 3
    # p <= 1 is of lse as it was rounded: dx lies between -w[t] and w[best] - w[t]
    wb, wt, s = w[best.long()].double(), w[t.long()].double(), (c * up.double())[:, None]
    ends = torch.stack((-s * wt, s * (wb - wt)))
    slack = 2.0 ** -6 * s.abs() * (wb.abs() + wt.abs())
    inside = (dx.double() >= ends.amin(0) - slack) & (dx.double() <= ends.amax(0) + slack)
    assert inside[alone].all()
    if tau is None:
        # and lse is the largest logit itself, its p one (dz and dx rounded once each).
        # (Distillation sums an entry's logit in another order: 66 u sum |x w| off,
        # at |z| >= 2^26 = kFar more than an exponent of 1, so p is anything up to 1.)
        assert ((dx.double() - s * (wb - wt)).abs() <= slack)[alone].all()


def test_gradients_against_differences():
    """dx and dw along a direction against the losses' central differences.  The
    steps are exact in bf16; f(1/2) - f(-1/2) = f'(0) + f'''/24, and the third
    derivative of a token's lse along dz is its third cumulant, at most the cube
    of dz's range (of the loss and of lse alike)."""
    T, V, D = 40, 300, 64
    g = torch.Generator(device=DEV).manual_seed(71)
    x = ((torch.randn(T, D, device=DEV, generator=g) * 8).round().clamp(-24, 24) / 8).bfloat16()
    w = ((torch.randn(V, D, device=DEV, generator=g) * 8).round().clamp(-28, 28) / 64).bfloat16()
    t = _targets(g, T, V, 0.2)
    up, ul = torch.randn(T, device=DEV, generator=g), torch.randn(T, device=DEV, generator=g)
    r = mg.head_loss(x, w, t)
    e = ref.entries(targets=t)
    dx, dw = mg.head_loss_bwd(x, w, t, r.lse, up, dlse=ul)
    _, _, tx, tw = ref.backward(x, w, *e, r.lse, up, up.double() + ul.double())
    weight = up.double().abs() + ul.double().abs()
    for name, grad, tol, h in (("dx", dx, tx, 1 / 64), ("dw", dw, tw, 1 / 512)):
        base = x if name == "dx" else w
        for _ in range(8):
            d = h * (torch.randint(0, 2, base.shape, device=DEV, generator=g) * 2 - 1).double()
            sides, slack = [], 0.0
            for sign in (1.0, -1.0):
                at = (base.double() + sign * d).bfloat16()
                assert torch.equal(at.double(), base.double() + sign * d)
                a, b = (at, w) if name == "dx" else (x, at)
                s = mg.head_loss(a, b, t)
                _, _, _, tl, ts, _ = ref.forward(a, b, *e)
                sides.append(((up.double() * s.loss.double()).sum() + (ul.double() * s.lse.double()).sum(), a.double() @ b.double().T))
                slack += float((weight * torch.maximum(tl, ts)).sum())
            dz = sides[0][1] - sides[1][1]
            third = float((weight * (dz.amax(1) - dz.amin(1)) ** 3)[t >= 0].sum()) / 24
            want, got = float(sides[0][0] - sides[1][0]), float((grad.double() * 2 * d).sum())
            assert abs(got - want) <= slack + third + float((tol * 2 * d.abs()).sum()), (name, got, want)


def test_misaligned_tensors_are_refused():
    T, V, D = 10, 50, 64
    g, x, w = _inputs(T, V, D, 72)
    t = _targets(g, T, V, 0.0)
    off = torch.empty(T * D + 4, dtype=torch.bfloat16, device=DEV)[4:].view(T, D)
    off.copy_(x)
    r = mg.head_loss(x, w, t)
    for call in (lambda: mg.head_loss(off, w, t),
                 lambda: mg.head_loss_bwd(off, w, t, r.lse, r.loss),
                 lambda: mg.head_loss_bwd(x, w, t, r.lse, r.loss, dx=off)):
        with pytest.raises(mg.MgemmError):
            call()


@pytest.mark.parametrize("T,V,D", [(1, 700, 72), (2, 3000, 136), (2, 70001, 520), (17, 2000, 1032), (33, 70001, 264), (64, 3000, 64), (64, 70001, 520)])
@pytest.mark.parametrize("ignored", [0.0, 0.5])
def test_few_tokens_keep_dz_in_two_values(T, V, D, ignored):
    """Up to 64 tokens: only the results' own rounding is left of the bounds."""
    g, x, w = _inputs(T, V, D, 80 + T)
    t = _targets(g, T, V, ignored)
    t[T // 2] = V - 1
    up = torch.randn(T, device=DEV, generator=g)
    r = mg.head_loss(x, w, t)
    e = ref.entries(targets=t)
    dlse = 0.3 * up
    dx, dw = mg.head_loss_bwd(x, w, t, r.lse, up, dlse=dlse)
    wx, ww, tx, tw = ref.backward(x, w, *e, r.lse, up, up.double() + dlse.double(), step=ref.H ** 2)
    _near("dx", dx, wx, tx)
    _near("dw", dw, ww, tw)
    teacher, index = _teacher(g, T, V, 5, torch.float32, ignored)
    index[T // 2, 0] = 0
    d = mg.head_distill(x, w, teacher, index, temperature=0.7)
    e = ref.entries(teacher=teacher, index=index, temperature=0.7)
    dx, dw = mg.head_distill_bwd(x, w, teacher, index, d.lse, d.logits, up, temperature=0.7)
    wx, ww, tx, tw = ref.backward(x, w, *e, d.lse, up, temperature=0.7, step=ref.H ** 2)
    _near("dx", dx, wx, tx)
    _near("dw", dw, ww, tw)


def test_buffers_that_overlap_are_refused():
    T, V, D = 20, 50, 64
    g, x, w = _inputs(T, V, D, 90)
    t = _targets(g, T, V, 0.0)
    r = mg.head_loss(x, w, t)
    room = torch.empty(T + V, D, dtype=torch.bfloat16, device=DEV)
    for buffers in (dict(dw=w), dict(dx=x), dict(dx=room[:T], dw=room[T - 1:T - 1 + V])):
        with pytest.raises(ValueError, match="overlap"):
            mg.head_loss_bwd(x, w, t, r.lse, r.loss, **buffers)
    dx, dw = mg.head_loss_bwd(x, w, t, r.lse, r.loss)
    ox, ow = mg.head_loss_bwd(x, w, t, r.lse, r.loss, dx=room[:T], dw=room[T:])       # side by side
    assert torch.equal(ox, dx) and torch.equal(ow, dw)
