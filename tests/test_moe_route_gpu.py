"""The router, its balance statistics and gradients, and the combine's
gradient against the 64-bit references on the GPU.

Tolerances.  Choices, counts and the row order are whole numbers: equal.  A
probability's exponent is (l - max) log2 e with two fp32 roundings of up to
2^-24 |l - max| log2 e (|l - max| <= 2^5 here: 2^-18 after the factor ln 2 and
both roundings), plus a few units of 2^-24 for the exponential, the sum and the
quotient: 2^-17 relative.  prob_sum adds at most 2^-20 of its value more.  A
gradient is a sum of a few such terms: 2^-15 of the sum of their magnitudes
(and half a bf16 step, 2^-8 of the value, for bf16 logits).
"""
import numpy as np
import pytest
import torch

import block_fp8_ref as ref
import moe_grouped_gemm_bf16_amd as mg

pytestmark = pytest.mark.gpu

P_TOL, G_TOL = 2.0 ** -17, 2.0 ** -15


def _say(*a):
    print("[case]", *a, flush=True)


def _np(t):
    return t.detach().cpu().numpy()


def _logits(T, E, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) * 2).to(dtype)


def _check_route(r, l, k, normalize, mask=None, first=0, local=None):
    want = ref.route(l.double().numpy(), k, normalize, None if mask is None else mask.numpy(), first, local)
    for name in ("experts", "counts", "tokens", "offsets", "gather", "token_rows"):
        assert (_np(getattr(r, name)) == want[name]).all(), name
    for name in ("weights", "lse", "prob_sum"):
        got, w = _np(getattr(r, name)).astype(np.float64), want[name]
        floor = 2.0 ** -20 if name == "lse" else 1e-37         # lse near 0: its terms are of order 1
        assert got.shape == w.shape and (np.abs(got - w) <= P_TOL * np.abs(w) + floor).all(), name
    loss = _np(r.loss).astype(np.float64)
    # z: lse enters squared; balance: counts times probabilities
    assert np.abs(loss - want["loss"]).max() <= 2 * P_TOL * np.abs(want["loss"]).max() + 1e-30
    return want


SHAPES = [(1, 1, 1), (1, 8, 2), (3, 16, 16), (16, 128, 8), (64, 33, 4), (65, 60, 4), (255, 64, 6), (256, 130, 8), (257, 256, 8),
          (1000, 100, 10), (4099, 31, 5), (300, 257, 3), (300, 512, 12), (70, 1000, 9), (300, 1024, 64), (20011, 72, 6)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_route(i, dtype):
    T, E, k = SHAPES[i]
    _say("route", T, E, k, dtype)
    l = _logits(T, E, dtype, i)
    _check_route(mg.moe_route(l.cuda(), k, normalize=i % 2 == 0), l, k, i % 2 == 0)


@pytest.mark.parametrize("T,E,k", [(256, 100, 64), (40000, 80, 40), (600000, 8, 4)])
def test_route_of_many_entries_per_workgroup(T, E, k):
    # more entries than a wave holds in registers between counting and placing.
    # prob_sum: at most 37 + 38 additions in a row, 2^-17.8, beside a
    # probability's 2^-18.5 (|l - max| < 20): within 2^-17
    _say("route entries", T, E, k)
    l = _logits(T, E, torch.float32, T)
    _check_route(mg.moe_route(l.cuda(), k), l, k, True)
    m = torch.rand(T, generator=torch.Generator().manual_seed(1)) < 0.9
    _check_route(mg.moe_route(l.cuda(), k, normalize=False, mask=m.cuda(), first=1, local=E - 3), l, k, False, m, 1, E - 3)


@pytest.mark.parametrize("T", [5, 700])
def test_route_mask_infinities_nan_and_lowest_values(T):
    _say("route masks", T)
    E, k = 24, 5
    for dtype in (torch.float32, torch.bfloat16):
        l = _logits(T, E, dtype, 40)
        low = torch.finfo(dtype).min
        l[:, 3] = -np.inf                       # an expert switched off
        l[:, 7] = float("nan")
        l[0] = -np.inf                          # nothing left
        l[1, 2:] = low                          # two real logits, the rest at the lowest value
        l[2] = low                              # all at the lowest value: uniform
        l[3, :20] = -np.inf                     # fewer than k
        l[4, 5], l[4, 6] = np.inf, np.inf
        mask = torch.ones(T, dtype=torch.bool)
        mask[T - T // 5:] = False
        l[T - 1] = float("nan")                 # in a masked place
        r = mg.moe_route(l.cuda(), k, mask=mask.cuda())
        want = ref.route(l.double().numpy(), k, True, mask.numpy())
        for name in ("experts", "counts", "tokens", "offsets", "gather", "token_rows"):
            assert (_np(getattr(r, name)) == want[name]).all(), name
        assert np.abs(_np(r.weights) - want["weights"]).max() <= P_TOL
        assert np.abs(_np(r.prob_sum) - want["prob_sum"]).max() <= P_TOL * max(1.0, want["prob_sum"].max())
        assert (_np(r.experts)[0] == -1).all() and (_np(r.weights)[0] == 0).all() and r.lse[0] == 0
        if T > 5:
            # gradients: zero where nothing counts, exact elsewhere
            dw = torch.randn(T, k, generator=torch.Generator().manual_seed(1))
            dl = torch.tensor([0.5, 0.0])
            d = _np(mg.moe_route_bwd(l.cuda(), r.weights, r.experts, r.lse, r.counts, r.tokens, dw.cuda(), dl.cuda()).float())
            g, mag = ref.route_bwd(want, dw.double().numpy(), dl.double().numpy(), True)
            step = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
            assert (np.abs(d - g) <= G_TOL * mag + step * np.abs(g) + 1e-37).all()
            off = (torch.isnan(l) | (l == -np.inf)).numpy()       # (row 2 has neither)
            assert (d[0] == 0).all() and (d[T - 1] == 0).all() and (d[off] == 0).all()


def test_route_ties_go_to_the_lower_index():
    _say("ties")
    l = torch.zeros(300, 130)
    l[:, 77] = 1.0
    r = mg.moe_route(l.cuda(), 4)
    assert (r.experts.cpu() == torch.tensor([77, 0, 1, 2])).all()
    _check_route(r, l, 4, True)


@pytest.mark.parametrize("T", [40, 3000])
@pytest.mark.parametrize("first,local", [(0, 8), (8, 16), (31, 1)])
def test_route_local_experts(T, first, local):
    _say("local", T, first, local)
    l = _logits(T, 32, torch.float32, 9)
    _check_route(mg.moe_route(l.cuda(), 3, first=first, local=local), l, 3, True, None, first, local)


def test_route_without_tokens():
    _say("no tokens")
    for mask in (None, torch.zeros(0, dtype=torch.uint8, device="cuda")):
        r = mg.moe_route(torch.zeros(0, 40, device="cuda"), 2, mask=mask)
        for t in (r.counts, r.prob_sum, r.tokens, r.loss, r.offsets):
            assert (t == 0).all()
        assert r.gather.numel() == 0 and r.offsets.numel() == 41
    d = mg.moe_route_bwd(torch.zeros(0, 40, device="cuda"), r.weights, r.experts, r.lse, r.counts, r.tokens)
    assert d.shape == (0, 40)
    r = mg.moe_route(torch.randn(900, 40, device="cuda"), 2, mask=torch.zeros(900, dtype=torch.bool, device="cuda"))
    for t in (r.counts, r.prob_sum, r.tokens, r.loss, r.offsets, r.lse, r.weights):
        assert (t == 0).all()
    assert (r.gather == -1).all() and (r.token_rows == -1).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (17, 60, 4), (130, 128, 8), (333, 256, 8), (90, 300, 3), (50, 1024, 64), (5000, 40, 5)])
def test_route_gradient(T, E, k, normalize, dtype):
    _say("route_bwd", T, E, k, normalize, dtype)
    l = _logits(T, E, dtype, T + E)
    ld = l.cuda()
    r = mg.moe_route(ld, k, normalize=normalize)
    want = ref.route(l.double().numpy(), k, normalize)
    g = torch.Generator().manual_seed(3)
    dw = torch.randn(T, k, generator=g)
    dl = torch.tensor([0.3, 0.1])
    for a, b in ((dw, dl), (dw, None), (None, dl), (None, None)):
        d = mg.moe_route_bwd(ld, r.weights, r.experts, r.lse, r.counts, r.tokens, None if a is None else a.cuda(),
                             None if b is None else b.cuda(), normalize=normalize)
        assert d.dtype == dtype
        exact, mag = ref.route_bwd(want, None if a is None else a.double().numpy(), np.zeros(2) if b is None else b.double().numpy(), normalize)
        step = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
        err = np.abs(_np(d.float()) - exact)
        # (bf16: a value below 2^-133 is a subnormal half step off at most)
        assert (err <= G_TOL * mag + step * np.abs(exact) + 1e-37).all(), float((err / np.maximum(G_TOL * mag + step * np.abs(exact), 1e-300)).max())


def test_route_gradient_against_differences_of_the_kernel_s_own_losses():
    """The losses' gradient along a direction against differences of moe_route's
    losses (counts unchanged by a small step)."""
    _say("differences")
    T, E, k = 400, 32, 4
    l = _logits(T, E, torch.float32, 77)
    r = mg.moe_route(l.cuda(), k)
    u = torch.randn(T, E, generator=torch.Generator().manual_seed(5))
    h = 2.0 ** -7
    up, dn = mg.moe_route((l + h * u).cuda(), k), mg.moe_route((l - h * u).cuda(), k)
    f = _np(r.counts) / _np(r.counts).sum()
    for i, dl in ((0, [1.0, 0.0]), (1, [0.0, 1.0])):
        d = mg.moe_route_bwd(l.cuda(), r.weights, r.experts, r.lse, r.counts, r.tokens, None, torch.tensor(dl).cuda())
        along = (_np(d).astype(np.float64) * u.double().numpy()).sum()
        if i == 0:            # counts held fixed
            vals = [E * (f * _np(x.prob_sum).astype(np.float64)).sum() / T for x in (up, dn)]
        else:
            vals = [float(x.loss[1]) for x in (up, dn)]
        diff = (vals[0] - vals[1]) / (2 * h)
        # 2^-17 of a value of order 1 (balance) or 16 (z) over 2 h = 2^-6, and h^2 times a third derivative of order 1
        assert abs(diff - along) <= (2.0 ** -11 if i == 0 else 2.0 ** -7) + h * h


def test_counts_summed_over_ranks_enter_the_gradient():
    _say("summed counts")
    l = _logits(200, 16, torch.float32, 8)
    r = mg.moe_route(l.cuda(), 2)
    want = ref.route(l.double().numpy(), 2, True)
    more = torch.arange(16, dtype=torch.int32)
    want["counts"] = want["counts"] + more.numpy()
    want["tokens"] = want["tokens"] + 60
    d = mg.moe_route_bwd(l.cuda(), r.weights, r.experts, r.lse, r.counts + more.cuda(), r.tokens + 60, None, torch.tensor([1.0, 1.0]).cuda())
    exact, mag = ref.route_bwd(want, None, np.array([1.0, 1.0]), True)
    assert (np.abs(_np(d) - exact) <= G_TOL * mag).all()


def test_counts_over_ranks_that_pass_31_bits_together():
    _say("large counts")
    l = _logits(200, 16, torch.float32, 8)
    r = mg.moe_route(l.cuda(), 2)
    want = ref.route(l.double().numpy(), 2, True)
    counts = torch.full((16,), 1 << 28, dtype=torch.int32)                  # 2^32 in all
    counts[3] = (1 << 31) - 1
    want["counts"], want["tokens"] = counts.numpy().astype(np.int64), np.array([(1 << 31) - 1], np.int64)
    d = mg.moe_route_bwd(l.cuda(), r.weights, r.experts, r.lse, counts.cuda(), torch.full((1,), (1 << 31) - 1, dtype=torch.int32, device="cuda"),
                         None, torch.tensor([1e9, 1e9]).cuda())
    exact, mag = ref.route_bwd(want, None, np.array([1e9, 1e9]), True)
    assert (np.abs(_np(d) - exact) <= G_TOL * mag).all()


@pytest.mark.parametrize("T,k,D", [(1, 1, 8), (5, 8, 264), (100, 3, 2048), (33, 64, 520), (300, 2, 72)])
def test_combine_gradient(T, k, D):
    _say("combine_bwd", T, k, D)
    rng = np.random.default_rng(T * k)
    M = T * k + 5
    rows_at = rng.permutation(M)[:T * k].astype(np.int32).reshape(T, k)
    rows_at[rng.random((T, k)) < 0.2] = -1
    rows_at[0, 0] = M + 3 if T > 1 else rows_at[0, 0]           # out of range: no row
    dout, rows = (torch.from_numpy(rng.standard_normal(s)).bfloat16() for s in ((T, D), (M, D)))
    w = torch.from_numpy(rng.standard_normal((T, k))).float()
    drows = torch.full((M, D), 3.0, dtype=torch.bfloat16, device="cuda")
    got, dw = mg.moe_combine_bwd(dout.cuda(), rows.cuda(), torch.from_numpy(rows_at).cuda(), w.cuda(), drows=drows)
    want, wd, mag = np.full((M, D), 3.0), np.zeros((T, k)), np.zeros((T, k))
    a, b = dout.double().numpy(), rows.double().numpy()
    for t in range(T):
        for j in range(k):
            r = rows_at[t, j]
            if 0 <= r < M:
                want[r] = float(w[t, j]) * a[t]
                wd[t, j], mag[t, j] = (b[r] * a[t]).sum(), np.abs(b[r] * a[t]).sum()
    # one fp32 and one bf16 rounding; a dot product of D terms, each lane's D / 64 and six more adds in order
    assert (np.abs(_np(got.float()) - want) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(want)).all()
    assert (np.abs(_np(dw) - wd) <= (D / 64 + 16) * 2.0 ** -24 * mag).all()
    ones, none = mg.moe_combine_bwd(dout.cuda(), rows.cuda(), torch.from_numpy(rows_at).cuda())
    assert none is None
    for t in range(T):
        for j in range(k):
            if 0 <= rows_at[t, j] < M:
                assert torch.equal(ones[rows_at[t, j]].cpu(), dout[t])
    named = np.unique(rows_at[(rows_at >= 0) & (rows_at < M)])
    assert (_np(ones.float())[np.setdiff1d(np.arange(M), named)] == 0).all()


def test_combine_gradient_matches_the_combine():
    """<combine(rows, w), g> has the gradient that moe_combine_bwd gives: its
    directional derivative against the forward kernel itself."""
    _say("combine identity")
    T, k, D = 64, 4, 512
    g = torch.Generator().manual_seed(2)
    rows_at = torch.randperm(T * k, generator=g).int().view(T, k).cuda()
    rows, dout = (torch.randn(n, D, generator=g).bfloat16().cuda() for n in (T * k, T))
    w = torch.randn(T, k, generator=g).cuda()
    drows, dw = mg.moe_combine_bwd(dout, rows, rows_at, w)
    y = mg.moe_combine(rows, rows_at, w).double()
    a = float((y * dout.double()).sum())
    b = float((rows.double() * drows.double()).sum())
    c = float((w.double() * dw.double()).sum())
    mag = float((y.abs() * dout.double().abs()).sum() + (rows.double() * drows.double()).abs().sum())
    assert abs(a - b) <= 2.0 ** -8 * mag and abs(a - c) <= 2.0 ** -8 * mag


def test_route_replayed_graph_and_streams():
    _say("route graph")
    for T in (100, 3000):
        l = _logits(T, 64, torch.float32, T).cuda()
        dw, dl = torch.randn(T, 6, device="cuda"), torch.tensor([0.1, 0.2], device="cuda")
        rows, dout = (torch.randn(n, 64, device="cuda").bfloat16() for n in (6 * T, T))

        def chain():
            r = mg.moe_route(l, 6)
            d = mg.moe_route_bwd(l, r.weights, r.experts, r.lse, r.counts, r.tokens, dw, dl)
            return [*r, d, *mg.moe_combine_bwd(dout, rows, r.token_rows, r.weights)]
        chain()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kept = chain()
        streams = [torch.cuda.Stream() for _ in range(2)]
        for i in range(3):
            l.copy_(l.roll(1, 1))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            eager = chain()
            outs = []
            torch.cuda.synchronize()
            for st in streams:
                with torch.cuda.stream(st):
                    outs.append(chain())
            torch.cuda.synchronize()
            for n, (a, b) in enumerate(zip(kept, eager)):
                assert torch.equal(a, b), (i, n)
                assert all(torch.equal(o[n], b) for o in outs)


def test_sums_over_ranks_in_place_leave_the_saved_outputs_valid():
    r = mg.moe_route(_logits(40, 16, torch.float32, 3).cuda(), 2)
    for t in (r.counts, r.tokens, r.prob_sum):
        t.add_(1)
    assert all(t._version == 0 for t in (r.weights, r.experts, r.lse, r.loss, r.offsets, r.gather, r.token_rows))


def test_bindings_refuse():
    l = torch.zeros(6, 8, device="cuda")
    with pytest.raises(ValueError, match="k must be"):
        mg.moe_route(l, 9)
    with pytest.raises(ValueError, match="k must be"):
        mg.moe_route(l, 0)
    with pytest.raises(ValueError, match="not among"):
        mg.moe_route(l, 2, first=4, local=5)
    with pytest.raises(ValueError, match="mask"):
        mg.moe_route(l, 2, mask=torch.ones(5, dtype=torch.bool, device="cuda"))
    with pytest.raises(TypeError, match="mask"):
        mg.moe_route(l, 2, mask=torch.ones(6, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        mg.moe_route(torch.zeros(8, 6, device="cuda").t(), 2)
    with pytest.raises(mg.MgemmError):
        mg.moe_route(torch.zeros(2, 1025, device="cuda"), 2)
    r = mg.moe_route(l, 2)
    with pytest.raises(ValueError, match="dloss"):
        mg.moe_route_bwd(l, r.weights, r.experts, r.lse, r.counts, r.tokens, dloss=torch.zeros(3, device="cuda"))
    with pytest.raises(ValueError, match="dweights"):
        mg.moe_route_bwd(l, r.weights, r.experts, r.lse, r.counts, r.tokens, dweights=torch.zeros(6, 3, device="cuda"))
    with pytest.raises(ValueError, match="entries"):
        mg.moe_route_bwd(l, r.weights, r.experts, r.lse, r.counts[:7].contiguous(), r.tokens)
    x = torch.zeros(12, 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="dout"):
        mg.moe_combine_bwd(x, x, r.token_rows, r.weights)
