"""Block-scaled fp8 quantizers and products against the 64-bit references on
the GPU.

Tolerances.  A bf16 result is off by at most half a step, 2^-8 of its value.
The matrix core sums a block's 128 products after aligning them to the largest
and dropping low bits: within 2^-11 of the sum of the magnitudes, whatever the
values (measured at most 2^-11.5 on magnitudes spread over 2^+-12, 2^-14.7 on
normals).  The fp32 fmas over the blocks add (blocks + 4) 2^-24 of the same
sum, under 2^-14 for any reduction here; 2^-10.8 covers both.  Products of
small integers with power-of-two scales are exact in every order, so there the
bf16 bits must be those of the exact sum.  The quantizers' arithmetic is a
correctly rounded fp32 sequence: codes and scales must be the reference's bits.
"""
import numpy as np
import pytest
import torch

import block_fp8_ref as ref
import moe_grouped_gemm_bf16_amd as mg

pytestmark = pytest.mark.gpu

SUM_TOL = 2.0 ** -10.8
BF16 = 2.0 ** -8


def _say(*a):
    print("[case]", *a, flush=True)


def _np(t):
    return t.detach().cpu().numpy()


def _offsets(sizes):
    return np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _operands(sizes, N, K, dgrad, seed, extra=0, spread=0.0):
    """Random codes and scales: (q, s, w8, ws, off) as arrays."""
    rng = np.random.default_rng(seed)
    M, R, E = sum(sizes) + extra, N if dgrad else K, len(sizes)
    x = rng.standard_normal((M, R)) * np.exp2(spread * rng.standard_normal((M, R)))
    w = rng.standard_normal((E * N, K))
    q, s = ref.quantize(x, 1)
    w8, ws = np.zeros((E, N, K), np.uint8), np.zeros((E, -(-N // 128), -(-K // 128)), np.float32)
    for e in range(E):
        w8[e], ws[e] = ref.quantize(w[e * N:(e + 1) * N], 128)
    ws *= np.exp2(rng.integers(-3, 4, ws.shape)).astype(np.float32)       # blocks differ
    return q, np.ascontiguousarray(s.T), w8, ws, _offsets(sizes)


def _call(dgrad, q, s, w8, ws, off, **kw):
    f = mg.dgrad_fp8 if dgrad else mg.fwd_fp8
    return f(_dev(q), _dev(s), _dev(w8), _dev(ws), _dev(off), **kw)


def _check(got, q, s, w8, ws, off, dgrad):
    exact, mag = ref.product(ref.dequant_rows(q, s), ref.dequant_weights(w8, ws), off, dgrad)
    o = int(off[-1])
    got = _np(got.float())[:o].astype(np.float64)
    err = np.abs(got - exact[:o])
    tol = BF16 * np.abs(exact[:o]) + SUM_TOL * mag[:o]
    assert np.isfinite(got).all() and (err <= tol).all(), float((err / np.maximum(tol, 1e-300)).max())


# rows per expert, N, K: one row; odd widths; empty experts; rows that end a
# tile, start one and cross several; long reductions; the few-row form's cases
PRODUCTS = [
    ([1], 16, 16), ([1], 128, 128), ([5, 0, 3], 48, 272), ([0, 0, 7, 0], 144, 2064),
    ([200, 0, 184, 128], 128, 256), ([127, 128, 129, 0, 1], 272, 400), ([300], 1040, 144),
    ([33, 64, 2, 0, 0, 95], 400, 720), ([1] * 40, 96, 1168), ([2, 0, 1, 17, 33, 0, 0, 0], 176, 4112),
    ([257, 40], 384, 1536),
]


@pytest.mark.parametrize("dgrad", [False, True])
@pytest.mark.parametrize("i", range(len(PRODUCTS)))
def test_product_against_exact_sums(i, dgrad):
    sizes, N, K = PRODUCTS[i]
    _say("product", sizes, N, K, "dgrad" if dgrad else "fwd")
    ops = _operands(sizes, N, K, dgrad, 100 + i, extra=3, spread=1.0 if i % 2 else 0.0)
    _check(_call(dgrad, *ops), *ops, dgrad)


@pytest.mark.parametrize("dgrad", [False, True])
@pytest.mark.parametrize("sizes", [[3, 0, 2], [150, 0, 133, 6]])
def test_product_of_small_integers_is_the_exact_sum_rounded(sizes, dgrad):
    _say("integers", sizes, dgrad)
    N, K, E = 272, 656, len(sizes)
    rng = np.random.default_rng(7)
    M, R = sum(sizes), N if dgrad else K
    q = ref.encode(rng.integers(-3, 4, (M, R)))
    w8 = ref.encode(rng.integers(-3, 4, (E, N, K)))
    s = np.exp2(rng.integers(0, 4, (-(-R // 128), M))).astype(np.float32)
    ws = np.exp2(rng.integers(-2, 2, (E, -(-N // 128), -(-K // 128)))).astype(np.float32)
    off = _offsets(sizes)
    exact, _ = ref.product(ref.dequant_rows(q, s), ref.dequant_weights(w8, ws), off, dgrad)
    want = torch.from_numpy(exact).float().bfloat16()           # |sum| 2^2 < 2^24: exact in fp32
    assert torch.equal(_call(dgrad, q, s, w8, ws, off).cpu(), want)


@pytest.mark.parametrize("dgrad", [False, True])
@pytest.mark.parametrize("sizes", [[2, 1], [130, 70]])
def test_rows_behind_the_last_are_left_and_hints_do_not_matter(sizes, dgrad):
    _say("tail", sizes, dgrad)
    N, K = 144, 272
    ops = _operands(sizes, N, K, dgrad, 11, extra=40)
    for hint in (0, 1, 10 ** 6):
        out = torch.full((sum(sizes) + 40, K if dgrad else N), 7.0, dtype=torch.bfloat16, device="cuda")
        got = _call(dgrad, *ops, max_m_per_e=hint, out=out)
        assert got is out
        _check(out, *ops, dgrad)
        assert (out[sum(sizes):] == 7.0).all()


@pytest.mark.parametrize("dgrad", [False, True])
def test_nan_stays_in_its_row_and_its_weights_outputs(dgrad):
    _say("nan", dgrad)
    sizes, N, K = [40, 0, 9], 256, 272
    for rows in (sizes, [2, 0, 1]):
        q, s, w8, ws, off = _operands(rows, N, K, dgrad, 12)
        q[1, 5] = 0x7F
        s[1, 2] = np.inf                     # an infinite scale: that row only
        M = sum(rows)
        bad = np.zeros(M, bool)
        bad[[1, 2]] = True
        got = _np(_call(dgrad, q, s, w8, ws, off).float())
        assert np.isnan(got[1]).all() and not np.isfinite(got[2]).any() and np.isfinite(got[~bad]).all()


def test_reduction_of_length_zero_writes_zeros():
    _say("empty reduction")
    off = torch.tensor([0, 3, 5], dtype=torch.int32, device="cuda")
    u8 = dict(dtype=torch.uint8, device="cuda")
    out = torch.full((8, 32), 5.0, dtype=torch.bfloat16, device="cuda")
    mg.fwd_fp8(torch.zeros(8, 0, **u8), torch.zeros(0, 8, device="cuda"), torch.zeros(2, 32, 0, **u8), torch.zeros(2, 1, 0, device="cuda"), off, out=out)
    assert (out[:5] == 0).all() and (out[5:] == 5.0).all()
    out.fill_(5.0)
    mg.dgrad_fp8(torch.zeros(8, 0, **u8), torch.zeros(0, 8, device="cuda"), torch.zeros(2, 0, 32, **u8), torch.zeros(2, 0, 1, device="cuda"), off, out=out)
    assert (out[:5] == 0).all() and (out[5:] == 5.0).all()
    y = mg.fwd_fp8(torch.zeros(0, 32, **u8), torch.zeros(1, 0, device="cuda"), torch.zeros(2, 32, 32, **u8), torch.zeros(2, 1, 1, device="cuda"), off * 0)
    assert y.shape == (0, 32)


def test_products_past_32_bit_offsets():
    # 5.4 GB of weights, the last expert's beyond 2^32 bytes
    E, N, K, M = 21, 16384, 15728, 300
    _say("large", E, N, K)
    torch.manual_seed(0)
    w8 = torch.randint(0, 120, (E, N, K), dtype=torch.uint8, device="cuda")
    ws = torch.rand(E, N // 128, -(-K // 128), device="cuda") * 1e-4
    off = torch.tensor([0] * E + [M], dtype=torch.int32, device="cuda")
    for dgrad in (False, True):
        R = N if dgrad else K
        q = torch.randint(0, 120, (M, R), dtype=torch.uint8, device="cuda")
        s = torch.rand(-(-R // 128), M, device="cuda") * 1e-4
        y = (mg.dgrad_fp8 if dgrad else mg.fwd_fp8)(q, s, w8, ws, off)
        table = torch.from_numpy(ref.e4m3_values()).cuda()
        rows = torch.tensor([0, 127, 299], device="cuda")
        x = table[q[rows].int()] * s[:, rows].t().double().repeat_interleave(128, 1)[:, :R]
        cols = torch.tensor([0, 1, 5000, (K if dgrad else N) - 1], device="cuda")
        blk = ws[-1].double()
        if dgrad:
            w = table[w8[-1][:, cols].int()] * blk[:, cols // 128].repeat_interleave(128, 0)
            want = (x[:, :, None] * w[None]).sum(1)
        else:
            w = table[w8[-1][cols].int()] * blk[cols // 128].repeat_interleave(128, 1)[:, :K]
            want = (x[:, None] * w[None]).sum(2)
        got = y[rows][:, cols].double()
        assert ((got - want).abs() <= (BF16 + SUM_TOL) * want.abs()).all()        # all terms positive


def _sampled(q, s, w8, ws, dgrad, y, rows, cols):
    """Outputs (rows, cols) of the last expert against exact sums, all terms positive."""
    table = torch.from_numpy(ref.e4m3_values()).cuda()
    R, K = q.shape[1], w8.shape[2]
    x = table[q[rows].int()] * s[:, rows].t().double().repeat_interleave(128, 1)[:, :R]
    blk = ws[-1].double()
    if dgrad:
        want = torch.stack([(x * (table[w8[-1][:, c].int()] * blk[:, c // 128].repeat_interleave(128)[:R])).sum(1) for c in cols.tolist()], 1)
    else:
        w = table[w8[-1][cols].int()] * blk[cols // 128].repeat_interleave(128, 1)[:, :K]
        want = (x[:, None] * w[None]).sum(2)
    # a block's sum 2^-11, the fmas over the blocks, the result's rounding
    tol = BF16 + 2.0 ** -11 + (-(-R // 128) + 4) * 2.0 ** -24
    assert ((y[rows][:, cols].double() - want).abs() <= tol * want.abs()).all()


@pytest.mark.parametrize("M", [100, 700])
def test_every_form_past_32_bit_offsets(M):
    # 5.4 GB of weights; 100 rows take the few-row forms, 700 the tiled ones
    E, N, K = 21, 16384, 15728
    _say("large", E, N, K, M)
    g = torch.Generator("cuda").manual_seed(M)
    d = dict(device="cuda", generator=g)
    w8 = torch.randint(0, 120, (E, N, K), dtype=torch.uint8, **d)
    ws = torch.rand(E, N // 128, -(-K // 128), **d) * 1e-4
    off = torch.tensor([0] * E + [M], dtype=torch.int32, device="cuda")
    for dgrad in (False, True):
        R = N if dgrad else K
        q, s = torch.randint(0, 120, (M, R), dtype=torch.uint8, **d), torch.rand(-(-R // 128), M, **d) * 1e-4
        y = (mg.dgrad_fp8 if dgrad else mg.fwd_fp8)(q, s, w8, ws, off)
        _sampled(q, s, w8, ws, dgrad, y, torch.tensor([0, 31, 64, M - 1], device="cuda"), torch.tensor([0, 1, 5000, (K if dgrad else N) - 1], device="cuda"))


@pytest.mark.parametrize("M,P,R", [(3, 128, 2 ** 22), (70, 64, 2 ** 22), (300, 8208, 2 ** 18)])
def test_long_reductions(M, P, R):
    _say("long", M, P, R)
    g = torch.Generator("cuda").manual_seed(R)
    d = dict(device="cuda", generator=g)
    off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    for dgrad in (False, True):
        N, K = (R, P) if dgrad else (P, R)
        w8, ws = torch.randint(0, 100, (1, N, K), dtype=torch.uint8, **d), torch.rand(1, -(-N // 128), -(-K // 128), **d) * 1e-4
        q, s = torch.randint(0, 100, (M, R), dtype=torch.uint8, **d), torch.rand(-(-R // 128), M, **d) * 1e-4
        y = (mg.dgrad_fp8 if dgrad else mg.fwd_fp8)(q, s, w8, ws, off)
        _sampled(q, s, w8, ws, dgrad, y, torch.tensor([0, M - 1], device="cuda"), torch.tensor([0, 63, P - 1], device="cuda"))


def test_two_streams_and_a_replayed_graph_give_the_eager_bits():
    _say("streams and graph")
    cases = [(False, *_operands([130, 0, 61], 272, 400, False, 21)), (False, *_operands([2, 0, 1], 272, 400, False, 22)),
             (True, *_operands([130, 0, 61], 272, 400, True, 23))]
    dev = [(d, [_dev(a) for a in ops]) for d, *ops in cases]
    run = lambda d, a, out=None: (mg.dgrad_fp8 if d else mg.fwd_fp8)(*a, out=out)   # noqa: E731
    want = [run(d, a) for d, a in dev]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for st in streams:
        with torch.cuda.stream(st):
            got.append([run(d, a) for _ in range(3) for d, a in dev])
    torch.cuda.synchronize()
    for g in got:
        for i, y in enumerate(g):
            assert torch.equal(y, want[i % len(dev)])
    outs = [torch.zeros_like(w) for w in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for (d, a), o in zip(dev, outs):
            run(d, a, o)
    for i in range(3):
        for o in outs:
            o.zero_()
        # other operands in place before the second and third replay
        for _, a in dev:
            a[0].copy_(a[0].roll(1, 0))
        graph.replay()
        torch.cuda.synchronize()
        for (d, a), o in zip(dev, outs):
            assert torch.equal(o, run(d, a)), i


# -- the tiled forms: enough 64-column pieces that the few-row form is not taken -----

# rows per expert, output width, reduction; in the large tiles the last three
TILED = [
    ([300], 8208, 144), ([127, 128, 129, 0, 1], 8208, 400), ([257, 40], 8400, 1536), ([33, 64, 2, 0, 0, 95], 8208, 720),
    ([200, 0, 184, 128], 8192, 16), ([4097], 8208, 144), ([2100, 0, 1877, 3], 8208, 272), ([1500, 0, 3000, 70, 1], 8336, 1040),
    ([3400], 8208, 144), ([1700, 0, 1620, 3], 8208, 272),
]


def _random_operands(sizes, P, R, dgrad, seed, extra=0):
    """Random codes and scales as device tensors: (q, s, w8, ws, off)."""
    g = torch.Generator("cuda").manual_seed(seed)
    N, K = (R, P) if dgrad else (P, R)
    M, E, d = sum(sizes) + extra, len(sizes), dict(device="cuda", generator=g)
    code = lambda *shape: torch.randint(0, 120, shape, dtype=torch.uint8, **d) | (torch.randint(0, 2, shape, dtype=torch.uint8, **d) << 7)  # noqa: E731
    scale = lambda *shape: torch.rand(shape, **d) + 0.5                                                                                 # noqa: E731
    return code(M, R), scale(-(-R // 128), M), code(E, N, K), scale(E, -(-N // 128), -(-K // 128)), torch.from_numpy(_offsets(sizes)).cuda()


def _exact_on_device(q, s, w8, ws, off, dgrad):
    """Exact sums and sums of the magnitudes, fp64."""
    table = torch.from_numpy(ref.e4m3_values()).cuda()
    R, N, K = q.shape[1], w8.shape[1], w8.shape[2]
    x = table[q.int()] * s.t().double().repeat_interleave(128, 1)[:, :R]
    out = [torch.zeros(q.shape[0], K if dgrad else N, dtype=torch.float64, device="cuda") for _ in range(2)]
    off = off.tolist()
    for e in range(len(off) - 1):
        w = table[w8[e].int()] * ws[e].double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
        w = w if dgrad else w.t().contiguous()
        rows = slice(off[e], off[e + 1])
        out[0][rows], out[1][rows] = x[rows] @ w, x[rows].abs() @ w.abs()
    return out


@pytest.mark.parametrize("dgrad", [False, True])
@pytest.mark.parametrize("i", range(len(TILED)))
def test_tiled_product_against_exact_sums(i, dgrad):
    sizes, P, R = TILED[i]
    _say("tiled", sizes, P, R, "dgrad" if dgrad else "fwd")
    ops = _random_operands(sizes, P, R, dgrad, 200 + i, extra=5)
    M = sum(sizes)
    exact, mag = _exact_on_device(*ops, dgrad)
    for hint in (0, 1, max(sizes)):
        out = torch.full((M + 5, P), 7.0, dtype=torch.bfloat16, device="cuda")
        (mg.dgrad_fp8 if dgrad else mg.fwd_fp8)(*ops, max_m_per_e=hint, out=out)
        assert (out[M:] == 7.0).all()
        err = (out[:M].double() - exact[:M]).abs()
        assert (err <= BF16 * exact[:M].abs() + SUM_TOL * mag[:M]).all(), hint


@pytest.mark.parametrize("dgrad", [False, True])
@pytest.mark.parametrize("sizes", [[150, 0, 133, 6], [3000, 0, 1100]])
def test_tiled_product_of_small_integers_is_the_exact_sum_rounded(sizes, dgrad):
    _say("tiled integers", sizes, dgrad)
    P, R = 8208, 656
    g = torch.Generator("cuda").manual_seed(8)
    d = dict(device="cuda", generator=g)
    codes = torch.from_numpy(ref.encode(np.arange(-3, 4))).cuda()
    N, K = (R, P) if dgrad else (P, R)
    M, E = sum(sizes), len(sizes)
    q, w8 = codes[torch.randint(0, 7, (M, R), **d)], codes[torch.randint(0, 7, (E, N, K), **d)]
    s = torch.exp2(torch.randint(0, 4, (-(-R // 128), M), **d).float())
    ws = torch.exp2(torch.randint(-2, 2, (E, -(-N // 128), -(-K // 128)), **d).float())
    off = torch.from_numpy(_offsets(sizes)).cuda()
    exact, _ = _exact_on_device(q, s, w8, ws, off, dgrad)
    # |sum| <= 656 * 9 * 8 * 2 < 2^17 in steps of 2^-2: exact in fp32 in any order
    assert torch.equal((mg.dgrad_fp8 if dgrad else mg.fwd_fp8)(q, s, w8, ws, off), exact.float().bfloat16())


@pytest.mark.parametrize("dgrad", [False, True])
@pytest.mark.parametrize("sizes", [[140, 0, 129], [3000, 0, 1100]])
def test_tiled_nan_stays_in_its_row(sizes, dgrad):
    _say("tiled nan", sizes, dgrad)
    q, s, w8, ws, off = _random_operands(sizes, 8208, 272, dgrad, 13)
    q[1, 5] = 0x7F
    s[1, 2] = np.inf
    # behind the last row of a tile and of an expert
    q[128, 0] = 0xFF
    bad = torch.zeros(sum(sizes), dtype=torch.bool, device="cuda")
    bad[[1, 2, 128]] = True
    got = (mg.dgrad_fp8 if dgrad else mg.fwd_fp8)(q, s, w8, ws, off)
    assert torch.isnan(got[1]).all() and not torch.isfinite(got[2]).any() and torch.isnan(got[128]).all()
    assert torch.isfinite(got[~bad]).all()


def test_tiled_products_on_two_streams_and_in_a_graph():
    _say("tiled graph")
    dev = [(d, _random_operands(n, 8208, 400, d, 30)) for d in (False, True) for n in ([130, 0, 61], [3000, 0, 1100])]
    run = lambda d, a, out=None: (mg.dgrad_fp8 if d else mg.fwd_fp8)(*a, out=out)   # noqa: E731
    want = [run(d, a) for d, a in dev]
    torch.cuda.synchronize()
    got = []
    for st in [torch.cuda.Stream() for _ in range(2)]:
        with torch.cuda.stream(st):
            got.append([run(d, a) for _ in range(2) for d, a in dev])
    torch.cuda.synchronize()
    for y in got:
        assert all(torch.equal(v, want[i % len(dev)]) for i, v in enumerate(y))
    outs = [torch.zeros_like(w) for w in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for (d, a), o in zip(dev, outs):
            run(d, a, o)
    for i in range(3):
        for o in outs:
            o.zero_()
        for _, a in dev:
            a[0].copy_(a[0].roll(1, 0))
        graph.replay()
        torch.cuda.synchronize()
        for (d, a), o in zip(dev, outs):
            assert torch.equal(o, run(d, a)), i


# -- quantizers ------------------------------------------------------------------

def _rows_input(M, K, dtype, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K)) * np.exp2(rng.integers(-8, 9, (M, 1)))
    x[rng.random(M) < 0.1] = 0.0
    return torch.from_numpy(x).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", [(1, 16), (1, 2048), (31, 144), (32, 512), (33, 528), (100, 1040), (7, 7168)])
def test_quantize_rows_bits(M, K, dtype):
    _say("quantize", M, K, dtype)
    x = _rows_input(M, K, dtype, M + K)
    codes, scales = mg.fp8_quantize(x.cuda())
    want, ws = ref.quantize(x.float().numpy(), 1)
    assert (_np(codes) == want).all() and (_np(scales) == ws.T).all()
    assert codes.shape == (M, K) and scales.shape == (-(-K // 128), M)


def test_quantize_gathers_skips_the_tail_and_zeroes_bad_indexes():
    _say("quantize gather")
    T, K, M = 20, 272, 70
    x = _rows_input(T, K, torch.bfloat16, 5)
    rng = np.random.default_rng(6)
    g = rng.integers(0, T, M).astype(np.int32)
    g[[3, 50]] = [-1, T]                                   # out of range: zeros
    off = _offsets([20, 0, 41])
    codes = torch.full((M, K), 9, dtype=torch.uint8, device="cuda")
    scales = torch.full((3, M), -1.0, device="cuda")
    r = mg.fp8_quantize(x.cuda(), gather=_dev(g), offsets=_dev(off), out=codes, scales=scales)
    assert r[0] is codes and r[1] is scales
    rows = np.where(((g < 0) | (g >= T))[:, None], 0.0, x.float().numpy()[np.clip(g, 0, T - 1)])
    want, ws = ref.quantize(rows, 1)
    assert (_np(codes)[:61] == want[:61]).all() and (_np(scales)[:, :61] == ws.T[:, :61]).all()
    assert (codes[61:] == 9).all() and (scales[:, 61:] == -1.0).all()
    empty = mg.fp8_quantize(x.cuda()[:0], gather=_dev(g))          # no rows to gather from
    assert (empty[0] == 0).all()


def test_quantize_extremes():
    _say("quantize extremes")
    x = np.zeros((6, 128), np.float32)
    x[0, 3] = 3.3e38                       # the scale's inverse is tiny
    x[1, :] = 1e-42                        # below the floor of the scale, subnormal
    x[2, 5], x[2, 6] = np.nan, 1.0
    x[3, 5], x[3, 6] = np.inf, 1.0
    x[4, :] = -448.0 * 2.0 ** -90
    x[5, 0], x[5, 1] = 2.0 ** -100, -(2.0 ** -101)
    codes, scales = (_np(t) for t in mg.fp8_quantize(torch.from_numpy(x).cuda()))
    assert codes[0, 3] == 126 and np.isfinite(scales[0, 0])
    assert (codes[1] == 0).all()
    assert (codes[2, 5] & 127) == 127 and codes[2, 6] == 126
    assert (codes[3, 5] & 127) == 127 and np.isinf(scales[0, 3])
    assert (codes[4] == 254).all() and scales[0, 4] == np.float32(2.0 ** -90)
    assert codes[5, 0] == 126 and codes[5, 1] == 0x80 | ref.encode(224.0)


@pytest.mark.parametrize("M,I", [(1, 16), (33, 144), (64, 1408)])
def test_quantize_swiglu(M, I):
    _say("quantize swiglu", M, I)
    rng = np.random.default_rng(M + I)
    gu = torch.from_numpy(rng.standard_normal((M, 2 * I)) * 3).bfloat16()
    gu[0, 0], gu[0, I] = -200.0, 50.0                  # silu underflows to -0
    codes, scales = (_np(t) for t in mg.fp8_quantize_swiglu(gu.cuda()))
    g, u = gu.double().numpy()[:, :I], gu.double().numpy()[:, I:]
    h = g / (1 + np.exp(-g)) * u
    nb = -(-I // 128)
    amax = np.stack([np.abs(h[:, 128 * b:128 * b + 128]).max(1) for b in range(nb)])
    # exponential, reciprocal and two products: a few 2^-24 each, the exponent's
    # argument |g| log2 e < 2^5 rounded before it: 2^-18 in all
    assert (np.abs(scales - amax / 448) <= 2.0 ** -18 * amax / 448).all()
    back = ref.dequant_rows(codes, scales)
    step = np.repeat(scales.T.astype(np.float64), 128, 1)[:, :I] * 2.0 ** -10
    assert (np.abs(back - h) <= (2.0 ** -4 + 2.0 ** -17) * np.abs(h) + step).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E,N,K", [(1, 1, 16), (2, 128, 128), (3, 130, 272), (2, 40, 1040)])
def test_quantize_weights_bits(E, N, K, dtype):
    _say("quantize weights", E, N, K, dtype)
    w = (torch.from_numpy(np.random.default_rng(E + N).standard_normal((E, N, K))) / 16).to(dtype)
    w[0, :, :16] = 0
    codes, scales = mg.fp8_quantize_weights(w.cuda())
    for e in range(E):
        want, ws = ref.quantize(w[e].float().numpy(), 128)
        assert (_np(codes[e]) == want).all() and (_np(scales[e]) == ws).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E,N,K", [(5, 300, 272), (9, 128, 1168), (17, 40, 128)])
def test_quantize_weights_of_many_block_rows_bits(E, N, K, dtype):
    # from eight rows of blocks on, their order over the workgroups differs
    _say("quantize weights rows", E, N, K, dtype)
    w = (torch.from_numpy(np.random.default_rng(E + N).standard_normal((E, N, K))) / 16).to(dtype)
    w *= torch.exp2(torch.arange(E, dtype=torch.float32))[:, None, None].to(dtype)
    codes, scales = mg.fp8_quantize_weights(w.cuda())
    for e in range(E):
        want, ws = ref.quantize(w[e].float().numpy(), 128)
        assert (_np(codes[e]) == want).all() and (_np(scales[e]) == ws).all()


def test_quantize_past_32_bit_offsets():
    M, K = 140001, 16400
    _say("quantize large", M, K)
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator("cuda").manual_seed(1))
    codes, scales = mg.fp8_quantize(x)
    for r in (0, 70000, 131000, M - 1):
        want, ws = ref.quantize(_np(x[r:r + 1].float()), 1)
        assert (_np(codes[r]) == want[0]).all() and (_np(scales[:, r]) == ws[0]).all()


def test_quantizers_in_a_graph_and_on_another_stream():
    _say("quantize graph")
    x = _rows_input(70, 528, torch.bfloat16, 9).cuda()
    w = torch.randn(2, 144, 272, device="cuda")
    gu = torch.randn(40, 288, device="cuda").bfloat16()
    calls = [lambda: mg.fp8_quantize(x), lambda: mg.fp8_quantize_weights(w), lambda: mg.fp8_quantize_swiglu(gu)]
    want = [c() for c in calls]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        other = [c() for c in calls]
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = [c() for c in calls]
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(want, other, kept):
            for u, v, z in zip(a, b, c):
                assert torch.equal(u, v) and torch.equal(u, z)


def test_bindings_refuse_shapes_strides_and_devices():
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    u8 = torch.zeros(8, 32, dtype=torch.uint8, device="cuda")
    s, w8, ws = torch.zeros(1, 8, device="cuda"), torch.zeros(2, 16, 32, dtype=torch.uint8, device="cuda"), torch.zeros(2, 1, 1, device="cuda")
    with pytest.raises(ValueError, match="scales"):
        mg.fwd_fp8(u8, s.t().contiguous(), w8, ws, off)
    with pytest.raises(ValueError, match="contiguous"):
        mg.fwd_fp8(torch.zeros(32, 8, dtype=torch.uint8, device="cuda").t(), s, w8, ws, off)
    with pytest.raises(ValueError, match="offsets"):
        mg.fwd_fp8(u8, s, w8, ws, off[:2])
    with pytest.raises(ValueError, match="dy8"):
        mg.dgrad_fp8(u8, s, w8, ws, off)
    with pytest.raises(ValueError, match="out"):
        mg.fwd_fp8(u8, s, w8, ws, off, out=torch.zeros(8, 32, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(mg.MgemmError):
        mg.fwd_fp8(torch.zeros(8, 24, dtype=torch.uint8, device="cuda"), s, torch.zeros(2, 16, 24, dtype=torch.uint8, device="cuda"), ws, off)
    with pytest.raises(mg.MgemmError):
        mg.fp8_quantize(torch.zeros(8, 24, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        mg.fp8_quantize(torch.zeros(8, 64, device="cuda")[:, :32])
    with pytest.raises(mg.MgemmError):                       # 4 bytes past alignment
        mg.fp8_quantize(torch.zeros(8 * 32 + 1, device="cuda")[1:].view(8, 32))
    with pytest.raises(ValueError, match="GPU"):
        mg.fp8_quantize(torch.zeros(8, 32, device="cuda"), gather=torch.zeros(4, dtype=torch.int32))
