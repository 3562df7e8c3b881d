"""Block-scaled fp8 products whose two scales multiply to what fp32 does not
hold: any pair of scales gives the defined sum, in every form of the kernels.

One reduction block has weight scales of 2^30 and one of 1.45 2^-46.  Row 0 has
the scale 2^100 in the first and only zero codes there (its sum is that of the
other blocks), row 1 the same scale and one smallest code (its outputs reach
2^115), row 2 the scale 2^-100 in the second, the largest codes there and
nothing elsewhere (the factor 1.45 2^-146 as one fp32 number would be 3.4% off).

Tolerance: half a bf16 step, 2^-8 of the value or 2^-134 below the normal
numbers; 2^-10.8 of the sum of the magnitudes for a block's sum in the matrix
core (2^-11) and the fmas over at most 64 blocks.
"""
import numpy as np
import pytest
import torch

import block_fp8_ref as ref
import moe_grouped_gemm_bf16_amd as mg

pytestmark = pytest.mark.gpu

# rows per expert, output width, reduction
FORMS = [
    ([3], 16, 256), ([5, 0, 4], 272, 656), ([3] + [1] * 30, 96, 1168),                # few rows, 32 and 64 columns
    ([150, 0, 133, 6], 8208, 656), ([4, 257, 40], 8400, 400), ([3000, 0, 1100], 8208, 272),     # tiles of 128 and of 256
]


def _operands(sizes, P, R, dgrad, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    d = dict(device="cuda", generator=g)
    E, M, nr, np_ = len(sizes), sum(sizes), -(-R // 128), -(-P // 128)
    code = lambda *n: torch.randint(0, 120, n, dtype=torch.uint8, **d) | (torch.randint(0, 2, n, dtype=torch.uint8, **d) << 7)   # noqa: E731
    q, w = code(M, R), code(E, P, R)
    s, ws = torch.rand(nr, M, **d) + 0.5, torch.rand(E, np_, nr, **d) + 0.5
    ws[:, :, 0] *= 2.0 ** 30
    s[0] *= 2.0 ** -30
    ws[:, :, 1] = 1.45 * 2.0 ** -46
    w[:, :, 128:256] = torch.randint(119, 127, (E, P, min(R, 256) - 128), dtype=torch.uint8, **d)
    w[:, :, 7] &= 0x87                                       # at most 7 2^-9
    s[0, 0], q[0, :128] = 2.0 ** 100, 0
    s[0, 1], q[1, :128] = 2.0 ** 100, 0
    q[1, 7] = 1                                              # 2^-9
    q[2] = 0
    s[1, 2], q[2, 128:256] = 2.0 ** -100, 126                # 448
    off = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32), device="cuda")
    if dgrad:
        w, ws = w.transpose(1, 2).contiguous(), ws.transpose(1, 2).contiguous()
    return q, s, w, ws, off


def _exact(q, s, w8, ws, off, dgrad):
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
@pytest.mark.parametrize("i", range(len(FORMS)))
def test_scales_whose_product_leaves_fp32(i, dgrad):
    sizes, P, R = FORMS[i]
    print("[case] scale range", sizes, P, R, dgrad, flush=True)
    ops = _operands(sizes, P, R, dgrad, 500 + i)
    exact, mag = _exact(*ops, dgrad)
    assert exact[1].abs().max() > 2.0 ** 108 and 2.0 ** -126 < exact[2].abs().max() < 2.0 ** -120
    got = (mg.dgrad_fp8 if dgrad else mg.fwd_fp8)(*ops).double()
    assert torch.isfinite(got).all(), torch.nonzero(~torch.isfinite(got).all(1)).view(-1)[:8].tolist()
    bad = (got - exact).abs() > 2.0 ** -8 * exact.abs() + 2.0 ** -10.8 * mag + 2.0 ** -134
    assert not bad.any(), torch.nonzero(bad.any(1)).view(-1)[:8].tolist()


@pytest.mark.parametrize("dgrad", [False, True])
@pytest.mark.parametrize("sizes", [[5, 0, 4], [150, 0, 133, 6], [3000, 0, 1100]])
def test_other_rows_do_not_depend_on_a_row_with_such_scales(sizes, dgrad):
    """The bits of a row are the same whether or not rows beside it have scales
    out of range."""
    print("[case] neighbours", sizes, dgrad, flush=True)
    f = mg.dgrad_fp8 if dgrad else mg.fwd_fp8
    q, s, w8, ws, off = _operands(sizes, 8208, 656, dgrad, 9)
    got = f(q, s, w8, ws, off)
    s = s.clone()
    s[0, :2], s[1, 2] = 2.0 ** -30, 1.0
    assert torch.equal(got[3:], f(q, s, w8, ws, off)[3:])


@pytest.mark.parametrize("dgrad", [False, True])
@pytest.mark.parametrize("sizes", [[5, 0, 4], [150, 0, 133, 6], [3000, 0, 1100]])
def test_rows_of_zeros_with_scales_out_of_range(sizes, dgrad):
    """Zero codes (of either sign) give zero with any finite scale, and a scale
    that is no number makes its row none, whatever the codes."""
    print("[case] zero rows", sizes, dgrad, flush=True)
    q, s, w8, ws, off = _operands(sizes, 8208, 656, dgrad, 10)
    q[:5] = 0
    q[1, ::3] = 0x80
    s[:, 0], s[:, 1] = 3e38, 2.0 ** -100 / 448
    s[0, 2], s[0, 3], s[0, 4] = 3e38, np.inf, np.nan
    got = (mg.dgrad_fp8 if dgrad else mg.fwd_fp8)(q, s, w8, ws, off)
    assert (got[:3] == 0).all() and torch.isnan(got[3:5]).all()
    exact, mag = _exact(q, s, w8, ws, off, dgrad)
    assert ((got[5:].double() - exact[5:]).abs() <= 2.0 ** -8 * exact[5:].abs() + 2.0 ** -10.8 * mag[5:] + 2.0 ** -134).all()
