"""Offsets that break the precondition (decreasing, below 0, past M) in the fp8
products: the kernels take the running maximum of the clamped offsets, so every
row belongs to one expert at most, nothing outside the output is written and
the number of tiles stays under what the host's limit counts with.

The GPU part's tolerance: half a bf16 step, 2^-8 of the value, and 2^-10.8 of
the sum of the magnitudes (a block's sum in the matrix core 2^-11, the fmas over
the blocks)."""
import numpy as np
import pytest
import torch

import block_fp8_ref as ref
import moe_grouped_gemm_bf16_amd as mg


def effective(off, M):
    return np.maximum.accumulate(np.clip(np.asarray(off, np.int64), 0, M))


def tiles(off, bq):
    return int((-(-np.diff(off) // bq)).sum())


def _broken(M, E, seed):
    rng = np.random.default_rng(seed)
    kinds = [rng.integers(-M, 2 * M, E + 1), np.where(np.arange(E + 1) % 2, M, 0), np.where(np.arange(E + 1) % 2, 2 ** 31 - 1, -2 ** 31),
             np.arange(E, -1, -1) * (M // E), np.full(E + 1, M)]
    return [k.astype(np.int32) for k in kinds]


def test_tiles_of_the_running_maximum_stay_under_the_host_s_count():
    """The count per expert from its own two clamped offsets does not: with 0 and
    M in turn half the experts have all the rows."""
    worst = 0
    for M, E, bq in ((1000, 7, 32), (4097, 1024, 32), (65536, 1024, 128), (300, 64, 256)):
        for i in range(20):
            for off in _broken(M, E, i):
                assert tiles(effective(off, M), bq) <= -(-M // bq) + E
                c = np.clip(off.astype(np.int64), 0, M)
                alone = int((-(-(np.maximum(c[1:], c[:-1]) - c[:-1]) // bq)).sum())
                worst = max(worst, alone / (-(-M // bq) + E))
    assert worst > 100


# experts, rows, output width, reduction: few rows (two widths), tiles of 128 and of 256
FORMS = [(4, 40, 96, 272), (70, 200, 176, 400), (3, 300, 8208, 272), (70, 600, 8208, 144), (3, 4200, 8208, 272)]


@pytest.mark.gpu
@pytest.mark.parametrize("dgrad", [False, True])
@pytest.mark.parametrize("form", range(len(FORMS)))
def test_products_with_broken_offsets(form, dgrad):
    E, M, P, R = FORMS[form]
    g = torch.Generator("cuda").manual_seed(form)
    d = dict(device="cuda", generator=g)
    code = lambda *n: torch.randint(0, 120, n, dtype=torch.uint8, **d) | (torch.randint(0, 2, n, dtype=torch.uint8, **d) << 7)   # noqa: E731
    N, K = (R, P) if dgrad else (P, R)
    q, w8, s = code(M, R), code(E, N, K), torch.rand(-(-R // 128), M, **d) + 0.5
    ws = torch.rand(E, -(-N // 128), -(-K // 128), **d) + 0.5
    table = torch.from_numpy(ref.e4m3_values()).cuda()
    x = table[q.int()] * s.t().double().repeat_interleave(128, 1)[:, :R]
    for off in _broken(M, E, form) + [np.linspace(0, M, E + 1).astype(np.int32)]:
        print("[case] broken offsets", FORMS[form], dgrad, off[:6].tolist(), flush=True)
        out = torch.full((M + 3, P), 7.0, dtype=torch.bfloat16, device="cuda")
        (mg.dgrad_fp8 if dgrad else mg.fwd_fp8)(q, s, w8, ws, torch.from_numpy(off).cuda(), out=out[:M])
        eff = effective(off, M)
        want = torch.full((M + 3, P), 7.0, dtype=torch.float64, device="cuda")
        mag = torch.zeros_like(want)
        for e in range(E):
            a, b = int(eff[e]), int(eff[e + 1])
            if a == b:
                continue
            w = table[w8[e].int()] * ws[e].double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
            w = w if dgrad else w.t().contiguous()
            want[a:b], mag[a:b] = x[a:b] @ w, x[a:b].abs() @ w.abs()
        assert ((out.double() - want).abs() <= 2.0 ** -8 * want.abs() * (mag > 0) + 2.0 ** -10.8 * mag).all()
