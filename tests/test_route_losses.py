"""The router's balance and z losses one by one, on logits that prefer some
experts (so that the balance loss is well above 1), with masks, infinities and
logits that no vector load may read whole."""
import numpy as np
import pytest
import torch

import block_fp8_ref as ref
import moe_grouped_gemm_bf16_amd as mg
from route_losses import losses_off

P_TOL = 2.0 ** -17


def _logits(T, E, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) * 2 + 1.5 * torch.randn(E, generator=g)).to(dtype)


def test_a_constant_balance_is_told_apart():
    """Mistakes planted in the reference's losses: a balance of 1, losses off by
    2^-14 and a NaN are outside the bounds."""
    for T, E, k in SHAPES[:6]:
        want = ref.route(_logits(T, E, torch.float32, T).double().numpy(), k, True)["loss"]
        assert losses_off(want, want) == []
        assert losses_off([1.0, want[1]], want) == ["balance"]
        assert losses_off(want * (1 + 2.0 ** -14), want) == ["balance", "z"]
        assert losses_off([np.nan, want[1]], want) == ["balance"]


SHAPES = [(16, 128, 8), (255, 64, 6), (256, 130, 8), (257, 256, 8), (1000, 100, 10), (300, 1024, 64), (20011, 72, 6), (40000, 80, 40), (600000, 8, 4)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_losses(T, E, k, dtype):
    print("[case] losses", T, E, k, dtype, flush=True)
    l = _logits(T, E, dtype, T)
    m = torch.rand(T, generator=torch.Generator().manual_seed(1)) < 0.9
    for mask in (None, m):
        r = mg.moe_route(l.cuda(), k, mask=None if mask is None else mask.cuda())
        want = ref.route(l.double().numpy(), k, True, None if mask is None else mask.numpy())
        assert want["loss"][0] > 1.05
        got = r.loss.cpu().numpy()
        assert losses_off(got, want["loss"]) == [], (got, want["loss"])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [7, 700])
def test_lse_and_losses_beside_masks_infinities_and_nan(T):
    """lse of every token, and the losses while lse^2 is in range."""
    E, k = 24, 5
    for dtype in (torch.float32, torch.bfloat16):
        print("[case] losses masks", T, dtype, flush=True)
        l = _logits(T, E, dtype, 40)
        l[:, 3] = -np.inf
        l[:, 7] = float("nan")
        l[0] = -np.inf
        l[1, 2:] = torch.finfo(dtype).min
        l[3, :20] = -np.inf
        mask = torch.ones(T, dtype=torch.bool)
        mask[T - T // 5:] = False
        l[T - 1] = float("nan")
        for extra in (False, True):
            if extra:                                        # two tokens whose lse is a largest number
                l[2] = torch.finfo(dtype).min
                l[4, 5], l[4, 6] = np.inf, np.inf
            r = mg.moe_route(l.cuda(), k, mask=mask.cuda())
            want = ref.route(l.double().numpy(), k, True, mask.numpy())
            lse = r.lse.cpu().double().numpy()
            assert (np.abs(lse - want["lse"]) <= P_TOL * np.abs(want["lse"]) + 2.0 ** -20).all()
            got = r.loss.cpu().double().numpy()
            if extra:
                assert np.isposinf(got[1])                   # lse^2 is no fp32 number
                got[1] = want["loss"][1]
            assert losses_off(got, want["loss"]) == [], (got, want["loss"])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(5, 16, 2), (300, 64, 6), (90, 256, 8), (300, 512, 9), (700, 136, 20)])
@pytest.mark.parametrize("by", [1, 2, 4])
def test_logits_off_the_vector_loads_alignment(T, E, k, dtype, by):
    """Logits (and the gradient's output) that start `by` values into an aligned
    buffer, with an expert count that vector loads divide: the same bits as from
    an aligned one."""
    print("[case] misaligned", T, E, k, dtype, by, flush=True)
    l = _logits(T, E, dtype, 3).cuda()
    buf = torch.full((T * E + 2 * by,), 9.0, dtype=dtype, device="cuda")
    off = buf[by:by + T * E].view(T, E)
    off.copy_(l)
    a, b = mg.moe_route(l, k), mg.moe_route(off, k)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    want = ref.route(l.cpu().double().numpy(), k, True)
    assert (b.experts.cpu().numpy() == want["experts"]).all() and (b.gather.cpu().numpy() == want["gather"]).all()
    dw, dl = torch.randn(T, k, device="cuda"), torch.tensor([0.3, 0.1], device="cuda")
    g = mg.moe_route_bwd(l, a.weights, a.experts, a.lse, a.counts, a.tokens, dw, dl)
    res = torch.full((T * E + 2 * by,), 9.0, dtype=dtype, device="cuda")
    h = mg.moe_route_bwd(off, a.weights, a.experts, a.lse, a.counts, a.tokens, dw, dl, out=res[by:by + T * E].view(T, E))
    assert torch.equal(g, h)
    assert (res[:by] == 9.0).all() and (res[by + T * E:] == 9.0).all()
