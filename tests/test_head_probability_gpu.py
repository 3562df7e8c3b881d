"""The probabilities in the output head's gradients are 1 at most, whichever
kernel forms them, however large the logits are and at every temperature.

One entry of the vocabulary (entry 0) has all of a token's probability, the
teacher's or target's entry (entry 1) none: dz is a p at entry 0 and -a at entry
1.  Column 1 of w is 1 at entry 0 and 0 elsewhere, and column 1 of x is 0, so that
dx[:, 1] = a p: p can be read off."""
import pytest
import torch

import moe_grouped_gemm_bf16_amd as mg

pytestmark = pytest.mark.gpu
DEV = "cuda"
U, H = 2.0 ** -24, 2.0 ** -8

# tiles of 64 x 64; of 256 x 128 and 256 x 256; two 16-bit values per dz; the
# same in tiles of 64 x 64; pieces of the vocabulary
SHAPES = [(200, 1500, 64), (1500, 9000, 136), (64, 70001, 520), (64, 3000, 64), (65600, 4500, 16)]


def _case(T, V, D, sign, largest, seed):
    """c z of entry 0 is spread from 1e3 to `largest`, the others' are at least
    half of it lower (sign > 0) or as much again (sign < 0)."""
    print("[case]", T, V, D, sign, largest, flush=True)
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = torch.zeros(V, D, device=DEV)
    w[:, 2:] = 0.01 * torch.randn(V, D - 2, device=DEV, generator=g)
    w[:, 0] = 64.0 if sign > 0 else 128.0
    w[0] = 0.0
    w[0, 0], w[0, 1] = (128.0, 1.0) if sign > 0 else (64.0, 1.0)
    x = torch.randn(T, D, device=DEV, generator=g)
    size = torch.exp(torch.rand(T, device=DEV, generator=g) * torch.log(torch.tensor(largest / 1e3))) * 1e3
    x[:, 0] = sign * size / w[0, 0]
    x[:, 1] = 0.0
    return x.bfloat16(), w.bfloat16()


def _check(p, lse):
    """p: dx[:, 1] over its weight a.  One rounding of dz relative to a (two 16-bit
    values have less) and one of dx, and 16 u for a's own roundings and the
    exponentials; from below also lse's two roundings, 2 u |lse|, and 4 u |lse|
    for the reference's and the scale's: below exp(-6 u |lse|) of 1."""
    assert p.isfinite().all()
    high = (1 + H) * (1 + H) * (1 + 16 * U)
    low = torch.exp(-6 * U * lse.double().abs()) * (1 - H) * (1 - H) * (1 - 16 * U)
    assert float(p.max()) <= high, float(p.max())
    assert (p >= low).all(), float((p / low).min())


@pytest.mark.parametrize("T,V,D", SHAPES)
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("tau", [0.7, 3.0, 1.0])
def test_distillation(T, V, D, sign, tau):
    for i, largest in enumerate((1e7, 1e9)):
        x, w = _case(T, V, D, sign, largest * tau, i)
        teacher = torch.zeros(T, 1, device=DEV)
        index = torch.ones(T, 1, device=DEV, dtype=torch.int32)
        r = mg.head_distill(x, w, teacher, index, temperature=tau)
        dx, _ = mg.head_distill_bwd(x, w, teacher, index, r.lse, r.logits, torch.ones(T, device=DEV), temperature=tau)
        _check(dx[:, 1].double() * float(torch.tensor(tau, dtype=torch.float32)), r.lse)


@pytest.mark.parametrize("T,V,D", SHAPES)
@pytest.mark.parametrize("sign", [1, -1])
def test_cross_entropy_with_a_log_sum_exp_joined_elsewhere(T, V, D, sign):
    # parts of a vocabulary are joined by the caller, to fp32's rounding
    x, w = _case(T, V, D, sign, 1e7, 7)
    t = torch.ones(T, device=DEV, dtype=torch.int32)
    r = mg.head_loss(x, w, t)
    lse = torch.nextafter(r.lse, torch.full_like(r.lse, -torch.inf))
    dx, _ = mg.head_loss_bwd(x, w, t, lse, torch.ones(T, device=DEV))
    _check(dx[:, 1].double(), r.lse)
