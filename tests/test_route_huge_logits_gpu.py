"""The router's z-loss gradient where lse is near the largest fp32 value (a
logit of +inf counts as that, a padded row may hold the lowest value in every
place) and the coefficient 2 dloss / n is above 1: the term 2 dloss lse / n
leaves fp32 although p times it does not.

Tolerance: fp32 products and sums of a probability (2^-17 relative, see the
router's tests): 2^-15 of the sum of the magnitudes; half a bf16 step, 2^-8,
for bf16 logits."""
import numpy as np
import pytest
import torch

import block_fp8_ref as ref
import moe_grouped_gemm_bf16_amd as mg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E", [6, 64, 300])
@pytest.mark.parametrize("normalize", [False, True])
def test_z_gradient_of_huge_logits(E, dtype, normalize):
    print("[case] huge logits", E, dtype, normalize, flush=True)
    l = (torch.randn(3, E, generator=torch.Generator().manual_seed(E)) * 2).to(dtype)
    l[0, 2] = float("inf")                                   # p = 1 there, 0 elsewhere
    l[1] = torch.finfo(dtype).min                            # uniform
    dl = torch.tensor([0.5, 4.0])                            # 2 dloss / n = 8 / 3
    dw = torch.randn(3, 2, generator=torch.Generator().manual_seed(1))
    r = mg.moe_route(l.cuda(), 2, normalize=normalize)
    got = mg.moe_route_bwd(l.cuda(), r.weights, r.experts, r.lse, r.counts, r.tokens, dw.cuda(), dl.cuda(), normalize=normalize)
    got = got.double().cpu().numpy()
    want = ref.route(l.double().numpy(), 2, normalize)
    exact, mag = ref.route_bwd(want, dw.double().numpy(), dl.double().numpy(), normalize)
    held = np.abs(exact) < 3e38                              # the result itself is an fp32 (and bf16) number
    assert held.sum() == 3 * E - 1                           # all but the chosen one's of row 0, which is infinite
    assert np.isposinf(got[0, 2])
    step = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    assert np.isfinite(got[held]).all(), np.argwhere(held & ~np.isfinite(got))[:6].tolist()
    assert (np.abs(got - exact)[held] <= (2.0 ** -15 * mag + step * np.abs(exact) + 1e-37)[held]).all()
