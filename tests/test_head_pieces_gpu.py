"""The output head where the vocabulary goes in several pieces or is as long as it
may be, and with hidden rows longer than other tests have, against
tests/head_ref.py (64 bits; its bounds are the tolerances)."""
import math

import pytest
import torch

import moe_grouped_gemm_bf16_amd as mg
import test_head_gpu as head

pytestmark = pytest.mark.gpu
DEV = "cuda"

# 16640 tokens: pieces of 16128 entries, the last one of 7744; whole and cut tiles
# along the tokens, the columns and the vocabulary.  40 tokens: a piece of 2^20
# entries and one of 300, tiles of fewer rows, dz as one value.  16500 tokens: two
# pieces, the second of one entry.
PIECES = [(16640, 40000, 520), (40, (1 << 20) + 300, 520), (16500, 16128 + 1, 264)]


@pytest.mark.parametrize("T,V,D", PIECES)
def test_loss_in_pieces(T, V, D):
    head._loss_case(T, V, D, ignored=0.2, z_loss=True, seed=T, uniform=False)


@pytest.mark.parametrize("T,V,D", PIECES)
def test_distillation_in_pieces(T, V, D):
    print("[case]", T, V, D, flush=True)
    k = 5
    g, x, w = head._inputs(T, V, D, 3)
    # distinct entries over the whole vocabulary, so over all pieces
    index = torch.randint(0, V // k, (T, k), device=DEV, generator=g, dtype=torch.int32)
    index += torch.arange(k, device=DEV, dtype=torch.int32) * (V // k)
    index[::7, 4] = V - 1                                  # of the last piece, with the piece before
    index[1::7, 3], index[2::7, :2], index[3::7] = index[1::7, 0], -1, -1
    teacher = torch.randn(T, k, device=DEV, generator=g)
    head._distill_check(x, w, teacher, index, 1.5, torch.randn(T, device=DEV, generator=g))


@pytest.mark.parametrize("T,V,D", [(1, 5000, 16392), (200, 3000, 16392), (600, 9000, 10248)])
def test_long_hidden_rows(T, V, D):
    head._loss_case(T, V, D, ignored=0.1, z_loss=True, seed=D, uniform=False)


def test_the_longest_vocabulary():
    """V = 2^31 - 256: all entries 0 but three, the last one among them."""
    V, D, T = (1 << 31) - 256, 8, 3
    at, z = [0, (1 << 30) + 77, V - 1], [16.0, 24.0, 20.0]
    w = torch.zeros(V, D, dtype=torch.bfloat16, device=DEV)
    for j, (v, value) in enumerate(zip(at, z)):
        w[v, j] = value
    x = torch.zeros(T, D, dtype=torch.bfloat16, device=DEV)
    for t in range(T):
        x[t, t] = 1.0                                      # token t sees entry at[t] alone
    r = mg.head_loss(x, w, torch.tensor([at[0], 5, at[2]], dtype=torch.int32, device=DEV))
    for t in range(T):
        lse = math.log(V - 1 + math.exp(z[t]))
        logit = (z[0], 0.0, z[2])[t]
        # equal terms: a wave's tile and a thread's chain of tiles add up to 2^23
        # ones each exactly or to u of the sum, 2^14 additions in a chain at most
        tol = 2.0 ** -24 * (2 ** 14 + 100 + 4 * lse)
        assert abs(float(r.lse[t]) - lse) <= tol and float(r.logit[t]) == logit
        assert abs(float(r.loss[t]) - (lse - logit)) <= tol
