"""Limits of the output head's calls that are decided on the host.  Every call
here is refused before anything is launched, with or without a device."""
import pytest

from moe_grouped_gemm_bf16_amd import _lib

L = _lib.LIB
SHAPE = _lib.MG_ERR_SHAPE
A = 0x10000          # an aligned address; no call below passes the checks


@pytest.mark.parametrize("T", [1, 128, 129])
@pytest.mark.parametrize("short", [1, 2, 255])
def test_the_forward_refuses_a_vocabulary_whose_last_tile_ends_past_31_bits(T, short):
    # 2^31 - 256 entries are whole tiles of 256; one entry more is a tile whose end
    # 32-bit counts cannot hold.  (The workspace is asked first: where it names a
    # size, the calls are not made.)
    V = (1 << 31) - short
    assert L.mg_head_workspace(T, V, 8) == 0
    assert L.mg_head_loss(A, A, A, T, V, 8, 0, A, A, A, A, 1 << 60, None) == SHAPE
    assert L.mg_head_distill(A, A, A, 0, A, T, V, 8, 3, 0, 1.0, A, A, A, A, 1 << 60, None) == SHAPE


def test_the_longest_vocabulary_has_a_workspace():
    V = (1 << 31) - 256
    assert L.mg_head_workspace(1, V, 8) >= V // 256 * 4 * 8
    # the gradients take it in pieces and have no such end
    assert L.mg_head_bwd_workspace(1, (1 << 31) - 1, 8, 0) > 0


def test_both_ends_of_the_temperature_are_taken():
    # (no tokens: nothing to launch)
    import numpy as np
    low, high = np.float32(1e-37), np.float32(1e37)
    for tau, status in ((low, 0), (high, 0), (np.nextafter(low, np.float32(0)), SHAPE),
                        (np.nextafter(high, np.float32(np.inf)), SHAPE)):
        tau = float(tau)
        assert L.mg_head_distill(A, A, A, 0, A, 0, 9, 16, 3, 0, tau, A, A, A, A, 0, None) == status, tau
        assert L.mg_head_distill_bwd(A, A, A, 0, A, A, A, A, 0, 9, 16, 3, 0, tau, A, None, A, 0, None) == status, tau
