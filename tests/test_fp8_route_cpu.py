"""Block-scaled fp8 and router calls on the host: the references the GPU tests
use, pinned by brute force, and every refusal that needs no device."""
import numpy as np
import pytest
import torch

import block_fp8_ref as ref
import moe_grouped_gemm_bf16_amd as mg
from moe_grouped_gemm_bf16_amd import _lib

L = _lib.LIB
OK, NUL, SHAPE, ALIGN, DEV, LAUNCH, OFFS = range(7)
A = 0x10000          # a 16-byte-aligned fake address, never dereferenced


# -- the references ------------------------------------------------------------

def test_encode_is_nearest_even_by_brute_force():
    table = ref.e4m3_values()
    rng = np.random.default_rng(1)
    mids = (table[:126] + table[1:127]) / 2
    vals = np.concatenate([table[:127], -table[:127], mids, -mids, rng.standard_normal(500) * 100,
                           rng.standard_normal(500) * 0.01])
    vals = vals[np.abs(vals) <= 448]
    got = ref.encode(vals)
    for v, c in zip(vals, got):
        d = np.abs(table[:127] - abs(v))
        near = np.nonzero(d == d.min())[0]
        want = near[0] if len(near) == 1 else [i for i in near if i % 2 == 0][0]
        assert (c & 127) == want and (c >> 7) == np.signbit(v), v


def test_torch_conversion_agrees_with_the_reference_encoding():
    x = np.random.default_rng(2).standard_normal(4000).astype(np.float32) * 60
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert (ref.encode(x.astype(np.float64)) == want).all()


def test_quantize_reference_covers_the_range_and_zero_blocks():
    x = np.random.default_rng(3).standard_normal((5, 144)).astype(np.float32)
    x[2, :128] = 0
    codes, scales = ref.quantize(x, 1)
    assert (codes[2, :128] == 0).all() and scales[2, 0] == np.float32(2.0 ** -100) / np.float32(448)
    back = ref.dequant_rows(codes, np.ascontiguousarray(scales.T))
    step = np.repeat(scales.astype(np.float64), 128, 1)[:, :144] * 2.0 ** -10     # half a subnormal step
    assert (np.abs(back - x) <= 2.0 ** -4 * np.abs(x) * (1 + 1e-6) + step).all()
    for r in (0, 1, 3, 4):
        assert (codes[r, :128] & 127).max() == 126                 # the maximum sits at 448


@pytest.mark.parametrize("normalize", [False, True])
def test_route_gradient_reference_against_differences(normalize):
    rng = np.random.default_rng(4)
    T, E, k = 5, 7, 3
    l = rng.standard_normal((T, E))
    l[1, 2] = -np.inf
    l[4] = -np.inf
    dw, dl = rng.standard_normal((T, k)), np.array([0.7, 0.3])
    r = ref.route(l, k, normalize)
    got, _ = ref.route_bwd(r, dw, dl, normalize)
    h = 1e-5
    for t in range(T):
        for e in range(E):
            if not np.isfinite(l[t, e]):
                assert got[t, e] == 0
                continue
            a, b = l.copy(), l.copy()
            a[t, e] += h
            b[t, e] -= h
            d = (ref.route_loss(a, r, dw, dl, normalize) - ref.route_loss(b, r, dw, dl, normalize)) / (2 * h)
            # central difference: h^2 times a third derivative of order 1, and 1e-16 / h
            assert abs(d - got[t, e]) < 1e-8


def test_route_reference_by_hand():
    r = ref.route(np.array([[1.0, 3.0, 3.0], [0.0, -np.inf, -np.inf], [2.0, 1.0, 0.0]]), 2, True, mask=[1, 1, 0])
    assert r["experts"].tolist() == [[1, 2], [0, -1], [-1, -1]]
    assert r["weights"].tolist() == [[0.5, 0.5], [1.0, 0.0], [0.0, 0.0]]
    assert r["counts"].tolist() == [1, 1, 1] and r["tokens"].tolist() == [2]
    assert r["offsets"].tolist() == [0, 1, 2, 3]
    assert r["gather"].tolist() == [1, 0, 0, -1, -1, -1]
    assert r["token_rows"].tolist() == [[1, 2], [0, -1], [-1, -1]]


# -- refusals of the C entry points ---------------------------------------------

@pytest.mark.parametrize("fn", ["mgemm_fwd_fp8", "mgemm_dgrad_fp8"])
def test_product_argument_errors(fn):
    f = getattr(L, fn)
    # (q8, q_scale, w8, w_scale, offsets, out, M, N, K, E, max_m_per_e, stream)
    assert f(A, A, A, A, A, A, 512, 128, 256, 0, 0, None) == SHAPE         # E < 1
    assert f(A, A, A, A, A, A, 512, 128, 256, 1025, 0, None) == SHAPE
    assert f(A, A, A, A, A, A, 512, 136, 256, 4, 0, None) == SHAPE         # N % 16
    assert f(A, A, A, A, A, A, 512, 128, 264, 4, 0, None) == SHAPE         # K % 16
    assert f(A, A, A, A, A, A, -1, 128, 256, 4, 0, None) == SHAPE
    assert f(A, A, A, A, A, A, 512, 128, 1 << 23, 4, 0, None) == SHAPE
    assert f(A, A, A, A, A, A, 512, 128, 256, 4, -1, None) == SHAPE        # bad hint
    assert f(A, A, A, A, A, A, 1 << 30, 1 << 22, 1 << 22, 4, 0, None) == SHAPE   # tile count
    for i in range(6):
        args = [A] * 6
        args[i] = None
        assert f(*args, 512, 128, 256, 4, 0, None) == NUL
    for i, by in ((0, 8), (1, 2), (2, 4), (3, 1), (4, 2), (5, 8)):
        args = [A] * 6
        args[i] = A + by
        assert f(*args, 512, 128, 256, 4, 0, None) == ALIGN
    assert f(None, None, None, None, None, None, 0, 128, 256, 4, 0, None) == OK


def test_quantizer_argument_errors():
    f = L.mg_fp8_quantize
    # (x, x_fp32, gather, offsets, codes, scales, M, T, K, E, stream)
    assert f(A, 0, None, None, A, A, 8, 8, 24, 0, None) == SHAPE            # K % 16
    assert f(A, 0, None, None, A, A, -1, 8, 32, 0, None) == SHAPE
    assert f(A, 0, A, None, A, A, 8, -1, 32, 0, None) == SHAPE
    assert f(A, 0, None, A, A, A, 8, 8, 32, 0, None) == SHAPE               # offsets, E < 1
    assert f(None, 0, None, None, A, A, 8, 8, 32, 0, None) == NUL
    assert f(A, 0, None, None, None, A, 8, 8, 32, 0, None) == NUL
    assert f(A, 0, None, None, A, None, 8, 8, 32, 0, None) == NUL
    assert f(A + 8, 0, None, None, A, A, 8, 8, 32, 0, None) == ALIGN
    assert f(A, 0, None, None, A + 8, A, 8, 8, 32, 0, None) == ALIGN
    assert f(A, 0, None, None, A, A + 2, 8, 8, 32, 0, None) == ALIGN
    assert f(A, 0, A + 2, None, A, A, 8, 8, 32, 0, None) == ALIGN
    assert f(None, 0, None, None, None, None, 0, 8, 32, 0, None) == OK
    assert f(None, 0, None, None, None, None, 8, 8, 0, 0, None) == OK
    g = L.mg_fp8_quantize_swiglu
    # (gu, offsets, codes, scales, M, I, E, stream)
    assert g(A, None, A, A, 8, 24, 0, None) == SHAPE
    assert g(None, None, A, A, 8, 32, 0, None) == NUL
    assert g(A, None, A + 4, A, 8, 32, 0, None) == ALIGN
    assert g(None, None, None, None, 0, 32, 0, None) == OK
    h = L.mg_fp8_quantize_weights
    # (w, w_fp32, codes, scales, E, N, K, stream)
    assert h(A, 0, A, A, 2, 8, 24, None) == SHAPE
    assert h(A, 0, A, A, -1, 8, 32, None) == SHAPE
    assert h(A, 0, A, A, 1 << 20, 1 << 20, 1 << 20, None) == SHAPE          # block count
    assert h(None, 0, A, A, 2, 8, 32, None) == NUL
    assert h(A + 8, 0, A, A, 2, 8, 32, None) == ALIGN
    assert h(None, 0, None, None, 2, 0, 32, None) == OK


def test_sizes_past_the_grid():
    h = L.mg_fp8_quantize_weights
    assert h(A, 0, A, A, 1 << 24, 1, 16, None) == SHAPE
    assert h(A, 0, A, A, 1 << 12, 1 << 12, 1 << 14, None) == SHAPE
    assert h(None, 0, A, A, (1 << 24) - 1, 1, 16, None) == NUL            # the sizes alone are fine
    # (x8, x_scale, w8, w_scale, offsets, y, M, N, K, E, max_m_per_e, stream)
    for f in (L.mgemm_fwd_fp8, L.mgemm_dgrad_fp8):
        assert f(A, A, A, A, A, A, 2 ** 31 - 256, 16, 16, 2, 0, None) == SHAPE      # the last tile's end
        assert f(A, A, A, A, None, A, 2 ** 31 - 257, 16, 16, 2, 0, None) == NUL     # the sizes alone are fine
    # T k past 64 bits
    assert L.mg_moe_route(*_route_args(T=1 << 58, E=64, k=64, local=64)) == SHAPE
    assert L.mg_moe_route_workspace(2 ** 63 - 1, 64) == 0


def _route_args(**kw):
    a = dict(logits=A, bf16=0, mask=None, T=8, E=16, k=2, normalize=1, first=0, local=16, weights=A, experts=A, lse=A, counts=A, prob_sum=A,
             tokens=A, loss=A, offsets=A, gather=A, token_rows=A, workspace=A, bytes=1 << 20, stream=None)
    a.update(kw)
    return tuple(a.values())


def test_route_argument_errors():
    f = L.mg_moe_route
    assert f(*_route_args(E=0)) == SHAPE and f(*_route_args(E=1025)) == SHAPE
    assert f(*_route_args(k=0)) == SHAPE and f(*_route_args(k=17)) == SHAPE
    assert f(*_route_args(E=128, local=128, k=65)) == SHAPE
    assert f(*_route_args(T=-1)) == SHAPE and f(*_route_args(T=1 << 30)) == SHAPE      # T k
    assert f(*_route_args(first=-1)) == SHAPE and f(*_route_args(first=1)) == SHAPE
    assert f(*_route_args(local=0)) == SHAPE and f(*_route_args(local=17)) == SHAPE
    assert f(*_route_args(first=2 ** 31 - 1)) == SHAPE
    assert f(*_route_args(T=100000, bytes=16)) == SHAPE                                # workspace
    for name in ("logits", "weights", "experts", "lse", "counts", "prob_sum", "tokens", "loss", "offsets", "gather", "token_rows"):
        assert f(*_route_args(**{name: None})) == NUL, name
        assert f(*_route_args(**{name: A + 1})) == ALIGN, name
    assert f(*_route_args(T=100000, workspace=None)) == NUL
    assert f(*_route_args(T=100000, workspace=A + 2)) == ALIGN
    assert f(*_route_args(bf16=1, logits=A + 1)) == ALIGN
    assert L.mg_moe_route_workspace(1, 64) == 0
    assert L.mg_moe_route_workspace(-1, 64) == 0 and L.mg_moe_route_workspace(8, 0) == 0
    assert 0 < L.mg_moe_route_workspace(1 << 20, 64) == L.mg_moe_route_workspace(1 << 24, 64)


def test_route_bwd_argument_errors():
    f = L.mg_moe_route_bwd
    base = dict(logits=A, bf16=0, weights=A, experts=A, lse=A, counts=A, tokens=A, dweights=A, dloss=A, dlogits=A, T=8, E=16, k=2, normalize=1,
                stream=None)

    def call(**kw):
        return f(*{**base, **kw}.values())
    assert call(E=0) == SHAPE and call(k=17) == SHAPE and call(T=-1) == SHAPE
    for name in ("logits", "weights", "experts", "lse", "counts", "tokens", "dlogits"):
        assert call(**{name: None}) == NUL, name
    for name in ("logits", "weights", "experts", "lse", "counts", "tokens", "dweights", "dloss", "dlogits"):
        assert call(**{name: A + 1}) == ALIGN, name
    assert call(T=0, logits=None) == OK


def test_combine_bwd_argument_errors():
    f = L.mg_moe_combine_bwd
    # (dout, rows, token_rows, weights, drows, dweights, M, T, k, D, stream)
    assert f(A, A, A, A, A, A, 100, 10, 0, 64, None) == SHAPE
    assert f(A, A, A, A, A, A, 100, 10, 65, 64, None) == SHAPE
    assert f(A, A, A, A, A, A, 100, 10, 4, 60, None) == SHAPE
    assert f(A, A, A, A, A, A, -1, 10, 4, 64, None) == SHAPE
    assert f(None, A, A, A, A, A, 100, 10, 4, 64, None) == NUL
    assert f(A, None, A, A, A, A, 100, 10, 4, 64, None) == NUL
    assert f(A, A, None, A, A, A, 100, 10, 4, 64, None) == NUL
    assert f(A, A, A, A, None, A, 100, 10, 4, 64, None) == NUL
    assert f(A + 8, A, A, A, A, A, 100, 10, 4, 64, None) == ALIGN
    assert f(A, A, A, A, A + 8, A, 100, 10, 4, 64, None) == ALIGN
    assert f(A, A, A, A, A, A + 2, 100, 10, 4, 64, None) == ALIGN
    assert f(None, None, None, None, None, None, 100, 0, 4, 64, None) == OK


def test_rows_named_twice_are_found():
    def check(v, M):
        v = np.ascontiguousarray(v, np.int32)
        return L.mg_check_rows_host(v.ctypes.data, v.size, M)
    assert check([0, 2, -1, -1, 1, 7, 7], 7) == OK              # 7 and -1: no row
    assert check([0, 2, -1, 2], 7) == OFFS
    assert L.mg_check_rows_host(None, 3, 7) == NUL
    assert check([0], -1) == SHAPE


# -- refusals of the binding ------------------------------------------------------

def test_binding_refuses_on_the_host():
    u8, f32 = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(1, 8)
    w8, ws, off = torch.zeros(2, 16, 32, dtype=torch.uint8), torch.zeros(2, 1, 1), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        mg.fwd_fp8(u8, f32, w8, ws, off)
    with pytest.raises(TypeError, match="uint8"):
        mg.dgrad_fp8(u8.float(), f32, w8, ws, off)
    with pytest.raises(TypeError, match="bfloat16 or torch.float32"):
        mg.fp8_quantize(torch.zeros(8, 32, dtype=torch.float16))
    with pytest.raises(TypeError):
        mg.fp8_quantize_swiglu(torch.zeros(8, 32))
    with pytest.raises(TypeError):
        mg.fp8_quantize_weights(torch.zeros(2, 8, 32, dtype=torch.float64))
    with pytest.raises(TypeError, match="logits"):
        mg.moe_route(torch.zeros(4, 8, dtype=torch.float16), 2)
    with pytest.raises(ValueError, match="GPU"):
        mg.moe_route(torch.zeros(4, 8), 2)
    with pytest.raises(TypeError):
        mg.moe_combine_bwd(torch.zeros(4, 8), torch.zeros(8, 8, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32))
