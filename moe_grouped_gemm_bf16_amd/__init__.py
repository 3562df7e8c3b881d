"""MoE grouped GEMM for AMD Instinct MI355X (gfx950).

Thin Python binding over the C ABI of libmgemm.so (include/mgemm.h): argument
checks and marshalling only.  Every step of the computation runs in the HIP
kernels; PyTorch provides device memory and the current stream.

  fwd(x, w, offsets)      Y[i] = x[i] W[e]^T          M-grouped forward
  dgrad(dy, w, offsets)   dX[i] = dy[i] W[e]          M-grouped input gradient
  wgrad(dy, x, offsets)   dW[e] = sum_i dy[i]^T x[i]  K-grouped fp32 weight gradient
  fwd_swiglu(x, w13, offsets, gather)                  gate-up forward, SwiGLU fused,
      h[i] = silu(x[r] w1[e]^T) * (x[r] w3[e]^T), r = gather[i]   rows gathered by index
  grouped_list([(A_g, B_g), ...])   D_g = A_g B_g^T    independent GEMMs, per-group shapes
  moe_route(logits, k)    gate, row order, balance and z losses; moe_route_bwd, its gradient
  moe_combine(rows, token_rows, weights)               and moe_combine_bwd, its gradient
  head_loss(x, w, targets)  cross entropy of the output head, no logits kept; head_loss_bwd
  head_distill(x, w, teacher, index)  the same from a teacher's top logits; head_distill_bwd
  fwd_fp8, dgrad_fp8      block-scaled fp8 products on the codes of fp8_quantize,
      fp8_quantize_swiglu and fp8_quantize_weights

Page-shaped aliases follow the RapidGEMM README ("Kernels"):
  Mgemm(x, w, cnt, max_M_per_E, transpose_B) and Kgemm(grad, X, cnt, descriptor).
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from ._lib import LIB, GemmDesc, MgemmError, check, status_str  # noqa: F401

__all__ = ["fwd", "dgrad", "wgrad", "wgrad_noalloc", "fwd_swiglu", "dgrad_swiglu",
           "moe_combine", "grouped_list", "list_descriptors", "grouped_list_desc",
           "mx_scales_blocked", "fwd_mx", "wgrad_mx", "wgrad_mx_tm", "fp8_quantize", "fp8_quantize_swiglu",
           "fp8_quantize_weights", "fwd_fp8", "dgrad_fp8", "Route", "moe_route", "moe_route_bwd",
           "moe_combine_bwd", "HeadLoss", "head_loss", "head_loss_bwd", "HeadDistill",
           "head_distill", "head_distill_bwd", "Mgemm", "Kgemm",
           "MgemmError", "status_str", "LIB"]


# The current device and the current stream's handle, without the Python objects
# that the public calls make (2 us of a call), where this torch has these calls.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


def _run(name: str, dev: torch.device, *args) -> None:
    """LIB.name(*args, stream) with dev current, on its current stream."""
    index = dev.index
    if index == _current_device():
        status = getattr(LIB, name)(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            status = getattr(LIB, name)(*args, _raw_stream(index))
    check(status, name)


def _ptr(t: torch.Tensor | None) -> int:
    return 0 if t is None else t.data_ptr()


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, ndim: int) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _same_device(dev, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the data on {dev}")


def _offsets(offsets: torch.Tensor, E: int, dev) -> torch.Tensor:
    _need(offsets, "offsets", torch.int32, 1)
    if offsets.numel() != E + 1:
        raise ValueError(f"offsets must have E+1 = {E + 1} entries, got {offsets.numel()}")
    if offsets.device != dev:
        raise ValueError("offsets must be on the same device as the data")
    return offsets


def fwd(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, max_m_per_e: int = 0,
        out: torch.Tensor | None = None) -> torch.Tensor:
    """M-grouped forward: out[i] = x[i] @ w[e].T for offsets[e] <= i < offsets[e+1].

    x bf16 [M, K], w bf16 [E, N, K], offsets int32 [E+1] (device).  Rows past
    offsets[E] of `out` are left untouched (uninitialised when `out` is None)."""
    _need(x, "x", torch.bfloat16, 2)
    _need(w, "w", torch.bfloat16, 3)
    M, K = x.shape
    E, N, K2 = w.shape
    if K2 != K:
        raise ValueError(f"x is [M, {K}] but w is [E, N, {K2}]")
    _offsets(offsets, E, x.device)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    else:
        _need(out, "out", torch.bfloat16, 2)
        if tuple(out.shape) != (M, N):
            raise ValueError(f"out must be [{M}, {N}]")
    _same_device(x.device, w=w, out=out)
    _run("mgemm_fwd", x.device, x.data_ptr(), w.data_ptr(), offsets.data_ptr(), out.data_ptr(), M,
         N, K, E, int(max_m_per_e))
    return out


def dgrad(dy: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, max_m_per_e: int = 0,
          out: torch.Tensor | None = None) -> torch.Tensor:
    """M-grouped input gradient: out[i] = dy[i] @ w[e] for the rows of expert e.

    dy bf16 [M, N], w bf16 [E, N, K]; returns bf16 [M, K]."""
    _need(dy, "dy", torch.bfloat16, 2)
    _need(w, "w", torch.bfloat16, 3)
    M, N = dy.shape
    E, N2, K = w.shape
    if N2 != N:
        raise ValueError(f"dy is [M, {N}] but w is [E, {N2}, K]")
    _offsets(offsets, E, dy.device)
    if out is None:
        out = torch.empty((M, K), dtype=torch.bfloat16, device=dy.device)
    else:
        _need(out, "out", torch.bfloat16, 2)
        if tuple(out.shape) != (M, K):
            raise ValueError(f"out must be [{M}, {K}]")
    _same_device(dy.device, w=w, out=out)
    _run("mgemm_dgrad", dy.device, dy.data_ptr(), w.data_ptr(), offsets.data_ptr(), out.data_ptr(),
         M, N, K, E, int(max_m_per_e))
    return out


def wgrad(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor, E: int | None = None,
          out: torch.Tensor | None = None, accumulate: bool = False) -> torch.Tensor:
    """K-grouped fp32 weight gradient: out[e] (=|+=) dy[rows_e].T @ x[rows_e].

    dy bf16 [M, N], x bf16 [M, K]; returns fp32 [E, N, K].  E defaults to
    offsets.numel() - 1.  With accumulate=True the sum is added into `out`."""
    return _wgrad("kgemm_wgrad", dy, x, offsets, E, out, accumulate)


def wgrad_noalloc(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor, out: torch.Tensor,
                  E: int | None = None, accumulate: bool = False) -> torch.Tensor:
    """wgrad through kgemm_wgrad_noalloc: the library allocates nothing (its
    token-split workspace is a static device array shared by every call on
    the GPU, so calls that can overlap race).  `out` (fp32 [E, N, K]) is
    required: the binding allocates nothing either."""
    if out is None:
        raise ValueError("wgrad_noalloc needs `out`")
    return _wgrad("kgemm_wgrad_noalloc", dy, x, offsets, E, out, accumulate)


def _wgrad(fn: str, dy, x, offsets, E, out, accumulate):
    _need(dy, "dy", torch.bfloat16, 2)
    _need(x, "x", torch.bfloat16, 2)
    M, N = dy.shape
    M2, K = x.shape
    if M2 != M:
        raise ValueError(f"dy has {M} rows but x has {M2}")
    if E is None:
        E = offsets.numel() - 1
    _offsets(offsets, E, dy.device)
    if out is None:
        if accumulate:
            raise ValueError("accumulate=True needs `out`")
        out = torch.empty((E, N, K), dtype=torch.float32, device=dy.device)
    else:
        _need(out, "out", torch.float32, 3)
        if tuple(out.shape) != (E, N, K):
            raise ValueError(f"out must be [{E}, {N}, {K}]")
    _same_device(dy.device, x=x, out=out)
    _run(fn, dy.device, dy.data_ptr(), x.data_ptr(), offsets.data_ptr(), out.data_ptr(), M, N, K, E,
         1 if accumulate else 0)
    return out


def fwd_swiglu(x: torch.Tensor, w13: torch.Tensor, offsets: torch.Tensor,
               gather: torch.Tensor | None = None, max_m_per_e: int = 0,
               out: torch.Tensor | None = None, gu_out: torch.Tensor | None = None
               ) -> torch.Tensor:
    """Gate-up forward with SwiGLU fused, on rows gathered through an index.

    w13 bf16 [E, 2I, K] stacks each expert's gate (rows 0..I-1) and up
    (rows I..2I-1) weights.  With `gather` (int32 [M], device), row i of the
    expert-grouped problem is x[gather[i]] of the token-major x bf16 [T, K];
    without it x is bf16 [M, K], already grouped.  Returns h bf16 [M, I]:
    h[i, j] = silu(g) * u, g = x[r] . w13[e, j], u = x[r] . w13[e, I + j].
    With `gu_out` (bf16 [M, 2I]) the pre-activation g | u is written too, for
    dgrad_swiglu.  Rows past offsets[E] of `out` are left untouched."""
    _need(x, "x", torch.bfloat16, 2)
    _need(w13, "w13", torch.bfloat16, 3)
    T, K = x.shape
    E, N2, K2 = w13.shape
    if K2 != K:
        raise ValueError(f"x is [T, {K}] but w13 is [E, 2I, {K2}]")
    if N2 % 2:
        raise ValueError(f"w13 must stack two halves (2I rows), got {N2}")
    I = N2 // 2
    if gather is None:
        M = T
        gptr = 0
    else:
        _need(gather, "gather", torch.int32, 1)
        if gather.device != x.device:
            raise ValueError("gather must be on the same device as the data")
        M = gather.numel()
        gptr = gather.data_ptr()
    _offsets(offsets, E, x.device)
    if out is None:
        out = torch.empty((M, I), dtype=torch.bfloat16, device=x.device)
    else:
        _need(out, "out", torch.bfloat16, 2)
        if tuple(out.shape) != (M, I):
            raise ValueError(f"out must be [{M}, {I}]")
    guptr = 0
    if gu_out is not None:
        _need(gu_out, "gu_out", torch.bfloat16, 2)
        if tuple(gu_out.shape) != (M, 2 * I):
            raise ValueError(f"gu_out must be [{M}, {2 * I}]")
        guptr = gu_out.data_ptr()
    _same_device(x.device, w13=w13, out=out, gu_out=gu_out)
    _run("mgemm_fwd_swiglu_gu", x.device, x.data_ptr(), gptr, w13.data_ptr(), offsets.data_ptr(),
         out.data_ptr(), guptr, M, T, I, K, E, int(max_m_per_e))
    return out


def dgrad_swiglu(dy: torch.Tensor, w2: torch.Tensor, gu: torch.Tensor, offsets: torch.Tensor,
                 max_m_per_e: int = 0, out: torch.Tensor | None = None) -> torch.Tensor:
    """Down-projection input gradient fused with the SwiGLU backward.

    dy bf16 [M, N], w2 bf16 [E, N, I] (the down weights), gu bf16 [M, 2I] (the
    saved pre-activation g | u).  Returns dgu bf16 [M, 2I]: with
    dh = dy[i] @ w2[e], dgu[i, j] = dh u silu'(g), dgu[i, I + j] = dh silu(g)."""
    _need(dy, "dy", torch.bfloat16, 2)
    _need(w2, "w2", torch.bfloat16, 3)
    _need(gu, "gu", torch.bfloat16, 2)
    M, N = dy.shape
    E, N2, I = w2.shape
    if N2 != N:
        raise ValueError(f"dy is [M, {N}] but w2 is [E, {N2}, I]")
    if tuple(gu.shape) != (M, 2 * I):
        raise ValueError(f"gu must be [{M}, {2 * I}]")
    _offsets(offsets, E, dy.device)
    if out is None:
        out = torch.empty((M, 2 * I), dtype=torch.bfloat16, device=dy.device)
    else:
        _need(out, "out", torch.bfloat16, 2)
        if tuple(out.shape) != (M, 2 * I):
            raise ValueError(f"out must be [{M}, {2 * I}]")
    _same_device(dy.device, w2=w2, gu=gu, out=out)
    _run("mgemm_dgrad_swiglu", dy.device, dy.data_ptr(), w2.data_ptr(), gu.data_ptr(),
         offsets.data_ptr(), out.data_ptr(), M, N, I, E, int(max_m_per_e))
    return out


def _matrix(t: torch.Tensor, name: str) -> int:
    """Row stride of a bf16 matrix view whose rows are contiguous; the row
    length where no stride is needed (one row, or rows of no elements, whose
    stride torch reports as 1)."""
    if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or t.dim() != 2:
        raise TypeError(f"{name} must be a 2-D bfloat16 tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU device")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    return int(t.stride(0)) if t.shape[0] > 1 and t.shape[1] > 0 else int(t.shape[1])


def list_descriptors(groups, outs) -> torch.Tensor:
    """Device array of mg_gemm_desc for groups [(A [m, k], B [n, k]), ...] and
    outputs [D [m, n], ...] (row-strided views are fine).  The copy to the
    device is synchronous, so the host staging buffer outlives it."""
    descs = (GemmDesc * len(groups))()
    dev = None
    for g, ((a, b), d) in enumerate(zip(groups, outs)):
        lda, ldb, ldd = _matrix(a, f"A[{g}]"), _matrix(b, f"B[{g}]"), _matrix(d, f"D[{g}]")
        m, k = a.shape
        n, k2 = b.shape
        if k2 != k or tuple(d.shape) != (m, n):
            raise ValueError(f"group {g}: A {tuple(a.shape)}, B {tuple(b.shape)}, D {tuple(d.shape)}")
        dev = a.device if dev is None else dev
        if a.device != dev or b.device != dev or d.device != dev:
            raise ValueError("all groups must live on one device")
        descs[g] = GemmDesc(a.data_ptr(), b.data_ptr(), d.data_ptr(), m, n, k, lda, ldb, ldd)
    st = LIB.mg_check_list_host(descs, len(groups))
    check(st, "mg_check_list_host")
    raw = torch.frombuffer(bytearray(bytes(descs)), dtype=torch.uint8)
    return raw.to(dev)


def grouped_list_desc(desc: torch.Tensor, G: int) -> None:
    """mgemm_list on a device descriptor array (from list_descriptors)."""
    if desc.dtype != torch.uint8 or not desc.is_cuda or desc.numel() != 48 * G:
        raise ValueError("desc must be the device uint8 array of G descriptors")
    _run("mgemm_list", desc.device, desc.data_ptr(), int(G))


def grouped_list(groups, outs=None):
    """Independent GEMMs D_g = A_g @ B_g.T with per-group shapes in one launch.

    groups: [(A_g bf16 [m_g, k_g], B_g bf16 [n_g, k_g]), ...]; outs: optional
    [D_g bf16 [m_g, n_g], ...] (allocated when None).  Returns the D list."""
    if not groups:
        return []
    if outs is None:
        outs = [torch.empty((a.shape[0], b.shape[0]), dtype=torch.bfloat16, device=a.device)
                for a, b in groups]
    desc = list_descriptors(groups, outs)
    grouped_list_desc(desc, len(groups))
    return outs


def mx_scales_blocked(scales: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """E8M0 scales [..., rows, K/32] (uint8) -> the blocked layout
    [..., ceil(K/128), rows, 4] that fwd_mx reads (absent blocks 127)."""
    if not isinstance(scales, torch.Tensor) or scales.dtype != torch.uint8 or scales.dim() < 2:
        raise TypeError("scales must be a uint8 tensor [..., rows, K/32]")
    _need(scales, "scales", torch.uint8, scales.dim())
    *lead, rows, nb = scales.shape
    batch = 1
    for d in lead:
        batch *= d
    shape = (*lead, (nb + 3) // 4, rows, 4)
    if out is None:
        out = torch.empty(shape, dtype=torch.uint8, device=scales.device)
    else:
        _need(out, "out", torch.uint8, len(shape))
        if tuple(out.shape) != shape:
            raise ValueError(f"out must be {shape}")
    _same_device(scales.device, out=out)
    _run("mg_mx_scales_blocked", scales.device, scales.data_ptr(), out.data_ptr(), rows, 32 * nb,
         batch)
    return out


def fwd_mx(x8: torch.Tensor, x_scale: torch.Tensor, w8: torch.Tensor, w_scale: torch.Tensor,
           offsets: torch.Tensor, max_m_per_e: int = 0,
           out: torch.Tensor | None = None) -> torch.Tensor:
    """MXFP8 M-grouped forward: out[i] = X[i] @ W[e].T with X, W the E4M3
    codes x8 [M, K], w8 [E, N, K] (uint8) times their E8M0 block scales.

    x_scale: blocked [ceil(K/128), M, 4]; w_scale: blocked [E, ceil(K/128), N, 4]
    (mx_scales_blocked makes them from [M, K/32] and [E, N, K/32]).  out bf16
    [M, N]; rows past offsets[E] are left untouched."""
    _need(x8, "x8", torch.uint8, 2)
    _need(w8, "w8", torch.uint8, 3)
    M, K = x8.shape
    E, N, K2 = w8.shape
    if K2 != K:
        raise ValueError(f"x8 is [M, {K}] but w8 is [E, N, {K2}]")
    kt = (K + 127) // 128
    _need(x_scale, "x_scale", torch.uint8, 3)
    _need(w_scale, "w_scale", torch.uint8, 4)
    if tuple(x_scale.shape) != (kt, M, 4) or tuple(w_scale.shape) != (E, kt, N, 4):
        raise ValueError(f"blocked scales must be [{kt}, {M}, 4] and [{E}, {kt}, {N}, 4]")
    _offsets(offsets, E, x8.device)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x8.device)
    else:
        _need(out, "out", torch.bfloat16, 2)
        if tuple(out.shape) != (M, N):
            raise ValueError(f"out must be [{M}, {N}]")
    _same_device(x8.device, x_scale=x_scale, w8=w8, w_scale=w_scale, out=out)
    _run("mgemm_fwd_mx", x8.device, x8.data_ptr(), x_scale.data_ptr(), w8.data_ptr(),
         w_scale.data_ptr(), offsets.data_ptr(), out.data_ptr(), M, N, K, E, int(max_m_per_e))
    return out


def _codes_out(M, K, dev, out, scales):
    # (sizes as separate arguments: 1.3 us of the host's time, as a tuple 1.6)
    nb = (K + 127) // 128
    if out is None:
        out = torch.empty(M, K, dtype=torch.uint8, device=dev)
    else:
        _need(out, "out", torch.uint8, 2)
        if tuple(out.shape) != (M, K):
            raise ValueError(f"out must be {[M, K]}")
        _same_device(dev, out=out)
    if scales is None:
        scales = torch.empty(nb, M, dtype=torch.float32, device=dev)
    else:
        _need(scales, "scales", torch.float32, 2)
        if tuple(scales.shape) != (nb, M):
            raise ValueError(f"scales must be [{nb}, {M}]")
        _same_device(dev, scales=scales)
    return out, scales


def _rows_offsets(offsets, dev):
    if offsets is None:
        return 0
    _need(offsets, "offsets", torch.int32, 1)
    if offsets.numel() < 2:
        raise ValueError("offsets must have E+1 entries")
    _same_device(dev, offsets=offsets)
    return offsets.numel() - 1


def fp8_quantize(x: torch.Tensor, gather: torch.Tensor | None = None,
                 offsets: torch.Tensor | None = None, out: torch.Tensor | None = None,
                 scales: torch.Tensor | None = None):
    """Rows to block-scaled fp8: (uint8 E4M3 codes [M, K], fp32 scales [ceil(K/128), M]).

    x bf16 or fp32 [M, K]; each row's 128 columns get the scale max|x| / 448.
    With `gather` (int32 [M]) row i is x[gather[i]] of x [T, K] (an index
    outside [0, T) gives zeros).  With `offsets` (int32 [E+1]) rows past
    offsets[E] are left untouched.  K a multiple of 16."""
    if not isinstance(x, torch.Tensor) or x.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("x must be a torch.bfloat16 or torch.float32 tensor")
    _need(x, "x", x.dtype, 2)
    T, K = x.shape
    M = T
    if gather is not None:
        _need(gather, "gather", torch.int32, 1)
        _same_device(x.device, gather=gather)
        M = gather.numel()
    E = _rows_offsets(offsets, x.device)
    out, scales = _codes_out(M, K, x.device, out, scales)
    _run("mg_fp8_quantize", x.device, x.data_ptr(), 1 if x.dtype == torch.float32 else 0,
         _ptr(gather), _ptr(offsets), out.data_ptr(), scales.data_ptr(), M, T, K, E)
    return out, scales


def fp8_quantize_swiglu(gu: torch.Tensor, offsets: torch.Tensor | None = None,
                        out: torch.Tensor | None = None, scales: torch.Tensor | None = None):
    """fp8_quantize of silu(g) u, in fp32 from gu = g | u (bf16 [M, 2I]):
    (codes [M, I], scales [ceil(I/128), M]); I a multiple of 16."""
    _need(gu, "gu", torch.bfloat16, 2)
    M, I2 = gu.shape
    if I2 % 2:
        raise ValueError(f"gu must hold two halves (2I columns), got {I2}")
    E = _rows_offsets(offsets, gu.device)
    out, scales = _codes_out(M, I2 // 2, gu.device, out, scales)
    _run("mg_fp8_quantize_swiglu", gu.device, gu.data_ptr(), _ptr(offsets), out.data_ptr(),
         scales.data_ptr(), M, I2 // 2, E)
    return out, scales


def fp8_quantize_weights(w: torch.Tensor, out: torch.Tensor | None = None,
                         scales: torch.Tensor | None = None):
    """Weights (bf16 or fp32 [E, N, K]) to block-scaled fp8: (uint8 codes
    [E, N, K], fp32 scales [E, ceil(N/128), ceil(K/128)]), one scale per
    128 x 128 block.  K a multiple of 16."""
    if not isinstance(w, torch.Tensor) or w.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("w must be a torch.bfloat16 or torch.float32 tensor")
    _need(w, "w", w.dtype, 3)
    E, N, K = w.shape
    shape = (E, (N + 127) // 128, (K + 127) // 128)
    if out is None:
        out = torch.empty(E, N, K, dtype=torch.uint8, device=w.device)
    else:
        _need(out, "out", torch.uint8, 3)
        if tuple(out.shape) != (E, N, K):
            raise ValueError(f"out must be [{E}, {N}, {K}]")
    if scales is None:
        scales = torch.empty(*shape, dtype=torch.float32, device=w.device)
    else:
        _need(scales, "scales", torch.float32, 3)
        if tuple(scales.shape) != shape:
            raise ValueError(f"scales must be {list(shape)}")
    _same_device(w.device, out=out, scales=scales)
    _run("mg_fp8_quantize_weights", w.device, w.data_ptr(), 1 if w.dtype == torch.float32 else 0,
         out.data_ptr(), scales.data_ptr(), E, N, K)
    return out, scales


def fwd_fp8(x8: torch.Tensor, x_scale: torch.Tensor, w8: torch.Tensor, w_scale: torch.Tensor,
            offsets: torch.Tensor, max_m_per_e: int = 0,
            out: torch.Tensor | None = None) -> torch.Tensor:
    """Block-scaled fp8 M-grouped forward: out[i] = X[i] @ W[e].T.

    x8 uint8 E4M3 codes [M, K] with x_scale fp32 [ceil(K/128), M] (one scale per
    row and 128 columns, as fp8_quantize returns them), w8 [E, N, K] with
    w_scale fp32 [E, ceil(N/128), ceil(K/128)] (one per 128 x 128 block, as
    fp8_quantize_weights returns them); N and K multiples of 16.  out bf16
    [M, N]; rows past offsets[E] are left untouched."""
    return _product_fp8("mgemm_fwd_fp8", False, x8, x_scale, w8, w_scale, offsets, max_m_per_e, out)


def dgrad_fp8(dy8: torch.Tensor, dy_scale: torch.Tensor, w8: torch.Tensor, w_scale: torch.Tensor,
              offsets: torch.Tensor, max_m_per_e: int = 0,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """Block-scaled fp8 M-grouped input gradient: out[i] = DY[i] @ W[e].

    dy8 uint8 E4M3 codes [M, N] with dy_scale fp32 [ceil(N/128), M]; w8 and
    w_scale as for fwd_fp8.  out bf16 [M, K]."""
    return _product_fp8("mgemm_dgrad_fp8", True, dy8, dy_scale, w8, w_scale, offsets, max_m_per_e,
                        out)


def _product_fp8(fn, dgrad, q8, q_scale, w8, w_scale, offsets, max_m_per_e, out):
    q, scale = ("dy8", "dy_scale") if dgrad else ("x8", "x_scale")
    _need(q8, q, torch.uint8, 2)
    _need(w8, "w8", torch.uint8, 3)
    M, R = q8.shape
    E, N, K = w8.shape
    if R != (N if dgrad else K):
        raise ValueError(f"{q} is [M, {R}] but w8 is [E, {N}, {K}]")
    _need(q_scale, scale, torch.float32, 2)
    _need(w_scale, "w_scale", torch.float32, 3)
    nn, nk, nr = (N + 127) // 128, (K + 127) // 128, (R + 127) // 128
    if tuple(q_scale.shape) != (nr, M) or tuple(w_scale.shape) != (E, nn, nk):
        raise ValueError(f"scales must be [{nr}, {M}] and [{E}, {nn}, {nk}]")
    _offsets(offsets, E, q8.device)
    P = K if dgrad else N
    if out is None:
        out = torch.empty(M, P, dtype=torch.bfloat16, device=q8.device)
    else:
        _need(out, "out", torch.bfloat16, 2)
        if tuple(out.shape) != (M, P):
            raise ValueError(f"out must be [{M}, {P}]")
    _same_device(q8.device, w8=w8, out=out, w_scale=w_scale, **{scale: q_scale})
    _run(fn, q8.device, q8.data_ptr(), q_scale.data_ptr(), w8.data_ptr(), w_scale.data_ptr(),
         offsets.data_ptr(), out.data_ptr(), M, N, K, E, int(max_m_per_e))
    return out


def wgrad_mx(dyt8: torch.Tensor, dyt_scale: torch.Tensor, xt8: torch.Tensor,
             xt_scale: torch.Tensor, offsets: torch.Tensor, E: int | None = None,
             out: torch.Tensor | None = None, accumulate: bool = False) -> torch.Tensor:
    """MXFP8 K-grouped weight gradient: out[e] (=/+=) DYT[:, rows_e] @ XT[:, rows_e].T.

    dyt8 [N, M], xt8 [K, M]: uint8 E4M3 codes quantized along the tokens (token
    axis last); dyt_scale [M/128, N, 4], xt_scale [M/128, K, 4]: blocked E8M0
    scales (mx_scales_blocked of [N, M/32] and [K, M/32]).  offsets int32 [E+1]
    with every entry a multiple of 128.  out fp32 [E, N, K]."""
    _need(dyt8, "dyt8", torch.uint8, 2)
    _need(xt8, "xt8", torch.uint8, 2)
    N, M = dyt8.shape
    K, M2 = xt8.shape
    if M2 != M:
        raise ValueError(f"dyt8 is [N, {M}] but xt8 is [K, {M2}]")
    if E is None:
        E = offsets.numel() - 1
    _need(dyt_scale, "dyt_scale", torch.uint8, 3)
    _need(xt_scale, "xt_scale", torch.uint8, 3)
    if tuple(dyt_scale.shape) != (M // 128, N, 4) or tuple(xt_scale.shape) != (M // 128, K, 4):
        raise ValueError(f"blocked scales must be [{M // 128}, {N}, 4] and [{M // 128}, {K}, 4]")
    _offsets(offsets, E, dyt8.device)
    if out is None:
        if accumulate:
            raise ValueError("accumulate=True needs an `out` to add into")
        out = torch.empty((E, N, K), dtype=torch.float32, device=dyt8.device)
    else:
        _need(out, "out", torch.float32, 3)
        if tuple(out.shape) != (E, N, K):
            raise ValueError(f"out must be [{E}, {N}, {K}]")
    _same_device(dyt8.device, dyt_scale=dyt_scale, xt8=xt8, xt_scale=xt_scale, out=out)
    _run("kgemm_wgrad_mx", dyt8.device, dyt8.data_ptr(), dyt_scale.data_ptr(), xt8.data_ptr(),
         xt_scale.data_ptr(), offsets.data_ptr(), out.data_ptr(), M, N, K, E,
         1 if accumulate else 0)
    return out


def wgrad_mx_tm(dy8: torch.Tensor, dy_scale: torch.Tensor, x8: torch.Tensor,
                x_scale: torch.Tensor, offsets: torch.Tensor, E: int | None = None,
                out: torch.Tensor | None = None, accumulate: bool = False) -> torch.Tensor:
    """MXFP8 K-grouped weight gradient on token-major operands:
    out[e] (=/+=) DY[rows_e].T @ X[rows_e].

    dy8 [M, N], x8 [M, K]: uint8 E4M3 codes quantized along the tokens (token
    axis first, as the layer holds them); dy_scale [M/128, N, 4], x_scale
    [M/128, K, 4]: blocked E8M0 scales (mx_scales_blocked of [N, M/32] and
    [K, M/32]).  offsets int32 [E+1] with every entry a multiple of 128.
    out fp32 [E, N, K]."""
    _need(dy8, "dy8", torch.uint8, 2)
    _need(x8, "x8", torch.uint8, 2)
    M, N = dy8.shape
    M2, K = x8.shape
    if M2 != M:
        raise ValueError(f"dy8 is [{M}, N] but x8 is [{M2}, K]")
    if E is None:
        E = offsets.numel() - 1
    _need(dy_scale, "dy_scale", torch.uint8, 3)
    _need(x_scale, "x_scale", torch.uint8, 3)
    if tuple(dy_scale.shape) != (M // 128, N, 4) or tuple(x_scale.shape) != (M // 128, K, 4):
        raise ValueError(f"blocked scales must be [{M // 128}, {N}, 4] and [{M // 128}, {K}, 4]")
    _offsets(offsets, E, dy8.device)
    if out is None:
        if accumulate:
            raise ValueError("accumulate=True needs an `out` to add into")
        out = torch.empty((E, N, K), dtype=torch.float32, device=dy8.device)
    else:
        _need(out, "out", torch.float32, 3)
        if tuple(out.shape) != (E, N, K):
            raise ValueError(f"out must be [{E}, {N}, {K}]")
    _same_device(dy8.device, dy_scale=dy_scale, x8=x8, x_scale=x_scale, out=out)
    _run("kgemm_wgrad_mx_tm", dy8.device, dy8.data_ptr(), dy_scale.data_ptr(), x8.data_ptr(),
         x_scale.data_ptr(), offsets.data_ptr(), out.data_ptr(), M, N, K, E, 1 if accumulate else 0)
    return out


def moe_combine(rows: torch.Tensor, token_rows: torch.Tensor,
                weights: torch.Tensor | None = None, out: torch.Tensor | None = None
                ) -> torch.Tensor:
    """out[t] = sum_j weights[t, j] rows[token_rows[t, j]] (bf16 [T, D]).

    rows bf16 [M, D]; token_rows int32 [T, k] (-1 = no row); weights fp32
    [T, k] or None (all 1).  The backward of the row gather of fwd_swiglu, or
    the layer's weighted output combine."""
    _need(rows, "rows", torch.bfloat16, 2)
    _need(token_rows, "token_rows", torch.int32, 2)
    M, D = rows.shape
    T, k = token_rows.shape
    wptr = 0
    if weights is not None:
        _need(weights, "weights", torch.float32, 2)
        if tuple(weights.shape) != (T, k):
            raise ValueError(f"weights must be [{T}, {k}]")
        wptr = weights.data_ptr()
    if out is None:
        out = torch.empty((T, D), dtype=torch.bfloat16, device=rows.device)
    else:
        _need(out, "out", torch.bfloat16, 2)
        if tuple(out.shape) != (T, D):
            raise ValueError(f"out must be [{T}, {D}]")
    _same_device(rows.device, token_rows=token_rows, weights=weights, out=out)
    _run("mg_moe_combine", rows.device, rows.data_ptr(), token_rows.data_ptr(), wptr,
         out.data_ptr(), M, T, k, D)
    return out


def moe_combine_bwd(dout: torch.Tensor, rows: torch.Tensor, token_rows: torch.Tensor,
                    weights: torch.Tensor | None = None, drows: torch.Tensor | None = None):
    """Gradient of moe_combine: (drows bf16 [M, D], dweights fp32 [T, k]).

    drows[token_rows[t, j]] = weights[t, j] dout[t], dweights[t, j] =
    rows[token_rows[t, j]] . dout[t]; dweights is None without weights.  No row
    may be named twice by token_rows (moe_route names none twice); rows that
    none names are left untouched in `drows`.  Where it is None they are zeros:
    the whole of [M, D] is filled first, so a caller with a buffer passes it
    (8192 x 8 rows of 2048: 113 us with one, 146 us without)."""
    _need(dout, "dout", torch.bfloat16, 2)
    _need(rows, "rows", torch.bfloat16, 2)
    _need(token_rows, "token_rows", torch.int32, 2)
    M, D = rows.shape
    T, k = token_rows.shape
    if tuple(dout.shape) != (T, D):
        raise ValueError(f"dout must be [{T}, {D}]")
    dweights = None
    if weights is not None:
        _need(weights, "weights", torch.float32, 2)
        if tuple(weights.shape) != (T, k):
            raise ValueError(f"weights must be [{T}, {k}]")
        dweights = torch.empty(T, k, dtype=torch.float32, device=rows.device)
    if drows is None:
        drows = torch.zeros((M, D), dtype=torch.bfloat16, device=rows.device)
    else:
        _need(drows, "drows", torch.bfloat16, 2)
        if tuple(drows.shape) != (M, D):
            raise ValueError(f"drows must be [{M}, {D}]")
    _same_device(rows.device, dout=dout, token_rows=token_rows, weights=weights, drows=drows)
    _run("mg_moe_combine_bwd", rows.device, dout.data_ptr(), rows.data_ptr(), token_rows.data_ptr(),
         _ptr(weights), drows.data_ptr(), _ptr(dweights), M, T, k, D)
    return drows, dweights


class Route(NamedTuple):
    """What moe_route computes (sizes for T tokens, E experts, k per token)."""
    weights: torch.Tensor     # fp32 [T, k]   gate weights (moe_combine's weights)
    experts: torch.Tensor     # int32 [T, k]  chosen experts, -1 = none
    lse: torch.Tensor         # fp32 [T]      log-sum-exp of the logits
    counts: torch.Tensor      # int32 [E]     entries per expert
    prob_sum: torch.Tensor    # fp32 [E]      sum of the probabilities
    tokens: torch.Tensor      # int32 [1]     tokens that count
    loss: torch.Tensor        # fp32 [2]      balance loss, z loss
    offsets: torch.Tensor     # int32 [local + 1]  row ranges of the local experts
    gather: torch.Tensor      # int32 [T k]   token of each row, -1 behind the last
    token_rows: torch.Tensor  # int32 [T, k]  row of each entry, -1 = none


def _logits(logits: torch.Tensor) -> None:
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a torch.Tensor")
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"logits must be torch.float32 or torch.bfloat16, got {logits.dtype}")
    _need(logits, "logits", logits.dtype, 2)


def moe_route(logits: torch.Tensor, k: int, normalize: bool = True,
              mask: torch.Tensor | None = None, first: int = 0,
              local: int | None = None) -> Route:
    """Router: gate, row order and balance of logits [T, E] (fp32 or bf16).

    The k largest logits of a token choose its experts (ties to the lower
    index); `normalize` divides their softmax probabilities by their sum.
    `mask` (bool or uint8 [T]) leaves out padding tokens; an expert whose logit
    is -inf (or NaN) is never chosen.  offsets, gather and token_rows describe
    the rows of experts first .. first + local - 1 (all by default), as
    fwd_swiglu, fp8_quantize and moe_combine take them.  loss = (balance, z):
    E sum_e (counts_e / sum counts) (prob_sum_e / n), and the mean of lse^2."""
    _logits(logits)
    T, E = logits.shape
    k = int(k)
    if not 1 <= k <= min(E, 64):
        raise ValueError(f"k must be in [1, min(E, 64)] = [1, {min(E, 64)}], got {k}")
    local = E - first if local is None else int(local)
    if first < 0 or local < 1 or first + local > E:
        raise ValueError(f"experts {first} .. {first + local - 1} are not among {E}")
    if mask is not None:
        if isinstance(mask, torch.Tensor) and mask.dtype == torch.bool:
            mask = mask.view(torch.uint8)
        _need(mask, "mask", torch.uint8, 1)
        if mask.numel() != T:
            raise ValueError(f"mask must have {T} entries, got {mask.numel()}")
        _same_device(logits.device, mask=mask)
    dev = logits.device
    # one allocation per type, the outputs (and the workspace) being parts of it
    words = LIB.mg_moe_route_workspace(T, E) // 4
    n = T * k
    f = torch.empty(n + T + E + 2, dtype=torch.float32, device=dev)
    i = torch.empty(3 * n + E + 2 + local + words, dtype=torch.int32, device=dev)
    weights, lse, prob_sum, loss = f.split_with_sizes((n, T, E, 2))
    experts, gather, token_rows, counts, tokens, offsets, work = i.split_with_sizes(
        (n, n, n, E, 1, local + 1, words))
    # what a sum over ranks replaces has a version of its own: autograd's check
    # of the saved others does not see it
    counts, tokens, prob_sum = counts.data, tokens.data, prob_sum.data
    r = Route(weights.view(T, k), experts.view(T, k), lse, counts, prob_sum, tokens, loss, offsets,
              gather, token_rows.view(T, k))
    _run("mg_moe_route", dev, logits.data_ptr(), 1 if logits.dtype == torch.bfloat16 else 0,
         _ptr(mask), T, E, k, 1 if normalize else 0, int(first), local, r.weights.data_ptr(),
         r.experts.data_ptr(), r.lse.data_ptr(), r.counts.data_ptr(), r.prob_sum.data_ptr(),
         r.tokens.data_ptr(), r.loss.data_ptr(), r.offsets.data_ptr(), r.gather.data_ptr(),
         r.token_rows.data_ptr(), work.data_ptr(), 4 * words)
    return r


def moe_route_bwd(logits: torch.Tensor, weights: torch.Tensor, experts: torch.Tensor,
                  lse: torch.Tensor, counts: torch.Tensor, tokens: torch.Tensor,
                  dweights: torch.Tensor | None = None, dloss: torch.Tensor | None = None,
                  normalize: bool = True, out: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of moe_route to the logits (their type, [T, E]).

    weights, experts, lse, counts and tokens are the forward's; for a balance
    over several ranks' tokens, counts and tokens are their sums.  dweights
    (fp32 [T, k]) is the gradient of the weights, dloss (fp32 [2]) that of
    (balance, z); either may be None.  `normalize` as in the forward."""
    _logits(logits)
    T, E = logits.shape
    _need(experts, "experts", torch.int32, 2)
    k = experts.shape[1]
    if experts.shape[0] != T:
        raise ValueError(f"experts must be [{T}, k]")
    for name, t in (("weights", weights), ("dweights", dweights)):
        if t is not None or name == "weights":
            _need(t, name, torch.float32, 2)
            if tuple(t.shape) != (T, k):
                raise ValueError(f"{name} must be [{T}, {k}]")
    _need(lse, "lse", torch.float32, 1)
    _need(counts, "counts", torch.int32, 1)
    _need(tokens, "tokens", torch.int32, 1)
    if lse.numel() != T or counts.numel() != E or tokens.numel() != 1:
        raise ValueError(f"lse, counts and tokens must have {T}, {E} and 1 entries")
    if dloss is not None:
        _need(dloss, "dloss", torch.float32, 1)
        if dloss.numel() != 2:
            raise ValueError("dloss must have 2 entries (balance, z)")
    if out is None:
        out = torch.empty_like(logits)
    else:
        _need(out, "out", logits.dtype, 2)
        if tuple(out.shape) != (T, E):
            raise ValueError(f"out must be [{T}, {E}]")
    _same_device(logits.device, weights=weights, experts=experts, lse=lse, counts=counts,
                 tokens=tokens, dweights=dweights, dloss=dloss, out=out)
    _run("mg_moe_route_bwd", logits.device, logits.data_ptr(),
         1 if logits.dtype == torch.bfloat16 else 0, weights.data_ptr(), experts.data_ptr(),
         lse.data_ptr(), counts.data_ptr(), tokens.data_ptr(), _ptr(dweights), _ptr(dloss),
         out.data_ptr(), T, E, k, 1 if normalize else 0)
    return out


class HeadLoss(NamedTuple):
    """What head_loss computes, fp32 [T] each."""
    loss: torch.Tensor        # lse - logit
    lse: torch.Tensor         # log-sum-exp of the token's logits
    logit: torch.Tensor       # logit of its target


class HeadDistill(NamedTuple):
    """What head_distill computes, in fp32."""
    loss: torch.Tensor        # [T]     divergence from the teacher's entries
    lse: torch.Tensor         # [T]     log-sum-exp of the token's logits / temperature
    logits: torch.Tensor      # [T, k]  logits of the entries


def _head(x: torch.Tensor, w: torch.Tensor, first: int) -> tuple:
    _need(x, "x", torch.bfloat16, 2)
    _need(w, "w", torch.bfloat16, 2)
    T, D = x.shape
    V, D2 = w.shape
    if D2 != D:
        raise ValueError(f"x is [T, {D}] but w is [V, {D2}]")
    if first < 0 or first + V > 2 ** 31:
        raise ValueError(f"vocabulary entries {first} .. {first + V - 1} are no int32 indices")
    return T, V, D


def _per_token(T: int, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None:
            _need(t, name, torch.float32, 1)
            if t.numel() != T:
                raise ValueError(f"{name} must have {T} entries, got {t.numel()}")


def _targets(targets: torch.Tensor, T: int) -> None:
    _need(targets, "targets", torch.int32, 1)
    if targets.numel() != T:
        raise ValueError(f"targets must have {T} entries, got {targets.numel()}")


def _teacher(teacher: torch.Tensor, index: torch.Tensor, T: int, temperature: float) -> int:
    if not isinstance(teacher, torch.Tensor) or teacher.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("teacher must be a torch.float32 or torch.bfloat16 tensor")
    _need(teacher, "teacher", teacher.dtype, 2)
    _need(index, "index", torch.int32, 2)
    k = index.shape[1]
    if tuple(index.shape) != (T, k) or tuple(teacher.shape) != (T, k):
        raise ValueError(f"teacher and index must be [{T}, k]")
    if not 1 <= k <= 256:
        raise ValueError(f"k must be in [1, 256], got {k}")
    if not 0.0 < temperature < float("inf"):
        raise ValueError(f"temperature must be positive and finite, got {temperature}")
    return k


def _overlap(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether two contiguous 16-bit tensors share memory."""
    return a.data_ptr() < b.data_ptr() + 2 * b.numel() and b.data_ptr() < a.data_ptr() + 2 * a.numel()


def _head_grads(x, w, dx, dw, need_dx, need_dw, words):
    """The gradients' tensors (None where not wanted) and the workspace."""
    out = []
    for name, like, t, need in (("dx", x, dx, need_dx), ("dw", w, dw, need_dw)):
        if not need:
            if t is not None:
                raise ValueError(f"{name} is given but need_{name} is False")
        elif t is None:
            t = torch.empty_like(like)
        else:
            _need(t, name, torch.bfloat16, 2)
            if t.shape != like.shape:
                raise ValueError(f"{name} must be {list(like.shape)}")
        out.append(t)
    _same_device(x.device, dx=out[0], dw=out[1])
    # the caller's buffers: the weights are still read while gradients are written
    for name, t, given, others in (("dx", out[0], dx, (x, w)), ("dw", out[1], dw, (x, w, out[0]))):
        if given is not None and any(o is not None and _overlap(t, o) for o in others):
            raise ValueError(f"{name} may not overlap x, w or the other gradient")
    return *out, torch.empty(words, dtype=torch.uint8, device=x.device)


def head_loss(x: torch.Tensor, w: torch.Tensor, targets: torch.Tensor, first: int = 0) -> HeadLoss:
    """Cross entropy of the output head, without keeping the logits z = x w^T.

    x bf16 [T, D], w bf16 [V, D] (D a multiple of 8, V of any size up to
    2^31 - 256), targets int32 [T].
    loss = lse - logit per token, lse = logsumexp(z), logit = z[target].  A
    token with a negative target does not count: its loss, lse and logit are 0.
    Where the vocabulary is spread over ranks, `first` is the index of w's row
    0 and a target in another part has logit 0 here: with the parts' lse joined
    (torch.logaddexp) and their logits summed, loss = lse - logit."""
    T, V, D = _head(x, w, first)
    _targets(targets, T)
    _same_device(x.device, w=w, targets=targets)
    loss, lse, logit = torch.empty(3 * T, dtype=torch.float32, device=x.device).split_with_sizes((T, T, T))
    size = LIB.mg_head_workspace(T, V, D)
    work = torch.empty(size, dtype=torch.uint8, device=x.device)
    _run("mg_head_loss", x.device, x.data_ptr(), w.data_ptr(), targets.data_ptr(), T, V, D, int(first),
         loss.data_ptr(), lse.data_ptr(), logit.data_ptr(), work.data_ptr(), size)
    return HeadLoss(loss, lse, logit)


def head_loss_bwd(x: torch.Tensor, w: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor,
                  dloss: torch.Tensor, dlse: torch.Tensor | None = None, first: int = 0,
                  dx: torch.Tensor | None = None, dw: torch.Tensor | None = None,
                  need_dx: bool = True, need_dw: bool = True):
    """Gradient of head_loss: (dx bf16 [T, D], dw bf16 [V, D]).

    lse is the forward's (over ranks: the joined one; dx is then a part of a
    sum).  dloss and dlse (fp32 [T]) are the gradients of loss and of lse (a z
    loss on top: 2 c lse); tokens that do not count have none.  Either gradient
    may be left out (need_dx, need_dw) and is None then."""
    T, V, D = _head(x, w, first)
    _targets(targets, T)
    _per_token(T, lse=lse, dloss=dloss, dlse=dlse)
    _same_device(x.device, w=w, targets=targets, lse=lse, dloss=dloss, dlse=dlse)
    size = LIB.mg_head_bwd_workspace(T, V, D, 0)
    dx, dw, work = _head_grads(x, w, dx, dw, need_dx, need_dw, size)
    _run("mg_head_loss_bwd", x.device, x.data_ptr(), w.data_ptr(), targets.data_ptr(), lse.data_ptr(),
         dloss.data_ptr(), _ptr(dlse), T, V, D, int(first), _ptr(dx), _ptr(dw), work.data_ptr(), size)
    return dx, dw


def head_distill(x: torch.Tensor, w: torch.Tensor, teacher: torch.Tensor, index: torch.Tensor,
                 temperature: float = 1.0, first: int = 0) -> HeadDistill:
    """Distillation of the output head from a teacher's k top logits per token.

    teacher fp32 or bf16 [T, k], index int32 [T, k] (k <= 256): the teacher's
    logits and their places in the vocabulary, -1 for no entry (a value of -inf
    or NaN is none either).  q = softmax(teacher / temperature) over a token's
    entries, loss = sum q (log q - log p) with p = softmax(z / temperature) over
    the vocabulary; a token without entries has loss and lse 0.  `first` as in
    head_loss: with joined lse and summed logits, loss = sum q (log q + lse -
    logits / temperature)."""
    T, V, D = _head(x, w, first)
    k = _teacher(teacher, index, T, temperature)
    _same_device(x.device, w=w, teacher=teacher, index=index)
    loss, lse, logits = torch.empty((2 + k) * T, dtype=torch.float32,
                                    device=x.device).split_with_sizes((T, T, T * k))
    size = LIB.mg_head_workspace(T, V, D)
    work = torch.empty(size, dtype=torch.uint8, device=x.device)
    _run("mg_head_distill", x.device, x.data_ptr(), w.data_ptr(), teacher.data_ptr(),
         1 if teacher.dtype == torch.bfloat16 else 0, index.data_ptr(), T, V, D, k, int(first),
         float(temperature), loss.data_ptr(), lse.data_ptr(), logits.data_ptr(), work.data_ptr(), size)
    return HeadDistill(loss, lse, logits.view(T, k))


def head_distill_bwd(x: torch.Tensor, w: torch.Tensor, teacher: torch.Tensor, index: torch.Tensor,
                     lse: torch.Tensor, logits: torch.Tensor, dloss: torch.Tensor,
                     temperature: float = 1.0, first: int = 0, dx: torch.Tensor | None = None,
                     dw: torch.Tensor | None = None, need_dx: bool = True, need_dw: bool = True):
    """Gradient of head_distill: (dx bf16 [T, D], dw bf16 [V, D]).

    lse and logits are the forward's, dloss (fp32 [T]) the gradient of its
    loss; the teacher gets none.  Otherwise as head_loss_bwd."""
    T, V, D = _head(x, w, first)
    k = _teacher(teacher, index, T, temperature)
    _per_token(T, lse=lse, dloss=dloss)
    _need(logits, "logits", torch.float32, 2)
    if tuple(logits.shape) != (T, k):
        raise ValueError(f"logits must be [{T}, {k}]")
    _same_device(x.device, w=w, teacher=teacher, index=index, lse=lse, logits=logits, dloss=dloss)
    size = LIB.mg_head_bwd_workspace(T, V, D, k)
    dx, dw, work = _head_grads(x, w, dx, dw, need_dx, need_dw, size)
    _run("mg_head_distill_bwd", x.device, x.data_ptr(), w.data_ptr(), teacher.data_ptr(),
         1 if teacher.dtype == torch.bfloat16 else 0, index.data_ptr(), lse.data_ptr(),
         logits.data_ptr(), dloss.data_ptr(), T, V, D, k, int(first), float(temperature), _ptr(dx),
         _ptr(dw), work.data_ptr(), size)
    return dx, dw


def Mgemm(x: torch.Tensor, w: torch.Tensor, cnt: torch.Tensor, max_M_per_E: int = 0,
          transpose_B: bool = True) -> torch.Tensor:
    """RapidGEMM-shaped M-grouped GEMM (README, "Kernels").

    w is stored [E, N, K].  transpose_B=True uses it transposed (the forward,
    x [M, K] -> [M, N]); transpose_B=False uses it as stored (the input
    gradient, x [M, N] -> [M, K]).  cnt: cumulative row offsets with a leading
    zero."""
    if transpose_B:
        return fwd(x, w, cnt, max_M_per_E)
    return dgrad(x, w, cnt, max_M_per_E)


def Kgemm(grad: torch.Tensor, X: torch.Tensor, cnt: torch.Tensor,
          descriptor: str | None = None) -> torch.Tensor:
    """RapidGEMM-shaped K-grouped fp32 weight gradient (README, "Kernels").

    descriptor names which weight is differentiated ("gw13": fused gate/up
    projection, "gw2": down projection); shapes come from the tensors, so it
    is only a label here."""
    if descriptor not in (None, "gw13", "gw2"):
        raise ValueError(f"descriptor must be 'gw13', 'gw2' or None, got {descriptor!r}")
    return wgrad(grad, X, cnt)
