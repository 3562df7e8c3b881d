"""Child process of test_validation_gpu.py: run with MGEMM_VALIDATE=1 in its
environment (the library reads it once per process).  Prints one line per check
and exits non-zero on the first failure."""
import sys

import numpy as np
import torch

import moe_grouped_gemm_bf16_amd as mg
from moe_grouped_gemm_bf16_amd._lib import MG_ERR_OFFSETS, MgemmError


def refused(fn, what, *untouched):
    """fn raises MG_ERR_OFFSETS and leaves the tensors, filled with 7, alone."""
    for t in untouched:
        t.fill_(7)
    try:
        fn()
    except MgemmError as ex:
        assert ex.status == MG_ERR_OFFSETS, f"{what}: status {ex.status}"
        torch.cuda.synchronize()
        assert all(bool((t == 7).all()) for t in untouched), f"{what}: a refused call wrote its output"
        print("[child] refused:", what, flush=True)
        return
    raise AssertionError(f"{what}: not refused")


def main():
    torch.manual_seed(0)
    dev = dict(device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, **dev)   # noqa: E731
    E, M, N, K = 3, 20, 32, 48
    x, w = torch.randn(M, K, **dev).bfloat16(), torch.randn(E, N, K, **dev)
    good = i32([0, 5, 12, 18])
    bad = {"decreasing": i32([0, 12, 5, 18]), "past M": i32([0, 5, 12, M + 1]), "no leading zero": i32([1, 5, 12, 18])}

    x8, xs = mg.fp8_quantize(x, offsets=good, out=torch.zeros(M, K, dtype=torch.uint8, **dev), scales=torch.zeros(1, M, **dev))
    plain8, plains = mg.fp8_quantize(x)
    assert torch.equal(x8[:18], plain8[:18]) and torch.equal(xs[:, :18], plains[:, :18])
    w8, ws = mg.fp8_quantize_weights(w)
    y = mg.fwd_fp8(x8, xs, w8, ws, good)
    dy8, dys = mg.fp8_quantize(y, offsets=good, out=torch.zeros(M, N, dtype=torch.uint8, **dev), scales=torch.zeros(1, M, **dev))
    dx = mg.dgrad_fp8(dy8, dys, w8, ws, good)
    gu = torch.randn(M, 2 * N, **dev).bfloat16()
    mg.fp8_quantize_swiglu(gu, offsets=good)
    assert torch.isfinite(y[:18]).all() and torch.isfinite(dx[:18]).all()
    print("[child] valid offsets pass", flush=True)

    outs = {n: torch.empty(M, c, dtype=t, **dev) for n, c, t in (("y", N, torch.bfloat16), ("dx", K, torch.bfloat16), ("c", K, torch.uint8), ("h", N, torch.uint8))}
    s = torch.empty(1, M, **dev)
    for name, off in bad.items():
        refused(lambda: mg.fwd_fp8(x8, xs, w8, ws, off, out=outs["y"]), "fwd_fp8, " + name, outs["y"])
        refused(lambda: mg.dgrad_fp8(dy8, dys, w8, ws, off, out=outs["dx"]), "dgrad_fp8, " + name, outs["dx"])
        refused(lambda: mg.fp8_quantize(x, offsets=off, out=outs["c"], scales=s), "fp8_quantize, " + name, outs["c"], s)
        refused(lambda: mg.fp8_quantize_swiglu(gu, offsets=off, out=outs["h"], scales=s), "fp8_quantize_swiglu, " + name, outs["h"], s)

    T, k = 4, 3
    rows, dout, wt = torch.randn(12, 64, **dev).bfloat16(), torch.randn(T, 64, **dev).bfloat16(), torch.rand(T, k, **dev)
    at = i32(np.arange(12).reshape(T, k).tolist())
    at[1, 1], at[2, 0] = -1, 40                              # no row, out of range: neither names one
    drows, dw = mg.moe_combine_bwd(dout, rows, at, wt)
    assert torch.equal(drows[0], (wt[0, 0] * dout[0].float()).bfloat16()) and float(dw[1, 1]) == 0
    print("[child] rows named once pass", flush=True)
    at[3, 2] = 0
    refused(lambda: mg.moe_combine_bwd(dout, rows, at, wt, drows=drows), "moe_combine_bwd, a row named twice", drows)
    print("[child] ok", flush=True)


if __name__ == "__main__":
    main()
    sys.exit(0)
