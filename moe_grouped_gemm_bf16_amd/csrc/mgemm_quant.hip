// Block-scaled fp8 quantizers: values to E4M3 codes with one fp32 scale per
// row and 128 columns (activations) or per 128 x 128 block (weights):
//   a = max(max |x| over the block, 2^-100),  scale = a / 448,
//   code = e4m3(x (448 / a))            (448: the largest E4M3 value)
// with both quotients correctly rounded fp32 divisions and the product rounded
// once to fp32 and once, to nearest even, to E4M3.  The floor 2^-100 keeps
// 448 / a finite; a block of zeros gets it and zero codes.  A NaN, or an
// infinity (whose scale is infinite), gives NaN codes, so the outputs of that
// row's products are NaN and no other row's.
//
// HBM-bound (2 bytes in, 1 byte out per bf16 value): 16 lanes hold one block's
// 128 columns, 8 each, so its maximum is four lane-row rotations away, and
// a wave's rows are all loaded before the first is used.  The scales, whose rows
// run along M, leave through LDS in runs.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mgemm_launch.h"

namespace mg {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr float kTop = 448.0f;
constexpr float kFloor = 0x1p-100f;
constexpr int kRowsPerWave = 2;

template <int CTRL>
__device__ __forceinline__ float rotate_max(float x) {
  const int y = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xF, 0xF, false);
  return fmaxf(x, __builtin_bit_cast(float, y));
}
// Maximum over the 16 lanes of a lane row.
__device__ __forceinline__ float row_max(float x) {
  x = rotate_max<0x128>(x);
  x = rotate_max<0x124>(x);
  x = rotate_max<0x122>(x);
  return rotate_max<0x121>(x);
}

// STREAM: the value is read once, and should not push others out of the caches.
template <bool STREAM, typename V>
__device__ __forceinline__ V read16(const V* p) {
  if constexpr (STREAM) return __builtin_nontemporal_load(p);
  else return *p;
}

// Eight values as loaded: bf16 (one 16-byte piece) or fp32 (two).
template <typename T>
struct Eight;
template <>
struct Eight<uint16_t> {
  u32x4 v;
  __device__ __forceinline__ void zero() { v = u32x4{0u, 0u, 0u, 0u}; }
  template <bool STREAM>
  __device__ __forceinline__ void load(const uint16_t* p) { v = read16<STREAM>(reinterpret_cast<const u32x4*>(p)); }
  __device__ __forceinline__ void to(float (&f)[8]) const {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      f[2 * q] = __builtin_bit_cast(float, v[q] << 16);
      f[2 * q + 1] = __builtin_bit_cast(float, v[q] & 0xFFFF0000u);
    }
  }
};
template <>
struct Eight<float> {
  f32x4 lo, hi;
  __device__ __forceinline__ void zero() { lo = hi = f32x4{0.f, 0.f, 0.f, 0.f}; }
  template <bool STREAM>
  __device__ __forceinline__ void load(const float* p) {
    lo = read16<STREAM>(reinterpret_cast<const f32x4*>(p));
    hi = read16<STREAM>(reinterpret_cast<const f32x4*>(p + 4));
  }
  __device__ __forceinline__ void to(float (&f)[8]) const {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      f[q] = lo[q];
      f[4 + q] = hi[q];
    }
  }
};

__device__ __forceinline__ float abs_max8(const float (&f)[8]) {
  float a = fabsf(f[0]);
#pragma unroll
  for (int q = 1; q < 8; ++q) a = fmaxf(a, fabsf(f[q]));
  return a;
}

__device__ __forceinline__ u32x2 encode8(const float (&f)[8], float inv) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h] * inv, f[4 * h + 1] * inv, 0, false);
    v = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h + 2] * inv, f[4 * h + 3] * inv, v, true);
    w[h] = (uint32_t)v;
  }
  return u32x2{w[0], w[1]};
}

// Workgroup -> item, in runs of `run` neighbouring items: workgroup b runs on
// XCD b % 8, and a run (the pieces of the same rows) stays on one, whose cache
// then holds whole lines where a piece's codes end inside a 128-byte line.
// What is left behind the last eight runs is taken in order.
__device__ __forceinline__ uint32_t in_runs(uint32_t b, uint32_t blocks, uint32_t run) {
  const uint32_t runs = blocks / run & ~7u, at = b >> 3;
  return b < runs * run ? ((at / run) * 8 + (b & 7)) * run + at % run : b;
}

// Rows: a workgroup takes 4 RW rows x 4 blocks; wave w rows RW w .. + RW - 1,
// its four lane rows the four blocks.  SWI: x holds g | u of 2 K columns and
// the value is silu(g) u.  Workgroups go along the columns first: the pieces
// of a row that are in flight together are neighbours in memory (32768 x 4096
// bf16: 98 us with the rows first, 73 us so; 66 us with streaming reads, which
// gathered rows, read again for every expert, do not get; 61 us with two rows
// per wave in place of eight: 6.7 TB/s).  Where K is no multiple of 128 codes'
// lines are shared by pieces, and a row's pieces go to one XCD (16384 x 6832:
// 79 us without, 65 us with; where K is one, gathered rows lose: 32768 rows of
// 4096 from 4096 tokens 49 us without, 57 us with).  Gathered rows are bound by
// the vector unit (80% busy at K = 2048): a token's maximum and codes are formed
// anew for each of its rows.
constexpr int kBlocks = 4;

template <typename T, bool SWI, bool GATHER>
__global__ __launch_bounds__(256) void fp8_rows_kernel(Fp8RowsArgs a) {
  constexpr int RW = kRowsPerWave, kRows = 4 * RW;
  __shared__ float scales[kBlocks][kRows];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int blk = lane >> 4;
  const int64_t nb = (a.K + 127) / 128;
  const uint32_t gx = (uint32_t)((nb + kBlocks - 1) / kBlocks), gy = gridDim.x / gx;
  const uint32_t item = in_runs(blockIdx.x, gridDim.x, a.K % 128 ? gx : 1);
  const int64_t b0 = (int64_t)(item % gx) * kBlocks;
  const int64_t col = (b0 + blk) * 128 + 8 * (lane & 15);
  int64_t end = a.M;
  if (a.offsets != nullptr) {
    const int64_t o = a.offsets[a.E];
    end = o < 0 ? 0 : (o < end ? o : end);
  }
  const T* x = static_cast<const T*>(a.x);
  const int64_t ld = SWI ? 2 * a.K : a.K;
  for (int64_t r0 = (int64_t)(item / gx) * kRows; r0 < end; r0 += (int64_t)gy * kRows) {
    Eight<T> v[RW], u[SWI ? RW : 1];
    int64_t src[RW];                                   // the rows' places in x, -1 = zeros
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      const int64_t r = r0 + RW * wave + i;
      src[i] = r < end && col < a.K ? r : -1;
      if (GATHER && src[i] >= 0) {
        src[i] = a.gather[r];
        if (src[i] >= a.T) src[i] = -1;                // an index out of range
      }
    }
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      v[i].zero();
      if (SWI) u[SWI ? i : 0].zero();
      if (src[i] >= 0) {
        v[i].template load<!GATHER>(x + src[i] * ld + col);
        if (SWI) u[SWI ? i : 0].template load<!GATHER>(x + src[i] * ld + a.K + col);
      }
    }
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      float f[8];
      v[i].to(f);
      if (SWI) {
        float w[8];
        u[SWI ? i : 0].to(w);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float ex = __builtin_amdgcn_exp2f(-f[q] * 1.4426950408889634f);
          f[q] = f[q] * __builtin_amdgcn_rcpf(1.0f + ex) * w[q];
        }
      }
      const float am = fmaxf(row_max(abs_max8(f)), kFloor);
      const int64_t r = r0 + RW * wave + i;
      const u32x2 c = encode8(f, kTop / am);
      if (r < end && col < a.K)
        *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(a.codes) + r * a.K + col) = c;
      if ((lane & 15) == 0) scales[blk][RW * wave + i] = am / kTop;
    }
    __syncthreads();
    if (threadIdx.x < kBlocks * kRows) {
      const int b = threadIdx.x / kRows, r = threadIdx.x % kRows;
      if (b0 + b < nb && r0 + r < end) a.scales[(b0 + b) * a.M + r0 + r] = scales[b][r];
    }
    __syncthreads();
  }
}

// Weights: a workgroup takes one 128 x 128 block, 16 lanes per row, eight rows
// per lane, and finds the block's maximum through LDS; a row of blocks goes to
// one XCD (fp32, 20 x 1808 x 6832: 358 us without, 269 us with, 4.6 TB/s;
// 32 x 4096 x 2048: 251 and 234 us).
template <typename T>
__global__ __launch_bounds__(256) void fp8_weights_kernel(const T* __restrict__ w,
                                                          uint8_t* __restrict__ codes,
                                                          float* __restrict__ scales, int64_t N,
                                                          int64_t K) {
  __shared__ float part[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t nk = (K + 127) / 128, nn = (N + 127) / 128;
  const uint32_t item = in_runs(blockIdx.x, gridDim.x, (uint32_t)nk);
  const int64_t kb = item % nk, en = item / nk;
  const int64_t e = en / nn, n0 = (en - e * nn) * 128;
  const int64_t col = kb * 128 + 8 * (lane & 15);
  Eight<T> v[8];
  float am = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t n = n0 + 16 * i + 4 * wave + (lane >> 4);
    v[i].zero();
    if (n < N && col < K) v[i].template load<true>(w + (e * N + n) * K + col);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float f[8];
    v[i].to(f);
    am = fmaxf(am, abs_max8(f));
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) am = fmaxf(am, __shfl_xor(am, d, 64));
  if (lane == 0) part[wave] = am;
  __syncthreads();
  am = fmaxf(fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3])), kFloor);
  const float inv = kTop / am;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t n = n0 + 16 * i + 4 * wave + (lane >> 4);
    float f[8];
    v[i].to(f);
    if (n < N && col < K) *reinterpret_cast<u32x2*>(codes + (e * N + n) * K + col) = encode8(f, inv);
  }
  if (threadIdx.x == 0) scales[en * nk + kb] = am / kTop;
}

}  // namespace

int launch_fp8_rows(const Fp8RowsArgs& a, bool fp32, bool swiglu, hipStream_t s) {
  const int64_t gx = ((a.K + 127) / 128 + kBlocks - 1) / kBlocks;
  int64_t gy = (a.M + 4 * kRowsPerWave - 1) / (4 * kRowsPerWave);
  const int64_t most = kMaxBlocks256 / gx;              // grid-stride beyond
  if (gy > most) gy = most;
  const dim3 g((unsigned)(gx * gy)), b(256);
  const bool gather = a.gather != nullptr;
  if (swiglu) hipLaunchKernelGGL((fp8_rows_kernel<uint16_t, true, false>), g, b, 0, s, a);
  else if (fp32 && gather) hipLaunchKernelGGL((fp8_rows_kernel<float, false, true>), g, b, 0, s, a);
  else if (fp32) hipLaunchKernelGGL((fp8_rows_kernel<float, false, false>), g, b, 0, s, a);
  else if (gather) hipLaunchKernelGGL((fp8_rows_kernel<uint16_t, false, true>), g, b, 0, s, a);
  else hipLaunchKernelGGL((fp8_rows_kernel<uint16_t, false, false>), g, b, 0, s, a);
  return (int)hipGetLastError();
}

int launch_fp8_weights(const void* w, bool fp32, uint8_t* codes, float* scales, int64_t E, int64_t N,
                       int64_t K, hipStream_t s) {
  const int64_t blocks = E * ((N + 127) / 128) * ((K + 127) / 128);
  const dim3 g((unsigned)blocks), b(256);
  if (fp32)
    hipLaunchKernelGGL((fp8_weights_kernel<float>), g, b, 0, s, static_cast<const float*>(w), codes,
                       scales, N, K);
  else
    hipLaunchKernelGGL((fp8_weights_kernel<uint16_t>), g, b, 0, s, static_cast<const uint16_t*>(w),
                       codes, scales, N, K);
  return (int)hipGetLastError();
}

}  // namespace mg
