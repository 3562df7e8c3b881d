// Device-side pieces that the grouped GEMM kernels share: vector types, buffer
// descriptors and direct-to-LDS loads, and the M-grouped tile scheduler.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mgemm_launch.h"

namespace mg {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr uint32_t kOOB = 0x80000000u;   // offset bit past any buffer range

// 128-bit raw buffer descriptor: base, stride 0, range `bytes`.  Loads past
// the range return zero.  All inputs are wave-uniform.
__device__ __forceinline__ i32x4 make_rsrc(const void* base, uint32_t bytes) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  i32x4 r;
  r.x = (int32_t)__builtin_amdgcn_readfirstlane((uint32_t)b);
  r.y = (int32_t)(__builtin_amdgcn_readfirstlane((uint32_t)(b >> 32)) & 0xFFFFu);
  r.z = (int32_t)__builtin_amdgcn_readfirstlane(bytes);
  r.w = 0x00020000;
  return r;
}

// Direct-to-LDS 16-byte load: lane l's 16 bytes land at LDS byte address
// lds_addr + 16 l (lds_addr wave-uniform).  Issued as inline assembly so that
// the compiler does not serialise it against the LDS reads of other stages;
// completion is awaited explicitly with vmcnt before the stage's barrier.
__device__ __forceinline__ void dma16(const i32x4& rsrc, uint32_t lds_addr, uint32_t voff) {
  uint32_t save;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %1\n\t"
      "buffer_load_dwordx4 %2, %3, 0 offen lds\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(save)
      : "s"(lds_addr), "v"(voff), "s"(rsrc)
      : "memory");
}

// Direct-to-LDS 4-byte load: lane l's dword lands at lds_addr + 4 l.
__device__ __forceinline__ void dma4(const i32x4& rsrc, uint32_t lds_addr, uint32_t voff) {
  uint32_t save;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %1\n\t"
      "buffer_load_dword %2, %3, 0 offen lds\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(save)
      : "s"(lds_addr), "v"(voff), "s"(rsrc)
      : "memory");
}

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t lds_u32(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)(
      (const __attribute__((address_space(3))) void*)p);
}

// ------------------------------------------------------------- scheduler --

// Exclusive prefix sum over the block of per-thread values; returns the
// thread's exclusive prefix and writes the block total to *total.
template <int NT>
__device__ __forceinline__ int block_exclusive_scan(int x, int* scratch, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int incl = x;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    int y = __shfl_up(incl, d, 64);
    if (lane >= d) incl += y;
  }
  if (lane == 63) scratch[wave] = incl;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) {
    int s = scratch[w];
    before += (w < wave) ? s : 0;
    all += s;
  }
  *total = all;
  return before + incl - x;
}

struct Tile {
  int e;        // expert
  int q0;       // first Q index of the tile (global row for M-grouped, n for K-grouped)
  int q_end;    // one past the last valid Q index
  int p0;       // first P index
  int r_begin;  // reduction range [r_begin, r_end) of this work item
  int r_end;
  int split;    // K-grouped: -1 for a whole tile, else 2 x split-tile id + half
};

// Scheduler state kept in LDS / registers for the whole launch.
struct Sched {
  int* scan;    // [16] scan scratch
  int* pref;    // [E+1] M-grouped: exclusive prefix of M-tiles per expert
  int* offs;    // [E+1] copy of the offsets
  int* inv;     // [E]   K-grouped: rank (heaviest first) -> expert
  int* mine;    // [2E]  K-grouped: this workgroup's (rank | rho << 16, count) entries
  int* keys;    // [64]  K-grouped: balancing scratch
  int nmine;    // K-grouped: entries in `mine`
  int total;    // number of tiles
  int E, tilesP, tilesQ, red;
  int gm;       // M-grouped: M-tiles per raster group
  int bw;       // K-grouped: P-tiles per band
  int per;      // K-grouped: tiles per expert
  bool split;   // K-grouped: heavy tiles may be split in two token halves
  bool whole;   // K-grouped: each XCD takes whole experts (see kchunk_start)
  const ListDesc* list;   // descriptor list (E groups), else null
};

// Offsets are read clamped to [0, M] and made non-decreasing per expert, so
// that even offsets breaking the documented precondition cannot move any read
// or write outside the tensors (the results are then meaningless, not unsafe).
__device__ __forceinline__ int clamp_off(const int32_t* offsets, int i, int M) {
  const int o = offsets[i];
  return o < 0 ? 0 : (o > M ? M : o);
}

// M-grouped set-up: tiles are, for every expert, ceil(m_e / BQ) M-tiles times
// tilesP P-tiles; empty experts contribute none.
template <int NT, int BQ>
__device__ void setup_mgrouped(const int32_t* __restrict__ offsets, int E, int M, Sched& S) {
  constexpr int kPer = (kMaxExperts + NT - 1) / NT;
  const int e0 = threadIdx.x * kPer;
  int cnt[kPer];
  int mine = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = e0 + j;
    cnt[j] = 0;
    if (e < E) {
      const int lo = clamp_off(offsets, e, M);
      const int hi = max(lo, clamp_off(offsets, e + 1, M));
      S.offs[e] = lo;
      if (e == E - 1) S.offs[E] = hi;
      const int m = hi - lo;
      cnt[j] = m > 0 ? (m + BQ - 1) / BQ : 0;
      mine += cnt[j];
    }
  }
  int mtiles;
  int run = block_exclusive_scan<NT>(mine, S.scan, &mtiles);
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = e0 + j;
    if (e < E) S.pref[e] = run;
    run += cnt[j];
  }
  if (threadIdx.x == 0) S.pref[E] = mtiles;
  __syncthreads();
  S.total = mtiles * S.tilesP;
}

// M-grouped tile id L -> tile.  Ids run expert by expert; within an expert,
// in groups of gm M-tiles (the last group may be shorter), M-tile fastest,
// then P-tile.
template <int PSTEP, int BQ>
__device__ __forceinline__ void decode_mgrouped(int L, const Sched& S, Tile& t) {
  const int tilesP = S.tilesP;
  // the expert whose id range [pref[e] tilesP, pref[e+1] tilesP) holds L: the
  // largest e with pref[e] tilesP <= L (empty experts share their successor's
  // prefix)
  int lo = 0, hi = S.E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (S.pref[mid] * tilesP <= L) lo = mid; else hi = mid - 1;
  }
  const int e = lo;
  const int local = L - S.pref[e] * tilesP;
  const int mt = S.pref[e + 1] - S.pref[e];
  const int g = local / (S.gm * tilesP);
  const int rem = local - g * S.gm * tilesP;
  const int gh = min(S.gm, mt - g * S.gm);
  const int tp = rem / gh;
  const int m = g * S.gm + (rem - tp * gh);
  t.e = e;
  t.q0 = S.offs[e] + m * BQ;
  t.q_end = max(S.offs[e + 1], S.offs[e]);
  t.p0 = tp * PSTEP;
  t.r_begin = 0;
  t.r_end = S.red;
}

}  // namespace mg
