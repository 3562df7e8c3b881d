// The router of a mixture-of-experts layer, from its logits to the row order
// that the grouped products and the token combine read, with the statistics of
// its balance, and the gradient of all of it.  For token t with logits l_t
// (NaN counts as -inf, +inf as the largest finite value; an expert at -inf is
// never chosen):
//   p_te = exp(l_te - lse_t),  lse_t = log sum_e exp(l_te)
//   experts[t, j]: the k largest logits in descending order, ties to the lower
//     index; weights[t, j] = p of the chosen, or that over their sum
//   counts_e = number of (t, j) with experts[t, j] = e,  prob_sum_e = sum_t p_te
//   n = number of tokens that count (unmasked, with a logit above -inf)
//   balance = E sum_e (counts_e / sum counts) (prob_sum_e / n)
//   z = sum_t lse_t^2 / n
// and the stable order of the rows by (expert, token).  Gradient, counts and n
// held fixed, with upstream gradients dw, b (of balance) and c (of z):
//   dl_te = p_te (g_e - sum_f p_tf g_f + 2 c lse_t / n),  g_e = b E counts_e / (n sum counts)
//           + the gate's part:  normalised  w_j (dw_j - sum_i w_i dw_i) at the chosen
//                               plain       w_j dw_j at the chosen - p_te sum_i w_i dw_i
//
// A token is held by L lanes, V logits each, one read of the logits per pass.
// L = 16 up to 256 experts: every reduction is then four rotations of a lane
// row, and one instruction serves four tokens of a wave.  The choice of up to
// KL = 8 or 16 experts sorts: a lane's logits become 64-bit floats whose low
// mantissa bits, free after the conversion from 32 bits, hold the expert, so
// that one comparison orders by logit and then by index and the maximum and
// minimum instructions exchange two entries; every lane sorts its own, and
// four rotations each merge two descending lists into the upper half (k rounds
// of a maximum each took 44 us of T = 65536, E = 256, k = 8, this takes
// 30 us; 32-bit keys, which do not hold fp32 logits whole, took no less).
// More than 16 experts are taken in rounds.
//
// The order is a counting sort in three launches: the token pass writes each
// workgroup's counts, probability sums, lse^2 sum and n; a scan over the
// workgroups turns the counts into bases; the placing pass ranks its own
// workgroup's entries in order.  All of it is integer arithmetic or sums in a
// fixed order: results are bitwise reproducible.  Up to kOneTokens tokens one
// workgroup does all three in one launch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "mgemm_launch.h"

namespace mg {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kNT = 1024;             // threads of the token and placing passes
constexpr int kSmallNT = 256;         // of the one-launch form for few tokens
constexpr int kMaxGroups = 256;       // workgroups of the token pass
constexpr int kOneTokens = 256;       // tokens that one workgroup takes alone
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float neg_inf() { return -__builtin_huge_valf(); }

// A lane-row rotation (every lane has a source, so no old value is needed).
template <int CTRL>
__device__ __forceinline__ int dpp(int x) {
  return __builtin_amdgcn_mov_dpp(x, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __builtin_bit_cast(float, dpp<CTRL>(__builtin_bit_cast(int, x)));
}
// Reductions over the L lanes (16 or 64) of a token; every lane gets the result.
template <int L, typename T, typename F>
__device__ __forceinline__ T reduce(T x, F f) {
  x = f(x, dpp<0x128>(x));            // rotations of the 16-lane row by 8, 4, 2, 1
  x = f(x, dpp<0x124>(x));
  x = f(x, dpp<0x122>(x));
  x = f(x, dpp<0x121>(x));
  if (L == 64) {
    x = f(x, __shfl_xor(x, 16, 64));
    x = f(x, __shfl_xor(x, 32, 64));
  }
  return x;
}
template <int L>
__device__ __forceinline__ float max_of(float x) {
  return reduce<L>(x, [](float a, float b) { return fmaxf(a, b); });
}
template <int L>
__device__ __forceinline__ float sum_of(float x) {
  return reduce<L>(x, [](float a, float b) { return a + b; });
}
template <int L>
__device__ __forceinline__ int min_of(int x) {
  return reduce<L>(x, [](int a, int b) { return min(a, b); });
}

// The experts of a lane: value v is expert (v / C) C L + sub C + v % C, so that
// the L lanes' loads of C values (16 bytes) are contiguous.
template <typename T, int L, int V>
struct Lanes {
  static constexpr int kVec = 16 / (int)sizeof(T);
  static constexpr int C = V < kVec ? V : kVec;
  static __device__ __forceinline__ int expert(int sub, int v) { return (v / C) * C * L + sub * C + v % C; }
  static __device__ __forceinline__ float value(float x) { return x; }
  static __device__ __forceinline__ float value(uint16_t x) {
    return __builtin_bit_cast(float, (uint32_t)x << 16);
  }
  // A token's logits; `vec`: E a multiple of C and the rows aligned to C values.
  static __device__ __forceinline__ void load(const T* row, int E, int sub, bool on, bool vec,
                                              float (&x)[V]) {
#pragma unroll
    for (int b = 0; b < V / C; ++b) {
      T tmp[C];
      const int e0 = b * C * L + sub * C;
      if (vec) {
        if (on && e0 < E) {
          __builtin_memcpy(tmp, __builtin_assume_aligned(row + e0, C * sizeof(T)), C * sizeof(T));
#pragma unroll
          for (int c = 0; c < C; ++c) x[b * C + c] = value(tmp[c]);
        } else {
#pragma unroll
          for (int c = 0; c < C; ++c) x[b * C + c] = neg_inf();
        }
      } else {
#pragma unroll
        for (int c = 0; c < C; ++c)
          x[b * C + c] = on && e0 + c < E ? value(row[e0 + c]) : neg_inf();
      }
    }
    // NaN: never chosen, no probability; +inf: the largest finite value
#pragma unroll
    for (int v = 0; v < V; ++v) {
      x[v] = x[v] != x[v] ? neg_inf() : fminf(x[v], 3.40282347e38f);
    }
  }
};

// Workspace of `groups` workgroups: counts / bases int32 [groups][E], prob_sum
// fp32 [groups][E], lse^2 sums fp32 [groups], tokens int32 [groups], total of
// the lse^2 sums (one float).
struct Work {
  int32_t* counts;
  float* prob;
  float* z;
  int32_t* n;
  float* ztotal;
  __device__ __host__ __forceinline__ Work(void* p, int groups, int E) {
    counts = static_cast<int32_t*>(p);
    prob = reinterpret_cast<float*>(counts + (int64_t)groups * E);
    z = prob + (int64_t)groups * E;
    n = reinterpret_cast<int32_t*>(z + groups);
    ztotal = reinterpret_cast<float*>(n + groups);
  }
};

// Block-wide exclusive prefix of one int per thread (scratch: NT / 64 ints).
template <int NT>
__device__ __forceinline__ int block_prefix(int x, int* scratch, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int incl = x;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(incl, d, 64);
    if (lane >= d) incl += y;
  }
  __syncthreads();
  if (lane == 63) scratch[wave] = incl;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < NT / 64; ++w) {
    before += w < wave ? scratch[w] : 0;
    all += scratch[w];
  }
  *total = all;
  return before + incl - x;
}

// ---------------------------------------------------------------- token pass --

// 64-bit maximum and minimum as single instructions (no operand is a NaN).
__device__ __forceinline__ double max64(double a, double b) {
  double r;
  asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
__device__ __forceinline__ double min64(double a, double b) {
  double r;
  asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
__device__ __forceinline__ void exchange(double& a, double& b) {   // a >= b afterwards
  const double hi = max64(a, b);
  b = min64(a, b);
  a = hi;
}

// A logit and its expert as one key: keys order by descending logit, then
// ascending expert.  An excluded logit (-inf) has the lowest key.
constexpr double kNoKey = -1.7976931348623157e308;
__device__ __forceinline__ double key_of(float x, int e) {
  x += 0.0f;                                           // -0 is 0
  const uint64_t d = __builtin_bit_cast(uint64_t, max64((double)x, kNoKey));
  const uint32_t code = (uint32_t)e ^ (__builtin_bit_cast(int, x) < 0 ? 0u : 1023u);
  return __builtin_bit_cast(double, d | code);
}
__device__ __forceinline__ bool has_key(double k) { return k > -1e300; }
__device__ __forceinline__ float key_logit(double k) {
  return (float)__builtin_bit_cast(double, __builtin_bit_cast(uint64_t, k) & ~uint64_t(0x1FFFFFFF));
}
__device__ __forceinline__ int key_expert(double k) {
  return (int)((__builtin_bit_cast(uint64_t, k) & 1023u) ^ (k < 0.0 ? 0u : 1023u));
}
static_assert(kMaxExperts <= 1024, "an expert's ten bits in a key");

// Bitonic sequence of N (a power of two) to descending order.
template <int N>
__device__ __forceinline__ void bitonic_sort(double* v) {
#pragma unroll
  for (int d = N / 2; d >= 1; d /= 2)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((i & d) == 0) exchange(v[i], v[i + d]);
}
// Any N values to descending order: Batcher's odd-even merge sort (19
// exchanges of 8 values, a bitonic sort has 24).
template <int N, int STEP = 1>
__device__ __forceinline__ void odd_even_merge(double* v) {   // two sorted halves of N entries, STEP apart
  if constexpr (N == 2) {
    exchange(v[0], v[STEP]);
  } else {
    odd_even_merge<N / 2, 2 * STEP>(v);
    odd_even_merge<N / 2, 2 * STEP>(v + STEP);
#pragma unroll
    for (int i = 1; i + 1 < N; i += 2) exchange(v[i * STEP], v[(i + 1) * STEP]);
  }
}
template <int N>
__device__ __forceinline__ void sort_down(double* v) {
  if constexpr (N > 1) {
    sort_down<N / 2>(v);
    sort_down<N / 2>(v + N / 2);
    odd_even_merge<N>(v);
  }
}
// The N largest of two descending lists of N, descending.
template <int N>
__device__ __forceinline__ void merge_top(double* a, const double* b) {
#pragma unroll
  for (int i = 0; i < N; ++i) a[i] = max64(a[i], b[N - 1 - i]);
  bitonic_sort<N>(a);
}

template <int CTRL>
__device__ __forceinline__ double dpp64(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)dpp<CTRL>((int)(uint32_t)u), hi = (uint32_t)dpp<CTRL>((int)(uint32_t)(u >> 32));
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
template <int N, int CTRL>
__device__ __forceinline__ void merge_rotated(double* a) {
  double b[N];
#pragma unroll
  for (int i = 0; i < N; ++i) b[i] = dpp64<CTRL>(a[i]);
  merge_top<N>(a, b);
}

// The KL largest of a token's keys (V of this lane's), descending, in every lane.
template <int L, int V, int KL>
__device__ __forceinline__ void top_keys(const double (&key)[V], double (&top)[KL]) {
  constexpr int C = V < KL ? V : KL;
#pragma unroll
  for (int i = 0; i < KL; ++i) top[i] = i < C ? key[i] : kNoKey;
  sort_down<C>(top);
#pragma unroll
  for (int c = 1; c < V / C; ++c) {
    double other[KL];
#pragma unroll
    for (int i = 0; i < KL; ++i) other[i] = i < C ? key[c * C + i] : kNoKey;
    sort_down<C>(other);
    merge_top<KL>(top, other);
  }
  merge_rotated<KL, 0x128>(top);       // rotations of the 16-lane row by 8, 4, 2, 1
  merge_rotated<KL, 0x124>(top);
  merge_rotated<KL, 0x122>(top);
  merge_rotated<KL, 0x121>(top);
  if (L == 64) {
#pragma unroll
    for (int d = 16; d <= 32; d *= 2) {
      double other[KL];
#pragma unroll
      for (int i = 0; i < KL; ++i) other[i] = __shfl_xor(top[i], d, 64);
      merge_top<KL>(top, other);
    }
  }
}

// Gate of the tokens [t0, t1): weights, experts, lse; and the workgroup's
// counts (LDS hist [E]), probability sums (LDS prob [NT / 64][E], one row per
// wave), lse^2 sum and token count (returned in every thread).
template <typename T, int L, int V, int KL, int NT>
__device__ void gate_tokens(const RouteArgs& a, int64_t t0, int64_t t1, int* hist, float* prob,
                            float* chosen_val, int* chosen_idx, float* zsum, int* ntok) {
  using LN = Lanes<T, L, V>;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = lane % L;
  constexpr int kPerWave = 64 / L, kTokens = NT / L;
  const bool vec = a.E % LN::C == 0 &&
                   (reinterpret_cast<uintptr_t>(a.logits) & (LN::C * sizeof(T) - 1)) == 0;
  for (int e = threadIdx.x; e < a.E; e += NT) hist[e] = 0;
  __syncthreads();
  float ps[V];
#pragma unroll
  for (int v = 0; v < V; ++v) ps[v] = 0.f;
  float z = 0.f;
  int n = 0;
  for (int64_t tb = t0; tb < t1; tb += kTokens) {
    const int64_t t = tb + wave * kPerWave + lane / L;
    const bool on = t < t1 && (a.mask == nullptr || a.mask[t < t1 ? t : t0] != 0);
    float x[V];
    LN::load(static_cast<const T*>(a.logits) + (t < t1 ? t : t0) * a.E, a.E, sub, on, vec, x);
    double best[KL];
    float top = neg_inf();
    if (KL > 1) {
      double key[V];
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = key_of(x[v], LN::expert(sub, v));
      top_keys<L, V, KL>(key, best);
      if (has_key(best[0])) top = key_logit(best[0]);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) top = fmaxf(top, x[v]);
      top = max_of<L>(top);
    }
    const bool live = top > neg_inf();
    const float base = live ? top : 0.f;
    float s = 0.f, p[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      p[v] = __builtin_amdgcn_exp2f((x[v] - base) * kLog2e);
      s += p[v];
    }
    s = sum_of<L>(s);
    const float inv = live ? 1.0f / s : 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) ps[v] = __builtin_fmaf(p[v], inv, ps[v]);
    const float lse = live ? top + logf(s) : 0.f;
    if (live && sub == 0) {
      z = __builtin_fmaf(lse, lse, z);
      ++n;
    }
    if (KL > 1) {
      // lane j of the token writes its j-th choice
      double mine = kNoKey;
#pragma unroll
      for (int j = 0; j < KL; ++j) mine = sub == j ? best[j] : mine;
      const bool got = sub < a.k && has_key(mine);
      const float ex = got ? __builtin_amdgcn_exp2f((key_logit(mine) - base) * kLog2e) : 0.f;
      const float csum = sum_of<L>(ex);
      if (t < t1 && sub < a.k) {
        const int e = got ? key_expert(mine) : -1;
        a.weights[t * a.k + sub] = ex * (a.normalize ? (live ? 1.0f / csum : 0.f) : inv);
        a.experts[t * a.k + sub] = e;
        if (got) atomicAdd(&hist[e], 1);
      }
      if (t < t1 && sub == 0) a.lse[t] = lse;
      continue;
    }
    // k rounds: the best of the lanes' best, the lowest expert that has it
    const int slot0 = (wave * kPerWave + lane / L) * a.k;      // this token's choices in LDS
    float csum = 0.f;
    for (int j = 0; j < a.k; ++j) {
      float lb = neg_inf();
      int le = 0x7FFFFFFF;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (x[v] > lb) {
          lb = x[v];
          le = LN::expert(sub, v);
        }
      const float m = max_of<L>(lb);
      const int win = min_of<L>(lb == m && m > neg_inf() ? le : 0x7FFFFFFF);
      const float ex = __builtin_amdgcn_exp2f((m - base) * kLog2e);
      csum += m > neg_inf() ? ex : 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (LN::expert(sub, v) == win) x[v] = neg_inf();
      if (sub == 0) {
        chosen_val[slot0 + j] = m > neg_inf() ? ex : 0.f;
        chosen_idx[slot0 + j] = m > neg_inf() ? win : -1;
      }
    }
    __builtin_amdgcn_wave_barrier();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (t < t1) {
      const float scale = a.normalize ? (live ? 1.0f / csum : 0.f) : inv;
      for (int j = sub; j < a.k; j += L) {
        const int e = chosen_idx[slot0 + j];
        a.weights[t * a.k + j] = chosen_val[slot0 + j] * scale;
        a.experts[t * a.k + j] = e;
        if (e >= 0) atomicAdd(&hist[e], 1);
      }
      if (sub == 0) a.lse[t] = lse;
    }
    __builtin_amdgcn_wave_barrier();
  }
  // probability sums: the wave's tokens by lane exchange, one row per wave
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (L == 16) {
      ps[v] += __shfl_xor(ps[v], 16, 64);
      ps[v] += __shfl_xor(ps[v], 32, 64);
    }
    const int e = LN::expert(sub, v);
    if (lane < L && e < a.E) prob[wave * a.E + e] = ps[v];
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    z += __shfl_xor(z, d, 64);
    n += __shfl_xor(n, d, 64);
  }
  __shared__ float zw[NT / 64];
  __shared__ int nw[NT / 64];
  if (lane == 0) {
    zw[wave] = z;
    nw[wave] = n;
  }
  __syncthreads();
  z = 0.f;
  n = 0;
  for (int w = 0; w < NT / 64; ++w) {
    z += zw[w];
    n += nw[w];
  }
  *zsum = z;
  *ntok = n;
}

// ----------------------------------------------------------------- placing --

// Offsets of the local experts (LDS start [E], the first row of each local
// expert) from the counts; thread e holds counts[e] (E <= NT).
template <int NT>
__device__ int local_starts(const RouteArgs& a, int count, int* start, int* scratch) {
  const int e = threadIdx.x, le = e - a.first;
  const bool mine = e < a.E && le >= 0 && le < a.local;
  int rows;
  const int at = block_prefix<NT>(mine ? count : 0, scratch, &rows);
  if (e < a.E) start[e] = mine ? at : 0;
  if (blockIdx.x == 0) {
    if (mine) a.offsets[le] = at;
    if (e == 0) a.offsets[a.local] = rows;
  }
  __syncthreads();
  return rows;
}

// Rank the entries (token, slot) [i0, i1) of this workgroup in order and write
// their rows.  start[e] (LDS): the next row of expert e for this workgroup.
// Each wave counts its own part first (cnt [NT / 64][E]); of a part of up to
// 64 kHeld entries the experts stay in registers in between.
constexpr int kHeld = 4;
template <int NT>
struct Part {                            // a wave's entries [w0, w1)
  int64_t w0, w1;
  bool held;
  int mine[kHeld];
  __device__ __forceinline__ int local(const RouteArgs& a, int64_t i) const {
    const int e = i < w1 ? a.experts[i] : -1;
    return e >= a.first && e < a.first + a.local ? e : -1;
  }
  __device__ __forceinline__ void load(const RouteArgs& a, int64_t i0, int64_t i1) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t len = ((i1 - i0 + NT / 64 - 1) / (NT / 64) + 63) / 64 * 64;
    w0 = i0 + wave * len;
    w1 = w0 + len < i1 ? w0 + len : i1;
    held = len <= 64 * kHeld;
#pragma unroll
    for (int h = 0; h < kHeld; ++h) mine[h] = held ? local(a, w0 + 64 * h + lane) : -1;
  }
};

template <int NT>
__device__ void place(const RouteArgs& a, const Part<NT>& part, int64_t i0, int64_t i1, int rows,
                      const int* start, int* cnt) {
  constexpr int kWaves = NT / 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t w0 = part.w0, w1 = part.w1;
  const bool held = part.held;
  for (int i = threadIdx.x; i < kWaves * a.E; i += NT) cnt[i] = 0;
  __syncthreads();
  int* my = cnt + wave * a.E;
  if (held) {
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
      if (part.mine[h] >= 0) atomicAdd(&my[part.mine[h]], 1);
  } else {
    for (int64_t i = w0 + lane; i < w1; i += 64) {
      const int e = part.local(a, i);
      if (e >= 0) atomicAdd(&my[e], 1);
    }
  }
  __syncthreads();
  // counts of the waves before, on top of the workgroup's start
  for (int e = threadIdx.x; e < a.E; e += NT) {
    int run = start[e], c[kWaves];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) c[w] = cnt[w * a.E + e];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      cnt[w * a.E + e] = run;
      run += c[w];
    }
  }
  __syncthreads();
  int bits = 0;
  while ((1 << bits) < a.E) ++bits;
  auto rank = [&](int64_t b, int e) {
    // lanes with the same expert, by the bits of its index
    uint64_t same = __ballot(e >= 0);
    for (int q = 0; q < bits; ++q) {
      const uint64_t bal = __ballot((e >> q) & 1);
      same &= (e >> q) & 1 ? bal : ~bal;
    }
    int row = -1;
    const uint64_t below = same & ((uint64_t(1) << lane) - 1);
    if (e >= 0) row = my[e] + __popcll(below);
    __builtin_amdgcn_wave_barrier();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (e >= 0 && below == 0) my[e] = row + __popcll(same);
    __builtin_amdgcn_wave_barrier();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    const int64_t i = b + lane;
    if (i < w1) {
      a.token_rows[i] = row;
      if (row >= 0) a.gather[row] = (int32_t)((uint32_t)i / (uint32_t)a.k);
    }
  };
  if (held) {
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
      if (w0 + 64 * h < w1) rank(w0 + 64 * h, part.mine[h]);
  } else {
    for (int64_t b = w0; b < w1; b += 64) rank(b, part.local(a, b + lane));
  }
  for (int64_t i = i0 + threadIdx.x; i < i1; i += NT)
    if (i >= rows) a.gather[i] = -1;                   // behind the last row
}

// Losses from the totals; thread e holds counts[e] and prob_sum[e].
template <int NT>
__device__ void losses(const RouteArgs& a, int count, float prob, float ztotal, int n) {
  __shared__ double red[2][NT / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double cp = (double)count * (double)prob, c = (double)count;
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    cp += __shfl_xor(cp, d, 64);
    c += __shfl_xor(c, d, 64);
  }
  if (lane == 0) {
    red[0][wave] = cp;
    red[1][wave] = c;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    cp = c = 0.0;
    for (int w = 0; w < NT / 64; ++w) {
      cp += red[0][w];
      c += red[1][w];
    }
    a.loss[0] = n > 0 ? (float)(a.E * cp / (c * n)) : 0.f;
    a.loss[1] = n > 0 ? ztotal / (float)n : 0.f;
  }
}

// Dynamic LDS of a token pass: hist [E], start [E], scratch [NT / 64], prob
// [NT / 64][E] (later cnt) and, for choices in rounds, values and experts
// [NT / L][k].
template <int L, int KL, int NT>
struct Lds {
  int *hist, *start, *scratch, *chosen_idx, *cnt;
  float *prob, *chosen_val;
  __device__ __forceinline__ Lds(char* p, int E, int k) {
    hist = reinterpret_cast<int*>(p);
    start = hist + E;
    scratch = start + E;
    prob = reinterpret_cast<float*>(scratch + NT / 64);
    cnt = reinterpret_cast<int*>(prob);
    chosen_val = prob + NT / 64 * E;
    chosen_idx = reinterpret_cast<int*>(chosen_val + (NT / L) * k);
  }
  static size_t bytes(int E, int k) {
    return 4 * ((size_t)(2 + NT / 64) * E + NT / 64 + (KL > 1 ? 0 : 2 * (size_t)(NT / L) * k));
  }
};

// ONE: the only workgroup, which finishes everything; else the first of three launches.
template <typename T, int L, int V, int KL, int NT, bool ONE>
__global__ __launch_bounds__(NT) void route_tokens_kernel(RouteArgs a) {
  extern __shared__ __attribute__((aligned(16))) char dyn[];
  const Lds<L, KL, NT> s(dyn, a.E, a.k);
  const int64_t t0 = (int64_t)blockIdx.x * a.per_group;
  const int64_t t1 = t0 + a.per_group < a.T ? t0 + a.per_group : a.T;
  float z;
  int n;
  gate_tokens<T, L, V, KL, NT>(a, t0, t1, s.hist, s.prob, s.chosen_val, s.chosen_idx, &z, &n);
  const int e = threadIdx.x;
  float prob = 0.f;
  int count = 0;
  if (e < a.E) {
    for (int w = 0; w < NT / 64; ++w) prob += s.prob[w * a.E + e];
    count = s.hist[e];
  }
  if (ONE) {
    if (e < a.E) {
      a.counts[e] = count;
      a.prob_sum[e] = prob;
    }
    if (e == 0) a.tokens[0] = n;
    const int rows = local_starts<NT>(a, count, s.start, s.scratch);
    losses<NT>(a, count, prob, z, n);
    // the experts written above are read by other waves of this workgroup
    __threadfence_block();
    __syncthreads();
    Part<NT> part;
    part.load(a, 0, a.T * a.k);
    place<NT>(a, part, 0, a.T * a.k, rows, s.start, s.cnt);
    return;
  }
  const Work w(a.workspace, gridDim.x, a.E);
  if (e < a.E) {
    w.counts[(int64_t)blockIdx.x * a.E + e] = count;
    w.prob[(int64_t)blockIdx.x * a.E + e] = prob;
  }
  if (e == 0) {
    w.z[blockIdx.x] = z;
    w.n[blockIdx.x] = n;
  }
}

// 64 experts per workgroup, a wave's lanes; the waves share the token pass's
// workgroups, at most kMaxGroups / kWaves each, held in registers.
__global__ __launch_bounds__(kNT) void route_scan_kernel(RouteArgs a, int groups) {
  constexpr int kWaves = kNT / 64;
  __shared__ int cs[kWaves][64];
  __shared__ float ps[kWaves][64];
  constexpr int kPer = kMaxGroups / kWaves;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const Work w(a.workspace, groups, a.E);
  const int e = blockIdx.x * 64 + lane;
  int c[kPer];
  float p[kPer];
  int csum = 0;
  float psum = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int g = wave * kPer + i;
    const bool on = g < groups && e < a.E;
    c[i] = on ? w.counts[(int64_t)g * a.E + e] : 0;
    p[i] = on ? w.prob[(int64_t)g * a.E + e] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    csum += c[i];
    psum += p[i];
  }
  cs[wave][lane] = csum;
  ps[wave][lane] = psum;
  __syncthreads();
  int run = 0;
  for (int v = 0; v < wave; ++v) run += cs[v][lane];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int g = wave * kPer + i;
    if (g < groups && e < a.E) w.counts[(int64_t)g * a.E + e] = run;
    run += c[i];
  }
  if (wave == kWaves - 1 && e < a.E) {
    float total = 0.f;
    for (int v = 0; v < kWaves; ++v) total += ps[v][lane];
    a.counts[e] = run;
    a.prob_sum[e] = total;
  }
  if (blockIdx.x == 0 && wave == 0) {
    float z = 0.f;
    int n = 0;
    for (int g = lane; g < groups; g += 64) {
      z += w.z[g];
      n += w.n[g];
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
      z += __shfl_xor(z, d, 64);
      n += __shfl_xor(n, d, 64);
    }
    if (lane == 0) {
      *w.ztotal = z;
      a.tokens[0] = n;
    }
  }
}

__global__ __launch_bounds__(kNT) void route_place_kernel(RouteArgs a) {
  extern __shared__ __attribute__((aligned(16))) char dyn[];
  int* start = reinterpret_cast<int*>(dyn);
  int* scratch = start + a.E;
  int* cnt = scratch + kNT / 64;
  const Work w(a.workspace, gridDim.x, a.E);
  const int e = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * a.per_group;
  const int64_t t1 = t0 + a.per_group < a.T ? t0 + a.per_group : a.T;
  // what the steps below wait for, loaded together
  const int count = e < a.E ? a.counts[e] : 0;
  const int base = e < a.E ? w.counts[(int64_t)blockIdx.x * a.E + e] : 0;
  Part<kNT> part;
  part.load(a, t0 * a.k, t1 * a.k);
  const int rows = local_starts<kNT>(a, count, start, scratch);
  if (blockIdx.x == 0) losses<kNT>(a, count, e < a.E ? a.prob_sum[e] : 0.f, *w.ztotal, a.tokens[0]);
  if (e < a.E) start[e] += base;
  __syncthreads();
  place<kNT>(a, part, t0 * a.k, t1 * a.k, rows, start, cnt);
}

// ----------------------------------------------------------------- gradient --

constexpr int kBT = 256;              // threads of the gradient kernel

template <typename T, int L, int V>
__global__ __launch_bounds__(kBT) void route_bwd_kernel(RouteBwdArgs a) {
  using LN = Lanes<T, L, V>;
  extern __shared__ __attribute__((aligned(16))) float gate[];       // [kBT / L][E]
  __shared__ long long csum[kBT / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = threadIdx.x % L;
  float* mine = gate + (threadIdx.x / L) * a.E;
  const bool losses = a.dloss != nullptr;
  float g[V], zc = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) g[v] = 0.f;
  if (losses) {
    long long c = 0;                     // (sums over ranks may pass 31 bits together)
    for (int e = threadIdx.x; e < a.E; e += kBT) c += a.counts[e];
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) c += __shfl_xor(c, d, 64);
    if (lane == 0) csum[wave] = c;
    __syncthreads();
    c = 0;
    for (int w = 0; w < kBT / 64; ++w) c += csum[w];
    const float n = (float)a.tokens[0];
    const float b = c > 0 && n > 0.f ? a.dloss[0] * (float)a.E / ((float)c * n) : 0.f;
    zc = n > 0.f ? 2.0f * a.dloss[1] / n : 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = LN::expert(sub, v);
      g[v] = e < a.E ? b * (float)a.counts[e] : 0.f;
    }
  }
  const bool vec = a.E % LN::C == 0 &&
                   ((reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.dlogits)) &
                    (LN::C * sizeof(T) - 1)) == 0;
  constexpr int kTokens = kBT / L;
  for (int64_t tb = (int64_t)blockIdx.x * kTokens; tb < a.T; tb += (int64_t)gridDim.x * kTokens) {
    const int64_t t = tb + threadIdx.x / L;
    const bool in = t < a.T;
    const int64_t tt = in ? t : a.T - 1;
    const bool live = in && a.experts[tt * a.k] >= 0;
    float x[V], p[V];
    // everything the token needs is loaded before the first use: its choices
    // are the lanes' (further ones, where k > L, are loaded in place)
    LN::load(static_cast<const T*>(a.logits) + tt * a.E, a.E, sub, in, vec, x);
    const float lse = a.lse[tt];
    auto choice = [&](int j, int& e, float& w, float& d) {
      e = a.experts[tt * a.k + j];
      w = a.weights[tt * a.k + j];
      d = a.dweights[tt * a.k + j];
      if (!live || e >= a.E) e = -1;
    };
    int ce = -1;
    float cw = 0.f, cd = 0.f;
    if (a.dweights != nullptr && sub < a.k) choice(sub, ce, cw, cd);
    // the softmax anew, not exp(l - lse): where the logits are huge (all of
    // them the type's lowest value, say) lse has lost the log of the sum
    float best = neg_inf(), sum = 0.f, pg = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) best = fmaxf(best, x[v]);
    best = max_of<L>(best);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      p[v] = live ? __builtin_amdgcn_exp2f((x[v] - best) * kLog2e) : 0.f;
      sum += p[v];
    }
    sum = sum_of<L>(sum);
    const float inv = live && sum > 0.f ? 1.0f / sum : 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      p[v] *= inv;
      pg = __builtin_fmaf(p[v], g[v], pg);
    }
    pg = sum_of<L>(pg);
    float dot = 0.f;
    if (a.dweights != nullptr) {
      for (int e = sub; e < a.E; e += L) mine[e] = 0.f;
      if (ce >= 0) dot = cw * cd;
      for (int j = sub + L; j < a.k; j += L) {
        int e;
        float w, d;
        choice(j, e, w, d);
        if (e >= 0) dot = __builtin_fmaf(w, d, dot);
      }
      dot = sum_of<L>(dot);
      __builtin_amdgcn_wave_barrier();
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (ce >= 0) mine[ce] = cw * (a.normalize ? cd - dot : cd);
      for (int j = sub + L; j < a.k; j += L) {
        int e;
        float w, d;
        choice(j, e, w, d);
        if (e >= 0) mine[e] = w * (a.normalize ? d - dot : d);
      }
      __builtin_amdgcn_wave_barrier();
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
    // (the z term as (p lse) zc: lse is up to the largest number, zc may be above
    // one, and p is what keeps their product one)
    const float common = -pg - (a.normalize ? 0.f : dot);
    T* out = static_cast<T*>(a.dlogits) + tt * a.E;
#pragma unroll
    for (int b = 0; b < V / LN::C; ++b) {
      const int e0 = LN::expert(sub, b * LN::C);
      T tmp[LN::C];
#pragma unroll
      for (int c = 0; c < LN::C; ++c) {
        const int v = b * LN::C + c;
        float d = __builtin_fmaf(p[v] * lse, zc, p[v] * (g[v] + common));
        if (a.dweights != nullptr && e0 + c < a.E) d += mine[e0 + c];
        if constexpr (sizeof(T) == 4) tmp[c] = d;
        else tmp[c] = __builtin_bit_cast(uint16_t, (__bf16)d);
      }
      if (vec) {
        if (in && e0 < a.E)
          __builtin_memcpy(__builtin_assume_aligned(out + e0, LN::C * sizeof(T)), tmp, LN::C * sizeof(T));
      } else {
#pragma unroll
        for (int c = 0; c < LN::C; ++c)
          if (in && e0 + c < a.E) out[e0 + c] = tmp[c];
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

int groups_of(int64_t T) {
  if (T <= kOneTokens) return 1;
  const int64_t g = (T + 63) / 64;
  return (int)(g < kMaxGroups ? g : kMaxGroups);
}

template <typename T, int L, int V, int KL>
int launch_tokens(RouteArgs a, hipStream_t s) {
  int groups = groups_of(a.T);
  a.per_group = groups == 1 ? (a.T > 0 ? a.T : 1) : ((a.T + groups - 1) / groups + 63) / 64 * 64;
  if (groups == 1) {
    // few tokens: a quarter of the waves, which is what their barriers cost
    // (T = 16, E = 128, k = 8: 6.5 us against 12)
    if constexpr (L == 16) {
      if (a.T <= 64) {
        hipLaunchKernelGGL((route_tokens_kernel<T, L, V, KL, kSmallNT, true>), dim3(1),
                           dim3(kSmallNT), (Lds<L, KL, kSmallNT>::bytes(a.E, a.k)), s, a);
        return (int)hipGetLastError();
      }
    }
    hipLaunchKernelGGL((route_tokens_kernel<T, L, V, KL, kNT, true>), dim3(1), dim3(kNT),
                       (Lds<L, KL, kNT>::bytes(a.E, a.k)), s, a);
    return (int)hipGetLastError();
  }
  groups = (int)((a.T + a.per_group - 1) / a.per_group);
  hipLaunchKernelGGL((route_tokens_kernel<T, L, V, KL, kNT, false>), dim3(groups), dim3(kNT),
                     (Lds<L, KL, kNT>::bytes(a.E, a.k)), s, a);
  int err = (int)hipGetLastError();
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL(route_scan_kernel, dim3((a.E + 63) / 64), dim3(kNT), 0, s, a, groups);
  if ((err = (int)hipGetLastError()) != hipSuccess) return err;
  hipLaunchKernelGGL(route_place_kernel, dim3(groups), dim3(kNT),
                     4 * ((size_t)(1 + kNT / 64) * a.E + kNT / 64), s, a);
  return (int)hipGetLastError();
}

template <typename T, int L, int V>
int launch_bwd(const RouteBwdArgs& a, hipStream_t s) {
  constexpr int kTokens = kBT / L;
  int64_t blocks = (a.T + kTokens - 1) / kTokens;
  // grid-stride beyond five workgroups per compute unit: each reads the counts
  // first, and eight of them leave a last wave that is mostly empty (65536 x
  // 256: 33 us with 1024 to 1280, 39 with 1536, 41 with 2048)
  if (blocks > 1280) blocks = 1280;
  hipLaunchKernelGGL((route_bwd_kernel<T, L, V>), dim3((unsigned)blocks), dim3(kBT),
                     a.dweights != nullptr ? (size_t)4 * kTokens * a.E : 0, s, a);
  return (int)hipGetLastError();
}

// Lanes and logits per lane by the expert count.
template <typename T, typename F>
int by_experts(int E, F f) {
  if (E <= 64) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 4>{});
  if (E <= 128) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 8>{});
  if (E <= 256) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 16>{});
  if (E <= 512) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 8>{});
  return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 16>{});
}

}  // namespace

int64_t route_workspace_bytes(int64_t T, int32_t E) {
  const int64_t g = groups_of(T);
  return g == 1 ? 0 : 4 * (2 * g * E + 2 * g + 1);
}

namespace {
template <typename T>
int launch_route_of(const RouteArgs& a, hipStream_t s) {
  return by_experts<T>(a.E, [&](auto l, auto v) {
    constexpr int L = decltype(l)::value, V = decltype(v)::value;
    if (a.k <= 8) return launch_tokens<T, L, V, 8>(a, s);
    if (a.k <= 16) return launch_tokens<T, L, V, 16>(a, s);
    return launch_tokens<T, L, V, 1>(a, s);
  });
}
}  // namespace

int launch_route(const RouteArgs& a, bool bf16, hipStream_t s) {
  return bf16 ? launch_route_of<uint16_t>(a, s) : launch_route_of<float>(a, s);
}

int launch_route_bwd(const RouteBwdArgs& a, bool bf16, hipStream_t s) {
  if (bf16)
    return by_experts<uint16_t>(a.E, [&](auto l, auto v) {
      return launch_bwd<uint16_t, decltype(l)::value, decltype(v)::value>(a, s);
    });
  return by_experts<float>(a.E, [&](auto l, auto v) {
    return launch_bwd<float, decltype(l)::value, decltype(v)::value>(a, s);
  });
}

}  // namespace mg
