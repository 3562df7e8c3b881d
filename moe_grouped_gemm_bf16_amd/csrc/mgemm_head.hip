// Losses of the output head on gfx950: cross entropy over a vocabulary and
// distillation from a teacher's top logits, and their gradients, from the
// hidden rows x [T, D] and the head's weights w [V, D] without keeping the
// logits z[t, v] = x[t] . w[v].
//
// Both losses see z through lse[t] = log sum_v exp(c z[t, v]) (c = 1 / the
// temperature) and through a few entries per token, so both gradients are
//   dz[t, v] = a[t] p[t, v] - sum over the entries at v of their weights b q,
//   p = exp(c z - lse),   dx = dz w,   dw = dz^T x,
// three matrix products of 2 T D V operations backward (z again, since it was
// not kept) against one forward.  All run on one kernel, nt_kernel below, as
// C[q, p] = sum_r Q[q, r] P[p, r]:
//   logits (forward, backward)  P = w rows, Q = x rows, r = hidden column
//   input gradient              P = dz rows (tokens), Q = w columns, r = vocabulary
//   weight gradient             P = x columns, Q = dz columns (vocabulary), r = token
// The forward's epilogue turns a tile of logits into one (maximum, sum of
// exponentials) per token and 64 or 128 vocabulary entries; the backward's turns
// it into dz, in 16 bits, for a piece of the vocabulary at a time.  dz lies in
// panels of 64 vocabulary entries, [v / 64][token][64]: whether a product reads
// it along the vocabulary or along the tokens, it reads 128 contiguous bytes.
// Operands that are strided along r (w and x as the gradients read them, dz in
// the weight gradient) are staged as they lie and transposed by the LDS read.
//
// Tokens that do not count (no target, no teacher's entry) are left out before
// the products: rows[] lists the others, x is packed by it (not if all count).
// The number that count stays on the device.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "mgemm_launch.h"

namespace mg {
namespace {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) const bf16x8 lds_frag;

constexpr uint32_t kOOB = 0x80000000u;       // offset bit past any buffer range

// 128-bit raw buffer descriptor: loads past `bytes` return zero.
__device__ __forceinline__ i32x4 make_rsrc(const void* base, uint32_t bytes) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  i32x4 r;
  r.x = (int32_t)__builtin_amdgcn_readfirstlane((uint32_t)b);
  r.y = (int32_t)(__builtin_amdgcn_readfirstlane((uint32_t)(b >> 32)) & 0xFFFFu);
  r.z = (int32_t)__builtin_amdgcn_readfirstlane(bytes);
  r.w = 0x00020000;
  return r;
}

// Direct-to-LDS load: lane l's 16 bytes land at lds_addr + 16 l.  In assembly
// so that the compiler does not wait for it before other LDS reads; the waits
// are the stage loop's own.  The compiler writes m0, which holds the address, and
// knows nothing of the load: the wait state between them stands here.  (With m0
// saved and restored in the block instead the wait state took 1% to 2% more time:
// loss of 8192 x 131072 x 4096 6.17 -> 6.31 ms; so 6.18.)
__device__ __forceinline__ void dma16(const i32x4& rsrc, uint32_t lds_addr, uint32_t voff) {
  asm volatile(
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, 0 offen lds"
      :
      : "{m0}"(lds_addr), "v"(voff), "s"(rsrc)
      : "memory");
}

template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// One operand of a product, rows of `stride` bytes, each in blocks of 64 values
// `step` bytes apart.  Its rows are the product's rows and the values its
// reduction steps, or (strided, below) the other way round.
struct Operand {
  const void* base;
  uint32_t stride;
  uint32_t step;
};

// A token that counts, as the backward's epilogue takes it.
struct Token {
  float lse;            // lse / c, as the logits
  float a;              // weight of the probabilities
  float b;              // weight of the entries
  int32_t target;       // vocabulary entry of w, -1 for none or several (written apart)
};

// kDzPair: dz as a sum of two 16-bit values, the second in rows of its own, for
// few tokens (see kPairs).
enum { kStats = 0, kDz = 1, kDx = 2, kDw = 3, kDzPair = 4 };
constexpr bool is_dz(int epi) { return epi == kDz || epi == kDzPair; }

// How a product's tiles are cut, by the number of tokens that count.
struct Plan {
  int32_t large;        // tiles along P of 256 x 256, the others of 256 x 128
  int32_t splits;       // parts of the reduction (gradients)
  int32_t rows;         // rows of P that a small tile takes: 256, or fewer (logits)
};

struct NtArgs {
  Operand P, Q;
  const void* x_all;        // what is taken for x when all tokens count
  const int32_t* n;         // device: tokens that count, NULL: all
  const Plan* plan_at;      // device, NULL: `plan`
  Plan plan;
  int32_t np, nq, K;        // rows of P and of Q and reduction steps; those that are
                            // tokens hold T
  int32_t tokens;           // T
  int32_t gq;               // tiles along Q that run beside each other
  int32_t add;              // input gradient: add to what is there
  int32_t first;            // logits: vocabulary entry of P's row 0 ...
  int64_t target_first;     // ... and, of targets[], of w's row 0
  float scale;              // logits: c log2(e)
  float2* part;             // forward: [parts][T] (largest logit, sum of exponentials from it)
  float* logit;             // forward: logit of a token's target, or NULL
  const Token* token;       // logits: per counting token, or
  const int32_t* targets;   // (forward of all tokens) its target
  const float* top;         // backward: [2], largest |a|, |b| and its inverse
  uint16_t* dz;             // [V' / 64][T'][64]
  int64_t rows_t;           // T'
  float* dx;                // [splits][T'][D] fp32
  uint16_t* dw;             // [V, D]
  float* dw_parts;          // [splits][V][D] fp32
  int32_t D;
};

// Tile of BP x BQ outputs, WP x WQ waves of (32 MB) x 64 each, 64 reduction
// steps a stage, two stages in LDS.  Every operand tile is staged as two
// units, its first half and its second; a wave holds MB blocks of 16 rows of
// each P half and two of each Q half.  So a stage is four products of a P half and a Q half,
// and a unit can be refilled as soon as its fragments are in registers, while
// the rest of the stage is still multiplied: a load has five of the eight
// phases of two stages (1.7 us of 256 x 256 tiles) before its data are read.
template <int MB_, int WP_, int WQ_>
struct Cfg {
  static constexpr int MB = MB_, WP = WP_, WQ = WQ_;
  static constexpr int BP = WP * 32 * MB, BQ = WQ * 64;
  static constexpr int UP = BP / 2 * 128, UQ = BQ / 2 * 128;     // bytes of a unit
  static constexpr int SP = BP / 2 / 64, SQ = BQ / 2 / 64;       // loads of a unit per wave
  static constexpr int LDS = 4 * (UP + UQ);
  static_assert(WP * WQ == 8 && SP >= 1 && SQ >= 1, "eight waves");
  static_assert(4 * UP <= 65536 && 4 * UQ <= 65536, "read offsets of 16 bits");
};
typedef Cfg<4, 2, 4> Large;      // 256 x 256
typedef Cfg<2, 4, 2> Small;      // 256 x 128

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// One operand of the tile: N waves along it, each with M blocks of 16 rows in
// either half.
// RS (strided): the unit holds [64 reduction steps][16 M N] values as they lie
// in memory and a fragment is read by the LDS transpose loads: lane i of 16
// addresses step i / 4 and values 4 (i % 4) .. + 3 and receives value i of four
// steps.  Otherwise [16 M N rows][64 steps], read with 128-bit loads.
// Bank conflicts: 16-byte chunk c of a row lies at c ^ (row % 8) of its eight (a
// 128-bit load takes lanes 0-3, 12-15, 20-23 and 24-27 together, which are then
// in different places; two rows span the banks).  Strided, 32 lanes read two chunks of steps 0-3 and 8-11:
// at c ^ 2 (row % 4 + 4 (row / 8 % 2)) of 16, or c ^ 2 (row / 2 % 2 +
// 2 (row / 8 % 2)) of eight, these lie in different places.
template <bool RS, int M, int N>
struct Side {
  static constexpr int U = 16 * M * N;          // rows (strided: values) of a unit
  static constexpr int BYTES = U * 128;
  static constexpr int S = U / 64;              // loads of a unit per wave
  static constexpr int kReads = RS ? 4 * M : 2 * M;
  static_assert(U == 128 || U == 64, "row swizzle");
  uint32_t at[RS ? M : 2];     // fragment addresses, by block or by slice of 32 steps
  uint32_t lds;                // the operand's first unit
  uint32_t row, chunk;         // load: byte offset of the lane's row; its chunk's bytes
  uint64_t base;
  uint32_t stride, step, most; // most: offset of the last row (strided: valid values)
  int first;                   // strided: step of the lane in a stage

  __device__ __forceinline__ void init(const Operand& o, uint32_t lds_, int w, int wave, int lane) {
    lds = lds_;
    stride = o.stride;
    step = o.step;
    const int i = lane & 15, g = lane >> 4;
    if constexpr (RS) {
      const int r = 8 * g + (i >> 2);
      const int swz = U == 128 ? (i >> 2) + 4 * (g & 1) : ((i >> 3) & 1) + 2 * (g & 1);
#pragma unroll
      for (int b = 0; b < M; ++b) {
        const int c = (2 * (w * M + b) + ((i & 3) >> 1)) ^ (2 * swz);
        at[b] = lds + (uint32_t)(r * U * 2 + 16 * c + 8 * (i & 1));
      }
      constexpr int kRow = U / 8;                              // chunks of a row
      const int lr = lane / kRow;                              // row within 1 KiB
      first = 64 / kRow * (wave * S) + lr;
      row = (uint32_t)first * stride;
      const int to = U == 128 ? (lr & 3) + 4 * (wave & 1) : ((lr >> 1) & 1) + 2 * (wave & 1);
      chunk = 16u * (uint32_t)((lane % kRow) ^ (2 * to));
    } else {
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)
        at[kk] = lds + (uint32_t)((w * 16 * M + i) * 128) +
                 (uint32_t)(((4 * kk + g) ^ (i & 7)) << 4);
      row = (uint32_t)(8 * S * wave + (lane >> 3)) * stride;
      chunk = (uint32_t)(((lane & 7) ^ (lane >> 3)) << 4);
    }
  }
  // Rows from o0 of n, steps from k0 (a multiple of 128).  Rows past the end
  // repeat the last one (their results are not stored); strided, values past it
  // are zeros.
  __device__ __forceinline__ void source(const void* p, int o0, int n, int k0) {
    const uint64_t b = reinterpret_cast<uint64_t>(p);
    if constexpr (RS) {
      base = b + (uint64_t)(o0 >> 6) * step + (uint64_t)k0 * stride;
      most = (uint32_t)min(2 * U, n - o0);
    } else {
      base = b + (uint64_t)o0 * stride + (uint64_t)(k0 >> 6) * step;
      most = (uint32_t)(min(2 * U, n - o0) - 1) * stride;
    }
  }
  __device__ __forceinline__ void advance() { base += RS ? 128 * (uint64_t)stride : 2 * (uint64_t)step; }

  // Refill of a unit with a stage, `left` steps of the reduction being left at
  // the buffer pair's start.  Steps past the end are zeros.
  template <int HALF, int BUF>
  __device__ __forceinline__ void load(uint32_t live, int left, int wave) const {
    const i32x4 rsrc = make_rsrc(reinterpret_cast<const void*>(base), live);
#pragma unroll
    for (int s = 0; s < S; ++s) {
      uint32_t off;
      if constexpr (RS) {
        constexpr int kRows = 512 / U;                         // steps of a load
        const uint32_t col = chunk >> 1;                       // value in the unit
        off = row + (uint32_t)(BUF * 64 + kRows * s) * stride +
              (col >> 6) * step + HALF * (U / 64) * step + 2 * (col & 63);
        off |= first + BUF * 64 + kRows * s < left && HALF * U + col < most ? 0u : kOOB;
      } else {
        off = min(row + (uint32_t)(8 * s + U * HALF) * stride, most) + chunk + BUF * step;
        off |= (int)(chunk >> 1) + BUF * 64 < left ? 0u : kOOB;
      }
      dma16(rsrc, lds + (2u * BUF + HALF) * BYTES + (uint32_t)(wave * S + s) * 1024u, off);
    }
  }
  template <int HALF, int BUF>
  __device__ __forceinline__ void read(bf16x8 (&f)[M][2]) const {
    constexpr uint32_t unit = (2 * BUF + HALF) * BYTES;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int b = 0; b < M; ++b) {
        if constexpr (RS) {
          const uint32_t a = at[b] + unit + kk * 32 * U * 2;
          const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)a);
          const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)(a + 4 * U * 2));
          f[b][kk] = __builtin_bit_cast(bf16x8, (s16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
          f[b][kk] = *(lds_frag*)(uintptr_t)(at[kk] + unit + b * 2048);
        }
      }
  }
};

template <class C, bool PRS, bool QRS>
struct Core {
  f32x4 acc[2 * C::MB][4];
  bf16x8 A0[C::MB][2], A1[C::MB][2], B0[2][2], B1[2][2];
  Side<PRS, C::MB, C::WP> P;
  Side<QRS, 2, C::WQ> Q;
  uint32_t live;
  int wave, left;

  __device__ __forceinline__ void init(const NtArgs& a, char* lds) {
    const int lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_char*)lds;
    P.init(a.P, lds0, wave / C::WQ, wave, lane);
    Q.init(a.Q, lds0 + 4 * C::UP, wave % C::WQ, wave, lane);
  }
  // The tile that the next loads bring; without one they read nothing.
  __device__ __forceinline__ void source(const void* p, const void* q, bool live_, int p0, int np, int q0,
                                         int nq, int k0, int K) {
    P.source(p, p0, np, k0);
    Q.source(q, q0, nq, k0);
    live = live_ ? 0x7fffffffu : 0u;
    left = K - k0;
  }
  __device__ __forceinline__ void advance() {
    P.advance();
    Q.advance();
    left -= 128;
  }
  template <int HALF, int BUF>
  __device__ __forceinline__ void loadP() const { P.template load<HALF, BUF>(live, left, wave); }
  template <int HALF, int BUF>
  __device__ __forceinline__ void loadQ() const { Q.template load<HALF, BUF>(live, left, wave); }

  // 16 x 16 x 32 products: an accumulator is read and written once in 32 steps.
  // (With 32 x 32 x 16 ones, once in 16, the chip drew more power and ran at 1.60
  // GHz, not 1.70: loss of 8192 x 131072 x 4096 in 6.68 ms, with these 6.38.)
  template <int HP, int HQ>
  __device__ __forceinline__ void mul(const bf16x8 (&A)[C::MB][2], const bf16x8 (&B)[2][2]) {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int i = 0; i < C::MB; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[C::MB * HP + i][2 * HQ + j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              A[i][kk], B[j][kk], acc[C::MB * HP + i][2 * HQ + j], 0, 0, 0);
  }
  // The reads between the products, evenly.
  template <int R>
  __device__ __forceinline__ void mix() {
    constexpr int each = (R + 7) / 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, C::MB / 2, 0);
      if (i * each < R) __builtin_amdgcn_sched_group_barrier(0x100, each, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  // All waves' fragment reads so far are done (their units may be refilled),
  // and all but the youngest N loads of every wave have landed.
  template <int N>
  __device__ __forceinline__ void edge() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    wait_vm<N>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  }
  // Loads of four units may be in flight at an edge: the two that the next two
  // phases read were issued five and six phases before.
  static constexpr int kFlight = 2 * C::SP + 2 * C::SQ;

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 2 * C::MB; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{};
  }
  __device__ __forceinline__ void start() {
    loadP<0, 0>(); loadQ<0, 0>(); loadQ<1, 0>(); loadP<1, 0>();
    loadP<0, 1>(); loadQ<1, 1>(); loadQ<0, 1>(); loadP<1, 1>();
    edge<3 * C::SP + 3 * C::SQ>();
    P.template read<0, 0>(A0);
    Q.template read<0, 0>(B0);
    edge<kFlight>();
    advance();
  }
  // Two stages, eight phases: each multiplies one pair of halves, reads the
  // half that a later phase needs into registers that are free, and refills
  // the unit that was read two phases before (of the stages 128 steps on).
  __device__ __forceinline__ void pair() {
    constexpr int RP = decltype(P)::kReads, RQ = decltype(Q)::kReads;
    loadP<0, 0>(); Q.template read<1, 0>(B1); mul<0, 0>(A0, B0); mix<RQ>();
    loadQ<0, 0>(); P.template read<1, 0>(A1); mul<0, 1>(A0, B1); mix<RP>(); edge<kFlight>();
    loadQ<1, 0>(); P.template read<0, 1>(A0); mul<1, 1>(A1, B1); mix<RP>();
    loadP<1, 0>(); Q.template read<1, 1>(B1); mul<1, 0>(A1, B0); mix<RQ>(); edge<kFlight>();
    loadP<0, 1>(); Q.template read<0, 1>(B0); mul<0, 1>(A0, B1); mix<RQ>();
    loadQ<1, 1>(); P.template read<1, 1>(A1); mul<0, 0>(A0, B0); mix<RP>(); edge<kFlight>();
    loadQ<0, 1>(); P.template read<0, 0>(A0); mul<1, 0>(A1, B0); mix<RP>();
    loadP<1, 1>(); Q.template read<0, 0>(B0); mul<1, 1>(A1, B1); mix<RQ>(); edge<kFlight>();
    advance();
  }
};

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ float low_half(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float high_half(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// Four blocks of 16 x 16 results, 16 bits each, lane l holding of row l % 16
// and block b columns 4 (l / 16) .. + 3 in x[b], to 16 bytes of one row: out[e]
// is of row (l % 16 & ~1) + e, block l / 16, columns 8 (l % 2) .. + 7.  So a
// store writes up to 128 contiguous bytes per row, where the registers as they
// are would give 32: the stores' requests, not their bytes, are what an
// epilogue waits for (dw of 96 tokens, V = 32768, D = 2048: 48 -> 35 us when a
// row's 16 bytes became 64).
__device__ __forceinline__ void regroup(const u32x2 (&x)[4], u32x4 (&out)[2], int lane) {
  uint32_t r[8];                     // block l / 16 of the lane's row, 16 columns
#pragma unroll
  for (int d = 0; d < 2; ++d) {
    // the other half wave's blocks, then the other 16 lanes' of each half
    const auto a = __builtin_amdgcn_permlane32_swap(x[0][d], x[2][d], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(x[1][d], x[3][d], false, false);
    const auto lo = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    r[d] = lo[0];
    r[2 + d] = lo[1];
    r[4 + d] = hi[0];
    r[6 + d] = hi[1];
  }
  const bool odd = lane & 1;
#pragma unroll
  for (int d = 0; d < 4; ++d) {      // second eight columns of the even row for the first of the odd one
    const uint32_t u = (uint32_t)__builtin_amdgcn_mov_dpp((int)r[d], 0xB1, 0xF, 0xF, true);
    const uint32_t v = (uint32_t)__builtin_amdgcn_mov_dpp((int)r[4 + d], 0xB1, 0xF, 0xF, true);
    out[0][d] = odd ? v : r[d];
    out[1][d] = odd ? r[4 + d] : u;
  }
}

// exp(c z - lse) is 2^(s z - r), one fma with s = c log2(e) and r = s lse / c
// rounded; what r's rounding takes off, in all exponents alike, goes to the
// factor before them.  Where r is past kFar that could be too much for a factor
// and the difference is taken first (a branch of the whole wave, for such tokens).
// z is above lse by the rounding of lse and of lse / c only, which is more the
// larger they are (2^-23 |lse| in all): no exponent is taken above that of z = lse,
// so that p <= 1 (at a temperature of 0.7 it was 2 for c z up to 1e7, 17 up to
// 4.6e7).  The minimum, one instruction per value, takes no time that can be
// measured: gradient of 8192 x 131072 x 4096 in 19.54 ms, without it 19.59.
constexpr float kFar = 67108864.f;
// z - lse, not above 0.  (A comparison, so that NaN stays.)
__device__ __forceinline__ float below(float z, float lse) {
  const float d = z - lse;
  return d > 0.f ? 0.f : d;
}

// A work item: tile (ip, iq) and, input gradient, part of the reduction.
// Items run along P within groups of gq tiles of Q.
struct Item {
  int ip, iq, s;
};
__device__ __forceinline__ Item item_of(int id, int tp, int tq, int gq) {
  Item t;
  t.s = id / (tp * tq);
  id -= t.s * tp * tq;
  const int g = id / (gq * tp), r = id - g * gq * tp, gh = min(gq, tq - g * gq);
  t.ip = r / gh;
  t.iq = g * gq + (r - t.ip * gh);
  return t;
}

// Products of all four calls.  One workgroup per compute unit walks its list
// of tiles; the loads run two stages ahead, on into the next tile, so that
// they go on during the epilogue.  Workgroup b runs on XCD b % 8, and every
// XCD has a contiguous range of tiles, gq of them along Q at a time, that
// share operand rows in its L2.  Bound by the matrix cores (busy 67% to 72% of
// the cycles) and by the clock that their power leaves (1.7 to 1.8 GHz): 8192
// tokens, V = 131072, D = 4096, forward 6.0 to 6.5 ms on different cards, 1350 to
// 1460 TFLOP/s (the product alone by the library: 1503); backward 19.4 to 20.5,
// 1290 to 1360.
// The weight gradient's loop on 256 x 256 tiles has more values than registers: three
// are read back from scratch in every pair of stages, and such a read waits for the
// loads in flight as well.
template <int EPI, class C>
__device__ __forceinline__ void products(const NtArgs& a, const int n_tok, const int tp0, const int tp_end,
                                         const int most_splits, const int rows, const int part0, char* lds) {
  constexpr bool kSplit = EPI == kDx || EPI == kDw;
  constexpr bool kLogits = EPI == kStats || is_dz(EPI);
  constexpr bool kCut = kLogits && C::BQ < 256;       // tiles may take fewer rows of P
  const int own = kCut ? rows : 256;
  const int np = EPI == kDx ? n_tok : a.np;
  const int nq = kLogits ? n_tok : a.nq;
  const int K = EPI == kDw ? n_tok : a.K;
  const int tp = tp_end - tp0, tq = (nq + C::BQ - 1) / C::BQ;      // tiles tp0 .. tp_end - 1 along P
  // pairs of stages; an empty reduction takes one of zeros
  const int pairs = max(1, (K + 127) >> 7);
  const int splits = kSplit ? min(most_splits, pairs) : 1;
  const int total = tp * tq * splits, xcd = blockIdx.x & 7, wgs = gridDim.x >> 3;
  const int per = total >> 3, rem = total & 7;
  // (the weight gradient's list begins at the other end of an XCD's workgroups:
  // the input gradient's has left those with the least)
  const int wg = blockIdx.x >> 3;
  int id = xcd * per + min(xcd, rem) + (EPI == kDw ? wgs - 1 - wg : wg);
  const int end = xcd * per + min(xcd, rem) + per + (xcd < rem ? 1 : 0);
  if (id >= end) return;
  // x, as it is where all tokens count
  const bool all = n_tok == a.tokens;
  const void* Pp = EPI == kDw && all ? a.x_all : a.P.base;
  const void* Qp = kLogits && all ? a.x_all : a.Q.base;

  Core<C, EPI == kDw, !kLogits> c;
  c.init(a, lds);
  auto range = [&](const Item& t, int& k0, int& m) {     // pairs [k0, k0 + m) of the item
    k0 = 0;
    m = pairs;
    if (kSplit) {
      const int each = pairs / splits, more = pairs - each * splits;
      k0 = t.s * each + min(t.s, more);
      m = each + (t.s < more ? 1 : 0);
    }
  };
  auto aim = [&](const Item& t, bool live) {
    int k0, m;
    range(t, k0, m);
    const int p0 = (tp0 + t.ip) * own;
    c.source(Pp, Qp, live, p0, kCut ? min(np, p0 + own) : np, t.iq * C::BQ, nq, 128 * k0, K);
    return m;
  };
  Item t = item_of(id, tp, tq, a.gq), ahead = t;
  int nid = id;
  int left = aim(t, true) - 1;       // pairs until the loads move on to the next tile
  c.start();
  const int lane = threadIdx.x & 63, l16 = lane & 15, g4 = lane >> 4;
  const int wp = c.wave / C::WQ, wq = c.wave % C::WQ;
  constexpr int MP = 2 * C::MB;
  // acc[i][j][e]: P row pw + p_row(i) + 4 g4 + e, Q row qw + q_row(j) + l16
  auto p_row = [](int i) { return i / C::MB * (C::BP / 2) + 16 * (i % C::MB); };
  auto q_row = [](int j) { return j / 2 * (C::BQ / 2) + 16 * (j % 2); };

  while (true) {
    int k0, m;
    range(t, k0, m);
    c.zero();
    for (int k = 0; k < m; ++k) {
      if (left == 0) {
        nid += wgs;
        const bool live = nid < end;
        if (live) ahead = item_of(nid, tp, tq, a.gq);
        left = aim(ahead, live);
      }
      c.pair();
      --left;
    }
    const int p0 = (tp0 + t.ip) * own, p_end = kCut ? min(np, p0 + own) : np, pw = p0 + wp * 16 * C::MB, qw = t.iq * C::BQ + wq * 32;

    if constexpr (EPI == kStats) {
      if (p0 + C::BP > p_end) {
        const int rows = p_end - pw - 4 * g4;
#pragma unroll
        for (int i = 0; i < MP; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (p_row(i) + e >= rows) {
#pragma unroll
              for (int j = 0; j < 4; ++j) c.acc[i][j][e] = -INFINITY;
            }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int q = qw + q_row(j) + l16;
        if (a.logit != nullptr) {
          int at = -1;
          if (q < nq) {
            if (a.targets != nullptr) {
              const int64_t v = (int64_t)a.targets[q] - a.target_first;
              at = v >= 0 && v < np ? (int)v : -1;
            } else {
              at = a.token[q].target;
            }
          }
          const int rel = at - pw;
          const bool here = at >= 0 && rel >= 0 && (kCut ? at < p_end : rel < C::BP) && ((rel >> 2) & 3) == g4 &&
                            rel % (C::BP / 2) < 16 * C::MB;
          if (__builtin_amdgcn_ballot_w64(here) != 0) {
            float z = 0.f;
#pragma unroll
            for (int i = 0; i < MP; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) z = rel - 4 * g4 == p_row(i) + e ? c.acc[i][j][e] : z;
            if (here) a.logit[q] = z;
          }
        }
        float top = c.acc[0][j][0];
#pragma unroll
        for (int i = 0; i < MP; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) top = fmaxf(top, c.acc[i][j][e]);
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        float ref = top == -INFINITY ? 0.f : top * a.scale;
        const bool far = fabsf(ref) > kFar;
        if (__builtin_amdgcn_ballot_w64(far) != 0) {
          const float from = far ? top : 0.f;
#pragma unroll
          for (int i = 0; i < MP; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) c.acc[i][j][e] -= from;
          ref = far ? 0.f : ref;
        }
        const float off = far || top == -INFINITY ? 0.f : __builtin_fmaf(top, a.scale, -ref);
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int i = 0; i < MP; ++i)
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            s0 += __builtin_amdgcn_exp2f(__builtin_fmaf(c.acc[i][j][e], a.scale, -ref));
            s1 += __builtin_amdgcn_exp2f(__builtin_fmaf(c.acc[i][j][e + 1], a.scale, -ref));
          }
        s0 += s1;
        s0 += __shfl_xor(s0, 16);
        s0 += __shfl_xor(s0, 32);
        s0 *= __builtin_amdgcn_exp2f(-off);
        if (g4 == 0 && q < nq) a.part[(int64_t)(part0 + t.ip * C::WP + wp) * a.tokens + q] = make_float2(top, s0);
      }
    }

    if constexpr (is_dz(EPI)) {
      const bool edge_p = p0 + C::BP > np;
      const float inv = a.top[1];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int q = qw + q_row(j) + l16;
        Token tk = {0.f, 0.f, 0.f, -1};
        if (q < nq) tk = a.token[q];
        const float wb = tk.b * inv;
        float wa = tk.a * inv, ref = tk.lse * a.scale;
        const bool far = fabsf(ref) > kFar;
        if (__builtin_amdgcn_ballot_w64(far) != 0) {
#pragma unroll
          for (int i = 0; i < MP; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) c.acc[i][j][e] = far ? below(c.acc[i][j][e], tk.lse) : c.acc[i][j][e];
          ref = far ? 0.f : ref;
        }
        const float off = far ? 0.f : __builtin_fmaf(tk.lse, a.scale, -ref);
        wa *= __builtin_amdgcn_exp2f(-off);
        const int rel = tk.target < 0 ? -1 : tk.target - a.first - pw;
        const bool told = __builtin_amdgcn_ballot_w64(rel >= 0 && rel < C::BP) != 0;
#pragma unroll
        for (int i = 0; i < MP; i += 4) {
          u32x2 pk[4], low[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              // (the minimum keeps NaN; p <= 1, as below() has it)
              const float to = __builtin_elementwise_minimum(__builtin_fmaf(c.acc[i + u][j][e], a.scale, -ref), off);
              v[e] = wa * __builtin_amdgcn_exp2f(to);
              if (told) v[e] -= rel - 4 * g4 == p_row(i + u) + e ? wb : 0.f;
              if (edge_p) v[e] = p_row(i + u) + e < np - pw - 4 * g4 ? v[e] : 0.f;
            }
            // the one rounding of dz: a 16-bit operand of the two products
            pk[u] = u32x2{pack2(v[0], v[1]), pack2(v[2], v[3])};
            if (EPI == kDzPair)
              low[u] = u32x2{pack2(v[0] - low_half(pk[u][0]), v[1] - high_half(pk[u][0])),
                             pack2(v[2] - low_half(pk[u][1]), v[3] - high_half(pk[u][1]))};
          }
          u32x4 out[2];
          regroup(pk, out, lane);
          // the lane's block, its two rows of dz
          const int pb = pw + p_row(i) + (C::MB == 4 ? 16 * g4 : (g4 >> 1) * (C::BP / 2) + 16 * (g4 & 1));
          char* dz = reinterpret_cast<char*>(a.dz) +
                     ((int64_t)(pb >> 6) * a.rows_t + qw + q_row(j) + (l16 & ~1)) * 128 + 2 * (pb & 63) + 16 * (lane & 1);
          if constexpr (EPI == kDzPair) {
            u32x4 rest[2];
            regroup(low, rest, lane);
            const int q2 = qw + q_row(j) + (l16 & ~1);
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (q2 + e < nq && (!kCut || pb < p_end)) {
                *reinterpret_cast<u32x4*>(dz + 128 * e) = out[e];
                *reinterpret_cast<u32x4*>(dz + 128 * (nq + e)) = rest[e];
              }
          } else if (!kCut || pb < p_end) {
            *reinterpret_cast<u32x4*>(dz) = out[0];
            *reinterpret_cast<u32x4*>(dz + 128) = out[1];
          }
          __builtin_amdgcn_sched_barrier(0);      // four blocks' values at a time: registers
        }
      }
    }

    if constexpr (EPI == kDx) {
      // P = tokens, Q = hidden columns: 32 consecutive columns per row and store
      auto store = [&](auto whole, auto add) {
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          const int d = qw + q_row(j) + 16 * (g4 & 1) + l16, p4 = pw + 4 * (g4 & ~1);
          const int rows = d < nq ? np - p4 : 0;
          float* to = a.dx + ((int64_t)t.s * a.rows_t + p4) * a.D + d;
#pragma unroll
          for (int i = 0; i < MP; ++i) {
            asm volatile("" : "+v"(to));      // a block's addresses at a time: registers
            float* at = to + (int64_t)p_row(i) * a.D;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              // rows 4 g4 + e of 16 columns each -> of 32: the even 16 lanes' row, the odd ones'
              const auto v = __builtin_amdgcn_permlane16_swap(__float_as_uint(c.acc[i][j][e]),
                                                              __float_as_uint(c.acc[i][j + 1][e]), false, false);
#pragma unroll
              for (int u = 0; u < 2; ++u)
                if (whole.value || p_row(i) + 4 * u + e < rows) {
                  // (adding: once per element and launch, so there is no order to
                  // depend on, and no load to wait for)
                  float* here = at + (int64_t)(4 * u + e) * a.D;
                  if (add.value) unsafeAtomicAdd(here, __uint_as_float(v[u]));
                  else *here = __uint_as_float(v[u]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      };
      const bool whole = p0 + C::BP <= np && t.iq * C::BQ + C::BQ <= nq;
      if (whole && a.add) store(std::true_type{}, std::true_type{});
      else if (whole) store(std::true_type{}, std::false_type{});
      else if (a.add) store(std::false_type{}, std::true_type{});
      else store(std::false_type{}, std::false_type{});
    }

    if constexpr (EPI == kDw) {
      // P = hidden columns, Q = vocabulary entries
      const float scale = a.top[0];
      if (splits > 1) {          // parts in fp32, joined by head_sum_kernel
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int q = qw + q_row(j) + l16;
          float* to = a.dw_parts + ((int64_t)t.s * nq + q) * a.D + pw + 4 * g4;
#pragma unroll
          for (int i = 0; i < MP; ++i)
            if (q < nq && pw + p_row(i) + 4 * g4 < np) *reinterpret_cast<f32x4*>(to + p_row(i)) = c.acc[i][j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int q2 = qw + q_row(j) + (l16 & ~1);
#pragma unroll
          for (int i = 0; i < MP; i += 4) {
            u32x2 pk[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
              pk[u] = u32x2{pack2(c.acc[i + u][j][0] * scale, c.acc[i + u][j][1] * scale),
                            pack2(c.acc[i + u][j][2] * scale, c.acc[i + u][j][3] * scale)};
            u32x4 out[2];
            regroup(pk, out, lane);
            const int d = pw + p_row(i) + (C::MB == 4 ? 16 * g4 : (g4 >> 1) * (C::BP / 2) + 16 * (g4 & 1)) + 8 * (lane & 1);
            uint16_t* to = a.dw + (int64_t)q2 * a.D + d;
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (q2 + e < nq && d < np) *reinterpret_cast<u32x4*>(to + (int64_t)e * a.D) = out[e];
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      }
    }

    id += wgs;
    if (id >= end) break;
    t = ahead;
  }
  // the loads in flight write this workgroup's LDS, which its next tiles take
  wait_vm<0>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Parts of the forward's sums: before tile ip along P, and of all its tiles.
__host__ __device__ __forceinline__ int parts_before(int ip, int large) {
  return ip < large ? ip * Large::WP : large * Large::WP + (ip - large) * Small::WP;
}
__host__ __device__ __forceinline__ int parts_of(int64_t V, const Plan& p) {
  return parts_before((int)((V + p.rows - 1) / p.rows), p.large);
}

template <int EPI>
__device__ __forceinline__ void product(const NtArgs& a, char* lds) {
  const int n = a.n != nullptr ? __builtin_amdgcn_readfirstlane(*a.n) : a.tokens;
  Plan plan = a.plan;
  if (a.plan_at != nullptr) {
    plan.large = __builtin_amdgcn_readfirstlane(a.plan_at->large);
    plan.splits = __builtin_amdgcn_readfirstlane(a.plan_at->splits);
    if (EPI == kStats || is_dz(EPI)) plan.rows = __builtin_amdgcn_readfirstlane(a.plan_at->rows);
  }
  const int tp = EPI == kStats || is_dz(EPI) ? (a.np + plan.rows - 1) / plan.rows : ((EPI == kDx ? n : a.np) + 255) / 256;
  const int large = min(plan.large, tp);
  products<EPI, Large>(a, n, 0, large, plan.splits, plan.rows, 0, lds);
  products<EPI, Small>(a, n, large, tp, plan.splits, plan.rows, parts_before(large, large), lds);
}

template <int EPI>
__global__ __launch_bounds__(512, 2) void nt_kernel(const NtArgs a) {
  extern __shared__ char lds[];
  product<EPI>(a, lds);
}

// Both gradients of a piece: a workgroup whose part of dx is done goes on with
// dw, so that neither waits for the other's last tiles.
__global__ __launch_bounds__(512, 2) void grads_kernel(const NtArgs x, const NtArgs w) {
  extern __shared__ char lds[];
  if (x.dx != nullptr) product<kDx>(x, lds);
  if (w.dw != nullptr) product<kDw>(w, lds);
}

// The logits' product of small problems, on tiles of 64 x 64 whose reduction is
// shared by the workgroup's eight waves, 64 steps in turn: where 256 x 128 tiles
// would be fewer than the compute units, four to eight times as many
// workgroups, each with an eighth of the steps (V = 700, 256 tokens, D = 4096:
// the forward 53 -> 20 us).  A wave stages its own 64 x 64 parts of both operands
// (16 KiB), takes them to registers, sends for the next and multiplies: no wave
// waits for another until their sums meet in LDS, in a fixed order.
template <int EPI>
__global__ __launch_bounds__(512, 2) void tile64_kernel(const NtArgs a) {
  extern __shared__ char lds[];
  float4* red = reinterpret_cast<float4*>(lds);          // [8 waves][16][64 lanes]
  const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nq = a.n != nullptr ? __builtin_amdgcn_readfirstlane(*a.n) : a.tokens, np = a.np, K = a.K;
  const int p0 = blockIdx.x * 64, q0 = blockIdx.y * 64;
  if (q0 >= nq) return;
  if (p0 >= np) {                                        // (parts are counted in tiles of 256)
    if (EPI == kStats && threadIdx.x < 64 && q0 + threadIdx.x < nq)
      a.part[(int64_t)blockIdx.x * a.tokens + q0 + threadIdx.x] = make_float2(-INFINITY, 0.f);
    return;
  }
  const char* Q = static_cast<const char*>(nq == a.tokens ? a.x_all : a.Q.base);
  // rows past the end repeat the last one, steps past it are zeros
  const uint32_t mine = (uint32_t)(uintptr_t)(lds_char*)lds + (uint32_t)wave * 16384u;
  const uint32_t r8 = lane >> 3, chunk = 16u * ((lane & 7) ^ r8);       // of even eights of rows
  const uint32_t most[2] = {(uint32_t)(min(64, np - p0) - 1) * a.P.stride, (uint32_t)(min(64, nq - q0) - 1) * a.Q.stride};
  const uint32_t stride[2] = {a.P.stride, a.Q.stride};
  const uint64_t base[2] = {reinterpret_cast<uint64_t>(a.P.base) + (uint64_t)p0 * a.P.stride,
                            reinterpret_cast<uint64_t>(Q) + (uint64_t)q0 * a.Q.stride};
  auto load = [&](int block) {
    const uint32_t past[2] = {(int)(chunk >> 1) + 64 * block < K ? 0u : kOOB,
                              (int)((chunk ^ 16u) >> 1) + 64 * block < K ? 0u : kOOB};
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      const i32x4 rsrc = make_rsrc(reinterpret_cast<const void*>(base[o] + 128 * (uint64_t)block), 0x7fffffffu);
#pragma unroll
      for (int r = 0; r < 8; ++r)
        dma16(rsrc, mine + 8192u * o + 1024u * r,
              (min((r8 + 8 * r) * stride[o], most[o]) + (chunk ^ (16u * (r & 1)))) | past[r & 1]);
    }
  };
  f32x16 acc[2][2] = {};
  const int blocks = (K + 63) / 64;
  if (wave < blocks) load(wave);
  for (int b = wave; b < blocks; b += 8) {
    bf16x8 f[4][4];                                      // w, w, x, x
    wait_vm<0>();
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        f[i][kk] = *(lds_frag*)(uintptr_t)(mine + 4096u * i + 128u * l32 +
                                           (uint32_t)(((2 * kk + h) ^ (l32 & 7) ^ ((l32 >> 3) & 1)) << 4));
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    if (b + 8 < blocks) load(b + 8);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[i][kk], f[2 + j][kk], acc[i][j], 0, 0, 0);
  }
  __syncthreads();                                       // the sums take the staged data's place
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        red[(wave * 16 + (2 * i + j) * 4 + g) * 64 + lane] =
            make_float4(acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]);
  __syncthreads();
  // the wave's share: rows 32 i + 16 (wave & 1) + 8 g + 4 h + e, g < 2, of token q
  const int i = wave >> 2, j = (wave >> 1) & 1, pw = p0 + 32 * i + 16 * (wave & 1) + 4 * h;
  const int q = q0 + 32 * j + l32;
  float v[8];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    float4 s = red[((2 * i + j) * 4 + 2 * (wave & 1) + g) * 64 + lane];
#pragma unroll
    for (int w = 1; w < 8; ++w) {
      const float4 o = red[(w * 16 + (2 * i + j) * 4 + 2 * (wave & 1) + g) * 64 + lane];
      s.x += o.x; s.y += o.y; s.z += o.z; s.w += o.w;
    }
    v[4 * g] = s.x; v[4 * g + 1] = s.y; v[4 * g + 2] = s.z; v[4 * g + 3] = s.w;
  }
  if constexpr (EPI == kStats) {
    int at = -1;
    if (a.logit != nullptr && q < nq) {
      if (a.targets != nullptr) {
        const int64_t t = (int64_t)a.targets[q] - a.target_first;
        at = t >= 0 && t < np ? (int)t : -1;
      } else {
        at = a.token[q].target;
      }
    }
    float top = -INFINITY;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int p = pw + 8 * (e >> 2) + (e & 3);
      if (at >= 0 && p == at) a.logit[q] = v[e];
      v[e] = p < np ? v[e] : -INFINITY;
      top = fmaxf(top, v[e]);
    }
    top = fmaxf(top, __shfl_xor(top, 32));
    const float from = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += __builtin_amdgcn_exp2f((v[e] - from) * a.scale);
    sum += __shfl_xor(sum, 32);
    __syncthreads();
    float2* of = reinterpret_cast<float2*>(lds);         // [4 sixteens of rows][64 tokens]
    if (h == 0) of[(2 * i + (wave & 1)) * 64 + 32 * j + l32] = make_float2(top, sum);
    __syncthreads();
    if (threadIdx.x < 64 && q0 + threadIdx.x < nq) {
      float2 r = of[threadIdx.x];
#pragma unroll
      for (int w = 1; w < 4; ++w) {
        const float2 o = of[64 * w + threadIdx.x];
        const float m = fmaxf(r.x, o.x), base = m == -INFINITY ? 0.f : m;
        r.y = r.y * __builtin_amdgcn_exp2f((r.x - base) * a.scale) + o.y * __builtin_amdgcn_exp2f((o.x - base) * a.scale);
        r.x = m;
      }
      a.part[(int64_t)blockIdx.x * a.tokens + q0 + threadIdx.x] = r;
    }
  } else {
    Token tk = {0.f, 0.f, 0.f, -1};
    if (q < nq) tk = a.token[q];
    const float inv = a.top[1], wa = tk.a * inv, wb = tk.b * inv;
    const int rel = tk.target < 0 ? -1 : tk.target - a.first;
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int p = pw + 8 * (e >> 2) + (e & 3);
      float z = wa * __builtin_amdgcn_exp2f(below(v[e], tk.lse) * a.scale);
      z -= p == rel ? wb : 0.f;
      v[e] = p < np ? z : 0.f;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = pack2(v[2 * e], v[2 * e + 1]);
    char* dz = reinterpret_cast<char*>(a.dz) + ((int64_t)blockIdx.x * a.rows_t + q) * 128 + 2 * (pw - p0);
    if (EPI == kDzPair && q >= nq) return;
    *reinterpret_cast<u32x2*>(dz) = u32x2{o[0], o[1]};
    *reinterpret_cast<u32x2*>(dz + 16) = u32x2{o[2], o[3]};
    if (EPI == kDzPair) {
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = pack2(v[2 * e] - low_half(o[e]), v[2 * e + 1] - high_half(o[e]));
      dz += 128 * (int64_t)nq;
      *reinterpret_cast<u32x2*>(dz) = u32x2{o[0], o[1]};
      *reinterpret_cast<u32x2*>(dz + 16) = u32x2{o[2], o[3]};
    }
  }
}

// ------------------------------------------------------------ token passes --

// An entry of the teacher: NaN counts as -inf, +inf as the largest value.
__device__ __forceinline__ float teacher_value(const HeadArgs& a, int64_t i) {
  float v = a.teacher_bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.teacher)[i] << 16)
                           : static_cast<const float*>(a.teacher)[i];
  return v != v ? -INFINITY : fminf(v, 3.402823466e38f);
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

constexpr int kEntryLanes = 4;       // entries per lane: k <= 256

// The teacher's distribution of one token over its entries, entry 64 i + lane
// in q[i] (0 where there is none); returns whether there is any.  lq: log q.
__device__ __forceinline__ bool teacher_row(const HeadArgs& a, int64_t t, int lane,
                                            float (&q)[kEntryLanes], float (&lq)[kEntryLanes],
                                            int (&at)[kEntryLanes]) {
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kEntryLanes; ++i) {
    const int j = 64 * i + lane;
    at[i] = j < a.k ? a.index[t * a.k + j] : -1;
    lq[i] = at[i] >= 0 ? teacher_value(a, t * a.k + j) : -INFINITY;
    if (lq[i] == -INFINITY) at[i] = -1;
    top = fmaxf(top, lq[i]);
  }
  top = wave_max(top);
  if (top == -INFINITY) return false;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kEntryLanes; ++i) {
    lq[i] = at[i] >= 0 ? (lq[i] - top) * (float)a.c : -INFINITY;
    q[i] = at[i] >= 0 ? expf(lq[i]) : 0.f;
    sum += q[i];
  }
  sum = wave_sum(sum);
  const float log_sum = logf(sum);
#pragma unroll
  for (int i = 0; i < kEntryLanes; ++i) {
    q[i] /= sum;
    lq[i] -= log_sum;
  }
  return true;
}

// Which tokens have an entry of the teacher.  One wave per token.
__global__ __launch_bounds__(256) void head_flags_kernel(const HeadArgs a, uint8_t* flag) {
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (t >= a.T) return;
  bool any = false;
  for (int j = lane; j < a.k; j += 64)
    any |= a.index[t * a.k + j] >= 0 && teacher_value(a, t * a.k + j) > -INFINITY;
  const bool counts = __builtin_amdgcn_ballot_w64(any) != 0;
  if (lane == 0) flag[t] = counts;
}

// The products' plans.  Times in ns: a tile of 256 x 256 takes 2800 per pair of
// stages (128 steps), one of 256 x 128 1660 (2070 where w's rows do not start
// on 128 bytes: its staged rows are then two reads of L2 each), and its epilogue
// `el`, `es` more; tiles run in rounds of the chip's 256 compute units.
// (Measured on 2048 tokens, V = 65536, D = 512 to 2064, either size alone.)
constexpr float kLargePair = 2800.f, kSmallPair = 1660.f, kSmallPairOdd = 2070.f;
struct Cost {
  int el, es;
};
__host__ __device__ __forceinline__ Cost cost_of(int epi) {
  return epi == kStats ? Cost{3600, 1900} : epi == kDz ? Cost{10000, 5500} : epi == kDw ? Cost{10000, 3000} : Cost{5000, 3000};
}
__host__ __device__ __forceinline__ float rounds_of(uint32_t tiles) { return (float)((tiles + 255) >> 8); }

// How many tiles along P are large: whole rounds of them, or all; what is left
// over in small ones, where it would fill half a round or less.
struct Timed {
  Plan plan;
  float time;
};
constexpr int kFewTokens = 128, kLeastRows = 64;
__host__ __device__ __forceinline__ Timed plan_of(int epi, int np, int nq, int K, bool few) {
  const uint32_t tp = (np + 255) / 256, tl = (nq + 255) / 256, ts = (nq + 127) / 128;
  const int pairs = K > 128 ? (K + 127) / 128 : 1;
  const Cost e = cost_of(epi);
  const float small_pair = (epi == kStats || epi == kDz) && K % 64 != 0 ? kSmallPairOdd : kSmallPair;
  const float large = kLargePair * pairs + e.el, small = small_pair * pairs + e.es;
  const uint32_t full = tp * tl / 256;
  Timed best = {{(int)tp, 1, 256}, -1.f};
#pragma unroll
  for (uint32_t i = 0; i < 4; ++i) {
    // all, none, all whole rounds, all but one of them
    if (i > 1 && (tl == 0 || full < i - 2)) continue;
    const uint32_t m = i == 0 ? tp : i == 1 ? 0 : (full - (i - 2)) * 256 / tl;
    const float t = rounds_of(m * tl) * large + rounds_of((tp - m) * ts) * small + (m > 0 && m < tp ? 3000.f : 0.f);
    if (best.time < 0.f || t < best.time) best = {{(int)m, 1, 256}, t};
  }
  // Few tokens (w is read once, and that is the time): small tiles that take
  // fewer rows each, so that all rounds are full.  (The forward's kernel in us, D =
  // 3328, V = 65721 or 257 tiles, 60 tokens: 120 -> 101; V = 151936, 128 tokens of
  // 4096: 257 -> 233.  For 256 tokens of 1024, V = 20000: 24 -> 25; for 10 of 184, V =
  // 112369, where the tiles' epilogues count: 26.7 -> 28.0.)
  if ((epi == kStats || epi == kDz) && few && nq > 0 && nq <= kFewTokens && K >= 512) {
    const uint32_t most = (tp + 255) / 256 * 256;
    const int rows = (int)(((uint32_t)np + most - 1) / most + 15) / 16 * 16;
    best.plan = {0, 1, rows < kLeastRows ? kLeastRows : rows};
  }
  return best;
}

// A gradient's tile size and parts of its reduction, choice i of 24: parts 1,
// 2, 3, 4, 6, 8, 12, .. 64, every part's way to memory and back at 5.1 TB/s.
__host__ __device__ __forceinline__ Timed split_choice(int epi, int i, int np, int nq, int K) {
  const int k = i >> 1, s = k < 2 ? k + 1 : (k & 1 ? 4 : 3) << (k - 2) / 2;
  const uint32_t pairs = K > 128 ? (K + 127) / 128 : 1, tp = (np + 255) / 256;
  const Cost e = cost_of(epi);
  const float each = (float)((pairs + s - 1) / s);
  const uint32_t tiles = tp * (i & 1 ? (nq + 127) / 128 : (nq + 255) / 256);
  const float rounds = ceilf((float)tiles * (float)s * (1.f / 256.f));
  const float time = rounds * (i & 1 ? kSmallPair * each + e.es : kLargePair * each + e.el) +
                     (float)s * (float)np * (float)nq * (1.f / 640.f) + (epi == kDw && s > 1 ? 2000.f : 0.f);
  return {{i & 1 ? 0 : (int)tp, s, 256}, time};
}
// The best of them, found by a wave.
__device__ __forceinline__ Plan split_plan(int epi, int np, int nq, int K, int most, int lane) {
  Timed p = split_choice(epi, lane < 24 ? lane : 0, np, nq, K);
  if (p.plan.splits > most) p.time = INFINITY;
  float least = p.time;
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) least = fminf(least, __shfl_xor(least, d));
  const int at = __builtin_ctzll(__builtin_amdgcn_ballot_w64(p.time == least));
  return Plan{__builtin_amdgcn_readlane(p.plan.large, at), __builtin_amdgcn_readlane(p.plan.splits, at), 256};
}

enum { kPlanLogits = 0, kPlanDx = 1, kPlanDw = 2, kPlans = 3 };

// The counting tokens in order: pos[t] their place (-1 for the others),
// rows[place] the token, n their number; per place what the epilogues need,
// the products' plans and, backward, the largest weight.  The first workgroup
// writes all that.  With `pack` every workgroup goes through the tokens, and
// packs its share of the rows of x (stride `ld`; nothing where all tokens count
// and x's own rows start on 128 bytes): for short batches, one launch for two.
// Eight tokens per thread and turn, so that a turn's loads are in flight
// together.  flag: the teacher's, or NULL: looked up here.
constexpr int kPlaceList = 64;         // rows of a workgroup's share
constexpr int kPlaceFlags = 1024;      // tokens whose entries this kernel looks up itself
struct PlaceArgs {
  const uint8_t* flag;
  int32_t* pos;
  int32_t* rows;
  int32_t* n;
  Token* token;
  Plan* plans;
  float* top;                // backward: [2]
  uint16_t* pack;
  int32_t ld, piece, dx_splits, dw_splits;
  int32_t pair;              // the gradients' products take every token twice
};
template <int PER>       // tokens of a thread in a turn, 1024 apart
__global__ __launch_bounds__(1024) void head_place_kernel(const HeadArgs a, const PlaceArgs o) {
  __shared__ int counts[2][128];
  __shared__ float tops[16];
  __shared__ int list[kPlaceList];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool head = blockIdx.x == 0;
  int base = 0, turn = 0;
  float most = 0.f;
  for (int64_t b = 0; b < a.T; b += 1024 * PER, turn ^= 1) {
    bool in[PER];
    int32_t target[PER];
    float up[PER], lse[PER], dlse[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const int64_t t = b + 1024 * e + threadIdx.x;
      const bool there = t < a.T;
      target[e] = -1;
      in[e] = false;
      if (there) {
        if (a.index == nullptr) {
          target[e] = a.targets[t];
          in[e] = target[e] >= 0;
        } else if (o.flag != nullptr) {
          in[e] = o.flag[t] != 0;
        } else if (PER == 1) {
          bool any = false;
          for (int j = 0; j < a.k && !any; j += 8) {
            int at[8];
            float v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const int64_t i = t * a.k + min(j + u, a.k - 1);
              at[u] = a.index[i];
              v[u] = teacher_value(a, i);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) any |= at[u] >= 0 && v[u] > -INFINITY;
          }
          in[e] = any;
        }
      }
      if (head && there && a.dloss != nullptr) {
        up[e] = a.dloss[t];
        lse[e] = a.lse_in[t];
        dlse[e] = a.dlse != nullptr ? a.dlse[t] : 0.f;
      }
    }
    // places: by e, then wave, then lane
    uint64_t mask[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      mask[e] = __builtin_amdgcn_ballot_w64(in[e]);
      if (lane == 0) counts[turn][16 * e + wave] = __popcll(mask[e]);
    }
    __syncthreads();
    int sum[2], total = 0;                     // counts before each (e, wave), 64 of them per register
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int v = 64 * u + lane < 16 * PER ? counts[turn][64 * u + lane] : 0;
      int s = v;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int w = __shfl_up(s, d);
        if (lane >= d) s += w;
      }
      sum[u] = total + s - v;
      total += __builtin_amdgcn_readlane(s, 63);
    }
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const int64_t t = b + 1024 * e + threadIdx.x;
      const int before = base + __builtin_amdgcn_readlane(sum[e / 4], (16 * e + wave) & 63) +
                         __popcll(mask[e] & ((1ull << lane) - 1));
      if (t >= a.T) continue;
      if (in[e] && o.pack != nullptr && before % gridDim.x == blockIdx.x) list[before / gridDim.x] = (int)t;
      if (!head) continue;
      o.pos[t] = in[e] ? before : -1;
      if (!in[e]) continue;
      o.rows[before] = (int32_t)t;
      Token k = {0.f, 0.f, 0.f, -1};
      if (a.index == nullptr) {
        const int64_t at = (int64_t)target[e] - a.first;
        k.target = at >= 0 && at < a.V ? (int32_t)at : -1;
      }
      if (a.dloss != nullptr) {
        k.lse = (float)((double)lse[e] / a.c);
        k.b = up[e] * (float)a.c;
        k.a = a.dlse != nullptr ? k.b + dlse[e] : k.b;
        most = fmaxf(most, fmaxf(fabsf(k.a), fabsf(k.b)));
      }
      o.token[before] = k;
    }
    base += total;
  }
  if (head) {
    const int rows = o.pair ? 2 * base : base;             // of dz
    if (threadIdx.x == 0) o.n[0] = base, o.n[1] = rows;
    if (threadIdx.x == 960)
      o.plans[kPlanLogits] = plan_of(o.top == nullptr ? kStats : kDz, o.piece, base, (int)a.D, o.top != nullptr || a.T <= kFewTokens).plan;
    if (o.top != nullptr) {
      if (wave == 13) {
        const Plan p = split_plan(kDx, rows, (int)a.D, o.piece, o.dx_splits, lane);
        if (lane == 0) o.plans[kPlanDx] = p;
      }
      if (wave == 14) {
        Plan p = split_plan(kDw, (int)a.D, o.piece, rows, o.dw_splits, lane);
        if (p.splits == 1) p = plan_of(kDw, (int)a.D, o.piece, rows, false).plan;
        if (lane == 0) o.plans[kPlanDw] = p;
      }
      most = wave_max(most);
      if (lane == 0) tops[wave] = most;
      __syncthreads();
      if (threadIdx.x == 0) {
        for (int w = 1; w < 16; ++w) most = fmaxf(most, tops[w]);
        // a weight past the range where its inverse is a normal number is left as it is
        const bool fit = most > 1e-37f && most < 1e37f;
        o.top[0] = fit ? most : 1.f;
        o.top[1] = fit ? 1.f / most : 1.f;
      }
    }
  }
  if (o.pack == nullptr || (base == a.T && o.ld == a.D && !o.pair)) return;
  __syncthreads();
  for (int i = wave; i * (int64_t)gridDim.x + blockIdx.x < base; i += 16) {
    const u32x4* from = reinterpret_cast<const u32x4*>(a.x + (int64_t)list[i] * a.D);
    u32x4* to = reinterpret_cast<u32x4*>(o.pack + ((int64_t)i * gridDim.x + blockIdx.x) * o.ld);
    for (int c = lane; c < a.D / 8; c += 64) {
      const u32x4 v = from[c];
      to[c] = v;
      if (o.pair) to[c + (int64_t)base * o.ld / 8] = v;
    }
  }
}

// xc[place] = x[rows[place]], as the kernel above.  One wave per row.
__global__ __launch_bounds__(256) void head_pack_kernel(const uint16_t* x, const int32_t* rows,
                                                        const int32_t* n, int32_t T, int32_t D,
                                                        uint16_t* xc, int32_t ld) {
  const int count = *n;
  if (count == T && ld == D) return;
  for (int64_t p = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); p < count; p += (int64_t)gridDim.x * 4) {
    const u32x4* from = reinterpret_cast<const u32x4*>(x + (int64_t)rows[p] * D);
    u32x4* to = reinterpret_cast<u32x4*>(xc + p * ld);
    for (int i = threadIdx.x & 63; i < D / 8; i += 64) to[i] = from[i];
  }
}

// lse of every token from its parts, and the loss of a target.  TT tokens per
// workgroup of NT threads, NT / TT threads to a token's parts.  The sum's
// logarithm, the reference and the difference from the logit are put together
// in 64 bits: each is up to log V, their sum may be far smaller.
template <int TT, int NT>
__global__ __launch_bounds__(NT) void head_join_kernel(const HeadArgs a, const int32_t parts_, const Plan* plan_at,
                                                       const int32_t* pos, const float2* part,
                                                       const float* logit, double* lse64) {
  __shared__ float2 got[NT / 64][TT];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, tok = threadIdx.x % TT;
  const int64_t t = (int64_t)blockIdx.x * TT + tok;
  const int parts = plan_at != nullptr ? parts_of(a.V, *plan_at) : parts_;
  int p = -1;
  if (t < a.T) p = pos != nullptr ? pos[t] : a.index != nullptr || a.targets[t] >= 0 ? (int)t : -1;
  float top = -INFINITY, sum = 0.f;
  auto join = [&](const float2 v) {
    const float m = fmaxf(top, v.x), ref = m == -INFINITY ? 0.f : m;
    sum = sum * __builtin_amdgcn_exp2f((top - ref) * a.scale) + v.y * __builtin_amdgcn_exp2f((v.x - ref) * a.scale);
    top = m;
  };
  if (p >= 0) {
#pragma unroll 4
    for (int i = threadIdx.x / TT; i < parts; i += NT / TT) join(part[(int64_t)i * a.T + p]);
  }
#pragma unroll
  for (int d = TT; d < 64; d <<= 1) join(make_float2(__shfl_xor(top, d), __shfl_xor(sum, d)));
  if (lane < TT) got[wave][lane] = make_float2(top, sum);
  __syncthreads();
  if (threadIdx.x >= TT || t >= a.T) return;
  for (int w = 1; w < NT / 64; ++w) join(got[w][threadIdx.x]);
  const double lse = p >= 0 ? (double)top * a.c + log((double)sum) : 0.0;
  a.lse[t] = (float)lse;
  if (a.index != nullptr) {
    lse64[t] = lse;
  } else {
    const int64_t at = (int64_t)a.targets[t] - a.first;
    const float z = p >= 0 && at >= 0 && at < a.V ? logit[p] : 0.f;
    a.logits[t] = z;
    a.loss[t] = (float)(lse - (double)z);
  }
}

// The logits of the entries of one token whose rows of w are given (row, -1 for
// none; entry 64 i + lane), four entries at a time, 8 columns per lane and
// step; wave `part` of `of` takes its share of the fours.
__device__ __forceinline__ void entry_logits(const HeadArgs& a, int64_t t, int lane,
                                             const int (&row)[kEntryLanes], int part, int of,
                                             float (&z)[kEntryLanes]) {
  const uint16_t* x = a.x + t * a.D;
  int turn = 0;
#pragma unroll
  for (int i = 0; i < kEntryLanes; ++i) {
    z[i] = 0.f;
    uint64_t todo = __builtin_amdgcn_ballot_w64(row[i] >= 0);
    while (todo != 0) {
      int j[4], r[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        j[e] = todo != 0 ? __builtin_ctzll(todo) : j[0];      // (past the last one: the first again)
        todo &= todo - 1;
        r[e] = __builtin_amdgcn_readlane(row[i], j[e]);
      }
      if (turn++ % of != part) continue;
      float s[4] = {};
#pragma unroll 2
      for (int d = 8 * lane; d < a.D; d += 512) {
        const u32x4 xv = *reinterpret_cast<const u32x4*>(x + d);
        u32x4 wv[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) wv[e] = *reinterpret_cast<const u32x4*>(a.w + (int64_t)r[e] * a.D + d);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float lo = __uint_as_float(xv[c] << 16), hi = __uint_as_float(xv[c] & 0xffff0000u);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[e] = __builtin_fmaf(lo, __uint_as_float(wv[e][c] << 16), s[e]);
            s[e] = __builtin_fmaf(hi, __uint_as_float(wv[e][c] & 0xffff0000u), s[e]);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[e] = wave_sum(s[e]);
        if (lane == j[e]) z[i] = s[e];
      }
    }
  }
}

__device__ __forceinline__ void entry_rows(const HeadArgs& a, const int (&at)[kEntryLanes],
                                           int (&row)[kEntryLanes]) {
#pragma unroll
  for (int i = 0; i < kEntryLanes; ++i) {
    const int64_t rel = at[i] < 0 ? -1 : (int64_t)at[i] - a.first;
    row[i] = rel >= 0 && rel < a.V ? (int)rel : -1;
  }
}

// sum over the entries of q (log q + lse - c z), in 64 bits (see the join).
__device__ __forceinline__ float entry_loss(const HeadArgs& a, const float (&q)[kEntryLanes],
                                            const float (&lq)[kEntryLanes], const float (&z)[kEntryLanes],
                                            double lse) {
  double loss = 0.0;
#pragma unroll
  for (int i = 0; i < kEntryLanes; ++i)
    if (q[i] > 0.f) loss += (double)q[i] * ((double)lq[i] + (lse - (double)z[i] * a.c));
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) loss += __shfl_xor(loss, d);
  return (float)loss;
}

// Distillation: the logits of a token's entries and its loss.  One wave per token.
// Bound by the gather of w's rows: 7376 tokens of 64 entries, D = 2048, 313 us,
// 6.2 TB/s of them (the last-level cache's share included).
__global__ __launch_bounds__(256) void head_entries_kernel(const HeadArgs a, const double* lse64) {
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (t >= a.T) return;
  float q[kEntryLanes], lq[kEntryLanes], z[kEntryLanes];
  int at[kEntryLanes], row[kEntryLanes];
  const bool any = teacher_row(a, t, lane, q, lq, at);
  entry_rows(a, at, row);
  entry_logits(a, t, lane, row, 0, 1, z);
#pragma unroll
  for (int i = 0; i < kEntryLanes; ++i)
    if (64 * i + lane < a.k) a.logits[t * a.k + 64 * i + lane] = z[i];
  const float loss = any ? entry_loss(a, q, lq, z, lse64[t]) : 0.f;
  if (lane == 0) a.loss[t] = loss;
}

// Both in one for short batches: a workgroup per token, its waves sharing the
// parts and then the entries.
__global__ __launch_bounds__(512) void head_finish_kernel(const HeadArgs a, const int32_t parts, const Plan* plan_at,
                                                          const int32_t* pos, const float2* part) {
  __shared__ float2 got[8];
  __shared__ float zs[64 * kEntryLanes];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = blockIdx.x;
  float q[kEntryLanes], lq[kEntryLanes], z[kEntryLanes];
  int at[kEntryLanes], row[kEntryLanes];
  const bool any = teacher_row(a, t, lane, q, lq, at);
  const int count = plan_at != nullptr ? parts_of(a.V, *plan_at) : parts;
  const int p = !any ? -1 : pos != nullptr ? pos[t] : (int)t;
  float top = -INFINITY, sum = 0.f;
  auto join = [&](const float2 v) {
    const float m = fmaxf(top, v.x), ref = m == -INFINITY ? 0.f : m;
    sum = sum * __builtin_amdgcn_exp2f((top - ref) * a.scale) + v.y * __builtin_amdgcn_exp2f((v.x - ref) * a.scale);
    top = m;
  };
  if (p >= 0) {
#pragma unroll 4
    for (int i = threadIdx.x; i < count; i += 512) join(part[(int64_t)i * a.T + p]);
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) join(make_float2(__shfl_xor(top, d), __shfl_xor(sum, d)));
  if (lane == 0) got[wave] = make_float2(top, sum);
  if (threadIdx.x < 64 * kEntryLanes) zs[threadIdx.x] = 0.f;
  __syncthreads();
  entry_rows(a, at, row);
  entry_logits(a, t, lane, row, wave, 8, z);
#pragma unroll
  for (int i = 0; i < kEntryLanes; ++i)
    if (z[i] != 0.f) zs[64 * i + lane] = z[i];           // (each entry of one wave)
  __syncthreads();
  if (wave != 0) return;
  for (int w = 1; w < 8; ++w) join(got[w]);
  const double lse = any ? (double)top * a.c + log((double)sum) : 0.0;
#pragma unroll
  for (int i = 0; i < kEntryLanes; ++i) {
    z[i] = zs[64 * i + lane];
    if (64 * i + lane < a.k) a.logits[t * a.k + 64 * i + lane] = z[i];
  }
  const float loss = any ? entry_loss(a, q, lq, z, lse) : 0.f;
  if (lane == 0) {
    a.loss[t] = loss;
    a.lse[t] = (float)lse;
  }
}

// Distillation, backward: dz at the entries of a token, from their logits.
// entry[j]: its place in w (-1: none here, or told by an earlier entry of the
// same place, whose q then holds both), value[j]: a p - b q, in 16 bits.  With
// dz (the whole vocabulary's) they are put there at once, with `second` what the
// rounding left as well, *second rows on.
__global__ __launch_bounds__(256) void head_entry_values_kernel(const HeadArgs a, const int32_t* pos,
                                                                const Token* token, const float* top,
                                                                int32_t* entry, uint16_t* value,
                                                                int64_t rows_t, uint16_t* dz, const int32_t* second) {
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (t >= a.T) return;
  const int p = pos[t];
  float q[kEntryLanes], lq[kEntryLanes];
  int at[kEntryLanes];
  const bool any = teacher_row(a, t, lane, q, lq, at);
  float sum[kEntryLanes];
  bool early[kEntryLanes];
#pragma unroll
  for (int i = 0; i < kEntryLanes; ++i) sum[i] = 0.f, early[i] = false;
  if (any) {
#pragma unroll
    for (int o = 0; o < kEntryLanes; ++o)
      for (int l = 0; l < 64 && 64 * o + l < a.k; ++l) {
        const int v = __builtin_amdgcn_readlane(at[o], l);
        const float w = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(q[o]), l));
#pragma unroll
        for (int i = 0; i < kEntryLanes; ++i)
          if (at[i] == v) {
            sum[i] += w;
            early[i] |= 64 * o + l < 64 * i + lane;
          }
      }
  }
#pragma unroll
  for (int i = 0; i < kEntryLanes; ++i) {
    const int j = 64 * i + lane;
    if (j >= a.k) continue;
    int where = -1;
    uint32_t bits = 0, rest = 0;
    if (any && at[i] >= 0 && !early[i] && at[i] >= a.first && at[i] - a.first < a.V) {
      where = (int)(at[i] - a.first);
      const Token k = token[p];
      const float pr = __builtin_amdgcn_exp2f(below(a.logits_in[t * a.k + j], k.lse) * a.scale);
      const float v = k.a * top[1] * pr - k.b * top[1] * sum[i];
      bits = pack2(v, 0.f) & 0xffffu;
      rest = pack2(v - low_half(bits), 0.f) & 0xffffu;
    }
    if (dz != nullptr) {
      if (where >= 0) {
        uint16_t* to = dz + ((int64_t)(where >> 6) * rows_t + p) * 64 + (where & 63);
        *to = (uint16_t)bits;
        if (second != nullptr) to[64 * (int64_t)*second] = (uint16_t)rest;
      }
    } else {
      entry[t * a.k + j] = where;
      value[t * a.k + j] = (uint16_t)bits;
    }
  }
}

// These values into the piece [v0, v0 + count) of dz.
__global__ __launch_bounds__(256) void head_entry_store_kernel(const int32_t* pos, const int32_t* entry,
                                                               const uint16_t* value, int64_t total,
                                                               int32_t k, int32_t v0, int32_t count,
                                                               int64_t rows_t, uint16_t* dz) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int v = entry[i];
    if (v < v0 || v - v0 >= count) continue;
    const int64_t p = pos[i / k], c = v - v0;
    dz[((c >> 6) * rows_t + p) * 64 + (c & 63)] = value[i];
  }
}

// dx[t] = top sum over the parts of dx32[part][place], one rounding; zeros for
// tokens that do not count.  From workgroup dx_blocks on: dw, where its
// reduction was in parts.  A thread per 8 columns.
struct SumArgs {
  const int32_t* pos;
  const int32_t* n;
  const Plan* plans;
  const float* top;
  const float* dx32;
  const float* dw32;
  uint16_t* dx;
  uint16_t* dw;
  int64_t T, V, rows_t;
  int32_t D, pairs;            // pairs of stages of dx's reduction
  int32_t pair;                // every token's dx is in two rows
  unsigned dx_blocks, dw_blocks;
};
__global__ __launch_bounds__(256) void head_sum_kernel(const SumArgs a) {
  const bool w = blockIdx.x >= a.dx_blocks;
  const float scale = a.top[0];
  int splits;
  if (w) {
    splits = min(a.plans[kPlanDw].splits, max(1, (*a.n + 127) >> 7));
    if (splits <= 1) return;                             // it is written
  } else {
    splits = min(a.plans[kPlanDx].splits, a.pairs);
  }
  const int64_t per_row = a.D / 8, total = (w ? a.V : a.T) * per_row;
  const int64_t step = (int64_t)(w ? a.dw_blocks : a.dx_blocks) * 256;
  const float* parts = w ? a.dw32 : a.dx32;
  const int64_t part = (w ? a.V : a.rows_t) * a.D;
  for (int64_t i = (int64_t)(blockIdx.x - (w ? a.dx_blocks : 0)) * 256 + threadIdx.x; i < total; i += step) {
    const int64_t r = i / per_row;
    const int d = 8 * (int)(i - r * per_row);
    const int64_t p = w ? r : a.pos[r];
    u32x4 v = {0, 0, 0, 0};
    if (p >= 0) {
      float s[8] = {};
#pragma unroll 4
      for (int k = 0; k < splits; ++k) {
        const float4* f = reinterpret_cast<const float4*>(parts + k * part + p * a.D + d);
        const float4 lo = f[0], hi = f[1];
        s[0] += lo.x; s[1] += lo.y; s[2] += lo.z; s[3] += lo.w;
        s[4] += hi.x; s[5] += hi.y; s[6] += hi.z; s[7] += hi.w;
        if (a.pair && !w) {
          const float4* g = reinterpret_cast<const float4*>(parts + k * part + (p + *a.n) * a.D + d);
          const float4 lo2 = g[0], hi2 = g[1];
          s[0] += lo2.x; s[1] += lo2.y; s[2] += lo2.z; s[3] += lo2.w;
          s[4] += hi2.x; s[5] += hi2.y; s[6] += hi2.z; s[7] += hi2.w;
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = pack2(s[2 * e] * scale, s[2 * e + 1] * scale);
    }
    *reinterpret_cast<u32x4*>((w ? a.dw : a.dx) + r * a.D + d) = v;
  }
}

// The weights' gradient of no tokens.
__global__ __launch_bounds__(256) void head_zero_kernel(u32x4* out, int64_t count) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (int64_t)gridDim.x * 256)
    out[i] = u32x4{0, 0, 0, 0};
}

// -------------------------------------------------------------------- host --

int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

// Parts of a workspace, each on a 256-byte boundary.
struct Parts {
  int64_t size = 0;
  char* base = nullptr;
  template <class X>
  X* take(int64_t count) {
    X* p = base != nullptr ? reinterpret_cast<X*>(base + size) : nullptr;
    size += up(count * (int64_t)sizeof(X), 256);
    return p;
  }
};

struct Common {
  uint8_t* flag;
  int32_t* pos;
  int32_t* rows;
  int32_t* n;
  Plan* plans;
  Token* token;
  uint16_t* xc;
};
Common take_common(Parts& w, int64_t T, int64_t D, int64_t rows) {
  Common c;
  c.flag = w.take<uint8_t>(T);
  c.pos = w.take<int32_t>(T);
  c.rows = w.take<int32_t>(T);
  c.n = w.take<int32_t>(2);
  c.plans = w.take<Plan>(kPlans);
  c.token = w.take<Token>(T);
  c.xc = w.take<uint16_t>(rows * up(D, 64));
  return c;
}

// Batches of so few tokens that there is little to leave out: the forward
// takes them as they are, without the three passes before the product.
constexpr int64_t kAsTheyAre = 128;

struct Forward {
  Common c;
  float2* part;
  float* logit;
  double* lse64;
};

Forward take_forward(Parts& w, int64_t T, int64_t V, int64_t D) {
  Forward f{};
  if (T > kAsTheyAre) f.c = take_common(w, T, D, T);
  // (plan_of's rows of a tile add up to 256 tiles)
  f.part = w.take<float2>(((V + 255) / 256 + (T <= kFewTokens ? 256 : 0)) * Small::WP * T);
  f.logit = w.take<float>(T);
  f.lse64 = w.take<double>(T);
  return f;
}

// Vocabulary entries of a piece: as many as make 2^28 values of dz (512 MiB),
// whole tiles, at least 4096.
int64_t piece_of(int64_t T, int64_t V) {
  const int64_t most = (int64_t(1) << 28) / up(T, 256) / 256 * 256, all = up(V, 256);
  const int64_t piece = most < 4096 ? 4096 : most;
  return piece < all ? piece : all;
}

struct Backward {
  Common c;
  float* top;
  uint16_t* dz;
  float* dx32;
  float* dw32;
  int32_t* entry;
  uint16_t* value;
  int64_t rows_t, piece;
  int32_t dx_splits, dw_splits;
  bool pair;
};

// Batches of so few tokens that a tile of the gradients' products has room for
// each twice take dz as two 16-bit values, the second what the first's rounding
// left.  With one or two tokens a few of dz's values make up the gradients, and
// nothing averages their roundings (relative error of dx and dw, 1 or 2 tokens:
// 0.0025 to 0.0034 with one value, 0.0017 with two, which is the results' own
// rounding); from some ten tokens on one value gives 0.0019 to 0.0024.  It costs
// stores and products: 14 x 90642 x 3312 477 -> 494 us.
constexpr int64_t kPairs = 64;

// Most parts of the gradients' reductions: of at least 256 steps each, 256 MiB
// in all; of dw's only where its tiles are few and the vocabulary one piece.
int32_t dx_splits(int64_t T, int64_t D, int64_t piece) {
  int64_t s = (int64_t(1) << 26) / (up(T, 256) * D);
  if (s > piece / 256) s = piece / 256;
  return (int32_t)(s < 1 ? 1 : s > 64 ? 64 : s);
}
int32_t dw_splits(int64_t T, int64_t V, int64_t D, int64_t piece) {
  if (V > piece || ((D + 255) / 256) * ((V + 127) / 128) > 128) return 1;
  int64_t s = (int64_t(1) << 26) / (V * D);
  if (s > T / 256) s = T / 256;
  return (int32_t)(s < 1 ? 1 : s > 64 ? 64 : s);
}

Backward take_backward(Parts& w, int64_t T, int64_t V, int64_t D, int64_t k) {
  Backward b{};
  b.piece = piece_of(T, V);
  b.pair = T <= kPairs && V <= b.piece;
  b.c = take_common(w, T, D, b.pair ? 2 * T : T);
  b.rows_t = up(T, 256);
  b.dx_splits = dx_splits(T, D, b.piece);
  b.dw_splits = dw_splits(T, V, D, b.piece);
  b.top = w.take<float>(2);
  b.dz = w.take<uint16_t>(b.rows_t * b.piece);
  b.dx32 = w.take<float>(b.dx_splits * b.rows_t * D);
  if (b.dw_splits > 1) b.dw32 = w.take<float>(b.dw_splits * V * D);
  if (V > b.piece) {
    b.entry = w.take<int32_t>(T * k);
    b.value = w.take<uint16_t>(T * k);
  }
  return b;
}

unsigned blocks_for(int64_t items, int64_t per, int64_t most) {
  const int64_t b = (items + per - 1) / per;
  return (unsigned)(b < 1 ? 1 : b > most ? most : b);
}

#define MG_RUN(call)                       \
  do {                                     \
    const int err_ = (call);               \
    if (err_ != hipSuccess) return err_;   \
  } while (0)

// Lets a kernel have more than 64 KiB of LDS, once per device (`done`, a bit
// for each; past 64 devices every time).
template <class F>
hipError_t allow_lds(F* kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  hipError_t err = hipGetDevice(&dev);
  if (err != hipSuccess) return err;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return hipSuccess;
  err = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (err == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return err;
}
template <int EPI>
int run_nt(const NtArgs& a, hipStream_t s) {
  static std::atomic<uint64_t> done{0};
  MG_RUN(allow_lds(&nt_kernel<EPI>, Large::LDS, done));
  hipLaunchKernelGGL(nt_kernel<EPI>, dim3(256), dim3(512), Large::LDS, s, a);
  return hipGetLastError();
}

// Whether the logits of these sizes go in tiles of 64 x 64: where one round of
// them takes the place of fewer, longer ones.  (Forward in us by large or small
// tiles and by these, 1 to 256 tokens: 256 tiles 10.0 -> 7.8 at D = 256, 48 ->
// 26 at D = 4096; 512 tiles 11.8 -> 12.6 at D = 256, 54 -> 52 at D = 4096; 1024
// tiles 12.5 -> 19.7 and 60 -> 93.)
bool tile64(int64_t np, int64_t nq, int64_t K) {
  const int64_t tiles = ((np + 255) / 256 * 4) * ((nq + 63) / 64);
  return tiles <= 256 || (tiles <= 512 && K >= 1536);
}
template <int EPI>
int run_tile64(const NtArgs& a, hipStream_t s) {
  constexpr int kLds = 8 * 16 * 64 * 16;
  static std::atomic<uint64_t> done{0};
  MG_RUN(allow_lds(&tile64_kernel<EPI>, kLds, done));
  hipLaunchKernelGGL(tile64_kernel<EPI>, dim3((unsigned)((a.np + 255) / 256 * 4), (unsigned)((a.nq + 63) / 64)),
                     dim3(512), kLds, s, a);
  return hipGetLastError();
}

// Which tokens count, their order and, packed, their rows of x.
int place_tokens(const HeadArgs& a, const Common& c, int64_t piece, int32_t dx_splits, int32_t dw_splits,
                 bool pair, float* top, hipStream_t s) {
  PlaceArgs o{};
  if (a.index != nullptr && a.T > kPlaceFlags) {
    hipLaunchKernelGGL(head_flags_kernel, dim3((unsigned)((a.T + 3) / 4)), dim3(256), 0, s, a, c.flag);
    MG_RUN(hipGetLastError());
    o.flag = c.flag;
  }
  const bool both = a.T <= 256 * kPlaceList;
  o.pos = c.pos;
  o.rows = c.rows;
  o.n = c.n;
  o.token = c.token;
  o.plans = c.plans;
  o.top = top;
  o.pack = both ? c.xc : nullptr;
  o.ld = (int32_t)up(a.D, 64);
  o.piece = (int32_t)piece;
  o.dx_splits = dx_splits;
  o.dw_splits = dw_splits;
  o.pair = pair;
  const dim3 grid(both ? blocks_for(a.T, 16, 256) : 1);
  if (a.T <= kPlaceFlags) hipLaunchKernelGGL(head_place_kernel<1>, grid, dim3(1024), 0, s, a, o);
  else hipLaunchKernelGGL(head_place_kernel<8>, grid, dim3(1024), 0, s, a, o);
  MG_RUN(hipGetLastError());
  if (both) return hipSuccess;
  hipLaunchKernelGGL(head_pack_kernel, dim3(blocks_for(a.T, 4, 2048)), dim3(256), 0, s, a.x, c.rows, c.n,
                     (int32_t)a.T, (int32_t)a.D, c.xc, o.ld);
  return hipGetLastError();
}

// The logits' product, from vocabulary entry v0 on.
NtArgs logits_args(const HeadArgs& a, const Common& c, int64_t v0, int64_t count) {
  NtArgs g{};
  g.P = {a.w + v0 * a.D, (uint32_t)a.D * 2u, 128u};
  // x's rows packed, or as they are where all count and every row starts on 128
  // bytes: a staged row that crosses a line is two reads of L2 each time
  const bool packed = c.xc != nullptr;
  g.Q = {c.xc, (uint32_t)(packed ? up(a.D, 64) : a.D) * 2u, 128u};
  g.x_all = packed && a.D % 64 != 0 ? c.xc : a.x;
  g.n = c.n;
  g.plan_at = c.plans != nullptr ? c.plans + kPlanLogits : nullptr;
  g.np = (int32_t)count;
  g.nq = g.tokens = (int32_t)a.T;
  g.K = g.D = (int32_t)a.D;
  g.first = (int32_t)v0;
  g.target_first = a.first;
  g.gq = 8;
  g.scale = a.scale;
  g.token = c.token;
  return g;
}

}  // namespace

int64_t head_workspace_bytes(int64_t T, int64_t V, int64_t D) {
  Parts w;
  take_forward(w, T, V, D);
  return w.size;
}

int64_t head_bwd_workspace_bytes(int64_t T, int64_t V, int64_t D, int32_t k) {
  Parts w;
  take_backward(w, T, V, D, k);
  return w.size;
}

int launch_head(const HeadArgs& a, hipStream_t s) {
  Parts w;
  w.base = static_cast<char*>(a.workspace);
  const Forward f = take_forward(w, a.T, a.V, a.D);
  if (f.c.pos != nullptr) MG_RUN(place_tokens(a, f.c, a.V, 1, 1, false, nullptr, s));
  NtArgs g = logits_args(a, f.c, 0, a.V);
  g.targets = f.c.pos != nullptr ? nullptr : a.targets;
  g.part = f.part;
  g.logit = a.index == nullptr ? f.logit : nullptr;
  const int tp = (int)((a.V + 255) / 256);
  int parts;
  if (tile64(a.V, a.T, a.D)) {
    parts = parts_before(tp, 0);
    g.plan_at = nullptr;
    MG_RUN(run_tile64<kStats>(g, s));
  } else {
    g.plan = plan_of(kStats, (int)a.V, (int)a.T, (int)a.D, a.T <= kFewTokens).plan;
    parts = parts_of(a.V, g.plan);
    MG_RUN(run_nt<kStats>(g, s));
  }
  if (a.index != nullptr && a.T < 1024) {
    hipLaunchKernelGGL(head_finish_kernel, dim3((unsigned)a.T), dim3(512), 0, s, a, parts, g.plan_at, f.c.pos,
                       f.part);
    return hipGetLastError();
  }
  if (a.T < 1024)
    hipLaunchKernelGGL((head_join_kernel<1, 256>), dim3((unsigned)a.T), dim3(256), 0, s, a, parts, g.plan_at,
                       f.c.pos, f.part, f.logit, f.lse64);
  else
    hipLaunchKernelGGL((head_join_kernel<16, 1024>), dim3((unsigned)((a.T + 15) / 16)), dim3(1024), 0, s, a,
                       parts, g.plan_at, f.c.pos, f.part, f.logit, f.lse64);
  MG_RUN(hipGetLastError());
  if (a.index != nullptr) {
    hipLaunchKernelGGL(head_entries_kernel, dim3((unsigned)((a.T + 3) / 4)), dim3(256), 0, s, a, f.lse64);
    MG_RUN(hipGetLastError());
  }
  return hipSuccess;
}

int launch_head_bwd(const HeadArgs& a, hipStream_t s) {
  if (a.T == 0) {
    hipLaunchKernelGGL(head_zero_kernel, dim3(blocks_for(a.V * (a.D / 8), 256, 4096)), dim3(256), 0, s,
                       reinterpret_cast<u32x4*>(a.dw), a.V * (a.D / 8));
    return hipGetLastError();
  }
  Parts w;
  w.base = static_cast<char*>(a.workspace);
  const Backward b = take_backward(w, a.T, a.V, a.D, a.index != nullptr ? a.k : 0);
  const int32_t T = (int32_t)a.T, D = (int32_t)a.D;
  const int64_t entries = a.index != nullptr ? a.T * a.k : 0;
  const bool one = a.V <= b.piece;
  MG_RUN(place_tokens(a, b.c, b.piece, b.dx_splits, b.dw_splits, b.pair, b.top, s));
  auto entry_values = [&](uint16_t* dz) {
    hipLaunchKernelGGL(head_entry_values_kernel, dim3((unsigned)((a.T + 3) / 4)), dim3(256), 0, s, a, b.c.pos,
                       b.c.token, b.top, b.entry, b.value, b.rows_t, dz, b.pair ? b.c.n : nullptr);
    return (int)hipGetLastError();
  };
  if (entries > 0 && !one) MG_RUN(entry_values(nullptr));
  for (int64_t v0 = 0; v0 < a.V; v0 += b.piece) {
    const int64_t count = a.V - v0 < b.piece ? a.V - v0 : b.piece;
    NtArgs g = logits_args(a, b.c, v0, count);
    g.top = b.top;
    g.dz = b.dz;
    g.rows_t = b.rows_t;
    const bool small = tile64(count, T, D);
    if (b.pair) MG_RUN(small ? run_tile64<kDzPair>(g, s) : run_nt<kDzPair>(g, s));
    else MG_RUN(small ? run_tile64<kDz>(g, s) : run_nt<kDz>(g, s));
    if (entries > 0 && one) {
      MG_RUN(entry_values(b.dz));
    } else if (entries > 0) {
      hipLaunchKernelGGL(head_entry_store_kernel, dim3(blocks_for(entries, 256, 2048)), dim3(256), 0, s,
                         b.c.pos, b.entry, b.value, entries, a.k, (int32_t)v0, (int32_t)count, b.rows_t, b.dz);
      MG_RUN(hipGetLastError());
    }
    const Operand dz = {b.dz, 128u, (uint32_t)(b.rows_t * 128)};
    NtArgs h{};
    h.n = b.c.n + 1;
    h.tokens = T;
    h.D = D;
    h.gq = 4;
    h.top = b.top;
    h.rows_t = b.rows_t;
    NtArgs x = h;
    x.P = dz;
    x.Q = {a.w + v0 * a.D, (uint32_t)D * 2u, 128u};
    x.plan_at = b.c.plans + kPlanDx;
    x.np = T;
    x.nq = D;
    x.K = (int32_t)count;
    x.add = v0 > 0;
    x.dx = a.dx != nullptr ? b.dx32 : nullptr;
    h.P = g.Q;
    h.x_all = b.pair ? b.c.xc : g.x_all;
    h.Q = dz;
    h.plan_at = b.c.plans + kPlanDw;
    h.np = D;
    h.nq = (int32_t)count;
    h.K = T;
    h.dw = a.dw != nullptr ? a.dw + v0 * a.D : nullptr;
    h.dw_parts = b.dw32;
    static std::atomic<uint64_t> done{0};
    MG_RUN(allow_lds(&grads_kernel, Large::LDS, done));
    hipLaunchKernelGGL(grads_kernel, dim3(256), dim3(512), Large::LDS, s, x, h);
    MG_RUN(hipGetLastError());
  }
  SumArgs o{};
  o.pos = b.c.pos;
  o.n = b.c.n;
  o.plans = b.c.plans;
  o.top = b.top;
  o.dx32 = b.dx32;
  o.dw32 = b.dw32;
  o.dx = a.dx;
  o.dw = a.dw;
  o.pair = b.pair;
  o.T = a.T;
  o.V = a.V;
  o.rows_t = b.rows_t;
  o.D = D;
  o.pairs = (int32_t)(((one ? a.V : b.piece) + 127) / 128);
  if (a.dx != nullptr) o.dx_blocks = blocks_for(a.T * (D / 8), 256, 4096);
  if (a.dw != nullptr && b.dw_splits > 1) o.dw_blocks = blocks_for(a.V * (D / 8), 256, 4096);
  if (o.dx_blocks + o.dw_blocks == 0) return hipSuccess;
  hipLaunchKernelGGL(head_sum_kernel, dim3(o.dx_blocks + o.dw_blocks), dim3(256), 0, s, o);
  return hipGetLastError();
}

}  // namespace mg
