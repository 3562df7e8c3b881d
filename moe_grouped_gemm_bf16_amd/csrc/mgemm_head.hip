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
// not kept) against one forward.  All four run on one kernel, nt_kernel below:
// C[q, p] = sum_r Q[q, r] P[p, r] with both operands contiguous along r.
//   logits (forward, backward)  P = w rows, Q = x rows, r = hidden column
//   input gradient              P = dz rows (tokens), Q = w^T rows, r = vocabulary
//   weight gradient             P = dz^T rows (vocabulary), Q = x^T rows, r = token
// The forward's epilogue turns a tile of logits into one (maximum, sum of
// exponentials) per token and 128 vocabulary entries; the backward's turns it
// into dz, in 16 bits, for a piece of the vocabulary at a time.  dz, its
// transpose and the transposes of x and of w's piece lie in panels of 64
// reduction steps, [r / 64][row][64]: a staged row is 128 contiguous bytes and
// a tile's rows follow each other, whatever the widths.
//
// Tokens that do not count (no target, no teacher's entry) are left out before
// the products: rows[] lists the others, x is packed by it (not if all count).
// The number that count stays on the device.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "mgemm_launch.h"

namespace mg {
namespace {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) const bf16x8 lds_frag;

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
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
// are the stage loop's own.
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

template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// One operand of a product: row i at base + i stride, reduction step k at
// (k / 64) kstep + 2 (k % 64) of the row.
struct Operand {
  const void* base;
  uint32_t stride;      // bytes between rows
  uint32_t kstep;       // bytes between blocks of 64 reduction steps
};

// A token that counts, as the backward's epilogue takes it.
struct Token {
  float lse2;           // lse log2(e)
  float a;              // weight of the probabilities
  float b;              // weight of the entries
  int32_t target;       // vocabulary entry of w, -1 for none or several (written apart)
};

enum { kStats = 0, kDz = 1, kDx = 2, kDw = 3 };

struct NtArgs {
  Operand P, Q;
  const void* Q_all;        // logits: x itself, taken when all tokens count
  const int32_t* n;         // device: tokens that count
  int32_t np, nq, K;        // rows of P and of Q and reduction steps; those that are
                            // tokens hold their upper bound
  int32_t tokens;           // that bound: T
  int32_t first;            // logits: vocabulary entry of P's row 0
  int32_t gq;               // tiles along Q that run beside each other
  int32_t splits;           // input gradient: parts of the reduction
  int32_t add;              // input gradient: add to what is there
  float scale;              // logits: c log2(e)
  float2* part;             // forward: [2 tiles along P][T] (maximum, sum)
  float* logit;             // forward: logit of a token's target, or NULL
  const Token* token;       // logits: per counting token
  const float* top;         // backward: [2], largest |a|, |b| and its inverse
  uint16_t* dz;             // [V' / 64][T'][64] (or NULL: not wanted)
  uint16_t* dzt;            // [T' / 64][V'][64] (or NULL)
  int64_t rows_t, rows_v;   // T', V' of these
  float* dx;                // [splits][T'][D] fp32
  uint16_t* dw;             // [V, D]
  int32_t D;
};

// Tile of BP x BQ outputs, WP x WQ waves of (64 MH) x 64 each, 64 reduction
// steps a stage, two stages in LDS.  Every operand tile is staged as two
// units, the rows of the waves' first halves and those of their second, so a
// stage is the four products of a P half and a Q half, and a unit can be
// refilled as soon as its fragments are in registers, while the rest of the
// stage is still multiplied: a load has five of the eight phases of two stages
// (about 1.3 us of 256 x 256 tiles) before its data are read.
template <int MH_, int WP_, int WQ_>
struct Cfg {
  static constexpr int MH = MH_, WP = WP_, WQ = WQ_;
  static constexpr int BP = WP * 64 * MH, BQ = WQ * 64;
  static constexpr int UP = BP / 2 * 128, UQ = BQ / 2 * 128;     // bytes of a unit
  static constexpr int SP = BP / 2 / 64, SQ = BQ / 2 / 64;       // loads of a unit per wave
  static constexpr int LDS = 4 * (UP + UQ);
  static_assert(WP * WQ == 8 && SP >= 1 && SQ >= 1, "eight waves");
  static_assert(4 * UP <= 65536 && 4 * UQ <= 65536, "read offsets of 16 bits");
};
typedef Cfg<2, 2, 4> Large;      // 256 x 256
typedef Cfg<1, 4, 2> Small;      // 256 x 128

template <class C>
struct Core {
  f32x16 acc[2 * C::MH][2];
  bf16x8 A0[C::MH][4], A1[C::MH][4], B0[4], B1[4];
  uint32_t aP[4], aQ[4];               // fragment addresses by slice of 16 steps
  uint32_t rowP, rowQ, maxP, maxQ, chunk;
  uint64_t baseP, baseQ;
  uint32_t lds0, live;
  uint32_t strideP, strideQ, kstepP, kstepQ;
  int wave, K, kd;

  // LDS rows of 128 bytes in 16-byte chunks; chunk c of row r lies at c ^ (r % 8),
  // so 32 rows read at one chunk touch every bank group equally often.
  __device__ __forceinline__ void init(const NtArgs& a, int K_, char* lds) {
    const int lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    lds0 = (uint32_t)(uintptr_t)(lds_char*)lds;
    const int wp = wave / C::WQ, wq = wave % C::WQ, l32 = lane & 31, h = lane >> 5;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const uint32_t c = (uint32_t)(((2 * kk + h) ^ (l32 & 7)) << 4);
      aP[kk] = lds0 + (uint32_t)((wp * 32 * C::MH + l32) * 128) + c;
      aQ[kk] = lds0 + (uint32_t)(4 * C::UP) + (uint32_t)((wq * 32 + l32) * 128) + c;
    }
    K = K_;
    strideP = a.P.stride;
    strideQ = a.Q.stride;
    kstepP = a.P.kstep;
    kstepQ = a.Q.kstep;
    // row of a unit -> row of the tile: half h of wave w holds rows
    // (2 w + h) 32 MH .. of P, (2 w + h) 32 .. of Q
    const int uP = 8 * C::SP * wave + (lane >> 3), uQ = 8 * C::SQ * wave + (lane >> 3);
    rowP = (uint32_t)((uP / (32 * C::MH)) * 64 * C::MH + uP % (32 * C::MH)) * strideP;
    rowQ = (uint32_t)((uQ / 32) * 64 + uQ % 32) * strideQ;
    chunk = (uint32_t)(((lane & 7) ^ ((lane >> 3) & 7)) << 4);
  }

  // The tile whose stages the next loads bring: rows from p0 of np, q0 of nq,
  // steps from k0.  Rows past the end repeat the last one (their results are
  // not stored), steps past the end are zeros.  Without a tile nothing is read.
  __device__ __forceinline__ void source(const NtArgs& a, const void* Q, bool live_, int p0, int np,
                                         int q0, int nq, int k0, int K_) {
    maxP = (uint32_t)(min(C::BP, np - p0) - 1) * strideP;
    maxQ = (uint32_t)(min(C::BQ, nq - q0) - 1) * strideQ;
    baseP = reinterpret_cast<uint64_t>(a.P.base) + (uint64_t)p0 * strideP + (uint64_t)(k0 >> 6) * kstepP;
    baseQ = reinterpret_cast<uint64_t>(Q) + (uint64_t)q0 * strideQ + (uint64_t)(k0 >> 6) * kstepQ;
    live = live_ ? 0x7fffffffu : 0u;
    K = K_;
    kd = 0;
  }
  __device__ __forceinline__ void advance() {
    baseP += 2 * (uint64_t)kstepP;
    baseQ += 2 * (uint64_t)kstepQ;
    kd += 128;
  }

  template <bool IsQ, int HALF, int BUF>
  __device__ __forceinline__ void load() {
    constexpr int S = IsQ ? C::SQ : C::SP;
    const i32x4 rsrc = make_rsrc(reinterpret_cast<const void*>(IsQ ? baseQ : baseP), live);
    const bool in = (int)(chunk >> 1) + kd + BUF * 64 < K;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      // segment s of the wave: 8 unit rows further
      const uint32_t add = (uint32_t)(8 * s + (IsQ ? 32 : 32 * C::MH) * HALF) * (IsQ ? strideQ : strideP);
      const uint32_t r = min((IsQ ? rowQ : rowP) + add, IsQ ? maxQ : maxP);
      const uint32_t off = (r + chunk + BUF * (IsQ ? kstepQ : kstepP)) | (in ? 0u : kOOB);
      dma16(rsrc, lds0 + (IsQ ? 4u * C::UP + (2u * BUF + HALF) * C::UQ : (2u * BUF + HALF) * C::UP) +
                      (uint32_t)(wave * S + s) * 1024u, off);
    }
  }
  template <int HALF, int BUF>
  __device__ __forceinline__ void readP(bf16x8 (&f)[C::MH][4]) {
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int i = 0; i < C::MH; ++i)
        f[i][kk] = *(lds_frag*)(uintptr_t)(aP[kk] + (2 * BUF + HALF) * C::UP + i * 4096);
  }
  template <int HALF, int BUF>
  __device__ __forceinline__ void readQ(bf16x8 (&f)[4]) {
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
      f[kk] = *(lds_frag*)(uintptr_t)(aQ[kk] + (2 * BUF + HALF) * C::UQ);
  }
  template <int HP, int HQ>
  __device__ __forceinline__ void mul(const bf16x8 (&A)[C::MH][4], const bf16x8 (&B)[4]) {
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int i = 0; i < C::MH; ++i)
        acc[C::MH * HP + i][HQ] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            A[i][kk], B[kk], acc[C::MH * HP + i][HQ], 0, 0, 0);
  }
  // Reads between the products, one for one.
  template <int R>
  __device__ __forceinline__ void mix() {
#pragma unroll
    for (int i = 0; i < 4 * C::MH; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if (i < R) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
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
    for (int i = 0; i < 2 * C::MH; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = f32x16{};
  }
  __device__ __forceinline__ void start() {
    load<false, 0, 0>(); load<true, 0, 0>(); load<true, 1, 0>(); load<false, 1, 0>();
    load<false, 0, 1>(); load<true, 1, 1>(); load<true, 0, 1>(); load<false, 1, 1>();
    edge<3 * C::SP + 3 * C::SQ>();
    readP<0, 0>(A0);
    readQ<0, 0>(B0);
    edge<kFlight>();
    advance();
  }
  // Two stages, eight phases: each multiplies one pair of halves, reads the
  // half that a later phase needs into registers that are free, and refills
  // the unit that was read two phases before (of the stages 128 steps on).
  __device__ __forceinline__ void pair() {
    constexpr int RP = 4 * C::MH, RQ = 4;
    load<false, 0, 0>(); readQ<1, 0>(B1); mul<0, 0>(A0, B0); mix<RQ>();
    load<true, 0, 0>();  readP<1, 0>(A1); mul<0, 1>(A0, B1); mix<RP>(); edge<kFlight>();
    load<true, 1, 0>();  readP<0, 1>(A0); mul<1, 1>(A1, B1); mix<RP>();
    load<false, 1, 0>(); readQ<1, 1>(B1); mul<1, 0>(A1, B0); mix<RQ>(); edge<kFlight>();
    load<false, 0, 1>(); readQ<0, 1>(B0); mul<0, 1>(A0, B1); mix<RQ>();
    load<true, 1, 1>();  readP<1, 1>(A1); mul<0, 0>(A0, B0); mix<RP>(); edge<kFlight>();
    load<true, 0, 1>();  readP<0, 0>(A0); mul<1, 0>(A1, B0); mix<RP>();
    load<false, 1, 1>(); readQ<0, 0>(B0); mul<1, 1>(A1, B1); mix<RQ>(); edge<kFlight>();
    advance();
  }
};

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}

// 4 x 4 transpose over the four lanes of a quad: lane i brings column i of
// four rows as (row 0, row 1), (row 2, row 3) and gets row i of four columns.
__device__ __forceinline__ u32x2 quad_transpose(uint32_t lo, uint32_t hi, int lane) {
  const bool up = lane & 2;
  const uint32_t send = up ? lo : hi, own = up ? hi : lo;
  const uint32_t recv = (uint32_t)__builtin_amdgcn_mov_dpp((int)send, 0x4E, 0xF, 0xF, true);  // lane ^ 2
  const uint32_t x = up ? recv : own, y = up ? own : recv;   // columns (i & 1), (i & 1) + 2
  const uint32_t rx = (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0xB1, 0xF, 0xF, true);       // lane ^ 1
  const uint32_t ry = (uint32_t)__builtin_amdgcn_mov_dpp((int)y, 0xB1, 0xF, 0xF, true);
  const uint32_t sel = (lane & 1) ? 0x03020706u : 0x05040100u;   // r's bytes are 4-7
  u32x2 v;
  v.x = __builtin_amdgcn_perm(rx, x, sel);
  v.y = __builtin_amdgcn_perm(ry, y, sel);
  return v;
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
// share operand rows in its L2.
template <int EPI, class C>
__global__ __launch_bounds__(512, 2) void nt_kernel(const NtArgs a) {
  extern __shared__ char lds[];
  const int n_tok = a.n != nullptr ? __builtin_amdgcn_readfirstlane(*a.n) : a.tokens;
  const int np = EPI == kDx ? n_tok : a.np;
  const int nq = EPI == kStats || EPI == kDz ? n_tok : a.nq;
  const int K = EPI == kDw ? (n_tok + 7) & ~7 : a.K;
  const int tp = (np + C::BP - 1) / C::BP, tq = (nq + C::BQ - 1) / C::BQ;
  // pairs of stages; an empty reduction takes one of zeros
  const int pairs = max(1, (K + 127) >> 7);
  const int splits = EPI == kDx ? min(a.splits, pairs) : 1;
  const int total = tp * tq * splits, xcd = blockIdx.x & 7, wgs = gridDim.x >> 3;
  const int per = total >> 3, rem = total & 7;
  int id = xcd * per + min(xcd, rem) + (int)(blockIdx.x >> 3);
  const int end = xcd * per + min(xcd, rem) + per + (xcd < rem ? 1 : 0);
  if (id >= end) return;
  const void* Q = (EPI == kStats || EPI == kDz) && n_tok == a.tokens ? a.Q_all : a.Q.base;

  Core<C> c;
  c.init(a, K, lds);
  auto range = [&](const Item& t, int& k0, int& m) {     // pairs [k0, k0 + m) of the item
    if (EPI == kDx) {
      const int each = pairs / splits, more = pairs - each * splits;
      k0 = t.s * each + min(t.s, more);
      m = each + (t.s < more ? 1 : 0);
    } else {
      k0 = 0;
      m = pairs;
    }
  };
  auto aim = [&](const Item& t, bool live) {
    int k0, m;
    range(t, k0, m);
    c.source(a, Q, live, t.ip * C::BP, np, t.iq * C::BQ, nq, 128 * k0, K - 128 * k0);
    return m;
  };
  Item t = item_of(id, tp, tq, a.gq), ahead = t;
  int nid = id;
  int left = aim(t, true) - 1;       // pairs until the loads move on to the next tile
  c.start();
  const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5;
  const int wp = c.wave / C::WQ, wq = c.wave % C::WQ;
  constexpr int MP = 2 * C::MH;

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
    // acc[i][j][4 g + e]: P row 32 i + 8 g + 4 h + e, Q row 32 j + l32 of the wave's part
    const int pw = t.ip * C::BP + wp * 32 * MP, qw = t.iq * C::BQ + wq * 64;

    if constexpr (EPI == kStats) {
      if (t.ip * C::BP + C::BP > np) {
#pragma unroll
        for (int i = 0; i < MP; ++i)
#pragma unroll
          for (int g = 0; g < 16; ++g)
            if (pw + 32 * i + 8 * (g >> 2) + 4 * h + (g & 3) >= np) {
              c.acc[i][0][g] = -INFINITY;
              c.acc[i][1][g] = -INFINITY;
            }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int q = qw + 32 * j + l32;
        if (a.logit != nullptr) {
          const int at = q < nq ? a.token[q].target - pw : -1;
          if (__builtin_amdgcn_ballot_w64(at >= 0 && at < 32 * MP) != 0) {
            const int rel = at - 4 * h;
            float z = 0.f;
#pragma unroll
            for (int i = 0; i < MP; ++i)
#pragma unroll
              for (int g = 0; g < 16; ++g)
                z = rel == 32 * i + 8 * (g >> 2) + (g & 3) ? c.acc[i][j][g] : z;
            if (at >= 0 && at < 32 * MP && ((at >> 2) & 1) == h) a.logit[q] = z;
          }
        }
        float top = c.acc[0][j][0];
#pragma unroll
        for (int i = 0; i < MP; ++i)
#pragma unroll
          for (int g = 0; g < 16; ++g) top = fmaxf(top, c.acc[i][j][g]);
        top = fmaxf(top, __shfl_xor(top, 32)) * a.scale;
        const float ref = top == -INFINITY ? 0.f : top;
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int i = 0; i < MP; ++i)
#pragma unroll
          for (int g = 0; g < 16; g += 2) {
            s0 += __builtin_amdgcn_exp2f(__builtin_fmaf(c.acc[i][j][g], a.scale, -ref));
            s1 += __builtin_amdgcn_exp2f(__builtin_fmaf(c.acc[i][j][g + 1], a.scale, -ref));
          }
        s0 += s1;
        s0 += __shfl_xor(s0, 32);
        if (h == 0 && q < nq)
          a.part[(int64_t)(t.ip * C::WP + wp) * a.tokens + q] = make_float2(top, s0);
      }
    }

    if constexpr (EPI == kDz) {
      const bool edge_p = t.ip * C::BP + C::BP > np;
      const float inv = a.top[1];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int q = qw + 32 * j + l32;
        Token tk = {INFINITY, 0.f, 0.f, -1};
        if (q < nq) tk = a.token[q];
        const float wa = tk.a * inv, wb = tk.b * inv;
        const int at = tk.target < 0 ? -1 : tk.target - a.first - pw;
        const bool told = __builtin_amdgcn_ballot_w64(at >= 0 && at < 32 * MP) != 0;
        // 32 x 64 values of a wave are 64 panel rows of 128 bytes in either order
        char* dz = reinterpret_cast<char*>(a.dz) + ((int64_t)(pw >> 6) * a.rows_t + q) * 128 + 8 * h;
        char* dzt = reinterpret_cast<char*>(a.dzt) +
                    ((int64_t)(qw >> 6) * a.rows_v + pw + 4 * h + (lane & 3)) * 128 + 64 * j + 2 * (l32 & ~3);
#pragma unroll
        for (int i = 0; i < MP; ++i) {
          f32x16 v;
#pragma unroll
          for (int g = 0; g < 16; ++g)
            v[g] = wa * __builtin_amdgcn_exp2f(__builtin_fmaf(c.acc[i][j][g], a.scale, -tk.lse2));
          if (told) {
#pragma unroll
            for (int g = 0; g < 16; ++g) v[g] -= at - 4 * h == 32 * i + 8 * (g >> 2) + (g & 3) ? wb : 0.f;
          }
          if (edge_p) {
#pragma unroll
            for (int g = 0; g < 16; ++g) v[g] = 32 * i + 8 * (g >> 2) + (g & 3) < np - pw - 4 * h ? v[g] : 0.f;
          }
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            // the one rounding of dz: 16-bit operands of the two products
            const uint32_t lo = pack2(v[4 * g], v[4 * g + 1]), hi = pack2(v[4 * g + 2], v[4 * g + 3]);
            if (a.dz != nullptr) *reinterpret_cast<u32x2*>(dz + 64 * (i & 1) + 16 * g) = u32x2{lo, hi};
            if (a.dzt != nullptr)
              *reinterpret_cast<u32x2*>(dzt + 1024 * g) = quad_transpose(lo, hi, lane);
          }
          if (i & 1) dz += a.rows_t * 128;
          dzt += 4096;
          __builtin_amdgcn_sched_barrier(0);      // a block's values at a time: registers
        }
      }
    }

    if constexpr (EPI == kDx) {
      // P = tokens, Q = hidden columns: 32 consecutive columns per half wave
      auto store = [&](auto whole, auto add) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int d = qw + 32 * j + l32;
          const int rows = d < nq ? np - pw - 4 * h : 0;
          float* to = a.dx + ((int64_t)t.s * a.rows_t + pw + 4 * h) * a.D + d;
#pragma unroll
          for (int i = 0; i < MP; ++i) {
            asm volatile("" : "+v"(to));      // a block's addresses at a time: registers
#pragma unroll
            for (int g = 0; g < 16; ++g) {
              if (whole.value || 32 * i + 8 * (g >> 2) + (g & 3) < rows) {
                // (adding: once per element and launch, so there is no order to
                // depend on, and no load to wait for)
                if (add.value) unsafeAtomicAdd(to, c.acc[i][j][g]);
                else *to = c.acc[i][j][g];
              }
              to += (g & 3) == 3 ? 5 * (int64_t)a.D : a.D;
            }
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      };
      const bool whole = t.ip * C::BP + C::BP <= np && t.iq * C::BQ + C::BQ <= nq;
      if (whole && a.add) store(std::true_type{}, std::true_type{});
      else if (whole) store(std::true_type{}, std::false_type{});
      else if (a.add) store(std::false_type{}, std::true_type{});
      else store(std::false_type{}, std::false_type{});
    }

    if constexpr (EPI == kDw) {
      const float scale = a.top[0];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int d = qw + 32 * j + (l32 & ~3);
#pragma unroll
        for (int i = 0; i < MP; ++i)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const u32x2 v = quad_transpose(
                pack2(c.acc[i][j][4 * g] * scale, c.acc[i][j][4 * g + 1] * scale),
                pack2(c.acc[i][j][4 * g + 2] * scale, c.acc[i][j][4 * g + 3] * scale), lane);
            const int p = pw + 32 * i + 8 * g + 4 * h + (lane & 3);
            if (p < np && d < nq) *reinterpret_cast<u32x2*>(a.dw + (int64_t)p * a.D + d) = v;
          }
      }
    }

    id += wgs;
    if (id >= end) break;
    t = ahead;
  }
  wait_vm<0>();       // the loads in flight write this workgroup's LDS
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
    lq[i] = at[i] >= 0 ? (lq[i] - top) * a.inv_temperature : -INFINITY;
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

// Which tokens count (pos[t] = 0, else -1): one thread per token, or, for a
// teacher's entries, one wave.
__global__ __launch_bounds__(256) void head_counts_kernel(const HeadArgs a, int32_t* pos) {
  if (a.index == nullptr) {
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t < a.T) pos[t] = a.targets[t] >= 0 ? 0 : -1;
    return;
  }
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (t >= a.T) return;
  bool any = false;
  for (int j = lane; j < a.k; j += 64)
    any |= a.index[t * a.k + j] >= 0 && teacher_value(a, t * a.k + j) > -INFINITY;
  const bool counts = __builtin_amdgcn_ballot_w64(any) != 0;
  if (lane == 0) pos[t] = counts ? 0 : -1;
}

// The counting tokens in order: pos[t] becomes a token's place (-1 for none),
// rows[place] its token, n their number; per place what the epilogues need,
// and, backward, the largest weight.  One workgroup.
__global__ __launch_bounds__(1024) void head_place_kernel(const HeadArgs a, int32_t* pos, int32_t* rows,
                                                          int32_t* n, Token* token, float* top) {
  __shared__ int counts[16];
  __shared__ float tops[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int base = 0;
  float most = 0.f;
  for (int64_t b = 0; b < a.T; b += 1024) {
    const int64_t t = b + threadIdx.x;
    const bool in = t < a.T && pos[t] >= 0;
    const uint64_t mask = __builtin_amdgcn_ballot_w64(in);
    if (lane == 0) counts[wave] = __popcll(mask);
    __syncthreads();
    int before = base + __popcll(mask & ((1ull << lane) - 1)), all = 0;
    for (int w = 0; w < 16; ++w) {
      const int v = counts[w];
      if (w < wave) before += v;
      all += v;
    }
    if (in) {
      pos[t] = before;
      rows[before] = (int32_t)t;
      Token k = {0.f, 0.f, 0.f, -1};
      if (a.index == nullptr) {
        const int64_t at = (int64_t)a.targets[t] - a.first;
        k.target = at >= 0 && at < a.V ? (int32_t)at : -1;
      }
      if (a.dloss != nullptr) {
        k.lse2 = a.lse_in[t] * kLog2e;
        k.b = a.dloss[t] * a.inv_temperature;
        k.a = a.dlse != nullptr ? k.b + a.dlse[t] : k.b;
        most = fmaxf(most, fmaxf(fabsf(k.a), fabsf(k.b)));
      }
      token[before] = k;
    }
    base += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) *n = base;
  if (top == nullptr) return;
  most = wave_max(most);
  if (lane == 0) tops[wave] = most;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 16; ++w) most = fmaxf(most, tops[w]);
    // a weight past the range where its inverse is a normal number is left as it is
    const bool fit = most > 1e-37f && most < 1e37f;
    top[0] = fit ? most : 1.f;
    top[1] = fit ? 1.f / most : 1.f;
  }
}

// xc[place] = x[rows[place]], unless all tokens count.  One wave per row.
__global__ __launch_bounds__(256) void head_pack_kernel(const uint16_t* x, const int32_t* rows,
                                                        const int32_t* n, int32_t T, int32_t D,
                                                        uint16_t* xc) {
  const int count = *n;
  if (count == T) return;
  for (int64_t p = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); p < count; p += (int64_t)gridDim.x * 4) {
    const u32x4* from = reinterpret_cast<const u32x4*>(x + (int64_t)rows[p] * D);
    u32x4* to = reinterpret_cast<u32x4*>(xc + p * D);
    for (int i = threadIdx.x & 63; i < D / 8; i += 64) to[i] = from[i];
  }
}

// Panels of the transpose: out[r / 64][c][r % 64] = in[row(r)][c], zeros for
// r past the end of its panel's valid rows.  rows: row(r) = rows[r], or NULL.
// n: valid rows on the device, or NULL for `count`.  One workgroup per 64 rows
// and 128 columns.
__global__ __launch_bounds__(256) void head_transpose_kernel(const uint16_t* in, const int32_t* rows,
                                                             const int32_t* n, int32_t count, int32_t D,
                                                             uint16_t* out) {
  __shared__ __attribute__((aligned(16))) uint16_t tile[64][128 + 8];
  const int valid = n != nullptr ? *n : count;
  const int64_t r0 = (int64_t)blockIdx.x * 64;
  const int c0 = blockIdx.y * 128;
  if (r0 >= valid) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int s = threadIdx.x + 256 * i, r = s >> 4, c = 8 * (s & 15);
    u32x4 v = {0, 0, 0, 0};
    if (r0 + r < valid && c0 + c < D) {
      const int64_t row = rows != nullptr ? rows[r0 + r] : r0 + r;
      v = *reinterpret_cast<const u32x4*>(in + row * D + c0 + c);
    }
    *reinterpret_cast<u32x4*>(&tile[r][c]) = v;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int s = threadIdx.x + 256 * i, c = s >> 3, r = 8 * (s & 7);
    if (c0 + c >= D) continue;
    u32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      v[e] = (uint32_t)tile[r + 2 * e][c] | (uint32_t)tile[r + 2 * e + 1][c] << 16;
    *reinterpret_cast<u32x4*>(out + ((int64_t)blockIdx.x * D + c0 + c) * 64 + r) = v;
  }
}

// lse of every token from its parts, and the loss of a target.  64 tokens per
// workgroup of 16 waves, a lane per token, the parts dealt to the waves.
__global__ __launch_bounds__(1024) void head_join_kernel(const HeadArgs a, const int32_t* pos,
                                                         const float2* part, int32_t parts,
                                                         const float* logit) {
  __shared__ float2 got[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * 64 + lane;
  const int p = t < a.T ? pos[t] : -1;
  float top = -INFINITY, sum = 0.f;
  if (p >= 0)
    for (int i = wave; i < parts; i += 16) {
      const float2 v = part[(int64_t)i * a.T + p];
      const float m = fmaxf(top, v.x), ref = m == -INFINITY ? 0.f : m;
      sum = sum * exp2f(top - ref) + v.y * exp2f(v.x - ref);
      top = m;
    }
  got[wave][lane] = make_float2(top, sum);
  __syncthreads();
  if (wave != 0 || t >= a.T) return;
  for (int w = 1; w < 16; ++w) {
    const float2 v = got[w][lane];
    const float m = fmaxf(top, v.x), ref = m == -INFINITY ? 0.f : m;
    sum = sum * exp2f(top - ref) + v.y * exp2f(v.x - ref);
    top = m;
  }
  const float lse = p >= 0 ? kLn2 * (top + log2f(sum)) : 0.f;
  a.lse[t] = lse;
  if (a.index == nullptr) {
    const int64_t at = (int64_t)a.targets[t] - a.first;
    const float z = p >= 0 && at >= 0 && at < a.V ? logit[p] : 0.f;
    a.logits[t] = z;
    a.loss[t] = lse - z;
  }
}

// Distillation: the logits of a token's entries and its loss.  One wave per
// token; 8 columns per lane and step.
__global__ __launch_bounds__(256) void head_entries_kernel(const HeadArgs a) {
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (t >= a.T) return;
  float q[kEntryLanes], lq[kEntryLanes], z[kEntryLanes];
  int at[kEntryLanes];
  const bool any = teacher_row(a, t, lane, q, lq, at);
  const uint16_t* x = a.x + t * a.D;
#pragma unroll
  for (int i = 0; i < kEntryLanes; ++i) {
    z[i] = 0.f;
    for (int j = 0; j < 64 && 64 * i + j < a.k; ++j) {
      const int v = __builtin_amdgcn_readlane(at[i], j) ;
      if (v < a.first || v - a.first >= a.V) continue;
      const uint16_t* w = a.w + (int64_t)(v - a.first) * a.D;
      float s = 0.f;
      for (int d = 8 * lane; d < a.D; d += 512) {
        const u32x4 xv = *reinterpret_cast<const u32x4*>(x + d), wv = *reinterpret_cast<const u32x4*>(w + d);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s = __builtin_fmaf(__uint_as_float(xv[e] << 16), __uint_as_float(wv[e] << 16), s);
          s = __builtin_fmaf(__uint_as_float(xv[e] & 0xffff0000u), __uint_as_float(wv[e] & 0xffff0000u), s);
        }
      }
      s = wave_sum(s);
      if (lane == j) z[i] = s;
    }
  }
  float loss = 0.f;
  const float lse = any ? a.lse[t] : 0.f;
#pragma unroll
  for (int i = 0; i < kEntryLanes; ++i) {
    const int j = 64 * i + lane;
    if (j < a.k) a.logits[t * a.k + j] = z[i];
    if (any && q[i] > 0.f) loss += q[i] * (lq[i] + lse - z[i] * a.inv_temperature);
  }
  loss = wave_sum(loss);
  if (lane == 0) a.loss[t] = loss;
}

// Distillation, backward: dz at the entries of a token, from their logits.
// entry[j]: its place in w (-1: none here, or told by an earlier entry of the
// same place, whose q then holds both), value[j]: a p - b q, in 16 bits.
__global__ __launch_bounds__(256) void head_entry_values_kernel(const HeadArgs a, const int32_t* pos,
                                                                const Token* token, const float* top,
                                                                int32_t* entry, uint16_t* value) {
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
    uint32_t bits = 0;
    if (any && at[i] >= 0 && !early[i] && at[i] >= a.first && at[i] - a.first < a.V) {
      where = (int)(at[i] - a.first);
      const Token k = token[p];
      const float pr = exp2f(__builtin_fmaf(a.logits_in[t * a.k + j], a.inv_temperature * kLog2e, -k.lse2));
      bits = pack2(k.a * top[1] * pr - k.b * top[1] * sum[i], 0.f) & 0xffffu;
    }
    entry[t * a.k + j] = where;
    value[t * a.k + j] = (uint16_t)bits;
  }
}

// These values into the piece [v0, v0 + count) of dz and of its transpose.
__global__ __launch_bounds__(256) void head_entry_store_kernel(const int32_t* pos, const int32_t* entry,
                                                               const uint16_t* value, int64_t total,
                                                               int32_t k, int32_t v0, int32_t count,
                                                               int64_t rows_t, int64_t rows_v,
                                                               uint16_t* dz, uint16_t* dzt) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int v = entry[i];
    if (v < v0 || v - v0 >= count) continue;
    const int64_t p = pos[i / k], c = v - v0;
    if (dz != nullptr) dz[((c >> 6) * rows_t + p) * 64 + (c & 63)] = value[i];
    if (dzt != nullptr) dzt[((p >> 6) * rows_v + c) * 64 + (p & 63)] = value[i];
  }
}

// dx[t] = top sum over the parts of dx32[part][place], one rounding; zeros for
// tokens that do not count.  A thread per 8 columns.
__global__ __launch_bounds__(256) void head_dx_kernel(const int32_t* pos, const float* dx32,
                                                      int32_t splits, int64_t rows_t, int64_t T,
                                                      int32_t D, const float* top, uint16_t* dx) {
  const int64_t total = T * (D / 8);
  const float scale = top[0];
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t t = i / (D / 8);
    const int d = 8 * (int)(i - t * (D / 8));
    const int p = pos[t];
    u32x4 v = {0, 0, 0, 0};
    if (p >= 0) {
      float s[8] = {};
      for (int k = 0; k < splits; ++k) {
        const float4* f = reinterpret_cast<const float4*>(dx32 + (k * rows_t + p) * D + d);
        const float4 lo = f[0], hi = f[1];
        s[0] += lo.x; s[1] += lo.y; s[2] += lo.z; s[3] += lo.w;
        s[4] += hi.x; s[5] += hi.y; s[6] += hi.z; s[7] += hi.w;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = pack2(s[2 * e] * scale, s[2 * e + 1] * scale);
    }
    *reinterpret_cast<u32x4*>(dx + t * D + d) = v;
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
  int32_t* pos;
  int32_t* rows;
  int32_t* n;
  Token* token;
  uint16_t* xc;
};
Common take_common(Parts& w, int64_t T, int64_t D) {
  Common c;
  c.pos = w.take<int32_t>(T);
  c.rows = w.take<int32_t>(T);
  c.n = w.take<int32_t>(1);
  c.token = w.take<Token>(T);
  c.xc = w.take<uint16_t>(T * D);
  return c;
}

struct Forward {
  Common c;
  float2* part;
  float* logit;
  int32_t parts;
  bool small;
};

// Whether a product of np x nq outputs takes 256 x 128 tiles.
bool small_tiles(int64_t np, int64_t nq, int64_t splits) {
  const int64_t large = up(((np + 255) / 256) * ((nq + 255) / 256) * splits, 256) / 256;
  const int64_t small = up(((np + 255) / 256) * ((nq + 127) / 128) * splits, 256) / 256;
  return small * 10 < large * 18;
}

Forward take_forward(Parts& w, int64_t T, int64_t V, int64_t D) {
  Forward f;
  f.c = take_common(w, T, D);
  f.small = small_tiles(V, T, 1);
  f.parts = (int32_t)((V + 255) / 256 * (f.small ? Small::WP : Large::WP));
  f.part = w.take<float2>(f.parts * T);
  f.logit = w.take<float>(T);
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
  uint16_t* dzt;
  uint16_t* xt;
  uint16_t* wt;
  float* dx32;
  int32_t* entry;
  uint16_t* value;
  int64_t rows_t, piece;
  int32_t splits;
};

// Parts of the input gradient's reduction: enough for 256 tiles, of at least
// 1024 steps each.
int32_t dx_splits(int64_t T, int64_t D, int64_t piece) {
  const int64_t tiles = ((T + 255) / 256) * ((D + 127) / 128);
  int64_t s = 256 / tiles;
  if (s > piece / 1024) s = piece / 1024;
  return (int32_t)(s < 1 ? 1 : s > 64 ? 64 : s);
}

Backward take_backward(Parts& w, int64_t T, int64_t V, int64_t D, int64_t k) {
  Backward b;
  b.c = take_common(w, T, D);
  b.rows_t = up(T, 256);
  b.piece = piece_of(T, V);
  b.splits = dx_splits(T, D, b.piece);
  b.top = w.take<float>(2);
  b.dz = w.take<uint16_t>(b.rows_t * b.piece);
  b.dzt = w.take<uint16_t>(b.rows_t * b.piece);
  b.xt = w.take<uint16_t>(b.rows_t * D);
  b.wt = w.take<uint16_t>(b.piece * D);
  b.dx32 = w.take<float>(b.splits * b.rows_t * D);
  b.entry = w.take<int32_t>(T * k);
  b.value = w.take<uint16_t>(T * k);
  return b;
}

unsigned blocks_for(int64_t items, int64_t per, int64_t most) {
  const int64_t b = (items + per - 1) / per;
  return (unsigned)(b < 1 ? 1 : b > most ? most : b);
}

template <int EPI, class C>
int run_nt(const NtArgs& a, hipStream_t s) {
  static const hipError_t set = hipFuncSetAttribute(reinterpret_cast<const void*>(&nt_kernel<EPI, C>),
                                                    hipFuncAttributeMaxDynamicSharedMemorySize, C::LDS);
  if (set != hipSuccess) return set;
  hipLaunchKernelGGL((nt_kernel<EPI, C>), dim3(256), dim3(512), C::LDS, s, a);
  return hipGetLastError();
}
template <int EPI>
int run_nt(const NtArgs& a, bool small, hipStream_t s) {
  return small ? run_nt<EPI, Small>(a, s) : run_nt<EPI, Large>(a, s);
}

#define MG_RUN(call)                       \
  do {                                     \
    const int err_ = (call);               \
    if (err_ != hipSuccess) return err_;   \
  } while (0)

// Which tokens count, their order and, packed, their rows of x.
int place_tokens(const HeadArgs& a, const Common& c, float* top, hipStream_t s) {
  const int64_t per = a.index != nullptr ? 4 : 256;
  hipLaunchKernelGGL(head_counts_kernel, dim3((unsigned)((a.T + per - 1) / per)), dim3(256), 0, s, a, c.pos);
  MG_RUN(hipGetLastError());
  hipLaunchKernelGGL(head_place_kernel, dim3(1), dim3(1024), 0, s, a, c.pos, c.rows, c.n, c.token, top);
  MG_RUN(hipGetLastError());
  hipLaunchKernelGGL(head_pack_kernel, dim3(blocks_for(a.T, 4, 2048)), dim3(256), 0, s, a.x, c.rows, c.n,
                     (int32_t)a.T, (int32_t)a.D, c.xc);
  return hipGetLastError();
}

// The logits' product, from vocabulary entry v0 on.
NtArgs logits_args(const HeadArgs& a, const Common& c, int64_t v0, int64_t count) {
  NtArgs g{};
  g.P = {a.w + v0 * a.D, (uint32_t)a.D * 2u, 128u};
  g.Q = {c.xc, (uint32_t)a.D * 2u, 128u};
  g.Q_all = a.x;
  g.n = c.n;
  g.np = (int32_t)count;
  g.nq = g.tokens = (int32_t)a.T;
  g.K = g.D = (int32_t)a.D;
  g.first = (int32_t)v0;
  g.gq = 8;
  g.splits = 1;
  g.scale = a.inv_temperature * kLog2e;
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
  MG_RUN(place_tokens(a, f.c, nullptr, s));
  NtArgs g = logits_args(a, f.c, 0, a.V);
  g.part = f.part;
  g.logit = a.index == nullptr ? f.logit : nullptr;
  MG_RUN(run_nt<kStats>(g, f.small, s));
  hipLaunchKernelGGL(head_join_kernel, dim3((unsigned)((a.T + 63) / 64)), dim3(1024), 0, s, a, f.c.pos,
                     f.part, f.parts, f.logit);
  MG_RUN(hipGetLastError());
  if (a.index != nullptr) {
    hipLaunchKernelGGL(head_entries_kernel, dim3((unsigned)((a.T + 3) / 4)), dim3(256), 0, s, a);
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
  MG_RUN(place_tokens(a, b.c, b.top, s));
  if (entries > 0) {
    hipLaunchKernelGGL(head_entry_values_kernel, dim3((unsigned)((a.T + 3) / 4)), dim3(256), 0, s, a,
                       b.c.pos, b.c.token, b.top, b.entry, b.value);
    MG_RUN(hipGetLastError());
  }
  const unsigned cols = (unsigned)((D + 127) / 128);
  if (a.dw != nullptr) {
    hipLaunchKernelGGL(head_transpose_kernel, dim3((unsigned)((T + 63) / 64), cols), dim3(256), 0, s, a.x,
                       b.c.rows, b.c.n, T, D, b.xt);
    MG_RUN(hipGetLastError());
  }
  for (int64_t v0 = 0; v0 < a.V; v0 += b.piece) {
    const int64_t count = a.V - v0 < b.piece ? a.V - v0 : b.piece;
    NtArgs g = logits_args(a, b.c, v0, count);
    g.top = b.top;
    g.dz = a.dx != nullptr ? b.dz : nullptr;
    g.dzt = a.dw != nullptr ? b.dzt : nullptr;
    g.rows_t = b.rows_t;
    g.rows_v = b.piece;
    MG_RUN(run_nt<kDz>(g, small_tiles(count, T, 1), s));
    if (entries > 0) {
      hipLaunchKernelGGL(head_entry_store_kernel, dim3(blocks_for(entries, 256, 2048)), dim3(256), 0, s,
                         b.c.pos, b.entry, b.value, entries, a.k, (int32_t)v0, (int32_t)count, b.rows_t,
                         b.piece, g.dz, g.dzt);
      MG_RUN(hipGetLastError());
    }
    if (a.dx != nullptr) {
      hipLaunchKernelGGL(head_transpose_kernel, dim3((unsigned)((count + 63) / 64), cols), dim3(256), 0, s,
                         a.w + v0 * a.D, nullptr, nullptr, (int32_t)count, D, b.wt);
      MG_RUN(hipGetLastError());
      NtArgs h{};
      h.P = {b.dz, 128u, (uint32_t)(b.rows_t * 128)};
      h.Q = {b.wt, 128u, (uint32_t)(a.D * 128)};
      h.n = b.c.n;
      h.np = h.tokens = T;
      h.nq = h.D = D;
      h.K = (int32_t)up(count, 8);
      h.gq = 8;
      h.splits = b.splits;
      h.add = v0 > 0;
      h.dx = b.dx32;
      h.rows_t = b.rows_t;
      MG_RUN(run_nt<kDx>(h, small_tiles(T, D, b.splits), s));
    }
    if (a.dw != nullptr) {
      NtArgs h{};
      h.P = {b.dzt, 128u, (uint32_t)(b.piece * 128)};
      h.Q = {b.xt, 128u, (uint32_t)(a.D * 128)};
      h.n = b.c.n;
      h.np = (int32_t)count;
      h.tokens = h.K = T;
      h.nq = h.D = D;
      h.gq = 8;
      h.splits = 1;
      h.top = b.top;
      h.dw = a.dw + v0 * a.D;
      MG_RUN(run_nt<kDw>(h, small_tiles(count, D, 1), s));
    }
  }
  if (a.dx != nullptr) {
    hipLaunchKernelGGL(head_dx_kernel, dim3(blocks_for(a.T * (D / 8), 256, 4096)), dim3(256), 0, s, b.c.pos,
                       b.dx32, b.splits, b.rows_t, a.T, D, b.top, a.dx);
    MG_RUN(hipGetLastError());
  }
  return hipSuccess;
}

}  // namespace mg
