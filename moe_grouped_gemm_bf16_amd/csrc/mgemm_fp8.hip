// gfx950 kernels of the block-scaled fp8 M-grouped products: E4M3 operands with
// one fp32 scale per row and 128 reduction steps of the activations and one per
// 128 x 128 block of the weights.
//   FWD    y[i, n]  = sum_b xs[b, i] ws[e, n / 128, b]
//                     sum_{k in block b} x8[i, k] w8[e, n, k]
//   DGRAD  dx[i, k] = sum_b dys[b, i] ws[e, b, k / 128]
//                     sum_{n in block b} dy8[i, n] w8[e, n, k]
// for offsets[e] <= i < offsets[e+1]; bf16 out.
//
// A stage of 128 reduction steps is one scale block, and one 16x16x128 fp8
// matrix-core product reduces it whole: the product starts from zero, and its
// four fp32 results per lane are added to the fp32 accumulators with one fma
// each, the factor being xs ws.  The output's contiguous dimension is the
// product's first operand (P: weights), so a lane holds four consecutive
// outputs of one row; the row's scale is then one register per 16 rows, and
// the weights' scale is uniform over a wave's 128 P indices.  The fma of one
// result block (16 cycles of the vector unit) runs under the next product
// (32 cycles of the matrix core).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "mgemm_launch.h"

namespace mg {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x2 __attribute__((ext_vector_type(2)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kBlk = 128;                 // reduction steps per scale block and LDS stage
constexpr uint32_t kOOB = 0x80000000u;    // offset bit past any buffer range

// Raw buffer descriptor over `bytes` bytes from `base` (both wave-uniform);
// loads past the range return zero.
__device__ __forceinline__ i32x4 rsrc_of(const void* base, uint32_t bytes) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  i32x4 r;
  r.x = (int32_t)__builtin_amdgcn_readfirstlane((uint32_t)b);
  r.y = (int32_t)(__builtin_amdgcn_readfirstlane((uint32_t)(b >> 32)) & 0xFFFFu);
  r.z = (int32_t)__builtin_amdgcn_readfirstlane(bytes);
  r.w = 0x00020000;
  return r;
}

// Direct-to-LDS loads of one stage: four 1-KiB pieces of P, four of Q (lane
// l's 16 bytes of piece j land at lds + 1024 j + 16 l) and one dword per lane
// of the scales.  One block, so that m0, which holds the LDS address, is saved
// and restored once (the scalar unit is a third of the loop's issue slots when
// every load does it); a wait state separates each m0 write from its load.
// Awaited with vmcnt before the barrier that publishes the stage.
__device__ __forceinline__ void load_stage(const i32x4& rp, const i32x4& rq, const i32x4& rs,
                                           uint32_t lp, uint32_t lq, uint32_t ls,
                                           const uint32_t (&vp)[4], const uint32_t (&vq)[4],
                                           uint32_t vs) {
  uint32_t save;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %4, %13, 0 offen lds\n\t"
      "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tbuffer_load_dwordx4 %5, %13, 0 offen lds\n\t"
      "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tbuffer_load_dwordx4 %6, %13, 0 offen lds\n\t"
      "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tbuffer_load_dwordx4 %7, %13, 0 offen lds\n\t"
      "s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %8, %14, 0 offen lds\n\t"
      "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tbuffer_load_dwordx4 %9, %14, 0 offen lds\n\t"
      "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tbuffer_load_dwordx4 %10, %14, 0 offen lds\n\t"
      "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tbuffer_load_dwordx4 %11, %14, 0 offen lds\n\t"
      "s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dword %12, %15, 0 offen lds\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(save)
      : "s"(lp), "s"(lq), "s"(ls), "v"(vp[0]), "v"(vp[1]), "v"(vp[2]), "v"(vp[3]), "v"(vq[0]),
        "v"(vq[1]), "v"(vq[2]), "v"(vq[3]), "v"(vs), "s"(rp), "s"(rq), "s"(rs)
      : "memory", "scc");
}

// The same for eight pieces of one operand.
__device__ __forceinline__ void load_block(const i32x4& r, uint32_t to, const uint32_t (&v)[8]) {
  uint32_t save;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %10, 0 offen lds\n\t"
      "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tbuffer_load_dwordx4 %3, %10, 0 offen lds\n\t"
      "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tbuffer_load_dwordx4 %4, %10, 0 offen lds\n\t"
      "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tbuffer_load_dwordx4 %5, %10, 0 offen lds\n\t"
      "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tbuffer_load_dwordx4 %6, %10, 0 offen lds\n\t"
      "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tbuffer_load_dwordx4 %7, %10, 0 offen lds\n\t"
      "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tbuffer_load_dwordx4 %8, %10, 0 offen lds\n\t"
      "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tbuffer_load_dwordx4 %9, %10, 0 offen lds\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(save)
      : "s"(to), "v"(v[0]), "v"(v[1]), "v"(v[2]), "v"(v[3]), "v"(v[4]), "v"(v[5]), "v"(v[6]),
        "v"(v[7]), "s"(r)
      : "memory", "scc");
}

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t lds_addr_of(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)(
      (const __attribute__((address_space(3))) void*)p);
}

// One scale block's product: 16 P rows x 16 Q rows x 128 steps, from zero.
// (The instruction's own power-of-two scales are 2^0 = code 127.)
__device__ __forceinline__ f32x4 product(const i32x8& p, const i32x8& q) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(p, q, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0,
                                                          127, 0, 127);
}

// The factor of a block's sum is its two scales' product s.  Where that is odd,
// neither a normal number nor zero, it is taken as m c, c = 2^+-64: a sum (0, or
// 2^-18 to 2^24.6) times c is exact, and that times m is rounded once, as with a
// factor that fits.  (Zero from an underflow drops a block that adds less than
// 2^-125, 2^-150 times 128 products of at most 448^2.  m past the largest number
// is that, so that a sum of zero stays zero; an infinite or NaN scale stays so.)
struct Factor {
  float m, c;
};
__device__ __forceinline__ bool factor_odd(float s) { return __builtin_amdgcn_classf(s, 0x297); }
__device__ __forceinline__ Factor split_factor(float a, float b, float s) {
  const bool small = fabsf(s) < 1.0f;
  const float k = small ? 0x1p32f : 0x1p-32f;
  float m = (a * k) * (b * k);
  if (fabsf(a) <= 3.40282347e38f && fabsf(b) <= 3.40282347e38f) m = fminf(fmaxf(m, -3.40282347e38f), 3.40282347e38f);
  return {m, small ? 0x1p-64f : 0x1p64f};
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}

// ---------------------------------------------------------------- scheduler --

// The experts' row ranges and tile counts, in LDS: offs[e] is the running
// maximum of the offsets clamped to [0, M] (a broken offsets array then gives
// no row to two experts, moves no access out of the tensors and makes no more
// tiles than the host counted with), pref[e] the exclusive prefix of
// ceil(rows / BQ).
struct Experts {
  int* offs;
  int* pref;
  int E, mtiles;
};

// Inclusive scan over the wave's lanes (operands not negative, 0 neutral), by
// row shifts: through LDS it takes 0.2 us more before a workgroup's first load.
template <typename F>
__device__ __forceinline__ int wave_scan(int x, F f) {
  x = f(x, __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false));   // rows: 1, 2, 4, 8 lanes below
  x = f(x, __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false));
  x = f(x, __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false));
  x = f(x, __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false));
  x = f(x, __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false));   // a row's last lane to the next row
  return f(x, __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false));
}

template <int BQ>
__device__ __forceinline__ void setup_experts(const int32_t* __restrict__ offsets, int M,
                                              Experts& X) {
  // every wave scans all experts (kMaxExperts / 64 per lane at most); wave 0 writes
  const int lane = threadIdx.x & 63, per = (X.E + 63) / 64;
  const bool writer = threadIdx.x < 64;
  auto clamped = [&](int e) { return min(max(offsets[e], 0), M); };
  int sum = 0;
  int least = 0;                        // below 0: an offset falls
  for (int j = 0; j < per; ++j) {
    const int e = lane * per + j;
    if (e >= X.E) break;
    const int lo = clamped(e), hi = clamped(e + 1);
    least = min(least, hi - lo);
    sum += (max(hi, lo) - lo + BQ - 1) / BQ;
  }
  int top = 0;                          // the maximum of the lanes' before
  if (__builtin_expect(__builtin_amdgcn_ballot_w64(least < 0) != 0, 0)) {
    int most = 0;
    for (int j = 0; j < per; ++j)
      if (lane * per + j < X.E) most = max(most, clamped(lane * per + j));
    most = wave_scan(most, [](int p, int q) { return max(p, q); });
    top = __shfl_up(most, 1, 64);
    if (lane == 0) top = 0;
    sum = 0;
    int lo = top;
    for (int j = 0; j < per; ++j) {
      const int e = lane * per + j;
      if (e >= X.E) break;
      lo = max(lo, clamped(e));
      sum += (max(lo, clamped(e + 1)) - lo + BQ - 1) / BQ;
    }
  }
  const int incl = wave_scan(sum, [](int p, int q) { return p + q; });
  X.mtiles = __builtin_amdgcn_readlane(incl, 63);
  if (writer) {
    int run = incl - sum, lo = top;
    for (int j = 0; j < per; ++j) {
      const int e = lane * per + j;
      if (e >= X.E) break;
      lo = max(lo, clamped(e));
      const int hi = max(lo, clamped(e + 1));
      X.offs[e] = lo;
      X.pref[e] = run;
      run += (hi - lo + BQ - 1) / BQ;
      if (e == X.E - 1) {
        X.offs[X.E] = hi;
        X.pref[X.E] = run;
      }
    }
  }
  __syncthreads();
}

struct Tile {
  int e, q0, q_end, p0;
};

// Tile id L -> tile: expert by expert, inside an expert in groups of gm
// M-tiles (M-tile fastest, then P-tile), so that the tiles that run at the
// same time on one XCD share weight and activation panels in its L2.  Ids are
// asked for in ascending order: the expert search goes on from the last one.
template <int BP, int BQ>
struct Decode {
  int first = 0, after = 0;                 // the current expert's tile ids,
  int e = 0, lo = 0, hi = 0;                // index and rows
  uint32_t group, rcp;                      // tiles of a full group, 2^32 / group
  __device__ __forceinline__ void init(int tilesP, int gm) {
    group = (uint32_t)gm * (uint32_t)tilesP;
    rcp = __builtin_amdgcn_readfirstlane(0xFFFFFFFFu / group);
  }
  __device__ __forceinline__ Tile at(int L, const Experts& X, int tilesP, int gm) {
    if (L >= after) {
      int a = e, b = X.E - 1;
      while (a < b) {
        const int mid = (a + b + 1) >> 1;
        if (X.pref[mid] * tilesP <= L) a = mid; else b = mid - 1;
      }
      e = __builtin_amdgcn_readfirstlane(a);
      first = __builtin_amdgcn_readfirstlane(X.pref[e]) * tilesP;
      after = __builtin_amdgcn_readfirstlane(X.pref[e + 1]) * tilesP;
      lo = __builtin_amdgcn_readfirstlane(X.offs[e]);
      hi = __builtin_amdgcn_readfirstlane(X.offs[e + 1]);
    }
    const uint32_t local = (uint32_t)(L - first);
    // local / group: the estimate from the reciprocal is at most two low
    uint32_t g = __umulhi(local, rcp), rem = local - g * group;
    if (rem >= group) { ++g; rem -= group; }
    if (rem >= group) { ++g; rem -= group; }
    const int mt = (hi - lo + BQ - 1) / BQ;
    const uint32_t gh = (uint32_t)min(gm, mt - (int)g * gm);
    const uint32_t tp = rem / gh;
    Tile t;
    t.e = e;
    t.q0 = lo + ((int)g * gm + (int)(rem - tp * gh)) * BQ;
    t.q_end = hi;
    t.p0 = (int)tp * BP;
    return t;
  }
};

// The tiles of this workgroup.  Workgroup b runs on XCD b % 8; every XCD takes
// a contiguous range of tile ids, its nx workgroups every nx-th of them.  Where
// the last round has at most nx / 2 tiles, HALVES gives each to two workgroups
// of half the rows (a tile's time follows its rows, see the row skip of the
// tiled kernel), so a round that is a quarter full costs half a round.
template <int BP, int BQ, bool HALVES>
struct Items {
  Decode<BP, BQ> dec;
  int i, items, lo, full, step;
  bool halves;
  __device__ __forceinline__ void init(int total, int tilesP, int gm) {
    dec.init(tilesP, gm);
    const int x = blockIdx.x & 7;
    const int q8 = total >> 3, r8 = total & 7;
    const int count = q8 + (x < r8 ? 1 : 0);
    lo = x * q8 + min(x, r8);
    step = gridDim.x >> 3;
    full = HALVES ? count / step * step : count;
    const int rest = count - full;
    halves = HALVES && 2 * rest <= step;
    items = full + (halves ? 2 * rest : rest);
    i = blockIdx.x >> 3;
  }
  // The next tile, or false behind the last; halves without rows are passed over.
  __device__ __forceinline__ bool next(const Experts& X, int tilesP, int gm, Tile& t) {
    bool found = false;
    while (!found && i < items) {
      const int u = i - full;
      const bool half = halves && u >= 0;
      t = dec.at(lo + (half ? full + (u >> 1) : i), X, tilesP, gm);
      i += step;
      if (half) {
        t.q0 += (u & 1) * (BQ / 2);
        t.q_end = min(t.q_end, t.q0 + BQ / 2);
      }
      found = __builtin_amdgcn_readfirstlane(t.q0 < t.q_end);
    }
    t.q0 = __builtin_amdgcn_readfirstlane(t.q0);
    t.q_end = __builtin_amdgcn_readfirstlane(t.q_end);
    t.p0 = __builtin_amdgcn_readfirstlane(t.p0);
    i = __builtin_amdgcn_readfirstlane(i);
    return found;
  }
};

// ------------------------------------------------------------- tiled kernel --

// BP x BQ output tile, WP x WQ waves; ST LDS stages of 128 steps.  Every wave
// loads four 1-KiB pieces of the P tile and four of the Q tile of a stage.
template <int BP_, int BQ_, int WP_, int WQ_, int ST_>
struct Fp8Cfg {
  static constexpr int BP = BP_, BQ = BQ_, WP = WP_, WQ = WQ_, ST = ST_;
  static constexpr int NW = WP * WQ, NT = 64 * NW;
  static constexpr int WTP = BP / WP, WTQ = BQ / WQ, MP = WTP / 16, MQ = WTQ / 16;
  static constexpr int P_BYTES = BP * kBlk, DATA = (BP + BQ) * kBlk;
  static constexpr int SCALES = NW * 256, STAGE = DATA + SCALES;
  static constexpr int LOADS = 9;                        // per wave and stage (load_stage)
  static constexpr int AHEAD = MP == 8 ? 1 : 2;          // P fragments read ahead
  static constexpr int RING = AHEAD == 1 ? 2 : 4;        // and their registers
  static_assert(BP == 32 * NW && BQ == 32 * NW, "load_stage: four segments of each operand");
  static_assert(MP % 4 == 0 && MQ % 2 == 0 && WTP <= 128 && 128 % WTP == 0, "wave tile");
  static_assert(BQ / 64 + 1 <= NW && BQ % 64 == 0, "scale loads");
  static_assert((MP - 1) % RING != 0, "the next stage's first fragment has a free slot");
};

template <bool DG, class C>
__global__ __launch_bounds__(C::NT, 2) void fp8_gemm_kernel(Fp8Args a) {
  __shared__ __attribute__((aligned(16))) char lds[C::ST * C::STAGE];
  __shared__ int sched[2 * (kMaxExperts + 1)];
  // reduction length, output width, leading dimensions of the code arrays
  const int red = (int)(DG ? a.N : a.K), Pdim = (int)(DG ? a.K : a.N);
  const int ldP = (int)a.K, ldQ = red;
  const int nk = (red + kBlk - 1) / kBlk;
  const int nn = (int)((a.N + kBlk - 1) / kBlk), nkb = (int)((a.K + kBlk - 1) / kBlk);
  const int tilesP = (Pdim + C::BP - 1) / C::BP;
  Experts X{sched, sched + kMaxExperts + 1, a.E, 0};
  setup_experts<C::BQ>(a.offsets, (int)a.M, X);
  const int total = X.mtiles * tilesP;
  const int nx = gridDim.x >> 3;
  int gm = 1;
  while (gm * gm < nx) ++gm;
  gm = max(gm, (nx + tilesP - 1) / tilesP);

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // (waves w and w + 4 share a SIMD: this order spreads the first half of the
  // rows over all four)
  const int wp = wave % C::WP, wq = wave / C::WP;
  const int l16 = lane & 15, g4 = lane >> 4;

  // ---- producer.  Steps-contiguous tiles are [rows][128] bytes in 16-byte
  // chunks, chunk c of row r at c ^ (r % 8) ^ (r / 8 % 4): 16 rows read at one
  // chunk hit 16 distinct 16-byte banks.  DGRAD's weights are staged as they
  // lie, [128 n][BP k], chunk c of row r at c ^ (2 (r % 8)) ^ (r / 32 % 2)
  // (BP = 256) or c ^ (2 (r / 2 % 4)) ^ (r / 32 % 2) (BP = 128): the transpose
  // reads of 8 rows by two lane groups, 32 rows apart, then hit 16 distinct
  // banks.  The lane's offsets are the same for every tile and stage; the
  // descriptors move.
  const uint32_t lds0 = lds_addr_of(lds);
  // Piece j of the wave's four of an operand lies 8 rows (DGRAD's weights:
  // 1024 / BP) below piece j - 1, and its chunk differs from piece 0's by an
  // exclusive or, so the eight offsets take few operations and no register
  // between stages (a wave's 128 accumulators leave room for none).
  constexpr int CPR = DG ? C::BP / 16 : 8;                 // chunks per row of P
  // (BP = 256: rows 4 apart; 128: rows 8 apart, the same chunk; else r / 8 % 4)
  auto pxor = [](int j) { return !DG ? 16 * j : C::BP == 256 ? 128 * (j & 1) : 0; };

  Items<C::BP, C::BQ, true> items;
  items.init(total, tilesP, gm);
  // tiles that the producer has begun and the consumer not yet: with a
  // reduction of one stage the producer is ST tiles ahead
  Tile ahead[C::ST + 1];
  int nahead = 0;
  bool live = false;
  // the next stage's descriptors, advanced by a stage's bytes each time
  i32x4 rp = {0, 0, 0, 0x00020000}, rq = rp, rs = rp;
  const int64_t stepP = DG ? (int64_t)kBlk * ldP : kBlk;
  int64_t stepS = 0;                 // bytes between the wave's scales of two blocks
  uint32_t vs = kOOB;                // this lane's scale
  int outP = 0, pleft = 0, produced = 0;
  uint32_t pbuf = 0;
  auto advance = [](i32x4& r, int64_t bytes) {
    const uint64_t b = (((uint64_t)(uint32_t)r.y << 32) | (uint32_t)r.x) + (uint64_t)bytes;
    r.x = __builtin_amdgcn_readfirstlane((uint32_t)b);
    r.y = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32));
  };
  auto next_tile = [&]() {
    Tile t = {0, 0, 0, 0};
    live = items.next(X, tilesP, gm, t);
    if (!live) return;
#pragma unroll
    for (int u = 0; u <= C::ST; ++u)
      if (u == nahead) ahead[u] = t;
    ++nahead;
    pleft = red;
    const uint8_t* w = static_cast<const uint8_t*>(a.w8) + (int64_t)t.e * a.N * a.K;
    outP = __builtin_amdgcn_readfirstlane(min(Pdim - t.p0, C::BP));
    const int outQ = min(t.q_end - t.q0, C::BQ);
    // Ranges end a stage's columns after the last valid row's start, so rows
    // past it are out of range (a row is at least that long) while the base
    // moves; columns past the reduction's (or DGRAD's output's) end are put
    // out of range by their lanes' offsets (see produce).
    const uint32_t cols = (uint32_t)min(red, kBlk);
    rp = rsrc_of(DG ? w + t.p0 : w + (int64_t)t.p0 * a.K,
                 DG ? (uint32_t)(kBlk - 1) * (uint32_t)ldP + (uint32_t)outP
                    : (uint32_t)(outP - 1) * (uint32_t)ldP + cols);
    rq = rsrc_of(static_cast<const uint8_t*>(a.q8) + (int64_t)t.q0 * ldQ,
                 (uint32_t)(outQ - 1) * (uint32_t)ldQ + cols);
    // scales: waves 0 .. BQ/64 - 1 load 64 rows' each, the next wave the
    // weights' (one per 128 P indices); the other waves' load reads nothing
    const float* s = a.qs;
    uint32_t range = 0;
    vs = kOOB;
    stepS = 0;
    if (wave < C::BQ / 64) {
      s = a.qs + t.q0;
      stepS = 4 * a.M;
      range = (uint32_t)min((int)a.M - t.q0, C::BQ) * 4u;
      vs = (uint32_t)(wave * 64 + lane) * 4u;
    } else if (wave == C::BQ / 64) {
      const int pb = t.p0 / kBlk;
      const int blocks = min((C::BP + kBlk - 1) / kBlk, (DG ? nkb : nn) - pb);
      const uint32_t step = DG ? 4u : (uint32_t)nkb * 4u;
      s = a.ws + (int64_t)t.e * nn * nkb + (DG ? (int64_t)pb : (int64_t)pb * nkb);
      stepS = DG ? 4 * (int64_t)nkb : 4;
      range = (uint32_t)(blocks - 1) * step + 4u;
      if (lane < blocks) vs = (uint32_t)lane * step;
    }
    rs = rsrc_of(s, range);
  };
  // Issue the producer's next stage into the LDS buffer that is free.
  auto produce = [&]() {
    if (!live || nk == 0) return;
    const uint32_t buf = lds0 + pbuf;
    const uint32_t lp = buf + (uint32_t)(wave * 4) * 1024u;
    const uint32_t lq = buf + (uint32_t)C::P_BYTES + (uint32_t)(wave * 4) * 1024u;
    const uint32_t ls = buf + (uint32_t)C::DATA + (uint32_t)wave * 256u;
    const bool tail = pleft < kBlk;
    uint32_t vp[4], vq[4];
    uint32_t ln = (uint32_t)lane;
    asm volatile("" : "+v"(ln));                 // (what follows is not kept between stages)
    const int prow = wave * (4 * 64 / CPR) + (int)(ln / CPR);
    const int psw = !DG ? (prow & 7) ^ ((prow >> 3) & 3)
                        : C::BP == 256 ? (2 * (prow & 7)) ^ ((prow >> 5) & 1)
                                       : (2 * ((prow >> 1) & 3)) ^ ((prow >> 5) & 1);
    const int qrow = wave * 32 + (int)(ln >> 3);
    const int pc0 = 16 * ((int)(ln % CPR) ^ psw);
    const int qc0 = 16 * ((int)(ln & 7) ^ (qrow & 7) ^ ((qrow >> 3) & 3));
    const uint32_t pb = (uint32_t)prow * (uint32_t)ldP;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      vp[j] = pb + (uint32_t)(j * (64 / CPR)) * (uint32_t)ldP + (uint32_t)(pc0 ^ pxor(j));
      // FWD: both operands are rows of K steps, and the offsets are the same
      vq[j] = !DG ? vp[j]
                  : (uint32_t)(qrow + 8 * j) * (uint32_t)ldQ + (uint32_t)(qc0 ^ (16 * j));
    }
    if (tail || (DG && outP < C::BP)) {
      // columns past the end hold the next row's bytes: out of range instead
      const int lim = DG ? outP : pleft;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        vp[j] = (pc0 ^ pxor(j)) < lim ? vp[j] : kOOB;
        vq[j] = ((DG ? qc0 : pc0) ^ (16 * j)) < pleft ? vq[j] : kOOB;
      }
      // DGRAD's rows past the reduction's end
      if (DG && tail)
        rp.z = __builtin_amdgcn_readfirstlane((pleft - 1) * ldP + outP);
    }
    load_stage(rp, rq, rs, lp, lq, ls, vp, vq, vs);
    ++produced;
    pbuf = pbuf == (uint32_t)((C::ST - 1) * C::STAGE) ? 0u : pbuf + (uint32_t)C::STAGE;
    pleft -= kBlk;
    if (pleft <= 0) {
      next_tile();
    } else {
      advance(rp, stepP);
      advance(rq, kBlk);
      advance(rs, stepS);
    }
  };

  // ---- consumer: fragment addresses.  Lane l of a fragment holds row l % 16
  // and the 32 steps 32 (l / 16) .. + 31 of the block.
  const uint32_t sw16 = 16u * (uint32_t)((2 * g4) ^ (l16 & 7) ^ (l16 >> 3));
  const uint32_t offQ = (uint32_t)C::P_BYTES + (uint32_t)(wq * C::WTQ + l16) * 128u + sw16;
  const uint32_t offP = (uint32_t)(wp * C::WTP + l16) * 128u + sw16;
  // DGRAD: within 16 lanes, lane L addresses 8 bytes of row L / 2 (columns
  // 8 (L % 2)) and receives column L of 8 consecutive rows
  const int trow = 32 * g4 + (l16 >> 1);
  const uint32_t tsw = (C::BP == 256 ? 2u * (uint32_t)(l16 >> 1) : 2u * (uint32_t)((l16 >> 2) & 3)) ^
                       (uint32_t)(g4 & 1);
  const uint32_t offT = (uint32_t)trow * C::BP + 16u * ((uint32_t)(wp * C::MP) ^ tsw) +
                        8u * (uint32_t)(l16 & 1);
  auto frag = [&](const char* base, uint32_t off) {
    const i32x4 lo = *reinterpret_cast<const i32x4*>(base + off);
    const i32x4 hi = *reinterpret_cast<const i32x4*>(base + (off ^ 16u));
    return (i32x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  auto readQ = [&](const char* st, int j) {
    return frag(st + j * 2048, offQ ^ (uint32_t)(32 * (j & 1)));
  };
  auto readP = [&](const char* st, int i) {
    if constexpr (DG) {
      typedef __attribute__((address_space(3))) i32x2 lds_i32x2;
      const uint32_t o = offT ^ (uint32_t)(16 * i);
      auto tr = [&](uint32_t off) {
        return __builtin_amdgcn_ds_read_tr8_b64_v2i32(
            (lds_i32x2*)((__attribute__((address_space(3))) char*)(
                             (__attribute__((address_space(3))) void*)st) + off));
      };
      const i32x2 a0 = tr(o), a1 = tr(o + 8 * C::BP), a2 = tr(o + 16 * C::BP), a3 = tr(o + 24 * C::BP);
      const i32x4 lo = __builtin_shufflevector(a0, a1, 0, 1, 2, 3);
      const i32x4 hi = __builtin_shufflevector(a2, a3, 0, 1, 2, 3);
      return (i32x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
      return frag(st + i * 2048, offP ^ (uint32_t)(32 * (i & 1)));
    }
  };
  f32x4 acc[C::MP][C::MQ];
#pragma unroll
  for (int i = 0; i < C::MP; ++i)
#pragma unroll
    for (int j = 0; j < C::MQ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  i32x8 fp[C::RING], fq[C::MQ];
  float rawq[C::MQ], raww;
  auto read_scales = [&](const char* st) {
    const float* sc = reinterpret_cast<const float*>(st + C::DATA);
#pragma unroll
    for (int j = 0; j < C::MQ; ++j) rawq[j] = sc[wq * C::WTQ + 16 * j + l16];
    raww = sc[C::BQ + wp * C::WTP / kBlk];
  };

  auto store = [&](const Tile& t) {
    uint16_t* out = reinterpret_cast<uint16_t*>(a.out);
#pragma unroll
    for (int j = 0; j < C::MQ; ++j) {
      const int m = t.q0 + wq * C::WTQ + 16 * j + l16;
#pragma unroll
      for (int i = 0; i < C::MP; i += 2) {
        // lanes regrouped so that each stores 8 consecutive outputs: after
        // the swap of lane rows between blocks i and i + 1, lane row rho holds
        // outputs 8 (rho / 2) .. + 7 of block i + rho % 2
        uint32_t x0 = pack_bf16(acc[i][j][0], acc[i][j][1]);
        uint32_t x1 = pack_bf16(acc[i][j][2], acc[i][j][3]);
        uint32_t y0 = pack_bf16(acc[i + 1][j][0], acc[i + 1][j][1]);
        uint32_t y1 = pack_bf16(acc[i + 1][j][2], acc[i + 1][j][3]);
        const auto r0 = __builtin_amdgcn_permlane16_swap(x0, y0, false, false);
        const auto r1 = __builtin_amdgcn_permlane16_swap(x1, y1, false, false);
        const int col = t.p0 + wp * C::WTP + 16 * (i + (g4 & 1)) + 8 * (g4 >> 1);
        if (col < Pdim && m < t.q_end)
          *reinterpret_cast<u32x4*>(out + (int64_t)m * Pdim + col) = u32x4{r0[0], r1[0], r0[1], r1[1]};
      }
    }
  };

  next_tile();
#pragma unroll
  for (int i = 0; i < C::ST; ++i) produce();
  if (produced >= C::ST) wait_vmcnt<(C::ST - 1) * C::LOADS>();
  else wait_vmcnt<0>();
  __syncthreads();
  int g = 0;                                   // stages consumed
  uint32_t cbuf = 0;                           // and the buffer of the current one
  // The first reads of the stage in cbuf.
  auto first_reads = [&]() {
    read_scales(lds + cbuf);
    fp[0] = readP(lds + cbuf, 0);
    if (C::AHEAD == 2) fp[1] = readP(lds + cbuf, 1);
#pragma unroll
    for (int j = 0; j < C::MQ; ++j) fq[j] = readQ(lds + cbuf, j);
  };
  // On to the next stage: the current one is in registers and the next has
  // landed; one barrier frees the one buffer and publishes the other.  (Behind
  // the launch's last stage the reads fetch values that nothing uses.)
  auto next_stage = [&]() {
    if (g + C::ST <= produced) wait_vmcnt<(C::ST - 2) * C::LOADS>();
    else wait_vmcnt<0>();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __syncthreads();
    produce();
    ++g;
    cbuf = cbuf == (uint32_t)((C::ST - 1) * C::STAGE) ? 0u : cbuf + (uint32_t)C::STAGE;
  };
  first_reads();
  while (nahead > 0) {
    const Tile t = ahead[0];
#pragma unroll
    for (int u = 0; u < C::ST; ++u) ahead[u] = ahead[u + 1];
    --nahead;
    if (nk == 0) next_tile();                  // nothing to load: zeros are stored
    // a wave none of whose rows exist takes part in the loads only: a tile of
    // half the rows leaves the matrix cores to the other half's waves
    const bool rows = __builtin_amdgcn_readfirstlane(t.q0 + wq * C::WTQ < t.q_end);
    if (!rows) {
      for (int kt = 0; kt < nk; ++kt) next_stage();
      first_reads();
      continue;
    }
    for (int kt = 0; kt < nk; ++kt) {
      float s[C::MQ];
      f32x4 part[2][C::MQ];
      // result block (i, j) of the stage into its accumulator.  The empty use
      // pins it here: a product has no side effects, and the compiler would
      // else move whole rows of them behind the waits and the barrier below,
      // with every fragment held in registers until then.
      auto add = [&](int i, int j) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[i][j][e] = __builtin_fmaf(part[i & 1][j][e], s[j], acc[i][j][e]);
        asm volatile("" : "+v"(acc[i][j]));
      };
      const char* st = lds + cbuf;
#pragma unroll
      for (int i = 0; i < C::MP; ++i) {
        const bool last = i == C::MP - 1;
        if (i + C::AHEAD < C::MP) fp[(i + C::AHEAD) % C::RING] = readP(st, i + C::AHEAD);
        __builtin_amdgcn_sched_barrier(0);           // (the read stays ahead of the products)
        if (last) {
          next_stage();
          read_scales(lds + cbuf);
          fp[0] = readP(lds + cbuf, 0);
          if (C::AHEAD == 2) fp[1] = readP(lds + cbuf, 1);
        }
#pragma unroll
        for (int j = 0; j < C::MQ; ++j) {
          part[i & 1][j] = product(fp[i % C::RING], fq[j]);
          if (last) fq[j] = readQ(lds + cbuf, j);
          if (i > 0) add(i - 1, j);
        }
        if (i == 0) {                                // (under the first products, no sums to add yet)
          bool odd = false;
#pragma unroll
          for (int j = 0; j < C::MQ; ++j) {
            asm volatile("" ::"v"(part[0][j]));      // (not moved behind the branch)
            s[j] = rawq[j] * raww;
            odd |= factor_odd(s[j]);
          }
          if (__builtin_expect(__builtin_amdgcn_ballot_w64(odd) != 0, 0)) {
            // Rows with an odd factor: the stage is added to them here, and with
            // the factor 0 below.  (The check costs at most 1% where tiles are
            // small: 8 experts, 512 rows each, N = 768, K = 2512: 24.9 -> 25.2 us;
            // such rows in every tile make it 45 us.)  A row of zero codes, whose
            // scale is the quantizer's least and may make an odd factor with any
            // small weight's, needs no sums.
            uint32_t any = 0;
#pragma unroll
            for (int j = 0; j < C::MQ; ++j) {
              uint32_t bits = 0;
#pragma unroll
              for (int w = 0; w < 8; ++w) bits |= (uint32_t)fq[j][w];
              any |= factor_odd(s[j]) ? bits & 0x7F7F7F7Fu : 0u;
            }
            const bool sums = __builtin_amdgcn_ballot_w64(any != 0) != 0;
            Factor f[C::MQ];
#pragma unroll
            for (int j = 0; j < C::MQ; ++j) {
              f[j] = factor_odd(s[j]) ? split_factor(rawq[j], raww, s[j]) : Factor{0.f, 1.f};
              if (factor_odd(s[j])) s[j] = 0.f * f[j].m;     // (NaN of a scale that is none)
            }
            if (sums) {
#pragma unroll
              for (int r = 0; r < C::MP; ++r) {
                const i32x8 p = readP(st, r);
#pragma unroll
                for (int j = 0; j < C::MQ; ++j) {
                  const f32x4 v = product(p, fq[j]);
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    acc[r][j][e] = __builtin_fmaf(v[e] * f[j].c, f[j].m, acc[r][j][e]);
                  // (one at a time: with more registers here the usual path is 2% slower)
                  __builtin_amdgcn_sched_barrier(0);
                }
              }
            }
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int j = 0; j < C::MQ; ++j) add(C::MP - 1, j);
    }
    store(t);
#pragma unroll
    for (int i = 0; i < C::MP; ++i)
#pragma unroll
      for (int j = 0; j < C::MQ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  wait_vmcnt<0>();
}

// ------------------------------------------------------------ few-row kernel --

// Where experts have few rows a weight fragment meets one or two row blocks, so
// no tile is shared between waves.  A workgroup of NW waves computes 16 PB P
// indices x 32 rows; the waves take every NW-th scale block, U blocks in
// flight, and their fp32 sums meet in LDS in wave order.  FWD's fragments (16
// rows x 128 contiguous bytes) come straight from memory into registers;
// DGRAD's weights, whose steps lie in different rows, pass through a part of
// LDS of the wave's own, from which they are read transposed.
constexpr int kFewQ = 32;

template <bool DG, int PB, int NW, int U>
__global__ __launch_bounds__(64 * NW, DG || PB == 2 ? 4 : 3) void fp8_few_rows_kernel(Fp8Args a) {
  constexpr int P = 16 * PB;
  static_assert(128 % P == 0, "one weight scale per tile and block");
  static_assert(!DG || PB == 4, "the weights' places in LDS");
  constexpr int kBlock = kBlk * P;                   // DGRAD: one block's weights
  constexpr int kSums = 2 * PB * 64 * 16, kOwn = DG && U * kBlock > kSums ? U * kBlock : kSums;
  __shared__ int sched[2 * (kMaxExperts + 1)];
  __shared__ __attribute__((aligned(16))) char own[NW][kOwn];
  const int red = (int)(DG ? a.N : a.K), Pdim = (int)(DG ? a.K : a.N);
  const int64_t ldw = a.K;
  const int nk = (red + kBlk - 1) / kBlk, np = (Pdim + kBlk - 1) / kBlk;
  const int tilesP = (Pdim + P - 1) / P;
  Experts X{sched, sched + kMaxExperts + 1, a.E, 0};
  setup_experts<kFewQ>(a.offsets, (int)a.M, X);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g4 = lane >> 4;
  // DGRAD: block u's 128 rows of 64 bytes, chunk c of row r at c ^ (r / 4 % 2)
  // ^ (2 (r / 32 % 2)): the transpose reads of 8 rows by two lane groups, 32
  // rows apart, hit 16 distinct 16-byte banks.  Piece j of a block is rows
  // 16 j .. + 15, a lane's chunk being that of piece 0 with j / 2 % 2 in bit 1.
  const int drow = lane >> 2, dcol = 16 * ((lane & 3) ^ ((drow >> 2) & 1));
  const int trow = 32 * g4 + (l16 >> 1);
  const uint32_t toff = (uint32_t)trow * P + 16u * (uint32_t)(2 * (g4 & 1) ^ ((trow >> 2) & 1)) +
                        8u * (uint32_t)(l16 & 1);
  Items<P, kFewQ, false> items;
  items.init(X.mtiles * tilesP, tilesP, max(X.mtiles, 1));
  Tile t = {0, 0, 0, 0};
  while (items.next(X, tilesP, max(X.mtiles, 1), t)) {
    const int rows = min(t.q_end - t.q0, kFewQ), cols = min(Pdim - t.p0, P);
    const bool two = rows > 16;
    const uint8_t* w = static_cast<const uint8_t*>(a.w8) + (int64_t)t.e * a.N * a.K;
    const auto rw = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(w + (DG ? 0 : (int64_t)t.p0 * ldw)), (short)0,
        DG ? 0 : cols * (int)ldw, 0x00020000);
    const auto rx = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(static_cast<const uint8_t*>(a.q8)) + (int64_t)t.q0 * red, (short)0,
        rows * red, 0x00020000);
    // the weights' scale of block kb
    const int64_t sblock = DG ? np : 1;
    const float* wsc = a.ws + (DG ? (int64_t)t.e * nk * np + t.p0 / kBlk
                                  : ((int64_t)t.e * np + t.p0 / kBlk) * nk);
    f32x4 acc[PB][2];
#pragma unroll
    for (int i = 0; i < PB; ++i) acc[i][0] = acc[i][1] = f32x4{0.f, 0.f, 0.f, 0.f};
    // 32 bytes of row `row`, zeros past the reduction's end or the valid rows
    auto frag = [&](auto rs, int row, int kb) {
      const uint32_t col = (uint32_t)(kb * kBlk + 32 * g4);
      const uint32_t off = (uint32_t)row * (uint32_t)red + col;
      const i32x4 lo = __builtin_bit_cast(
          i32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, (int)(off | (col < (uint32_t)red ? 0u : kOOB)), 0, 0));
      const i32x4 hi = __builtin_bit_cast(
          i32x4, __builtin_amdgcn_raw_buffer_load_b128(
                     rs, (int)((off + 16u) | (col + 16u < (uint32_t)red ? 0u : kOOB)), 0, 0));
      return (i32x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    // DGRAD: block kb's weights to the wave's LDS; rows and columns past their
    // ends, and blocks past nk, are zeros
    auto stage = [&](int u, int kb) {
      const int left = min(red - kb * kBlk, kBlk);
      const i32x4 rs = rsrc_of(w + (int64_t)(left > 0 ? kb : 0) * kBlk * ldw + t.p0,
                               left > 0 ? (uint32_t)(left - 1) * (uint32_t)ldw + (uint32_t)cols : 0u);
      const uint32_t to = lds_addr_of(own[wave]) + (uint32_t)(u * kBlock);
      uint32_t off[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = dcol ^ (32 * ((j >> 1) & 1));
        off[j] = c < cols ? (uint32_t)(16 * j + drow) * (uint32_t)ldw + (uint32_t)c : kOOB;
      }
      load_block(rs, to, off);
    };
    auto staged = [&](int u, int i) {
      typedef __attribute__((address_space(3))) i32x2 lds_i32x2;
      auto tr = [&](uint32_t off) {
        return __builtin_amdgcn_ds_read_tr8_b64_v2i32(
            (lds_i32x2*)((__attribute__((address_space(3))) char*)(
                             (__attribute__((address_space(3))) void*)own[wave]) + u * kBlock + off));
      };
      // rows 8 further: r / 4 % 2 and r / 32 % 2 are the same
      const uint32_t o = toff ^ (uint32_t)(16 * i);
      const i32x2 a0 = tr(o), a1 = tr(o + 8 * P), a2 = tr(o + 16 * P), a3 = tr(o + 24 * P);
      const i32x4 lo = __builtin_shufflevector(a0, a1, 0, 1, 2, 3);
      const i32x4 hi = __builtin_shufflevector(a2, a3, 0, 1, 2, 3);
      return (i32x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    for (int k0 = wave; k0 < nk; k0 += NW * U) {
      i32x8 fw[U][PB], fx[U][2];
      float s[U][2];
      // (the reads of the last round's blocks are done)
      if constexpr (DG) asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int kb = k0 + NW * u;                  // past nk: the loads read zeros
        if constexpr (DG) {
          stage(u, kb);
        } else {
#pragma unroll
          for (int i = 0; i < PB; ++i) fw[u][i] = frag(rw, 16 * i + l16, kb);
        }
        fx[u][0] = frag(rx, l16, kb);
        if (two) fx[u][1] = frag(rx, 16 + l16, kb);
        const bool in = kb < nk;
        const float sw = in ? wsc[kb * sblock] : 0.f;
        const float* xs = a.qs + (int64_t)(in ? kb : 0) * a.M + t.q0;
        s[u][0] = in && l16 < rows ? xs[l16] * sw : 0.f;
        s[u][1] = in && 16 + l16 < rows ? xs[16 + l16] * sw : 0.f;
      }
      if constexpr (DG) wait_vmcnt<0>();
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if constexpr (DG) {
#pragma unroll
          for (int i = 0; i < PB; ++i) fw[u][i] = staged(u, i);
        }
        auto add = [&](int h) {
          Factor f = {s[u][h], 1.f};
          if (__builtin_expect(__builtin_amdgcn_ballot_w64(factor_odd(f.m)) != 0, 0)) {
            // from the two scales, read again (a factor of a block past nk or of
            // a row past the last is zero, so the address is in the scales)
            const int kb = min(k0 + NW * u, nk - 1);
            if (factor_odd(f.m)) f = split_factor(a.qs[(int64_t)kb * a.M + t.q0 + 16 * h + l16], wsc[kb * sblock], f.m);
          }
#pragma unroll
          for (int i = 0; i < PB; ++i) {
            const f32x4 p = product(fw[u][i], fx[u][h]);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][h][e] = __builtin_fmaf(p[e] * f.c, f.m, acc[i][h][e]);
          }
        };
        add(0);
        if (two) add(1);
      }
    }
    auto sums = [&](int v) { return reinterpret_cast<f32x4*>(own[v]); };
    if constexpr (DG) asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    else __syncthreads();                            // the previous tile's sums are read
#pragma unroll
    for (int i = 0; i < PB; ++i) {
      sums(wave)[(2 * i) * 64 + lane] = acc[i][0];
      sums(wave)[(2 * i + 1) * 64 + lane] = acc[i][1];
    }
    __syncthreads();
    for (int b = wave; b < 2 * PB; b += NW) {        // a wave finishes result block b
      f32x4 r = sums(0)[b * 64 + lane];
#pragma unroll
      for (int v = 1; v < NW; ++v) r += sums(v)[b * 64 + lane];
      const int m = 16 * (b & 1) + l16, n = t.p0 + 16 * (b >> 1) + 4 * g4;
      if (m < rows && n < Pdim)
        *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(a.out) + (int64_t)(t.q0 + m) * Pdim + n) =
            u32x2{pack_bf16(r[0], r[1]), pack_bf16(r[2], r[3])};
    }
    if constexpr (DG) __syncthreads();               // the sums are read, the next tile's loads may land
  }
}

int device_cus() {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  int n = cache[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0)
      n = 256;
    cache[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// Upper bound of a launch's tiles: sum_e ceil(m_e / BQ) P-tiles.
int64_t tile_bound(const Fp8Args& a, int64_t pdim, int64_t max_m, int bp, int bq) {
  int64_t mt = (a.M + bq - 1) / bq + (a.E < a.M ? a.E : a.M);
  if (max_m > 0) {
    const int64_t alt = (int64_t)a.E * ((max_m + bq - 1) / bq);
    if (alt < mt) mt = alt;
  }
  return mt * ((pdim + bp - 1) / bp);
}

unsigned grid_of(int64_t tiles, int64_t cap) {
  cap &= ~int64_t(7);
  if (cap < 8) cap = 8;
  const int64_t g = (tiles + 7) & ~int64_t(7);
  return (unsigned)(g < cap ? g : cap);
}

// 256 x 256 tiles, one workgroup of 8 waves per compute unit, and 128 x 128
// tiles, two workgroups of 4 waves.
using Big = Fp8Cfg<256, 256, 2, 4, 2>;
using Small = Fp8Cfg<128, 128, 2, 2, 2>;

template <class C>
void launch_tiled(bool dgrad, const Fp8Args& a, int64_t tiles, int64_t cap, hipStream_t s) {
  // (twice the tiles: the last round's may be halved)
  const dim3 g(grid_of(2 * tiles, cap)), b(C::NT);
  if (dgrad) hipLaunchKernelGGL((fp8_gemm_kernel<true, C>), g, b, 0, s, a);
  else hipLaunchKernelGGL((fp8_gemm_kernel<false, C>), g, b, 0, s, a);
}

}  // namespace

int launch_fp8(bool dgrad, const Fp8Args& a, int64_t max_m, hipStream_t s) {
  const int64_t pdim = dgrad ? a.K : a.N;
  const int64_t cus = device_cus();
  // Which kernel: by the number of tiles that the buffer's rows give if they
  // spread evenly (the host does not see the offsets, nor how far the last of
  // them lies below M; every expert's last tile is half full on average).
  // Results do not depend on the spread, only speed.
  const int64_t live = a.E < a.M ? a.E : a.M;
  // Few rows: tiles of 32 rows.  With too few 128 x 128 tiles to fill the chip,
  // or too few rows to reuse a staged weight tile, a round of those is bound by
  // what its products do not hide, and this kernel is faster.  Measured (us,
  // this / tiled), FWD: 8 experts, N = 768, K = 2048: 6.0 / 17 at 1 row each,
  // 11 / 17 at 64, 22 / 17 at 128; N = 1408, K = 7168: 20 / 49 at 1 row, 46 / 49
  // at 64; 64 experts, N = 4096, K = 2048: 58 / 66 at 1, 95 / 99 at 4, 118 / 102
  // at 16 rows.  DGRAD: 3 experts, N = 3520, K = 2288: 10 / 30 at 1 row each,
  // 18 / 31 at 128; 16 experts: 29 / 34 at 16, 33 / 34 at 32, 47 / 41 at 64;
  // 64 experts, N = 416, K = 5904: 42 / 45 at 16, 51 / 45 at 32.
  int64_t mt = a.M / kFewQ + live / 2;
  if (mt < live) mt = live;
  const int64_t t64 = mt * ((pdim + 63) / 64);
  auto few = [&](auto kernel, int p, int nw, int64_t cap) {
    hipLaunchKernelGGL(kernel, dim3(grid_of(tile_bound(a, pdim, max_m, p, kFewQ), cap * cus)),
                       dim3(64 * nw), 0, s, a);
    return (int)hipGetLastError();
  };
  if (dgrad && (a.M <= 16 * live || t64 <= 4 * cus))
    // (16 experts, N = 768, K = 2048, 32 rows each: 9 us, with two blocks in
    // flight 12, LDS then holding one workgroup; 3 experts, N = 3520, K = 2288, 1
    // row: 10 us, with four waves 12)
    return few(fp8_few_rows_kernel<true, 4, 8, 1>, 64, 8, 4);
  if (!dgrad && (a.M < 8 * live || t64 <= 2 * cus))
    // eight waves per 32-column tile while there are few tiles (1 row for each
    // of 8 experts, K = 7168: 20 us against 25), else four per 64 columns, which
    // reads the rows half as often (16 rows, N = 4096: 17 against 20)
    return t64 <= cus ? few(fp8_few_rows_kernel<false, 2, 8, 2>, 32, 8, 4)
                      : few(fp8_few_rows_kernel<false, 4, 4, 2>, 64, 4, 8);
  // Tiled: the rounds of tiles over the chip times what a stage of a round
  // takes: 2 us for 256 x 256 tiles, 1.25 us for 128 x 128 tiles with two
  // workgroups per compute unit (0.9 us with one), less for a last round with
  // so few tiles that they are halved.  Measured over 96 shapes, this picks the
  // faster or one within 10% (us, large / small: FWD 8 experts, 2048 rows each,
  // N = 4096, K = 2048: 154 / 166; 1024 rows: 88 / 85; 128 rows: 25 / 23; DGRAD
  // 8 experts, 1024 rows, N = 4096, K = 2048: 108 / 96).
  auto tiles = [&](int64_t b) { return (2 * a.M / b + live + 1) / 2 * ((pdim + b - 1) / b); };
  auto rounds = [](double r, double full, double few, double last) {
    const int64_t n = (int64_t)r;
    const double part = r - (double)n;
    return full * (double)n + (part == 0 ? 0 : part <= few ? last : full);
  };
  const int64_t ts = tiles(128);
  const double big = rounds((double)tiles(256) / cus, 2.0, 0.5, 1.5);
  const double small = ts <= cus ? 0.9 : rounds((double)ts / (2 * cus), 1.25, ts < 2 * cus ? 0 : 0.3, 0.4);
  if (big <= small)
    launch_tiled<Big>(dgrad, a, tile_bound(a, pdim, max_m, Big::BP, Big::BQ), cus, s);
  else
    launch_tiled<Small>(dgrad, a, tile_bound(a, pdim, max_m, Small::BP, Small::BQ), 2 * cus, s);
  return (int)hipGetLastError();
}

}  // namespace mg
