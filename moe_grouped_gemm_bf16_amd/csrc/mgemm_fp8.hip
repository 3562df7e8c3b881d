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

// Direct-to-LDS loads: lane l's 16 (4) bytes land at lds_addr + 16 l (4 l).
// Awaited with vmcnt(0) before the barrier that publishes the stage.
__device__ __forceinline__ void to_lds16(const i32x4& rsrc, uint32_t lds_addr, uint32_t voff) {
  uint32_t save;
  asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\tbuffer_load_dwordx4 %2, %3, 0 offen lds\n\t"
               "s_mov_b32 m0, %0"
               : "=&s"(save) : "s"(lds_addr), "v"(voff), "s"(rsrc) : "memory");
}
__device__ __forceinline__ void to_lds4(const i32x4& rsrc, uint32_t lds_addr, uint32_t voff) {
  uint32_t save;
  asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\tbuffer_load_dword %2, %3, 0 offen lds\n\t"
               "s_mov_b32 m0, %0"
               : "=&s"(save) : "s"(lds_addr), "v"(voff), "s"(rsrc) : "memory");
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

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}

// ---------------------------------------------------------------- scheduler --

// The experts' row ranges and tile counts, in LDS: offs[e] is the clamped,
// non-decreasing offset (a broken offsets array then cannot move an access out
// of the tensors), pref[e] the exclusive prefix of ceil(rows / BQ).
struct Experts {
  int* offs;
  int* pref;
  int E, mtiles;
};

template <int BQ>
__device__ __forceinline__ void setup_experts(const int32_t* __restrict__ offsets, int M,
                                              Experts& X) {
  // every wave scans all experts (kMaxExperts / 64 per lane at most); wave 0 writes
  const int lane = threadIdx.x & 63, per = (X.E + 63) / 64;
  const bool writer = threadIdx.x < 64;
  int sum = 0;
  for (int j = 0; j < per; ++j) {
    const int e = lane * per + j;
    if (e >= X.E) break;
    const int lo = min(max(offsets[e], 0), M), hi = max(lo, min(max(offsets[e + 1], 0), M));
    sum += (hi - lo + BQ - 1) / BQ;
  }
  int incl = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(incl, d, 64);
    if (lane >= d) incl += y;
  }
  X.mtiles = __builtin_amdgcn_readlane(incl, 63);
  if (writer) {
    int run = incl - sum;
    for (int j = 0; j < per; ++j) {
      const int e = lane * per + j;
      if (e >= X.E) break;
      const int lo = min(max(offsets[e], 0), M), hi = max(lo, min(max(offsets[e + 1], 0), M));
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
// same time on one XCD share weight and activation panels in its L2.
template <int BP, int BQ>
__device__ __forceinline__ Tile tile_of(int L, const Experts& X, int tilesP, int gm) {
  int lo = 0, hi = X.E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (X.pref[mid] * tilesP <= L) lo = mid; else hi = mid - 1;
  }
  const int e = __builtin_amdgcn_readfirstlane(lo);
  const int local = L - X.pref[e] * tilesP;
  const int mt = X.pref[e + 1] - X.pref[e];
  const int g = local / (gm * tilesP);
  const int rem = local - g * gm * tilesP;
  const int gh = min(gm, mt - g * gm);
  const int tp = rem / gh;
  Tile t;
  t.e = e;
  t.q0 = __builtin_amdgcn_readfirstlane(X.offs[e] + (g * gm + rem - tp * gh) * BQ);
  t.q_end = __builtin_amdgcn_readfirstlane(X.offs[e + 1]);
  t.p0 = __builtin_amdgcn_readfirstlane(tp * BP);
  return t;
}

// Workgroup b runs on XCD b % 8; every XCD takes a contiguous range of tile
// ids, its workgroups every nx-th of them.
struct Walk {
  int at, end, step;
  __device__ __forceinline__ void init(int total) {
    const int x = blockIdx.x & 7, c = blockIdx.x >> 3;
    const int q8 = total >> 3, r8 = total & 7;
    const int lo = x * q8 + min(x, r8);
    end = lo + q8 + (x < r8 ? 1 : 0);
    at = lo + c;
    step = gridDim.x >> 3;
  }
};

// ------------------------------------------------------------- tiled kernel --

// BP x BQ output tile, WP x WQ waves; kStages LDS stages of 128 steps.
template <int BP_, int BQ_, int WP_, int WQ_, int ST_>
struct Fp8Cfg {
  static constexpr int BP = BP_, BQ = BQ_, WP = WP_, WQ = WQ_, ST = ST_;
  static constexpr int NW = WP * WQ, NT = 64 * NW;
  static constexpr int WTP = BP / WP, WTQ = BQ / WQ, MP = WTP / 16, MQ = WTQ / 16;
  static constexpr int P_BYTES = BP * kBlk, DATA = (BP + BQ) * kBlk;
  static constexpr int SCALES = NW * 256, STAGE = DATA + SCALES;
  static constexpr int SPW = DATA / 1024 / NW;           // 1 KiB loads per wave and stage
  static constexpr int SEGS_P = P_BYTES / 1024;
  static_assert(DATA / 1024 % NW == 0 && SEGS_P % SPW == 0 && SPW % 4 == 0, "loads per wave");
  static_assert(MP % 4 == 0 && WTP <= 128 && 128 % WTP == 0, "one weight scale per wave");
  static_assert(BQ / 64 + 1 <= NW && BQ % 64 == 0, "scale loads");
};

template <bool DG, class C>
__global__ __launch_bounds__(C::NT) void fp8_gemm_kernel(Fp8Args a) {
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
  const int wp = wave / C::WQ, wq = wave % C::WQ;
  const int l16 = lane & 15, g4 = lane >> 4;

  // ---- producer: stage loads of this wave, 1 KiB segments seg0 .. + SPW of
  // its operand's tile.  Steps-contiguous tiles are [rows][128] bytes in
  // 16-byte chunks, chunk c of row r at c ^ (r % 8) ^ (r / 8 % 4): 16 rows
  // read at one chunk hit 16 distinct 16-byte banks.  DGRAD's weights are
  // staged as they lie, [128 n][BP k], chunk c of row r at
  // c ^ (2 (r % 8)) ^ (r / 32 % 2) (BP = 256) or
  // c ^ (2 (r / 2 % 4)) ^ (r / 32 % 2) (BP = 128): the transpose reads of 8
  // rows by two lane groups, 32 rows apart, then hit 16 distinct banks.
  const bool isP = wave * C::SPW < C::SEGS_P;
  const int seg0 = isP ? wave * C::SPW : wave * C::SPW - C::SEGS_P;
  const uint32_t lds0 = lds_addr_of(lds);
  const uint32_t data0 = lds0 + (isP ? 0u : (uint32_t)C::P_BYTES) + (uint32_t)seg0 * 1024u;
  const uint32_t scale0 = lds0 + (uint32_t)C::DATA + (uint32_t)wave * 256u;
  const int ld = isP ? ldP : ldQ;
  const bool strided = DG && isP;
  constexpr int RPS = 1024 / (DG ? C::BP : kBlk);          // strided: rows per segment
  const int c0 = (lane & 7) ^ (lane >> 3);
  const uint32_t row0 = strided ? (uint32_t)(seg0 * RPS + lane / (C::BP / 16)) * (uint32_t)ld
                                : (uint32_t)(seg0 * 8 + (lane >> 3)) * (uint32_t)ld;

  Walk pw;
  pw.init(total);
  bool live = false;
  const uint8_t* psrc = nullptr;     // the operand's tile at reduction step 0
  const float* pscale = nullptr;     // the wave's scales at block 0
  int64_t pscale_step = 0;
  uint32_t psc_off = kOOB;           // this lane's scale, bytes from pscale
  uint32_t psc_range = 0;
  int pouter = 0, pkt = 0, produced = 0;
  auto next_tile = [&]() {
    live = pw.at < pw.end && nk > 0;
    if (!live) return;
    const Tile t = tile_of<C::BP, C::BQ>(pw.at, X, tilesP, gm);
    pw.at += pw.step;
    pkt = 0;
    const uint8_t* w = static_cast<const uint8_t*>(a.w8) + (int64_t)t.e * a.N * a.K;
    if (isP) {
      psrc = DG ? w + t.p0 : w + (int64_t)t.p0 * a.K;
      pouter = min(Pdim - t.p0, C::BP);
    } else {
      psrc = static_cast<const uint8_t*>(a.q8) + (int64_t)t.q0 * ldQ;
      pouter = min(t.q_end - t.q0, C::BQ);
    }
    // scales: waves 0 .. BQ/64 - 1 load 64 rows' each, the next wave the
    // weights' (one per 128 P indices); the other waves load nothing
    psc_off = kOOB;
    psc_range = 0;
    if (wave < C::BQ / 64) {
      pscale = a.qs + t.q0;
      pscale_step = a.M;
      const int rows = min((int)a.M - t.q0, C::BQ);
      psc_range = (uint32_t)rows * 4u;
      psc_off = (uint32_t)(wave * 64 + lane) * 4u;
    } else if (wave == C::BQ / 64) {
      const int pb = t.p0 / kBlk;
      const float* s = a.ws + (int64_t)t.e * nn * nkb;
      const int blocks = min((C::BP + kBlk - 1) / kBlk, (DG ? nkb : nn) - pb);
      pscale = DG ? s + pb : s + (int64_t)pb * nkb;
      pscale_step = DG ? nkb : 1;
      const uint32_t step = DG ? 4u : (uint32_t)nkb * 4u;
      psc_range = (uint32_t)(blocks - 1) * step + 4u;
      if (lane < blocks) psc_off = (uint32_t)lane * step;
    } else {
      pscale = a.qs;
      pscale_step = 0;
    }
  };
  // Issue the producer's next stage into LDS stage buffer produced % ST.
  auto produce = [&]() {
    if (!live) return;
    const int r0 = pkt * kBlk;
    const uint32_t buf = (uint32_t)(produced % C::ST) * (uint32_t)C::STAGE;
    i32x4 rs;
    if (strided) {
      const int rr = min(red - r0, kBlk);
      rs = rsrc_of(psrc + (int64_t)r0 * ld, (uint32_t)(rr - 1) * (uint32_t)ld + (uint32_t)pouter);
    } else {
      rs = rsrc_of(psrc + r0, (uint32_t)(pouter - 1) * (uint32_t)ld + (uint32_t)min(red - r0, kBlk));
    }
    const i32x4 ss = rsrc_of(pscale + pkt * pscale_step, psc_range);
    // (an opaque copy: the loads' offsets are not kept in registers between stages)
    uint32_t ro = row0;
    asm volatile("" : "+v"(ro));
#pragma unroll
    for (int j = 0; j < C::SPW; ++j) {
      uint32_t off;
      if (strided) {
        const int seg = seg0 + j, row = seg * RPS + lane / (C::BP / 16);
        const int sw = C::BP == 256 ? (2 * (row & 7)) ^ ((row >> 5) & 1)
                                    : (2 * ((row >> 1) & 3)) ^ ((row >> 5) & 1);
        const int col = 16 * ((lane % (C::BP / 16)) ^ sw);
        off = (ro + (uint32_t)(j * RPS) * (uint32_t)ld + (uint32_t)col) | (col < pouter ? 0u : kOOB);
      } else {
        const int col = 16 * (c0 ^ (j & 3));
        off = (ro + (uint32_t)(j * 8) * (uint32_t)ld + (uint32_t)col) |
              (r0 + col < red ? 0u : kOOB);
      }
      to_lds16(rs, data0 + buf + (uint32_t)j * 1024u, off);
    }
    to_lds4(ss, scale0 + buf, psc_off);
    ++produced;
    if (++pkt == nk) next_tile();
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
  auto readQ = [&](int g, int j) {
    const char* st = lds + (g % C::ST) * C::STAGE;
    return frag(st + j * 2048, offQ ^ (uint32_t)(32 * (j & 1)));
  };
  auto readP = [&](int g, int i) {
    const char* st = lds + (g % C::ST) * C::STAGE;
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
  static_assert(C::MQ % 2 == 0, "swizzle parity");

  f32x4 acc[C::MP][C::MQ];
#pragma unroll
  for (int i = 0; i < C::MP; ++i)
#pragma unroll
    for (int j = 0; j < C::MQ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  i32x8 fp[4], fq[C::MQ];
  float rawq[C::MQ], raww;
  auto read_scales = [&](int g) {
    const float* sc = reinterpret_cast<const float*>(lds + (g % C::ST) * C::STAGE + C::DATA);
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
  for (int s = 0; s < C::ST; ++s) produce();
  Walk cw;
  cw.init(total);
  auto first_reads = [&](int g) {
    read_scales(g);
    fp[0] = readP(g, 0);
    fp[1] = readP(g, 1);
  };
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (produced > 0) {
    first_reads(0);
#pragma unroll
    for (int j = 0; j < C::MQ; ++j) fq[j] = readQ(0, j);
  }
  int g = 0;
  for (; cw.at < cw.end; cw.at += cw.step) {
    const Tile t = tile_of<C::BP, C::BQ>(cw.at, X, tilesP, gm);
    for (int kt = 0; kt < nk; ++kt, ++g) {
      float s[C::MQ];
#pragma unroll
      for (int j = 0; j < C::MQ; ++j) s[j] = rawq[j] * raww;
      f32x4 part[C::MQ];
#pragma unroll
      for (int i = 0; i < C::MP; ++i) {
        if (i + 2 < C::MP) fp[(i + 2) & 3] = readP(g, i + 2);
        const bool last = i == C::MP - 1;
        if (last) {
          // stage g is in registers and stage g + 1 has landed: one barrier
          // frees the one buffer and publishes the other
          asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
          __syncthreads();
          produce();
          first_reads(g + 1);          // (of the launch's last stage: unused values)
        }
#pragma unroll
        for (int j = 0; j < C::MQ; ++j) {
          part[j] = product(fp[i & 3], fq[j]);
          if (last) fq[j] = readQ(g + 1, j);
        }
#pragma unroll
        for (int j = 0; j < C::MQ; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(part[j][e], s[j], acc[i][j][e]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    store(t);
#pragma unroll
    for (int i = 0; i < C::MP; ++i)
#pragma unroll
      for (int j = 0; j < C::MQ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// ------------------------------------------------------------ few-row kernel --

// FWD where experts have few rows: the weights are read once and nothing is
// reused, so there is no LDS staging.  A workgroup of four waves computes 32
// P indices x 32 rows; the waves take every fourth scale block, each loading
// its fragments straight into registers (16 rows x 128 contiguous bytes per
// fragment), four blocks in flight, and their fp32 sums meet in LDS in wave
// order.
constexpr int kFewP = 32, kFewQ = 32, kFewU = 4;

__global__ __launch_bounds__(256) void fp8_few_rows_kernel(Fp8Args a) {
  __shared__ int sched[2 * (kMaxExperts + 1)];
  __shared__ __attribute__((aligned(16))) f32x4 sums[4][4][64];
  const int N = (int)a.N, K = (int)a.K;
  const int nk = (K + kBlk - 1) / kBlk, nn = (N + kBlk - 1) / kBlk;
  const int tilesP = (N + kFewP - 1) / kFewP;
  Experts X{sched, sched + kMaxExperts + 1, a.E, 0};
  setup_experts<kFewQ>(a.offsets, (int)a.M, X);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g4 = lane >> 4;
  Walk w;
  for (w.init(X.mtiles * tilesP); w.at < w.end; w.at += w.step) {
    const Tile t = tile_of<kFewP, kFewQ>(w.at, X, tilesP, 1 << 20);
    const int rows = min(t.q_end - t.q0, kFewQ), cols = min(N - t.p0, kFewP);
    const bool two = rows > 16;
    const i32x4 rw = rsrc_of(static_cast<const uint8_t*>(a.w8) + ((int64_t)t.e * N + t.p0) * K,
                             (uint32_t)cols * (uint32_t)K);
    const i32x4 rx = rsrc_of(static_cast<const uint8_t*>(a.q8) + (int64_t)t.q0 * K,
                             (uint32_t)rows * (uint32_t)K);
    const float* wsc = a.ws + ((int64_t)t.e * nn + t.p0 / kBlk) * nk;
    f32x4 acc[2][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i >> 1][i & 1] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto frag = [&](const i32x4& rs, int row, int kb) {
      const uint32_t col = (uint32_t)(kb * kBlk + 32 * g4);
      const uint32_t off = (uint32_t)row * (uint32_t)K + col;
      const auto d = __builtin_amdgcn_make_buffer_rsrc(
          reinterpret_cast<void*>(((uint64_t)(uint32_t)rs.y << 32) | (uint32_t)rs.x), (short)0, rs.z, rs.w);
      const i32x4 lo = __builtin_bit_cast(
          i32x4, __builtin_amdgcn_raw_buffer_load_b128(d, (int)(off | (col < (uint32_t)K ? 0u : kOOB)), 0, 0));
      const i32x4 hi = __builtin_bit_cast(
          i32x4, __builtin_amdgcn_raw_buffer_load_b128(
                     d, (int)((off + 16u) | (col + 16u < (uint32_t)K ? 0u : kOOB)), 0, 0));
      return (i32x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    for (int k0 = wave; k0 < nk; k0 += 4 * kFewU) {
      i32x8 fw[kFewU][2], fx[kFewU][2];
      float s[kFewU][2];
#pragma unroll
      for (int u = 0; u < kFewU; ++u) {
        const int kb = k0 + 4 * u;                   // past nk: the loads read zeros
        fw[u][0] = frag(rw, l16, kb);
        fw[u][1] = frag(rw, 16 + l16, kb);
        fx[u][0] = frag(rx, l16, kb);
        if (two) fx[u][1] = frag(rx, 16 + l16, kb);
        const bool in = kb < nk;
        const float sw = in ? wsc[kb] : 0.f;
        const float* xs = a.qs + (int64_t)(in ? kb : 0) * a.M + t.q0;
        s[u][0] = in && l16 < rows ? xs[l16] * sw : 0.f;
        s[u][1] = in && 16 + l16 < rows ? xs[16 + l16] * sw : 0.f;
      }
#pragma unroll
      for (int u = 0; u < kFewU; ++u) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const f32x4 p = product(fw[u][i], fx[u][0]);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][0][e] = __builtin_fmaf(p[e], s[u][0], acc[i][0][e]);
        }
        if (two) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const f32x4 p = product(fw[u][i], fx[u][1]);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][1][e] = __builtin_fmaf(p[e], s[u][1], acc[i][1][e]);
          }
        }
      }
    }
    __syncthreads();                                 // the previous tile's sums are read
#pragma unroll
    for (int b = 0; b < 4; ++b) sums[wave][b][lane] = acc[b >> 1][b & 1];
    __syncthreads();
    // wave b finishes result block b
    const int i = wave >> 1, j = wave & 1;
    f32x4 r = sums[0][wave][lane];
#pragma unroll
    for (int v = 1; v < 4; ++v) r += sums[v][wave][lane];
    const int m = 16 * j + l16, n = t.p0 + 16 * i + 4 * g4;
    if (m < rows && n < N)
      *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(a.out) + (int64_t)(t.q0 + m) * N + n) =
          u32x2{pack_bf16(r[0], r[1]), pack_bf16(r[2], r[3])};
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

using Cfg = Fp8Cfg<128, 128, 2, 2, 2>;

}  // namespace

int launch_fp8(bool dgrad, const Fp8Args& a, int64_t max_m, hipStream_t s) {
  const int64_t pdim = dgrad ? a.K : a.N;
  const int cus = device_cus();
  // Few rows per expert: nothing of a weight tile is reused, and the kernel
  // that reads it straight into registers has shorter start-up.  Measured
  // (forward, N = 768, K = 2048, eight experts of one row each): 12 us against
  // 19 us; at 8 rows for each of 64 experts (N = 1536): 44 us against 39 us.
  if (!dgrad && a.M < 8 * (int64_t)a.E) {
    const int64_t tiles = tile_bound(a, pdim, max_m, kFewP, kFewQ);
    hipLaunchKernelGGL(fp8_few_rows_kernel, dim3(grid_of(tiles, 8 * cus)), dim3(256), 0, s, a);
  } else {
    const dim3 g(grid_of(tile_bound(a, pdim, max_m, Cfg::BP, Cfg::BQ), 2 * cus)), b(Cfg::NT);
    if (dgrad) hipLaunchKernelGGL((fp8_gemm_kernel<true, Cfg>), g, b, 0, s, a);
    else hipLaunchKernelGGL((fp8_gemm_kernel<false, Cfg>), g, b, 0, s, a);
  }
  return (int)hipGetLastError();
}

}  // namespace mg
