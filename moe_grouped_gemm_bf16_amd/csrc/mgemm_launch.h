// Internal interface between the C-ABI layer and the gfx950 kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mg {

enum { kFwd = 0, kDgrad = 1, kWgrad = 2, kFwdSwiglu = 3, kList = 4, kFwdMx = 5, kWgradMx = 6,
       kDgradSwiglu = 7, kWgradMxT = 8 };

// Largest expert count a launch accepts: the device-side scheduler keeps the
// per-expert tile prefix in LDS, two entries per thread of a 512-thread block.
constexpr int kMaxExperts = 1024;

// Most workgroups of 256 threads in one grid dimension: a dimension holds less
// than 2^32 threads.
constexpr int64_t kMaxBlocks256 = (int64_t(1) << 24) - 1;

// One group of the descriptor-list call (same layout as mg_gemm_desc of the
// C ABI): D [m, n] = A [m, k] B [n, k]^T, row strides in elements.
struct ListDesc {
  const void* a;
  const void* b;
  void* d;
  int32_t m, n, k;
  int32_t lda, ldb, ldd;
};

struct KernelArgs {
  const void* p_src;        // FWD/DGRAD: W [E,N,K]; FWD_SWIGLU: W13 [E,N=2I,K]; WGRAD: X [M,K];
                            // FWD_MX: W8 [E,N,K] E4M3 codes; WGRAD_MX: X^T [K,M] E4M3 codes;
                            // WGRAD_MX_T: X8 [M,K] E4M3 codes (token-major)
  const void* q_src;        // FWD: X [M,K]; FWD_SWIGLU: X [M or T,K]; DGRAD/WGRAD: dY [M,N];
                            // FWD_MX: X8 [M,K] E4M3 codes; WGRAD_MX: dY^T [N,M] E4M3 codes;
                            // WGRAD_MX_T: dY8 [M,N] E4M3 codes (token-major)
  const int32_t* offsets;   // [E+1], device
  void* out;                // FWD: Y [M,N] bf16; FWD_SWIGLU: H [M,N/2] bf16; DGRAD: dX [M,K] bf16;
                            // DGRAD_SWIGLU: dGU [M,2K] bf16 (dg | du);
                            // WGRAD, WGRAD_MX, WGRAD_MX_T: dW [E,N,K] fp32
  int64_t M, N, K;
  int32_t E;
  int32_t accumulate;       // WGRAD only: add into `out`
  const ListDesc* list;     // LIST: E descriptors (device)
  const int32_t* gather;    // FWD_SWIGLU: row i of the problem is row gather[i] of x (or NULL)
  int64_t T;                // FWD_SWIGLU with gather: rows of x
  float* ws;                // WGRAD token split: 2 slots of 256 x 256 fp32 per split tile
  uint32_t* tickets;        // one word per split tile (see ticket_mark)
  uint32_t ticket_mark;     // this launch's odd ticket value, 2 g + 1 for a launch count g
  const uint8_t* p_scale;   // FWD_MX: W's E8M0 scales, blocked [E][ceil(K/128)][N][4];
                            // WGRAD_MX, WGRAD_MX_T: X's, blocked [M/128][K][4]
  const uint8_t* q_scale;   // FWD_MX: X's E8M0 scales, blocked [ceil(K/128)][M][4];
                            // WGRAD_MX, WGRAD_MX_T: dY's, blocked [M/128][N][4]
  void* aux;                // FWD_SWIGLU: optional gu [M, N] bf16 out (pre-activation g | u);
                            // DGRAD_SWIGLU: gu [M, 2K] bf16 in
};

// Token-order combine: out[t, :] = sum_j w[t, j] rows[token_rows[t, j], :]
// (bf16 rows [M, D], token_rows int32 [T, k], weights fp32 [T, k] or NULL, out
// bf16 [T, D]).  Returns a hipError_t value.
int launch_moe_combine(const uint16_t* rows, const int32_t* token_rows, const float* weights,
                       uint16_t* out, int64_t M, int64_t T, int32_t k, int64_t D, hipStream_t s);

// Rearrange E8M0 scales [batch][rows][K/32] into the blocked layout
// [batch][ceil(K/128)][rows][4] (absent blocks 127).  Returns a hipError_t value.
int launch_mx_scales_blocked(const uint8_t* src, uint8_t* dst, int64_t rows, int64_t K,
                             int64_t batch, hipStream_t s);

// Block-scaled fp8 products: E4M3 codes, one fp32 scale per row and 128
// reduction steps of q8, one per 128 x 128 block of w8.
struct Fp8Args {
  const void* w8;           // [E, N, K]
  const float* ws;          // [E, ceil(N/128), ceil(K/128)]
  const void* q8;           // forward: x8 [M, K]; input gradient: dy8 [M, N]
  const float* qs;          // forward: [ceil(K/128), M]; input gradient: [ceil(N/128), M]
  const int32_t* offsets;   // [E+1], device
  void* out;                // bf16: y [M, N] or dx [M, K]
  int64_t M, N, K;
  int32_t E;
};
int launch_fp8(bool dgrad, const Fp8Args& a, int64_t max_m_per_e, hipStream_t s);

// Rows to block-scaled fp8: codes [M, K], scales [ceil(K/128), M]; with
// `gather`, row i is row gather[i] of x [T, K]; with `offsets` (E entries + 1,
// device) only rows below offsets[E] are written.  With swiglu x is g | u
// [M, 2 K] (bf16) and the values silu(g) u.
struct Fp8RowsArgs {
  const void* x;
  const int32_t* gather;
  const int32_t* offsets;
  void* codes;
  float* scales;
  int64_t M, T, K;
  int32_t E;
};
int launch_fp8_rows(const Fp8RowsArgs& a, bool fp32, bool swiglu, hipStream_t s);
// Weights [E, N, K] to codes [E, N, K] and scales [E, ceil(N/128), ceil(K/128)].
int launch_fp8_weights(const void* w, bool fp32, uint8_t* codes, float* scales, int64_t E, int64_t N,
                       int64_t K, hipStream_t s);

// Router forward (see mg_moe_route); per_group is set by the launch.
struct RouteArgs {
  const void* logits;       // [T, E] fp32 or bf16
  const uint8_t* mask;      // [T] or NULL
  int64_t T;
  int32_t E, k, normalize, first, local;
  float* weights;           // [T, k]
  int32_t* experts;         // [T, k]
  float* lse;               // [T]
  int32_t* counts;          // [E]
  float* prob_sum;          // [E]
  int32_t* tokens;          // [1]
  float* loss;              // [2]
  int32_t* offsets;         // [local + 1]
  int32_t* gather;          // [T k]
  int32_t* token_rows;      // [T, k]
  void* workspace;
  int64_t per_group;        // tokens per workgroup of the token pass
};
int64_t route_workspace_bytes(int64_t T, int32_t E);
int launch_route(const RouteArgs& a, bool bf16, hipStream_t s);

struct RouteBwdArgs {
  const void* logits;       // [T, E] fp32 or bf16
  const float* weights;     // [T, k]
  const int32_t* experts;   // [T, k]
  const float* lse;         // [T]
  const int32_t* counts;    // [E]
  const int32_t* tokens;    // [1]
  const float* dweights;    // [T, k] or NULL
  const float* dloss;       // [2] or NULL
  void* dlogits;            // [T, E] as the logits
  int64_t T;
  int32_t E, k, normalize;
};
int launch_route_bwd(const RouteBwdArgs& a, bool bf16, hipStream_t s);

// Gradient of the token-order combine: drows[token_rows[t, j]] = w[t, j] dout[t]
// and, with weights, dweights[t, j] = <rows[token_rows[t, j]], dout[t]>.
int launch_moe_combine_bwd(const uint16_t* dout, const uint16_t* rows, const int32_t* token_rows,
                           const float* weights, uint16_t* drows, float* dweights, int64_t M,
                           int64_t T, int32_t k, int64_t D, hipStream_t s);

// Losses of the output head: cross entropy (targets) or distillation (teacher,
// index), and their gradients (see mg_head_loss and mg_head_distill).
struct HeadArgs {
  const uint16_t* x;          // [T, D] bf16
  const uint16_t* w;          // [V, D] bf16
  int64_t T, V, D;
  int64_t first;              // vocabulary index of w's row 0
  const int32_t* targets;     // [T], cross entropy
  const void* teacher;        // [T, k] fp32 or bf16, distillation
  const int32_t* index;       // [T, k], or NULL: cross entropy
  int32_t k, teacher_bf16;
  double c;                   // 1 / temperature (1 for cross entropy)
  float scale;                // c log2(e)
  float* loss;                // forward: [T]
  float* lse;                 // [T]
  float* logits;              // [T] or [T, k]
  const float* lse_in;        // backward: the forward's
  const float* logits_in;     // [T, k]
  const float* dloss;         // [T]
  const float* dlse;          // [T] or NULL
  uint16_t* dx;               // [T, D] bf16 or NULL
  uint16_t* dw;               // [V, D] bf16 or NULL
  void* workspace;
};
int64_t head_workspace_bytes(int64_t T, int64_t V, int64_t D);
int64_t head_bwd_workspace_bytes(int64_t T, int64_t V, int64_t D, int32_t k);
int launch_head(const HeadArgs& a, hipStream_t s);
int launch_head_bwd(const HeadArgs& a, hipStream_t s);

// Where the weight gradient's token split takes its workspace from.
enum WsKind {
  kWsStream = 0,   // a device allocation per (device, stream), made on first use
  kWsStatic = 1,   // the library's static device array (one per device); never allocates
};

// Enqueue one grouped GEMM on stream `s`.  Returns a hipError_t value.
int launch_grouped(int mode, const KernelArgs& a, int64_t max_m_per_e, hipStream_t s,
                   WsKind ws = kWsStream);

}  // namespace mg
