// Internal launchers shared between the kernel files and the C-ABI layer.
#pragma once

#include <hip/hip_runtime.h>
#include <hip/hip_ext.h>
#include <stdint.h>

namespace moe {

// ---- dequant.hip
hipError_t launch_dequant(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t cols,
                          float* out, hipStream_t st);

// ---- lora.hip: low-rank adapters beside a projection
// The second half of an adapter's term, added where the projection is computed:
// out[t][o] += sum_r B[a_t][o][r] u[t][r] with u already scaled and zero past the adapter's
// rank.  B null: no adapters.
struct LoraSeg {
  const uint16_t* B = nullptr;         // [N][n_out][R]
  const int32_t* adapter = nullptr;    // [T]; ids outside [0, N) have no term
  const int32_t* rank = nullptr;       // nullable [N]
  const float* u = nullptr;            // [T][R], the GEMV's operand
  const uint16_t* ut = nullptr;        // [U_TERMS][T][rank_pad(R)] bf16, the matrix cores' operand: u is their sum
  int32_t N = 0, R = 0;
};
constexpr int U_TERMS = 3;  // of eight bits each: all 24 of an fp32 value
constexpr int LORA_MAX_RANK = 128;
constexpr int LORA_MAX_ADAPTERS = 1024;
// ranks on the matrix cores come in K steps of 32
__host__ __device__ constexpr int rank_pad(int R) { return (R + 31) / 32 * 32; }
struct LoraArgs {
  const uint16_t* x;       // [T][K]
  const uint16_t* A;       // [N][R][K]
  const uint16_t* B;       // [N][n_out][R]
  const float* scale;      // [N]
  const int32_t* rank;     // nullable [N]
  const int32_t* adapter;  // [T]
  int64_t T;
  int32_t K, N, R;
};
size_t lora_ws_bytes(int64_t T, int32_t K, int32_t N, int32_t R);
// u of every token into the workspace; *seg names it for launch_dense
hipError_t launch_lora_shrink(const LoraArgs& a, void* ws, LoraSeg* seg, hipStream_t st);

// ---- dense_gemv.hip
// One output "segment" of a dense bf16 GEMV over rows of W[rows][K].
struct DenseSeg {
  const uint16_t* W;
  int32_t rows;
  int32_t router;    // 0: out = bf16 [T][rows]; 1: out = fp32 [T][rows] (fp64-folded), wnorm, xnorm
  void* out;
  float* wnorm;      // router only: [rows] Euclidean row norms of W (fp32 sum of squares, rounded sqrt)
  float* xnorm;      // router only: [T] Euclidean norms of the tokens
  const float* add = nullptr;  // bf16 outputs only, nullable: fp32 [T][add_rows][rows] added before the rounding
  int32_t add_rows = 0;
};
// Relative accumulation error bound of router logits from launch_dense_gemv, per
// unit of |x_t| |w_e| (see the kernel for its derivation).
constexpr double GEMV_ROUTER_GAMMA = 16.0 / 8388608.0;  // 16 * 2^-23
// lora, when given, is the adapters' term of the last segment
// clear, when given, is memory that the launch sets besides
struct Clear {
  int32_t* zero = nullptr;  // nzero words, 32 apart, to 0
  int32_t nzero = 0;
  uint4* ones = nullptr;    // nones pieces of 16 bytes to all ones
  int32_t nones = 0;
};
hipError_t launch_dense_gemv(const uint16_t* x, int64_t T, int32_t K, const DenseSeg* segs, int nseg,
                             hipStream_t st, const LoraSeg* lora = nullptr, const Clear* clear = nullptr);

// ---- dense_mfma.hip: the same projections on the matrix cores for token batches
constexpr double DENSE_MFMA_ROUTER_GAMMA = 66.0 / 8388608.0;  // 66 * 2^-23
bool dense_uses_mfma(int64_t T, int32_t K);
// relative error bound of the router logits of launch_dense for T tokens of width K
double dense_router_gamma(int64_t T, int32_t K);
hipError_t launch_dense_mfma(const uint16_t* x, int64_t T, int32_t K, const DenseSeg& s, hipStream_t st,
                             const LoraSeg* lora = nullptr);
// the GEMV for few tokens, the matrix-core GEMM otherwise
hipError_t launch_dense(const uint16_t* x, int64_t T, int32_t K, const DenseSeg* segs, int nseg, hipStream_t st,
                        const LoraSeg* lora = nullptr);

// ---- route.hip
struct RouteArgs {
  const float* logits_fast;  // [T][E] unbiased fast logits (nullptr in topk mode)
  const float* xnorm;       // [T]
  const float* wnorm;       // [E]
  double gamma;              // relative error bound of logits_fast per |x||w|
  const float* exact_logits; // topk mode: [T][E] caller logits taken as exact (already biased)
  const float* bias;         // nullable
  int64_t bias_stride;
  const uint16_t* x;         // [T][d] for exact recompute
  const uint16_t* router_w;  // [E][d]
  int32_t d;
  int64_t T;
  int32_t E, k, renormalize, flags;
  int32_t* idx;              // [T][k]
  float* w;                  // [T][k]
  float* logits_out;         // nullable [T][E] biased logits
  int32_t* stats;            // [4] counters: tokens needing recompute, logits recomputed, Kulisch uses
  const uint16_t* h;         // nullable [T][L] latent rows to quantise for the experts
  int32_t L;
  int32_t mxfp8;             // 1: quantise h as MXFP8 (one term), 0: two exact e4m3 terms
  QRows hq;
};
hipError_t launch_route(const RouteArgs& a, hipStream_t st);

// Grouping of routed rows by expert.  tiles[0, n_active) = {expert, offset, count, first
// row} of the active experts, ascending; tiles[n_active, max_tiles) = {-1, 0, 0, -1}.
struct PermOut {
  int32_t* counts;    // [E]
  int32_t* offsets;   // [E+1]
  int32_t* perm;      // [T*k]
  int4* tiles;        // [max_tiles]
  int32_t* n_active;  // [1]
  int32_t max_tiles;  // min(E, T*k)
};
// routing, quantisation of h and the grouping in one block, for T <= ROUTE_FUSED_TOKENS
constexpr int ROUTE_FUSED_TOKENS = 8;
hipError_t launch_route_permute_small(const RouteArgs& a, const PermOut& p, hipStream_t st);
// grouping of the rows of routed tokens (distinct valid experts per token),
// T <= 64 and T*k <= ROUTE_SMALL_ROWS
constexpr int ROUTE_SMALL_ROWS = 1024;
constexpr int ROUTE_PLACE_TOKENS = 64;
hipError_t launch_place_rows(const int32_t* idx, int64_t T, int32_t k, int32_t E, const PermOut& p,
                             hipStream_t st);

// ---- permute.hip
constexpr int PERM_CHUNK = 2048;
size_t permute_ws_bytes(int64_t rows, int32_t E);
hipError_t launch_permute(const int32_t* idx, int64_t rows, int32_t E, const PermOut& out, void* ws,
                          hipStream_t st);

// ---- expert_mfma.hip
// Packed expert layout (moe_pack_experts): bytes of one 16-row group of a matrix with K
// columns, and of one expert.
__host__ __device__ constexpr int64_t packed_group_bytes(int K) {
  return (int64_t)(K / 128) * 1024 + (int64_t)((K / 128 + 3) / 4) * 256;
}
__host__ __device__ constexpr int64_t packed_expert_bytes(int L, int F) {
  return 2 * (int64_t)(F / 16) * packed_group_bytes(L) + (int64_t)(L / 16) * packed_group_bytes(F);
}
hipError_t launch_pack_experts(const uint8_t* src, uint8_t* dst, int E, int L, int F, hipStream_t st);

// Start and end events stamped by a kernel's own dispatch (hipExtLaunchKernelGGL): they
// bracket that kernel alone, with no launch gap; both null for a plain launch.
struct KernelEvents {
  hipEvent_t begin = nullptr, end = nullptr;
};
template <typename... Args, typename F = void (*)(Args...)>
inline hipError_t dispatch(const KernelEvents& ev, F kernel, dim3 grid, dim3 block, uint32_t lds, hipStream_t st,
                           Args... args) {
  if (ev.begin || ev.end)
    hipExtLaunchKernelGGL(kernel, grid, block, lds, st, ev.begin, ev.end, 0u, args...);
  else
    hipLaunchKernelGGL(kernel, grid, block, lds, st, args...);
  return hipGetLastError();
}

struct MxArgs {
  const uint8_t* blob;
  int32_t packed;            // 1: blob in the packed layout, 0: checkpoint records
  int32_t L, F, k;
  int64_t T;
  const int4* tiles;         // [max_active] {expert, offset in perm, rows, first row}; expert -1: none
  int32_t max_active;        // grid bound: min(E, T*k)
  const int32_t* perm;       // [T*k] slots t*k+j grouped by expert
  QRows hq;                  // [T][L] latent rows h, two-term e4m3
  QRows aq;                  // [T*k][F] GLU outputs by slot, two-term e4m3 (MXFP8 mode: lo term zero)
  int32_t mxfp8;             // activation format of aq (and of hq): MXFP8, else two exact e4m3 terms
  uint16_t* a_bf16;          // nullable [T*k][F] GLU outputs by slot, bf16
  float* y;                  // [T*k][L] down outputs by slot
  unsigned long long* clock; // nullable: MOE_CLOCK_SLOTS {start, end} pairs of the kernel's blocks (clock_begin/end)
  double* sal;               // nullable [T*k][sal_chunks]: per slot, the sum of y^2 over each block of latent rows
  int32_t sal_chunks;        // latent-row blocks of the down kernel that runs (down_*_sal_chunks)
};
hipError_t launch_gateup_mx(const MxArgs& p, hipStream_t st, const KernelEvents& ev = KernelEvents());
hipError_t launch_down_mx(const MxArgs& p, hipStream_t st, const KernelEvents& ev = KernelEvents());
bool down_combine_fits(int64_t T, int32_t k);
// latent-row blocks per routed row of each down kernel: the REAP partials it writes
int32_t down_mx_sal_chunks(int32_t L);
int32_t down_combine_sal_chunks(int32_t L);
hipError_t launch_down_combine_mx(const MxArgs& p, const int32_t* idx, const float* w, uint16_t* z,
                                  hipStream_t st, const KernelEvents& ev = KernelEvents());
hipError_t launch_quantize_rows(const uint16_t* src, int64_t rows, int K, const QRows& q, bool mxfp8, hipStream_t st);

// ---- expert_gemm.hip: grouped GEMMs for experts with many routed rows
// tiles of up to 64 routed rows per active expert, built from counts/offsets, followed by
// their count (GEMM_TILES_TAIL_BYTES): gemm_tiles_bytes in all
constexpr int GEMM_TILES_TAIL_BYTES = 16;
int64_t gemm_max_tiles(int64_t rows, int32_t E);
size_t gemm_tiles_bytes(int64_t rows, int32_t E);
hipError_t launch_gemm_tiles(const int32_t* counts, const int32_t* offsets, int32_t E, int4* gtiles,
                             int64_t max_gtiles, hipStream_t st);
hipError_t launch_gateup_gemm(const MxArgs& p, const int4* gtiles, int64_t max_gtiles, hipStream_t st,
                              const KernelEvents& ev = KernelEvents());
hipError_t launch_down_gemm(const MxArgs& p, const int4* gtiles, int64_t max_gtiles, hipStream_t st,
                            const KernelEvents& ev = KernelEvents());
int32_t down_gemm_sal_chunks(int32_t L);

// ---- stream.hip: expert records fetched from host memory into HBM slots
// copies the record of active expert j (tiles[j].x, j < *n_active) from src (device-
// readable host memory, expert_bytes per record) into slot j of dst
hipError_t launch_gather_experts(const uint8_t* src, int64_t expert_bytes, const int4* tiles, const int32_t* n_active,
                                 int32_t max_slots, uint8_t* dst, hipStream_t st);
// the grouping renumbered to slots (active expert j -> expert j): tiles_s [max_slots],
// counts_s [max_slots], offsets_s [max_slots + 1], idx_s [rows]
hipError_t launch_remap_to_slots(const int4* tiles, const int32_t* n_active, int32_t max_slots, const int32_t* counts,
                                 const int32_t* offsets, const int32_t* idx, int64_t rows, int4* tiles_s,
                                 int32_t* counts_s, int32_t* offsets_s, int32_t* idx_s, hipStream_t st);

// ---- reap.hip: saliency[e] += sum over e's rows (perm order) of w[slot] ||y[slot]||_2
hipError_t launch_reap_saliency(const float* y, const float* w, const int32_t* perm, const int32_t* offsets,
                                int32_t E, int32_t L, double* saliency, hipStream_t st);
// the same sums from the down kernels' partials: ||y[slot]||^2 = sum over c of sal[slot][c]
hipError_t launch_reap_partials(const double* sal, int32_t nch, const float* w, const int32_t* perm,
                                const int32_t* offsets, int32_t E, double* saliency, hipStream_t st);
// bias[e] = 0 for the n_keep experts of highest saliency (ties to the lower index, NaN
// lowest), -inf for the others
hipError_t launch_reap_keep_bias(const double* saliency, int32_t E, int32_t n_keep, float* bias, hipStream_t st);

// ---- decode.hip: a few tokens' layer behind the router logits and the latent rows
constexpr int DECODE_MAX_TOKENS = 8;
constexpr int DECODE_MAX_ROWS = 64;   // T * k
int32_t decode_counters(int32_t L);   // counters, 32 words apart, zero when the kernel starts
struct DecodeArgs {
  RouteArgs r;               // h set; idx, w and hq unused
  const uint8_t* blob;
  int32_t F;
  const uint16_t* latent_up;  // [d][L]
  uint8_t* aq;               // decode_aq_bytes(T*k, F): the GLU rows by slot, quantised
  uint16_t* z;               // [T][L], all ones when the kernel starts
  uint32_t* u;               // [T][R of lora] fp32 bits, likewise
  uint16_t* out;             // [T][d]
  float* y;                  // [T*k][L]
  int32_t* ctr;              // [32 * decode_counters(L)]
  LoraSeg lora;              // of latent_up, its u unused
  const uint16_t* lora_a;    // [N][R][L]
  const float* lora_scale;   // [N]
  // the caller's, nullable
  int32_t* idx;
  float* w;
  int32_t* counts;
  int32_t* offsets;
  int32_t* perm;
  // set by the launcher
  int32_t stage_offset;              // the waves' LDS rows of the down operand
  int32_t up_rows, slab_rows, slab_offset;  // a block's up rows, and those of them that wait in its LDS
};
size_t decode_aq_bytes(int64_t rows, int32_t F);
hipError_t launch_decode(const DecodeArgs& a, bool packed, hipStream_t st);

// ---- combine.hip
hipError_t launch_combine(const float* y, const float* w, int64_t T, int32_t k, int32_t L, uint16_t* z,
                          hipStream_t st);

// ---- ffn.hip: the dense gated block and its backward pass
struct FfnLayout {
  size_t a, dgu, finite, part, total;  // workspace: GLU rows, dG | dU, x and dout for low halves, pieces of split sums
};
struct FfnArgs {
  const uint16_t *x, *w_gate, *w_up, *w_down;  // [T][d], [F][d], [F][d], [d][F]
  int64_t T;
  int32_t d, F;
  uint16_t *out, *gate, *up;  // [T][d]; nullable [T][F]
};
struct FfnBackArgs {
  const uint16_t *dout, *x, *w_gate, *w_up, *w_down, *gate, *up;
  int64_t T;
  int32_t d, F;
  uint16_t *dx, *dw_gate, *dw_up, *dw_down;  // nullable (dw_gate and dw_up together)
};
FfnLayout ffn_layout(int64_t T, int32_t d, int32_t F);
FfnLayout ffn_backward_layout(int64_t T, int32_t d, int32_t F);
hipError_t launch_ffn(const FfnArgs& p, void* ws, hipStream_t st);
hipError_t launch_ffn_backward(const FfnBackArgs& p, void* ws, hipStream_t st);

// Blocks of up to 256 threads a launch: a launch counts its threads in 32 bits, and 2^24 rows, a block
// each, are one too many.  Calls of more blocks take a launch for each part.
constexpr int64_t LAUNCH_BLOCKS = (int64_t)1 << 23;

// ---- norms.hip: the norms, gate and sum between two blocks of a residual stream
struct NormArgs {
  const uint16_t *y, *residual, *post, *pre, *gate;  // y, post, pre, gate nullable
  int64_t gate_stride;                               // 0: one row for all tokens, or d
  int64_t T;
  int32_t d;
  float scale, eps;
  uint16_t *out, *normed;  // with y; with pre
};
struct NormBackArgs {
  const uint16_t *dout, *dnormed, *y, *out, *post, *pre, *gate;
  int64_t gate_stride;
  int64_t T;
  int32_t d;
  float scale, eps;
  uint16_t *dresidual, *dy, *dgate_rows;  // nullable
  float *dpre, *dpost, *dgate;            // nullable, [d]
  float* part;                            // set by the launcher: [3][blocks][d]
  int32_t sums;                           // set by the launcher: which of dpre, dpost, dgate
};
size_t norms_backward_ws_bytes(int64_t T, int32_t d);
hipError_t launch_block_norms(const NormArgs& a, hipStream_t st);
hipError_t launch_block_norms_backward(const NormBackArgs& a, void* ws, hipStream_t st);

// ---- int8.hip: a projection in 8-bit integers and its quantiser
struct Int8Layout {
  size_t scale, q, part, total;  // workspace: the tokens' scales and codes, pieces of split sums
};
Int8Layout int8_layout(int64_t T, int32_t n_in, int32_t n_out, bool quantize);
hipError_t launch_quantize_int8(const uint16_t* x, int64_t T, int32_t n, int8_t* q, float* scale, hipStream_t st);
hipError_t launch_linear_int8(const int8_t* q, const float* xs, const int8_t* W, const float* ws, int64_t T, int32_t n_in,
                              int32_t n_out, uint16_t* out, int32_t* part, hipStream_t st);

}  // namespace moe
