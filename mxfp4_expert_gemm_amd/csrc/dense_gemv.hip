// Dense bf16 GEMV for few tokens: router logits and the latent projections.
//
// out[t][r] = sum_i x[t][i] * W[r][i] over rows of W[rows][K] (kimi-k3-mlx digest,
// architecture table: the router scores 896 experts from the 7168-wide token;
// Stable LatentMoE projects 7168 -> 3584 and back with bf16 matrices).
//
// Memory-bound: every weight byte is read once per token group, so sums are kept in
// fp64 (fp32 partials of 8 exact products folded into fp64) at no cost in time; the
// bf16 outputs are then the correctly rounded sums but for fp64-level ties.  One wave owns one
// row; lane l reads 16 bytes (8 bf16) at column 8*(64c + l) for chunk c, so each
// load instruction covers 1 KiB of the row contiguously, and reads the matching token
// values from the block's copy of the token rows in LDS.  Products of bf16 pairs are
// exact in fp32 (v_dot2_f32_bf16).
//
// Router rows fold each 8-element chunk partial into an fp64 accumulator.  Error
// bound: a chunk partial is 4 dot2 steps from zero, at most 8 fp32 roundings of
// partial sums bounded by the chunk's sum of |products| (2^-23 each, covering
// round-toward-zero too); the fp64 folds and the 6-step wave tree add at most
// (NCH + 6) * 2^-53 relative to the sum of |products|.  With S = sum |x_i w_i|
// <= |x| |w|, the error of the fp64 logit is below 8.0001 * 2^-23 * |x||w|;
// GEMV_ROUTER_GAMMA = 16 * 2^-23 leaves a factor of two for the fp32 norm sums.
// A token or router row holding a subnormal bf16 value (which the dot instructions
// might flush) gets the norm +inf: its logits are all recomputed exactly.
#include "common.h"
#include "kernels.h"

namespace moe {

struct DenseParams {
  const uint16_t* x;
  int64_t T;
  int64_t t_base;  // first token of this launch
  int32_t K;
  int32_t nseg;
  DenseSeg seg[2];
  LoraSeg lora;  // of the last segment
  Clear clear;
};

// The token rows are staged once per block in LDS (their loads issued first, then the
// weight row's, so the wait for them leaves the weight loads in flight): the registers
// then hold only the weight row, and more waves fit a SIMD, so the router + latent-down
// grid (4480 rows at one token) and the latent-up grid (7168 rows) run in one round.
//
// LORA: the last segment's rows also take their adapters' term, sum_r B[a_t][row][r] u[t][r].
// Lane l holds ranks l and l + 64 of each token; the products (exact in fp64) join the lane's
// fp64 sum before the wave reduction, so the term costs two loads a lane and token, issued
// behind the weight row's (they wait for the adapter's id and rank), and no rounding of its own.
template <int NCH, int G, bool LORA>
__global__ void __launch_bounds__(256) dense_gemv_kernel(DenseParams p) {
  constexpr int XN = G * NCH * 64;            // 16-byte pieces of the block's token rows
  constexpr int XPT = (XN + 255) / 256;       // per thread
  __shared__ uint4 xs[XN];
  const int lane = lane_id();
  const int wave = threadIdx.x / WAVE;
  int64_t row = (int64_t)blockIdx.x * 4 + wave;
  // the segment is chosen with scalar selects so every field stays in kernel-argument
  // registers (an indexed p.seg[si] would be read from memory after the loads)
  const bool second = row >= p.seg[0].rows;
  if (second) row -= p.seg[0].rows;
  const DenseSeg s = second ? p.seg[1] : p.seg[0];
  // a wave past the last row works on the segment's last row and writes nothing (no
  // wave leaves before the block's barrier)
  const bool valid = !second || (p.nseg >= 2 && row < p.seg[1].rows);
  if (!valid) row = s.rows - 1;
  const int32_t K = p.K;
  const int64_t t0 = p.t_base + (int64_t)blockIdx.y * G;
  // asked of the kernel's arguments first: the grid's size comes from memory, 0.12 us for every launch
  if (p.clear.nzero > 0 && blockIdx.y == 0) {
    for (int i = blockIdx.x * 256 + threadIdx.x; i < p.clear.nzero; i += gridDim.x * 256) p.clear.zero[32 * i] = 0;
    for (int i = blockIdx.x * 256 + threadIdx.x; i < p.clear.nones; i += gridDim.x * 256)
      p.clear.ones[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
  }

  uint4 xv[XPT];
#pragma unroll
  for (int u = 0; u < XPT; ++u) {
    const int i = threadIdx.x + 256 * u < XN ? threadIdx.x + 256 * u : XN - 1;
    const int g = i / (NCH * 64), rem = i - g * (NCH * 64);
    const int col = 8 * rem;  // piece rem = 64 c + lane of token g
    const int64_t t = t0 + g < p.T ? t0 + g : p.T - 1;
    xv[u] = *reinterpret_cast<const uint4*>(p.x + t * K + (col < K ? col : 0));
    if (col >= K || t0 + g >= p.T) xv[u] = make_uint4(0, 0, 0, 0);
  }
  uint4 wr[NCH];
  const uint16_t* wrow = s.W + row * K;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int col = 8 * (64 * c + lane);
    wr[c] = load_nt16(wrow + (col < K ? col : 0));
    if (col >= K) wr[c] = make_uint4(0, 0, 0, 0);
  }
  uint16_t lb[LORA ? G : 1][2];
  float lu[LORA ? G : 1][2];
  if constexpr (LORA) {
    const bool mine = second || p.nseg < 2;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int64_t t = t0 + g < p.T ? t0 + g : p.T - 1;
      const int a = p.lora.adapter[t];
      const bool on = mine && (uint32_t)a < (uint32_t)p.lora.N;
      const int rk = !on ? 0 : !p.lora.rank ? p.lora.R : min(p.lora.rank[a], p.lora.R);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = lane + WAVE * h;
        lb[g][h] = 0;
        lu[g][h] = 0.f;
        if (r < rk) {
          lb[g][h] = p.lora.B[((int64_t)a * s.rows + row) * p.lora.R + r];
          lu[g][h] = p.lora.u[t * p.lora.R + r];
        }
      }
    }
  }
#pragma unroll
  for (int u = 0; u < XPT; ++u)
    if (threadIdx.x + 256 * u < XN) xs[threadIdx.x + 256 * u] = xv[u];
  lds_barrier();  // the weight loads stay in flight
  auto xr = [&](int g, int c) -> uint4 { return xs[g * (NCH * 64) + 64 * c + lane]; };

  if (!s.router) {
    // latent projections: fp32 chunk partials folded into fp64, rounded once to bf16
    double acc[G];
#pragma unroll
    for (int g = 0; g < G; ++g) acc[g] = 0.0;
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const uint4 xc = xr(g, c);
        float pc = dot2(xc.x, wr[c].x, 0.f);
        pc = dot2(xc.y, wr[c].y, pc);
        pc = dot2(xc.z, wr[c].z, pc);
        pc = dot2(xc.w, wr[c].w, pc);
        acc[g] += (double)pc;
      }
    if constexpr (LORA) {
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int h = 0; h < 2; ++h) acc[g] += (double)lu[g][h] * (double)bf16f(lb[g][h]);
    }
    uint16_t* out = reinterpret_cast<uint16_t*>(s.out);
    double v = wave_sums<G>(acc);  // lane g: token g
    if (valid && lane < G && t0 + lane < p.T) {
      for (int a = 0; a < s.add_rows; ++a) v += (double)s.add[((t0 + lane) * s.add_rows + a) * s.rows + row];
      out[(t0 + lane) * s.rows + row] = f64_to_bf16(v);
    }
    return;
  }

  // router row: fp32 chunk partials folded into fp64
  double acc[G];
  float wn = 0.f;
  uint32_t wsub = 0;
#pragma unroll
  for (int g = 0; g < G; ++g) acc[g] = 0.0;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    wn = dot2(wr[c].x, wr[c].x, wn);
    wn = dot2(wr[c].y, wr[c].y, wn);
    wn = dot2(wr[c].z, wr[c].z, wn);
    wn = dot2(wr[c].w, wr[c].w, wn);
    wsub |= bf16x2_subnormal(wr[c].x) | bf16x2_subnormal(wr[c].y) | bf16x2_subnormal(wr[c].z) |
            bf16x2_subnormal(wr[c].w);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint4 xc = xr(g, c);
      float pc = dot2(xc.x, wr[c].x, 0.f);
      pc = dot2(xc.y, wr[c].y, pc);
      pc = dot2(xc.z, wr[c].z, pc);
      pc = dot2(xc.w, wr[c].w, pc);
      acc[g] += (double)pc;
    }
  }
  float* out = reinterpret_cast<float*>(s.out);
  const double logit = wave_sums<G>(acc);  // lane g: token g
  if (valid && lane < G && t0 + lane < p.T) out[(t0 + lane) * s.rows + row] = (float)logit;
  wn = wave_sum_dpp(wn);
  const bool wany = __any(wsub != 0u);
  if (valid && lane == 0 && blockIdx.y == 0) s.wnorm[row] = wany ? __builtin_inff() : sqrtf(wn);
  if (valid && row == 0) {  // one wave per token group writes the token norms
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float xn = 0.f;
      uint32_t xsub = 0;
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const uint4 xc = xr(g, c);
        xn = dot2(xc.x, xc.x, xn);
        xn = dot2(xc.y, xc.y, xn);
        xn = dot2(xc.z, xc.z, xn);
        xn = dot2(xc.w, xc.w, xn);
        xsub |= bf16x2_subnormal(xc.x) | bf16x2_subnormal(xc.y) | bf16x2_subnormal(xc.z) |
                bf16x2_subnormal(xc.w);
      }
      xn = wave_sum_dpp(xn);
      const bool xany = __any(xsub != 0u);
      if (lane == 0 && t0 + g < p.T) s.xnorm[t0 + g] = xany ? __builtin_inff() : sqrtf(xn);
    }
  }
}

template <int NCH, int G>
static hipError_t launch_nch_g(DenseParams p, hipStream_t st) {
  int64_t rows = p.seg[0].rows + (p.nseg > 1 ? p.seg[1].rows : 0);
  if (ceil_div(rows, 4) > 0x7FFFFFFF) return hipErrorInvalidValue;
  constexpr int64_t MAX_Y = 65535;  // the grid's second dimension; more tokens take more launches
  const int64_t groups = ceil_div(p.T, G);
  for (int64_t g0 = 0; g0 < groups; g0 += MAX_Y) {
    p.t_base = g0 * G;
    const dim3 grid((unsigned)ceil_div(rows, 4), (unsigned)(groups - g0 < MAX_Y ? groups - g0 : MAX_Y));
    if (p.lora.B)
      hipLaunchKernelGGL((dense_gemv_kernel<NCH, G, true>), grid, dim3(256), 0, st, p);
    else
      hipLaunchKernelGGL((dense_gemv_kernel<NCH, G, false>), grid, dim3(256), 0, st, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int NCH>
static hipError_t launch_nch(const DenseParams& p, hipStream_t st) {
  // Tokens per block: a weight row is read once for G of them (results do not depend on it).  As
  // many as leave a wave for each of the card's 1024 SIMDs, or two where a wave has four tokens:
  // fewer waves than that take longer, each, than they save in reads.  One, two and four a block,
  // us: 7168 wide, 3584 rows 2 tokens 15.1, 10.2, 16.4, 3 tokens 21.0, 17.2, 15.9, 8 tokens 49.6,
  // 29.1, 24.9; 896 rows 3 tokens 6.0, 6.3, 6.8, 4 tokens 7.2, 5.8, 6.8, 8 tokens 10.8, 8.4, 8.0; 4096
  // wide, 512 rows 4 tokens 3.4, 3.7, 5.0, 8 tokens 4.5, 4.0, 5.0, 16 tokens 6.2, 5.3, 5.5; 2048 wide, 2048
  // rows 4 tokens 5.6, 4.5, 4.0.
  const int64_t rows = p.seg[0].rows + (p.nseg > 1 ? p.seg[1].rows : 0);
  if (p.T >= 3 && rows * ceil_div(p.T, 4) >= 2048) return launch_nch_g<NCH, 4>(p, st);
  if (p.T >= 2 && rows * ceil_div(p.T, 2) >= 1024) return launch_nch_g<NCH, 2>(p, st);
  return launch_nch_g<NCH, 1>(p, st);
}

hipError_t launch_dense_gemv(const uint16_t* x, int64_t T, int32_t K, const DenseSeg* segs, int nseg,
                             hipStream_t st, const LoraSeg* lora, const Clear* clear) {
  DenseParams p;
  if (lora) p.lora = *lora;
  if (clear) p.clear = *clear;
  p.x = x;
  p.T = T;
  p.K = K;
  p.nseg = nseg;
  p.seg[0] = segs[0];
  p.seg[1] = nseg > 1 ? segs[1] : segs[0];
  if (T == 0) return hipSuccess;
  int nch = (int)ceil_div(K, 512);
  switch (nch) {
    case 1: return launch_nch<1>(p, st);
    case 2: return launch_nch<2>(p, st);
    case 3: case 4: return launch_nch<4>(p, st);
    case 5: case 6: case 7: return launch_nch<7>(p, st);
    case 8: return launch_nch<8>(p, st);
    case 9: case 10: case 11: case 12: case 13: case 14: return launch_nch<14>(p, st);
    case 15: case 16: return launch_nch<16>(p, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace moe
