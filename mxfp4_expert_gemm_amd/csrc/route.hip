// Routing kernels: batches (one wavefront per token), and the small batches whose routing,
// quantisation of the latent rows and grouping by expert share one block.  The selection
// itself, its certification and the exact recompute are in route_token.h.
#include "route_token.h"

namespace moe {

// the 8 values of group j of a latent row, quantised (the quad of lanes holding the four
// groups of a scale block is active together)
__device__ __forceinline__ void quantize_group8(const uint4 raw, const QRows& q, int64_t j, bool mxfp8) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16lo(w[i]);
    v[2 * i + 1] = bf16hi(w[i]);
  }
  uint32_t hi[2], lo[2], shi, slo;
  quantize_quad8_fmt(v, hi, lo, shi, slo, mxfp8);
  *reinterpret_cast<uint2*>(q.hi + 8 * j) = make_uint2(hi[0], hi[1]);
  *reinterpret_cast<uint2*>(q.lo + 8 * j) = make_uint2(lo[0], lo[1]);
  if ((j & 3) == 0) {
    q.shi[j >> 2] = (uint8_t)shi;
    q.slo[j >> 2] = (uint8_t)slo;
  }
}

// the token's latent row h as two e4m3 terms for the expert kernels, eight values per
// lane and group: for L <= 8 * 64 * QH_GROUPS every group's load is issued before the
// first is used (one memory round trip per row instead of one per two groups)
constexpr int QH_GROUPS = 8;
__device__ __forceinline__ void quantize_token_h(const RouteArgs& a, int64_t t) {
  if (!a.h) return;
  const QRows q{a.hq.hi + t * a.L, a.hq.lo + t * a.L, a.hq.shi + t * (a.L / 32), a.hq.slo + t * (a.L / 32)};
  const uint16_t* h = a.h + t * a.L;
  const int ng = a.L / 8, lane = lane_id();
  if (ng > QH_GROUPS * WAVE) {
    quantize_quads(h, q, a.L, lane, WAVE, a.mxfp8 != 0);
    return;
  }
  uint4 raw[QH_GROUPS];
#pragma unroll
  for (int u = 0; u < QH_GROUPS; ++u) {
    const int j = lane + WAVE * u;
    raw[u] = j < ng ? *reinterpret_cast<const uint4*>(h + 8 * j) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int u = 0; u < QH_GROUPS; ++u)
    if (lane + WAVE * u < ng) quantize_group8(raw[u], q, lane + WAVE * u, a.mxfp8 != 0);
}

// MINB blocks per CU: 4 caps the kernel at 128 registers a lane, spilling in the general
// path; for large batches the doubled occupancy over the 2 blocks of the uncapped build
// (172 registers) pays (prefill32k: 0.49 -> 0.33 ms), while a few dozen tokens, whose
// slowest token sets the kernel's length, run faster uncapped (decode64: 63 us against 71).
constexpr int64_t ROUTE_WIDE_TOKENS = 2048;  // 512 blocks: two per CU at the uncapped occupancy

template <int MINB>
__global__ void __launch_bounds__(256, MINB) route_kernel(RouteArgs a) {
  __shared__ RouteLds scratch[4];
  const int wave = threadIdx.x / WAVE;
  const int64_t t = (int64_t)blockIdx.x * 4 + wave;
  if (t >= a.T) return;
  route_token(a, t, &scratch[wave]);
  quantize_token_h(a, t);
}

hipError_t launch_route(const RouteArgs& a, hipStream_t st) {
  if (a.T == 0) return hipSuccess;
  if (a.E > ROUTE_MAXI * WAVE) return hipErrorInvalidValue;
  const dim3 grid((unsigned)ceil_div(a.T, 4));
  if (a.T >= ROUTE_WIDE_TOKENS)
    hipLaunchKernelGGL(route_kernel<4>, grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL(route_kernel<1>, grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

// ---- small batches: the grouping of routed rows by expert

// Block-wide grouping of the T*k routed rows r = t*k + j (expert sidx[r]; the k experts
// of a token are distinct and valid; T <= 64) by expert: counts, offsets, perm with
// tokens ascending inside each group, and the tile list.  Per expert, LDS holds the row
// count, the 64-bit mask of its tokens and its first row, all built with integer
// atomics (order-free); a row's place inside its group is the number of lower tokens in
// the mask.  One packed prefix sum over the experts gives offsets (low 16 bits) and tile
// slots (high 16 bits) together.
constexpr int PLACE_MAX_TOKENS = ROUTE_PLACE_TOKENS;
struct PlaceLds {
  int cnt[ROUTE_MAXI * WAVE];
  unsigned long long tmask[ROUTE_MAXI * WAVE];
  int first[ROUTE_MAXI * WAVE];
  int wsum[16];
};

__device__ void place_rows_block(const int* sidx, int T, int k, int E, PlaceLds* S, const PermOut& p) {
  const int tid = threadIdx.x, nt = blockDim.x, nw = nt / WAVE, wave = tid / WAVE, lane = lane_id();
  for (int e = tid; e < E; e += nt) {
    S->cnt[e] = 0;
    S->tmask[e] = 0ull;
    S->first[e] = 0x7FFFFFFF;
  }
  __syncthreads();
  const int rows = T * k;
  for (int r = tid; r < rows; r += nt) {
    const int e = sidx[r];
    atomicAdd(&S->cnt[e], 1);
    atomicOr(&S->tmask[e], 1ull << (r / k));
    atomicMin(&S->first[e], r);
  }
  __syncthreads();
  const int per = (E + nt - 1) / nt;  // consecutive experts per thread
  int loc = 0;
  for (int q = 0; q < per; ++q) {
    const int e = tid * per + q;
    if (e < E) loc += S->cnt[e] | ((S->cnt[e] > 0) << 16);
  }
  int wtot = 0;
  const int wex = wave_excl_scan(loc, wtot);
  if (lane == 0) S->wsum[wave] = wtot;
  __syncthreads();
  int run = wex, totals = 0;
  for (int w = 0; w < nw; ++w) {
    run += w < wave ? S->wsum[w] : 0;
    totals += S->wsum[w];
  }
  for (int q = 0; q < per; ++q) {
    const int e = tid * per + q;
    if (e < E) {
      const int c = S->cnt[e], off = run & 0xFFFF;
      p.counts[e] = c;
      p.offsets[e] = off;
      if (c > 0) p.tiles[run >> 16] = make_int4(e, off, c, S->first[e]);
      run += c | ((c > 0) << 16);
      S->cnt[e] = off;  // from here on: the group's first position
    }
  }
  const int nact = totals >> 16;
  if (tid == 0) {
    p.offsets[E] = totals & 0xFFFF;
    *p.n_active = nact;
  }
  for (int sl = nact + tid; sl < p.max_tiles; sl += nt) p.tiles[sl] = make_int4(-1, 0, 0, -1);
  __syncthreads();
  for (int r = tid; r < rows; r += nt) {
    const int e = sidx[r], t = r / k;
    p.perm[S->cnt[e] + __popcll(S->tmask[e] & ((1ull << t) - 1ull))] = r;
  }
}

// Routing of T <= ROUTE_FUSED_TOKENS tokens, the quantisation of their latent rows and
// the grouping by expert in one block.
__global__ void __launch_bounds__(512) route_permute_small_kernel(RouteArgs a, PermOut p) {
  __shared__ RouteLds scratch[8];
  __shared__ int sidx[ROUTE_FUSED_TOKENS * WAVE];
  __shared__ PlaceLds pl;
  const int wave = threadIdx.x / WAVE, nw = blockDim.x / WAVE;
  const int k = a.k, T = (int)a.T;
  for (int t = wave; t < T; t += nw) route_token(a, t, &scratch[wave]);
  // eight latent values per thread: by the waves that route no token when there are
  // some (they start at once), else by every thread, counted from the last one down so
  // that the waves with fewer tokens to route take the first ones
  if (a.h) {
    if (T < nw) {
      if (wave >= T)
        quantize_quads(a.h, a.hq, (int64_t)T * a.L, threadIdx.x - T * WAVE, blockDim.x - T * WAVE, a.mxfp8 != 0);
    } else {
      quantize_quads(a.h, a.hq, (int64_t)T * a.L, blockDim.x - 1 - threadIdx.x, blockDim.x, a.mxfp8 != 0);
    }
  }
  __syncthreads();  // token t's selection, ascending, is in scratch[t].oidx (one wave per token)
  if (T == 1) {
    // one token: its k distinct experts in ascending order are the k groups, one row
    // each.  Thread experts e = tid + i nt (i < NE, NE nt > E): offsets[e] = selections
    // below e, counts[e] = 1 if e is selected; each selection is read once.
    constexpr int NE = (ROUTE_MAXI * WAVE + 1 + 4 * WAVE - 1) / (4 * WAVE);
    const int* sel = scratch[0].oidx;
    const int nt = blockDim.x;
    int below[NE], upto[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) below[i] = upto[i] = 0;
    for (int j = 0; j < k; ++j) {
      const int sj = sel[j];
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const int e = threadIdx.x + i * nt;
        below[i] += sj < e;
        upto[i] += sj <= e;
      }
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = threadIdx.x + i * nt;
      if (e <= a.E) p.offsets[e] = below[i];
      if (e < a.E) p.counts[e] = upto[i] - below[i];
    }
    for (int j = threadIdx.x; j < k; j += blockDim.x) {
      p.perm[j] = j;
      p.tiles[j] = make_int4(sel[j], j, 1, j);
    }
    for (int sl = k + threadIdx.x; sl < p.max_tiles; sl += blockDim.x) p.tiles[sl] = make_int4(-1, 0, 0, -1);
    if (threadIdx.x == 0) *p.n_active = k;
    return;
  }
  for (int r = threadIdx.x; r < T * k; r += blockDim.x) sidx[r] = scratch[r / k].oidx[r % k];
  __syncthreads();
  place_rows_block(sidx, T, k, a.E, &pl, p);
}

// One token (decode) routed by a whole block, one expert per thread.  A single wave
// holding 14 experts per lane spends most of its time in dependent instruction chains;
// here the fast logits, radii and keys of route_token are computed once per thread
// (the same fp32 values), the cut tau is the k-th largest of the maxima of 64 groups of
// consecutive experts (at least k keys reach it, so the k best are candidates), and the
// candidates are compacted in expert order and ranked by all waves (four each).  Wave 0
// certifies the boundary against every other expert's upper end and writes the
// selection, the same values route_token writes when its fast path decides; when this
// one cannot decide (more than ROUTE_CAND candidates, an uncertain boundary, weights
// over all experts) wave 0 runs route_token instead.  The other waves quantise the
// latent row meanwhile (its loads are issued with the logits'); then every thread
// writes the grouping entries of its expert.
constexpr int RB_THREADS = 1024;
constexpr int RB_WAVES = RB_THREADS / WAVE;
constexpr int RB_GROUP = RB_THREADS / WAVE;  // experts per group: one group maximum per lane
constexpr int RB_QT = RB_THREADS - WAVE;     // threads of the latent row's quantisation
static_assert(ROUTE_CAND == WAVE && ROUTE_CAND <= 4 * RB_WAVES, "four candidates ranked per wave");

struct RouteBlockLds {
  RouteLds rl;  // wave 0's candidates, output pairs and fallback scratch
  unsigned long long cpk[ROUTE_CAND];  // candidate (key, ~expert): larger ranks first
  int crank[ROUTE_CAND];
  int selpre[ROUTE_CAND + 1];  // selected candidates before candidate i
  uint32_t gmax[WAVE];
  int wcnt[RB_WAVES];
  float wup[RB_WAVES];
  uint32_t tau;
  int decided;
};

// route_token as a call: its registers are not reserved in the block kernel, where it
// runs only when the block's selection cannot decide
__attribute__((noinline)) __device__ void route_token_call(RouteArgs a, RouteLds* L) { route_token(a, 0, L); }

__global__ void __launch_bounds__(RB_THREADS) route_permute_one_kernel(RouteArgs a, PermOut p) {
  __shared__ RouteBlockLds S;
  const int tid = threadIdx.x, lane = lane_id(), wave = tid / WAVE;
  const int E = a.E, k = a.k;
  const int e = tid;
  const bool have = e < E;
  const int ec = have ? e : E - 1;
  const float lf = a.logits_fast[ec];
  const float bv = a.bias ? a.bias[ec] : 0.f;
  const float wn = a.wnorm[ec];
  const float xn = a.xnorm[0];
  // the first group of the latent row this thread quantises
  const int64_t ng = a.h ? a.L / 8 : 0;
  const int64_t jq = tid - WAVE;
  const bool qg = wave > 0 && jq < ng;
  const uint4 hraw = qg ? *reinterpret_cast<const uint4*>(a.h + 8 * jq) : make_uint4(0u, 0u, 0u, 0u);

  const float gam = (float)a.gamma * (1.f + 0x1p-18f) * xn;
  const float pad = (float)a.d * 0x1p-124f;
  float c = -__builtin_inff(), R = 0.f;
  uint32_t key = 0u;
  if (have) {
    c = lf + bv;
    R = gam * wn + pad + 0x1p-20f * (fabsf(lf) + fabsf(bv));
    if (bv == -__builtin_inff()) {
      const float rr = gam * wn + pad + 0x1p-20f * fabsf(lf);
      const bool known = __builtin_isfinite(lf) && __builtin_isfinite(rr) && fabsf(lf) + rr < 0x1p127f;
      c = -__builtin_inff();
      R = known ? 0.f : __builtin_inff();
    } else if (!(__builtin_isfinite(c) && __builtin_isfinite(R))) {
      c = -__builtin_inff();
      R = __builtin_inff();
    }
    key = order_key(c);
  }
  // the maximum of each 16-lane row (a group), by DPP within the row
  static_assert(RB_GROUP == 16, "a group is one DPP row");
  uint32_t gm = key;
  gm = max(gm, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)gm, DPP_QUAD_1032, 0xF, 0xF, false));
  gm = max(gm, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)gm, DPP_QUAD_2301, 0xF, 0xF, false));
  gm = max(gm, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)gm, DPP_ROW_ROR4, 0xF, 0xF, false));
  gm = max(gm, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)gm, DPP_ROW_ROR8, 0xF, 0xF, false));
  if ((lane & (RB_GROUP - 1)) == 0) S.gmax[tid / RB_GROUP] = gm;
  lds_barrier();
  if (wave == 0) {
    const uint32_t t0 = kth_of_lanes(S.gmax[lane], k);
    if (lane == 0) S.tau = t0;
  }
  lds_barrier();
  const uint32_t tau = S.tau;
  const bool cand = key != 0u && key >= tau;
  const unsigned long long cb = __ballot(cand);
  float up = -__builtin_inff();
  if (have && !cand) up = R == __builtin_inff() ? __builtin_inff() : next_up(c + R);
  up = wave_max_dpp(up);
  if (lane == 0) {
    S.wcnt[wave] = __popcll(cb);
    S.wup[wave] = up;
  }
  lds_barrier();
  int base = 0, n_c = 0;
#pragma unroll
  for (int w = 0; w < RB_WAVES; ++w) {
    const int cw = S.wcnt[w];
    base += w < wave ? cw : 0;
    n_c += cw;
  }
  // this expert's place in the candidate list (for a non-candidate: the candidates below it)
  const int pos = base + __popcll(cb & ((1ull << lane) - 1ull));
  const bool fits = n_c <= ROUTE_CAND;
  if (fits && cand) {
    S.cpk[pos] = ((unsigned long long)key << 32) | (uint32_t)~(uint32_t)e;
    S.rl.cidx[pos] = e;
    S.rl.cval[pos] = c;
    S.rl.crad[pos] = R;
  }
  lds_barrier();
  if (fits) {
    // wave w ranks candidates 4w..4w+3 against all: rank = candidates ahead of it
    const unsigned long long pj = lane < n_c ? S.cpk[lane] : 0ull;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = 4 * wave + u;
      const unsigned long long pi = __shfl(pj, i);
      const int r = __popcll(__ballot(lane < n_c && pj > pi));
      if (lane == 0 && i < n_c) S.crank[i] = r;
    }
  }
  lds_barrier();
  if (wave == 0) {
    bool fast = fits && a.renormalize && !(a.flags & MOE_ROUTE_EXACT_ALL);
    if (fast) {
      const bool live = lane < n_c;
      const bool sel = live && S.crank[lane] < k;
      const float mc = live ? S.rl.cval[lane] : 0.f, mr = live ? S.rl.crad[lane] : 0.f;
      if (k < E) {
        float Mloc = __builtin_inff(), mloc = -__builtin_inff();
        if (sel) Mloc = mr == __builtin_inff() ? -__builtin_inff() : next_down(mc - mr);
        if (live && !sel) mloc = mr == __builtin_inff() ? __builtin_inff() : next_up(mc + mr);
        if (lane < RB_WAVES) mloc = fmaxf(mloc, S.wup[lane]);
        fast = wave_min_dpp(Mloc) > wave_max_dpp(mloc);
      }
      if (fast) {
        // candidates are in expert order, so the output place is the count of selected below
        const unsigned long long sb = __ballot(sel);
        const int op = __popcll(sb & ((1ull << lane) - 1ull));
        S.selpre[lane] = op;
        if (lane == 0) S.selpre[ROUTE_CAND] = __popcll(sb);
        if (sel) {
          S.rl.oidx[op] = S.rl.cidx[lane];
          S.rl.oval[op] = mc;
        }
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
        __builtin_amdgcn_wave_barrier();
        emit_topk(a, 0, &S.rl, 0.f, 1.f);
      }
    }
    if (!fast) route_token_call(a, &S.rl);
    if (lane == 0) S.decided = fast;
  } else {
    if (qg) quantize_group8(hraw, a.hq, jq, a.mxfp8 != 0);
    if (ng > RB_QT) quantize_quads(a.h, a.hq, a.L, jq + RB_QT, RB_QT, a.mxfp8 != 0);
  }
  lds_barrier();  // the k selected experts, ascending, are in S.rl.oidx
  const bool decided = S.decided;
  if (decided && a.logits_out && have) a.logits_out[e] = c;
  // one row per selected expert: offsets[e] = selected experts below e
  int below = 0, upto = 0;
  if (decided) {
    below = S.selpre[pos < n_c ? pos : ROUTE_CAND];
    upto = below + (cand && S.crank[pos] < k);
  } else {
    for (int j = 0; j < k; ++j) {
      const int sj = S.rl.oidx[j];
      below += sj < e;
      upto += sj <= e;
    }
  }
  if (e <= E) p.offsets[e] = below;
  if (tid == 0 && E == RB_THREADS) p.offsets[E] = k;
  if (have) p.counts[e] = upto - below;
  if (tid < k) {
    p.perm[tid] = tid;
    p.tiles[tid] = make_int4(S.rl.oidx[tid], tid, 1, tid);
  }
  for (int sl = k + tid; sl < p.max_tiles; sl += RB_THREADS) p.tiles[sl] = make_int4(-1, 0, 0, -1);
  if (tid == 0) *p.n_active = k;
}

// Grouping of the rows of routed tokens (distinct, valid experts per token) for
// T <= PLACE_MAX_TOKENS and T*k <= ROUTE_SMALL_ROWS, after route_kernel.
__global__ void __launch_bounds__(1024) place_rows_kernel(const int32_t* __restrict__ idx, int T, int k, int E,
                                                          PermOut p) {
  __shared__ int sidx[ROUTE_SMALL_ROWS];
  __shared__ PlaceLds pl;
  for (int r = threadIdx.x; r < T * k; r += blockDim.x) sidx[r] = idx[r];
  __syncthreads();
  place_rows_block(sidx, T, k, E, &pl, p);
}

hipError_t launch_place_rows(const int32_t* idx, int64_t T, int32_t k, int32_t E, const PermOut& p,
                             hipStream_t st) {
  if (T == 0) return hipSuccess;
  if (E > ROUTE_MAXI * WAVE || T > PLACE_MAX_TOKENS || T * k > ROUTE_SMALL_ROWS || k > WAVE)
    return hipErrorInvalidValue;
  hipLaunchKernelGGL(place_rows_kernel, dim3(1), dim3(1024), 0, st, idx, (int)T, k, E, p);
  return hipGetLastError();
}

hipError_t launch_route_permute_small(const RouteArgs& a, const PermOut& p, hipStream_t st) {
  if (a.T == 0) return hipSuccess;
  if (a.E > ROUTE_MAXI * WAVE || a.T > ROUTE_FUSED_TOKENS || a.k > WAVE) return hipErrorInvalidValue;
  if (a.T == 1 && a.E <= RB_THREADS && a.exact_logits == nullptr) {
    hipLaunchKernelGGL(route_permute_one_kernel, dim3(1), dim3(RB_THREADS), 0, st, a, p);
    return hipGetLastError();
  }
  // a wave per token, and at least one wave more that quantises the latent rows meanwhile
  // for T < 8
  const int nw = a.T < 4 ? 4 : 8;
  hipLaunchKernelGGL(route_permute_small_kernel, dim3(1), dim3(nw * WAVE), 0, st, a, p);
  return hipGetLastError();
}

}  // namespace moe
