// The layer for the few tokens of a decode step, in two launches: the router logits and the
// latent rows h (dense_gemv_kernel), then everything behind them in one grid.
//
// A decode step of a few tokens reads a few hundred MB once, so its time is the HBM's plus
// what each launch costs on the way: its first loads' latency, its last blocks' drain, and
// the routing, during which nothing streams.  Here one block per CU goes through the phases
//   route      every block routes all tokens for itself (a wave per token) and quantises h
//              into its LDS: no block waits for another's selection;
//   gate / up  work items of 32 FFN rows of one routed expert, a wave each;
//   down       work items of 16 latent rows of all routed experts, with the combine;
//   up         work items of a few output rows a wave;
// and phases hand over through counters in the workspace, not through launches.
//
// Progress.  A block claims an item from the phase's counter when it is about to work on it,
// moves on when none is left, and waits only for items that were claimed before, each by a
// block that runs and waits for earlier phases at most.  So the grid drains however many of
// its blocks are resident at a time, beside whatever else the GPU runs.  The counters are
// cleared by the launch before.
//
// The arithmetic of every value is that of the kernels moe_layer_forward runs on a batch of
// this size (dense_gemv_kernel, route_token, stream_group, the down kernel's fp64 combine),
// in the same order: the outputs are bit-identical.
#include "mfma_stream.h"
#include "route_token.h"

namespace moe {

constexpr int DEC_THREADS = 512;
constexpr int DEC_WAVES = DEC_THREADS / WAVE;
constexpr int DEC_ROWS = 32;   // FFN rows of a gate / up item: one scale block of the down operand
constexpr int DEC_GU_PF = 4;   // K steps in flight, of four weight streams a wave
constexpr int DEC_DN_PF = 8;   // of one or two
constexpr int DEC_LDS_STATIC = 24 * 1024;  // room for the statically allocated LDS
static_assert(DECODE_MAX_TOKENS <= DEC_WAVES && DECODE_MAX_ROWS <= WAVE, "a wave per token, a lane per routed row");

// a staged activation row: hi codes, lo codes, hi scales, lo scales
__host__ __device__ constexpr int dec_row_bytes(int K) { return (2 * K + K / 16 + 15) / 16 * 16; }
__device__ __forceinline__ ALds dec_row(uint8_t* row, int K) { return {row, row + K, row + 2 * K, row + 2 * K + K / 32}; }

// ---- phase counters, a 128-byte line each
enum { C_GATEUP, C_GATEUP_DONE, C_DOWN, C_DOWN_DONE, C_U, C_U_DONE, C_UP, C_COUNT };
static_assert(C_COUNT * 32 == DECODE_COUNTERS, "the first launch clears the counters");

__device__ __forceinline__ int claim(int32_t* ctr, int n, int* shared) {
  __syncthreads();  // the last claim has been read
  if (threadIdx.x == 0) *shared = __hip_atomic_fetch_add(ctr, n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  return *shared;
}
// the block's stores of n items are in memory before the count says so
__device__ __forceinline__ void publish(int32_t* ctr, int n) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // each wave's own stores have left
  __syncthreads();
  if (threadIdx.x == 0 && n > 0) {
    __threadfence();
    __hip_atomic_fetch_add(ctr, n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
}
__device__ __forceinline__ void await(int32_t* ctr, int n) {
  if (threadIdx.x == 0)
    while (__hip_atomic_load(ctr, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) < n) __builtin_amdgcn_s_sleep(1);
  __syncthreads();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
}
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// stream_group with NS weight streams that share one activation row group (ONE_A) or have one
// each: acc[q] += A_q W_q^T over all K steps, sb and ring filled by prime_stream
template <class W, int NS, int PF, bool ONE_A>
__device__ __forceinline__ void dec_stream(const W (&w)[NS], SBlock (&sb)[NS], uint4 (&ring)[NS][PF],
                                           const ALds (&ad)[ONE_A ? 1 : NS], bool on, int K, int g, f32x4 (&acc)[NS]) {
  const int nks = K / 128, nc = (nks + 15) / 16;
  SBlock sbn[NS];
  for (int c = 0; c < nc; ++c) {
#pragma unroll
    for (int q = 0; q < NS; ++q) w[q].sblock(sbn[q], c + 1 < nc ? c + 1 : c);
    unroll16([&](auto jc) {
      constexpr int J = decltype(jc)::value;
      const int ks = 16 * c + J;
      uint4 cw[NS];
#pragma unroll
      for (int q = 0; q < NS; ++q) {
        cw[q] = ring[q][J % PF];
        ring[q][J % PF] = w[q].load(ks + PF < nks ? ks + PF : nks - 1);
      }
      if (ks < nks) {
        AStep a;
#pragma unroll
        for (int q = 0; q < NS; ++q) {
          if (!ONE_A || q == 0) read_a(a, ad[ONE_A ? 0 : q], on ? 0 : 1, 1, K, ks, g);
          const uint32_t sw = w[q].template scale<J>(sb[q]);
          const i32x8 b = as_b(cw[q]);
          acc[q] = mx_mfma<W::opsel(J)>(a.hi, b, acc[q], a.shi, sw);
          acc[q] = mx_mfma<W::opsel(J)>(a.lo, b, acc[q], a.slo, sw);
        }
      }
    });
#pragma unroll
    for (int q = 0; q < NS; ++q) sb[q] = sbn[q];
  }
}

struct DecodeLds {
  union {
    RouteLds route[DEC_WAVES];
    float atile[DEC_WAVES][DECODE_MAX_TOKENS][DEC_ROWS + 1];  // an item's GLU outputs, a wave's own
    float ys[DECODE_MAX_ROWS][16];                            // an item's expert outputs by slot
  };
  int sel[DECODE_MAX_ROWS];    // expert of slot t k + j
  float w[DECODE_MAX_ROWS];    // its weight
  int gexp[DECODE_MAX_ROWS];   // distinct experts, and the slots of each
  int gn[DECODE_MAX_ROWS];
  int gslot[DECODE_MAX_ROWS][DECODE_MAX_TOKENS];
  int ng;
  int claimed;
};
static_assert(sizeof(DecodeLds) <= DEC_LDS_STATIC, "static LDS");

// Routing of all tokens into S, and h quantised into hq, by the whole block; the first block
// also writes what the caller asked for.
__device__ __forceinline__ void dec_route(const DecodeArgs& p, DecodeLds& S, uint8_t* hq) {
  const int tid = threadIdx.x, lane = lane_id(), wave = tid / WAVE;
  const int T = (int)p.r.T, k = p.r.k, E = p.r.E, L = p.r.L, n = T * k;
  const bool writer = blockIdx.x == 0;
  RouteArgs a = p.r;
  a.idx = S.sel;
  a.w = S.w;
  if (!writer) a.logits_out = nullptr;
  if (wave < T) route_token(a, wave, &S.route[wave]);
  // the waves that route nothing quantise meanwhile
  const int q0 = T < DEC_WAVES ? T : 0;
  if (wave >= q0)
    for (int t = 0; t < T; ++t) {
      const ALds r = dec_row(hq + t * dec_row_bytes(L), L);
      quantize_quads(a.h + (int64_t)t * L, QRows{r.hi, r.lo, r.shi, r.slo}, L, tid - q0 * WAVE,
                     DEC_THREADS - q0 * WAVE, a.mxfp8 != 0);
    }
  __syncthreads();
  if (wave == 0) {  // a lane per slot: the first slot of an expert leads its group
    const int e = lane < n ? S.sel[lane] : -1;
    unsigned long long mine = 0;
    for (int s = 0; s < n; ++s) {
      const unsigned long long m = __ballot(e == __builtin_amdgcn_readlane(e, s));
      if (e >= 0 && (m >> lane) & 1ull) mine = m;
    }
    const unsigned long long below = (1ull << lane) - 1ull;
    const bool lead = e >= 0 && (mine & below) == 0ull;
    const unsigned long long leads = __ballot(lead);
    if (e >= 0) {
      const int first = __ffsll((long long)mine) - 1;
      const int grp = __popcll(leads & ((1ull << first) - 1ull));
      S.gslot[grp][__popcll(mine & below)] = lane;
      if (lead) {
        S.gexp[grp] = e;
        S.gn[grp] = __popcll(mine);
      }
    }
    if (lane == 0) S.ng = __popcll(leads);
    if (writer && lane < n) {
      if (p.idx) p.idx[lane] = e;
      if (p.w) p.w[lane] = S.w[lane];
      if (p.perm) {
        int at = 0;
        for (int s = 0; s < n; ++s) at += S.sel[s] < e || (S.sel[s] == e && s < lane);
        p.perm[at] = lane;
      }
    }
  }
  if (writer && (p.counts || p.offsets))
    for (int e = tid; e <= E; e += DEC_THREADS) {
      int below = 0, same = 0;
      for (int s = 0; s < n; ++s) {
        below += S.sel[s] < e;
        same += S.sel[s] == e;
      }
      if (p.counts && e < E) p.counts[e] = same;
      if (p.offsets) p.offsets[e] = below;
    }
  __syncthreads();
}

// NS: routed rows a wave takes through the down matrices side by side.  UC chunks of 512
// latent columns of UR output rows are a wave's share of an up item.
template <class W, int NS, int UC, int UR>
__global__ void __launch_bounds__(DEC_THREADS) decode_kernel(DecodeArgs p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ DecodeLds S;
  const int tid = threadIdx.x, lane = lane_id(), wave = tid / WAVE;
  const int nl = lane & 15, g = lane >> 4;
  const int T = (int)p.r.T, k = p.r.k, L = p.r.L, F = p.F, d = p.r.d, n = T * k;
  const int arow = dec_row_bytes(F);

  dec_route(p, S, smem);
  const int ng = S.ng;

  // ---- gate / up
  const int nrb = F / DEC_ROWS, n1 = ng * nrb;
  {
    const int chunk = max(1, min(DEC_WAVES, (n1 + (int)gridDim.x - 1) / (int)gridDim.x));
    int mine = 0;
    for (;;) {
      const int c = claim(p.ctr + 32 * C_GATEUP, chunk, &S.claimed);
      if (c >= n1) break;
      mine += min(chunk, n1 - c);
      const int item = c + wave;
      if (wave < chunk && item < n1) {
        const int grp = item / nrb, rb = item - grp * nrb, e = S.gexp[grp], nt = S.gn[grp];
        const W w[4] = {W::make(p.blob, e, L, F, MAT_GATE, 2 * rb, lane), W::make(p.blob, e, L, F, MAT_GATE, 2 * rb + 1, lane),
                        W::make(p.blob, e, L, F, MAT_UP, 2 * rb, lane), W::make(p.blob, e, L, F, MAT_UP, 2 * rb + 1, lane)};
        SBlock sb[4];
        uint4 ring[4][DEC_GU_PF];
        prime_stream<W, 4, DEC_GU_PF>(w, sb, ring, L / 128);
        const bool on = nl < nt;
        const ALds ad[1] = {dec_row(smem + (on ? S.gslot[grp][nl] / k : 0) * dec_row_bytes(L), L)};
        f32x4 acc[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[q] = f32x4{0.f, 0.f, 0.f, 0.f};
        dec_stream<W, 4, DEC_GU_PF, true>(w, sb, ring, ad, on, L, g, acc);
        // lane: rows 16 h + nl of the item, tokens 4 g + j of the expert
        float(*at)[DEC_ROWS + 1] = S.atile[wave];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (4 * g + j < nt) at[4 * g + j][16 * h + nl] = bf16f(glu_bf16(acc[h][j], acc[2 + h][j]));
        wave_sync();
        // a quad of lanes per token, eight of the block's 32 values each
        const int m = lane >> 2, sub = lane & 3;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = m < nt ? at[m][8 * sub + i] : 0.f;
        uint32_t hi[2], lo[2], shi, slo;
        quantize_quad8_fmt(v, hi, lo, shi, slo, p.r.mxfp8 != 0);
        if (m < nt) {
          const ALds o = dec_row(p.aq + (int64_t)S.gslot[grp][m] * arow, F);
          *reinterpret_cast<uint2*>(o.hi + DEC_ROWS * rb + 8 * sub) = make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(o.lo + DEC_ROWS * rb + 8 * sub) = make_uint2(lo[0], lo[1]);
          if (sub == 0) {
            o.shi[rb] = (uint8_t)shi;
            o.slo[rb] = (uint8_t)slo;
          }
        }
      }
    }
    publish(p.ctr + 32 * C_GATEUP_DONE, mine);
  }

  // ---- down and combine: item = 16 latent rows of every routed row
  const int n2 = L / 16;
  {
    uint8_t* rows = smem + wave * NS * arow;
    bool ready = false;
    int mine = 0;
    for (;;) {
      const int c = claim(p.ctr + 32 * C_DOWN, 1, &S.claimed);
      if (c >= n2) break;
      ++mine;
      int s0 = wave * NS;
      W w[NS];
      SBlock sb[NS];
      uint4 ring[NS][DEC_DN_PF];
      auto prime = [&]() {
#pragma unroll
        for (int q = 0; q < NS; ++q)
          w[q] = W::make(p.blob, S.sel[min(s0 + q, n - 1)], L, F, MAT_DOWN, c, lane);
        prime_stream<W, NS, DEC_DN_PF>(w, sb, ring, F / 128);
      };
      if (s0 < n) prime();
      if (!ready) await(p.ctr + 32 * C_GATEUP_DONE, n1);
      ready = true;
      while (s0 < n) {
        ALds ad[NS];
#pragma unroll
        for (int q = 0; q < NS; ++q) {
          ad[q] = dec_row(rows + q * arow, F);
          const uint8_t* src = p.aq + (int64_t)min(s0 + q, n - 1) * arow;
          for (int i = 16 * lane; i < arow; i += 16 * WAVE)
            *reinterpret_cast<uint4*>(rows + q * arow + i) = *reinterpret_cast<const uint4*>(src + i);
        }
        wave_sync();
        f32x4 acc[NS];
#pragma unroll
        for (int q = 0; q < NS; ++q) acc[q] = f32x4{0.f, 0.f, 0.f, 0.f};
        dec_stream<W, NS, DEC_DN_PF, false>(w, sb, ring, ad, nl == 0, F, g, acc);
#pragma unroll
        for (int q = 0; q < NS; ++q)
          if (g == 0 && s0 + q < n) S.ys[s0 + q][nl] = acc[q][0];
        wave_sync();
        s0 += DEC_WAVES * NS;
        if (s0 < n) prime();
      }
      __syncthreads();
      for (int q = tid; q < T * 16; q += DEC_THREADS) {
        const int t = q >> 4, r = q & 15;
        double acc = 0.0;
        for (int j = 0; j < k; ++j) acc += (double)S.w[t * k + j] * (double)S.ys[t * k + j][r];
        p.z[(int64_t)t * L + c * 16 + r] = f64_to_bf16(acc);
      }
    }
    publish(p.ctr + 32 * C_DOWN_DONE, mine);
  }

  // ---- up (with the adapters' two products)
  uint16_t* zs = reinterpret_cast<uint16_t*>(smem);
  bool ready = false;
  auto stage_z = [&]() {  // every block that reads z holds all of it
    await(p.ctr + 32 * C_DOWN_DONE, n2);
    for (int i = tid; i < T * L / 8; i += DEC_THREADS)
      *reinterpret_cast<uint4*>(zs + 8 * i) = *reinterpret_cast<const uint4*>(p.z + 8 * i);
    __syncthreads();
    ready = true;
  };
  const bool lora = p.lora.B != nullptr;
  const int nu = T * p.lora.R;
  if (lora) {
    int mine = 0;
    for (;;) {  // item = a (token, rank) pair per wave
      const int c = claim(p.ctr + 32 * C_U, DEC_WAVES, &S.claimed);
      if (c >= nu) break;
      mine += min(DEC_WAVES, nu - c);
      if (!ready) stage_z();
      const int i = c + wave;
      if (i < nu) {
        const int t = i / p.lora.R, r = i - t * p.lora.R, a = p.lora.adapter[t];
        const bool have = (uint32_t)a < (uint32_t)p.lora.N;
        const int rk = !have ? 0 : p.lora.rank ? min(p.lora.rank[a], p.lora.R) : p.lora.R;
        float v = 0.f;
        if (r < rk) {
          const uint16_t* A = p.lora_a + ((int64_t)a * p.lora.R + r) * L;
          double acc = 0.0;
          for (int col = 8 * lane; col < L; col += 8 * WAVE) {
            const uint4 x = *reinterpret_cast<const uint4*>(zs + t * L + col);
            const uint4 av = *reinterpret_cast<const uint4*>(A + col);
            float q = dot2(x.x, av.x, 0.f);
            q = dot2(x.y, av.y, q);
            q = dot2(x.z, av.z, q);
            q = dot2(x.w, av.w, q);
            acc += (double)q;
          }
          v = (float)(wave_sum_dpp(acc) * (double)p.lora_scale[a]);
        }
        if (lane == 0) p.u[i] = v;
      }
    }
    publish(p.ctr + 32 * C_U_DONE, mine);
  }
  const int chunk = max(1, min(DEC_WAVES * UR, (d + (int)gridDim.x - 1) / (int)gridDim.x));
  bool uready = !lora;
  for (;;) {
    const int c = claim(p.ctr + 32 * C_UP, chunk, &S.claimed);
    if (c >= d) break;
    const int end = min(c + chunk, d);
    uint4 wr[UR][UC];
#pragma unroll
    for (int i = 0; i < UR; ++i) {
      const int row = min(c + wave + DEC_WAVES * i, d - 1);
#pragma unroll
      for (int q = 0; q < UC; ++q) {
        const int col = 8 * (WAVE * q + lane);
        wr[i][q] = load_nt16(p.latent_up + (int64_t)row * L + (col < L ? col : 0));
      }
    }
    if (!ready) stage_z();
    if (!uready) await(p.ctr + 32 * C_U_DONE, nu);
    uready = true;
    for (int t = 0; t < T; ++t) {
      double acc[UR];
#pragma unroll
      for (int i = 0; i < UR; ++i) acc[i] = 0.0;
#pragma unroll
      for (int q = 0; q < UC; ++q) {
        const int col = 8 * (WAVE * q + lane);
        if (col < L) {
          const uint4 x = *reinterpret_cast<const uint4*>(zs + t * L + col);
#pragma unroll
          for (int i = 0; i < UR; ++i) {
            float s = dot2(x.x, wr[i][q].x, 0.f);
            s = dot2(x.y, wr[i][q].y, s);
            s = dot2(x.z, wr[i][q].z, s);
            s = dot2(x.w, wr[i][q].w, s);
            acc[i] += (double)s;
          }
        }
      }
      if (lora) {
        const int a = p.lora.adapter[t];
        const bool have = (uint32_t)a < (uint32_t)p.lora.N;
        const int rk = !have ? 0 : p.lora.rank ? min(p.lora.rank[a], p.lora.R) : p.lora.R;
#pragma unroll
        for (int i = 0; i < UR; ++i) {
          const int row = min(c + wave + DEC_WAVES * i, d - 1);
          for (int r = lane; r < rk; r += WAVE)
            acc[i] += (double)p.u[t * p.lora.R + r] * (double)bf16f(p.lora.B[((int64_t)a * d + row) * p.lora.R + r]);
        }
      }
#pragma unroll
      for (int i = 0; i < UR; ++i) {
        const int row = c + wave + DEC_WAVES * i;
        const double v = wave_sum_dpp(acc[i]);
        if (lane == 0 && row < end) p.out[(int64_t)t * d + row] = f64_to_bf16(v);
      }
    }
  }
}

// ------------------------------------------------------------------------- host

size_t decode_aq_bytes(int64_t rows, int32_t F) { return (size_t)rows * dec_row_bytes(F); }

static int cu_count() {
  static const int n = [] {
    int dev = 0, v = 0;
    if (hipGetDevice(&dev) != hipSuccess ||
        hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || v < 1)
      v = 256;
    return v;
  }();
  return n;
}

template <class W, int NS, int UC, int UR>
static hipError_t launch_decode_as(const DecodeArgs& a, unsigned grid, size_t lds, hipStream_t st) {
  static const hipError_t e =
      hipFuncSetAttribute(reinterpret_cast<const void*>(&decode_kernel<W, NS, UC, UR>),
                          hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024 - DEC_LDS_STATIC);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((decode_kernel<W, NS, UC, UR>), dim3(grid), dim3(DEC_THREADS), lds, st, a);
  return hipGetLastError();
}

hipError_t launch_decode(const DecodeArgs& a, bool packed, hipStream_t st) {
  const int T = (int)a.r.T, n = T * a.r.k, L = a.r.L, F = a.F;
  if (T < 1 || T > DECODE_MAX_TOKENS || n > DECODE_MAX_ROWS || L % 128 || F % 128 || L > 7168 || F > 7168 ||
      a.r.E > ROUTE_MAXI * WAVE || a.r.d % 8)
    return hipErrorInvalidValue;
  const size_t avail = 160 * 1024 - DEC_LDS_STATIC;
  // two rows a wave side by side halve the waves' dependent steps; where sixteen staged rows
  // exceed the LDS, one
  const bool two = (size_t)2 * DEC_WAVES * dec_row_bytes(F) <= avail;
  size_t lds = (size_t)T * dec_row_bytes(L);
  lds = lds > (size_t)(two ? 2 : 1) * DEC_WAVES * dec_row_bytes(F) ? lds : (size_t)(two ? 2 : 1) * DEC_WAVES * dec_row_bytes(F);
  if (lds > avail) return hipErrorInvalidValue;
  // one block per CU, fewer where no phase has that many items
  int64_t items = (int64_t)n * (F / DEC_ROWS);
  if (items < L / 16) items = L / 16;
  if (items < a.r.d / DEC_WAVES) items = a.r.d / DEC_WAVES;
  const unsigned grid = (unsigned)(items < cu_count() ? items : cu_count());
  const bool wide = L > 7 * 512;
  auto go = [&](auto wt) -> hipError_t {
    using W = decltype(wt);
    if (two)
      return wide ? launch_decode_as<W, 2, 14, 2>(a, grid, lds, st) : launch_decode_as<W, 2, 7, 4>(a, grid, lds, st);
    return wide ? launch_decode_as<W, 1, 14, 2>(a, grid, lds, st) : launch_decode_as<W, 1, 7, 4>(a, grid, lds, st);
  };
  return packed ? go(PackedW{}) : go(RecordW{});
}

}  // namespace moe
