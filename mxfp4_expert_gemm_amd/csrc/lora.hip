// Low-rank adapters of many requests beside one shared projection: the first product,
//   u[t][r] = scale[a_t] * sum_i A[a_t][r][i] x[t][i],   r < rank[a_t], a_t the token's adapter,
// in fp32 (zero past the rank and for a token without an adapter).  The second product,
// sum_r B[a_t][o][r] u[t][r], is added where the projection itself is computed
// (dense_gemv.hip, dense_mfma.hip), so no [T][n_out] intermediate exists and the output is
// rounded once.
//
// Two forms.  Few (token, rank) pairs: a wave per pair, x[t] against one row of A, the
// way the GEMV reads a weight row; requests with one adapter share its rows in the L2.
// Many: the tokens are grouped by adapter and a tile of up to 64 of them runs on the matrix
// cores (v_mfma_f32_16x16x32_bf16), the K range cut into slices so that the grid fills the
// chip; the slices' fp32 partials are added in slice order by the kernel that also splits u
// into the bf16 terms the matrix-core projection reads.
#include "common.h"
#include "kernels.h"

namespace moe {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int LT_TOK = 64;       // tokens per matrix-core tile
constexpr int LT_SLICES = 8;     // at most so many K slices
constexpr int LT_MIN_K = 256;    // at least so much K per slice

struct LoraWs {
  float* u;         // [T][R]
  uint16_t* ut;     // [U_TERMS][T][rank_pad(R)]
  int32_t* perm;    // [T] tokens grouped by adapter
  int4* tiles;      // {adapter, first place in perm, tokens, 0}
  int32_t* ntiles;
  float* part;      // [slices][T][R]
  size_t total;
};

// at most so many tiles: one more than full ones for every adapter met
static int64_t lora_max_tiles(int64_t T, int32_t N) { return T / LT_TOK + (T < N ? T : N); }
static int lora_slices(int64_t T, int32_t K, int32_t N) {
  int64_t s = 1024 / lora_max_tiles(T, N);
  if (s > LT_SLICES) s = LT_SLICES;
  if (s > K / LT_MIN_K) s = K / LT_MIN_K;
  return s < 1 ? 1 : (int)s;
}
// The second form: its two extra launches and the detour through fp32 partials cost 10 to 25 us,
// a wave per pair reads x R times and A T times through the L2.  Whole projections with 4
// adapters, one after another over the tokens, 7168 -> 3584, first and second form: 64 tokens of
// rank 128 34.9 and 57.9 us, 256 of rank 64 55.5 and 68.5, 512 of rank 16 68.9 and 70.7, 512 of
// rank 64 144 and 144 (with 64 adapters 304 and 279), 1024 of rank 16 127 and 114; the projections in
// tiles of 64 x 64 throughout.
static bool lora_grouped(int64_t T, int32_t R) { return T > 512 || T * R > 16384; }

static LoraWs lora_ws(void* ws, int64_t T, int32_t K, int32_t N, int32_t R) {
  LoraWs l;
  size_t off = 0;
  char* base = static_cast<char*>(ws);
  auto take = [&](size_t bytes) {
    char* p = base + off;
    off = align_up(off + bytes, 256);
    return p;
  };
  const size_t t = (size_t)T, rp = (size_t)rank_pad(R);
  l.u = reinterpret_cast<float*>(take(t * (size_t)R * 4));
  l.ut = reinterpret_cast<uint16_t*>(take(U_TERMS * t * rp * 2));
  l.perm = nullptr;
  l.tiles = nullptr;
  l.ntiles = nullptr;
  l.part = nullptr;
  if (lora_grouped(T, R)) {
    l.perm = reinterpret_cast<int32_t*>(take(t * 4));
    l.tiles = reinterpret_cast<int4*>(take((size_t)lora_max_tiles(T, N) * 16));
    l.ntiles = reinterpret_cast<int32_t*>(take(4));
    l.part = reinterpret_cast<float*>(take((size_t)lora_slices(T, K, N) * t * (size_t)R * 4));
  }
  l.total = off;
  return l;
}
size_t lora_ws_bytes(int64_t T, int32_t K, int32_t N, int32_t R) { return lora_ws(nullptr, T, K, N, R).total; }

// ranks of a token's adapter in use (0 for a token without one)
__device__ __forceinline__ int token_rank(const LoraArgs& p, int a) {
  if ((uint32_t)a >= (uint32_t)p.N) return 0;
  return p.rank ? max(0, min(p.rank[a], p.R)) : p.R;
}

// u in the forms the projections read: fp32, and three bf16 terms whose sum it is.  Each term is
// the top half of what the earlier ones leave (exact differences), so the terms of a value have one
// sign, and a finite value above the largest bf16 stays finite; an infinity or NaN is its first term
// alone.
__device__ __forceinline__ void put_u(const LoraArgs& p, const LoraWs& w, int64_t t, int r, float v) {
  if (r < p.R) w.u[t * p.R + r] = v;
  const int RP = rank_pad(p.R);
  uint16_t* at = w.ut + t * RP + r;
  const bool finite = fabsf(v) <= 0x1.fffffep127f;
  float rest = v;
#pragma unroll
  for (int i = 0; i < U_TERMS; ++i) {
    const uint16_t top = v != v && i == 0 ? (uint16_t)0x7FC0 : (uint16_t)(__float_as_uint(rest) >> 16);
    at[(int64_t)i * p.T * RP] = top;
    rest = finite ? rest - bf16f(top) : 0.f;
  }
}

// A wave per (token, rank), ranks up to rank_pad(R).  Chunk partials of eight exact products
// are folded into fp64 like the GEMV's.
__global__ void __launch_bounds__(256) lora_shrink_rows_kernel(LoraArgs p, LoraWs w) {
  const int lane = lane_id();
  const int r = blockIdx.x * 4 + threadIdx.x / WAVE;
  const int64_t t = blockIdx.y;
  if (r >= rank_pad(p.R)) return;
  const int a = p.adapter[t];
  float v = 0.f;
  if (r < token_rank(p, a)) {
    const uint16_t* x = p.x + t * p.K;
    const uint16_t* A = p.A + ((int64_t)a * p.R + r) * p.K;
    constexpr int U = 8;  // chunks of eight values a lane has in flight
    double acc = 0.0;
    for (int c0 = 8 * lane; c0 < p.K; c0 += 8 * WAVE * U) {
      uint4 xv[U], av[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int c = c0 + 8 * WAVE * i;
        xv[i] = *reinterpret_cast<const uint4*>(x + (c < p.K ? c : 0));
        av[i] = *reinterpret_cast<const uint4*>(A + (c < p.K ? c : 0));
      }
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (c0 + 8 * WAVE * i < p.K) {
          float q = dot2(xv[i].x, av[i].x, 0.f);
          q = dot2(xv[i].y, av[i].y, q);
          q = dot2(xv[i].z, av[i].z, q);
          q = dot2(xv[i].w, av[i].w, q);
          acc += (double)q;
        }
    }
    v = (float)(wave_sum_dpp(acc) * (double)p.scale[a]);
  }
  if (lane == 0) put_u(p, w, t, r, v);
}

// The tokens grouped by adapter (those without one left out) and cut into tiles, by one
// block: counts, places and tiles are formed in LDS.  The order inside a group depends on the
// atomics and does not matter: a token's row of a matrix-core tile depends on no other row.
__global__ void __launch_bounds__(1024) lora_group_kernel(const int32_t* __restrict__ adapter, int64_t T, int N,
                                                          int32_t* __restrict__ perm, int4* __restrict__ tiles,
                                                          int32_t* __restrict__ ntiles) {
  __shared__ int cnt[LORA_MAX_ADAPTERS], sum[16], tsum[16];
  const int tid = threadIdx.x, lane = lane_id(), wave = tid / WAVE;
  cnt[tid] = 0;
  __syncthreads();
  // a wave's tokens of one adapter take one atomic: segments cost one or two a wave
  auto each = [&](auto&& f) {
    for (int64_t b = (int64_t)wave * WAVE; b < T; b += 1024) {
      const int64_t t = b + lane;
      const int a = t < T ? adapter[t] : -1;
      for (unsigned long long todo = __ballot((uint32_t)a < (uint32_t)N); todo;) {
        const int lead = __ffsll((long long)todo) - 1;
        const int ad = __builtin_amdgcn_readlane(a, lead);
        const unsigned long long same = __ballot(a == ad);
        todo &= ~same;
        f(ad, same, lead, t, a == ad);
      }
    }
  };
  each([&](int ad, unsigned long long same, int lead, int64_t, bool) {
    if (lane == lead) atomicAdd(&cnt[ad], __popcll(same));
  });
  __syncthreads();
  const int c = tid < N ? cnt[tid] : 0, nt = (c + LT_TOK - 1) / LT_TOK;
  int ctot = 0, ttot = 0;
  int at = wave_excl_scan(c, ctot), tl = wave_excl_scan(nt, ttot);
  if (lane == 0) {
    sum[wave] = ctot;
    tsum[wave] = ttot;
  }
  __syncthreads();
  int all = 0;
  for (int v = 0; v < 16; ++v) {
    at += v < wave ? sum[v] : 0;
    tl += v < wave ? tsum[v] : 0;
    all += tsum[v];
  }
  for (int i = 0; i < nt; ++i)
    tiles[tl + i] = make_int4(tid, at + i * LT_TOK, min(LT_TOK, c - i * LT_TOK), 0);
  if (tid == 0) *ntiles = all;
  __syncthreads();
  cnt[tid] = at;  // from here on: the adapter's next free place
  __syncthreads();
  each([&](int ad, unsigned long long same, int lead, int64_t t, bool mine) {
    int base = 0;
    if (lane == lead) base = atomicAdd(&cnt[ad], __popcll(same));
    base = __builtin_amdgcn_readlane(base, lead);
    if (mine) perm[base + __popcll(same & ((1ull << lane) - 1ull))] = (int32_t)t;
  });
}

// Tile blockIdx.x, K slice blockIdx.y, ranks from 16 RB blockIdx.z: wave w has tokens
// 16w .. 16w+15 of the tile and all RB blocks of 16 ranks.  Operands come straight from global memory in the instruction's
// order (lane l: row l%16, eight K values of block l/16): a block of ranks reads the tile's
// token rows once, the adapter's rows by four waves through the L1.  A wave has up to 24 KB
// of loads under way, 16 rows of 64 bytes each, and their latency is what bounds it: 41 us at
// 4096 x 7168, rank 32 (59 MB of x: 1.4 TB/s), of 283 with the projection.  Blocks of 16,
// 32, 64 or 128 ranks, 8 or 16 slices and 256 or 512 of K at least are within 5% of each other in
// the whole projection; 32 and 256 were never behind (600 tokens of rank 64, 3584 -> 7168: 82.6
// against 86.8 us with 64 and 512).
template <int RB>
__global__ void __launch_bounds__(256) lora_shrink_mfma_kernel(LoraArgs p, LoraWs w, int slices) {
  if ((int)blockIdx.x >= *w.ntiles) return;
  const int4 tile = w.tiles[blockIdx.x];
  const int lane = lane_id(), wave = threadIdx.x / WAVE, nl = lane & 15, g = lane >> 4;
  if (16 * wave >= tile.z) return;
  const int rk = token_rank(p, tile.x), rank0 = 16 * RB * blockIdx.z;
  const int row = 16 * wave + nl;
  const int64_t t = w.perm[tile.y + (row < tile.z ? row : tile.z - 1)];
  // slices are whole steps of 32
  const int steps = p.K / 32, per = (steps + slices - 1) / slices;
  const int s0 = blockIdx.y * per, s1 = min(steps, s0 + per);
  const uint16_t* x = p.x + t * p.K + 8 * g;
  const uint16_t* A[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    const int r = min(rank0 + 16 * b + nl, p.R - 1);
    A[b] = p.A + ((int64_t)tile.x * p.R + r) * p.K + 8 * g;
  }
  f32x4_t acc[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) acc[b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  constexpr int U = 8;  // steps in flight
  for (int s = s0; s < s1; s += U) {
    bf16x8_t xv[U], av[U][RB];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int k = 32 * min(s + i, s1 - 1);
      xv[i] = *reinterpret_cast<const bf16x8_t*>(x + k);
#pragma unroll
      for (int b = 0; b < RB; ++b) av[i][b] = *reinterpret_cast<const bf16x8_t*>(A[b] + k);
    }
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (s + i < s1)
#pragma unroll
        for (int b = 0; b < RB; ++b)
          acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv[i], av[i][b], acc[b], 0, 0, 0);
  }
  // acc[b][j] of lane l is token row 4 g + j, rank 16 b + nl
  float* out = w.part + (int64_t)blockIdx.y * p.T * p.R;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int m = 16 * wave + 4 * g + j;
    if (m >= tile.z) continue;
    const int64_t tm = w.perm[tile.y + m];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const int r = rank0 + 16 * b + nl;
      if (r < p.R) out[tm * p.R + r] = r < rk ? acc[b][j] : 0.f;
    }
  }
}

// the slices' partials added, scaled and put in the forms the projections read; a thread
// per (token, rank up to rank_pad(R))
__global__ void __launch_bounds__(256) lora_join_kernel(LoraArgs p, LoraWs w, int slices) {
  const int RP = rank_pad(p.R);
  const int64_t n = p.T * RP;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t t = i / RP;
    const int r = (int)(i - t * RP);
    const int a = p.adapter[t];
    float v = 0.f;
    if (r < token_rank(p, a)) {
      for (int s = 0; s < slices; ++s) v += w.part[((int64_t)s * p.T + t) * p.R + r];
      v *= p.scale[a];
    }
    put_u(p, w, t, r, v);
  }
}

template <int RB>
static void launch_shrink_mfma(const LoraArgs& a, const LoraWs& w, int slices, hipStream_t st) {
  const dim3 grid((unsigned)lora_max_tiles(a.T, a.N), (unsigned)slices, (unsigned)ceil_div(a.R, 16 * RB));
  hipLaunchKernelGGL(lora_shrink_mfma_kernel<RB>, grid, dim3(256), 0, st, a, w, slices);
}

hipError_t launch_lora_shrink(const LoraArgs& a, void* ws, LoraSeg* seg, hipStream_t st) {
  if (a.T == 0) return hipSuccess;
  if (a.N < 1 || a.N > LORA_MAX_ADAPTERS || a.R < 8 || a.R > LORA_MAX_RANK || a.R % 8 || a.K % 32)
    return hipErrorInvalidValue;
  const LoraWs w = lora_ws(ws, a.T, a.K, a.N, a.R);
  seg->B = a.B;
  seg->adapter = a.adapter;
  seg->rank = a.rank;
  seg->u = w.u;
  seg->ut = w.ut;
  seg->N = a.N;
  seg->R = a.R;
  if (!lora_grouped(a.T, a.R)) {
    const dim3 grid((unsigned)(rank_pad(a.R) / 4), (unsigned)a.T);
    hipLaunchKernelGGL(lora_shrink_rows_kernel, grid, dim3(256), 0, st, a, w);
    return hipGetLastError();
  }
  const int slices = lora_slices(a.T, a.K, a.N);
  hipLaunchKernelGGL(lora_group_kernel, dim3(1), dim3(1024), 0, st, a.adapter, a.T, a.N, w.perm, w.tiles, w.ntiles);
  if (a.R <= 16)
    launch_shrink_mfma<1>(a, w, slices, st);
  else
    launch_shrink_mfma<2>(a, w, slices, st);
  int64_t blocks = ceil_div(a.T * rank_pad(a.R), 256);
  if (blocks > 4096) blocks = 4096;
  hipLaunchKernelGGL(lora_join_kernel, dim3((unsigned)blocks), dim3(256), 0, st, a, w, slices);
  return hipGetLastError();
}

}  // namespace moe
