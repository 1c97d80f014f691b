// The dense gated feed-forward block and its backward pass, bf16 in and out, on the tiles of
// tile_gemm.h.
//   forward:   g = Wg x, u = Wu x (fp32), a = bf16(silu(g) u), out = bf16(Wd a)
//   backward:  dA = Wd^T dout (fp32), s = 1 / (1 + e^-g),
//              a = bf16(g s u), dU = bf16(dA g s), dG = bf16(dA u s (1 + g (1 - s))),
//              dx = bf16(Wg^T dG + Wu^T dU), dWg = bf16(dG^T x), dWu = bf16(dU^T x), dWd = bf16(dout^T a)
// a, dG and dU are rounded to bf16 once each, since the matrix cores read them: the results are off by
// 0.0023 to 0.0024 (rms, relative), of which 0.0017 is their own rounding.  Fewer roundings where
// they were found to cost nothing: up to four tokens forward a stays fp32 if it fits the LDS (gemv_wide),
// up to 64 tokens backward each is held in two halves (0.0017 both).  So a token's result depends on
// how many are with it, within those roundings.  Every sum is fp32 (the kept g and u are bf16 so that
// training holds 4 bytes for a token and inner channel and not 8).
//
// Measured (kernels; rates of 2 M N K operations, bytes of weights read):
//   4096 tokens, 7168 -> 3584: gate/up 300-350 us (1.2-1.4 PFLOP/s), down 160-190 (1.1-1.3)
//   4096 tokens, 4096 -> 8192, backward: dA 275-297 us (0.93-1.0 PFLOP/s: its epilogue reads g and u and
//     stores a, dG, dU, 43 us a turn of tiles during which the matrix cores wait), dx 364-396
//     (1.4-1.5), weights' gradients 593-650 (1.3-1.4)
//   33 tokens, 3584 -> 7168: gate/up 23 us (4.5 TB/s), down 13.4 (3.8 TB/s) and 4 to join its pieces
//   1 token, 7168 -> 8192: gate/up 36.7 us (6.4 TB/s), down 21.5 (5.5 TB/s)
//   77 tokens, 512 -> 1000, backward: 8.6 + 6.8 + 3.5 + 6 us, of which some 5 a launch are there with
//     8 x 8 matrices too
#include "common.h"
#include "kernels.h"
#include "mfma_stream.h"
#include "tile_gemm.h"

#include <algorithm>

namespace moe {

namespace {

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const bf16x2_t v = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
  const uint32_t d[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16lo(d[i]);
    v[2 * i + 1] = bf16hi(d[i]);
  }
}

// The epilogues' results come in whole pieces of eight: every width is a multiple of 8.
struct NoHeld {};

// rows of bf16: product 0's at out[0], from row `cut` on at out[1], product 1's at out[2]
struct EpiRows {
  uint16_t* out[3];
  int32_t cut;
  int32_t N[2];
  float* part;
  static constexpr bool BEGINS = false;
  using Held = NoHeld;
  __device__ __forceinline__ Held hold(int, int) const { return {}; }
  __device__ __forceinline__ void put(int which, int m, int n, int, const Held&, const float (&v)[8]) const {
    uint16_t* o = which ? out[2] + (int64_t)m * N[1] : m < cut ? out[0] + (int64_t)m * N[0] : out[1] + (int64_t)(m - cut) * N[0];
    store8(o + n, v);
  }
};

// a = bf16(silu(g) u), and g and u themselves where they are kept
struct EpiGlu {
  uint16_t *a, *gate, *up;
  int32_t F;
  float* part;
  static constexpr bool BEGINS = false;
  using Held = NoHeld;
  __device__ __forceinline__ Held hold(int, int) const { return {}; }
  __device__ __forceinline__ void put(int, int m, int n, int, const Held&, const float (&g)[8], const float (&u)[8]) const {
    const int64_t at = (int64_t)m * F + n;
    if (gate) {
      store8(gate + at, g);
      store8(up + at, u);
    }
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = silu_f32(g[i]) * u[i];
    store8(a + at, v);
  }
};

// s = 1 / (1 + e^-g), 1 - s and g s, each to a few fp32 ulps (and what |g| 2^-24 makes of the exponential)
// for every g: from e^-|g|, past the range of the hardware's 2^x, which ends at 2^-126, from 2^32 times it,
// as in silu_f32.
struct Sigmoid {
  float s, rest, gs;
};
__device__ __forceinline__ Sigmoid sigmoid_f32(float g) {
  const float x = -fabsf(g) * 1.44269504088896341f;
  const bool tiny = x < -120.f;
  const float e2 = __builtin_amdgcn_exp2f(tiny ? x + 32.f : x), sc = tiny ? 0x1p-32f : 1.f;
  const float e = e2 * sc, r = __builtin_amdgcn_rcpf(1.f + e), less = e * r;
  return g >= 0.f ? Sigmoid{r, less, g * r} : Sigmoid{less, r, (g * e2) * sc * r};
}

// what rounding v to bf16 leaves, or 0 where it does not stay finite
__device__ __forceinline__ float rounded_off(float v) {
  const float r = v - (float)(__bf16)v;
  return fabsf(r) < INFINITY ? r : 0.f;
}

// dA's tile meets the kept g and u: a, dG, dU.  dgu holds dG and dU side by side, [T][2 F].  LOW: behind
// the T rows of either lie as many of what the rounding of those left.  Those may be zero, or of the other
// sign, and an infinity that met them would make a NaN of the one that it gives with the rounded
// values: for the weights' gradients they meet copies of x and dout without what is not finite, made
// here, and dx leaves their sums out where it has to (the copies: 64 tokens, 512 -> 1000 0.8 us of 22.5; 11
// tokens, 3952 -> 72, few blocks for many columns, 2 of 25).
template <bool LOW>
struct EpiGluBack {
  const uint16_t *gate, *up;
  uint16_t *a, *dgu;
  int32_t F, T;
  float* part;
  const uint16_t *x, *dout;  // LOW: copied to finite, one behind the other
  uint16_t* finite;          // null: the weights' gradients are not asked for
  int32_t d;
  static constexpr bool BEGINS = LOW;
  __device__ __forceinline__ void begin() const {
    if (!finite) return;
    const int pieces = T * (d / 8);
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < 2 * pieces; i += gridDim.x * blockDim.x) {
      const uint4 v = reinterpret_cast<const uint4*>(i < pieces ? x : dout)[i < pieces ? i : i - pieces];
      reinterpret_cast<uint4*>(finite)[i] = make_uint4(finite2(v.x), finite2(v.y), finite2(v.z), finite2(v.w));
    }
  }
  struct Held {
    uint4 g, u;
  };
  __device__ __forceinline__ Held hold(int m, int n) const {
    const int64_t at = (int64_t)m * F + n;
    return {*reinterpret_cast<const uint4*>(gate + at), *reinterpret_cast<const uint4*>(up + at)};
  }
  __device__ __forceinline__ void put(int, int m, int n, int, const Held& h, const float (&d)[8]) const {
    float g[8], u[8], av[8], dg[8], du[8];
    unpack8(h.g, g);
    unpack8(h.u, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const Sigmoid t = sigmoid_f32(g[i]);
      av[i] = t.gs * u[i];
      du[i] = d[i] * t.gs;
      dg[i] = d[i] * (u[i] * (t.s + t.gs * t.rest));  // u meets the slope first: d u may be past fp32 where this is not
    }
    store8(a + (int64_t)m * F + n, av);
    uint16_t* o = dgu + (int64_t)m * 2 * F + n;
    store8(o, dg);
    store8(o + F, du);
    if constexpr (LOW) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        av[i] = rounded_off(av[i]);
        dg[i] = rounded_off(dg[i]);
        du[i] = rounded_off(du[i]);
      }
      store8(a + (int64_t)(m + T) * F + n, av);
      o += (int64_t)T * 2 * F;
      store8(o, dg);
      store8(o + F, du);
    }
  }
};

// Up to eight tokens on the vector units: one wave a row of the weights (GLU: the same row of both
// matrices), 16 bytes a lane and load, eight loads (of each) on their way, the block's tokens in LDS.
// Good for narrow blocks, where the call is short (5 tokens, 256 -> 344: 5.2 + 4.6 us).  Of wide ones it
// falls off past four tokens: 7168 -> 8192 58.7 us for one, 87 for four, 164 for five and 176 for
// eight, where nine on the tiles take 69.4; the tokens of 7168 values then fill 112 KB of a unit's
// LDS, so one block of four waves runs there and fills it anew for every four rows of weights.
// out[t][row] = sum_k w[row][k] in[t][k]; GLU: bf16(silu(g) u), and g and u where they are kept.
// Bound: HBM.  A lane's sum is at most K / 128 pairs of products one after another, in fp32, then a
// tree over the lanes.
// WIDE: a stays fp32 between the two launches (GLU writes it so, the other reads it so).
struct GemvArgs {
  const uint16_t *w, *w1;  // [rows][K]
  const void* in;          // [T][K]
  void* out;               // [T][rows]
  uint16_t *gate, *up;     // [T][rows], nullable
  int32_t T, K, rows;
};
constexpr int GEMV_TOKENS = 8;
// rows of a block: every block reads all tokens, which of fp32 values is as much as two rows of weights
// each (8192 -> 7168, one token: 22.7 us with four rows)
constexpr int gemv_rows(bool glu, bool wide) { return wide && !glu ? 8 : 4; }
template <int G, bool GLU, bool WIDE>
__global__ void __launch_bounds__(64 * gemv_rows(GLU, WIDE)) ffn_gemv_kernel(GemvArgs p) {
  constexpr int ROWS = gemv_rows(GLU, WIDE);
  constexpr int U = 8, M = GLU ? 2 : 1, P = WIDE && !GLU ? 2 : 1;  // P x 16 bytes: eight values of a token
  extern __shared__ __align__(16) uint8_t lds[];
  uint4* xs = reinterpret_cast<uint4*>(lds);  // [G][P][K / 8]
  const int lane = lane_id(), wave = threadIdx.x / WAVE;
  const int row = min((int)blockIdx.x * ROWS + wave, p.rows - 1);
  const bool mine = blockIdx.x * ROWS + wave < p.rows;
  const int pieces = p.K / 8;
  const uint4* w[2];
  w[0] = reinterpret_cast<const uint4*>(p.w + (int64_t)row * p.K);
  w[1] = GLU ? reinterpret_cast<const uint4*>(p.w1 + (int64_t)row * p.K) : w[0];
  uint4 held[M][U];
  auto load = [&](int base) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = base + 64 * u + lane;
#pragma unroll
      for (int m = 0; m < M; ++m) held[m][u] = at < pieces ? load_nt16(w[m] + at) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  load(0);
#pragma unroll
  for (int t = 0; t < G; ++t) {
    const uint4* x = static_cast<const uint4*>(p.in) + (int64_t)min(t, p.T - 1) * pieces * P;
    for (int i = threadIdx.x; i < pieces * P; i += 64 * ROWS) xs[(t * P + i % P) * pieces + i / P] = x[i];
  }
  lds_barrier();
  float acc[M][G];
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int t = 0; t < G; ++t) acc[m][t] = 0.f;
  for (int base = 0; base < pieces; base += 64 * U) {
    uint4 cur[M][U];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int m = 0; m < M; ++m) cur[m][u] = held[m][u];
    if (base + 64 * U < pieces) load(base + 64 * U);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = base + 64 * u + lane;
      if (base + 64 * u >= pieces) break;
#pragma unroll
      for (int t = 0; t < G; ++t) {
        const uint4 x = xs[t * P * pieces + min(at, pieces - 1)];
        const bool in = at < pieces;
        if constexpr (P == 2) {
          const uint4 y = xs[(t * P + 1) * pieces + min(at, pieces - 1)];
          float v[8], s = acc[0][t];
          unpack8(cur[0][u], v);
          const uint32_t b[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) s = __builtin_fmaf(__builtin_bit_cast(float, b[i]), v[i], s);
          acc[0][t] = in ? s : acc[0][t];
          continue;
        }
#pragma unroll
        for (int m = 0; m < M; ++m) {
          float s = acc[m][t];
          s = dot2(x.x, cur[m][u].x, s);
          s = dot2(x.y, cur[m][u].y, s);
          s = dot2(x.z, cur[m][u].z, s);
          s = dot2(x.w, cur[m][u].w, s);
          acc[m][t] = in ? s : acc[m][t];
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < G; ++t) {
    float v[M];
#pragma unroll
    for (int m = 0; m < M; ++m) v[m] = wave_sum_dpp(acc[m][t]);
    if (lane == 0 && mine && t < p.T) {
      const int64_t at = (int64_t)t * p.rows + row;
      if constexpr (GLU) {
        if constexpr (WIDE)
          static_cast<float*>(p.out)[at] = silu_f32(v[0]) * v[1];
        else
          static_cast<uint16_t*>(p.out)[at] = glu_bf16(v[0], v[1]);
        if (p.gate) {
          p.gate[at] = f32_to_bf16(v[0]);
          p.up[at] = f32_to_bf16(v[1]);
        }
      } else {
        static_cast<uint16_t*>(p.out)[at] = f32_to_bf16(v[0]);
      }
    }
  }
}
template <int G, bool GLU, bool WIDE>
hipError_t launch_gemv(const GemvArgs& a, hipStream_t st) {
  const size_t lds = (size_t)G * a.K * (WIDE && !GLU ? 4 : 2);
  if (lds > 65536) {
    static const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&ffn_gemv_kernel<G, GLU, WIDE>),
                                                    hipFuncAttributeMaxDynamicSharedMemorySize, 163840);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((ffn_gemv_kernel<G, GLU, WIDE>), dim3((unsigned)ceil_div(a.rows, gemv_rows(GLU, WIDE))),
                     dim3(64 * gemv_rows(GLU, WIDE)), lds, st, a);
  return hipGetLastError();
}
template <bool GLU>
hipError_t gemv(const GemvArgs& a, bool wide, hipStream_t st) {
  if (a.T > 4) return launch_gemv<8, GLU, false>(a, st);
  if (a.T > 2) return wide ? launch_gemv<4, GLU, true>(a, st) : launch_gemv<4, GLU, false>(a, st);
  if (a.T > 1) return wide ? launch_gemv<2, GLU, true>(a, st) : launch_gemv<2, GLU, false>(a, st);
  return launch_gemv<1, GLU, true>(a, st);  // of one token every width fits
}
// the tokens' rows have to fit the LDS
bool gemv_takes(int64_t T, int32_t K, int value_bytes = 2) {
  return T <= GEMV_TOKENS && (int64_t)(T <= 2 ? T : T <= 4 ? 4 : 8) * K * value_bytes <= 163840;
}
// Up to four tokens a stays fp32 where it fits: the results are off by their own rounding alone
// (8192 -> 7168, one token: 21.4 us, of a rounded 20.8).  Of eight tokens the reads of fp32 values
// would bind on the LDS.
bool gemv_wide(int64_t T, int32_t d, int32_t F) { return T <= 4 && gemv_takes(T, d) && gemv_takes(T, F, 4); }

int64_t k_tiles(int64_t K) { return ceil_div(K, 64); }
int splits_of(int64_t M, int64_t N, int64_t K, bool row_major) {
  const TileSize z = tile_size(M, N, k_tiles(K), row_major);
  return tile_splits(z, tiles_of(z, M, N), K / 64);
}
size_t part_bytes(int64_t M, int64_t N, int64_t K, bool row_major, int halves = 1) {
  const int s = splits_of(M, N, K, row_major);
  return s * halves > 1 ? (size_t)s * M * N * 4 : 0;
}
// of the weights' gradients, two products in one launch: one tile for both, by the three matrices'
// area in rows of d
TileSize weights_tile(int64_t T, int32_t d, int32_t F) { return tile_size(3 * (int64_t)F, d, k_tiles(T), true); }
int weights_splits(int64_t T, int32_t d, int32_t F) {
  const TileSize z = weights_tile(T, d, F);
  return tile_splits(z, tiles_of(z, 2 * (int64_t)F, d) + tiles_of(z, d, F), T / 64);
}
// Backward of few tokens: a, dG and dU are held in two halves of 8 bits each, since that is free there
// (one tile of rows and of K takes both).  Of more tokens each is rounded once.
constexpr int64_t HALVES_TOKENS = 64;
int halves_of(int64_t T) { return T <= HALVES_TOKENS ? 2 : 1; }
TileOperand operand(const void* p, int64_t ld_values, int32_t rows, const void* p1 = nullptr) {
  return TileOperand{{p, p1 ? p1 : p}, ld_values * 2, rows};
}

}  // namespace

FfnLayout ffn_layout(int64_t T, int32_t d, int32_t F) {
  FfnLayout l;
  l.a = 0;
  l.part = l.a + align_up((size_t)T * F * (gemv_wide(T, d, F) ? 4 : 2), 256);
  l.dgu = l.finite = 0;
  // used one after another: pieces of g and u, and of out
  const size_t glu = gemv_takes(T, d) ? 0 : part_bytes(T, 2 * (int64_t)F, d, false);
  const size_t out = gemv_takes(T, F) ? 0 : part_bytes(T, d, F, false);
  l.total = l.part + align_up(glu > out ? glu : out, 256);
  return l;
}
FfnLayout ffn_backward_layout(int64_t T, int32_t d, int32_t F) {
  FfnLayout l;
  const int h = halves_of(T);
  l.a = 0;
  l.dgu = l.a + align_up((size_t)T * F * 2 * h, 256);
  l.finite = l.dgu + align_up((size_t)T * F * 4 * h, 256);
  l.part = l.finite + (h > 1 ? align_up((size_t)T * d * 4, 256) : 0);
  // used one after another: pieces of dA, of dx, of the weights' gradients
  const int sw = weights_splits(T, d, F);
  size_t most = part_bytes(T, F, d, true);
  most = std::max(most, part_bytes(h * T, d, 2 * (int64_t)F, true, h));
  most = std::max(most, sw > 1 ? (size_t)sw * 3 * F * d * 4 : 0);
  l.total = l.part + align_up(most, 256);
  return l;
}

hipError_t launch_ffn(const FfnArgs& p, void* ws, hipStream_t st) {
  const FfnLayout l = ffn_layout(p.T, p.d, p.F);
  char* w = static_cast<char*>(ws);
  uint16_t* a = reinterpret_cast<uint16_t*>(w + l.a);
  float* part = reinterpret_cast<float*>(w + l.part);
  const int32_t T = (int32_t)p.T;
  hipError_t err;
  TileArgs t{};
  const bool wide = gemv_wide(T, p.d, p.F);
  if (gemv_takes(T, p.d)) {
    err = gemv<true>(GemvArgs{p.w_gate, p.w_up, p.x, a, p.gate, p.up, T, p.d, p.F}, wide, st);
  } else {
    t.m = operand(p.x, p.d, T);
    t.n = operand(p.w_gate, p.d, p.F, p.w_up);
    t.K = p.d;
    t.splits = splits_of(T, 2 * (int64_t)p.F, p.d, false);
    t.halves = 1;
    err = run_tiles<TILE_KMAJ, TILE_KMAJ, true, false>(tile_size(T, 2 * (int64_t)p.F, k_tiles(p.d), false), t, 1,
                                                EpiGlu{a, p.gate, p.up, p.F, part}, st);
  }
  if (err != hipSuccess) return err;
  if (gemv_takes(T, p.F)) return gemv<false>(GemvArgs{p.w_down, nullptr, a, p.out, nullptr, nullptr, T, p.F, p.d}, wide, st);
  t.m = operand(a, p.F, T);
  t.n = operand(p.w_down, p.F, p.d);
  t.K = p.F;
  t.splits = splits_of(T, p.d, p.F, false);
  t.halves = 1;
  const EpiRows e{{p.out, nullptr, nullptr}, T, {p.d, 0}, part};
  return run_tiles<TILE_KMAJ, TILE_KMAJ, false, false>(tile_size(T, p.d, k_tiles(p.F), false), t, 1, e, st);
}

// Three launches, and a join where dx's K is split: dA with a, dG and dU; dx, whose K is dG's and then dU's; and the weights' gradients,
// two products of the same K in one launch.
hipError_t launch_ffn_backward(const FfnBackArgs& p, void* ws, hipStream_t st) {
  const FfnLayout l = ffn_backward_layout(p.T, p.d, p.F);
  char* w = static_cast<char*>(ws);
  uint16_t* a = reinterpret_cast<uint16_t*>(w + l.a);
  uint16_t* dgu = reinterpret_cast<uint16_t*>(w + l.dgu);
  float* part = reinterpret_cast<float*>(w + l.part);
  const int32_t T = (int32_t)p.T;
  const int h = halves_of(T);
  TileArgs t{};
  t.m = operand(p.dout, p.d, T);
  t.n = operand(p.w_down, p.F, p.F);
  t.K = p.d;
  t.splits = splits_of(T, p.F, p.d, true);
  t.halves = 1;
  hipError_t err;
  const TileSize z = tile_size(T, p.F, k_tiles(p.d), true);
  uint16_t* finite = reinterpret_cast<uint16_t*>(w + l.finite);
  if (h > 1)  // never the large tiles
    err = run_middle_tiles<TILE_KMAJ, TILE_RMAJ, false, false>(
        z, t, 1, EpiGluBack<true>{p.gate, p.up, a, dgu, p.F, T, part, p.x, p.dout, p.dw_gate ? finite : nullptr, p.d}, st);
  else
    err = run_tiles<TILE_KMAJ, TILE_RMAJ, false, false>(
        z, t, 1, EpiGluBack<false>{p.gate, p.up, a, dgu, p.F, T, part, nullptr, nullptr, nullptr, p.d}, st);
  if (err == hipSuccess && p.dx) {
    t.m = operand(dgu, 2 * (int64_t)p.F, h * T, dgu + p.F);
    t.n = operand(p.w_gate, p.d, p.d, p.w_up);
    t.K = p.F;
    t.splits = splits_of(h * T, p.d, 2 * (int64_t)p.F, true);
    t.halves = h;
    const EpiRows e{{p.dx, nullptr, nullptr}, T, {p.d, 0}, part};
    err = run_tiles<TILE_KMAJ, TILE_RMAJ, false, false>(tile_size(h * T, p.d, k_tiles(2 * (int64_t)p.F), true), t, 2, e, st);
  }
  if (err == hipSuccess && p.dw_gate) {
    TileArgs u{};
    t.m = operand(dgu, 2 * (int64_t)p.F, 2 * p.F, dgu + 2 * (int64_t)p.F * T);  // the second halves, of h == 2
    t.n = operand(p.x, p.d, p.d, finite);
    u.m = operand(p.dout, p.d, p.d, finite + (int64_t)p.d * T);
    u.n = operand(a, p.F, p.F, a + (int64_t)p.F * T);
    t.K = u.K = T;
    t.splits = u.splits = weights_splits(T, p.d, p.F);
    t.halves = u.halves = 1;
    u.which = 1;
    u.part = (int64_t)t.splits * 2 * p.F * p.d;
    const EpiRows e{{p.dw_gate, p.dw_up, p.dw_down}, p.F, {p.d, p.F}, part};
    err = run_tiles<TILE_RMAJ, TILE_RMAJ, false, false>(weights_tile(T, p.d, p.F), t, h, e, st, &u);
  }
  return err;
}

}  // namespace moe
