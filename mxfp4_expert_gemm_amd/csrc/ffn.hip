// The dense gated feed-forward block and its backward pass, bf16 in and out, on the tiles of
// tile_gemm.h.
//   forward:   g = Wg x, u = Wu x (fp32), a = bf16(silu(g) u), out = bf16(Wd a)
//   backward:  dA = Wd^T dout (fp32), s = 1 / (1 + e^-g),
//              a = bf16(g s u), dU = bf16(dA g s), dG = bf16(dA u s (1 + g (1 - s))),
//              dx = bf16(Wg^T dG + Wu^T dU), dWg = bf16(dG^T x), dWu = bf16(dU^T x), dWd = bf16(dout^T a)
// a, dG and dU are rounded to bf16 since the matrix cores read them; every sum is fp32 (the kept
// g and u are bf16 so that training holds 4 bytes for a token and inner channel and not 8).
#include "common.h"
#include "kernels.h"
#include "mfma_stream.h"
#include "tile_gemm.h"

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

// rows of bf16, the first `cut` of them at out[0], the others at out[1]; or, of split sums, fp32
// pieces [split][M][N]
struct EpiRows {
  uint16_t* out[2];
  int32_t cut;
  float* part;
  int32_t M, N;
  using Held = NoHeld;
  __device__ __forceinline__ Held hold(int, int, int) const { return {}; }
  __device__ __forceinline__ void put(int m, int n, int, int split, const Held&, const float (&v)[8]) const {
    if (part) {
      float* p = part + ((int64_t)split * M + m) * N + n;
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      store8((m < cut ? out[0] + (int64_t)m * N : out[1] + (int64_t)(m - cut) * N) + n, v);
    }
  }
};

// a = bf16(silu(g) u), and g and u themselves where they are kept
struct EpiGlu {
  uint16_t *a, *gate, *up;
  int32_t F;
  using Held = NoHeld;
  __device__ __forceinline__ Held hold(int, int, int) const { return {}; }
  __device__ __forceinline__ void put(int m, int n, int, int, const Held&, const float (&g)[8], const float (&u)[8]) const {
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

// dA's tile meets the kept g and u: a, dG, dU.  dgu holds dG and dU side by side, [T][2 F].
struct EpiGluBack {
  const uint16_t *gate, *up;
  uint16_t *a, *dgu;
  int32_t F;
  struct Held {
    uint4 g, u;
  };
  __device__ __forceinline__ Held hold(int m, int n, int) const {
    const int64_t at = (int64_t)m * F + n;
    return {*reinterpret_cast<const uint4*>(gate + at), *reinterpret_cast<const uint4*>(up + at)};
  }
  __device__ __forceinline__ void put(int m, int n, int, int, const Held& h, const float (&d)[8]) const {
    float g[8], u[8], av[8], dg[8], du[8];
    unpack8(h.g, g);
    unpack8(h.u, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = 1.f / (1.f + __expf(-g[i])), gs = g[i] * s;
      av[i] = gs * u[i];
      du[i] = d[i] * gs;
      dg[i] = d[i] * u[i] * (s + gs * (1.f - s));
    }
    store8(a + (int64_t)m * F + n, av);
    uint16_t* o = dgu + (int64_t)m * 2 * F + n;
    store8(o, dg);
    store8(o + F, du);
  }
};

// out = bf16(sum over the splits), eight values a thread, in the splits' order
__global__ void __launch_bounds__(256) join_splits_kernel(const float* __restrict__ part, int64_t n8, int splits,
                                                          uint16_t* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n8) return;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < splits; ++s) {
    const float* p = part + (int64_t)s * n8 * 8 + 8 * i;
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    const float w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += w[j];
  }
  store8(out + 8 * i, v);
}

// which tiles a product takes
enum TileSize { TILE_32, TILE_64, TILE_128, TILE_224, TILE_256 };

// The K tiles are split where the tiles of the output alone leave compute units idle: no more
// pieces than bring the grid to one block a unit, of 16 steps of 32 at least.
int split_count(int64_t tiles, int64_t K) {
  const int64_t most = K / 512, want = 256 / tiles;
  const int64_t s = want < most ? want : most;
  return s < 1 ? 1 : s > 16 ? 16 : (int)s;
}
TileSize tile_size(int64_t M, int64_t N, bool row_major) {
  if (ceil_div(M, 256) * ceil_div(N, 256) >= 192) return tiles_of_224(M, N) ? TILE_224 : TILE_256;
  if (M > 64 || row_major) return TILE_128;
  return M > 32 ? TILE_64 : TILE_32;
}
int64_t tile_count(TileSize z, int64_t M, int64_t N) {
  switch (z) {
    case TILE_256: case TILE_224: return 256;  // not split
    case TILE_128: return ceil_div(M, 128) * ceil_div(N, 128);
    case TILE_64: return ceil_div(N, 32);
    default: return ceil_div(N, 32);
  }
}
int splits_of(int64_t M, int64_t N, int64_t K, bool row_major) {
  return split_count(tile_count(tile_size(M, N, row_major), M, N), K);
}
size_t part_bytes(int64_t M, int64_t N, int64_t K, bool row_major) {
  const int s = splits_of(M, N, K, row_major);
  return s > 1 ? (size_t)s * M * N * 4 : 0;
}

template <int MO, int NO>
hipError_t product_tiles(TileSize z, const TileArgs& a, int segs, const EpiRows& e, hipStream_t st) {
  if (z == TILE_256) return launch_tile_gemm<TileCfg<8, 8, 2, 2, 5, MO, NO, false>>(a, segs, e, st);
  if (z == TILE_224) return launch_tile_gemm<TileCfg<8, 7, 2, 2, 5, MO, NO, false>>(a, segs, e, st);
  if constexpr (MO == TILE_KMAJ && NO == TILE_KMAJ) {
    if (z == TILE_64) return launch_tile_gemm<TileCfg<2, 1, 2, 2, 13, MO, NO, false>>(a, segs, e, st);
    if (z == TILE_32) return launch_tile_gemm<TileCfg<1, 1, 2, 2, 13, MO, NO, false>>(a, segs, e, st);
  }
  return launch_tile_gemm<TileCfg<4, 4, 2, 2, 5, MO, NO, false>>(a, segs, e, st);
}

// out [M][N] (its rows from `cut` on at out1) = sum over `segs` segments of K; part: room for splits
template <int MO, int NO>
hipError_t product(TileArgs a, int segs, uint16_t* out, uint16_t* out1, int32_t cut, float* part, hipStream_t st) {
  const int64_t M = a.m.rows, N = a.n.rows;
  const bool rmaj = MO == TILE_RMAJ || NO == TILE_RMAJ;
  const TileSize z = tile_size(M, N, rmaj);
  a.splits = out1 ? 1 : splits_of(M, N, a.K * segs, rmaj);
  EpiRows e{{out, out1}, cut, a.splits > 1 ? part : nullptr, (int32_t)M, (int32_t)N};
  const hipError_t err = product_tiles<MO, NO>(z, a, segs, e, st);
  if (err != hipSuccess || a.splits == 1) return err;
  const int64_t n8 = M * N / 8;
  hipLaunchKernelGGL(join_splits_kernel, dim3((unsigned)ceil_div(n8, 256)), dim3(256), 0, st, part, n8, a.splits, out);
  return hipGetLastError();
}

TileOperand operand(const void* p, int64_t ld_values, int32_t rows, const void* p1 = nullptr) {
  return TileOperand{{p, p1 ? p1 : p}, ld_values * 2, rows};
}

size_t max2(size_t a, size_t b) { return a > b ? a : b; }

}  // namespace

FfnLayout ffn_layout(int64_t T, int32_t d, int32_t F) {
  FfnLayout l;
  l.a = 0;
  l.part = align_up((size_t)T * F * 2, 256);
  l.dgu = 0;
  l.total = l.part + align_up(part_bytes(T, d, F, false), 256);
  return l;
}
FfnLayout ffn_backward_layout(int64_t T, int32_t d, int32_t F) {
  FfnLayout l;
  l.a = 0;
  l.dgu = align_up((size_t)T * F * 2, 256);
  l.part = l.dgu + align_up((size_t)T * F * 4, 256);
  l.total = l.part + align_up(max2(part_bytes(T, d, 2 * (int64_t)F, true), part_bytes(d, F, T, true)), 256);
  return l;
}

hipError_t launch_ffn(const FfnArgs& p, void* ws, hipStream_t st) {
  const FfnLayout l = ffn_layout(p.T, p.d, p.F);
  uint16_t* a = reinterpret_cast<uint16_t*>(static_cast<char*>(ws) + l.a);
  float* part = reinterpret_cast<float*>(static_cast<char*>(ws) + l.part);
  TileArgs t{};
  t.m = operand(p.x, p.d, (int32_t)p.T);
  t.n = operand(p.w_gate, p.d, p.F, p.w_up);
  t.K = p.d;
  t.splits = 1;
  const EpiGlu e{a, p.gate, p.up, p.F};
  hipError_t err;
  switch (tile_size(p.T, 2 * (int64_t)p.F, false)) {
    case TILE_256: err = launch_tile_gemm<TileCfg<8, 8, 2, 2, 5, TILE_KMAJ, TILE_KMAJ, true>>(t, 1, e, st); break;
    case TILE_224: err = launch_tile_gemm<TileCfg<8, 7, 2, 2, 5, TILE_KMAJ, TILE_KMAJ, true>>(t, 1, e, st); break;
    case TILE_128: err = launch_tile_gemm<TileCfg<4, 4, 2, 2, 5, TILE_KMAJ, TILE_KMAJ, true>>(t, 1, e, st); break;
    case TILE_64: err = launch_tile_gemm<TileCfg<2, 2, 2, 2, 13, TILE_KMAJ, TILE_KMAJ, true>>(t, 1, e, st); break;
    default: err = launch_tile_gemm<TileCfg<1, 2, 2, 2, 13, TILE_KMAJ, TILE_KMAJ, true>>(t, 1, e, st); break;
  }
  if (err != hipSuccess) return err;
  t.m = operand(a, p.F, (int32_t)p.T);
  t.n = operand(p.w_down, p.F, p.d);
  t.K = p.F;
  return product<TILE_KMAJ, TILE_KMAJ>(t, 1, p.out, nullptr, (int32_t)p.T, part, st);
}

hipError_t launch_ffn_backward(const FfnBackArgs& p, void* ws, hipStream_t st) {
  const FfnLayout l = ffn_backward_layout(p.T, p.d, p.F);
  uint16_t* a = reinterpret_cast<uint16_t*>(static_cast<char*>(ws) + l.a);
  uint16_t* dgu = reinterpret_cast<uint16_t*>(static_cast<char*>(ws) + l.dgu);
  float* part = reinterpret_cast<float*>(static_cast<char*>(ws) + l.part);
  const int32_t T = (int32_t)p.T;
  TileArgs t{};
  t.m = operand(p.dout, p.d, T);
  t.n = operand(p.w_down, p.F, p.F);
  t.K = p.d;
  t.splits = 1;
  const EpiGluBack e{p.gate, p.up, a, dgu, p.F};
  hipError_t err;
  switch (tile_size(T, p.F, true)) {
    case TILE_256: err = launch_tile_gemm<TileCfg<8, 8, 2, 2, 5, TILE_KMAJ, TILE_RMAJ, false>>(t, 1, e, st); break;
    case TILE_224: err = launch_tile_gemm<TileCfg<8, 7, 2, 2, 5, TILE_KMAJ, TILE_RMAJ, false>>(t, 1, e, st); break;
    default: err = launch_tile_gemm<TileCfg<4, 4, 2, 2, 5, TILE_KMAJ, TILE_RMAJ, false>>(t, 1, e, st); break;
  }
  if (err == hipSuccess && p.dx) {
    t.m = operand(dgu, 2 * (int64_t)p.F, T, dgu + p.F);
    t.n = operand(p.w_gate, p.d, p.d, p.w_up);
    t.K = p.F;
    err = product<TILE_KMAJ, TILE_RMAJ>(t, 2, p.dx, nullptr, T, part, st);
  }
  if (err == hipSuccess && p.dw_gate) {
    t.m = operand(dgu, 2 * (int64_t)p.F, 2 * p.F);
    t.n = operand(p.x, p.d, p.d);
    t.K = T;
    err = product<TILE_RMAJ, TILE_RMAJ>(t, 1, p.dw_gate, p.dw_up, p.F, part, st);
  }
  if (err == hipSuccess && p.dw_down) {
    t.m = operand(p.dout, p.d, p.d);
    t.n = operand(a, p.F, p.F);
    t.K = T;
    err = product<TILE_RMAJ, TILE_RMAJ>(t, 1, p.dw_down, nullptr, p.d, part, st);
  }
  return err;
}

}  // namespace moe
