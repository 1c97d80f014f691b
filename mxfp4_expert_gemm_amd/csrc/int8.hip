// A projection in 8-bit integers: out[t][o] = bf16(x_scale[t] w_scale[o] sum_i q[t][i] W[o][i]), the
// sums exact in 32 bits, on the tiles of tile_gemm.h (v_mfma_i32_16x16x64_i8: the same bytes a
// step as the bf16 products, for twice the values); and the quantiser of its tokens,
//   q = 127 x / max|x| rounded to the nearest whole number, ties to even, x_scale = max|x| / 127.
// Measured: 8191 tokens, 3584 -> 7168: product 190-222 us (1.9-2.2 POP/s), quantiser 18-21 (4.2-4.9 TB/s
// of x and codes); 48 tokens, 7168 -> 3584: quantiser 4.2 us, product 9.2 (2.8 TB/s of weights: a
// stream this short is mostly its beginning and end), join 3.
#include "common.h"
#include "kernels.h"
#include "tile_gemm.h"

namespace moe {

namespace {

// 16 bytes at any even address: rows of odd widths lie so
typedef uint32_t any_u32x4_t __attribute__((ext_vector_type(4), aligned(2)));

struct EpiInt8 {
  const float *xs, *ws;
  uint16_t* out;
  int32_t N;
  int32_t* part;
  static constexpr bool BEGINS = false;
  struct Held {};
  __device__ __forceinline__ Held hold(int, int) const { return {}; }
  __device__ __forceinline__ void put(int, int m, int n, int left, const Held&, const int32_t (&v)[8]) const {
    const float s = xs[m];
    uint16_t* o = out + (int64_t)m * N + n;
    if (left >= 8) {
      const float4 a = *reinterpret_cast<const float4*>(ws + n), b = *reinterpret_cast<const float4*>(ws + n + 4);
      const float w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      uint32_t d[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const bf16x2_t c = {(__bf16)((float)v[2 * r] * s * w[2 * r]), (__bf16)((float)v[2 * r + 1] * s * w[2 * r + 1])};
        d[r] = __builtin_bit_cast(uint32_t, c);
      }
      *reinterpret_cast<any_u32x4_t*>(o) = any_u32x4_t{d[0], d[1], d[2], d[3]};
    } else {
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < left) o[r] = f32_to_bf16((float)v[r] * s * ws[n + r]);
    }
  }
};

// One row a block.  Rows of up to 8192 values stay in registers between the search for the largest
// and the codes; longer ones are read again.  The bits of |x| order like the values, with what is
// not finite above them: such a row gets the scale NaN and codes 0, so that all of its results are
// NaN.  127 x is exact in fp32 and the quotient's one Newton step makes every representable one
// exact, so a tie (x = max / 2 is 63.5) is seen as one; other quotients lie further from a border
// than their error.  Tiny and huge rows are scaled by a power of two first.
__device__ __forceinline__ uint32_t pack_codes(float a, float b, float c, float d) {
  return ((uint32_t)(int)a & 255u) | ((uint32_t)(int)b & 255u) << 8 | ((uint32_t)(int)c & 255u) << 16 | (uint32_t)(int)d << 24;
}
__global__ void __launch_bounds__(256) quantize_int8_kernel(const uint16_t* __restrict__ x, int32_t n, int8_t* __restrict__ q,
                                                            float* __restrict__ scale) {
  constexpr int C = 4;
  __shared__ uint32_t tops[4];
  const int64_t t = blockIdx.x;
  const uint16_t* row = x + t * n;
  uint4 v[C];
  uint32_t top = 0;
  auto look = [&](const uint4& w) {
    const uint32_t d[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = d[i] & 0x7FFFu, hi = (d[i] >> 16) & 0x7FFFu;
      top = max(top, max(lo, hi));
    }
  };
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = 8 * (threadIdx.x + 256 * c);
    v[c] = col < n ? *reinterpret_cast<const uint4*>(row + col) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int c = 0; c < C; ++c) look(v[c]);
  for (int col = 8 * (threadIdx.x + 256 * C); col < n; col += 8 * 256) look(*reinterpret_cast<const uint4*>(row + col));
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
  if (lane_id() == 0) tops[threadIdx.x / WAVE] = top;
  __syncthreads();
  top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));

  const bool finite = top < 0x7F80u;
  const float most = bf16f((uint16_t)top);
  if (threadIdx.x == 0) scale[t] = finite ? most / 127.f : __builtin_nanf("");
  const float f = most < 0x1p-60f ? 0x1p100f : most > 0x1p60f ? 0x1p-60f : 1.f;
  const float a = most * f, m = 127.f * f;
  const float inv = finite && top != 0 ? 1.f / a : 0.f;
  auto code = [&](float xv) {
    if (!finite) return 0.f;
    const float p = xv * m, r = p * inv;
    return rintf(fmaf(fmaf(-r, a, p), inv, r));
  };
  auto write = [&](const uint4& w, int col) {
    const uint32_t d[4] = {w.x, w.y, w.z, w.w};
    uint32_t o[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      o[h] = pack_codes(code(bf16lo(d[2 * h])), code(bf16hi(d[2 * h])), code(bf16lo(d[2 * h + 1])), code(bf16hi(d[2 * h + 1])));
    *reinterpret_cast<uint2*>(q + t * n + col) = make_uint2(o[0], o[1]);
  };
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = 8 * (threadIdx.x + 256 * c);
    if (col < n) write(v[c], col);
  }
  for (int col = 8 * (threadIdx.x + 256 * C); col < n; col += 8 * 256) write(*reinterpret_cast<const uint4*>(row + col), col);
}

int int8_splits(int64_t M, int64_t N, int64_t K) {
  const TileSize z = tile_size(M, N, ceil_div(K, 128), false);
  return tile_splits(z, tiles_of(z, M, N), K / 128);
}

}  // namespace

Int8Layout int8_layout(int64_t T, int32_t n_in, int32_t n_out, bool quantize) {
  Int8Layout l;
  const int s = int8_splits(T, n_out, n_in);
  l.scale = 0;
  l.q = (quantize ? align_up((size_t)T * 4, 256) : 0);
  l.part = l.q + (quantize ? align_up((size_t)T * n_in, 256) : 0);
  l.total = l.part + (s > 1 ? align_up((size_t)s * T * align_up(n_out, 8) * 4, 256) : 0);
  return l;
}
hipError_t launch_quantize_int8(const uint16_t* x, int64_t T, int32_t n, int8_t* q, float* scale, hipStream_t st) {
  hipError_t err = hipSuccess;
  for (int64_t t = 0; t < T && err == hipSuccess; t += LAUNCH_BLOCKS) {
    const unsigned rows = (unsigned)(T - t < LAUNCH_BLOCKS ? T - t : LAUNCH_BLOCKS);
    hipLaunchKernelGGL(quantize_int8_kernel, dim3(rows), dim3(256), 0, st, x + t * n, n, q + t * n, scale + t);
    err = hipGetLastError();
  }
  return err;
}

hipError_t launch_linear_int8(const int8_t* q, const float* xs, const int8_t* W, const float* ws, int64_t T, int32_t n_in,
                              int32_t n_out, uint16_t* out, int32_t* part, hipStream_t st) {
  TileArgs a{};
  a.m = TileOperand{{q, q}, n_in, (int32_t)T};
  a.n = TileOperand{{W, W}, n_in, n_out};
  a.K = n_in;
  a.splits = int8_splits(T, n_out, n_in);
  a.halves = 1;
  a.part = 0;
  const EpiInt8 e{xs, ws, out, n_out, part};
  return run_tiles<TILE_KMAJ, TILE_KMAJ, false, true>(tile_size(T, n_out, ceil_div(n_in, 128), false), a, 1, e, st);
}

}  // namespace moe
