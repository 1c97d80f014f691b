// What stands between two blocks of a residual stream, in one pass over it: the norm after a
// block, its gate and residual scale, the sum into the stream, and the norm before the next
// block; and the gradients of all of that.
//   forward:   v = y / rms(y) post (or v = y),  out = bf16(residual + scale gate v),
//              normed = bf16(out / rms(out) pre),  rms(t) = sqrt(mean t^2 + eps)
//   backward:  with r = out, rh = r / rms(r), e = dnormed pre:
//              G = dout + (e - rh mean(e rh)) / rms(r)   (the gradient of out and of residual)
//              dpre = sum_t dnormed rh,  dgate = scale G v (summed over t for one gate of all tokens)
//              with yh = y / rms(y), b = scale gate G, f = b post:
//              dpost = sum_t b yh,  dy = (f - yh mean(f yh)) / rms(y)   (dy = b without a norm)
// Bound: HBM.  A row is held in registers from its first load on, so each tensor is read and
// written once: 8 bytes an element forward, 12 backward, 2 and 4 more with a gate of each token.
// A row belongs to one wave, or to four or eight where it is long.  Sums are fp32, of squares scaled by
// a power of two where they would leave its range.
// Measured: forward 8192 x 7168 with a gate of each token 103 us (5.7 TB/s), one row 3.6; backward
// 8192 x 4096 108-111 us (3.7 TB/s: some 60 fp32 operations an element on half-filled units, with two
// rows' tensors in registers; 5 us of it for the look at each sum's range) and 6 for the join of the
// blocks' sums, 333 x 1000 6.2-6.5 and 4.
#include "common.h"
#include "kernels.h"

namespace moe {

namespace {

__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
  const uint32_t d[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16lo(d[i]);
    v[2 * i + 1] = bf16hi(d[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  uint32_t d[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bf16x2_t p = {(__bf16)v[2 * i], (__bf16)v[2 * i + 1]};
    d[i] = __builtin_bit_cast(uint32_t, p);
  }
  return make_uint4(d[0], d[1], d[2], d[3]);
}
__device__ __forceinline__ uint4 load16(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ void store16(uint16_t* p, const uint4& v) { *reinterpret_cast<uint4*>(p) = v; }

// N sums over the WPR waves of a row, to all of them.  `turn` alternates between two places of
// the LDS, so that one barrier is enough: a wave writes a place again only behind the next
// barrier, which every wave reaches after it has read the place.
template <int WPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* lds, int turn) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum_dpp(v[i]);
  if constexpr (WPR > 1) {
    const int wave = threadIdx.x / WAVE, nw = blockDim.x / WAVE;
    float* at = lds + turn * nw * 4;
    if (lane_id() == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) at[4 * wave + i] = v[i];
    lds_barrier();
    const int first = wave / WPR * WPR;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < WPR; ++w) s += at[4 * (first + w) + i];
      v[i] = s;
    }
  }
}

// The squares of a row.  Of values past 2^60, and with a tiny eps of those under 2^-50, the sum of
// their squares nears an end of fp32's range or leaves it; a wave that finds its sum there takes it
// again of its values times a power of two (a branch of whole waves, from registers).  Range says
// which: of a row's waves the largest counts, and the others' sums are brought to it.
enum Range { IN = 0, HIGH = 1, LOW = 2 };
__device__ __forceinline__ int range_of(float squares, float eps) {
  const float t = squares + eps;
  return t < 0x1p120f ? (t < 0x1p-100f ? LOW : IN) : HIGH;  // an infinity or NaN: HIGH
}
__device__ __forceinline__ float range_scale(int range) { return range == IN ? 1.f : range == HIGH ? 0x1p-72f : 0x1p72f; }
// the larger of two, and what a value scaled for `from` is to be multiplied with to be scaled for `to`
__device__ __forceinline__ int range_max(int a, int b) { return a == HIGH || b == HIGH ? HIGH : a == IN || b == IN ? IN : LOW; }
__device__ __forceinline__ float range_step(int from, int to) {
  return from == to ? 1.f : from == LOW && to == HIGH ? 0.f : 0x1p-72f;  // 2^-144 of what is below 1
}

// row_sums of s[0] a row's squares, s[1] products with its values, s[2] another row's squares, each of
// the range that r (of the first two) and y say; on return those are the row's.
template <int WPR, int N>
__device__ __forceinline__ void row_statistics(float (&s)[N], int& r, int& y, float* lds, int turn) {
  static_assert(N == 1 || N == 3, "squares; or squares, products, squares");
  if constexpr (WPR > 1) {
    const int wave = threadIdx.x / WAVE, nw = blockDim.x / WAVE;
    float4* at = reinterpret_cast<float4*>(lds) + turn * nw;
    if (lane_id() == 0) at[wave] = make_float4(s[0], N > 1 ? s[1] : 0.f, N > 1 ? s[2] : 0.f, __int_as_float(r | y << 2));
    lds_barrier();
    const float4* mine = at + wave / WPR * WPR;
    int any = 0;
    float sum[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < WPR; ++w) {
      const float4 v = mine[w];
      sum[0] += v.x;
      sum[1] += v.y;
      sum[2] += v.z;
      any |= __float_as_int(v.w);
    }
    any = __builtin_amdgcn_readfirstlane(any);
    if (any != 0) {
      r = y = LOW;
#pragma unroll 1
      for (int w = 0; w < WPR; ++w) {
        const int f = __float_as_int(mine[w].w);
        r = range_max(r, f & 3);
        y = range_max(y, f >> 2);
      }
      sum[0] = sum[1] = sum[2] = 0.f;
#pragma unroll 1
      for (int w = 0; w < WPR; ++w) {
        const float4 v = mine[w];
        const int f = __float_as_int(v.w);
        const float a = range_step(f & 3, r), b = range_step(f >> 2, y);
        sum[0] += v.x * a * a;
        sum[1] += v.y * a;
        sum[2] += v.z * b * b;
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = sum[i];
  }
}

// sum of (x kx) w (y ky), w null: 1.  Word by word, and nothing that was computed from them is kept for
// it or by it: it is rare, and stands where registers are few.
template <int C>
__device__ __forceinline__ float scaled_sum(const uint4 (&x)[C], const uint4 (&y)[C], const uint4* w, float kx, float ky) {
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const uint32_t a[4] = {x[c].x, x[c].y, x[c].z, x[c].w}, b[4] = {y[c].x, y[c].y, y[c].z, y[c].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t p = a[i], q = b[i], r = 0x3F803F80u;  // two ones
      if (w) r = i == 0 ? w[c].x : i == 1 ? w[c].y : i == 2 ? w[c].z : w[c].w;
      asm volatile("" : "+v"(p), "+v"(q), "+v"(r), "+v"(s));
      s += (bf16lo(p) * kx) * bf16lo(r) * (bf16lo(q) * ky);
      s += (bf16hi(p) * kx) * bf16hi(r) * (bf16hi(q) * ky);
    }
  }
  return s;
}

// 1 / rms of the row itself, from squares of values times range_scale(range)
__device__ __forceinline__ float inverse_rms(float squares, int range, float inv_d, float eps) {
  const float k = range_scale(range);
  return k / sqrtf(squares * inv_d + eps * k * k);
}

// 1 / rms of the row whose pieces x are, s the lane's sum of their squares
template <int WPR, int C>
__device__ __forceinline__ float row_inverse_rms(const uint4 (&x)[C], float s0, float inv_d, float eps, float* red, int turn) {
  float s[1] = {wave_sum_dpp(s0)};
  int range = range_of(s[0], eps), none = IN;
  if (range != IN) {
    const float k = range_scale(range);
    s[0] = wave_sum_dpp(scaled_sum<C>(x, x, nullptr, k, k));
  }
  row_statistics<WPR>(s, range, none, red, turn);
  return inverse_rms(s[0], range, inv_d, eps);
}

// WPR waves a row, C pieces of 8 columns a thread
template <int WPR, int C>
__global__ void __launch_bounds__(256) block_norms_kernel(NormArgs p) {
  constexpr int GT = WPR * WAVE, ROWS = 256 / GT;
  __shared__ __align__(16) float red[2 * 4 * 4];
  const int at = threadIdx.x % GT;
  int64_t t = (int64_t)blockIdx.x * ROWS + threadIdx.x / GT;
  if constexpr (ROWS > 1) {
    if (t >= p.T) return;  // a wave of its own: no barrier waits for it
  }
  const int64_t row = t * p.d;
  uint4 y[C], r[C], g[C], pw[C], nw[C];
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = 8 * (at + GT * c);
    const bool in = col < p.d;
    y[c] = in && p.y ? load16(p.y + row + col) : zero;
    r[c] = in ? load16(p.residual + row + col) : zero;
    g[c] = in && p.gate ? load16(p.gate + t * p.gate_stride + col) : zero;
    pw[c] = in && p.post ? load16(p.post + col) : zero;
    nw[c] = in && p.pre ? load16(p.pre + col) : zero;
  }
  const float inv_d = 1.f / (float)p.d;
  float m = p.scale;
  if (p.post) {
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float v[8];
      unpack8(y[c], v);
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i] * v[i];
    }
    m = row_inverse_rms<WPR>(y, s, inv_d, p.eps, red, 0);
  }
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (p.y) {
      float v[8], o[8], w[8];
      unpack8(y[c], v);
      unpack8(r[c], o);
      if (p.post) {
        unpack8(pw[c], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] * m * w[i] * p.scale;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= p.scale;
      }
      if (p.gate) {
        unpack8(g[c], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= w[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] += v[i];
      r[c] = pack8(o);
      const int col = 8 * (at + GT * c);
      if (col < p.d) store16(p.out + row + col, r[c]);
    }
    float v[8];
    unpack8(r[c], v);
#pragma unroll
    for (int i = 0; i < 8; ++i) s += v[i] * v[i];
  }
  if (!p.pre) return;
  const float k = row_inverse_rms<WPR>(r, s, inv_d, p.eps, red, 1);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = 8 * (at + GT * c);
    float v[8], w[8];
    unpack8(r[c], v);
    unpack8(nw[c], w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * k * w[i];
    if (col < p.d) store16(p.normed + row + col, pack8(v));
  }
}

// Sums over the tokens are kept by each thread for its columns over all rows of its group, joined
// over the block's groups in LDS, and written as one row of partial sums per block (which = 0
// dpre, 1 dpost, 2 dgate); join_norm_sums adds those in the blocks' order.  So the blocks are few
// and go on from row to row, the next row's loads on their way while one is worked on.
// Rows of one wave come in blocks of four waves, up to twice as many: a small batch spreads over more
// units (333 rows of 1000: 6.3 us from 8.8).
constexpr int back_threads(int wpr) { return wpr == 1 ? 256 : 512; }

template <int WPR, int C>
__global__ void __launch_bounds__(back_threads(WPR)) block_norms_backward_kernel(NormBackArgs p) {
  constexpr int GT = WPR * WAVE, ROWS = back_threads(WPR) / GT;
  extern __shared__ __align__(16) uint8_t lds[];
  float* red = reinterpret_cast<float*>(lds);           // [2][8 waves][4]
  float* sums = reinterpret_cast<float*>(lds) + 2 * 8 * 4;  // [ROWS - 1][columns], at the end
  const int at = threadIdx.x % GT, group = threadIdx.x / GT;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const float inv_d = 1.f / (float)p.d;
  const int64_t turns = ceil_div(p.T, (int64_t)gridDim.x * ROWS);

  uint4 nw[C], pw[C], gw[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = 8 * (at + GT * c);
    const bool in = col < p.d;
    nw[c] = in && p.pre ? load16(p.pre + col) : zero;
    pw[c] = in && p.post ? load16(p.post + col) : zero;
    gw[c] = in && p.gate && p.gate_stride == 0 ? load16(p.gate + col) : zero;
  }
  float apre[C][8], apost[C][8], agate[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) apre[c][i] = apost[c][i] = agate[c][i] = 0.f;

  uint4 dout[C], dn[C], y[C], r[C], g[C];
  auto load = [&](int64_t turn) {
    int64_t t = (turn * gridDim.x + blockIdx.x) * ROWS + group;
    if (t >= p.T) t = p.T - 1;  // read, and not used
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = 8 * (at + GT * c);
      const bool in = col < p.d;
      const int64_t e = t * p.d + col;
      dout[c] = in && p.dout ? load16(p.dout + e) : zero;
      dn[c] = in && p.dnormed ? load16(p.dnormed + e) : zero;
      r[c] = in && p.pre ? load16(p.out + e) : zero;
      y[c] = in && p.y ? load16(p.y + e) : zero;
      g[c] = in && p.gate && p.gate_stride ? load16(p.gate + e) : gw[c];
    }
  };
  load(0);
  for (int64_t turn = 0; turn < turns; ++turn) {
    const int64_t t = (turn * gridDim.x + blockIdx.x) * ROWS + group;
    const bool live = t < p.T;
    const int64_t row = t * p.d;
    uint4 cd[C], cn[C], cy[C], cr[C], cg[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      cd[c] = dout[c];
      cn[c] = dn[c];
      cy[c] = y[c];
      cr[c] = r[c];
      cg[c] = g[c];
    }
    if (turn + 1 < turns) load(turn + 1);
    float s[3] = {0.f, 0.f, 0.f};  // r^2, e r, y^2
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float a[8], b[8], w[8];
      if (p.pre) {
        unpack8(cr[c], a);
        unpack8(cn[c], b);
        unpack8(nw[c], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          s[0] += a[i] * a[i];
          s[1] += b[i] * w[i] * a[i];
        }
      }
      if (p.post) {
        unpack8(cy[c], a);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[2] += a[i] * a[i];
      }
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) s[i] = wave_sum_dpp(s[i]);
    int rr = p.pre ? range_of(s[0], p.eps) : IN, ry = p.post ? range_of(s[2], p.eps) : IN;
    if (rr != IN) {
      s[0] = wave_sum_dpp(scaled_sum<C>(cr, cr, nullptr, range_scale(rr), range_scale(rr)));
      s[1] = wave_sum_dpp(scaled_sum<C>(cn, cr, nw, 1.f, range_scale(rr)));
    }
    if (ry != IN) s[2] = wave_sum_dpp(scaled_sum<C>(cy, cy, nullptr, range_scale(ry), range_scale(ry)));
    row_statistics<WPR>(s, rr, ry, red, 0);
    if constexpr (C > 1) {  // not kept unpacked from above: past the branches there are no registers for it
#pragma unroll
      for (int c = 0; c < C; ++c) asm volatile("" : "+v"(cn[c].x), "+v"(cn[c].y), "+v"(cn[c].z), "+v"(cn[c].w));
    }
    const float ir = inverse_rms(s[0], rr, inv_d, p.eps);
    const float mean = s[1] * inv_d * (rr == IN ? ir : ir * range_scale(HIGH + LOW - rr)) * ir;  // mean(e rh) / rms(r)
    const float iy = p.post ? inverse_rms(s[2], ry, inv_d, p.eps) : 1.f;
    float f[C][8], q[1] = {0.f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = 8 * (at + GT * c);
      float G[8], a[8], b[8], w[8], gt[8];
      unpack8(cd[c], G);
      if (p.pre) {
        unpack8(cr[c], a);
        unpack8(cn[c], b);
        unpack8(nw[c], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float rh = a[i] * ir;
          G[i] += ir * (b[i] * w[i]) - rh * mean;
          if (live) apre[c][i] += b[i] * rh;
        }
      }
      if (live && col < p.d && p.dresidual) store16(p.dresidual + row + col, pack8(G));
      if (p.y) {
        unpack8(cy[c], a);
#pragma unroll
        for (int i = 0; i < 8; ++i) G[i] *= p.scale;
        if (p.post) {
          unpack8(pw[c], w);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = 1.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] *= iy;
        if (p.gate) {
          unpack8(cg[c], gt);
          float dg[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dg[i] = G[i] * (a[i] * w[i]);
            if (live) agate[c][i] += dg[i];
            G[i] *= gt[i];
          }
          if (p.gate_stride && p.dgate_rows && live && col < p.d) store16(p.dgate_rows + row + col, pack8(dg));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (live) apost[c][i] += G[i] * a[i];
          f[c][i] = G[i] * w[i];
          q[0] += f[c][i] * a[i];
        }
      }
    }
    if (p.y) {
      if (p.post) {
        row_sums<WPR>(q, red, 1);
        q[0] *= inv_d;
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int col = 8 * (at + GT * c);
        if (p.post) {
          float a[8];
          unpack8(cy[c], a);
#pragma unroll
          for (int i = 0; i < 8; ++i) f[c][i] = iy * (f[c][i] - a[i] * iy * q[0]);
        }
        if (live && col < p.d && p.dy) store16(p.dy + row + col, pack8(f[c]));
      }
    }
    if (WPR > 1 && !(p.y && p.post)) lds_barrier();  // one of the two places is read by all before it is written again
  }

  if (!p.part) return;
  auto join = [&](float (&acc)[C][8], int which) {
    if (!(p.sums >> which & 1)) return;
    lds_barrier();
    if (group > 0)
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float4*>(sums + ((group - 1) * C * GT + c * GT + at) * 8 + 4 * h) =
              make_float4(acc[c][4 * h], acc[c][4 * h + 1], acc[c][4 * h + 2], acc[c][4 * h + 3]);
    lds_barrier();
    if (group > 0) return;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = 8 * (at + GT * c);
      if (col >= p.d) continue;
      float* to = p.part + ((int64_t)which * gridDim.x + blockIdx.x) * p.d + col;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float4 v = make_float4(acc[c][4 * h], acc[c][4 * h + 1], acc[c][4 * h + 2], acc[c][4 * h + 3]);
        for (int o = 1; o < ROWS; ++o) {
          const float4 w = *reinterpret_cast<const float4*>(sums + ((o - 1) * C * GT + c * GT + at) * 8 + 4 * h);
          v.x += w.x;
          v.y += w.y;
          v.z += w.z;
          v.w += w.w;
        }
        *reinterpret_cast<float4*>(to + 4 * h) = v;
      }
    }
  };
  join(apre, 0);
  join(apost, 1);
  join(agate, 2);
}

// column sums of the blocks' rows: 16 slices of the rows a block, joined in their order
__global__ void __launch_bounds__(256) join_norm_sums(const float* __restrict__ part, int rows, int32_t d,
                                                      float* dpre, float* dpost, float* dgate) {
  __shared__ float4 sh[16][16];
  float* out = blockIdx.y == 0 ? dpre : blockIdx.y == 1 ? dpost : dgate;
  if (!out) return;
  const int x = threadIdx.x % 16, slice = threadIdx.x / 16;
  const int col = (blockIdx.x * 16 + x) * 4;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (col < d) {
    const float* p = part + (int64_t)blockIdx.y * rows * d + col;
    for (int r = slice; r < rows; r += 16) {
      const float4 w = *reinterpret_cast<const float4*>(p + (int64_t)r * d);
      v.x += w.x;
      v.y += w.y;
      v.z += w.z;
      v.w += w.w;
    }
  }
  sh[slice][x] = v;
  __syncthreads();
  if (slice == 0 && col < d) {
    for (int s = 1; s < 16; ++s) {
      const float4 w = sh[s][x];
      v.x += w.x;
      v.y += w.y;
      v.z += w.z;
      v.w += w.w;
    }
    *reinterpret_cast<float4*>(out + col) = v;
  }
}

// waves a row of the backward pass: two pieces of columns a thread, more do not fit its registers
// beside the three sums of each and the next row
int backward_waves(int32_t d) { return d <= 1024 ? 1 : d <= 4096 ? 4 : 8; }
int64_t backward_blocks(int64_t T, int32_t d) {
  const int w = backward_waves(d), most = 256 * 512 / back_threads(w);
  const int64_t n = ceil_div(T, back_threads(w) / (w * WAVE));
  return n < most ? n : most;
}

template <int WPR, int C>
hipError_t launch_forward(const NormArgs& a, hipStream_t st) {
  constexpr int64_t ROWS = 4 / WPR;
  hipError_t err = hipSuccess;
  for (int64_t t = 0; t < a.T && err == hipSuccess; t += LAUNCH_BLOCKS * ROWS) {
    NormArgs p = a;
    auto from = [&](auto* rows) { return rows ? rows + t * a.d : nullptr; };
    p.y = from(a.y);
    p.residual = from(a.residual);
    p.out = from(a.out);
    p.normed = from(a.normed);
    if (a.gate_stride) p.gate = from(a.gate);
    p.T = a.T - t < LAUNCH_BLOCKS * ROWS ? a.T - t : LAUNCH_BLOCKS * ROWS;
    hipLaunchKernelGGL((block_norms_kernel<WPR, C>), dim3((unsigned)ceil_div(p.T, ROWS)), dim3(256), 0, st, p);
    err = hipGetLastError();
  }
  return err;
}
template <int WPR, int C>
hipError_t launch_backward(const NormBackArgs& a, hipStream_t st) {
  constexpr int LDS = 2 * 8 * 4 * 4 + (back_threads(WPR) / (WPR * WAVE) - 1) * C * WPR * WAVE * 8 * 4;
  static_assert(LDS <= 65536, "no attribute needed");
  hipLaunchKernelGGL((block_norms_backward_kernel<WPR, C>), dim3((unsigned)backward_blocks(a.T, a.d)),
                     dim3(back_threads(WPR)), LDS, st, a);
  return hipGetLastError();
}

}  // namespace

size_t norms_backward_ws_bytes(int64_t T, int32_t d) { return (size_t)(3 * backward_blocks(T, d) * d) * 4; }

hipError_t launch_block_norms(const NormArgs& a, hipStream_t st) {
  const int c = (int)ceil_div(a.d, a.d <= 2048 ? 512 : 2048);
  if (a.d <= 2048) {
    switch (c) {
      case 1: return launch_forward<1, 1>(a, st);
      case 2: return launch_forward<1, 2>(a, st);
      case 3: return launch_forward<1, 3>(a, st);
      default: return launch_forward<1, 4>(a, st);
    }
  }
  switch (c) {
    case 2: return launch_forward<4, 2>(a, st);
    case 3: return launch_forward<4, 3>(a, st);
    default: return launch_forward<4, 4>(a, st);
  }
}

hipError_t launch_block_norms_backward(const NormBackArgs& a0, void* ws, hipStream_t st) {
  NormBackArgs a = a0;
  a.sums = (a.dpre ? 1 : 0) | (a.dpost ? 2 : 0) | (a.dgate ? 4 : 0);
  a.part = a.sums ? static_cast<float*>(ws) : nullptr;
  hipError_t err;
  if (a.d <= 512)
    err = launch_backward<1, 1>(a, st);
  else if (a.d <= 1024)
    err = launch_backward<1, 2>(a, st);
  else if (a.d <= 2048)
    err = launch_backward<4, 1>(a, st);
  else if (a.d <= 4096)
    err = launch_backward<4, 2>(a, st);
  else
    err = launch_backward<8, 2>(a, st);
  if (err != hipSuccess || !a.sums) return err;
  hipLaunchKernelGGL(join_norm_sums, dim3((unsigned)ceil_div(a.d, 64), 3), dim3(256), 0, st, a.part,
                     (int)backward_blocks(a.T, a.d), a.d, a.dpre, a.dpost, a.dgate);
  return hipGetLastError();
}

}  // namespace moe
