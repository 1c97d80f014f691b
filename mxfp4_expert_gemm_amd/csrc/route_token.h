// Router top-k with certified, exact selection: one token by one wavefront.
//
// The router picks the top-k of E experts per token (kimi-k3-mlx digest,
// architecture table: top-16 of 896) and its weights are probabilities renormalised
// over the kept experts (same digest, REAP section).  The selection is defined on
// the correctly rounded fp32 logit of the exact bf16 dot product, plus the bias in
// one fp32 add, ordered by (logit descending, expert index ascending).
//
// The fast logits come with a per-logit error radius r_e = gamma |x_t| |w_e| plus
// rounding padding, so the exact biased logit lies in [c_e - r_e, c_e + r_e].  With
// S the k best by centre, M = min over S of the lower ends and m = max over the rest
// of the upper ends: if M > m the set is certain.  Otherwise an expert whose lower
// end exceeds m is certainly in, one whose upper end is below M certainly out, and
// the ambiguous rest A (lo <= m, hi >= M) is recomputed exactly and ranked.
//
// Exact recompute of one logit: the wave sums the exact fp64 products with a
// rigorous error bound; when both ends of the bound round to the same fp32 that is
// the correctly rounded value.  Otherwise the products are accumulated exactly in a
// fixed-point integer (least significant bit 2^-266, 20 signed 64-bit digits of 32
// bits in LDS, updated with 64-bit LDS atomics, so the order of additions cannot
// matter) and rounded to nearest even once.
#pragma once

#include "common.h"
#include "kernels.h"

namespace moe {

constexpr int ROUTE_MAXI = 16;  // experts per lane: E <= 1024
constexpr int KDIG = 20;
constexpr int KLSB = 266;

struct WaveScratch {
  unsigned long long acc[KDIG];
  int special;  // bit 0 NaN, bit 1 +inf, bit 2 -inf
};

// ---- ordering: larger value first, NaN last, ties to the lower index
__device__ __forceinline__ bool ranks_before(double va, int ia, double vb, int ib) {
  bool na = va != va, nb = vb != vb;
  if (na != nb) return nb;
  if (!na && va != vb) return va > vb;
  return ia < ib;
}

__device__ __forceinline__ void wave_best(double& v, int& i) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    double ov = __shfl_xor(v, o);
    int oi = __shfl_xor(i, o);
    if (ranks_before(ov, oi, v, i)) {
      v = ov;
      i = oi;
    }
  }
}

__device__ __forceinline__ double wave_min_d(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmin(v, __shfl_xor(v, o));
  return v;
}
__device__ __forceinline__ double wave_max_d(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmax(v, __shfl_xor(v, o));
  return v;
}

// ---- exact dot product of two bf16 rows, correctly rounded to fp32

__device__ __forceinline__ void kulisch_add(WaveScratch* ws, uint32_t a, uint32_t b) {
  uint32_t sa = a >> 15, sb = b >> 15;
  uint32_t ea = (a >> 7) & 0xFFu, eb = (b >> 7) & 0xFFu;
  uint32_t fa = a & 0x7Fu, fb = b & 0x7Fu;
  bool a_nan = ea == 255 && fa, b_nan = eb == 255 && fb;
  bool a_inf = ea == 255 && !fa, b_inf = eb == 255 && !fb;
  bool a_zero = ea == 0 && !fa, b_zero = eb == 0 && !fb;
  if (a_nan || b_nan || (a_inf && b_zero) || (b_inf && a_zero)) {
    atomicOr(&ws->special, 1);
    return;
  }
  if (a_inf || b_inf) {
    atomicOr(&ws->special, (sa ^ sb) ? 4 : 2);
    return;
  }
  if (a_zero || b_zero) return;
  uint64_t ma = ea ? 128u + fa : fa, mb = eb ? 128u + fb : fb;
  int qa = ea ? (int)ea - 134 : -133, qb = eb ? (int)eb - 134 : -133;
  int o = qa + qb + KLSB;
  uint64_t v = (ma * mb) << (o & 31);
  uint64_t lo = v & 0xFFFFFFFFull, hi = v >> 32;
  if (sa ^ sb) {
    lo = 0ull - lo;
    hi = 0ull - hi;
  }
  atomicAdd(&ws->acc[o >> 5], lo);
  if (hi) atomicAdd(&ws->acc[(o >> 5) + 1], hi);
}

// digits (signed, lazy carries) -> correctly rounded fp32; run by one lane
__device__ __forceinline__ float kulisch_round(const WaveScratch* ws) {
  if ((ws->special & 1) || (ws->special & 6) == 6) return __uint_as_float(0x7FC00000u);
  if (ws->special & 2) return __uint_as_float(0x7F800000u);
  if (ws->special & 4) return __uint_as_float(0xFF800000u);
  uint32_t dig[KDIG];
  long long carry = 0;
  for (int i = 0; i < KDIG; ++i) {
    long long v = (long long)ws->acc[i] + carry;
    dig[i] = (uint32_t)v;
    carry = (v - (long long)dig[i]) >> 32;  // exact: a multiple of 2^32
  }
  bool neg = carry < 0;
  if (neg) {
    uint64_t c = 1;
    for (int i = 0; i < KDIG; ++i) {
      uint64_t v = (uint64_t)(~dig[i]) + c;
      dig[i] = (uint32_t)v;
      c = v >> 32;
    }
  }
  int top = -1;
  for (int i = KDIG - 1; i >= 0 && top < 0; --i)
    if (dig[i]) top = 32 * i + 31 - __clz(dig[i]);
  if (top < 0) return 0.f;
  int lsb = top - 23;
  if (lsb < KLSB - 149) lsb = KLSB - 149;  // fp32 subnormal spacing 2^-149
  auto bit = [&](int i) -> uint32_t { return i < 0 ? 0u : (dig[i >> 5] >> (i & 31)) & 1u; };
  uint32_t mant = 0;
  for (int i = top; i >= lsb; --i) mant = (mant << 1) | bit(i);
  uint32_t rb = bit(lsb - 1);
  bool sticky = false;
  for (int i = lsb - 2; i >= 0 && !sticky; --i) sticky = bit(i);
  if (rb && (sticky || (mant & 1u))) mant += 1;
  float r = ldexpf((float)mant, lsb - KLSB);
  return neg ? -r : r;
}

__device__ __forceinline__ float exact_dot_wave(const uint16_t* __restrict__ x, const uint16_t* __restrict__ w, int d,
                                WaveScratch* ws, int32_t* stats) {
  const int lane = lane_id();
  double s = 0.0, sa = 0.0;
  int nterm = 0;
  // EXU chunks of 8 products per lane are loaded before any is used, so the row costs
  // d / (8 WAVE EXU) memory round trips (two at d = 7168) rather than one per chunk
  constexpr int EXU = 7;
  const int nch = d / 8;
  for (int c0 = lane; c0 < nch; c0 += WAVE * EXU) {
    uint4 xv[EXU], wv[EXU];
#pragma unroll
    for (int u = 0; u < EXU; ++u) {
      const int c = c0 + WAVE * u;
      if (c < nch) {
        xv[u] = *reinterpret_cast<const uint4*>(x + 8 * c);
        wv[u] = *reinterpret_cast<const uint4*>(w + 8 * c);
      } else {
        xv[u] = wv[u] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
#pragma unroll
    for (int u = 0; u < EXU; ++u) {
      if (c0 + WAVE * u >= nch) continue;
      uint32_t xs[4] = {xv[u].x, xv[u].y, xv[u].z, xv[u].w}, wsv[4] = {wv[u].x, wv[u].y, wv[u].z, wv[u].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        double p0 = (double)bf16lo(xs[q]) * (double)bf16lo(wsv[q]);
        double p1 = (double)bf16hi(xs[q]) * (double)bf16hi(wsv[q]);
        s += p0;
        s += p1;
        sa += fabs(p0);
        sa += fabs(p1);
      }
      nterm += 8;
    }
  }
  s = wave_sum(s);
  sa = wave_sum(sa);
  int nmax = __shfl(nterm, 0);  // lane 0 has the most terms
  // each lane: nterm additions; tree: 6 more; products are exact in fp64
  double err = (double)(nmax + 8) * 0x1p-53 * sa * (1.0 + 0x1p-40) + 0x1p-1022;
  if (__builtin_isfinite(s) && __builtin_isfinite(sa)) {
    double e2 = err + 0x1p-52 * fabs(s);
    float lo = (float)(s - e2), hi = (float)(s + e2);
    if (lo == hi && __builtin_signbit(lo) == __builtin_signbit(hi)) return lo;  // a zero of unknown sign goes on
  }
  // fixed-point fallback
  if (stats && lane == 0) atomicAdd(&stats[2], 1);
  if (lane < KDIG) ws->acc[lane] = 0ull;
  if (lane == 0) ws->special = 0;
  __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
  __builtin_amdgcn_wave_barrier();
  for (int c = lane; c < d / 8; c += WAVE) {
    uint4 xv = *reinterpret_cast<const uint4*>(x + 8 * c);
    uint4 wv = *reinterpret_cast<const uint4*>(w + 8 * c);
    uint32_t xs[4] = {xv.x, xv.y, xv.z, xv.w}, wsv[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      kulisch_add(ws, xs[q] & 0xFFFFu, wsv[q] & 0xFFFFu);
      kulisch_add(ws, xs[q] >> 16, wsv[q] >> 16);
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
  __builtin_amdgcn_wave_barrier();
  float r = 0.f;
  if (lane == 0) r = kulisch_round(ws);
  return __shfl(r, 0);
}

// ---- selection by keys

// neighbouring floats (finite inputs; the infinities stay put)
__device__ __forceinline__ float next_down(float f) {
  if (f != f || f == -__builtin_inff()) return f;
  if (f == 0.f) return -__uint_as_float(1u);
  uint32_t u = __float_as_uint(f);
  return __uint_as_float(f > 0.f ? u - 1u : u + 1u);
}
__device__ __forceinline__ float next_up(float f) { return -next_down(-f); }

// order-preserving 32-bit key of a float: larger value -> larger key; -0 == +0;
// NaN maps to 1, below every number (every number's key is >= 0x007FFFFF); 0 is
// reserved for "not a candidate".
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 1u;
  uint32_t u = __float_as_uint(v == 0.f ? 0.f : v);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Marks in `sel` the kk largest keys of the wave (ties to the lower expert index,
// e = 64 i + lane).  Keys of 0 are never taken when at least kk keys are nonzero.
// Radix select on the key bits with ballot counts: no cross-lane data movement.
__device__ __forceinline__ uint32_t select_top(const uint32_t (&key)[ROUTE_MAXI], int kk) {
  uint32_t tau = 0;
  for (int b = 31; b >= 0; --b) {
    const uint32_t cand = tau | (1u << b);
    int cnt = 0;
#pragma unroll
    for (int i = 0; i < ROUTE_MAXI; ++i) cnt += __popcll(__ballot(key[i] >= cand));
    if (cnt >= kk) tau = cand;
  }
  uint32_t sel = 0;
  int need = kk;
#pragma unroll
  for (int i = 0; i < ROUTE_MAXI; ++i) {
    const bool gt = key[i] > tau;
    need -= __popcll(__ballot(gt));
    if (gt) sel |= 1u << i;
  }
  const int lane = lane_id();
#pragma unroll
  for (int i = 0; i < ROUTE_MAXI; ++i) {
    unsigned long long m = __ballot(key[i] == tau && tau != 0u);
    unsigned long long take = 0;
    while (need > 0 && m) {
      unsigned long long low = m & (0ull - m);
      take |= low;
      m ^= low;
      --need;
    }
    if ((take >> lane) & 1ull) sel |= 1u << i;
  }
  return sel;
}

// ---- routing of one token by one wave


// Per-wave LDS of the routing: Kulisch digits, the candidate list of the fast path and
// the selected (expert, logit) pairs in output order.
constexpr int ROUTE_CAND = WAVE;
struct RouteLds {
  WaveScratch ks;
  uint32_t ckey[ROUTE_CAND];
  int cidx[ROUTE_CAND];
  float cval[ROUTE_CAND], crad[ROUTE_CAND];
  alignas(16) int oidx[WAVE];
  float oval[WAVE];
};

// Writes idx/w of token t from the k selected (expert, logit) pairs in L->oidx/oval,
// ascending expert order.  Renormalised weights: softmax over the k logits (max and a
// fixed DPP tree, the same in every path).  Otherwise: over all E logits, whose
// max and sum over experts the caller passes in.
__device__ __forceinline__ void emit_topk(const RouteArgs& a, int64_t t, const RouteLds* L, float mx_all,
                                          float den_all) {
  const int lane = lane_id(), k = a.k;
  const bool mine = lane < k;
  const float v = mine ? L->oval[lane] : -__builtin_inff();
  float mx = mx_all, den = den_all;
  float ex;
  if (a.renormalize) {
    mx = wave_max_dpp(v);
    ex = mine ? expf(v - mx) : 0.f;
    den = wave_sum_dpp(ex);
  } else {
    ex = expf(v - mx);
  }
  if (mine) {
    a.idx[t * k + lane] = L->oidx[lane];
    a.w[t * k + lane] = ex / den;
  }
}

// max and sum of exp(v - max) over all experts of the lane arrays (softmax over E)
__device__ __forceinline__ void softmax_all(const float (&val)[ROUTE_MAXI], int E, float& mx, float& den) {
  const int lane = lane_id();
  mx = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < ROUTE_MAXI; ++i)
    if (i * WAVE + lane < E) mx = fmaxf(mx, val[i]);
  mx = wave_max_dpp(mx);
  den = 0.f;
#pragma unroll
  for (int i = 0; i < ROUTE_MAXI; ++i)
    if (i * WAVE + lane < E) den += expf(val[i] - mx);
  den = wave_sum_dpp(den);
}

// General path: selection over every expert by radix select on the keys, certification,
// exact recompute of the ambiguous logits.  Kept out of line: it runs only when the
// fast path below cannot decide (many ties, an uncertain boundary, MOE_ROUTE_EXACT_ALL).
__device__ __forceinline__ void route_token_general(const RouteArgs& a, int64_t t, RouteLds* L) {
  const int lane = lane_id();
  const int E = a.E, k = a.k;
  const bool topk_mode = a.exact_logits != nullptr;
  float val[ROUTE_MAXI];      // logit used for weights and export (exact where recomputed)
  float lo[ROUTE_MAXI], hi[ROUTE_MAXI];
  uint32_t key[ROUTE_MAXI];
  const double xn = topk_mode ? 0.0 : (double)a.xnorm[t];
  const double abs_pad = (double)a.d * 0x1p-125;
#pragma unroll
  for (int i = 0; i < ROUTE_MAXI; ++i) {
    const int e = i * WAVE + lane;
    val[i] = -__builtin_inff();
    lo[i] = -__builtin_inff();
    hi[i] = -__builtin_inff();
    key[i] = 0u;
    if (e < E) {
      if (topk_mode) {
        val[i] = a.exact_logits[t * E + e];
        key[i] = order_key(val[i]);
      } else {
        const float lf = a.logits_fast[t * E + e];
        const float b = a.bias ? a.bias[t * a.bias_stride + e] : 0.f;
        val[i] = lf + b;  // the fast biased logit, one fp32 rounding
        const double r = a.gamma * xn * (double)a.wnorm[e] * (1.0 + 0x1p-20) + abs_pad +
                         0x1p-21 * ((double)fabsf(lf) + (double)fabsf(b));
        const double c = (double)lf + (double)b;
        if (b == -__builtin_inff() && __builtin_isfinite(lf) && __builtin_isfinite(r) &&
            fabs((double)lf) + r < 0x1.fffffep127) {
          // a bias of -inf (an expert pruned away): the exact logit is finite, so the
          // biased logit is exactly -inf and never needs recomputing
          val[i] = lo[i] = hi[i] = -__builtin_inff();
          key[i] = order_key(-__builtin_inff());
        } else if (__builtin_isfinite(lf) && __builtin_isfinite(b) && __builtin_isfinite(r)) {
          // outward-rounded fp32 ends of the interval holding the exact biased logit
          float l32 = (float)(c - r), h32 = (float)(c + r);
          if ((double)l32 > c - r) l32 = next_down(l32);
          if ((double)h32 < c + r) h32 = next_up(h32);
          lo[i] = l32;
          hi[i] = h32;
          key[i] = order_key((float)c);
        } else {  // unknown: must be recomputed if it can matter
          lo[i] = -__builtin_inff();
          hi[i] = __builtin_inff();
          key[i] = order_key(-__builtin_inff());
        }
      }
    }
  }

  uint32_t sel = select_top(key, k);
  if (!topk_mode) {
    float mloc = -__builtin_inff(), Mloc = __builtin_inff();
#pragma unroll
    for (int i = 0; i < ROUTE_MAXI; ++i) {
      const int e = i * WAVE + lane;
      if (e < E) {
        if ((sel >> i) & 1u) Mloc = fminf(Mloc, lo[i]);
        else mloc = fmaxf(mloc, hi[i]);
      }
    }
    const float M = wave_min_dpp(Mloc), m = wave_max_dpp(mloc);
    const bool all = (a.flags & MOE_ROUTE_EXACT_ALL) != 0;
    if (all || (k < E && !(M > m))) {
      // amb: undecided experts, ranked below on exact values; known: those among them
      // whose interval is a point (a pruned expert's exact -inf), already in val
      uint32_t amb = 0, cin = 0, known = 0;
#pragma unroll
      for (int i = 0; i < ROUTE_MAXI; ++i) {
        const int e = i * WAVE + lane;
        if (e < E) {
          if (all) amb |= 1u << i;
          else if (((sel >> i) & 1u) && lo[i] > m) cin |= 1u << i;
          else if (lo[i] <= m && hi[i] >= M) {
            amb |= 1u << i;
            if (lo[i] == hi[i]) known |= 1u << i;
          }
        }
      }
      int n_in = 0, n_amb = 0;
#pragma unroll
      for (int i = 0; i < ROUTE_MAXI; ++i) {
        n_in += __popcll(__ballot((cin >> i) & 1u));
        unsigned long long bal = __ballot(((amb & ~known) >> i) & 1u);
        n_amb += __popcll(bal);
        while (bal) {
          const int l = __ffsll((long long)bal) - 1;
          bal &= bal - 1;
          const int e = i * WAVE + l;
          float v = exact_dot_wave(a.x + t * a.d, a.router_w + (int64_t)e * a.d, a.d, &L->ks, a.stats);
          if (a.bias) v = v + a.bias[t * a.bias_stride + e];
          if (lane == l) val[i] = v;
        }
      }
      if (a.stats && lane == 0) {
        atomicAdd(&a.stats[0], 1);
        atomicAdd(&a.stats[1], n_amb);
      }
      uint32_t ekey[ROUTE_MAXI];
#pragma unroll
      for (int i = 0; i < ROUTE_MAXI; ++i) ekey[i] = ((amb >> i) & 1u) ? order_key(val[i]) : 0u;
      sel = cin | select_top(ekey, k - n_in);
    }
  }

  // selected pairs in ascending expert order, then the weights
  int base = 0;
#pragma unroll
  for (int i = 0; i < ROUTE_MAXI; ++i) {
    const unsigned long long bal = __ballot((sel >> i) & 1u);
    if ((sel >> i) & 1u) {
      const int pos = base + __popcll(bal & ((1ull << lane) - 1ull));
      L->oidx[pos] = i * WAVE + lane;
      L->oval[pos] = val[i];
    }
    base += __popcll(bal);
    const int e = i * WAVE + lane;
    if (a.logits_out && e < E) a.logits_out[t * E + e] = val[i];
  }
  float mx_all = 0.f, den_all = 1.f;
  if (!a.renormalize) softmax_all(val, E, mx_all, den_all);
  __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
  __builtin_amdgcn_wave_barrier();
  emit_topk(a, t, L, mx_all, den_all);
}

// k-th largest of one key per lane (radix select with ballots), k <= WAVE
__device__ __forceinline__ uint32_t kth_of_lanes(uint32_t v, int k) {
  uint32_t tau = 0;
  for (int b = 31; b >= 0; --b) {
    const uint32_t cand = tau | (1u << b);
    if (__popcll(__ballot(v >= cand)) >= k) tau = cand;
  }
  return tau;
}

// Routing of token t (fills idx/w, ascending ids, and optionally logits_out).
//
// Fast path.  The keys of the fast biased logits c_e are cut at tau, the k-th largest
// of the 64 per-lane maxima: at least k keys reach tau, so the k best are among the
// candidates (key >= tau), usually a few dozen.  The candidates are ranked against
// each other, one per lane, and the selection is certified as in the general path
// with fp32 interval ends: radius R_e = gamma' |x||w_e| + pad' + 2^-20 (|lf| + |b|),
// with gamma' = gamma (1 + 2^-18) and pad' = d 2^-124, covers the radius of the
// general path plus the roundings of c_e = lf + b and of R_e itself (a few ulp of
// 2^-24 each), and the ends c - R and c + R are pushed one ulp outwards.  More than 64
// candidates or an uncertified boundary go to the general path, which starts over.
__device__ __forceinline__ void route_token(const RouteArgs& a, int64_t t, RouteLds* L) {
  const int lane = lane_id();
  const int E = a.E, k = a.k;
  const bool topk_mode = a.exact_logits != nullptr;
  if (a.flags & MOE_ROUTE_EXACT_ALL) {
    route_token_general(a, t, L);
    return;
  }
  float c[ROUTE_MAXI], R[ROUTE_MAXI];
  uint32_t key[ROUTE_MAXI];
  const float xn = topk_mode ? 0.f : a.xnorm[t];
  const float gam = (float)a.gamma * (1.f + 0x1p-18f) * xn;
  const float pad = (float)a.d * 0x1p-124f;
  // every load unconditional and from a pointer chosen once (lanes past E read the last
  // expert and are masked after; a missing operand reads the logits and is not used), so
  // no branch splits them and all are in flight together: one memory round trip
  const float* pl = (topk_mode ? a.exact_logits : a.logits_fast) + t * E;
  const bool has_bias = !topk_mode && a.bias != nullptr;
  const float* pb = has_bias ? a.bias + t * a.bias_stride : pl;
  const float* pw = topk_mode ? pl : a.wnorm;
  float lf[ROUTE_MAXI], bv[ROUTE_MAXI], wn[ROUTE_MAXI];
#pragma unroll
  for (int i = 0; i < ROUTE_MAXI; ++i) {
    const int e = i * WAVE + lane < E ? i * WAVE + lane : E - 1;
    lf[i] = pl[e];
    bv[i] = pb[e];
    wn[i] = pw[e];
  }
#pragma unroll
  for (int i = 0; i < ROUTE_MAXI; ++i) bv[i] = has_bias ? bv[i] : 0.f;
  uint32_t kmax = 0;
#pragma unroll
  for (int i = 0; i < ROUTE_MAXI; ++i) {
    const int e = i * WAVE + lane;
    c[i] = -__builtin_inff();
    R[i] = 0.f;
    key[i] = 0u;
    if (e < E) {
      if (topk_mode) {
        c[i] = lf[i];
      } else {
        c[i] = lf[i] + bv[i];
        R[i] = gam * wn[i] + pad + 0x1p-20f * (fabsf(lf[i]) + fabsf(bv[i]));
        if (bv[i] == -__builtin_inff()) {
          // pruned expert (bias -inf): exactly -inf when the exact logit is finite, which
          // the radius shows; else unknown
          const float rr = gam * wn[i] + pad + 0x1p-20f * fabsf(lf[i]);
          const bool known = __builtin_isfinite(lf[i]) && __builtin_isfinite(rr) && fabsf(lf[i]) + rr < 0x1p127f;
          c[i] = -__builtin_inff();
          R[i] = known ? 0.f : __builtin_inff();
        } else if (!(__builtin_isfinite(c[i]) && __builtin_isfinite(R[i]))) {
          c[i] = -__builtin_inff();  // unknown: the general path recomputes it if it can matter
          R[i] = __builtin_inff();
        }
      }
      key[i] = order_key(c[i]);
      kmax = key[i] > kmax ? key[i] : kmax;
    }
  }
  const uint32_t tau = kth_of_lanes(kmax, k);
  // candidates: keys >= tau, compacted in (lane, i) order
  int mine = 0;
#pragma unroll
  for (int i = 0; i < ROUTE_MAXI; ++i) mine += (key[i] != 0u && key[i] >= tau);
  int n_c = 0;
  int pos = wave_excl_scan(mine, n_c);
  if (n_c > ROUTE_CAND) {
    route_token_general(a, t, L);
    return;
  }
#pragma unroll
  for (int i = 0; i < ROUTE_MAXI; ++i)
    if (key[i] != 0u && key[i] >= tau) {
      L->ckey[pos] = key[i];
      L->cidx[pos] = i * WAVE + lane;
      L->cval[pos] = c[i];
      L->crad[pos] = R[i];
      ++pos;
    }
  __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
  __builtin_amdgcn_wave_barrier();
  // rank of this lane's candidate: (key descending, expert ascending)
  const bool live = lane < n_c;
  const uint32_t mk = live ? L->ckey[lane] : 0u;
  const int me = live ? L->cidx[lane] : 0x7FFFFFFF;
  int rank = 0;
  for (int j = 0; j < n_c; ++j) {  // register broadcasts: no memory round trip per step
    const uint32_t kj = (uint32_t)__builtin_amdgcn_readlane((int)mk, j);
    const int ej = __builtin_amdgcn_readlane(me, j);
    rank += (kj > mk) || (kj == mk && ej < me);
  }
  const bool sel = live && rank < k;
  const float mc = live ? L->cval[lane] : 0.f, mr = live ? L->crad[lane] : 0.f;
  if (!topk_mode && k < E) {
    // certification: min lower end over the selected, max upper end over the rest
    float Mloc = __builtin_inff(), mloc = -__builtin_inff();
    if (sel) Mloc = mr == __builtin_inff() ? -__builtin_inff() : next_down(mc - mr);
    if (live && !sel) mloc = mr == __builtin_inff() ? __builtin_inff() : next_up(mc + mr);
#pragma unroll
    for (int i = 0; i < ROUTE_MAXI; ++i)
      if (key[i] != 0u && key[i] < tau) mloc = fmaxf(mloc, R[i] == __builtin_inff() ? __builtin_inff() : next_up(c[i] + R[i]));
    const float M = wave_min_dpp(Mloc), m = wave_max_dpp(mloc);
    if (!(M > m)) {
      route_token_general(a, t, L);
      return;
    }
  }
  // output order: ascending expert id among the selected
  int op = 0;
  for (unsigned long long sm = __ballot(sel); sm; sm &= sm - 1)
    op += __builtin_amdgcn_readlane(me, __ffsll((long long)sm) - 1) < me;
  if (sel) {
    L->oidx[op] = me;
    L->oval[op] = mc;
  }
  if (a.logits_out) {
#pragma unroll
    for (int i = 0; i < ROUTE_MAXI; ++i) {
      const int e = i * WAVE + lane;
      if (e < E) a.logits_out[t * E + e] = c[i];
    }
  }
  float mx_all = 0.f, den_all = 1.f;
  if (!a.renormalize) softmax_all(c, E, mx_all, den_all);
  __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
  __builtin_amdgcn_wave_barrier();
  emit_topk(a, t, L, mx_all, den_all);
}

}  // namespace moe
