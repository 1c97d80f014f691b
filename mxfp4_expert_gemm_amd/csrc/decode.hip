// The layer for the few tokens of a decode step, in two launches: the router logits and the
// latent rows h (dense_gemv_kernel), then everything behind them in one grid.
//
// A decode step of a few tokens reads a few hundred MB once, so its time is the HBM's plus
// what each launch costs on the way: its first loads' latency, its last blocks' drain, and
// the routing, during which nothing streams.  Here one block per CU goes through the phases
//   route      every block routes all tokens for itself and quantises h into its LDS: no
//              block waits for another's selection;
//   gate / up  16 FFN rows of one routed expert for its tokens, a wave each; two of them make a
//              scale block of the down operand, which the later one quantises;
//   down       16 latent rows of up to 16 routed rows, a block each, with the combine where
//              that is all of them (else the block that finishes a group of rows combines);
//   up         a share of the output rows per block, whose weights are under way long
//              before: some into the LDS as the routing ends, some into registers while the
//              last gate / up items finish.
//
// Progress.  A block claims gate / up chunks and down items when it is about to work on them,
// and waits only for items of earlier phases, which it does when all of them are claimed, by
// blocks that run and wait for still earlier phases at most.  Nothing waits for up rows, which
// are dealt out in advance.  So the grid drains however many of its blocks are resident at a
// time, beside whatever else the GPU runs.
//
// Counters.  2048 atomic additions to one address take 23 us here (11 ns each, at the memory
// side, since the XCDs' L2s are not shared), to 32 addresses 1 us: an item counter is 32
// shards on lines of their own (item 32 j + s is the j-th of shard s, and a claimer whose shard
// is spent looks for another that has some left), and completion is counted per expert
// and per row group.  What one wave hands to another is written through to the memory side
// (agent-scope stores), and, where it is counted, waited for before; the reader's loads are
// agent-scope too.  A hand-over takes 0.8 us.  z and the adapters' u need no count: their
// words start as all ones, which none of them can be (a NaN is written as 0x7FC0 or
// 0x7FC00000), and a reader asks again until a word is another.  The launch
// before sets counters and words.
// That a relaxed agent-scope store has reached the memory side once vmcnt is zero, that later
// additions are seen behind it, and that a load issued after a polled value came back reads no
// older data, is how this chip works and what the order of the instructions here relies on.  The
// language's memory model would ask for release and acquire, which write back and invalidate a
// whole L2 each.
//
// Measured (7168-wide tokens, latent 3584, FFN 3072, 16 of 896 experts; packed experts but where
// records are named).  One token reads 397 MB in 86.3 us, 4.6 TB/s: 12.7 us the first launch;
// in the second the routing and the first chunk end at 10.5, a block's gate / up at 40 in the
// median and 53 at the latest, its down at 63 and 69, z is there at 71, and the up rows, which
// are on chip by then, take 3.  The first 10 us and the last 5 stream little, the blocks' spread
// at the two hand-overs costs as much again: that is what bounds it.  Against the five launches
// of moe_layer_forward, in graphs of 50 steps on experts of their own, here / there in us:
//   tokens                    1           2           3           4
//   packed experts         90.1 / 85.4  153 / 145   212 / 203   263 / 244
//   checkpoint records      122 / 119   200 / 211   285 / 305   351 / 376
// and eight MXFP8 tokens of a middle layer (2048, 1024, 512, 8 of 64, packed) 53.6 / 57.5, one
// token of it 30.4 / 24.0, four of a tiny layer over records 27.4 / 27.3, one over packed experts
// 22.5 / 21.3.  So it is for records, for many rows of few experts, and where five launches
// cost the host more than the card; several blocks a CU, which cover one another's spread, are
// worth more than three launches where the packed streams set the pace.
// Slower: a wave per down item; the latent rows and the routing in this launch too; more steps in
// flight per stream; counters without shards (one token 125 us).
//
// The arithmetic of every value is that of the kernels moe_layer_forward runs on a batch of
// this size (dense_gemv_kernel, the routing, stream_group, the fp64 combine), in the same
// order: the outputs are bit-identical.
#include "decode_chunks.h"
#include "mfma_stream.h"
#include "route_token.h"

namespace moe {

constexpr int DEC_THREADS = 512;
constexpr int DEC_WAVES = DEC_THREADS / WAVE;
constexpr int DEC_GU_PF = 4;   // K steps in flight, of a gate and an up stream
constexpr int DEC_DN_PF = 8;   // of a down stream
constexpr int DEC_SLOTS = 2 * DEC_WAVES;  // routed rows of a down item: two a wave
constexpr int DEC_SHARDS = 32;
constexpr int DEC_MAX_DIM = 7168;  // of latent and FFN
static_assert(DECODE_MAX_ROWS * (DEC_MAX_DIM / 32) < 0xFFFF, "pairs and chunks fit the halves of a GateUpPlan head");
static_assert(DECODE_MAX_TOKENS <= DEC_WAVES && DECODE_MAX_ROWS <= WAVE, "a wave per token, a lane per routed row");

// a staged activation row: hi codes, lo codes, hi scales, lo scales
__host__ __device__ constexpr int dec_row_bytes(int K) { return (2 * K + K / 16 + 15) / 16 * 16; }
__device__ __forceinline__ ALds dec_row(uint8_t* row, int K) { return {row, row + K, row + 2 * K, row + 2 * K + K / 32}; }

// ---- counters, each on a 128-byte line of its own
enum {
  C_GATEUP = 0,                         // claimed items, by shard
  C_DOWN = C_GATEUP + DEC_SHARDS,
  C_U = C_DOWN + DEC_SHARDS,
  C_EXPERT = C_U + DEC_SHARDS,          // quantised gate / up scale blocks, by expert
  C_ROWS = C_EXPERT + DECODE_MAX_ROWS   // finished down items, by row group
};
int32_t decode_counters(int32_t L) { return C_ROWS + L / 16; }
__device__ __forceinline__ int32_t* line(int32_t* ctr, int i) { return ctr + 32 * i; }

template <class V>
__device__ __forceinline__ void put(V* p, V v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <class V>
__device__ __forceinline__ V get(const V* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ int add1(int32_t* p) {
  return __hip_atomic_fetch_add(p, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// the wave's stores so far have reached the memory side
__device__ __forceinline__ void stores_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// words that are still to come
__device__ __forceinline__ bool missing16(unsigned long long v) {  // a 16-bit lane is all ones
  const unsigned long long t = ~v;
  return ((t - 0x0001000100010001ull) & ~t & 0x8000800080008000ull) != 0ull;
}
// A wait for another block, or for a tile, ends after so many polls (a few seconds) too, and with
// it every later one of the block: only a call that shares its workspace with one that overlaps
// it can wait for what never comes, and it then ends, with NaN outputs, instead of holding
// the GPU.  (The other waits in a block are for a wave that is claiming, which waits for
// nothing itself, and for wave 0's next down item, which it claims behind waits of this kind at
// most.)
constexpr int DEC_POLLS = 1 << 22;
template <class F>
__device__ __forceinline__ bool wait_for(int* late, F&& there) {
  for (int n = 0; !there(); ++n) {
    if (n == DEC_POLLS) __hip_atomic_store(late, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    if (__hip_atomic_load(late, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP)) return false;
    __builtin_amdgcn_s_sleep(2);
  }
  return true;
}
__device__ __forceinline__ unsigned long long await16(int* late, const uint16_t* p) {  // NaN where it is late
  unsigned long long v;
  wait_for(late, [&] { return !missing16(v = get(reinterpret_cast<const unsigned long long*>(p))); });
  return v;
}
__device__ __forceinline__ uint32_t await32(int* late, const uint32_t* p) {
  uint32_t v;
  wait_for(late, [&] { return (v = get(p)) != 0xFFFFFFFFu; });
  return v;
}

// Claims of one phase's n items by a wave.  take() sends the request for the wave's next item
// early; item() waits for it and is -1 when no item is left.
struct Claims {
  int32_t* ctr;
  int n, shard, asked;
  __device__ __forceinline__ Claims(int32_t* base, int n_) : ctr(base), n(n_), shard(blockIdx.x % DEC_SHARDS), asked(0) {}
  __device__ __forceinline__ void take() {
    if (lane_id() == 0) asked = add1(line(ctr, shard));
  }
  __device__ __forceinline__ int item() {
    for (;;) {
      const int i = DEC_SHARDS * __builtin_amdgcn_readfirstlane(asked) + shard;
      if (i < n) return i;
      const int lane = lane_id();
      const int at = lane < DEC_SHARDS ? (lane + shard) % DEC_SHARDS : 0;
      const int used = lane < DEC_SHARDS ? get(line(ctr, at)) : n;
      const unsigned long long left = __ballot(lane < DEC_SHARDS && DEC_SHARDS * used + at < n);
      if (!left) return -1;
      shard = (__ffsll((long long)left) - 1 + shard) % DEC_SHARDS;
      take();
    }
  }
};

// A weight stream as mfma_stream.h's, its addresses a wave-uniform base and a lane's 32-bit
// offset: a step then costs scalar additions only.  The vector instructions per step are what
// binds the down phase (1 KB of weights a step and stream) once loads are far enough ahead.
struct DecW {
  const uint8_t* c;  // codes
  const uint8_t* s;  // scales
};
template <class W>
struct DecLane;
template <>
struct DecLane<PackedW> {
  uint32_t oc, os;
  int nsc;
  static constexpr int SIDE = 1;
  __device__ __forceinline__ DecLane(int K, int lane) : oc(16 * lane), os(4 * lane), nsc((K / 128 + 3) / 4) {}
  // 16 rows `grp` of matrix `mat` of expert e
  __device__ __forceinline__ static DecW make(const uint8_t* blob, int e, int L, int F, int mat, int grp) {
    const PackedW w = PackedW::make(blob, e, L, F, mat, grp, 0);
    return {w.c, w.s};
  }
  __device__ __forceinline__ uint4 load(const DecW& w, int ks) const { return load_nt16(w.c + 1024 * ks + oc); }
  __device__ __forceinline__ void sblock(const DecW& w, SBlock& b, int blk) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 4 * blk + i;
      const uint32_t v = *reinterpret_cast<const uint32_t*>(w.s + 256 * (t < nsc ? t : nsc - 1) + os);
      b.d[i] = t < nsc ? v : 0x7F7F7F7Fu;
    }
  }
  template <int J>
  __device__ __forceinline__ uint32_t scale(const SBlock& b) const {
    return b.d[J >> 2];
  }
};
template <>
struct DecLane<RecordW> {
  uint32_t oc, os;
  int nsb, n, g;
  // a record's row gives 64 bytes a step: two steps' loads side by side read whole 128-byte lines
  static constexpr int SIDE = 2;
  __device__ __forceinline__ DecLane(int K, int lane)
      : oc((lane & 15) * (K / 2) + 16 * (lane >> 4)), os((lane & 15) * (K / 32)), nsb(K / 32), n(lane & 15), g(lane >> 4) {}
  __device__ __forceinline__ static DecW make(const uint8_t* blob, int e, int L, int F, int mat, int grp) {
    const RecordW w = RecordW::make(blob, e, L, F, mat, grp, 0);
    return {w.c, w.s};
  }
  __device__ __forceinline__ uint4 load(const DecW& w, int ks) const { return load_nt16(w.c + 64 * ks + oc); }
  __device__ __forceinline__ void sblock(const DecW& w, SBlock& b, int blk) const {
    const int off = 64 * blk + 16 * g;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int o = off + 4 * i;
      const uint32_t v = *reinterpret_cast<const uint32_t*>(w.s + os + (uint32_t)(o < nsb ? o : nsb - 4));
      b.d[i] = o < nsb ? v : 0x7F7F7F7Fu;
    }
  }
  template <int J>
  __device__ __forceinline__ uint32_t scale(const SBlock& b) const {
    return (uint32_t)__shfl((int)b.d[J & 3], n + 16 * (J >> 2)) >> (8 * g);
  }
};
template <int NS, int PF, class Ln>
__device__ __forceinline__ void dec_prime(const Ln& ln, const DecW (&w)[NS], SBlock (&sb)[NS], uint4 (&ring)[NS][PF],
                                          int nks) {
#pragma unroll
  for (int q = 0; q < NS; ++q) ln.sblock(w[q], sb[q], 0);
#pragma unroll
  for (int d = 0; d < PF; ++d)
#pragma unroll
    for (int q = 0; q < NS; ++q) ring[q][d] = ln.load(w[q], d < nks ? d : nks - 1);
}

// The activation operand of a lane: its tile row in the LDS, from 16 g on, or, for a row the
// tile does not have, zeros that do not move on (DEC_ZEROS bytes of them: 16 K steps and the
// second half of one), so that no step asks which it is.
constexpr int DEC_ZEROS = 16 * 128 + 80;
struct DecA {
  const uint8_t *hi, *lo, *shi, *slo;
  int on;
  __device__ __forceinline__ DecA(bool on_, uint8_t* row, const uint8_t* zeros, int K, int g) : on(on_) {
    hi = on_ ? row + 16 * g : zeros;
    lo = on_ ? row + K + 16 * g : zeros;
    shi = on_ ? row + 2 * K + g : zeros;
    slo = on_ ? row + 2 * K + K / 32 + g : zeros;
  }
  __device__ __forceinline__ void advance() {  // by 16 K steps
    hi += on ? 16 * 128 : 0;
    lo += on ? 16 * 128 : 0;
    shi += on ? 16 * 4 : 0;
    slo += on ? 16 * 4 : 0;
  }
  template <int J>
  __device__ __forceinline__ void read(AStep& a) const {
    const uint4 h0 = *reinterpret_cast<const uint4*>(hi + 128 * J), h1 = *reinterpret_cast<const uint4*>(hi + 128 * J + 64);
    const uint4 l0 = *reinterpret_cast<const uint4*>(lo + 128 * J), l1 = *reinterpret_cast<const uint4*>(lo + 128 * J + 64);
    a.hi[0] = (int)h0.x; a.hi[1] = (int)h0.y; a.hi[2] = (int)h0.z; a.hi[3] = (int)h0.w;
    a.hi[4] = (int)h1.x; a.hi[5] = (int)h1.y; a.hi[6] = (int)h1.z; a.hi[7] = (int)h1.w;
    a.lo[0] = (int)l0.x; a.lo[1] = (int)l0.y; a.lo[2] = (int)l0.z; a.lo[3] = (int)l0.w;
    a.lo[4] = (int)l1.x; a.lo[5] = (int)l1.y; a.lo[6] = (int)l1.z; a.lo[7] = (int)l1.w;
    a.shi = shi[4 * J];
    a.slo = slo[4 * J];
  }
};

// stream_group with NS weight streams on one activation row group: acc[q] += A W_q^T over all K
// steps, sb and ring filled by dec_prime.  With `chain` the ring goes on with the first
// steps of wn as w's loads end, and wn's scales are in sb after, as dec_prime would leave
// them (K / 128 a multiple of PF, so that the ring's slots fit).
template <class W, int NS, int PF>
__device__ __forceinline__ void dec_stream(const DecLane<W>& ln, const DecW (&w)[NS], const DecW (&wn)[NS], bool chain,
                                           SBlock (&sb)[NS], uint4 (&ring)[NS][PF], DecA ad, int K, f32x4 (&acc)[NS]) {
  constexpr int SIDE = DecLane<W>::SIDE;
  const int nks = K / 128, nc = (nks + 15) / 16;
  SBlock sbn[NS];
  for (int c = 0; c < nc; ++c) {
#pragma unroll
    for (int q = 0; q < NS; ++q) {
      const bool next = chain && c + 1 == nc;
      ln.sblock(next ? wn[q] : w[q], sbn[q], next ? 0 : c + 1 < nc ? c + 1 : c);
    }
    unroll_n<16 / SIDE>([&](auto jc) {
      constexpr int J2 = SIDE * decltype(jc)::value;
      const int ks2 = 16 * c + J2;
      uint4 cw[SIDE][NS];
#pragma unroll
      for (int q = 0; q < NS; ++q)
#pragma unroll
        for (int h = 0; h < SIDE; ++h) {
          cw[h][q] = ring[q][(J2 + h) % PF];
          // every step loads, on every path (see prime_stream): past w's steps, those of wn
          // that the ring's slot is for, or w's last again
          const int at = ks2 + h + PF;
          const bool next = chain && at >= nks;
          ring[q][(J2 + h) % PF] = ln.load(next ? wn[q] : w[q], next ? (at - nks) % PF : at < nks ? at : nks - 1);
        }
      unroll_n<SIDE>([&](auto hc) {
        constexpr int H = decltype(hc)::value, J = J2 + H;
        const int ks = ks2 + H;
        if (ks < nks) {
          AStep a;
          ad.template read<J>(a);
#pragma unroll
          for (int q = 0; q < NS; ++q) {
            const uint32_t sw = ln.template scale<J>(sb[q]);
            const i32x8 b = as_b(cw[H][q]);
            acc[q] = mx_mfma<W::opsel(J)>(a.hi, b, acc[q], a.shi, sw);
            acc[q] = mx_mfma<W::opsel(J)>(a.lo, b, acc[q], a.slo, sw);
          }
        }
      });
    });
    ad.advance();
#pragma unroll
    for (int q = 0; q < NS; ++q) sb[q] = sbn[q];
  }
}

struct DecodeLds {
  union {
    RouteLds route[DECODE_MAX_TOKENS];  // candidates and output of a token
    unsigned long long slots[ROUTE_MAXI * WAVE];  // of an expert, while they are grouped
    struct {
      uint16_t tile[DEC_TILES][DECODE_MAX_TOKENS][34];  // GLU outputs of a pair of items
      float ys[2][DEC_SLOTS][16];                       // expert outputs of a down item, by slot
    };
  };
  alignas(16) uint8_t zeros[DEC_ZEROS];
  uint32_t gmax[DEC_WAVES][WAVE];
  int wcnt[DEC_WAVES][16];
  float wup[DEC_WAVES];
  uint8_t crank[DECODE_MAX_TOKENS][ROUTE_CAND];
  uint32_t redo;               // tokens whose selection the block could not decide
  // the routing
  int sel[DECODE_MAX_ROWS];    // expert of slot t k + j
  float w[DECODE_MAX_ROWS];    // its weight
  int sgrp[DECODE_MAX_ROWS];   // its group: the distinct experts, and the slots of each
  int gexp[DECODE_MAX_ROWS];
  int gn[DECODE_MAX_ROWS];
  uint8_t gslot[DECODE_MAX_ROWS][DECODE_MAX_TOKENS];
  int ng;
  int late;  // a wait was given up
  unsigned long long chunk;  // the block's gate / up chunk, a word of GateUpPlan
  int tile_of[DEC_TILES], tile_n[DEC_TILES];  // the pair a tile is for, items of it there
  unsigned long long ditem[2];  // (sequence + 1) << 32 | down item, as wave 0 learns of it
};
constexpr size_t DEC_LDS = (160 * 1024 - sizeof(DecodeLds)) / 1024 * 1024;  // what is left for the launch to size

// route_token as a call: its registers are not reserved in the kernel, where it runs only
// when the block's own selection cannot decide
__attribute__((noinline)) __device__ void dec_route_alone(RouteArgs a, int64_t t, RouteLds* L) { route_token(a, t, L); }

// Routing of all tokens at once, W = 16 / EPT waves a token and EPT experts a lane: the values,
// cut, certification and output of route_token's fast path (see there).  What it cannot
// decide is left to route_token (S.redo).  load() brings a token's logits, select() works on
// them; every wave of the block calls both.
template <int EPT>
struct RouteBlock {
  static constexpr int W = 16 / EPT;
  float lf[EPT], bv[EPT], wn[EPT], xn;

  __device__ __forceinline__ static int expert(int i) { return (i * W + (threadIdx.x / WAVE) % W) * WAVE + lane_id(); }
  __device__ __forceinline__ void load(const RouteArgs& a) {
    const int t = min((int)threadIdx.x / WAVE / W, (int)a.T - 1);
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      const int e = min(expert(i), a.E - 1);
      lf[i] = a.logits_fast[(int64_t)t * a.E + e];
      bv[i] = a.bias ? a.bias[t * a.bias_stride + e] : 0.f;
      wn[i] = a.wnorm[e];
    }
    xn = a.xnorm[t];
  }
  __device__ __forceinline__ void select(const RouteArgs& a, DecodeLds& S) const {
    const int lane = lane_id(), wave = threadIdx.x / WAVE, t = wave / W, sub = wave % W;
    const int E = a.E, k = a.k;
    const bool token = t < a.T;
    RouteLds& L = S.route[token ? t : 0];
    const float gam = (float)a.gamma * (1.f + 0x1p-18f) * xn;
    const float pad = (float)a.d * 0x1p-124f;
    float c[EPT], R[EPT];
    uint32_t key[EPT], kmax = 0u;
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      c[i] = -__builtin_inff();
      R[i] = 0.f;
      key[i] = 0u;
      if (expert(i) < E) {
        c[i] = lf[i] + bv[i];
        R[i] = gam * wn[i] + pad + 0x1p-20f * (fabsf(lf[i]) + fabsf(bv[i]));
        if (bv[i] == -__builtin_inff()) {
          const float rr = gam * wn[i] + pad + 0x1p-20f * fabsf(lf[i]);
          const bool known = __builtin_isfinite(lf[i]) && __builtin_isfinite(rr) && fabsf(lf[i]) + rr < 0x1p127f;
          c[i] = -__builtin_inff();
          R[i] = known ? 0.f : __builtin_inff();
        } else if (!(__builtin_isfinite(c[i]) && __builtin_isfinite(R[i]))) {
          c[i] = -__builtin_inff();
          R[i] = __builtin_inff();
        }
        key[i] = order_key(c[i]);
        kmax = max(kmax, key[i]);
      }
    }
    S.gmax[wave][lane] = kmax;
    lds_barrier();
    // the cut: the k-th largest of the maxima of 64 groups (experts equal mod 64)
    uint32_t gm = 0u;
#pragma unroll
    for (int v = 0; v < W; ++v) gm = max(gm, S.gmax[wave - sub + v][lane]);
    const uint32_t tau = kth_of_lanes(gm, k);
    unsigned long long cb[EPT];
    float up = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      const bool cand = key[i] != 0u && key[i] >= tau;
      cb[i] = __ballot(cand);
      if (key[i] != 0u && !cand) up = fmaxf(up, R[i] == __builtin_inff() ? __builtin_inff() : next_up(c[i] + R[i]));
      if (lane == 0) S.wcnt[wave - sub][i * W + sub] = __popcll(cb[i]);
    }
    up = wave_max_dpp(up);
    if (lane == 0) S.wup[wave] = up;
    lds_barrier();
    int base[EPT], n_c = 0;
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int n = S.wcnt[wave - sub][v];
      if (v % W == sub) base[v / W] = n_c;
      n_c += n;
    }
    const bool fits = n_c <= ROUTE_CAND;
    if (token && fits)
#pragma unroll
      for (int i = 0; i < EPT; ++i)
        if ((cb[i] >> lane) & 1ull) {
          const int pos = base[i] + __popcll(cb[i] & ((1ull << lane) - 1ull));
          L.ckey[pos] = key[i];
          L.cidx[pos] = expert(i);
          L.cval[pos] = c[i];
          L.crad[pos] = R[i];
        }
    lds_barrier();
    if (token && fits) {  // a candidate's rank: those ahead of it are counted
      constexpr int PER = ROUTE_CAND / W;
      const bool live = lane < n_c;
      const uint32_t mk = live ? L.ckey[lane] : 0u;
      const int me = live ? L.cidx[lane] : 0x7FFFFFFF;
      for (int i = PER * sub; i < min(PER * sub + PER, n_c); ++i) {
        const uint32_t ki = (uint32_t)__builtin_amdgcn_readlane((int)mk, i);
        const int ei = __builtin_amdgcn_readlane(me, i);
        const int r = __popcll(__ballot(live && (mk > ki || (mk == ki && me < ei))));
        if (lane == 0) S.crank[t][i] = (uint8_t)r;
      }
    }
    lds_barrier();
    if (token && sub == 0) {
      bool fast = fits && a.renormalize && !(a.flags & MOE_ROUTE_EXACT_ALL);
      const bool live = fast && lane < n_c;
      const bool sel = live && S.crank[t][lane] < k;
      const float mc = live ? L.cval[lane] : 0.f, mr = live ? L.crad[lane] : 0.f;
      if (fast && k < E) {
        float Mloc = __builtin_inff(), mloc = -__builtin_inff();
        if (sel) Mloc = mr == __builtin_inff() ? -__builtin_inff() : next_down(mc - mr);
        if (live && !sel) mloc = mr == __builtin_inff() ? __builtin_inff() : next_up(mc + mr);
        if (lane < W) mloc = fmaxf(mloc, S.wup[wave + lane]);
        fast = wave_min_dpp(Mloc) > wave_max_dpp(mloc);
      }
      if (fast) {
        // candidates are in expert order, so the output place is the count of selected below
        const int op = __popcll(__ballot(sel) & ((1ull << lane) - 1ull));
        if (sel) {
          L.oidx[op] = L.cidx[lane];
          L.oval[op] = mc;
        }
        wave_sync();
        emit_topk(a, t, &L, 0.f, 1.f);
      } else if (lane == 0) {
        atomicOr(&S.redo, 1u << t);
      }
    }
    if (token && a.logits_out) {  // a redo overwrites what it recomputes
#pragma unroll
      for (int i = 0; i < EPT; ++i)
        if (expert(i) < E) a.logits_out[(int64_t)t * E + expert(i)] = c[i];
    }
  }
};

// Routing of all tokens into S, and h quantised into hq, by the whole block; the first block
// also writes what the caller asked for.  ahead() starts loads that the end of the routing
// hides; before() takes what is still on its way (a wait for an older load, afterwards, would
// wait for those too).
template <int EPT, class Fb, class Fn>
__device__ __forceinline__ void dec_route(const DecodeArgs& p, const RouteArgs& a, DecodeLds& S, uint8_t* hq,
                                          Fb&& before, Fn&& ahead) {
  const int tid = threadIdx.x;
  const int T = (int)a.T, L = a.L;
  RouteBlock<EPT> rb;
  rb.load(a);
  constexpr int U = 2;  // groups of eight latent values a thread has in flight
  const int per = L / 8, groups = T * per;
  uint4 raw[U];
  auto load_h = [&](int j0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + DEC_THREADS * u;
      if (DEC_THREADS * u < groups) raw[u] = *reinterpret_cast<const uint4*>(a.h + 8 * (int64_t)(j < groups ? j : 0));
    }
  };
  load_h(tid);
  for (int j0 = tid; j0 < groups; j0 += DEC_THREADS * U) {
    if (j0 != tid) load_h(j0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + DEC_THREADS * u;
      if (j < groups) {  // the four groups of a scale block are a quad of lanes
        const int t = j / per, jj = j - t * per;
        const ALds r = dec_row(hq + t * dec_row_bytes(L), L);
        const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[2 * i] = bf16lo(w[i]);
          v[2 * i + 1] = bf16hi(w[i]);
        }
        uint32_t hi[2], lo[2], shi, slo;
        quantize_quad8_fmt(v, hi, lo, shi, slo, a.mxfp8 != 0);
        *reinterpret_cast<uint2*>(r.hi + 8 * jj) = make_uint2(hi[0], hi[1]);
        *reinterpret_cast<uint2*>(r.lo + 8 * jj) = make_uint2(lo[0], lo[1]);
        if ((jj & 3) == 0) {
          r.shi[jj >> 2] = (uint8_t)shi;
          r.slo[jj >> 2] = (uint8_t)slo;
        }
      }
    }
  }
  rb.select(a, S);
  before();
  ahead();  // by most waves while few certify
}

// the selection's groups, the caller's routing outputs and the first gate / up chunk
__device__ __forceinline__ void dec_group(const DecodeArgs& p, const RouteArgs& a, DecodeLds& S) {
  const int tid = threadIdx.x, lane = lane_id(), wave = tid / WAVE;
  const int T = (int)a.T, k = a.k, n = T * k;
  const bool writer = blockIdx.x == 0;
  lds_barrier();  // loads that ahead() started stay in flight
  const uint32_t redo = S.redo;
  if (redo) {
    if (wave < T && (redo >> wave) & 1u) dec_route_alone(a, wave, &S.route[wave]);
    __syncthreads();
  }
  if (wave == 0) {
    const int e = lane < n ? S.sel[lane] : -1;
    if (T == 1) {  // a token's experts are distinct
      if (lane < n) {
        S.sgrp[lane] = lane;
        S.gexp[lane] = e;
        S.gn[lane] = 1;
        S.gslot[lane][0] = (uint8_t)lane;
      }
      if (lane == 0) S.ng = n;
    } else {  // a lane per slot: the first slot of an expert leads its group
      unsigned long long mine = 0;
      if (e >= 0) S.slots[e] = 0ull;
      wave_sync();
      if (e >= 0) atomicOr(&S.slots[e], 1ull << lane);
      wave_sync();
      if (e >= 0) mine = S.slots[e];
      const unsigned long long below = (1ull << lane) - 1ull;
      const bool lead = e >= 0 && (mine & below) == 0ull;
      const unsigned long long leads = __ballot(lead);
      if (e >= 0) {
        const int first = __ffsll((long long)mine) - 1;
        const int grp = __popcll(leads & ((1ull << first) - 1ull));
        S.sgrp[lane] = grp;
        S.gslot[grp][__popcll(mine & below)] = (uint8_t)lane;
        if (lead) {
          S.gexp[grp] = e;
          S.gn[grp] = __popcll(mine);
        }
      }
      if (lane == 0) S.ng = __popcll(leads);
    }
    if (writer && lane < n) {
      if (p.idx) p.idx[lane] = e;
      if (p.w) p.w[lane] = S.w[lane];
      if (p.perm) {
        int at = 0;
        for (int s = 0; s < n; ++s) at += S.sel[s] < e || (S.sel[s] == e && s < lane);
        p.perm[at] = lane;
      }
    }
  } else if (wave == 1 && lane < DEC_TILES) {
    S.tile_of[lane] = lane;
    S.tile_n[lane] = 0;
  }
  if (writer && (p.counts || p.offsets))
    for (int e = tid; e <= a.E; e += DEC_THREADS) {
      int below = 0, same = 0;
      for (int s = 0; s < n; ++s) {
        below += S.sel[s] < e;
        same += S.sel[s] == e;
      }
      if (p.counts && e < a.E) p.counts[e] = same;
      if (p.offsets) p.offsets[e] = below;
    }
}

// ranks of token t's adapter in use, and its id
__device__ __forceinline__ int dec_rank(const LoraSeg& l, int t, int& a) {
  a = l.adapter[t];
  if ((uint32_t)a >= (uint32_t)l.N) return 0;
  return l.rank ? min(l.rank[a], l.R) : l.R;
}

// UC chunks of 512 latent columns cover an up row; a wave holds UA of them through the down
// phase.
// ONE: one token.  Its phases run a few hundred instructions each and are met cold, so the code
// for more tokens (the up phase's four at a time) costs it 2 us by its place alone: 87.7 us as a
// kernel of its own against 89.9 (L 3584, packed), and nothing either way for two to eight.
template <class W, int UC, int UA, bool ONE>
__global__ void __launch_bounds__(DEC_THREADS) decode_kernel(DecodeArgs p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ DecodeLds S;
  const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
  const int nl = lane & 15, g = lane >> 4;
  const int T = ONE ? 1 : (int)p.r.T, k = p.r.k, L = p.r.L, F = p.F, d = p.r.d;
  const int hrow = dec_row_bytes(L), arow = dec_row_bytes(F);
  uint8_t* stage = smem + p.stage_offset + wave * arow;

  // the block's up rows: the first slab_rows wait in the LDS, the others are taken by the
  // waves in turn
  const int up0 = min(d, (int)blockIdx.x * p.up_rows), up1 = min(d, up0 + p.up_rows);
  const int slab1 = min(up1, up0 + p.slab_rows);
  uint16_t* slab = reinterpret_cast<uint16_t*>(smem + p.slab_offset);

  // ---- routing; the first claims are on their way meanwhile (wave 0's)
  Claims chunks(line(p.ctr, C_GATEUP), 0), downs(line(p.ctr, C_DOWN), 0);
  if (wave == 0) {
    chunks.take();
    downs.take();
  }
  RouteArgs ra = p.r;
  ra.idx = S.sel;
  ra.w = S.w;
  if (blockIdx.x != 0) ra.logits_out = nullptr;
  if (tid == 0) {  // read behind barriers
    S.redo = 0u;
    S.late = 0;
  }
  for (int i = tid; i < DEC_ZEROS / 4; i += DEC_THREADS) reinterpret_cast<uint32_t*>(S.zeros)[i] = 0u;
  auto ahead = [&]() {
    const int bytes = (slab1 - up0) * L * 2;
    for (int i = 1024 * wave; i < bytes; i += 1024 * DEC_WAVES)
      if (i + 16 * lane < bytes)
        lds_dma16(reinterpret_cast<const uint8_t*>(p.latent_up + (int64_t)up0 * L) + i + 16 * lane,
                  reinterpret_cast<const uint8_t*>(slab) + i);
  };
  auto before = [&]() { asm volatile("" ::"v"(chunks.asked), "v"(downs.asked)); };
  if (T == 1) dec_route<2>(p, ra, S, smem, before, ahead);
  else if (T == 2) dec_route<4>(p, ra, S, smem, before, ahead);
  else if (T <= 4) dec_route<8>(p, ra, S, smem, before, ahead);
  else dec_route<16>(p, ra, S, smem, before, ahead);
  dec_group(p, ra, S);
  if (wave == 0) wave_sync();
  lds_barrier();
  const int nrb = F / 32;
  const GateUpPlan plan(S.ng * nrb, (int)gridDim.x, DEC_WAVES);
  chunks.n = plan.n;
  const int nrg = L / 16, nsc = (T * k + DEC_SLOTS - 1) / DEC_SLOTS;
  downs.n = nrg * nsc;
  if (wave == 0) {
    const int c = chunks.item(), dn = downs.item();
    if (lane == 0) {
      S.chunk = (unsigned long long)GateUpPlan::first(c) << 32;
      S.ditem[0] = 1ull << 32 | (uint32_t)dn;
      S.ditem[1] = 0ull;
    }
  }
  lds_barrier();

  // ---- gate / up
  struct Half {
    int pair, seq, h;  // pair of the phase, of the block; which of its two items
  };
  auto next_half = [&](Half& x) -> bool {
    for (;;) {
      unsigned long long v = 0;
      if (lane == 0) v = atomicAdd(&S.chunk, 1ull);
      const uint32_t head = (uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32));
      const ChunkPlace at = plan.place(head, (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v));
      if (at.what == ChunkPlace::NONE) return false;
      if (at.what == ChunkPlace::ITEM) {
        x.pair = at.pair;
        x.seq = at.seq;
        x.h = at.half;
        return true;
      }
      if (at.what == ChunkPlace::NEXT) {
        chunks.take();
        const uint32_t next = plan.next(head, chunks.item());
        if (lane == 0)
          __hip_atomic_store(&S.chunk, (unsigned long long)next << 32, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
      } else {
        __builtin_amdgcn_s_sleep(1);
      }
    }
  };
  {
    DecW w[2], wn[2];
    SBlock sb[2];
    uint4 ring[2][DEC_GU_PF];
    const DecLane<W> ln(L, lane);
    const bool fit = (L / 128) % DEC_GU_PF == 0;
    auto make = [&](DecW(&m)[2], const Half& x) {
      const int grp = x.pair / nrb, r = 2 * (x.pair - grp * nrb) + x.h, e = __builtin_amdgcn_readfirstlane(S.gexp[grp]);
      m[0] = ln.make(p.blob, e, L, F, MAT_GATE, r);
      m[1] = ln.make(p.blob, e, L, F, MAT_UP, r);
    };
    Half x, y;
    bool more = next_half(x);
    if (more) {
      make(w, x);
      dec_prime(ln, w, sb, ring, L / 128);
    }
    while (more) {
      const int grp = x.pair / nrb, rb = x.pair - grp * nrb, nt = __builtin_amdgcn_readfirstlane(S.gn[grp]);
      const bool again = next_half(y);
      if (again) make(wn, y);
      else {
        wn[0] = w[0];
        wn[1] = w[1];
      }
      const bool on = nl < nt;
      f32x4 acc[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) acc[q] = f32x4{0.f, 0.f, 0.f, 0.f};
      dec_stream<W, 2, DEC_GU_PF>(ln, w, wn, again && fit, sb, ring,
                                  DecA(on, smem + (on ? S.gslot[grp][nl] / k : 0) * hrow, S.zeros, L, g), L, acc);
      if (again && !fit) dec_prime(ln, wn, sb, ring, L / 128);
      // lane: row nl of the item, tokens 4 g + j of the expert
      const int ti = x.seq % DEC_TILES;
      // the pair 16 before this one is complete; given up, the pair is not counted, and the rows
      // that need it become NaN
      const bool open = wait_for(&S.late, [&] {
        return __hip_atomic_load(&S.tile_of[ti], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP) == x.seq;
      });
      if (!__builtin_amdgcn_readfirstlane(open)) break;
      uint16_t(*at)[34] = S.tile[ti];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (4 * g + j < nt) at[4 * g + j][16 * x.h + nl] = glu_bf16(acc[0][j], acc[1][j]);
      wave_sync();
      int there = 0;
      if (lane == 0) there = atomicAdd(&S.tile_n[ti], 1);
      if (__builtin_amdgcn_readfirstlane(there) == 1) {
        wave_sync();
        // the pair is whole: a quad of lanes per token, eight of its 32 values each
        const int m = lane >> 2, sub = lane & 3;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = m < nt ? bf16f(at[m][8 * sub + i]) : 0.f;
        uint32_t hi[2], lo[2], shi, slo;
        quantize_quad8_fmt(v, hi, lo, shi, slo, p.r.mxfp8 != 0);
        if (m < nt) {
          const ALds o = dec_row(p.aq + (int64_t)S.gslot[grp][m] * arow, F);
          put(reinterpret_cast<unsigned long long*>(o.hi + 32 * rb + 8 * sub), (unsigned long long)hi[1] << 32 | hi[0]);
          put(reinterpret_cast<unsigned long long*>(o.lo + 32 * rb + 8 * sub), (unsigned long long)lo[1] << 32 | lo[0]);
          if (sub == 0) {
            put(o.shi + rb, (uint8_t)shi);
            put(o.slo + rb, (uint8_t)slo);
          }
        }
        wave_sync();
        if (lane == 0) {  // the tile is the 16th next pair's
          S.tile_n[ti] = 0;
          __hip_atomic_store(&S.tile_of[ti], x.seq + DEC_TILES, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_WORKGROUP);
        }
        stores_done();
        if (lane == 0) add1(line(p.ctr, C_EXPERT + grp));
      }
      more = again;
      x = y;
      w[0] = wn[0];
      w[1] = wn[1];
    }
  }
  if (p.stage_offset == 0) __syncthreads();  // the staged rows take the place of h

  // ---- down and combine
  uint4 wr[UA][UC];
  auto load_up = [&](int row, int r) {  // row of the matrix into wr[r]
    row = max(0, min(row, up1 - 1));
#pragma unroll
    for (int q = 0; q < UC; ++q) {
      const int col = 8 * (WAVE * q + lane);
      wr[r][q] = load_nt16(p.latent_up + (int64_t)row * L + (col < L ? col : 0));
    }
  };
  {
    const int n = T * k;
    DecW w[1], wn[1];
    SBlock sb[1];
    uint4 ring[1][DEC_DN_PF];
    const DecLane<W> ln(F, lane);
    const bool fit = (F / 128) % DEC_DN_PF == 0;
    // the block's seq-th item: wave 0 has claimed it and says so in the LDS
    auto item_of = [&](int seq) -> int {
      for (;;) {
        const unsigned long long v = __hip_atomic_load(&S.ditem[seq & 1], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        if (__builtin_amdgcn_readfirstlane((int)(v >> 32)) == seq + 1) return __builtin_amdgcn_readfirstlane((int)(uint32_t)v);
        __builtin_amdgcn_s_sleep(1);
      }
    };
    auto slot_of = [&](int item) { return item < 0 ? n : DEC_SLOTS * (item / nrg) + wave; };
    auto make = [&](int item, int s) {
      return ln.make(p.blob, __builtin_amdgcn_readfirstlane(S.sel[s]), L, F, MAT_DOWN, item % nrg);
    };
    int ditem = item_of(0), s = slot_of(ditem);
    if (s < n) {
      w[0] = make(ditem, s);
      dec_prime(ln, w, sb, ring, F / 128);
    }
#pragma unroll
    for (int r = 0; r < UA; ++r) load_up(slab1 + wave + DEC_WAVES * r, r);
    for (int seq = 0; ditem >= 0; ++seq) {
      const int rg = ditem % nrg;
      int nitem = -2;  // not asked yet
      while (s < n) {
        // the wave's next row: of this item, else of the block's next
        const bool second = s < DEC_SLOTS * (ditem / nrg) + DEC_WAVES && s + DEC_WAVES < n;
        if (!second) {
          if (wave == 0) {  // it has rows of every item; claimed no earlier, for a block that may be free by then
            downs.take();
            const int nx = downs.item();
            if (lane == 0)
              __hip_atomic_store(&S.ditem[(seq + 1) & 1], (unsigned long long)(seq + 2) << 32 | (uint32_t)nx,
                                 __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
          }
          nitem = item_of(seq + 1);
        }
        const int ns = second ? s + DEC_WAVES : slot_of(nitem);
        const bool again = ns < n;
        wn[0] = again ? make(second ? ditem : nitem, ns) : w[0];
        int32_t* ready = line(p.ctr, C_EXPERT + S.sgrp[s]);
        const bool there = wait_for(&S.late, [&] { return get(ready) >= nrb; });
        // the row by 8-byte agent-scope loads, SU of a lane in flight
        constexpr int SU = 13;
        const uint8_t* src = p.aq + (int64_t)s * arow;
        for (int i0 = 8 * lane; i0 < arow; i0 += 8 * WAVE * SU) {
          unsigned long long v[SU];
#pragma unroll
          for (int q = 0; q < SU; ++q) {
            const int i = i0 + 8 * WAVE * q;
            v[q] = get(reinterpret_cast<const unsigned long long*>(src + (i < arow ? i : 0)));
          }
#pragma unroll
          for (int q = 0; q < SU; ++q) {
            const int i = i0 + 8 * WAVE * q;
            if (i < arow) *reinterpret_cast<unsigned long long*>(stage + i) = v[q];
          }
        }
        wave_sync();
        f32x4 acc[1] = {f32x4{0.f, 0.f, 0.f, 0.f}};
        dec_stream<W, 1, DEC_DN_PF>(ln, w, wn, again && fit, sb, ring, DecA(nl == 0, stage, S.zeros, F, g), F, acc);
        if (again && !fit) dec_prime(ln, wn, sb, ring, F / 128);
        if (!there) acc[0][0] = __builtin_nanf("");
        if (g == 0) {
          if (nsc == 1) S.ys[seq & 1][s][nl] = acc[0][0];
          else put(p.y + (int64_t)s * L + 16 * rg + nl, acc[0][0]);
        }
        wave_sync();  // the next row may overwrite this one
        w[0] = wn[0];
        s = ns;
        if (!second) break;
      }
      if (nsc > 1) stores_done();
      if (nitem == -2) {  // no row of this item was the wave's
        nitem = item_of(seq + 1);
        s = slot_of(nitem);
        if (s < n) {
          w[0] = make(nitem, s);
          dec_prime(ln, w, sb, ring, F / 128);
        }
      }
      lds_barrier();
      if (wave == 0) {
        // z[t][l] = bf16(sum_j w[t][j] y[t k + j][l]) in slot order, in fp64, once every slot's
        // outputs of these rows are there
        int before = 0;
        if (nsc > 1 && lane == 0) before = add1(line(p.ctr, C_ROWS + rg));
        if (__builtin_amdgcn_readfirstlane(before) == nsc - 1) {
          for (int i = lane; i < T * 16; i += WAVE) {
            const int t = i / 16, r = i % 16;
            double acc = 0.0;
            constexpr int YU = 16;
            for (int j0 = 0; j0 < k; j0 += YU) {
              float v[YU];
#pragma unroll
              for (int u = 0; u < YU; ++u) {
                const int sl = t * k + min(j0 + u, k - 1);
                v[u] = nsc == 1 ? S.ys[seq & 1][sl][r] : get(p.y + (int64_t)sl * L + 16 * rg + r);
              }
#pragma unroll
              for (int u = 0; u < YU; ++u)
                if (j0 + u < k) acc += (double)S.w[t * k + j0 + u] * (double)v[u];
            }
            put(p.z + (int64_t)t * L + 16 * rg + r, f64_to_bf16(acc));
          }
        }
      }
      ditem = nitem;
    }
  }

  // ---- up (with the adapters' two products): every block holds all of z
  const bool lora = p.lora.B != nullptr;
  const int R = p.lora.R;
  Claims us(line(p.ctr, C_U), T * R);
  if (lora) us.take();
  stores_done();    // the slab's loads: behind the barriers every wave sees all of it
  lds_barrier();    // no wave reads its staged rows any more
  uint16_t* zs = reinterpret_cast<uint16_t*>(smem);
  float* ul = reinterpret_cast<float*>(smem + T * L * 2);                  // [T][R]
  uint16_t* bl = reinterpret_cast<uint16_t*>(ul + T * R);                 // [up row][T][R], where it fits
  const bool bfit = T * L * 2 + T * R * (4 + 2 * p.up_rows) <= p.slab_offset;
  int ui = -1;
  uint4 ua[UC];
  auto load_a = [&]() {  // a row of an adapter's first matrix, for (token, rank) pair ui
    ui = us.item();
    if (ui < 0) return;
    const int t = ui / R, r = ui - t * R;
    int a;
    const int rk = dec_rank(p.lora, t, a);
#pragma unroll
    for (int q = 0; q < UC; ++q) {
      const int col = 8 * (WAVE * q + lane);
      ua[q] = make_uint4(0u, 0u, 0u, 0u);
      if (r < rk && col < L) ua[q] = *reinterpret_cast<const uint4*>(p.lora_a + ((int64_t)a * R + r) * L + col);
    }
  };
  if (lora) {
    load_a();
    if (bfit)  // the rows of the second matrices, eight ranks a thread
      for (int i = tid; i < (up1 - up0) * T * (R / 8); i += DEC_THREADS) {
        const int row = i / (T * (R / 8)), t = i / (R / 8) % T, r = i % (R / 8) * 8;
        int a;
        const int rk = dec_rank(p.lora, t, a);
        if (r < rk)
          *reinterpret_cast<uint4*>(bl + (row * T + t) * R + r) =
              *reinterpret_cast<const uint4*>(p.lora.B + ((int64_t)a * d + up0 + row) * R + r);
      }
  }
  for (int i = 4 * tid; i < T * L; i += 4 * DEC_THREADS)
    *reinterpret_cast<unsigned long long*>(zs + i) = await16(&S.late, p.z + i);
  lds_barrier();
  if (lora) {
    while (ui >= 0) {
      us.take();
      const int t = ui / R, r = ui - t * R;
      int a;
      const int rk = dec_rank(p.lora, t, a);
      float v = 0.f;
      if (r < rk) {
        double acc = 0.0;
#pragma unroll
        for (int q = 0; q < UC; ++q) {
          const int col = 8 * (WAVE * q + lane);
          if (col < L) {
            const uint4 x = *reinterpret_cast<const uint4*>(zs + t * L + col);
            float s = dot2(x.x, ua[q].x, 0.f);
            s = dot2(x.y, ua[q].y, s);
            s = dot2(x.z, ua[q].z, s);
            s = dot2(x.w, ua[q].w, s);
            acc += (double)s;
          }
        }
        v = (float)(wave_sum_dpp(acc) * (double)p.lora_scale[a]);
      }
      // a NaN with a payload (a scale's) must not become the word that means "not there yet"
      if (lane == 0) put(p.u + ui, v != v ? 0x7FC00000u : __float_as_uint(v));
      load_a();
    }
    for (int i = tid; i < T * R; i += DEC_THREADS) ul[i] = __uint_as_float(await32(&S.late, p.u + i));
    lds_barrier();
  }
  // NR rows, DEC_WAVES apart, for every token, TP at a time: weights(r, q) is chunk q of the r-th
  auto rows_up = [&](int row0, int end, auto nr, auto tp, auto&& weights) {
    constexpr int NR = decltype(nr)::value, TP = decltype(tp)::value;
    for (int t0 = 0; t0 < T; t0 += TP) {
      double acc[NR * TP];
#pragma unroll
      for (int i = 0; i < NR * TP; ++i) acc[i] = 0.0;
#pragma unroll
      for (int q = 0; q < UC; ++q) {
        const int col = 8 * (WAVE * q + lane);
        if (col < L) {
          uint4 v[NR];
#pragma unroll
          for (int r = 0; r < NR; ++r) v[r] = weights(r, q);
#pragma unroll
          for (int t = 0; t < TP; ++t)
            if (TP == 1 || t0 + t < T) {
              const uint4 x = *reinterpret_cast<const uint4*>(zs + (t0 + t) * L + col);
#pragma unroll
              for (int r = 0; r < NR; ++r) {
                float s = dot2(x.x, v[r].x, 0.f);
                s = dot2(x.y, v[r].y, s);
                s = dot2(x.z, v[r].z, s);
                s = dot2(x.w, v[r].w, s);
                acc[r * TP + t] += (double)s;
              }
            }
        }
      }
      if (lora)
#pragma unroll
        for (int t = 0; t < TP; ++t)
          if (TP == 1 || t0 + t < T) {
            int a;
            const int rk = dec_rank(p.lora, t0 + t, a);
#pragma unroll
            for (int r = 0; r < NR; ++r) {
              const int row = min(row0 + DEC_WAVES * r, end - 1);
              const uint16_t* B = bfit ? bl + ((row - up0) * T + t0 + t) * R : p.lora.B + ((int64_t)a * d + row) * R;
              for (int i = lane; i < rk; i += WAVE)
                acc[r * TP + t] += (double)ul[(t0 + t) * R + i] * (double)bf16f(B[i]);
            }
          }
      if constexpr (TP == 1) {
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const double v = wave_sum_dpp(acc[r]);
          if (lane == 0 && row0 + DEC_WAVES * r < end)
            p.out[(int64_t)t0 * d + row0 + DEC_WAVES * r] = f64_to_bf16(v);
        }
      } else {
        const double v = wave_sums<NR * TP>(acc);  // lane r TP + t
        const int row = row0 + DEC_WAVES * (lane / TP), t = t0 + lane % TP;
        if (lane < NR * TP && row < end && t < T) p.out[(int64_t)t * d + row] = f64_to_bf16(v);
      }
    }
  };
  auto up_all = [&](auto tp) {
    for (int row = slab1 + wave; row < up1; row += DEC_WAVES * UA) {
      rows_up(row, up1, std::integral_constant<int, UA>{}, tp, [&](int r, int q) { return wr[r][q]; });
      if (row + DEC_WAVES * UA < up1)
#pragma unroll
        for (int r = 0; r < UA; ++r) load_up(row + DEC_WAVES * (UA + r), r);
    }
    for (int row = up0 + wave; row < slab1; row += DEC_WAVES * 2)
      rows_up(row, slab1, std::integral_constant<int, 2>{}, tp, [&](int r, int q) {
        const int at = min(row + DEC_WAVES * r, slab1 - 1) - up0;
        return *reinterpret_cast<const uint4*>(slab + at * L + 8 * (WAVE * q + lane));
      });
  };
  up_all(std::integral_constant<int, ONE ? 1 : 4>{});
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

template <class W, int UC, int UA, bool ONE>
static hipError_t launch_decode_as(const DecodeArgs& a, unsigned grid, size_t lds, hipStream_t st) {
  static const hipError_t e =
      hipFuncSetAttribute(reinterpret_cast<const void*>(&decode_kernel<W, UC, UA, ONE>),
                          hipFuncAttributeMaxDynamicSharedMemorySize, (int)DEC_LDS);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((decode_kernel<W, UC, UA, ONE>), dim3(grid), dim3(DEC_THREADS), lds, st, a);
  return hipGetLastError();
}

template <class W>
static hipError_t launch_decode_for(const DecodeArgs& a, unsigned grid, size_t lds, hipStream_t st) {
  const bool wide = a.r.L > 7 * 512;
  if (a.r.T == 1)
    return wide ? launch_decode_as<W, 14, 1, true>(a, grid, lds, st) : launch_decode_as<W, 7, 2, true>(a, grid, lds, st);
  return wide ? launch_decode_as<W, 14, 1, false>(a, grid, lds, st) : launch_decode_as<W, 7, 2, false>(a, grid, lds, st);
}

hipError_t launch_decode(const DecodeArgs& args, bool packed, hipStream_t st) {
  DecodeArgs a = args;
  const int T = (int)a.r.T, n = T * a.r.k, L = a.r.L, F = a.F;
  if (T < 1 || T > DECODE_MAX_TOKENS || n > DECODE_MAX_ROWS || L % 128 || F % 128 || L > DEC_MAX_DIM || F > DEC_MAX_DIM ||
      a.r.E > ROUTE_MAXI * WAVE || a.r.d % 8)
    return hipErrorInvalidValue;
  // one block per CU, fewer where no phase has that many items
  int64_t items = ceil_div((int64_t)n * (F / 16), DEC_WAVES);
  if (items < (L / 16) * ceil_div(n, DEC_SLOTS)) items = (L / 16) * ceil_div(n, DEC_SLOTS);
  if (items < a.r.d / DEC_WAVES) items = a.r.d / DEC_WAVES;
  const unsigned grid = (unsigned)(items < cu_count() ? items : cu_count());
  a.up_rows = (int32_t)ceil_div(a.r.d, grid);
  // LDS: the quantised h; each wave's staged row of the down operand behind it, or, where they
  // do not fit there, in its place (and the block meets a barrier); then the slab
  const size_t hq = (size_t)T * dec_row_bytes(L), rows = (size_t)DEC_WAVES * dec_row_bytes(F);
  a.stage_offset = hq + rows <= DEC_LDS ? (int32_t)hq : 0;
  size_t used = a.stage_offset + rows;
  if (used < hq) used = hq;
  const size_t zu = (size_t)T * ((size_t)L * 2 + (a.lora.B ? (size_t)a.lora.R * 4 : 0));  // z and u come over both
  if (used < zu) used = zu;
  used = align_up(used, 16);
  if (used > DEC_LDS) return hipErrorInvalidValue;
  a.slab_offset = (int32_t)used;
  const int64_t slab = (int64_t)((DEC_LDS - used) / ((size_t)L * 2));
  a.slab_rows = (int32_t)(slab < a.up_rows ? slab : a.up_rows);
  const size_t lds = used + (size_t)a.slab_rows * L * 2;
  return packed ? launch_decode_for<PackedW>(a, grid, lds, st) : launch_decode_for<RecordW>(a, grid, lds, st);
}

}  // namespace moe
