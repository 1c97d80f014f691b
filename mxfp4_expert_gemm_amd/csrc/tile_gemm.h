// Tiles of a matrix product on the matrix cores, for the dense block (ffn.hip) and the 8-bit
// projection (int8.hip):
//   C[m][n] = sum_k M(m, k) N(n, k),   the results handed to an epilogue, eight n at a time.
//
// Either operand is K-major (rows of consecutive k, as activations and weights lie in a forward
// product) or row-major in the other index (k is the slow one), which a backward pass needs for
// the same matrices: dx = dg W reads W by its rows, dW = dg^T x reads both by their tokens.
//
// A block of WM x WN waves owns a tile of 16 MI WM x 16 NJ WN results, a wave 16 MI x 16 NJ of
// them.  K moves in tiles of 128 bytes of it (64 bf16 or 128 8-bit values: whole lines of a K-major
// operand, half lines cost each line two trips from the L2), two steps of 64 bytes a tile.
// Operand tiles are loaded straight into LDS (16 bytes a lane) into a ring of R slots, M and N of
// a tile one after another: while tile t is worked on, M of tile t + (R - 1) / 2 is loaded during
// its first step, into the slot that N of tile t - 1 left, and N during its second, into the slot of
// M of tile t, one barrier for a tile.  R is odd, so the ring holds one operand more than whole
// tiles: five slots of 32 KB are all of the LDS.  The operands of the next step are read into
// registers while the current step's products run.
//
// A block goes on from tile to tile of its share, the first K tiles of the next one loading under
// the epilogue of the last.  Each XCD (blocks b with the same b mod 8) has a contiguous range of an
// order that goes through groups of 8 tiles in m, so that what is resident shares operands.
//
// The operand that the matrix instruction calls A (its rows go to a lane's four result registers)
// is N: lane l holds n = 4 (l / 16) + 0..3 of m = l % 16.  GLU: N has the rows of two matrices; an
// instruction's first eight are rows f .. f + 7 of the first and its other eight the same of the
// second.
//
// LDS layouts, in pieces of 16 bytes, free of bank conflicts for the reads:
//  K-major: a row is 8 pieces, piece c stored at c ^ (row % 8);
//  row-major: a k is RP/8 pieces, piece p stored at p ^ 2 (k % 4) ^ 8 (k / 8 % 2) (of 64 rows, whose k
//    alternate between the halves of 256 bytes, ^ 2 (k / 8 % 2)), read by the transposing LDS read:
//    16 lanes hand in 4 k x 16 rows, and lane i receives row i's four k; 32 lanes, of k and k + 8,
//    are served at once.  (With p ^ 2 (k % 4) alone those two met: 5.1e7 conflicts in the weights'
//    gradients of 4096 tokens, 18% of the cycles; the products hid them.)
// What bounds it at large sizes: a wave of 128 x 128 reads (128 + 128) x 64 bytes from LDS for 64
// products of 16 cycles, four waves half of the LDS's 128 bytes a cycle, the loads into LDS a
// quarter; the products themselves run at what the card's power allows (1.9 GHz under this load).
// Counted at 4096 tokens: the matrix cores busy for 74% of the units' cycles in the gate/up product, 68%
// in down, 51% in dA (its epilogue), 81% in dx, 72% in the weights' gradients; 53% in 8 bits, 8191 tokens
// (of twice the rate).
#pragma once

#include "common.h"

namespace moe {

typedef __bf16 tg_bf16x8 __attribute__((ext_vector_type(8)));
typedef float tg_f32x4 __attribute__((ext_vector_type(4)));
typedef int tg_i32x4 __attribute__((ext_vector_type(4)));
typedef short tg_s16x4 __attribute__((ext_vector_type(4)));

enum TileOrder { TILE_KMAJ = 0, TILE_RMAJ = 1 };

struct TileOperand {
  const void* p[2];  // second: the other K segment, or the second matrix (GLU)
  int64_t ld;        // bytes from a row (K-major) or a k (row-major) to the next
  int32_t rows;
};
struct TileArgs {
  TileOperand m, n;
  int64_t K;       // values of one K segment; K-major: whole pieces of 16 bytes
  int32_t splits;  // the K tiles are dealt to so many blocks; tile_join adds their results
  int32_t halves;  // 2: the second half of M's rows are the low bits of the first's; tile_join adds their results,
                   // without the second's where the first's are not finite (there 0 may have met an infinity)
  int32_t which;   // told to the epilogue: of two products in one launch, whose results these are
  int64_t part;    // where in the epilogue's part the product's pieces begin
  // set by the launcher
  int32_t nk;        // K tiles of a segment
  int32_t nkt;       // K tiles in all (nk, or 2 nk)
  int32_t ntm, ntn;
  int32_t nblocks;   // ntm * ntn * splits
};

// what a lane reads where a tile's k lie past K
static __device__ __align__(16) const uint32_t tile_zero[4] = {0u, 0u, 0u, 0u};

// 16 bytes a lane from scalar base + lane offset, or from a lane's own address, to LDS at lds + 16
// lane.  m0 is left changed: the compiler keeps nothing there on this target, it writes m0 right
// before its own uses.  A write of m0 needs one wait state before the load that reads it, and the
// compiler does not look for that inside asm: so they stand in one block with an s_nop between, or
// apart, as tile_dma_to and tile_dma_go, with an instruction in between that is asm volatile like
// them (one of the compiler's own may be moved away).
__device__ __forceinline__ void tile_dma_to(uint32_t lds) { asm volatile("s_mov_b32 m0, %0" ::"s"(lds)); }
__device__ __forceinline__ void tile_dma_go(const uint8_t* base, uint32_t off) {
  asm volatile("global_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base) : "memory");
}
__device__ __forceinline__ void tile_dma(const uint8_t* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(lds) : "memory");
}
__device__ __forceinline__ void tile_dma(const uint8_t* at, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(at), "s"(lds) : "memory");
}
// waits for all of the wave's loads into LDS but the last VM, and for its LDS reads, then for the block
template <int VM>
__device__ __forceinline__ void tile_wait_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(VM) : "memory");
}

// One operand's tile of ROWS rows.  SPLIT: its second half are rows of p[1].
template <int ORDER, int ROWS, int NW, bool SPLIT>
struct TileLoader {
  // a row-major tile is as wide as the next power of two: what it permutes stays inside
  static constexpr int RP = ORDER == TILE_KMAJ ? ROWS : ROWS <= 64 ? 64 : ROWS <= 128 ? 128 : 256;
  static constexpr int BYTES = RP * 128;
  static constexpr int NU = BYTES / (1024 * NW);  // loads of a wave for one tile
  static_assert(NU * 1024 * NW == BYTES, "whole loads");
  static_assert(!SPLIT || ORDER == TILE_KMAJ, "two matrices by their rows");
  // where a row-major k has its pieces
  static __device__ __forceinline__ int swizzle(int k) { return (2 * (k % 4)) ^ (k / 8 % 2 * (RP == 64 ? 2 : 8)); }
  uint32_t off[NU];
  const uint8_t* base[2];
  int64_t step, K16;  // bytes (K-major) or k (row-major) of a segment

  __device__ __forceinline__ void init(const TileOperand& o, int r0, int64_t K, int es, int wave, int lane) {
    constexpr int HALF = SPLIT ? ROWS / 2 : ROWS;
    const int left = o.rows - r0;
#pragma unroll
    for (int s = 0; s < 2; ++s)
      base[s] = static_cast<const uint8_t*>(o.p[s]) + (ORDER == TILE_KMAJ ? (int64_t)r0 * o.ld : (int64_t)r0 * 2);
    step = ORDER == TILE_KMAJ ? 128 : 64 * o.ld;
    K16 = ORDER == TILE_KMAJ ? K * es : K;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int p = NW * u + wave;
      if constexpr (ORDER == TILE_KMAJ) {  // rows past the last one are read as that one, and not used
        const int row = 8 * p + lane / 8, c = (lane % 8) ^ (row % 8), in = row % HALF;
        off[u] = (uint32_t)((in < left ? in : left - 1) * o.ld + 16 * c);
      } else {
        const int k = p * (512 / RP) + lane / (RP / 8), pos = lane % (RP / 8);
        const int piece = pos ^ swizzle(k), last = (left - 1) / 8;
        off[u] = (uint32_t)(k * o.ld + 16 * (piece < last ? piece : last));
      }
    }
  }
  __device__ __forceinline__ const uint8_t* at(int kt, int p, bool seg1) const {
    if constexpr (SPLIT) return base[p >= ROWS / 16 ? 1 : 0] + kt * step;  // 8 rows a load, half the rows
    return (seg1 ? base[1] : base[0]) + kt * step;
  }
  // load u of K tile kt (of its segment), all of whose k exist; or first where to, then the load
  __device__ __forceinline__ void load(int kt, bool seg1, int u, uint32_t lds, int wave) const {
    tile_dma(at(kt, NW * u + wave, seg1), off[u], lds + (NW * u + wave) * 1024);
  }
  __device__ __forceinline__ void load_to(int u, uint32_t lds, int wave) const { tile_dma_to(lds + (NW * u + wave) * 1024); }
  __device__ __forceinline__ void load_go(int kt, bool seg1, int u, int wave) const {
    tile_dma_go(at(kt, NW * u + wave, seg1), off[u]);
  }
  // all loads of a tile, some of whose k may lie past K: zeros
  __device__ __forceinline__ void load_tail(int kt, bool seg1, uint32_t lds, int wave, int lane) const {
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int p = NW * u + wave;
      bool in;
      if constexpr (ORDER == TILE_KMAJ)
        in = (int64_t)kt * 128 + 16 * ((lane % 8) ^ (lane / 8)) < K16;  // row 8 p + lane / 8
      else
        in = (int64_t)kt * 64 + p * (512 / RP) + lane / (RP / 8) < K16;
      const uint8_t* a = at(kt, p, seg1) + off[u];
      tile_dma(in ? a : reinterpret_cast<const uint8_t*>(tile_zero), lds + p * 1024);
    }
  }
};

// MI x NJ results of 16 x 16 a wave, WM x WN waves, R slots
template <int MI_, int NJ_, int WM_, int WN_, int R_, int MORD_, int NORD_, bool GLU_, bool I8_ = false>
struct TileCfg {
  static constexpr int MI = MI_, NJ = NJ_, WM = WM_, WN = WN_, R = R_, MORD = MORD_, NORD = NORD_;
  static constexpr bool GLU = GLU_, I8 = I8_;
  static constexpr int NW = WM * WN, BM = 16 * MI * WM, BN = 16 * NJ * WN;
  static constexpr int OUT_N = GLU ? BN / 2 : BN;  // columns of the result
  static constexpr int ES = I8 ? 1 : 2, BK = 128 / ES;
  using ML = TileLoader<MORD, BM, NW, false>;
  using NL = TileLoader<NORD, BN, NW, GLU>;
  static constexpr int SLOT = ML::BYTES > NL::BYTES ? ML::BYTES : NL::BYTES, LDS = R * SLOT;
  // One wave a SIMD where the accumulators need it.  The others' products may be split: those tiles
  // are taken where there are enough of them.
  static constexpr int WAVES = MI * NJ > 32 ? 1 : 2;
  static constexpr bool JOINS = WAVES == 2;
  // Few-token tiles stream their weights, all blocks at one pace: where rows are multiples of 4 KB
  // apart they would all ask the same memory channels at once, so there each block begins elsewhere
  // in K (one token, 8192 -> 7168: 22.5 us from 26; 7168 -> 8192, rows of 14 KB: 42.5 from 40.8).
  static constexpr bool TURN = R > 5;
  static constexpr int BLOCKS = 256 * (163840 / LDS);  // resident at once on 256 CUs
  static_assert(R % 2 == 1 && R >= 5, "two whole tiles (the first may be cut short) and one operand");
  static_assert(NW * 16 * 16 * NJ * 4 <= SLOT, "the epilogue passes 16 rows a wave through one slot");
};

// acc += n m for one step.  Where the accumulators take half of the registers they are held in the
// accumulation registers by hand: left to itself the compiler moves them back and forth (280 moves
// for the 128 products of a K tile).  It does not know these instructions, so what it must not do
// next to them is kept away: between two that share an accumulator lie 50 others, operands come
// from LDS reads, which it waits for, and tile_settle stands before and after the loop.
template <class C, class Acc>
__device__ __forceinline__ void tile_mfma(Acc& acc, const u32x4_t& n, const u32x4_t& m) {
  if constexpr (C::WAVES == 1) {
    if constexpr (C::I8)
      asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(acc) : "v"(n), "v"(m));
    else
      asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(n), "v"(m));
  } else if constexpr (C::I8) {
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(tg_i32x4, n), __builtin_bit_cast(tg_i32x4, m), acc, 0, 0, 0);
  } else {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(tg_bf16x8, n), __builtin_bit_cast(tg_bf16x8, m), acc, 0, 0, 0);
  }
}
// 32 wait states between what writes the accumulators before it and what reads them behind it (a
// product's result needs 18 at most)
template <class C, class Acc>
__device__ __forceinline__ void tile_settle(Acc (&acc)[C::MI][C::NJ]) {
  if constexpr (C::WAVES == 1) {
#pragma unroll
    for (int i = 0; i < C::MI; ++i)
#pragma unroll
      for (int j = 0; j < C::NJ; ++j) asm volatile("" : "+a"(acc[i][j]));
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
#pragma unroll
    for (int i = 0; i < C::MI; ++i)
#pragma unroll
      for (int j = 0; j < C::NJ; ++j) asm volatile("" : "+a"(acc[i][j]));
  }
}

// The epilogue's type Epi has
//   static constexpr bool BEGINS      void begin(), if so: what the grid's threads do before their tiles
//   struct Held                       what it reads from memory for eight results
//   Held hold(m, n)                   reads that, ahead of the results
//   void put(which, m, n, left, held, v)       eight results (left: columns from n on that exist), or with GLU
//   void put(which, m, n, left, held, v, w)    eight of each matrix
//   Value* part                       pieces of products whose K is split, which tile_join adds and calls
//                                     put with: [splits][rows of M][rows of N rounded up to 8], GLU [splits][2]..
template <class C, class Epi>
__global__ void __launch_bounds__(C::NW * 64, C::WAVES) tile_gemm_kernel(TileArgs p0, TileArgs p1, Epi epi) {
  constexpr int MI = C::MI, NJ = C::NJ, R = C::R, H = (R - 1) / 2, BM = C::BM, BN = C::BN;
  using ML = typename C::ML;
  using NL = typename C::NL;
  constexpr int MU = ML::NU, NU = NL::NU;
  using Acc = std::conditional_t<C::I8, tg_i32x4, tg_f32x4>;
  using Value = std::conditional_t<C::I8, int32_t, float>;
  extern __shared__ __align__(16) uint8_t lds[];

  if constexpr (Epi::BEGINS) epi.begin();
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / WAVE));
  const int wm = wave / C::WN, wn = wave % C::WN, rho = lane & 15, g = lane >> 4;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(lds));
  // this block's share: every gridDim / 8-th tile of its XCD's range
  const int all = p0.nblocks + p1.nblocks;
  const int range = (all + 7) / 8, first = (int)(blockIdx.x & 7) * range + (int)(blockIdx.x >> 3);
  const int end = min((int)(blockIdx.x & 7) * range + range, all), stride = gridDim.x >> 3;

  ML ml;
  NL nl;
  struct Place {  // of a tile of results
    int which, m0, n0, split, joins, tile, rows_m, rows_n;
    int64_t part;
  } at;
  int full, part, k0, nkt, turn = 0;
  auto start = [&](int lb) {
    constexpr int GROUP = 8;
    const bool second = lb >= p0.nblocks;
    const TileArgs& p = second ? p1 : p0;
    if (second) lb -= p0.nblocks;
    const int per = p.ntm * p.ntn;
    const int split = lb / per, tile = lb - split * per;
    const int span = GROUP * p.ntn, grp = tile / span, from = grp * GROUP;
    const int gs = p.ntm - from < GROUP ? p.ntm - from : GROUP;
    const int within = tile - grp * span;
    const int m0 = (from + within % gs) * BM, n0 = (within / gs) * C::OUT_N;
    at = Place{p.which, m0, n0, split, p.splits * p.halves, tile, p.m.rows, p.n.rows, p.part};
    full = (int)(p.K / C::BK);
    part = full == p.nk ? 0 : p.nkt / p.nk;
    k0 = (int)((int64_t)p.nkt * split / p.splits);
    nkt = (int)((int64_t)p.nkt * (split + 1) / p.splits) - k0;
    if constexpr (C::TURN) {
      const int whole = nkt - (k0 < part ? min(part - k0, nkt) : 0);
      turn = whole > 0 && p.n.ld % 4096 == 0 ? (tile * 11) % whole : 0;
    }
    ml.init(p.m, m0, p.K, C::ES, wave, lane);
    nl.init(p.n, n0, p.K, C::ES, wave, lane);
  };
  // K tile t of the share's tile.  Tiles that reach past K (one a segment) come first, so that only
  // the loads ahead of the loop have to look for them.
  auto place = [&](int t, bool& seg1) {
    int kt = k0 + t - part;
    if constexpr (C::TURN) {
      kt += turn;
      if (kt >= k0 + nkt - part) kt -= nkt - (k0 < part ? part - k0 : 0);
    }
    seg1 = kt >= full;
    return seg1 ? kt - full : kt;
  };
  auto load_first = [&]() {
    for (int t = 0; t < (nkt < H ? nkt : H); ++t) {
      bool seg1 = k0 + t == 1;
      const int kt = k0 + t < part ? full : place(t, seg1);
      ml.load_tail(kt, seg1, lds0 + 2 * t * C::SLOT, wave, lane);
      nl.load_tail(kt, seg1, lds0 + (2 * t + 1) * C::SLOT, wave, lane);
    }
  };

  // the operands of one step in registers
  u32x4_t fm[2][MI], fn[2][NJ];
  auto tr_read = [&](const uint8_t* from, int row_bytes) {
    typedef __attribute__((address_space(3))) tg_s16x4* lp;
    union {
      tg_s16x4 h[2];
      u32x4_t v;
    } r;
    r.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)from);
    r.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(from + 4 * row_bytes));
    return r.v;
  };
  auto read_tile = [&](const uint8_t* slot, auto orderc, auto widthc, int ks, int row, int col0) -> u32x4_t {
    if constexpr (decltype(orderc)::value == TILE_KMAJ) {
      return *reinterpret_cast<const u32x4_t*>(slot + row * 128 + 16 * ((4 * ks + g) ^ (rho & 7)));
    } else {  // lane: k = 32 ks + 8 g + rho / 4 (and + 4), four rows from 4 (rho % 4)
      constexpr int W = 2 * decltype(widthc)::value;
      const int k = 32 * ks + 8 * g + (rho >> 2), q = rho & 3;
      const int swizzle = (2 * (rho >> 2)) ^ ((g & 1) * (W == 128 ? 2 : 8));
      return tr_read(slot + k * W + 16 * ((col0 / 8 + (q >> 1)) ^ swizzle) + 8 * (q & 1), W);
    }
  };
  auto read_m = [&](const uint8_t* slot, int ks, int i) {
    const int r = 16 * MI * wm + 16 * i;
    return read_tile(slot, std::integral_constant<int, C::MORD>{}, std::integral_constant<int, ML::RP>{}, ks, r + rho, r);
  };
  auto read_n = [&](const uint8_t* slot, int ks, int j) {
    const int r = 16 * NJ * wn + 16 * j;
    const int row = C::GLU ? (rho >> 3) * (BN / 2) + r / 2 + (rho & 7) : r + rho;
    return read_tile(slot, std::integral_constant<int, C::NORD>{}, std::integral_constant<int, NL::RP>{}, ks, row, r);
  };
  Acc acc[MI][NJ];

  // The products of step KS, while the next step's operands are read into the other registers and,
  // with FETCH, the step's operand of tile td (M in the first step, N in the second) is loaded to `to`.
  // A product occupies the matrix cores for 16 cycles and its wave for 4, so what else there is to
  // issue is dealt out one by one between the products; a few instructions in a row leave them idle
  // (a read, its address and a load at every eighth product: 63% busy at 4096 tokens 7168 -> 3584).  The
  // reads end before three quarters of the products: the barrier that follows waits for the last.
  auto step = [&](auto ksc, auto fetchc, const uint8_t* next_m, const uint8_t* next_n, int td, uint32_t to) {
    constexpr int KS = decltype(ksc)::value;
    constexpr bool FETCH = decltype(fetchc)::value;
    constexpr int U = KS == 0 ? MU : NU, A = MI + NJ, S = MI * NJ;
    bool seg1 = false;
    const int kt = FETCH ? place(td, seg1) : 0;
    unroll_n<S>([&](auto sc) {
      constexpr int X = decltype(sc)::value, Q = X / NJ, JJ = X % NJ;
      // loads u at products floor(u S / U); reads r at floor(3 r S / 4 A)
      constexpr int U0 = (X * U + S - 1) / S, U1 = ((X + 1) * U + S - 1) / S;
      constexpr bool ASM = C::WAVES == 1;  // the product between m0 and the first load is asm
      if constexpr (FETCH && ASM && U1 > U0) {
        if constexpr (KS == 0)
          ml.load_to(U0, to, wave);
        else
          nl.load_to(U0, to, wave);
      }
      tile_mfma<C>(acc[Q][JJ], fn[KS][JJ], fm[KS][Q]);
      if constexpr (FETCH) {
        unroll_n<U1 - U0>([&](auto uc) {
          constexpr int V = U0 + decltype(uc)::value;
          if constexpr (ASM && V == U0) {
            if constexpr (KS == 0)
              ml.load_go(kt, seg1, V, wave);
            else
              nl.load_go(kt, seg1, V, wave);
          } else {
            if constexpr (KS == 0)
              ml.load(kt, seg1, V, to, wave);
            else
              nl.load(kt, seg1, V, to, wave);
          }
        });
      }
      constexpr int R0 = (4 * A * X + 3 * S - 1) / (3 * S), R1 = (4 * A * (X + 1) + 3 * S - 1) / (3 * S);
      constexpr int E0 = R0 < A ? R0 : A, E1 = X == S - 1 ? A : R1 < A ? R1 : A;
      unroll_n<E1 - E0>([&](auto rc) {
        constexpr int V = E0 + decltype(rc)::value;
        if constexpr (V < NJ)
          fn[KS ^ 1][V] = read_n(next_n, KS ^ 1, V);
        else
          fm[KS ^ 1][V - NJ] = read_m(next_m, KS ^ 1, V - NJ);
      });
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  // Tile t, its M in slot sm.  At the barrier every wave has the operands of its second step in
  // registers, which frees both slots, and tile t + 1 has landed; what was loaded behind that one (M
  // and N of tiles t + 2 .. t + H - 1, and M of tile t + H) may still be on its way.
  auto after = [](int slot, int by) { return slot + by >= R ? slot + by - R : slot + by; };
  auto run_tile = [&](auto fetchc, int t, int sm) {
    const int sn = after(sm, 1), next = after(sm, 2);
    const uint8_t *m = lds + sm * C::SLOT, *n = lds + sn * C::SLOT;
    step(std::integral_constant<int, 0>{}, fetchc, m, n, t + H, lds0 + after(sm, R - 1) * C::SLOT);
    if constexpr (decltype(fetchc)::value)
      tile_wait_barrier<(H - 1) * MU + (H - 2) * NU>();
    else
      tile_wait_barrier<0>();
    step(std::integral_constant<int, 1>{}, fetchc, lds + next * C::SLOT, lds + after(next, 1) * C::SLOT, t + H,
         lds0 + sm * C::SLOT);
    return next;
  };

  // one piece of a split K (GLU: of matrix `second`)
  auto store_part = [&](const Place& e, int second, int m, int n, const Value (&v)[8]) {
    const int64_t row = ((int64_t)e.split * (C::GLU ? 2 : 1) + second) * e.rows_m + m;
    Value* q = epi.part + e.part + row * ((e.rows_n + 7) & ~7) + n;
#pragma unroll
    for (int h = 0; h < 2; ++h) *reinterpret_cast<Acc*>(q + 4 * h) = Acc{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
  };

  // Sixteen rows of the wave's results at a time through its part of the last slot (which the first
  // loads of the next tile leave alone), so that memory is met in runs of whole rows: row rho is
  // 16 NJ words, four of them at a time stored at their place ^ rho % 8 (of an odd NJ, whose rows
  // alternate between the halves of 128 bytes, ^ rho / 2 % 4).
  auto epilogue = [&](const Place& e) {
    constexpr int PR = (C::GLU ? 8 : 16) * NJ / 8;        // pieces of eight results of a row (of one matrix)
    constexpr int P = 16 * PR, PL = (P + 63) / 64;        // of 16 rows, and of a lane
    uint8_t* mine = lds + (R - 1) * C::SLOT + wave * (16 * 64 * NJ);
    const int wcols = (C::GLU ? 8 : 16) * NJ * wn;
    auto where = [&](int s, int i, int& m, int& n) {
      const int x = lane + 64 * s, row = x / PR, piece = x - row * PR;
      m = e.m0 + 16 * MI * wm + 16 * i + row;
      n = e.n0 + wcols + 8 * piece;
      return x < P && m < e.rows_m && n < e.rows_n;
    };
    typename Epi::Held held[2][PL];
    auto hold = [&](int i) {
#pragma unroll
      for (int s = 0; s < PL; ++s) {
        int m, n;
        if (where(s, i, m, n)) held[i & 1][s] = epi.hold(m, n);
      }
    };
    hold(0);
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      if (i + 1 < MI) hold(i + 1);
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int word = C::GLU ? (g >> 1) * (8 * NJ) + 8 * j + 4 * (g & 1) : 16 * j + 4 * g;
        *reinterpret_cast<Acc*>(mine + rho * (64 * NJ) + 16 * ((word / 4) ^ (NJ % 2 ? (rho >> 1) & 3 : rho & 7))) = acc[i][j];
      }
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int s = 0; s < PL; ++s) {
        int m, n;
        const bool in = where(s, i, m, n);
        const int x = lane + 64 * s, row = x / PR, piece = x - row * PR;
        auto eight = [&](int word, Value (&v)[8]) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const Acc a = *reinterpret_cast<const Acc*>(mine + (row & 15) * (64 * NJ) +
                                                        16 * ((word / 4 + h) ^ (NJ % 2 ? (row >> 1) & 3 : row & 7)));
#pragma unroll
            for (int r = 0; r < 4; ++r) v[4 * h + r] = a[r];
          }
        };
        Value v[8], w[8];
        eight(8 * piece, v);
        if constexpr (C::GLU) eight(8 * NJ + 8 * piece, w);
        if (!in) continue;
        if (!C::JOINS || e.joins == 1) {
          if constexpr (C::GLU)
            epi.put(e.which, m, n, e.rows_n - n, held[i & 1][s], v, w);
          else
            epi.put(e.which, m, n, e.rows_n - n, held[i & 1][s], v);
        } else {
          store_part(e, 0, m, n, v);
          if constexpr (C::GLU) store_part(e, 1, m, n, w);
        }
      }
      __builtin_amdgcn_wave_barrier();
    }
  };

  if (first >= end) return;
  start(first);
  load_first();
  for (int lb = first;;) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = Acc{0, 0, 0, 0};
    if (lb == first && nkt >= H)
      tile_wait_barrier<(H - 1) * (MU + NU)>();  // the first K tile has landed
    else
      tile_wait_barrier<0>();  // the stores of the last epilogue are among what is waited for
#pragma unroll
    for (int j = 0; j < NJ; ++j) fn[0][j] = read_n(lds + C::SLOT, 0, j);
#pragma unroll
    for (int i = 0; i < MI; ++i) fm[0][i] = read_m(lds, 0, i);
    tile_settle<C>(acc);
    int slot = 0, t = 0;
    for (; t + H < nkt; ++t) slot = run_tile(std::true_type{}, t, slot);
    for (; t < nkt; ++t) slot = run_tile(std::false_type{}, t, slot);  // nothing left to load
    tile_settle<C>(acc);
    tile_wait_barrier<0>();  // the reads past the last step are done everywhere: the LDS is free
    const Place done = at;
    lb += stride;
    const bool more = lb < end;
    if (more) {
      start(lb);
      load_first();
    }
    epilogue(done);
    if (!more) break;
  }
}

// Tiles of 256 x 224 instead of 256 x 256, where fewer turns of the 256 CUs' blocks, or less work
// in the same number, come of it: a turn costs by the tile's width.
inline bool tiles_of_224(int64_t M, int64_t N) {
  auto turns = [&](int64_t width) { return ceil_div(ceil_div(M, 256) * ceil_div(N, width), 256); };
  return turns(224) * 7 < turns(256) * 8;
}

// The sums of the pieces of a split K, added in their order (the same call gives the same bits).  A
// launch of its own, 2 to 4 us: joined by whichever block of a tile comes last, the pieces had to pass the
// XCDs' own caches and one unit read all of a tile's (33 tokens, 7168 -> 3584: 20.4 us in all, 10.1 + 4 so).
struct TileJoin {  // of one product
  int64_t pieces, part;  // eight results each
  int32_t N, parts, which, halves;
};
template <class Value, bool GLU, class Epi>
__global__ void __launch_bounds__(256) tile_join_kernel(TileJoin p0, TileJoin p1, Epi epi) {
  int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const bool second = x >= p0.pieces;
  const TileJoin p = second ? p1 : p0;
  if (second) x -= p0.pieces;
  if (x >= p.pieces) return;
  typedef Value V4 __attribute__((ext_vector_type(4)));
  constexpr int G = GLU ? 2 : 1;
  const int32_t row = (p.N + 7) / 8;
  const int m = (int)(x / row), n = 8 * (int)(x - (int64_t)m * row);
  V4 a[2 * G];
#pragma unroll
  for (int i = 0; i < 2 * G; ++i) a[i] = V4{0, 0, 0, 0};
#pragma unroll 4
  for (int s = 0; s < p.parts; ++s)
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const V4* q = reinterpret_cast<const V4*>(epi.part + p.part + ((int64_t)(s * G + i) * p.pieces + x) * 8);
      a[2 * i] += q[0];
      a[2 * i + 1] += q[1];
    }
  Value v[G][8];
#pragma unroll
  for (int i = 0; i < G; ++i)
#pragma unroll
    for (int r = 0; r < 8; ++r) v[i][r] = a[2 * i + r / 4][r % 4];
  if constexpr (!GLU && std::is_same_v<Value, float>) {
    if (p.halves == 2) {
      bool finite = true;
#pragma unroll
      for (int r = 0; r < 8; ++r) finite = finite && fabsf(v[0][r]) < INFINITY;
      if (!finite) {  // the first halves' sums alone
        a[0] = a[1] = V4{0, 0, 0, 0};
        for (int s = 0; s < p.parts; s += 2) {
          const V4* q = reinterpret_cast<const V4*>(epi.part + p.part + ((int64_t)s * p.pieces + x) * 8);
          a[0] += q[0];
          a[1] += q[1];
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) v[0][r] = fabsf(v[0][r]) < INFINITY ? v[0][r] : a[r / 4][r % 4];
      }
    }
  }
  if constexpr (GLU)
    epi.put(p.which, m, n, p.N - n, epi.hold(m, n), v[0], v[1]);
  else
    epi.put(p.which, m, n, p.N - n, epi.hold(m, n), v[0]);
}

// the K tiles and tiles of results of one product
template <class C>
bool tile_plan(TileArgs& a, int segs) {
  a.ntm = (int32_t)ceil_div(a.m.rows, C::BM);
  a.ntn = (int32_t)ceil_div(a.n.rows, C::OUT_N);
  a.nk = (int32_t)ceil_div(a.K, C::BK);
  a.nkt = a.nk * segs;
  const int64_t nb = (int64_t)a.ntm * a.ntn * a.splits;
  a.nblocks = (int32_t)nb;
  return a.splits >= 1 && a.splits <= a.nkt && nb <= 0x3FFFFFF0 && a.m.rows % a.halves == 0 &&
         (C::JOINS || a.splits * a.halves == 1);
}
// One product, or two in one launch (of as many K segments each).
template <class C, class Epi>
hipError_t launch_tile_gemm(TileArgs a, int segs, const Epi& epi, hipStream_t st, const TileArgs* second = nullptr) {
  TileArgs b{};
  if (second) b = *second;
  if (!tile_plan<C>(a, segs) || (second && !tile_plan<C>(b, segs))) return hipErrorInvalidValue;
  const int64_t nb = (int64_t)a.nblocks + b.nblocks;
  const unsigned grid = (unsigned)(nb < C::BLOCKS ? (nb + 7) / 8 * 8 : C::BLOCKS);
  if constexpr (C::LDS > 65536) {
    static const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&tile_gemm_kernel<C, Epi>),
                                                    hipFuncAttributeMaxDynamicSharedMemorySize, C::LDS);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((tile_gemm_kernel<C, Epi>), dim3(grid), dim3(C::NW * 64), C::LDS, st, a, b, epi);
  if constexpr (C::JOINS) {
    using Value = std::conditional_t<C::I8, int32_t, float>;
    auto join = [](const TileArgs& p) {  // a piece of all of M's rows is one of each half
      if (p.nblocks == 0 || p.splits * p.halves == 1) return TileJoin{};
      return TileJoin{(int64_t)(p.m.rows / p.halves) * ceil_div(p.n.rows, 8), p.part, p.n.rows, p.splits * p.halves, p.which, p.halves};
    };
    const TileJoin ja = join(a), jb = join(b);
    if (ja.pieces + jb.pieces > 0)
      hipLaunchKernelGGL((tile_join_kernel<Value, C::GLU, Epi>), dim3((unsigned)ceil_div(ja.pieces + jb.pieces, 256)),
                         dim3(256), 0, st, ja, jb, epi);
  }
  return hipGetLastError();
}

// Tiles by the size of the output: 256 x 256 (or 224) where those fill three quarters of the units;
// otherwise few tokens take 16, 32, 48 or 64 rows by 64 columns in blocks of two waves, two blocks a
// unit, with a deep ring.  Outputs of more than 48,896 columns (each matrix of a GLU: 24,448) fill the
// units with large tiles whatever their rows, most of which then do not exist: one token in 8 bits,
// 7168 -> 49152 94.7 us (3.7 TB/s), -> 163840 263 (4.5), where 40960 columns, on tiles of 16 rows, take
// 64.1 (4.6).  Between them 128 x 128, two blocks a unit, or where those leave units idle and K is
// short, so that beginning and ending count and not the stream, 64 x 64 (77 tokens, 512 and 1000 wide:
// forward 14.5 us from 20.2, backward 24 from 31; 512 tokens, 1024 -> 1024: forward 18.5 from 27.5.
// With a longer K they lose: 100 tokens, 4096 -> 4096 46 from 36.8).
enum TileSize { TILE_16, TILE_32, TILE_48, TILE_64, TILE_SQUARE_64, TILE_128, TILE_224, TILE_256 };
inline TileSize tile_size(int64_t M, int64_t N, int64_t k_tiles, bool row_major) {
  if (ceil_div(M, 256) * ceil_div(N, 256) >= 192) return tiles_of_224(M, N) ? TILE_224 : TILE_256;
  if (M <= 64 && !row_major) return (TileSize)((M - 1) / 16);
  return ceil_div(M, 128) * ceil_div(N, 128) <= 128 && k_tiles <= 32 ? TILE_SQUARE_64 : TILE_128;
}
inline int64_t tiles_of(TileSize z, int64_t M, int64_t N) {
  const int64_t m = z == TILE_128 ? 128 : 64, n = z == TILE_128 ? 128 : 64;
  return ceil_div(M, m) * ceil_div(N, n);
}
// K is split where the tiles of the output alone leave units idle: no more pieces than bring the
// grid to a block a unit, of 8 K tiles at least, 16 at most (33 tokens, 7168 -> 3584, 56 tiles:
// 23 us whole, 12.1 in two, 10.1 in four, 10.6 in eight).  Below 24 K tiles the join costs what the
// pieces save or more (128 tokens, 1024 and 2048 wide: forward 16.8 us whole, 19.8 in two pieces each).
inline int tile_splits(TileSize z, int64_t tiles, int64_t k_tiles) {
  if (z >= TILE_224) return 1;
  const int64_t most = k_tiles < 24 ? 1 : k_tiles / 8, want = 256 / tiles, s = want < most ? want : most;
  return s < 1 ? 1 : s > 16 ? 16 : (int)s;
}
template <int MO, int NO, bool GLU, bool I8, class Epi>
hipError_t run_middle_tiles(TileSize z, const TileArgs& a, int segs, const Epi& e, hipStream_t st, const TileArgs* b = nullptr) {
  if (z == TILE_SQUARE_64) return launch_tile_gemm<TileCfg<2, 2, 2, 2, 5, MO, NO, GLU, I8>>(a, segs, e, st, b);
  return launch_tile_gemm<TileCfg<4, 4, 2, 2, 5, MO, NO, GLU, I8>>(a, segs, e, st, b);
}
template <int MO, int NO, bool GLU, bool I8, class Epi>
hipError_t run_tiles(TileSize z, const TileArgs& a, int segs, const Epi& e, hipStream_t st, const TileArgs* b = nullptr) {
  if (z == TILE_256) return launch_tile_gemm<TileCfg<8, 8, 2, 2, 5, MO, NO, GLU, I8>>(a, segs, e, st, b);
  if (z == TILE_224) return launch_tile_gemm<TileCfg<8, 7, 2, 2, 5, MO, NO, GLU, I8>>(a, segs, e, st, b);
  if constexpr (MO == TILE_KMAJ && NO == TILE_KMAJ) {
    switch (z) {
      case TILE_16: return launch_tile_gemm<TileCfg<1, 2, 1, 2, 9, MO, NO, GLU, I8>>(a, segs, e, st, b);
      case TILE_32: return launch_tile_gemm<TileCfg<2, 2, 1, 2, 9, MO, NO, GLU, I8>>(a, segs, e, st, b);
      case TILE_48: return launch_tile_gemm<TileCfg<3, 2, 1, 2, 9, MO, NO, GLU, I8>>(a, segs, e, st, b);
      case TILE_64: return launch_tile_gemm<TileCfg<4, 2, 1, 2, 9, MO, NO, GLU, I8>>(a, segs, e, st, b);
      default: break;
    }
  }
  return run_middle_tiles<MO, NO, GLU, I8>(z, a, segs, e, st, b);
}

}  // namespace moe
