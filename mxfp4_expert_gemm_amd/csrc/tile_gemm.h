// Tiles of a matrix product on the matrix cores, for the dense block (ffn.hip) and the 8-bit
// projection (int8.hip):
//   C[m][n] = sum_k M(m, k) N(n, k),   the results handed to an epilogue.
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
// registers while the current step's products run.  What bounds it at large sizes is the LDS: a
// wave of 128 x 128 reads (128 + 128) x 64 bytes for 64 products of 16 cycles, four waves half of
// the LDS's 128 bytes a cycle, the loads into LDS a quarter.
//
// The operand that the matrix instruction calls A (its rows go to a lane's four result registers)
// is N, so that a lane holds consecutive n; and the n of a wave are dealt to instructions so that
// a lane's NJ x 4 results are consecutive: row rho of instruction j is
// n = 4 NJ (rho / 4) + 4 j + rho % 4.  GLU: the tile's first half are rows of one matrix, its
// second the same rows of another; a lane holds both for the same f.
//
// LDS layouts, in pieces of 16 bytes, free of bank conflicts for the reads below:
//  K-major: a row is 8 pieces, piece c stored at c ^ key(row), key = the row's bits 0, 1 and SB, the
//    bit in which the rows read together by lanes 0-3 and 4-7 differ.
//  row-major: a k is R/8 pieces, piece p stored at p ^ f(k), read by the transposing LDS read: 16
//    lanes hand in 4 k x 16 rows, and lane i receives row i's four k.
#pragma once

#include "common.h"

namespace moe {

typedef __bf16 tg_bf16x8 __attribute__((ext_vector_type(8)));
typedef float tg_f32x4 __attribute__((ext_vector_type(4)));
typedef int tg_i32x4 __attribute__((ext_vector_type(4)));
typedef short tg_s16x4 __attribute__((ext_vector_type(4)));

enum TileOrder { TILE_KMAJ = 0, TILE_RMAJ = 1 };

struct TileOperand {
  const void* p[2];  // second: the other K segment, or the rows of a tile's second half (GLU)
  int64_t ld;        // bytes from a row (K-major) or a k (row-major) to the next
  int32_t rows;
};
struct TileArgs {
  TileOperand m, n;
  int64_t K;       // values of one K segment; K-major: a multiple of 16 bytes of them
  int32_t nk;      // K tiles of a segment
  int32_t nkt;     // K tiles in all (nk, or 2 nk)
  int32_t splits;  // the K tiles are dealt to so many blocks, each with an output of its own
  int32_t ntm, ntn;
  int32_t nblocks;  // ntm * ntn * splits
};

// what a lane reads where a tile's k lie past K
static __device__ __align__(16) const uint32_t tile_zero[4] = {0u, 0u, 0u, 0u};

// 16 bytes a lane from scalar base + lane offset, or from a lane's own address, to LDS at lds + 16
// lane.  m0 is left changed: the compiler keeps nothing there on this target, it writes m0 right
// before its own uses.
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

// One operand's tile of R rows.  SB, J: see above; SPLIT: the second half of the rows comes from p[1].
template <int ORDER, int R, int NW, int SB, int J, bool SPLIT>
struct TileLoader {
  static constexpr int BYTES = R * 128;
  static constexpr int NU = BYTES / (1024 * NW);  // loads of a wave for one tile
  static_assert(NU * 1024 * NW == BYTES, "whole loads");
  static_assert(ORDER == TILE_KMAJ || R >= 128, "row-major tiles permute within 16 pieces");
  uint32_t off[NU];
  const uint8_t* base[2];
  int64_t step, K16;  // bytes (K-major) or k (row-major) of a segment
  int nk;

  static __device__ __forceinline__ int key(int row) { return (row & 3) | ((row >> SB) & 1) << 2; }
  static __device__ __forceinline__ int fold(int k) {  // row-major: what a k's pieces are stored at
    return J == 8 ? (k & 3) : J == 4 ? (k & 1) | ((k >> 1) & 1) << 3 : (k & 3) << 1;
  }
  __device__ __forceinline__ void init(const TileOperand& o, int r0, int64_t K, int nk_, int es, int wave, int lane) {
    nk = nk_;
    const int half = SPLIT ? R / 2 : R;
    const int left = o.rows - r0;
#pragma unroll
    for (int s = 0; s < 2; ++s)
      base[s] = static_cast<const uint8_t*>(o.p[s]) + (ORDER == TILE_KMAJ ? (int64_t)r0 * o.ld : (int64_t)r0 * 2);
    if constexpr (ORDER == TILE_KMAJ) {
      step = 128;
      K16 = K * es;
    } else {
      step = 64 * o.ld;
      K16 = K;
    }
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int p = NW * u + wave;
      if constexpr (ORDER == TILE_KMAJ) {
        const int row = 8 * p + lane / 8, c = (lane % 8) ^ key(row);
        const int in = row % half;
        off[u] = (uint32_t)((in < left ? in : left - 1) * o.ld + 16 * c);
      } else {
        const int k = p * (512 / R) + lane / (R / 8), pos = lane % (R / 8);
        const int piece = pos ^ fold(k), last = (left - 1) / 8;
        off[u] = (uint32_t)(k * o.ld + 16 * (piece < last ? piece : last));
      }
    }
  }
  __device__ __forceinline__ const uint8_t* at(int kt, int u, bool seg1) const {
    if constexpr (SPLIT) return base[(u >= NU / 2) ? 1 : 0] + kt * step;
    return (seg1 ? base[1] : base[0]) + kt * step;
  }
  // load u of K tile kt (of its segment), all of whose k exist
  __device__ __forceinline__ void load(int kt, bool seg1, int u, uint32_t lds, int wave) const {
    tile_dma(at(kt, u, seg1), off[u], lds + (NW * u + wave) * 1024);
  }
  // all loads of a tile, some of whose k may lie past K: zeros
  __device__ __forceinline__ void load_tail(int kt, bool seg1, uint32_t lds, int wave, int lane) const {
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int p = NW * u + wave;
      bool in;
      if constexpr (ORDER == TILE_KMAJ) {
        const int row = 8 * p + lane / 8, c = (lane % 8) ^ key(row);
        in = (int64_t)kt * 128 + 16 * c < K16;
      } else {
        in = (int64_t)kt * 64 + p * (512 / R) + lane / (R / 8) < K16;
      }
      const uint8_t* a = at(kt, u, seg1) + off[u];
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
  static constexpr int ES = I8 ? 1 : 2, BK = 128 / ES;
  static constexpr int J = GLU ? NJ / 2 : NJ;  // a lane's consecutive n: 4 J
  static constexpr int SB = J == 8 ? 5 : J == 4 ? 4 : J == 2 ? 3 : 2;
  static constexpr int SLOT = (BM > BN ? BM : BN) * 128, LDS = R * SLOT;
  // one wave a SIMD where the accumulators need it
  static constexpr int WAVES = MI * NJ > 32 ? 1 : 2;
  static_assert(R % 2 == 1 && R >= 5, "two whole tiles (the first may be cut short) and one operand");
};

// acc += n m for one step.  Where the accumulators take half of the registers they are held in the
// accumulation registers by hand: left to itself the compiler moves them back and forth (280 moves
// for the 128 products of a K tile).  It does not know these instructions, so what it must not do
// next to them is kept away: between two that share an accumulator lie 63 others, operands come
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

template <class C, class Epi>
__global__ void __launch_bounds__(C::NW * 64, C::WAVES) tile_gemm_kernel(TileArgs p, Epi epi) {
  constexpr int MI = C::MI, NJ = C::NJ, R = C::R, H = (R - 1) / 2, NW = C::NW, BM = C::BM, BN = C::BN, J = C::J;
  using ML = TileLoader<C::MORD, BM, NW, 2, 1, false>;
  using NL = TileLoader<C::NORD, BN, NW, C::SB, J, C::GLU>;
  constexpr int MU = ML::NU, NU = NL::NU;
  using Acc = std::conditional_t<C::I8, tg_i32x4, tg_f32x4>;
  extern __shared__ __align__(16) uint8_t lds[];

  const int nbp = gridDim.x;
  const int lb = (blockIdx.x & 7) * (nbp >> 3) + (blockIdx.x >> 3);
  if (lb >= p.nblocks) return;
  constexpr int GROUP = 8;
  const int per = p.ntm * p.ntn, split = lb / per, tile = lb - split * per;
  const int span = GROUP * p.ntn, grp = tile / span, first = grp * GROUP;
  const int gs = p.ntm - first < GROUP ? p.ntm - first : GROUP;
  const int within = tile - grp * span;
  const int m0 = (first + within % gs) * BM, n0 = (within / gs) * (C::GLU ? BN / 2 : BN);
  const int k0 = (int)((int64_t)p.nkt * split / p.splits), k1 = (int)((int64_t)p.nkt * (split + 1) / p.splits);
  const int nkt = k1 - k0;

  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / WAVE));
  const int wm = wave / C::WN, wn = wave % C::WN, rho = lane & 15, g = lane >> 4;
  ML ml;
  NL nl;
  ml.init(p.m, m0, p.K, p.nk, C::ES, wave, lane);
  nl.init(p.n, n0, p.K, p.nk, C::ES, wave, lane);
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(lds));
  const int full = (int)(p.K / C::BK), part = (p.nkt - full * (p.nkt / p.nk)) != 0 ? p.nkt / p.nk : 0;

  // Tile t of this block's K range.  Tiles that reach past K (one a segment) come first, so that
  // only the loads ahead of the loop have to look for them.
  auto place = [&](int t, bool& seg1) {
    int kt = k0 + t - part;
    seg1 = kt >= full;
    return seg1 ? kt - full : kt;
  };
  auto first_m = [&](int t, uint32_t at) {
    bool seg1 = k0 + t == 1;
    const int kt = k0 + t < part ? full : place(t, seg1);
    ml.load_tail(kt, seg1, at, wave, lane);
  };
  auto first_n = [&](int t, uint32_t at) {
    bool seg1 = k0 + t == 1;
    const int kt = k0 + t < part ? full : place(t, seg1);
    nl.load_tail(kt, seg1, at, wave, lane);
  };

  // the operands of one step in registers
  u32x4_t fm[2][MI], fn[2][NJ];
  auto tr_read = [&](const uint8_t* at, int row_bytes) {
    typedef __attribute__((address_space(3))) tg_s16x4* lp;
    union {
      tg_s16x4 h[2];
      u32x4_t v;
    } r;
    r.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)at);
    r.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(at + 4 * row_bytes));
    return r.v;
  };
  auto read_m = [&](const uint8_t* slot, int ks, int i) -> u32x4_t {
    if constexpr (C::MORD == TILE_KMAJ) {
      const int row = 16 * MI * wm + 16 * i + rho;
      return *reinterpret_cast<const u32x4_t*>(slot + row * 128 + 16 * ((4 * ks + g) ^ ML::key(rho)));
    } else {
      const int k = 32 * ks + 8 * g + (rho >> 2), q = rho & 3;
      const int piece = 2 * MI * wm + 2 * i + (q >> 1);
      return tr_read(slot + k * (2 * BM) + 16 * (piece ^ ML::fold(rho >> 2)) + 8 * (q & 1), 2 * BM);
    }
  };
  auto read_n = [&](const uint8_t* slot, int ks, int j) -> u32x4_t {
    const int h = C::GLU ? j / J : 0, jj = C::GLU ? j % J : j;
    const int at = h * (BN / 2) + 16 * J * wn + 4 * jj;
    if constexpr (C::NORD == TILE_KMAJ) {
      const int row = at + 4 * J * (rho >> 2) + (rho & 3), key = (rho & 3) | ((rho >> 2) & 1) << 2;
      return *reinterpret_cast<const u32x4_t*>(slot + row * 128 + 16 * ((4 * ks + g) ^ key));
    } else {
      const int k = 32 * ks + 8 * g + (rho >> 2), col = at + 4 * J * (rho & 3);
      return tr_read(slot + k * (2 * BN) + 16 * ((col >> 3) ^ NL::fold(rho >> 2)) + 2 * (col & 7), 2 * BN);
    }
  };
  Acc acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = Acc{0, 0, 0, 0};

  // the products of step KS, while the next step's operands are read into the other registers and,
  // with FETCH, the step's operand of tile td (M in the first step, N in the second) is loaded to `to`
  auto step = [&](auto ksc, auto fetchc, const uint8_t* next_m, const uint8_t* next_n, int td, uint32_t to) {
    constexpr int KS = decltype(ksc)::value;
    constexpr bool FETCH = decltype(fetchc)::value;
    constexpr int U = KS == 0 ? MU : NU;
    unroll_n<MI>([&](auto qc) {
      constexpr int Q = decltype(qc)::value;
      if constexpr (FETCH) {
        bool seg1;
        const int kt = place(td, seg1);
        unroll_n<(Q + 1) * U / MI - Q * U / MI>([&](auto uc) {
          constexpr int X = Q * U / MI + decltype(uc)::value;
          if constexpr (KS == 0)
            ml.load(kt, seg1, X, to, wave);
          else
            nl.load(kt, seg1, X, to, wave);
        });
      }
      constexpr int A = MI + NJ, R0 = Q * A / MI, R1 = (Q + 1) * A / MI;
      unroll_n<R1 - R0>([&](auto rc) {
        constexpr int X = R0 + decltype(rc)::value;
        if constexpr (X < NJ)
          fn[KS ^ 1][X] = read_n(next_n, KS ^ 1, X);
        else
          fm[KS ^ 1][X - NJ] = read_m(next_m, KS ^ 1, X - NJ);
      });
      unroll_n<NJ>([&](auto jc) {
        constexpr int X = decltype(jc)::value;
        tile_mfma<C>(acc[Q][X], fn[KS][X], fm[KS][Q]);
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

  const int pre = nkt < H ? nkt : H;
  for (int t = 0; t < pre; ++t) {
    first_m(t, lds0 + 2 * t * C::SLOT);
    first_n(t, lds0 + (2 * t + 1) * C::SLOT);
  }
  if (nkt >= H)
    tile_wait_barrier<(H - 1) * (MU + NU)>();
  else
    tile_wait_barrier<0>();
#pragma unroll
  for (int j = 0; j < NJ; ++j) fn[0][j] = read_n(lds + C::SLOT, 0, j);
#pragma unroll
  for (int i = 0; i < MI; ++i) fm[0][i] = read_m(lds, 0, i);
  tile_settle<C>(acc);
  int slot = 0, t = 0;
  for (; t + H < nkt; ++t) slot = run_tile(std::true_type{}, t, slot);
  for (; t < nkt; ++t) slot = run_tile(std::false_type{}, t, slot);  // nothing left to load
  // the reads of the step past the end are still on their way
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  tile_settle<C>(acc);

  // lane: results m = 16 i + rho, n = 4 J g .. 4 J g + 4 J - 1 (of each half)
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int m = m0 + 16 * MI * wm + 16 * i + rho;
    const int n = n0 + 16 * J * wn + 4 * J * g;
    if (m < p.m.rows) epi.template row<C>(m, n, p.n.rows, split, acc[i]);
  }
}

template <class C, class Epi>
hipError_t launch_tile_gemm(TileArgs a, int segs, const Epi& epi, hipStream_t st) {
  a.ntm = (int32_t)ceil_div(a.m.rows, C::BM);
  a.ntn = (int32_t)ceil_div(a.n.rows, C::GLU ? C::BN / 2 : C::BN);
  a.nk = (int32_t)ceil_div(a.K, C::BK);
  a.nkt = a.nk * segs;
  const int64_t nb = (int64_t)a.ntm * a.ntn * a.splits;
  if (a.splits < 1 || a.splits > a.nkt || nb > 0x7FFFFFF0) return hipErrorInvalidValue;
  a.nblocks = (int32_t)nb;
  const unsigned grid = (unsigned)((nb + 7) / 8 * 8);
  if constexpr (C::LDS > 65536) {
    static const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&tile_gemm_kernel<C, Epi>),
                                                    hipFuncAttributeMaxDynamicSharedMemorySize, C::LDS);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((tile_gemm_kernel<C, Epi>), dim3(grid), dim3(C::NW * 64), C::LDS, st, a, epi);
  return hipGetLastError();
}

}  // namespace moe
