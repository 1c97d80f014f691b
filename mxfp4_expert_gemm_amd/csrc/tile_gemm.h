// Tiles of a matrix product on the matrix cores, for the dense block (ffn.hip) and the 8-bit
// projection (int8.hip):
//   C[m][n] = sum_k M(m, k) N(n, k),   the results handed to an epilogue.
//
// Either operand is K-major (rows of consecutive k, as activations and weights lie in a forward
// product) or row-major in the other index (k is the slow one), which a backward pass needs for
// the same matrices: dx = dg W reads W by its rows, dW = dg^T x reads both by their tokens.
//
// A block of WM x WN waves owns a tile of 16 MI WM x 16 NJ WN results, a wave 16 MI x 16 NJ of
// them.  K moves in tiles of 32 KS values (64 KS bytes; 64 KS 8-bit values), loaded straight into
// one of S stages of LDS S tiles ahead (lds loads of 16 bytes a lane), one barrier for a tile, and
// the operands of the next step of 32 are read into registers while the current step's products
// run.  What bounds it at large sizes is the LDS: a wave of 128 x 128 reads (128 + 128) x 64 bytes
// for 64 products of 16 cycles, four waves half of the LDS's 128 bytes a cycle, the loads into LDS
// a quarter.
//
// The operand that the matrix instruction calls A (its rows go to a lane's four result registers)
// is N, so that a lane holds consecutive n; and the n of a wave are dealt to instructions so that
// a lane's NJ x 4 results are consecutive: row rho of instruction j is
// n = 4 NJ (rho / 4) + 4 j + rho % 4.  GLU: the tile's first half are rows of one matrix, its
// second the same rows of another; a lane holds both for the same f.
//
// LDS layouts, in pieces of 16 bytes, free of bank conflicts for the reads below:
//  K-major: a row is 4 KS pieces, piece c stored at c ^ key(row) (KS = 2), or c ^ key(row) / 2
//    (KS = 1, where two rows share 128 bytes), key = the row's bits 0, 1 and SB, the bit in which
//    the rows read together by lanes 0-3 and 4-7 differ.
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
template <int VM>
__device__ __forceinline__ void tile_wait_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(VM) : "memory");
}

// One operand's tile of R rows.  SB, J: see above; SPLIT: the second half of the rows comes from p[1].
template <int ORDER, int R, int KS, int NW, int SB, int J, bool SPLIT>
struct TileLoader {
  static constexpr int BYTES = R * 64 * KS;
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
      step = 64 * KS;
      K16 = K * es;
    } else {
      step = (int64_t)(32 * KS) * o.ld;
      K16 = K;
    }
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int p = NW * u + wave;
      if constexpr (ORDER == TILE_KMAJ) {
        const int row = p * (16 / KS) + lane / (4 * KS), pos = lane % (4 * KS);
        const int c = pos ^ (KS == 1 ? key(row) >> 1 : key(row));
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
        const int row = p * (16 / KS) + lane / (4 * KS), pos = lane % (4 * KS);
        const int c = pos ^ (KS == 1 ? key(row) >> 1 : key(row));
        in = (int64_t)kt * (64 * KS) + 16 * c < K16;
      } else {
        in = (int64_t)kt * (32 * KS) + p * (512 / R) + lane / (R / 8) < K16;
      }
      const uint8_t* a = at(kt, u, seg1) + off[u];
      tile_dma(in ? a : reinterpret_cast<const uint8_t*>(tile_zero), lds + p * 1024);
    }
  }
};

// MI x NJ results of 16 x 16 a wave, WM x WN waves, K tiles of KS steps, S stages
template <int MI_, int NJ_, int WM_, int WN_, int KS_, int S_, int MORD_, int NORD_, bool GLU_, bool I8_ = false>
struct TileCfg {
  static constexpr int MI = MI_, NJ = NJ_, WM = WM_, WN = WN_, KS = KS_, S = S_, MORD = MORD_, NORD = NORD_;
  static constexpr bool GLU = GLU_, I8 = I8_;
  static constexpr int NW = WM * WN, BM = 16 * MI * WM, BN = 16 * NJ * WN;
  static constexpr int ES = I8 ? 1 : 2, BK = 64 * KS / ES;
  static constexpr int J = GLU ? NJ / 2 : NJ;  // a lane's consecutive n: 4 J
  static constexpr int SB = J == 8 ? 5 : J == 4 ? 4 : J == 2 ? 3 : 2;
  static constexpr int STAGE = (BM + BN) * 64 * KS, LDS = S * STAGE;
  // one wave a SIMD where the accumulators need it
  static constexpr int WAVES = MI * NJ > 32 ? 1 : 2;
};

template <class C, class Epi>
__global__ void __launch_bounds__(C::NW * 64, C::WAVES) tile_gemm_kernel(TileArgs p, Epi epi) {
  constexpr int MI = C::MI, NJ = C::NJ, KS = C::KS, S = C::S, NW = C::NW, BM = C::BM, BN = C::BN, J = C::J;
  using ML = TileLoader<C::MORD, BM, KS, NW, 2, 1, false>;
  using NL = TileLoader<C::NORD, BN, KS, NW, C::SB, J, C::GLU>;
  constexpr int NU = ML::NU + NL::NU;
  constexpr int M_BYTES = BM * 64 * KS;
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

  // Tile t of this block's K range, to stage t % S.  Tiles that reach past K (one a segment) come
  // first, so that only the first S loads have to look for them.
  auto load_one = [&](int t, uint32_t at, auto uc) {
    constexpr int U = decltype(uc)::value;
    int kt = k0 + t - part;
    const bool seg1 = kt >= full;
    if (seg1) kt -= full;
    if constexpr (U < ML::NU)
      ml.load(kt, seg1, U, at, wave);
    else
      nl.load(kt, seg1, U - ML::NU, at + M_BYTES, wave);
  };
  auto load_first = [&](int t, uint32_t at) {
    int kt = k0 + t;
    bool seg1 = kt == 1;
    if (kt < part) {
      kt = full;
    } else {
      kt -= part;
      seg1 = kt >= full;
      if (seg1) kt -= full;
    }
    ml.load_tail(kt, seg1, at, wave, lane);
    nl.load_tail(kt, seg1, at + M_BYTES, wave, lane);
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
  auto read_m = [&](const uint8_t* stage, int ks, int i) -> u32x4_t {
    if constexpr (C::MORD == TILE_KMAJ) {
      const int row = 16 * MI * wm + 16 * i + rho, c = 4 * ks + g, k = ML::key(rho);
      return *reinterpret_cast<const u32x4_t*>(stage + row * (64 * KS) + 16 * (KS == 1 ? c ^ (k >> 1) : c ^ k));
    } else {
      const int k = 32 * ks + 8 * g + (rho >> 2), q = rho & 3;
      const int piece = 2 * MI * wm + 2 * i + (q >> 1);
      return tr_read(stage + k * (2 * BM) + 16 * (piece ^ ML::fold(rho >> 2)) + 8 * (q & 1), 2 * BM);
    }
  };
  auto read_n = [&](const uint8_t* stage, int ks, int j) -> u32x4_t {
    const int h = C::GLU ? j / J : 0, jj = C::GLU ? j % J : j;
    const int at = h * (BN / 2) + 16 * J * wn + 4 * jj;
    if constexpr (C::NORD == TILE_KMAJ) {
      const int row = at + 4 * J * (rho >> 2) + (rho & 3), c = 4 * ks + g;
      const int k = (rho & 3) | ((rho >> 2) & 1) << 2;
      return *reinterpret_cast<const u32x4_t*>(stage + M_BYTES + row * (64 * KS) + 16 * (KS == 1 ? c ^ (k >> 1) : c ^ k));
    } else {
      const int k = 32 * ks + 8 * g + (rho >> 2), col = at + 4 * J * (rho & 3);
      return tr_read(stage + M_BYTES + k * (2 * BN) + 16 * ((col >> 3) ^ NL::fold(rho >> 2)) + 2 * (col & 7), 2 * BN);
    }
  };
  Acc acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = Acc{0, 0, 0, 0};

  // the products of one step from registers CUR, while the next step's operands are read into the
  // others and, with FETCH (or FETCH 2 and `fetch`), tile td is loaded to sd
  auto step = [&](auto curc, auto fetchc, bool fetch, const uint8_t* next, int ks_next, int td, uint32_t sd) {
    constexpr int CUR = decltype(curc)::value, FETCH = decltype(fetchc)::value;
    unroll_n<MI>([&](auto qc) {
      constexpr int Q = decltype(qc)::value;
      constexpr int U0 = Q * NU / MI, U1 = (Q + 1) * NU / MI;
      if constexpr (FETCH != 0 && U1 > U0) {
        if (FETCH == 1 || fetch)
          unroll_n<U1 - U0>([&](auto uc) { load_one(td, sd, std::integral_constant<int, U0 + decltype(uc)::value>{}); });
      }
      constexpr int A = MI + NJ, R0 = Q * A / MI, R1 = (Q + 1) * A / MI;
      unroll_n<R1 - R0>([&](auto rc) {
        constexpr int R = R0 + decltype(rc)::value;
        if constexpr (R < NJ)
          fn[CUR ^ 1][R] = read_n(next, ks_next, R);
        else
          fm[CUR ^ 1][R - NJ] = read_m(next, ks_next, R - NJ);
      });
      unroll_n<NJ>([&](auto jc) {
        constexpr int JJ = decltype(jc)::value;
        if constexpr (C::I8)
          acc[Q][JJ] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(tg_i32x4, fn[CUR][JJ]),
                                                             __builtin_bit_cast(tg_i32x4, fm[CUR][Q]), acc[Q][JJ], 0, 0, 0);
        else
          acc[Q][JJ] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(tg_bf16x8, fn[CUR][JJ]),
                                                               __builtin_bit_cast(tg_bf16x8, fm[CUR][Q]), acc[Q][JJ], 0, 0, 0);
      });
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  // Tile t.  At its last step every wave has its operands of tile t in registers, so that the
  // barrier frees t's stage, and tile t + 1 has landed; the tiles behind that one (S - 2 of them,
  // NU loads a wave each) may still be on their way.
  auto run_tile = [&](auto parc, auto fetchc, int t, int stage) {
    constexpr int P = decltype(parc)::value;  // the registers that hold the tile's first step
    const uint8_t* here = lds + stage * C::STAGE;
    const int sn = stage + 1 == S ? 0 : stage + 1;
    unroll_n<KS - 1>([&](auto kc) {
      constexpr int X = decltype(kc)::value;
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      step(std::integral_constant<int, (P + X) & 1>{}, std::integral_constant<int, 0>{}, false, here, X + 1, 0, 0);
    });
    if (decltype(fetchc)::value == 1 || t + S - 1 < nkt)
      tile_wait_barrier<(S - 2) * NU>();
    else
      tile_wait_barrier<0>();
    step(std::integral_constant<int, (P + KS - 1) & 1>{}, fetchc, t + S < nkt, lds + sn * C::STAGE, 0, t + S,
         lds0 + stage * C::STAGE);
  };

  const int pre = nkt < S ? nkt : S;
  for (int t = 0; t < pre; ++t) load_first(t, lds0 + t * C::STAGE);
  if (nkt >= S)
    tile_wait_barrier<(S - 1) * NU>();
  else
    tile_wait_barrier<0>();
#pragma unroll
  for (int j = 0; j < NJ; ++j) fn[0][j] = read_n(lds, 0, j);
#pragma unroll
  for (int i = 0; i < MI; ++i) fm[0][i] = read_m(lds, 0, i);
  // two tiles a turn (with an odd KS the registers swap from tile to tile), the last S or S + 1
  // tiles, which load nothing, or little, in a loop of their own: a branch in the first one costs
  // the accumulators their registers
  auto after = [](int stage) { return stage + 1 == S ? 0 : stage + 1; };
  int stage = 0, t = 0;
  for (; t + 1 + S < nkt; t += 2) {
    run_tile(std::integral_constant<int, 0>{}, std::integral_constant<int, 1>{}, t, stage);
    stage = after(stage);
    run_tile(std::integral_constant<int, KS & 1>{}, std::integral_constant<int, 1>{}, t + 1, stage);
    stage = after(stage);
  }
  for (; t < nkt; t += 2) {
    run_tile(std::integral_constant<int, 0>{}, std::integral_constant<int, 2>{}, t, stage);
    stage = after(stage);
    if (t + 1 < nkt) {
      run_tile(std::integral_constant<int, KS & 1>{}, std::integral_constant<int, 2>{}, t + 1, stage);
      stage = after(stage);
    }
  }
  // the reads of the step past the end are still on their way
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");

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
