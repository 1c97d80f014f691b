// How the gate / up phase of the few-token layer (decode.hip) deals out its work: pairs of
// items in chunks, a chunk at a time to a block, an item at a time to its waves.  Arithmetic
// only, host code too, so that a model of the claims runs on the CPU.
#pragma once
#include <stdint.h>

namespace moe {

constexpr int DEC_TILES = 16;  // pairs of gate / up items a block may have open
constexpr uint32_t DEC_NO_CHUNK = 0xFFFFFFFFu;

// What a wave finds at a place of its block's chunk.
struct ChunkPlace {
  enum What {
    ITEM,  // half `half` of pair `pair`, the block's seq-th
    NEXT,  // the chunk is spent, and this wave brings the next
    WAIT,  // another wave is bringing it
    NONE   // no chunk is left
  };
  What what;
  int pair, seq, half;
};

// The block's chunk is one 64-bit word: in its upper half the head (pairs of the block's
// earlier chunks) << 16 | chunk, in its lower half the places taken of it so far.
//
// Only pairs that exist are numbered.  A pair's tile in the LDS is handed on, when the pair is
// complete, to the one DEC_TILES later in the block's count; a number that no pair has would
// leave its tile with nobody to hand it on, and a block that comes that far after a last chunk
// of fewer than cp pairs (as it does when few of the grid's blocks are resident) would wait for
// it for ever.
struct GateUpPlan {
  int pairs, cp, n;  // pairs of the phase, of a chunk (the last may have fewer), chunks

  // chunks of consecutive pairs, about half as many items as waves or as many: a CU's waves then
  // read one stretch of memory.  (The 64-bit divisions, and the order of the cases below, are what
  // the kernel runs fastest with, by its code's place in the instruction cache: one token 87.9 us, three
  // over records 276, against 92.1 and 281 with narrower divisions and the rare cases first.)
  constexpr GateUpPlan(int pairs_, int grid, int waves) : pairs(pairs_), cp(1), n(0) {
    const int64_t most = (int64_t)grid * (waves / 2), turns = (pairs + most - 1) / most;
    const int64_t rounds = turns < 1 ? 1 : turns;
    cp = (int)((pairs + grid * rounds - 1) / (grid * rounds));
    n = (pairs + cp - 1) / cp;
  }
  constexpr int size(uint32_t head) const {
    const int left = pairs - (int)(head & 0xFFFFu) * cp;
    return left < cp ? left : cp;
  }
  constexpr ChunkPlace place(uint32_t head, uint32_t taken) const {
    const uint32_t items = head == DEC_NO_CHUNK ? 0u : 2u * (uint32_t)size(head);
    if (taken < items)
      return {ChunkPlace::ITEM, (int)((head & 0xFFFFu) * (uint32_t)cp + taken / 2), (int)((head >> 16) + taken / 2),
              (int)(taken & 1u)};
    return {items == 0u ? ChunkPlace::NONE : taken == items ? ChunkPlace::NEXT : ChunkPlace::WAIT, 0, 0, 0};
  }
  // the head of the chunk the block takes after `head`, chunk -1 being none
  static constexpr uint32_t first(int chunk) { return chunk < 0 ? DEC_NO_CHUNK : (uint32_t)chunk; }
  constexpr uint32_t next(uint32_t head, int chunk) const {
    return chunk < 0 ? DEC_NO_CHUNK : ((head >> 16) + (uint32_t)size(head)) << 16 | (uint32_t)chunk;
  }
};

}  // namespace moe
