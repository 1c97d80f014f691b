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
  // read one stretch of memory
  constexpr GateUpPlan(int pairs_, int grid, int waves) : pairs(pairs_), cp(1), n(0) {
    const int most = grid * (waves / 2);
    const int rounds = pairs > most ? (pairs + most - 1) / most : 1;
    cp = (pairs + grid * rounds - 1) / (grid * rounds);
    n = (pairs + cp - 1) / cp;
  }
  constexpr int size(uint32_t head) const {
    const int left = pairs - (int)(head & 0xFFFFu) * cp;
    return left < cp ? left : cp;
  }
  constexpr ChunkPlace place(uint32_t head, uint32_t taken) const {
    if (head == DEC_NO_CHUNK) return {ChunkPlace::NONE, 0, 0, 0};
    const uint32_t items = 2u * (uint32_t)size(head);
    if (taken > items) return {ChunkPlace::WAIT, 0, 0, 0};
    if (taken == items) return {ChunkPlace::NEXT, 0, 0, 0};
    const int i = (int)taken;
    return {ChunkPlace::ITEM, (int)(head & 0xFFFFu) * cp + i / 2, (int)(head >> 16) + i / 2, i & 1};
  }
  // the head of the chunk the block takes after `head`, chunk -1 being none
  static constexpr uint32_t first(int chunk) { return chunk < 0 ? DEC_NO_CHUNK : (uint32_t)chunk; }
  constexpr uint32_t next(uint32_t head, int chunk) const {
    return chunk < 0 ? DEC_NO_CHUNK : ((head >> 16) + (uint32_t)size(head)) << 16 | (uint32_t)chunk;
  }
};

}  // namespace moe
