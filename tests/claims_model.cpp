// A model of layer_decode's gate / up claims: blocks of eight waves that take chunks from sharded
// counters and items from their block's chunk, one item ahead, over the ring of tiles in which
// a pair's two halves meet.  Its arithmetic is the kernel's (decode_chunks.h).  Any wave may be
// the next to take a step; the order is drawn from a seed.
#include <cstdint>
#include <cstdio>
#include <vector>

#include "../mxfp4_expert_gemm_amd/csrc/decode_chunks.h"

using moe::ChunkPlace;
using moe::DEC_TILES;
using moe::GateUpPlan;

namespace {
constexpr int SHARDS = 32, WAVES = 8;

// What the model must be able to show: places of the last chunk that no pair has are numbered
// like the others, and skipped.
struct NumbersAbsentPairs : GateUpPlan {
  using GateUpPlan::GateUpPlan;
  ChunkPlace place(uint32_t head, uint32_t taken) const {
    if (head == moe::DEC_NO_CHUNK) return {ChunkPlace::NONE, 0, 0, 0};
    if (taken > 2u * cp) return {ChunkPlace::WAIT, 0, 0, 0};
    if (taken == 2u * cp) return {ChunkPlace::NEXT, 0, 0, 0};
    const int i = (int)taken, pair = (int)(head & 0xFFFFu) * cp + i / 2;
    if (pair >= pairs) return {ChunkPlace::WAIT, 0, 0, 0};  // the place is used up
    return {ChunkPlace::ITEM, pair, (int)(head >> 16) + i / 2, i & 1};
  }
  uint32_t next(uint32_t head, int chunk) const {
    return chunk < 0 ? moe::DEC_NO_CHUNK : ((head >> 16) + (uint32_t)cp) << 16 | (uint32_t)chunk;
  }
};

struct Wave {
  enum State { FETCH, CLAIM, TILE, DONE } state = FETCH;
  bool have = false, again = false;
  ChunkPlace x{}, y{};
  int shard = 0, asked = -1;
  uint32_t head = 0;
};

struct Block {
  uint32_t head = 0, taken = 0;
  int tile_of[DEC_TILES], tile_n[DEC_TILES];
  int next_seq = 0;
  Wave w[WAVES];
};

// 0: every item done once, each block's pairs numbered without a gap; 1: no wave can go on;
// 2: an item done twice or not at all, or a gap
template <class Plan>
int run(int pairs, int grid, int resident, uint64_t seed) {
  const Plan plan(pairs, grid, WAVES);
  std::vector<int> ctr(SHARDS, 0), done(2 * pairs, 0);
  std::vector<Block> blocks(resident);
  auto claim = [&](Wave& w) {  // one look at a shard; true when there is an answer in w.asked
    const int i = SHARDS * ctr[w.shard]++ + w.shard;
    if (i < plan.n) {
      w.asked = i;
      return true;
    }
    for (int s = 0; s < SHARDS; ++s) {
      const int at = (s + w.shard) % SHARDS;
      if (SHARDS * ctr[at] + at < plan.n) {
        w.shard = at;
        return false;
      }
    }
    w.asked = -1;
    return true;
  };
  for (int b = 0; b < resident; ++b) {
    for (int t = 0; t < DEC_TILES; ++t) blocks[b].tile_of[t] = t, blocks[b].tile_n[t] = 0;
    for (Wave& w : blocks[b].w) w.shard = b % SHARDS;
    while (!claim(blocks[b].w[0])) {
    }
    blocks[b].head = GateUpPlan::first(blocks[b].w[0].asked);
  }
  // one step of a wave; false when it changes nothing
  auto step = [&](Block& b, Wave& w) {
    switch (w.state) {
      case Wave::DONE: return false;
      case Wave::CLAIM:
        if (!claim(w)) return true;
        b.head = plan.next(w.head, w.asked);
        b.taken = 0;
        w.state = Wave::FETCH;
        return true;
      case Wave::FETCH: {
        const ChunkPlace at = plan.place(b.head, b.taken);
        if (b.head != moe::DEC_NO_CHUNK) ++b.taken;
        if (at.what == ChunkPlace::WAIT) return b.taken <= 2u * plan.cp;
        if (at.what == ChunkPlace::NEXT) {
          w.head = b.head;
          w.state = Wave::CLAIM;
          return true;
        }
        w.again = at.what == ChunkPlace::ITEM;
        if (w.again) w.y = at;
        if (w.have) {
          w.state = Wave::TILE;
        } else if (w.again) {
          w.x = w.y;
          w.have = true;
        } else {
          w.state = Wave::DONE;
        }
        return true;
      }
      case Wave::TILE: {
        const int t = w.x.seq % DEC_TILES;
        if (b.tile_of[t] != w.x.seq) return false;
        ++done[2 * w.x.pair + w.x.half];
        if (++b.tile_n[t] == 2) {
          b.tile_n[t] = 0;
          b.tile_of[t] = w.x.seq + DEC_TILES;
          ++b.next_seq;
        }
        w.x = w.y;
        w.state = w.again ? Wave::FETCH : Wave::DONE;
        return true;
      }
    }
    return false;
  };
  // Rounds over all waves in a drawn order, a drawn share of them held back in each (so that
  // some run far behind); a round in which none was held and none moved is the end.
  uint64_t r = seed * 0x9E3779B97F4A7C15ull + 1;
  auto draw = [&] {
    r ^= r << 13;
    r ^= r >> 7;
    r ^= r << 17;
    return r;
  };
  const int n = resident * WAVES;
  for (;;) {
    const int held = (int)(draw() % 4);  // quarters of the waves, in the mean
    const int off = (int)(draw() % n);
    bool moved = false, all_done = true;
    for (int i = 0; i < n; ++i) {
      const int v = (i + off) % n;
      Block& b = blocks[v / WAVES];
      Wave& w = b.w[v % WAVES];
      if ((int)(draw() % 4) < held) continue;
      moved = step(b, w) || moved;
    }
    if (!moved)
      for (int v = 0; v < n; ++v) moved = step(blocks[v / WAVES], blocks[v / WAVES].w[v % WAVES]) || moved;
    for (int v = 0; v < n; ++v) all_done = all_done && blocks[v / WAVES].w[v % WAVES].state == Wave::DONE;
    if (all_done) break;
    if (!moved) return 1;
  }
  int total = 0;
  for (const Block& b : blocks) {
    total += b.next_seq;
    for (int t = 0; t < DEC_TILES; ++t)  // the tile waits for the first number that was not given
      if (b.tile_n[t] || b.tile_of[t] < b.next_seq || b.tile_of[t] >= b.next_seq + DEC_TILES) return 2;
  }
  for (int d : done)
    if (d != 1) return 2;
  return total == pairs ? 0 : 2;
}
}  // namespace

// the kernel's plan (absent = 0), or the one that numbers absent pairs
extern "C" int claims_run(int pairs, int grid, int resident, uint64_t seed, int absent) {
  return absent ? run<NumbersAbsentPairs>(pairs, grid, resident, seed) : run<GateUpPlan>(pairs, grid, resident, seed);
}
extern "C" int claims_chunk(int pairs, int grid) { return GateUpPlan(pairs, grid, WAVES).cp; }
