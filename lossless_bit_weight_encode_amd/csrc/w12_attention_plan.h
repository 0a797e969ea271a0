// How a tree attention call is cut into items, each one block of rows over one chunk of tiles: integer arithmetic alone,
// run by the kernels (lengths are device memory) and, for the size of the workspace, bounded on the host.
#pragma once

#include <stdint.h>

namespace w12 {

constexpr int kTile = 64;            // tokens of a tile
constexpr int kBlockRows = 128;      // rows of a block
constexpr int kMostTiles = 1 << 24;  // of a request: it holds fewer than 2^30 tokens
// Least tiles of a chunk where all rows are up to 64 (twice as many for more than 32 chunks; us with them / without: one
// node over 8191 tokens 16.4 / 19.3, 12 nodes 19.0 / 21.1, but one node over 2047, always twice as many, 13.1 / 12.0), and
// elsewhere, where a partial result is as large as 2 tiles (63 nodes over 2047 tokens 19.2 us, with 6 tiles 19.8; over
// 8191 the same).
constexpr int kMinChunk = 2;
constexpr int kMinChunkLarge = 4;

__host__ __device__ constexpr int at_least(int v, int low) { return v < low ? low : v; }
__host__ __device__ constexpr int at_most(int v, int high) { return v > high ? high : v; }

// The blocks of a request: `full` of 128 rows, and a last one of `rest` waves' rows (0: none; 2: up to 64, whose
// other two waves take half of the tokens; 4).  A tile of a block costs its waves.
struct Blocks {
  int tiles, full, rest;
  __host__ __device__ int count() const { return full + (rest != 0); }
  __host__ __device__ int64_t cost() const { return (int64_t)tiles * (4 * full + rest); }
};

// Of `rows` rows over `len` tokens.
__host__ __device__ inline Blocks blocks_of(int rows, int len) {
  const int rem = rows % kBlockRows;
  return Blocks{(len + kTile - 1) / kTile, rows / kBlockRows, rem == 0 ? 0 : rem <= kBlockRows / 2 ? 2 : 4};
}

// Tiles of a chunk where requests share the chip: the cost of all tiles over `share`.  Where twice the blocks of all heads
// fit the chip, all items make one round: the cost is a tile of a block, half a chunk for each block is set
// aside for last chunks that are short, and a chunk that still gives too many items is lengthened by eighths, up to
// three times (us in one round / in about two: 16 requests of 24 nodes over up to 8000 tokens 80 / 86 in E4M3, 93 / 107 in
// BF16; 8 of 40 nodes, E4M3, 62 / 77; 4 of 12 nodes 41 / 43; 32 of 8 nodes over 4000 88 / 112).  Otherwise two rounds,
// whose items even out unequal lengths, and the cost is that of four waves.
__host__ __device__ inline int chunk_of(int64_t cost, int64_t share, int rows) {
  const int64_t tiles = (cost + share - 1) / share;
  return at_least(tiles > kMostTiles ? kMostTiles : (int)tiles, rows <= kBlockRows / 2 ? kMinChunk : kMinChunkLarge);
}

// Tiles of a chunk of one request, whose items (per = heads x blocks, for each chunk) have equally many tiles (of a last
// block of up to 64 rows, half a block's work): they go in whole rounds of the `slots` work-groups that the chip holds, the
// fewest that leave at most a quarter of the slots empty; a few items over a round would cost another one (us so / cut as
// several requests are: 63 nodes over 2047 tokens 19 / 27, over 8191 29 / 38, over 32767 68 / 74, 64 over 131001 232 / 233).
__host__ __device__ inline int one_request_chunk(const Blocks& k, int slots, int per, int rows) {
  int chunks = 1;
  for (int rounds = 1; rounds <= 4; ++rounds) {
    chunks = at_least(rounds * slots / at_least(per, 1), 1);
    if ((int64_t)4 * chunks * per >= 3 * rounds * slots) break;
  }
  const int least = rows <= kBlockRows / 2 ? at_most(at_least((k.tiles + 31) / 32, kMinChunk), 2 * kMinChunk) : kMinChunkLarge;
  return at_least((k.tiles + chunks - 1) / chunks, least);
}

struct Plan {
  int64_t items;
  int chunk;       // tiles of a chunk
};

__host__ __device__ inline int64_t items_of(const Blocks& c, int heads, int chunk) {
  return (int64_t)heads * c.count() * ((c.tiles + chunk - 1) / chunk);
}

// The items of a call of `rows` rows (nodes x group) in all.  blocks(b): request b's; sum(value): the sum of value(b)
// over the requests.
template <typename BlocksOf, typename Sum>
__host__ __device__ inline Plan plan_of(int requests, int heads, int rows, int target, BlocksOf blocks, Sum sum) {
  Plan p;
  const int slots = target / 2;
  if (requests == 1) {
    const Blocks k = blocks(0);
    p.chunk = one_request_chunk(k, slots, heads * k.count(), rows);
    p.items = items_of(k, heads, p.chunk);
  } else {
    const int64_t wanted = (int64_t)heads * at_least((rows + kBlockRows - 1) / kBlockRows, requests);
    const bool round = 2 * wanted <= slots;
    const int64_t cost = sum([&](int b) {
      const Blocks k = blocks(b);
      return heads * (round ? (int64_t)k.tiles * k.count() : k.cost());
    });
    p.chunk = chunk_of(cost, round ? slots - wanted / 2 : 4 * (int64_t)target, rows);
    for (int tries = 0;; ++tries) {
      p.items = sum([&](int b) { return items_of(blocks(b), heads, p.chunk); });
      if (!round || p.items <= slots || tries == 3) break;
      p.chunk += (p.chunk + 7) / 8;
    }
  }
  return p;
}

// Most items of a call whose ranges do not overlap.  Chunks are at least cost / (4 target) long and a tile costs at least 2,
// so whole chunks are at most 2 target; each head of each block has at most one more.  One request's items are at most
// four rounds, 2 target, or one for each head of each block.
__host__ __device__ inline int64_t most_items(int64_t rows, int requests, int heads, int target) {
  return 2 * (int64_t)target + ((rows + kBlockRows - 1) / kBlockRows + requests) * heads;
}

}  // namespace w12
