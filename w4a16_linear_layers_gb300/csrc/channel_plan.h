// channel_plan.h -- which kernel takes a per-channel W8A8 product, and how its
// work is divided.  Host arithmetic only, on the sizes and on how many clusters
// a device runs at one time: no CUDA, so that it is checked without a device.
#pragma once

#include <cstddef>
#include <cstdint>

namespace qlin {

constexpr int kSWarps = 8;                 // warps of a streaming block, along K
constexpr int kMaxSplits = 8;              // streaming blocks of a cluster, along K
constexpr int kKB = 64;                    // K of one step of a streaming warp
constexpr int kMaxParts = 4;               // pairs of a cluster

// Clusters that run at one time on a device, by their size: GPCs of different
// sizes each take whole ones (152 SMs take 36, 23 and 15 clusters of 4, 6 and 8
// blocks that fill an SM).
struct Room {
  int sm_count = 0;
  int pairs[kMaxParts + 1] = {};           // of so many pairs
  int narrow[kMaxSplits + 1] = {};         // of the streaming kernel's blocks: 32 channels, 8 tokens
  int wide[kMaxSplits + 1] = {};           // 64 channels, 8 tokens
  int tokens16[kMaxSplits + 1] = {};       // 32 channels, 16 tokens
};

// Blocks that share K: as many as run at one time for all tiles, while a warp's
// steps get fewer.
struct StreamSplit {
  int splits;
  int64_t steps;
};
inline StreamSplit split_stream(int64_t tiles, const int* room, int64_t K) {
  const int64_t nkb = K / kKB;
  StreamSplit best{1, (nkb + kSWarps - 1) / kSWarps};
  for (int c = 2; c <= kMaxSplits; ++c) {
    const int64_t steps = (nkb + kSWarps * c - 1) / (kSWarps * c);
    if (tiles <= room[c] && steps < best.steps) best = {c, steps};
  }
  return best;
}

// 16 tokens a block: two blocks an SM (three of 85 registers a thread spill:
// 16 x 5120 x 1024 6.2 us instead of 4.1).
inline int64_t stream16_tiles(int64_t M, int64_t N) { return (N + 31) / 32 * ((M + 15) / 16); }

// The streaming kernel's block (32 or 64 channels, 8 or 16 tokens) and the blocks
// of a cluster, which share K.
struct StreamPlan {
  int channels, tokens, splits;
};
inline StreamPlan plan_stream(int64_t M, int64_t N, int64_t K, const Room& room) {
  if (M > 8) return {32, 16, split_stream(stream16_tiles(M, N), room.tokens16, K).splits};
  // A step of a warp takes about 1.2 us, of 64 channels 1.5, mostly latency: the
  // fewer steps the better, while all blocks run at one time.  8 x 5120 x 5120 7.9
  // us (32 channels in 2 parts of K; unsplit 11.4, in 3 parts of 64 8.3), 8 x 17408
  // x 5120 18.7 (64 channels in 3 parts; 32 in 2 21.3), 8 x 17408 x 8192 26.7 (64 in
  // 2; 32 unsplit 38.6), 8 x 5120 x 10240 12.3 (32 unsplit; 64 14.4).  More tiles
  // of 32 than run at one time: N = 34816 32.6 us in 64, 38 in 32.
  const int64_t tiles = (N + 31) / 32, tiles2 = (N + 63) / 64;
  const StreamSplit narrow = split_stream(tiles, room.narrow, K);
  const StreamSplit wide = split_stream(tiles2, room.wide, K);
  if (tiles > room.narrow[1] || (tiles2 <= room.wide[1] && 152 * wide.steps < 120 * narrow.steps))
    return {64, 8, wide.splits};
  return {32, 8, narrow.splits};
}

constexpr size_t kCounterBytes = 1024;    // arrival counters of the cut tiles
constexpr int64_t kMinShare = 8;          // K steps of a pair's share of the cut tiles, at least

struct PairPlan {
  int T = 0;
  int64_t TT = 0, F2 = 0, G = 0, pairs = 0, band = 0, sk_tiles = 0, sk_pairs = 0;
  int64_t parts = 1;        // pairs of a cluster: they share a tile
  bool cut = false;         // some tile is shared between other pairs
  size_t part_bytes = 0;    // int32 partials of the shared tiles
  int64_t cost = 0;         // estimated time, in 10 ns
};

// A tile size: the time of a K step, of a tile's way out (where its steps take
// less) and of what is around a pair's tiles, in 10 ns, measured at N from 5120 to
// 219520; a step takes 37, 40, 44 and 56 now, and less where few tiles share HBM.
// Parts of a tile that meet in a cluster take 2 us; through the workspace
// 5 us and half a one for 64 tokens of each part, of which 1.5 are left where
// whole tiles follow.
struct PairSize {
  int T, step, out, base;
};
constexpr PairSize kPairSizes[4] = {{64, 38, 170, 330}, {96, 43, 210, 400}, {128, 47, 250, 450}, {192, 56, 320, 560}};

inline PairPlan plan_tiles(const PairSize& size, int64_t M, int64_t N, int64_t K, const Room& room) {
  PairPlan pl;
  const int64_t slots = room.sm_count / 2;
  pl.T = size.T;
  pl.TT = (M + size.T - 1) / size.T;
  pl.F2 = (N + 255) / 256;
  pl.G = K / 128;
  pl.band = pl.TT < 8 ? pl.TT : 8;
  const int64_t tiles = pl.TT * pl.F2;
  const int64_t rest = tiles % slots;
  const int64_t rounds = tiles / slots;
  pl.pairs = tiles < slots ? tiles : slots;
  const int64_t whole = size.step * pl.G > size.out ? size.step * pl.G : size.out;
  int64_t last = rest == 0 ? 0 : whole;   // time of the last round
  // The last round's tiles are cut along K unless they nearly fill it: into as
  // many equal parts as the pairs allow where that is two or more, else into
  // shares that cross tiles.
  if (rest != 0 && rest * 8 < slots * 7) {
    const int64_t most = slots / rest;
    int64_t n = most >= 2 ? rest * (most < pl.G / kMinShare ? most : pl.G / kMinShare) : slots;
    if (n * kMinShare > rest * pl.G) n = rest * pl.G / kMinShare;
    if (n > rest) {
      const int64_t meet = rounds > 0 ? 150 : 480 + 45 * ((n + rest - 1) / rest) * size.T / 64;
      const int64_t cut = size.step * ((rest * pl.G + n - 1) / n) + meet;
      if (cut < last) {
        pl.sk_tiles = rest;
        pl.sk_pairs = n;
        pl.cut = true;
        pl.part_bytes = static_cast<size_t>(n) * 4 * pl.T * 128 * sizeof(int32_t);
        if (pl.pairs < n) pl.pairs = n;
        last = cut;
      }
    }
  }
  // Few tiles: the pairs of a cluster share one, and meet in shared memory (64 x
  // 5120 x 5120 10.9 us, without 12.5; 512 x 5120 x 1024 12.8 and 14.4; 64 x 2048 x
  // 4096 6.9 and 8.7).
  for (int c = 2; c <= kMaxParts && c * kMinShare <= pl.G; ++c) {
    const int64_t shared = size.step * ((pl.G + c - 1) / c) + 200;
    if (tiles <= room.pairs[c] && shared < last) {
      pl.parts = c;
      pl.cut = false;
      pl.part_bytes = 0;
      pl.sk_tiles = tiles;
      pl.sk_pairs = pl.pairs = tiles * c;
      last = shared;
    }
  }
  pl.cost = size.base + whole * rounds + last;
  return pl;
}

inline PairPlan plan_pair(int64_t M, int64_t N, int64_t K, const Room& room) {
  PairPlan best;
  for (const PairSize& size : kPairSizes) {
    const PairPlan pl = plan_tiles(size, M, N, K, room);
    if (best.T == 0 || pl.cost < best.cost) best = pl;
  }
  return best;
}

// Batches that take the streaming kernel: up to 8 tokens always, and more where
// its blocks of 16 all run at one time and are done first.  A step of their warps
// takes 0.88 us, mostly latency.  Measured: 16 x 17408 x 1024 7.9 us against 15.1 in
// pairs, 64 x 5120 x 1024 6.9 and 7.5, 16 x 1152 x 8192 3.8 and 6.5; but 128 x 5120
// x 1024 9.7 and 8.3, 16 x 17408 x 5120 33.6 and 21.2, 16 x 5120 x 10240 23.2 and
// 16.9.  The estimate errs by what steps of few tiles take less: 64 x 17408 x 1024
// streams in 17.4 us and takes 15.6 in pairs.
inline bool streams(int64_t M, int64_t N, int64_t K, const Room& room) {
  if (M <= 8) return true;
  const int64_t tiles = stream16_tiles(M, N);
  if (tiles > room.tokens16[1]) return false;
  return 180 + 88 * split_stream(tiles, room.tokens16, K).steps < plan_pair(M, N, K, room).cost;
}

// The pair kernel reads fp16 codes: int8 ones from an image in the workspace.
inline size_t image_bytes(int64_t M, int64_t K) { return static_cast<size_t>(M) * K * 2; }

inline size_t plan_workspace_bytes(int64_t M, int64_t N, int64_t K, bool c16, const Room& room) {
  if (streams(M, N, K, room)) return 0;
  const PairPlan pl = plan_pair(M, N, K, room);
  return (pl.cut ? kCounterBytes + pl.part_bytes : 0) + (c16 ? 0 : image_bytes(M, K));
}

}  // namespace qlin
