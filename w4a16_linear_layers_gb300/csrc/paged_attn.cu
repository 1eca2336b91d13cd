// paged_attn.cu -- attention of the new tokens over the paged INT8 cache.
//
// For a row (token i of a sequence, query head h) over the tokens j it sees:
//   x_j = scale ks_j (q . kc_j)  (softcap tanh(x_j / softcap)),
//   out = sum_j exp(x_j) vs_j vc_j / sum_j exp(x_j),
// kc, vc the codes and ks, vs their scales, in one pass over the cache: sums of
// 2^(y_j - m) (vs_j vc_j) and of 2^(y_j - m), y_j = x_j log2(e), under a
// reference m of each row that follows the largest weight so far.
//
// What bounds it: HBM, 264 bytes a token and key/value head, which its rows (T
// new tokens times G query heads of the group) share.
//
// The work is the list of blocks of 16 tokens of all (sequence, key/value head,
// row tile) segments, in order, cut into equal shares: a thread block takes one,
// whatever the sequences' lengths.  The parts of a segment that shares cut meet
// in a second kernel; segments inside one are finished at once.
//
// A warp takes every eighth block of 16 tokens of its thread block's piece, on
// its own: it brings the 4224 bytes into its slots in shared memory by one bulk
// copy each, two or three ahead, and nothing in the loop waits for another warp.
// Scores are formed transposed, tokens x rows: the codes are operand A (m16 = the
// tokens), widened to fp16 on the way, and q, as fp16 times a power of two of
// its row, operand B (n8 = rows).  So 1 to 8 rows cost half of what rows as operand
// A would.  The weights, as fp16, are transposed between the lanes (movmatrix) and
// are operand B again of the output, formed as components x rows, with the value
// codes as operand A.  The warps' sums meet when the piece is done.
//
// The reference m is raised only where a weight would pass 2^15, and then to put
// the row's largest at 2^4: no exchange between lanes elsewhere (a tile of 128
// tokens that the block's warps shared, with a running maximum exchanged through
// shared memory and the components of the output divided between them, took 118
// us for 12 x 8 rows of 32 heads over 8192 tokens).
//
// mma.sync, not tcgen05: its operands come from registers, where the codes are
// widened; tcgen05's would have to be written to shared or tensor memory first,
// and the rows, mostly 4 to 32, fill a fraction of its tile.
//
// Precision.  Codes are exact in fp16, and so is q up to 2^-39 of its row's
// largest component.  Weights have fp16's 11 bits down to 2^-17 of the row's
// largest, and are at most 2^-28 of it off below that.  Scores, sums and
// outputs are fp32.
#include <cuda_fp16.h>

#include "f32x2.cuh"
#include "kv_cache.cuh"

namespace qlin {
namespace {

constexpr int kAttnWarps = 8;
constexpr int kAttnThreads = 32 * kAttnWarps;
constexpr int kTileBlocks = 8;      // of 16 tokens, of a tile
constexpr int kTile = 16 * kTileBlocks;
constexpr int kMinShare = kTileBlocks;
constexpr int kQStride = 272;       // bytes of a row of q: rows 16 bytes apart mod 128
constexpr int kPStride = 288;       // bytes of a row of weights: rows 32 bytes apart mod 128
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr float kNone = -1e30f;     // reference of a row that has seen nothing
// Logarithms of the weights that a row's reference may let through, and of its
// largest where it is set: 11 apart, so that few tiles set one (4 apart, a third
// of the tiles of 32 rows did).
constexpr float kMostWeight = 15.0f;
constexpr float kNewWeight = 4.0f;

template <int NR>
struct Shape {
  static constexpr int kRows = 8 * NR;
  static constexpr int kParts = NR == 4 ? 2 : 1;         // row parts, shared out among the warps for the scores
  static constexpr int kGroups = NR / kParts;            // 8-row groups of a part
  static constexpr int kTokenWarps = kAttnWarps / kParts;
  static constexpr int kStages = NR == 1 ? 3 : 2;
  // shared memory, in order
  static constexpr int kRing = kStages * kTileBlocks * kCacheBlock;
  static constexpr int kQ = kRing;
  static constexpr int kP = kQ + kRows * kQStride;
  static constexpr int kO = kP + 2 * kRows * kPStride;   // fp32 [rows][128]
  static constexpr int kPair = kO + kRows * 512;         // float2 [token warps][rows]: references; sums
  static constexpr int kRef = kPair + kTokenWarps * kRows * 8;    // float2 [rows]
  static constexpr int kKeep = kRef + kRows * 8;         // fp32 [rows]
  static constexpr int kFactor = kKeep + kRows * 4;      // fp32 [rows]
  static constexpr int kLow = kFactor + kRows * 4;       // int32 [rows]: first token seen
  static constexpr int kHigh = kLow + kRows * 4;         // and the one behind the last
  static constexpr int kBytes = kHigh + kRows * 4;
};

// What a stage of the ring holds.
struct alignas(16) Tile {
  int j0;              // first token
  int blocks;          // of 16 tokens
  uint32_t there;      // bit i: block i is on a page
  uint32_t flags;
  int64_t b;
  int seg;
  int len, fresh;      // of the sequence
  int cut;             // the piece starts inside its segment
};
enum : uint32_t { kFirst = 1, kLast = 2, kWhole = 4, kFinal = 8 };   // of a piece; the piece is a segment; of the share

// A row's reference m + c and the sum under it, of a part of its tokens.
struct alignas(16) Share {
  float m, c, l, none;
  // its reference over m of others
  __device__ __forceinline__ float over(float other) const { return (m - other) + c; }
};

struct AttnParams {
  PagedAttnArgs a;
  int G;               // query heads of a key/value head
  int row_tiles;       // of a sequence's T * G rows
  int* err;
  // workspace: where the cut segments are, then their parts
  int32_t* cuts;       // [grid][4]: segment, its first and last share, sequence; segment -1: none
  Share* part_share;   // [2 grid][rows]
  float* part_o;       // [2 grid][rows][128]
};

// Blocks of 16 of a sequence that its new rows see, and the first of them.
struct Span {
  int first, count;
};
__device__ __forceinline__ Span span_of(const PagedAttnArgs& a, const SeqLen& s) {
  Span p{0, 0};
  if (s.fresh == 0) return p;
  const int64_t lo = a.window > 0 ? s.len - s.fresh + 1 - a.window : 0;
  p.first = lo > 0 ? static_cast<int>(lo >> 4) : 0;
  p.count = ((s.len + 15) >> 4) - p.first;
  return p;
}

// Blocks of 16 that each of `grid` thread blocks takes.
__device__ __forceinline__ int64_t share_of(int64_t total, int grid) {
  const int64_t share = (total + grid - 1) / grid;
  return share < kMinShare ? kMinShare : share;
}

// A walk through a share: its pieces (parts of segments), in order.
struct Walk {
  int64_t left;        // blocks of the share still to come
  int64_t b;
  int seg, segs;       // segment of the sequence (key/value head, then row tile), and how many it has
  int off;             // block of the segment
  SeqLen seq;
  Span span;

  __device__ __forceinline__ void load(const PagedAttnArgs& a) {
    seq = seq_len(a.c, b, a.T);
    span = span_of(a, seq);
  }
  __device__ __forceinline__ int piece() const {
    const int rest = span.count - off;
    return left < rest ? static_cast<int>(left) : rest;
  }
  __device__ __forceinline__ void next(const PagedAttnArgs& a) {
    const int n = piece();
    left -= n;
    off += n;
    if (left == 0 || off < span.count) return;
    off = 0;
    if (++seg < segs) return;
    seg = 0;
    do {
      ++b;
      load(a);
    } while (span.count == 0);      // more blocks are to come, so there is one
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ f32x2 both(float v) { return pack2(v, v); }

// max over the 8 lanes that share lane & 3
__device__ __forceinline__ float max_over_g(float v) {
  v = fmaxf(v, __shfl_xor_sync(kAll, v, 4));
  v = fmaxf(v, __shfl_xor_sync(kAll, v, 8));
  return fmaxf(v, __shfl_xor_sync(kAll, v, 16));
}

// log2 of a power of two above |v|; |v| below 2^-90 taken as that
__device__ __forceinline__ float log2_above(float v) {
  return static_cast<float>(max(static_cast<int>(__float_as_uint(v) >> 23 & 255u) - 126, -90));
}

template <int NR, bool kCap>
__global__ void __launch_bounds__(kAttnThreads, 2) attn_kernel(const AttnParams p) {
  using S = Shape<NR>;
  constexpr int kStages = S::kStages, kGroups = S::kGroups, kOwn = S::kParts;   // kOwn: blocks of a tile that a warp scores
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kStages];     // the stage's blocks are there
  __shared__ uint64_t told[kStages];     // its Tile is written
  __shared__ Tile tiles[kStages];
  __shared__ int abort_flag, told_abort;
  __shared__ int64_t warp_sums[kAttnWarps];
  __shared__ Walk ahead;             // of the copies
  __shared__ int64_t before_b;
  const PagedAttnArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int segs = p.row_tiles * static_cast<int>(a.c.kv_heads);

  if (tid == 0) {
    abort_flag = told_abort = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&told[i]), 1);
    }
    fence_barrier_init();
  }
  grid_dep_launch();
  grid_dep_wait();

  // ---- this block's share.  Blocks of 16 of 256 sequences at a time: their
  // running sum, which places the share, and what they are in all.
  auto chunk = [&](int64_t b0, int& n, int64_t& incl, int64_t& all) {
    const int64_t b = b0 + tid;
    n = b < a.c.B ? span_of(a, seq_len(a.c, b, a.T)).count : 0;
    incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(kAll, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    all = 0;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) {
      if (w < warp) incl += warp_sums[w];
      all += warp_sums[w];
    }
    __syncthreads();
  };
  int n0;
  int64_t incl, all;
  chunk(0, n0, incl, all);
  int64_t total = all;
  for (int64_t b0 = kAttnThreads; b0 < a.c.B; b0 += kAttnThreads) {
    int n;
    int64_t i, s;
    chunk(b0, n, i, s);
    total += s;
  }
  total *= segs;
  const int64_t share = share_of(total, gridDim.x);
  const int64_t at = blockIdx.x * share;
  if (at >= total) {
    if (tid == 0) p.cuts[4 * blockIdx.x] = -1;
    return;
  }
  for (int64_t b0 = 0, before = 0;; b0 += kAttnThreads) {
    if (b0 > 0) chunk(b0, n0, incl, all);
    const int64_t from = (before + incl - n0) * segs;
    if (n0 > 0 && from <= at && at < from + static_cast<int64_t>(n0) * segs) {
      ahead.b = b0 + tid;
      ahead.segs = segs;
      ahead.seg = static_cast<int>((at - from) / n0);
      ahead.off = static_cast<int>((at - from) % n0);
      ahead.left = total - at < share ? total - at : share;
      ahead.load(a);
      before_b = from;
    }
    before += all;
    if (before * segs > at) break;
  }
  __syncthreads();

  // A copy that does not come ends the work, not the walk through the tiles, in
  // which the warps keep meeting: they go on with tiles told to be empty.
  const WaitCtx ctx{p.err, &abort_flag, kWaitLimitNs};
  const WaitCtx told_ctx{p.err, &told_abort, 8 * kWaitLimitNs};
  bool ok = true;

  // ---- copies: warp 0's lanes bring the blocks of a tile, one each.  The next
  // tile's pages are read a tile ahead of their use.
  int ahead_i = 0;                   // of the piece
  int ahead_page = 0;
  bool ahead_more = true;
  const int per_page = static_cast<int>(a.c.page_size) >> 4;
  auto look = [&]() {
    const int i = ahead_i + lane;
    if (lane < kTileBlocks && i < ahead.piece())
      ahead_page = __ldg(a.c.block_table + ahead.b * a.c.max_pages + (ahead.span.first + ahead.off + i) / per_page);
  };
  auto fetch = [&](int stage) {      // warp 0
    if (!ahead_more) return;
    const int n = ahead.piece(), left = n - ahead_i;
    const int first = ahead.span.first + ahead.off + ahead_i;
    const bool real = ok && lane < kTileBlocks && lane < left && ahead_page >= 0 && ahead_page < a.c.pages;
    const uint32_t there = __ballot_sync(kAll, real);
    const bool last = left <= kTileBlocks, final = last && ahead.left == n;
    if (lane == 0) {
      Tile& t = tiles[stage];
      t.j0 = 16 * first;
      t.blocks = left < kTileBlocks ? left : kTileBlocks;
      t.there = there;
      t.flags = (ahead_i == 0 ? kFirst : 0u) | (last ? kLast : 0u) | (n == ahead.span.count ? kWhole : 0u) | (final ? kFinal : 0u);
      t.b = ahead.b;
      t.seg = ahead.seg;
      t.len = ahead.seq.len;
      t.fresh = ahead.seq.fresh;
      t.cut = ahead.off;
      if (ok) mbar_arrive_expect_tx(smem_u32(&full[stage]), __popc(there) * kCacheBlock);
      mbar_arrive(smem_u32(&told[stage]));
    }
    __syncwarp();
    if (real) {
      const int in_page = (first + lane) % per_page;
      bulk_load(smem_u32(smem) + (stage * kTileBlocks + lane) * kCacheBlock,
                a.c.cache + ((ahead_page * a.c.kv_heads + ahead.seg / p.row_tiles) * per_page + in_page) * kCacheBlock, kCacheBlock,
                smem_u32(&full[stage]));
    }
    ahead_i += kTileBlocks;
    ahead_more = !final;
    if (last && !final) {
      __syncwarp();
      if (lane == 0) ahead.next(a);
      ahead_i = 0;
      __syncwarp();
    }
    if (ahead_more) look();
  };
  if (warp == 0) {
    if (lane == 0) {
      // the first boundary inside a segment announces it
      const int64_t s0 = before_b + static_cast<int64_t>(ahead.seg) * ahead.span.count;
      const int64_t first = s0 / share, last = (s0 + ahead.span.count - 1) / share;
      const bool cut = ahead.off > 0 && first == blockIdx.x - 1;
      *reinterpret_cast<int4*>(p.cuts + 4 * blockIdx.x) =
          make_int4(cut ? ahead.seg : -1, static_cast<int>(first), static_cast<int>(last), static_cast<int>(ahead.b));
    }
    __syncwarp();
    look();
    for (int i = 0; i < kStages; ++i) fetch(i);
  }
  __syncthreads();

  const int g = lane >> 2, q = lane & 3;
  // Scores: tokens tok and tok + 1 of the blocks own .. own + kOwn - 1 of a tile,
  // rows 8 (group0 + r) + 2 q and the next one.  The tokens are such that 8
  // lanes' reads of keys (g = 2 u and 2 u + 1, 4 chunks each) meet in no bank.
  const int tok = 2 * (g >> 1) + 8 * (g & 1);
  const int k_turn = 2 * ((tok >> 2) & 3);
  const int own = warp / S::kParts * kOwn;
  const int group0 = warp % S::kParts * kGroups;
  // Outputs: components 32 quarter + 4 g .. + 3 of all rows, from four blocks of a tile.
  const int quarter = warp & 3, half = warp >> 2;
  uint8_t* const qs = smem + S::kQ;
  uint8_t* const ps = smem + S::kP;
  float* const os = reinterpret_cast<float*>(smem + S::kO);
  float2* const pairs = reinterpret_cast<float2*>(smem + S::kPair);
  float2* const refs = reinterpret_cast<float2*>(smem + S::kRef);
  float* const keeps = reinterpret_cast<float*>(smem + S::kKeep);
  float* const factors = reinterpret_cast<float*>(smem + S::kFactor);
  int* const lows = reinterpret_cast<int*>(smem + S::kLow);
  int* const highs = reinterpret_cast<int*>(smem + S::kHigh);
  const int rows = static_cast<int>(a.T) * p.G;

  // Of the rows that a lane scores.  The reference is a score (top, its negative)
  // plus a small number (low), so that large scores do not swallow the logarithm
  // of the value scale in it.
  f32x2 factor[kGroups], top[kGroups], low[kGroups], sum[kGroups];
  uint4 qb[kGroups][4];              // q as operand B: components 16 (q + 4 (c / 2)) + 8 (c % 2) .. + 7
  float o[2][NR][4];
  int seen_from = 0, seen_to = 0;    // tokens that all rows see

  int stage = 0, phase = 0, turn = 0;
  for (int refill = -1;; refill = stage, phase ^= stage == kStages - 1, stage = stage == kStages - 1 ? 0 : stage + 1) {
    // (the tile behind this one is told while some warps are still here, so its
    // Tile may not be looked at before)
    (void)mbar_wait(smem_u32(&told[stage]), phase, told_ctx, 90);
    const Tile& tile = tiles[stage];
    const uint32_t flags = tile.flags;
    if (flags & kFirst) {
      // q of the piece's rows, what they see
      const int fresh = tile.fresh, len = tile.len, h = tile.seg / p.row_tiles;
      const int row0 = (tile.seg - h * p.row_tiles) * S::kRows;
      const uint16_t* const from = a.q + (tile.b * a.T * a.q_heads + h * p.G) * kHeadDim;
      uint2 x[NR];
#pragma unroll
      for (int k = 0; k < NR; ++k) {
        const int row = row0 + warp + kAttnWarps * k, t = row / p.G;
        x[k] = make_uint2(0, 0);
        if (row < rows && t < fresh)
          x[k] = __ldg(reinterpret_cast<const uint2*>(from + (t * a.q_heads + (row - t * p.G)) * kHeadDim) + lane);
      }
#pragma unroll
      for (int k = 0; k < NR; ++k) {
        const int r = warp + kAttnWarps * k, row = row0 + r, t = row / p.G;
        const float f[4] = {__uint_as_float(x[k].x << 16), __uint_as_float(x[k].x & 0xFFFF0000u), __uint_as_float(x[k].y << 16),
                            __uint_as_float(x[k].y & 0xFFFF0000u)};
        float most = fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3])));
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) most = fmaxf(most, __shfl_xor_sync(kAll, most, d));
        // into [2^14, 2^15)
        const int e = min(max(static_cast<int>(__float_as_uint(most) >> 23), 27), 254);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 + 127 - e) << 23);
        const __half2 lo = __floats2half2_rn(f[0] * up, f[1] * up), hi = __floats2half2_rn(f[2] * up, f[3] * up);
        *reinterpret_cast<uint2*>(qs + r * kQStride + 8 * lane) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
        if (lane == 0) {
          factors[r] = a.scale * __uint_as_float(static_cast<uint32_t>(e - 14) << 23) * (kCap ? 1.0f : kLog2e);
          const int i = len - fresh + t;
          const int64_t w = a.window > 0 ? a.window : 1LL << 40;
          lows[r] = i - w + 1 > 0 ? static_cast<int>(i - w + 1) : 0;
          highs[r] = a.causal ? i + 1 : i + w < len ? static_cast<int>(i + w) : len;
          if (row >= rows || t >= fresh) highs[r] = 0;
        }
      }
      __syncthreads();
      const int last_row = min(min(S::kRows, rows - row0), fresh * p.G - row0) - 1;   // < 0: none
      seen_from = last_row < 0 ? 0 : lows[last_row];
      seen_to = last_row < 0 ? 0 : highs[0];
#pragma unroll
      for (int r = 0; r < kGroups; ++r) {
        const int row = 8 * (group0 + r);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          qb[r][c] = *reinterpret_cast<const uint4*>(qs + (row + g) * kQStride + 32 * (q + 4 * (c >> 1)) + 16 * (c & 1));
        const float2 f = *reinterpret_cast<const float2*>(factors + row + 2 * q);
        factor[r] = pack2(f.x, f.y);
        top[r] = both(-kNone);
        low[r] = sum[r] = both(0.0f);
      }
#pragma unroll
      for (int r = 0; r < NR; ++r) {
#pragma unroll
        for (int c = 0; c < 4; ++c) o[0][r][c] = o[1][r][c] = 0.0f;
      }
    }

    ok = __all_sync(kAll, ok && mbar_wait(smem_u32(&full[stage]), phase, ctx, 91));
    const int j0 = tile.j0;
    // All rows see all of the tile's 128 tokens.  Elsewhere what a row does not see
    // gets no weight: blocks that are not there are gone through all the same, as
    // whatever finite codes stand in their place.
    const uint32_t there = ok ? tile.there : 0u;
    const bool all_seen = there == 0xFFu && j0 >= seen_from && j0 + kTile <= seen_to;
    const uint8_t* const ring = smem + stage * kTileBlocks * kCacheBlock;

    // ---- scores times log2(e)
    f32x2 x[kOwn][kGroups][2];
    float2 vs[kOwn];
#pragma unroll
    for (int n = 0; n < kOwn; ++n) {
      const uint8_t* const blk = ring + (own + n) * kCacheBlock;
      float s[kGroups][4];
#pragma unroll
      for (int r = 0; r < kGroups; ++r) {
#pragma unroll
        for (int c = 0; c < 4; ++c) s[r][c] = 0.0f;
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint4 ka = *reinterpret_cast<const uint4*>(blk + tok * kHeadDim + 16 * ((q + 4 * c) ^ k_turn));
        const uint4 kb = *reinterpret_cast<const uint4*>(blk + (tok + 1) * kHeadDim + 16 * ((q + 4 * c) ^ k_turn));
        uint32_t fa[4][4];
        biased_u8x4_to_f16x4(ka.x, fa[0][0], fa[0][2]);
        biased_u8x4_to_f16x4(kb.x, fa[0][1], fa[0][3]);
        biased_u8x4_to_f16x4(ka.y, fa[1][0], fa[1][2]);
        biased_u8x4_to_f16x4(kb.y, fa[1][1], fa[1][3]);
        biased_u8x4_to_f16x4(ka.z, fa[2][0], fa[2][2]);
        biased_u8x4_to_f16x4(kb.z, fa[2][1], fa[2][3]);
        biased_u8x4_to_f16x4(ka.w, fa[3][0], fa[3][2]);
        biased_u8x4_to_f16x4(kb.w, fa[3][1], fa[3][3]);
#pragma unroll
        for (int r = 0; r < kGroups; ++r) {
          mma(s[r], fa[0], qb[r][2 * c].x, qb[r][2 * c].y);
          mma(s[r], fa[1], qb[r][2 * c].z, qb[r][2 * c].w);
          mma(s[r], fa[2], qb[r][2 * c + 1].x, qb[r][2 * c + 1].y);
          mma(s[r], fa[3], qb[r][2 * c + 1].z, qb[r][2 * c + 1].w);
        }
      }
      const float2 ks = *reinterpret_cast<const float2*>(blk + kKScales + 4 * tok);
      vs[n] = *reinterpret_cast<const float2*>(blk + kVScales + 4 * tok);
#pragma unroll
      for (int r = 0; r < kGroups; ++r) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          x[n][r][c] = mul2(mul2(pack2(s[r][2 * c], s[r][2 * c + 1]), factor[r]), both(c == 0 ? ks.x : ks.y));
          if constexpr (kCap) {
            // tanh(y) = 1 - 2 / (1 + e^2y), with an error of about 2^-23
            float v[2];
            unpack2(x[n][r][c], v[0], v[1]);
#pragma unroll
            for (int k = 0; k < 2; ++k)
              v[k] = a.softcap * kLog2e * (1.0f - __fdividef(2.0f, 1.0f + ex2(v[k] * (2.0f * kLog2e / a.softcap))));
            x[n][r][c] = pack2(v[0], v[1]);
          }
        }
      }
    }
    if (!all_seen) {
#pragma unroll
      for (int n = 0; n < kOwn; ++n) {
        const bool here = (there >> (own + n)) & 1u;
        const int j = j0 + 16 * (own + n) + tok;
        if (!here) vs[n] = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int r = 0; r < kGroups; ++r) {
          const int2 lo = *reinterpret_cast<const int2*>(lows + 8 * (group0 + r) + 2 * q);
          const int2 hi = *reinterpret_cast<const int2*>(highs + 8 * (group0 + r) + 2 * q);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float v0, v1;
            unpack2(x[n][r][c], v0, v1);
            x[n][r][c] = pack2(here && j + c >= lo.x && j + c < hi.x ? v0 : -INFINITY, here && j + c >= lo.y && j + c < hi.y ? v1 : -INFINITY);
          }
        }
      }
    }

    // ---- weights, as if the references held
    uint8_t* const weights = ps + turn * (S::kRows * kPStride);
    f32x2 more[kGroups];
    auto weigh = [&]() {
      float far = -INFINITY;
#pragma unroll
      for (int r = 0; r < kGroups; ++r) more[r] = both(0.0f);
#pragma unroll
      for (int n = 0; n < kOwn; ++n) {
        float most[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int r = 0; r < kGroups; ++r) {
          float w[4];
          unpack2(sub2(add2(x[n][r][0], top[r]), low[r]), w[0], w[1]);
          unpack2(sub2(add2(x[n][r][1], top[r]), low[r]), w[2], w[3]);
          most[0] = fmaxf(most[0], fmaxf(w[0], w[1]));
          most[1] = fmaxf(most[1], fmaxf(w[2], w[3]));
#pragma unroll
          for (int k = 0; k < 4; ++k) w[k] = ex2(w[k]);
          const f32x2 p0 = pack2(w[0], w[1]), p1 = pack2(w[2], w[3]);
          more[r] = add2(more[r], add2(p0, p1));
          unpack2(mul2(p0, both(vs[n].x)), w[0], w[1]);
          unpack2(mul2(p1, both(vs[n].y)), w[2], w[3]);
          if (!all_seen) {      // hidden weights 0, whatever the scale holds
            float v[4];
            unpack2(x[n][r][0], v[0], v[1]);
            unpack2(x[n][r][1], v[2], v[3]);
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = v[k] == -INFINITY ? 0.0f : w[k];
          }
          uint8_t* const to = weights + (8 * (group0 + r) + 2 * q) * kPStride + 2 * (16 * (own + n) + tok);
          *reinterpret_cast<__half2*>(to) = __floats2half2_rn(w[0], w[2]);
          *reinterpret_cast<__half2*>(to + kPStride) = __floats2half2_rn(w[1], w[3]);
        }
        far = fmaxf(far, fmaxf(most[0] + log2_above(vs[n].x), most[1] + log2_above(vs[n].y)));
      }
      return far;
    };
    // (behind this barrier all warps are done with the tile before this one, so its stage is free)
    const bool raise = __syncthreads_or(weigh() > kMostWeight) != 0;
    if (warp == 0 && refill >= 0) {
      fence_proxy_async_smem();
      fetch(refill);
    }
    if (raise) {
      // References of the rows concerned up, what stands under them down.  Each
      // warp's largest score and, over that, weight of a row; then the warps'.
#pragma unroll
      for (int r = 0; r < kGroups; ++r) {
        float most[2] = {-INFINITY, -INFINITY}, over[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int n = 0; n < kOwn; ++n) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float v[2];
            unpack2(x[n][r][c], v[0], v[1]);
            most[0] = fmaxf(most[0], v[0]);
            most[1] = fmaxf(most[1], v[1]);
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          most[k] = max_over_g(most[k]);
          if (most[k] == -INFINITY) most[k] = kNone;
        }
#pragma unroll
        for (int n = 0; n < kOwn; ++n) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float v[2];
            unpack2(x[n][r][c], v[0], v[1]);
            const float lv = log2_above(c == 0 ? vs[n].x : vs[n].y);
            over[0] = fmaxf(over[0], v[0] - most[0] + lv);
            over[1] = fmaxf(over[1], v[1] - most[1] + lv);
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          over[k] = max_over_g(over[k]);
          if (g == 0) pairs[warp / S::kParts * S::kRows + 8 * (group0 + r) + 2 * q + k] = make_float2(most[k], over[k]);
        }
      }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < kGroups; ++r) {
        float m[2], c[2], keep[2];
        unpack2(top[r], m[0], m[1]);
        unpack2(low[r], c[0], c[1]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int row = 8 * (group0 + r) + 2 * q + k;
          float2 of[S::kTokenWarps];
          float most = kNone, over = -INFINITY;
#pragma unroll
          for (int w = 0; w < S::kTokenWarps; ++w) {
            of[w] = pairs[w * S::kRows + row];
            most = fmaxf(most, of[w].x);
          }
#pragma unroll
          for (int w = 0; w < S::kTokenWarps; ++w) over = fmaxf(over, (of[w].x - most) + of[w].y);
          const bool up = (most + m[k]) + (over - c[k]) > kMostWeight;
          over -= kNewWeight;
          keep[k] = up ? ex2((c[k] - over) - (most + m[k])) : 1.0f;
          if (up) {
            m[k] = -most;
            c[k] = over;
          }
          if (warp < S::kParts && g == 0) keeps[row] = keep[k];
        }
        top[r] = pack2(m[0], m[1]);
        low[r] = pack2(c[0], c[1]);
        sum[r] = mul2(sum[r], pack2(keep[0], keep[1]));
      }
      (void)weigh();
      __syncthreads();
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float2 k = *reinterpret_cast<const float2*>(keeps + 8 * r + 2 * q);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          o[0][r][c] *= (c & 1) ? k.y : k.x;
          o[1][r][c] *= (c & 1) ? k.y : k.x;
        }
      }
    }
#pragma unroll
    for (int r = 0; r < kGroups; ++r) sum[r] = add2(sum[r], more[r]);
    // ---- outputs
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int in_tile = 4 * half + k;
      const uint8_t* const v = ring + in_tile * kCacheBlock + kVCodes + 4 * q * kHeadDim + 32 * (quarter ^ q) + 4 * g;
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = *reinterpret_cast<const uint32_t*>(v + e * kHeadDim);
      uint32_t fa[2][4];
      biased_u8x4_to_f16x4(prmt(w[0], w[1], 0x5140u), fa[0][0], fa[0][1]);
      biased_u8x4_to_f16x4(prmt(w[2], w[3], 0x5140u), fa[0][2], fa[0][3]);
      biased_u8x4_to_f16x4(prmt(w[0], w[1], 0x7362u), fa[1][0], fa[1][1]);
      biased_u8x4_to_f16x4(prmt(w[2], w[3], 0x7362u), fa[1][2], fa[1][3]);
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const uint2 b = *reinterpret_cast<const uint2*>(weights + (8 * r + g) * kPStride + 32 * in_tile + 8 * q);
        mma(o[0][r], fa[0], b.x, b.y);
        mma(o[1][r], fa[1], b.x, b.y);
      }
    }
    turn ^= 1;

    if (flags & kLast) {
      // ---- the piece is done: sums over the warps, outputs of the two halves
#pragma unroll
      for (int r = 0; r < kGroups; ++r) {
        float l[2], m[2], c[2];
        unpack2(sum[r], l[0], l[1]);
        unpack2(top[r], m[0], m[1]);
        unpack2(low[r], c[0], c[1]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int d = 4; d <= 16; d <<= 1) l[k] += __shfl_xor_sync(kAll, l[k], d);
          const int row = 8 * (group0 + r) + 2 * q + k;
          if (g == 0) pairs[warp / S::kParts * S::kRows + row].x = l[k];
          if (g == 0 && warp < S::kParts) refs[row] = make_float2(-m[k], c[k]);
        }
      }
      if (half == 1) {
#pragma unroll
        for (int r = 0; r < NR; ++r) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
            *reinterpret_cast<float4*>(os + (8 * r + 2 * q + c) * kHeadDim + 32 * quarter + 4 * g) =
                make_float4(o[0][r][c], o[0][r][2 + c], o[1][r][c], o[1][r][2 + c]);
        }
      }
      __syncthreads();
      if (half == 0) {
        const int h = tile.seg / p.row_tiles, row0 = (tile.seg - h * p.row_tiles) * S::kRows, fresh = tile.fresh;
        const int64_t part = (2LL * blockIdx.x + (tile.cut > 0 ? 0 : 1)) * S::kRows;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int in_tile = 8 * r + 2 * q + c, row = row0 + in_tile, t = row / p.G;
            if (row >= rows || t >= fresh) continue;
            float l = 0.0f;
#pragma unroll
            for (int w = 0; w < S::kTokenWarps; ++w) l += pairs[w * S::kRows + in_tile].x;
            float4 v = *reinterpret_cast<const float4*>(os + in_tile * kHeadDim + 32 * quarter + 4 * g);
            v = make_float4(o[0][r][c] + v.x, o[0][r][2 + c] + v.y, o[1][r][c] + v.z, o[1][r][2 + c] + v.w);
            const int d = 32 * quarter + 4 * g;
            if (flags & kWhole) {
              const float back = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);      // 0: no token seen
              *reinterpret_cast<uint2*>(a.out + ((tile.b * a.T + t) * a.q_heads + h * p.G + (row - t * p.G)) * kHeadDim + d) =
                  make_uint2(bf16x2_rn(v.x * back, v.y * back), bf16x2_rn(v.z * back, v.w * back));
            } else {
              *reinterpret_cast<float4*>(p.part_o + (part + in_tile) * kHeadDim + d) = v;
              if (d == 0) p.part_share[part + in_tile] = Share{refs[in_tile].x, refs[in_tile].y, l, 0.0f};
            }
          }
        }
      }
      if (flags & kFinal) break;
    }
  }
  if (!ok) {      // the copies land before the block ends
    int never = 0;
    const WaitCtx drain{p.err, &never, kWaitLimitNs};
    for (int i = 0; i < kStages; ++i) {
      (void)mbar_wait(smem_u32(&full[stage]), phase, drain, 92);
      if (--stage < 0) {
        stage = kStages - 1;
        phase ^= 1;
      }
    }
  }
}

// A row's parts under one reference.
struct Joined {
  Share all{kNone, -200.0f, 0.0f, 0.0f};      // below every part's
  float4 o = make_float4(0, 0, 0, 0);         // components 4 lane .. + 3

  __device__ __forceinline__ void add(const Share& s, const float4& v) {
    const float m = fmaxf(all.m, s.m);
    const float was = all.over(m), is = s.over(m), c = fmaxf(was, is);
    const float f = ex2(was - c), g = ex2(is - c);
    all = Share{m, c, all.l * f + s.l * g, 0.0f};
    o = make_float4(o.x * f + v.x * g, o.y * f + v.y * g, o.z * f + v.z * g, o.w * f + v.w * g);
  }
  // parts k, k + step, .. of those that shares first .. first + parts - 1 left
  __device__ __forceinline__ void add_parts(const AttnParams& p, int64_t first, int parts, int k, int step, int tile_rows, int in_tile,
                                            int lane) {
    constexpr int kAhead = 4;
    for (; k < parts; k += kAhead * step) {
      float4 part[kAhead], v[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int at = k + i * step;
        if (at >= parts) break;
        const int64_t slot = at == 0 ? 2 * first + 1 : 2 * (first + at);
        part[i] = __ldg(reinterpret_cast<const float4*>(p.part_share + slot * tile_rows + in_tile));
        v[i] = __ldg(reinterpret_cast<const float4*>(p.part_o + (slot * tile_rows + in_tile) * kHeadDim) + lane);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (k + i * step < parts) add(Share{part[i].x, part[i].y, part[i].z, 0.0f}, v[i]);
    }
  }
  __device__ __forceinline__ void store(const AttnParams& p, int64_t b, int seg, int row, int t, int lane) const {
    const float back = all.l == 0.0f ? 0.0f : __fdiv_rn(1.0f, all.l);
    const int64_t to = ((b * p.a.T + t) * p.a.q_heads + seg / p.row_tiles * p.G + (row - t * p.G)) * kHeadDim + 4 * lane;
    *reinterpret_cast<uint2*>(p.a.out + to) = make_uint2(bf16x2_rn(o.x * back, o.y * back), bf16x2_rn(o.z * back, o.w * back));
  }
};

// The parts of the cut segment that share x announces: a warp takes a row at a time.
__global__ void __launch_bounds__(256) join_cuts_kernel(const AttnParams p, int tile_rows) {
  const int lane = threadIdx.x & 31;
  grid_dep_launch();
  grid_dep_wait();
  const int4 cut = __ldg(reinterpret_cast<const int4*>(p.cuts + 4 * (blockIdx.x + 1)));
  if (cut.x < 0) return;
  const int fresh = seq_len(p.a.c, cut.w, p.a.T).fresh;
  for (int in_tile = threadIdx.x >> 5; in_tile < tile_rows; in_tile += 8) {
    const int row = cut.x % p.row_tiles * tile_rows + in_tile, t = row / p.G;
    if (row >= static_cast<int>(p.a.T) * p.G || t >= fresh) return;
    Joined j;
    j.add_parts(p, cut.y, cut.z - cut.y + 1, 0, 1, tile_rows, in_tile, lane);
    j.store(p, cut.w, cut.x, row, t, lane);
  }
}

// The same where there are few segments, of many parts each: a block takes row y
// of segment x, and finds its parts from the lengths.
__global__ void __launch_bounds__(128) join_segments_kernel(const AttnParams p, int tile_rows, int grid) {
  __shared__ float4 acc[4][32];
  __shared__ Share of[4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const PagedAttnArgs& a = p.a;
  grid_dep_launch();
  grid_dep_wait();
  const int segs = p.row_tiles * static_cast<int>(a.c.kv_heads);
  const int b = blockIdx.x / segs, seg = blockIdx.x % segs, in_tile = blockIdx.y;
  int64_t total = 0, before = 0;
  for (int i = lane; i < static_cast<int>(a.c.B); i += 32) {
    const int n = span_of(a, seq_len(a.c, i, a.T)).count;
    total += n;
    if (i < b) before += n;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    total += __shfl_xor_sync(kAll, total, o);
    before += __shfl_xor_sync(kAll, before, o);
  }
  const SeqLen seq = seq_len(a.c, b, a.T);
  const int n = span_of(a, seq).count;
  const int row = seg % p.row_tiles * tile_rows + in_tile, t = row / p.G;
  if (n == 0 || row >= static_cast<int>(a.T) * p.G || t >= seq.fresh) return;
  const int64_t share = share_of(total * segs, grid);
  const int64_t s0 = before * segs + static_cast<int64_t>(seg) * n;
  const int64_t first = s0 / share;
  const int parts = static_cast<int>((s0 + n - 1) / share - first) + 1;
  if (parts == 1) return;       // written already
  Joined j;
  j.add_parts(p, first, parts, warp, 4, tile_rows, in_tile, lane);
  acc[warp][lane] = j.o;
  if (lane == 0) of[warp] = j.all;
  __syncthreads();
  if (warp != 0) return;
#pragma unroll
  for (int w = 1; w < 4; ++w) j.add(of[w], acc[w][lane]);
  j.store(p, b, seg, row, t, lane);
}

// 8-row groups of a tile for `rows` rows: as few as hold them, four at most.
int row_groups(int64_t rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : 4; }


template <int NR, bool kCap>
cudaError_t launch_groups(const AttnParams& p, int grid, cudaStream_t stream) {
  const auto kernel = attn_kernel<NR, kCap>;
  // per call: a device's first costs nothing more, and no state is kept
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<NR>::kBytes);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(kAttnThreads), Shape<NR>::kBytes, stream, p);
  if (e != cudaSuccess) return e;
  const int64_t segments = p.a.c.B * p.row_tiles * p.a.c.kv_heads;
  if (8 * segments <= grid) {   // of eight parts and more
    const int64_t rows = p.a.T * p.G;
    return launch_pdl(join_segments_kernel, dim3(static_cast<unsigned>(segments), static_cast<unsigned>(rows < 8 * NR ? rows : 8 * NR)),
                      dim3(128), 0, stream, p, 8 * NR, grid);
  }
  return launch_pdl(join_cuts_kernel, dim3(static_cast<unsigned>(grid - 1)), dim3(256), 0, stream, p, 8 * NR);
}

template <int NR>
cudaError_t launch_cap(const AttnParams& p, int grid, cudaStream_t stream) {
  return p.a.softcap > 0.0f ? launch_groups<NR, true>(p, grid, stream) : launch_groups<NR, false>(p, grid, stream);
}

}  // namespace

size_t paged_attn_workspace_bytes(int64_t, int64_t T, int64_t q_heads, int64_t kv_heads, int sm_count) {
  const int groups = row_groups(T * (q_heads / kv_heads));
  const size_t grid = 2 * static_cast<size_t>(sm_count);
  return grid * 16 + 2 * grid * 8 * groups * (sizeof(Share) + kHeadDim * sizeof(float));
}

cudaError_t launch_paged_attn(const PagedAttnArgs& a, int* err, int sm_count, cudaStream_t stream) {
  AttnParams p{};
  p.a = a;
  p.G = static_cast<int>(a.q_heads / a.c.kv_heads);
  const int groups = row_groups(a.T * p.G);
  const int64_t tiles = (a.T * p.G + 8 * groups - 1) / (8 * groups);
  if (a.T * p.G > 0x7FFFFFFFLL || tiles * a.c.kv_heads > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
  p.row_tiles = static_cast<int>(tiles);
  p.err = err;
  const int grid = 2 * sm_count;
  uint8_t* const ws = static_cast<uint8_t*>(a.workspace);
  p.cuts = reinterpret_cast<int32_t*>(ws);
  p.part_o = reinterpret_cast<float*>(ws + static_cast<size_t>(grid) * 16);
  p.part_share = reinterpret_cast<Share*>(p.part_o + 2 * static_cast<size_t>(grid) * 8 * groups * kHeadDim);
  switch (groups) {
    case 1: return launch_cap<1>(p, grid, stream);
    case 2: return launch_cap<2>(p, grid, stream);
    default: return launch_cap<4>(p, grid, stream);
  }
}

}  // namespace qlin
