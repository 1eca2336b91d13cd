// paged_attn.cu -- attention of the new tokens over the paged INT8 cache.
//
// For a row (token i of a sequence, query head h) over the tokens j it sees:
//   x_j = scale ks_j (q . kc_j)  (softcap tanh(x_j / softcap)),
//   out = sum_j exp(x_j) vs_j vc_j / sum_j exp(x_j),
// kc, vc the codes and ks, vs their scales, in one pass over the cache: sums of
// (2^(y_j - m) vs_j 2^-c) vc_j and of 2^(y_j - m), y_j = x_j log2(e), under two
// references of each row: a score m, which follows the largest so far, and a power of
// two 2^c, which follows the largest product of weight and value scale, so that this
// fits fp16 whatever the scales are, and the denominator does not depend on them.
//
// What bounds it: HBM, 264 bytes a token and key/value head, which its rows (T
// new tokens times G query heads of the group) share.
//
// The work is the list of blocks of 16 tokens of all (sequence, key/value head,
// row tile) segments, in order, cut into equal shares: a thread block takes one,
// whatever the sequences' lengths.  The parts of a segment that shares cut meet
// in a second kernel; segments inside one are finished at once.  A tile is 32 rows at
// most, and every tile of a sequence goes through all blocks that any of its new rows sees:
// made for a token or a drafted block; prompts are right, and far from what they could
// take (1 x 8192 new tokens of 32 on 8 heads: 4.65 ms).
//
// A thread block goes through its share 128 tokens at a time.  Scores are formed
// transposed, tokens x rows, warp w of four those of the tile's blocks w and w + 4:
// the key codes are operand A (m16 = a block's tokens), widened to fp16 on the way,
// and q, as fp16 times a power of two of its row, operand B (n8 = rows), in registers
// for a whole piece.  So 1 to 8 rows cost half of what rows as operand A would, and no
// code is widened twice.  The weights go as fp16 through shared memory, and the outputs
// are formed transposed too, components x rows, with the value codes as operand A: warp
// w takes 32 components.  Each warp brings its blocks of the tiles to come, one bulk
// copy a block, into a ring of tiles, where one is free behind the barrier of the tile
// after.
//
// Four warps of 255 registers and not eight of 128: with q of 32 rows read from
// shared memory by eight warps a tile, that was busy 57% of the time (12 x 8 tokens at
// 8192 65.0 us, four warps 58.8; 96 x 1 at 512 30.0 and 28.3).
//
// One barrier a tile: references are raised only where a weight, with its scale or
// without, would pass 2^15, and then to put the row's largest near 2^0, so that weights
// are formed and written as if they held, and the barrier that they need anyway says
// whether they did.  (With a running maximum exchanged before, two barriers and copies
// through one producer warp a tile took twice the time.)
//
// Where the time goes (two thread blocks an SM): with 32 rows a tile of 128 tokens
// takes one of them 4600 cycles, 1300 for scores, 700 weights, 300 the barrier, 700
// the copies' issue, 1200 outputs; the tensor pipe is 36% busy over the call, and the
// chain through a tile bounds it (12 x 8 tokens at 8192: 55.1 us, 2.9 TB/s; of 4 39.6).
// With 8 rows a tile takes 2200 to 3000 and the copies keep up (96 x 1 at 4096: 104.6 us, 6.0 TB/s;
// 1 x 131072: 47.1 us, 5.9 TB/s).  Beginning a share takes 4 us
// (lengths, the plan, a page, the first blocks: loads one behind the other), ending a
// piece 0.4: what short calls are made of (1 x 515: 6.4 us).
//
// mma.sync, not tcgen05: its operands come from registers, where the codes are
// widened; tcgen05's would have to be written to shared or tensor memory first,
// and the rows, mostly 4 to 32, fill a fraction of its tile.
//
// Precision.  Codes are exact in fp16, and so is q up to 2^-39 of its row's
// largest component.  The largest product of a weight and its value scale that a row
// has seen stands between 1 and 2^15, so these products have fp16's 11 bits down to
// 2^-14 of it, and are at most a step of 2^-24 off below that.  There a product gets,
// before it is rounded, up to half a step more or less, by its token: of the products that
// fall between two steps as many round up as their place between them says, so that a long
// tail of small ones, alike or not, has its sum (without that the sum of 131072 at 2^-20.7
// of the first was 5% off, at 2^-25.5 nothing).  Scores, weights, sums and outputs are
// fp32; a weight is 0 below 2^-126 of the row's largest.
#include <cfloat>

#include <algorithm>
#include <atomic>

#include <cuda_fp16.h>

#include "f32x2.cuh"
#include "kv_cache.cuh"

namespace qlin {
namespace {

constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = 32 * kAttnWarps;
constexpr int kTileBlocks = 8;      // of 16 tokens, of a tile
constexpr int kOf = kTileBlocks / kAttnWarps;     // of them that a warp scores: w, w + 4
constexpr int kTile = 16 * kTileBlocks;
constexpr int kMinShare = kTileBlocks;
constexpr int kPStride = 288;       // bytes of a row of weights: rows 32 bytes apart mod 128
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr float kNone = -FLT_MAX;     // reference of a row that has seen nothing: no score is below it
// Weights times their scales: what a row's references may let through (of the weights
// by themselves too), the logarithm of what a reference set in passing is lifted at, and
// of a power of two above the row's largest, not more than four times that, where one is
// set: 13 apart, so that few tiles set one, and not more, so that what is rounded to a step
// of 2^-24 is small beside the row's largest (12 x 8 tokens at 8192: 13 apart 56.6 us, 11
// apart 57.6, 9 apart 58.8).
constexpr float kMostWeight = 32768.0f;
constexpr float kLiftWeight = 4.0f;
constexpr float kNewWeight = 2.0f;
constexpr float kMostScale = 126.0f;      // c is between this and its negative

template <int NR, int kPerSm>
struct Shape {
  static constexpr int kRows = 8 * NR;
  static constexpr int kRowsOf = kRows / kAttnWarps;    // whose q a warp brings
  // Blocks in the ring: whole tiles, as many as the thread blocks of an SM have room
  // for.  A tile's blocks are sent when the one two (three) before is done, which with
  // few rows, whose tiles are short, is late in a ring of two tiles (96 x 1 at 4096 134 us,
  // 104 in three; 12 x 4 at 8192 44.4 and 40.7).
  static constexpr int kSlots = kPerSm == 2 && NR <= 2 ? 24 : 16;
  static_assert(kSlots % kTileBlocks == 0, "whole tiles");
  // shared memory, in order
  // weights of two tiles; and, where a piece begins, its q, in the place of its first tile's
  static constexpr int kP = kSlots * kCacheBlock;
  static constexpr int kPair = kP + 2 * kRows * kPStride;      // float2 [warps][rows]: references; sums
  static constexpr int kRef = kPair + kAttnWarps * kRows * 8;     // float4 [rows / 2]: two rows' references
  static constexpr int kKeep = kRef + kRows * 8;         // float2 [rows]: what raised references leave of the sums, of the outputs
  static constexpr int kFactor = kKeep + kRows * 8;      // fp32 [rows]
  // of two pieces:
  static constexpr int kTo = kFactor + kRows * 4;        // int32 [rows]: the row's head of the sequence's outputs, -1: none
  static constexpr int kLow = kTo + 2 * kRows * 4;       // int32 [rows]: first token seen
  static constexpr int kHigh = kLow + 2 * kRows * 4;     // and the one behind the last
  static constexpr int kBytes = kHigh + 2 * kRows * 4;
};

// A row's references m and 2^c and the sum of weights under m, of a part of its tokens.
struct alignas(16) Share {
  float m, c, l, none;
};

struct AttnParams {
  PagedAttnArgs a;
  int G;               // query heads of a key/value head
  int row_tiles;       // of a sequence's T * G rows
  bool planned;        // Plan is used; then
  int each;            // thread blocks of a segment, 0: fewer than segments
  // Quotients by these come from products (a division is a chain of 20 instructions,
  // and a share's beginning one of such chains): 2^40, 2^36, 2^40 and 2^38 over each,
  // rounded up
  uint64_t per_grid, per_each, per_group, per_page;
  float cap, per_cap;  // of scores times log2(e); 1 / softcap
  int* err;
  // workspace: where the cut segments are, then their parts
  int32_t* cuts;       // [grid][8]: segment (-1: none), its first and last share, sequence and its new tokens
  Share* part_share;   // [2 grid][rows]
  float* part_o;       // [2 grid][rows][128]
};

// x / d with m = 2^s / d rounded up: exact where x (d - 1) is below 2^s and x m below 2^64.
__device__ __forceinline__ int over(int x, uint64_t m, int s) { return static_cast<int>(static_cast<uint32_t>(x) * m >> s); }

// x / d where that is below 2^16 (fp32's quotient is then less than one off)
__device__ __forceinline__ int few_times(int x, int d) {
  const int q = static_cast<int>(__fdividef(static_cast<float>(x), static_cast<float>(d)));
  const int rest = x - q * d;
  return rest < 0 ? q - 1 : rest >= d ? q + 1 : q;
}

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
__device__ __forceinline__ int64_t share_of(const AttnParams& p, int64_t total, int grid) {
  const int64_t share = total < 1LL << 30 ? over(static_cast<int>(total) + grid - 1, p.per_grid, 40) : (total + grid - 1) / grid;
  return share < kMinShare ? kMinShare : share;
}

// The share that block `at` is in (of fewer than 2^16).
__device__ __forceinline__ int share_at(int64_t at, int64_t share) {
  return at < 1LL << 30 ? few_times(static_cast<int>(at), static_cast<int>(share)) : static_cast<int>(at / share);
}

// Segments that can be of eight parts and more each.
__host__ __device__ inline bool few_segments(int64_t segments, int64_t grid) { return 8 * segments <= grid; }

// How the work of up to 32 sequences, less than 2^31 blocks, is shared out; each
// warp finds it by itself, lane by sequence.  Either every thread block takes
// `share` blocks of the list, or (own) segments are cut into parts of their own: a
// thread block that holds parts of two begins and ends two pieces, 1 to 2 us more
// than the others.  Then the share is the smallest for which the parts,
// ceil(n_s / share) of a segment of n_s blocks, are no more than the thread blocks.
// That is done where it is at most kPieceBlocks over the even one (12 x 8 rows in a
// window of 2048, 2 over 41: 24.5 us, 27.0 with even shares; of 1000 tokens 17.4 and
// 19.2; at 8192, 15 over 126, 54.2 and 53.9), and where segments are few (then it is
// less than grid / (grid - segments) times the even one).
constexpr int kPieceBlocks = 5;
struct Plan {
  SeqLen seq;              // the lane's
  int share, blocks;       // of a thread block, of all
  bool own;
  int parts;               // of the lane's sequence's segments; blocks where not own
  int before;              // of the sequences before, for one segment

  __device__ __forceinline__ Plan(const AttnParams& p, int grid, int lane) {
    const int B = static_cast<int>(p.a.c.B), segs = p.row_tiles * static_cast<int>(p.a.c.kv_heads);
    seq = lane < B ? seq_len(p.a.c, lane, p.a.T) : SeqLen{0, 0};
    const int n = span_of(p.a, seq).count;
    blocks = __reduce_add_sync(kAll, n) * segs;
    // (exact: blocks are less than 2^31, and grid times that less than 2^40)
    const int even = max(over(blocks + grid - 1, p.per_grid, 40), kMinShare);
    const bool few = few_segments(B * segs, grid);
    share = even;
    own = false;
    if (p.each > 0) {
      // as many parts of each: enough, and hardly more where lengths are alike
      int lo = even, hi = max(over(__reduce_max_sync(kAll, n) + p.each - 1, p.per_each, 36), even);
      if (hi <= lo + 2) lo = hi;
      if (!few && hi > lo + kPieceBlocks) hi = lo + kPieceBlocks + 1;      // not taken
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (__reduce_add_sync(kAll, few_times(n + mid - 1, mid)) * segs <= grid) hi = mid;
        else lo = mid + 1;
      }
      own = few || lo <= even + kPieceBlocks;
      if (own) share = lo;
    }
    parts = own ? few_times(n + share - 1, share) : n;      // (shares are n / grid and more)
    int incl = parts;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kAll, incl, o);
      if (lane >= o) incl += v;
    }
    before = incl - parts;
  }
  // Where thread block c begins: sequence, segment, part (own) or block of it, and
  // of how many; false: nowhere
  __device__ __forceinline__ bool find(int c, int segs, int& b, int& seg, int& at, int& of) const {
    const int in_b = (own ? c : c * share) - before * segs;
    const uint32_t who = __ballot_sync(kAll, in_b >= 0 && in_b < parts * segs);
    if (who == 0) return false;
    b = __ffs(who) - 1;
    const int in = __shfl_sync(kAll, in_b, b);
    of = __shfl_sync(kAll, parts, b);
    seg = segs < 1 << 16 ? few_times(in, of) : in / of;
    at = in - seg * of;
    return true;
  }
};

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
  // total and fresh: total_len and new_len of the sequence behind b, read long before
  __device__ __forceinline__ void next(const PagedAttnArgs& a, int& total, int& fresh) {
    const int n = piece();
    left -= n;
    off += n;
    if (left == 0 || off < span.count) return;
    off = 0;
    if (++seg < segs) return;
    seg = 0;
    ++b;
    seq = seq_of(a.c, a.T, total, fresh);
    span = span_of(a, seq);
    while (span.count == 0) {      // more blocks are to come, so there is one
      ++b;
      load(a);
    }
    look_behind(a, total, fresh);
  }
  __device__ __forceinline__ void look_behind(const PagedAttnArgs& a, int& total, int& fresh) const {
    if (b + 1 < a.c.B) {
      total = __ldcg(a.c.total_len + b + 1);
      fresh = fresh_of(a.c, b + 1);
    }
  }
};

// A piece that the copies have come to, for when its tiles are gone through.
struct alignas(16) Piece {
  int64_t b;
  int seg, len, fresh;
  int cut;             // its first block of the segment
  int n;               // blocks of 16
  int j0;              // first token
  bool whole, final;   // it is a segment; the last one of the share
};
constexpr int kPieces = 8;      // more than the copies look ahead
constexpr int kTilesAhead = 4;  // and tiles, this one among them

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// cap tanh(x / cap) of four, 2^-20 of it off at most.  With y = |x| / cap:
// below 0.6 y + y^3 p(y^2), p of degree 4 fitted to it (2^-28); from there on
// 1 - 2 / (1 + e^2y), which would cancel below (at 0.6, where tanh is 0.537: e^2y 1.6
// steps of 2^-22 off by its argument and ex2, its sum half, the quotient of 0.463 one by
// its division: 1.2 in all), with the sign of x (for y below 0 it would cancel too, and
// be twice as far off).  Scores are mostly well below their
// caps, so a warp forms the second only where one of its scores needs it (12 x 8 tokens,
// all at 8192: 79.0 us under a cap of 30, 80.2 under one of 2, 71.2 without a cap).
constexpr float kSmall = 0.6f;
__device__ __forceinline__ void cap_scores(float (&v)[4], float cap, float per_cap) {
  float y[4], most = 0.0f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    y[k] = v[k] * per_cap;
    most = fmaxf(most, fabsf(y[k]));
    const float z = y[k] * y[k];
    float s = fmaf(z, -5.940188188e-3f, 2.083871700e-2f);
    s = fmaf(z, s, -5.379820615e-2f);
    s = fmaf(z, s, 1.333212405e-1f);
    s = fmaf(z, s, -3.333330750e-1f);
    v[k] = fmaf(y[k] * z, s, y[k]);
  }
  if (__any_sync(kAll, most >= kSmall)) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float l = 1.0f - __fdividef(2.0f, 1.0f + ex2(fabsf(y[k]) * (2.0f * kLog2e)));
      v[k] = fabsf(y[k]) < kSmall ? v[k] : copysignf(l, y[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] *= cap;
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

// log2 of a power of two above |v|, -126 for all smaller ones
__device__ __forceinline__ float log2_above(float v) {
  return static_cast<float>(static_cast<int>(__float_as_uint(v) >> 23 & 255u) - 126);
}

// 2^c, c whole and between -126 and 127
__device__ __forceinline__ float power_of_two(float c) { return __uint_as_float(static_cast<uint32_t>(static_cast<int>(c) + 127) << 23); }
// and c of it
__device__ __forceinline__ float log2_of(float f) { return static_cast<float>(static_cast<int>(__float_as_uint(f) >> 23) - 127); }

template <int NR, bool kCap, int kPerSm>
__global__ void __launch_bounds__(kAttnThreads, kPerSm) attn_kernel(const AttnParams p) {
  using S = Shape<NR, kPerSm>;
  constexpr int kSlots = S::kSlots, kRowsOf = S::kRowsOf;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kTilesAhead];    // a tile's blocks are there
  __shared__ Walk aheads[kAttnWarps];       // of each warp's copies
  __shared__ Piece pieces[kPieces];
  __shared__ Walk start;
  __shared__ int abort_flag;
  __shared__ int64_t warp_sums[kAttnWarps];
  const PagedAttnArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int segs = p.row_tiles * static_cast<int>(a.c.kv_heads);

  if (tid == 0) {
    abort_flag = 0;
    for (int i = 0; i < kTilesAhead; ++i) mbar_init(smem_u32(&full[i]), kTileBlocks);
    fence_barrier_init();
  }
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();      // (the joining kernel may read what this one's predecessors wrote at once)

  // ---- this block's share
  Walk walk;
  walk.segs = segs;
  if (p.planned) {
    const Plan plan(p, gridDim.x, lane);
    const int c = blockIdx.x;
    int b = 0, seg = 0, piece_at = 0, of = 1;
    const bool mine = plan.find(c, segs, b, seg, piece_at, of);
    // the first boundary inside a segment announces it
    int4 cut = make_int4(-1, 0, 0, b);
    if (mine) {
      walk.b = b;
      walk.seg = seg;
      walk.seq = SeqLen{__shfl_sync(kAll, plan.seq.len, b), __shfl_sync(kAll, plan.seq.fresh, b)};
      walk.span = span_of(a, walk.seq);
      if (plan.own) {
        walk.off = piece_at * plan.share;
        walk.left = min(walk.span.count - walk.off, plan.share);
        if (piece_at == 1) cut = make_int4(seg, c - 1, c - 2 + of, b);
      } else {
        const int from = c * plan.share;
        walk.off = piece_at;
        walk.left = min(plan.blocks - from, plan.share);
        if (piece_at > 0 && piece_at <= plan.share) cut = make_int4(seg, c - 1, few_times(from - piece_at + of - 1, plan.share), b);
      }
    }
    if (tid == 0) {
      *reinterpret_cast<int4*>(p.cuts + 8 * c) = cut;
      p.cuts[8 * c + 4] = walk.seq.fresh;
    }
    if (!mine) return;
  } else {
    // Blocks of 16 of as many sequences as threads at a time: their running sum, which places
    // the share, and what they are in all.
    SeqLen seq{0, 0};      // the thread's
    auto chunk = [&](int64_t b0, int& n, int64_t& incl, int64_t& all) {
      const int64_t b = b0 + tid;
      seq = b < a.c.B ? seq_len(a.c, b, a.T) : SeqLen{0, 0};
      n = span_of(a, seq).count;
      uint32_t in_warp = static_cast<uint32_t>(n);      // 32 spans of 2^26 blocks at most
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(kAll, in_warp, o);
        if (lane >= o) in_warp += v;
      }
      if (lane == 31) warp_sums[warp] = in_warp;
      incl = in_warp;
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
    const int64_t share = share_of(p, total, gridDim.x);
    const int64_t at = blockIdx.x * share;
    if (at >= total) {
      if (tid == 0) p.cuts[8 * blockIdx.x] = -1;
      return;
    }
    for (int64_t b0 = 0, before = 0;; b0 += kAttnThreads) {
      if (a.c.B > kAttnThreads) chunk(b0, n0, incl, all);
      const int64_t from = (before + incl - n0) * segs;
      if (n0 > 0 && from <= at && at < from + static_cast<int64_t>(n0) * segs) {
        start.b = b0 + tid;
        start.segs = segs;
        const int64_t in_b = at - from;
        start.seg = in_b < 1LL << 30 && segs < 1 << 16 ? few_times(static_cast<int>(in_b), n0) : static_cast<int>(in_b / n0);
        start.off = static_cast<int>(in_b - static_cast<int64_t>(start.seg) * n0);
        start.left = total - at < share ? total - at : share;
        start.seq = seq;
        start.span = span_of(a, seq);
        // the first boundary inside a segment announces it
        const int64_t s0 = from + static_cast<int64_t>(start.seg) * n0;
        const int first = share_at(s0, share), last = share_at(s0 + n0 - 1, share);
        p.cuts[8 * blockIdx.x + 4] = seq.fresh;
        *reinterpret_cast<int4*>(p.cuts + 8 * blockIdx.x) =
            make_int4(start.off > 0 && first == static_cast<int>(blockIdx.x) - 1 ? start.seg : -1, first, last, static_cast<int>(start.b));
      }
      before += all;
      if (before * segs > at) break;
    }
    __syncthreads();
    walk = start;
  }

  // A copy that does not come ends the work, not the walk through the tiles, in
  // which the warps keep meeting.
  const WaitCtx ctx{p.err, &abort_flag, kWaitLimitNs};
  bool ok = true;

  // ---- q of the piece to come, each warp's rows, brought while the piece before
  // it ends
  const int rows = static_cast<int>(a.T) * p.G;
  uint8_t* const ps = smem + S::kP;
  auto q_at = [&](int turn, int r) { return ps + (turn * S::kRows + r) * kPStride; };      // bf16, then fp16
  // lane by row: its head of the sequence's outputs, -1: none, and its new token
  int to_next = 0, token_next = 0;
  auto place = [&](int seg, int fresh, int& t) {
    const int h = p.row_tiles == 1 ? seg : seg / p.row_tiles, row = (seg - h * p.row_tiles) * S::kRows + lane;
    t = rows < 1 << 24 ? over(row, p.per_group, 40) : row / p.G;
    return lane < S::kRows && row < rows && t < fresh ? t * static_cast<int>(a.q_heads) + h * p.G + (row - t * p.G) : -1;
  };
  auto bring_q = [&](int64_t b, int to, int turn) {
    const uint16_t* const from = a.q + b * a.T * a.q_heads * kHeadDim + 8 * (lane & 15);
#pragma unroll
    for (int k = 0; k < kRowsOf; k += 2) {      // half a warp a row
      const int r = warp + kAttnWarps * (k + (lane >> 4));
      const int at = __shfl_sync(kAll, to, r);
      if (at >= 0)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(q_at(turn, r) + 16 * (lane & 15))),
                     "l"(from + static_cast<int64_t>(at) * kHeadDim)
                     : "memory");
    }
  };
  // ---- copies: this warp's blocks of each tile, one bulk copy each (whose issue
  // takes its thread 200 cycles), into the ring as soon as the tile that they displace
  // is done.  The pages of 32 tiles are read at once, lane by tile.
  Walk& ahead = aheads[warp];
  const int per_page = static_cast<int>(a.c.page_size) >> 4;
  const int page_blocks = per_page * static_cast<int>(a.c.kv_heads);
  int next_i = 0, next_n = 0;        // the tile's first block of the piece, the piece's blocks
  int first = 0, head_at = 0;        // the piece's first block of the sequence; the head's first block of a page
  int page[kOf], in_head[kOf];       // lane by tile: the blocks' pages, their places in the cache but for that
  int put = 0;
  bool coming = true;
  uint32_t on_page = 0;              // bits t % kTilesAhead, kOf each: the warp's blocks of tile t are on a page
  int to_send = 0, send_slot = warp; // the tile whose block is next, and where it goes
  int behind_total = 0, behind_fresh = 0;  // lane 0: see Walk
  auto look = [&]() {                // at the pages of 32 tiles
#pragma unroll
    for (int k = 0; k < kOf; ++k) {
      const int i = next_i + kTileBlocks * lane + warp + kAttnWarps * k;
      const int n = first + i, of_table = over(n, p.per_page, 38);
      in_head[k] = head_at + n - of_table * per_page;
      page[k] = i < next_n ? __ldg(a.c.block_table + ahead.b * a.c.max_pages + of_table) : -1;
    }
  };
  auto enter = [&]() {               // ahead's piece (each warp writes the same)
    next_i = 0;
    next_n = ahead.piece();
    first = ahead.span.first + ahead.off;
    head_at = (p.row_tiles == 1 ? ahead.seg : ahead.seg / p.row_tiles) * per_page;
    look();
    if (lane == 0)
      pieces[put] = Piece{ahead.b, ahead.seg, ahead.seq.len, ahead.seq.fresh, ahead.off, next_n, 16 * first, next_n == ahead.span.count,
                          next_n == ahead.left};
    put = (put + 1) % kPieces;
  };
  // tile: the one whose predecessors are done
  auto send = [&](int tile) {
    if (!coming || kTileBlocks * to_send >= kTileBlocks * tile + kSlots) return;
    const int from = next_i / kTileBlocks % 32;
    const int of = to_send % kTilesAhead;
#pragma unroll
    for (int k = 0; k < kOf; ++k) {
      const int on = __shfl_sync(kAll, page[k], from), in = __shfl_sync(kAll, in_head[k], from);
      const bool real = on >= 0 && on < a.c.pages;
      if (ok && lane == 0) {
        const uint32_t bar = smem_u32(&full[of]);
        const int slot = send_slot + kAttnWarps * k;
        mbar_arrive_expect_tx(bar, real ? kCacheBlock : 0);
        if (real)
          bulk_load(smem_u32(smem) + slot * kCacheBlock, a.c.cache + (static_cast<int64_t>(on) * page_blocks + in) * kCacheBlock,
                    kCacheBlock, bar);
      }
      const uint32_t bit = 1u << (of * kOf + k);
      on_page = (on_page & ~bit) | (real ? bit : 0u);
    }
    ++to_send;
    send_slot += kTileBlocks;
    if (send_slot >= kSlots) send_slot -= kSlots;
    next_i += kTileBlocks;
    if (next_i < next_n) {
      if (from == 31) look();
    } else {
      coming = ahead.left > next_n;
      __syncwarp();
      if (coming) {
        if (lane == 0) ahead.next(a, behind_total, behind_fresh);
        __syncwarp();
        enter();
      }
    }
  };
  if (lane == 0) {
    ahead = walk;
    walk.look_behind(a, behind_total, behind_fresh);
  }
  __syncwarp();
  enter();
  to_next = place(walk.seg, walk.seq.fresh, token_next);
  bring_q(walk.b, to_next, 0);
  for (int i = 0; kTileBlocks * i < kSlots; ++i) send(0);
  const int g = lane >> 2, q = lane & 3;
  // Scores: tokens tok and tok + 1 of the warp's block, rows 8 r + 2 q and the
  // next one.  The tokens are such that 8 lanes' reads of keys (g = 2 u and
  // 2 u + 1, 4 chunks each) meet in no bank.
  const int tok = 2 * (g >> 1) + 8 * (g & 1);
  const int k_turn = 2 * ((tok >> 2) & 3);
  // What is added to token t's products, in steps: the bits of t % 128 backwards as a
  // fraction, so that any 2^i tokens in a row, or at equal distances of a power of two,
  // have equally spaced ones; moved in the same way from tile to tile.  Here 1 more
  // (the exponent's) and 1/2 - 1/256 as well.
  const uint32_t jitter = 0x33800000u | __brev(tok + 16 * warp) >> 25 << 16;
  constexpr float kJitterMid = 1.49609375f * 0x1p-24f;
  // Outputs: components 32 warp + 4 g .. + 3 of all rows.
  float2* const pairs = reinterpret_cast<float2*>(smem + S::kPair);
  float4* const refs = reinterpret_cast<float4*>(smem + S::kRef);
  float2* const keeps = reinterpret_cast<float2*>(smem + S::kKeep);
  int* const tos = reinterpret_cast<int*>(smem + S::kTo);
  float* const factors = reinterpret_cast<float*>(smem + S::kFactor);
  int* const lows = reinterpret_cast<int*>(smem + S::kLow);
  int* const highs = reinterpret_cast<int*>(smem + S::kHigh);

  // Of a row's references -m and 2^-c are held.
  f32x2 sum[NR];
  uint4 qb[NR][4];
  auto q_part = [&](int turn, int r, int c) {  // operand B: components 16 (q + 4 (c / 2)) + 8 (c % 2) .. + 7
    return *reinterpret_cast<const uint4*>(q_at(turn, 8 * r + g) + 32 * (q + 4 * (c >> 1)) + 16 * (c & 1));
  };
  float o[2][NR][4];
  int seen_from = 0, seen_to = 0;    // tokens that all rows see

  int tile = 0, slot = 0, turn = 0, get = 0, odd = 0;      // slot: of the tile's first block
  int i = 0, n = 0, j0 = 0;          // the tile's first block of the piece, the piece's blocks, the tile's first token
  for (;;) {
    const Piece& piece = pieces[get];
    const bool begins = i >= n;
    if (begins) {
      __syncwarp();
      // q of the piece's rows, what they see
      i = 0;
      n = piece.n;
      j0 = piece.j0;
      // lane by row: its place, and what it sees
      odd ^= 1;
      const int to = to_next;
      const bool real = to >= 0;
      const int len = piece.len, token = len - piece.fresh + token_next;
      const int64_t w = a.window > 0 ? a.window : 1LL << 40;
      const int low = real && token - w + 1 > 0 ? static_cast<int>(token - w + 1) : 0;
      const int high = !real ? 0 : a.causal ? token + 1 : token + w < len ? static_cast<int>(token + w) : len;
      seen_from = __reduce_max_sync(kAll, low);
      seen_to = __reduce_min_sync(kAll, real ? high : len);
      if (warp == 0 && lane < S::kRows) {
        tos[odd * S::kRows + lane] = to;
        lows[odd * S::kRows + lane] = low;
        highs[odd * S::kRows + lane] = high;
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
      uint2 x[kRowsOf];
#pragma unroll
      for (int k = 0; k < kRowsOf; ++k) {
        const int r = warp + kAttnWarps * k;
        x[k] = __shfl_sync(kAll, to, r) >= 0 ? *reinterpret_cast<const uint2*>(q_at(turn, r) + 8 * lane) : make_uint2(0, 0);
      }
#pragma unroll
      for (int k = 0; k < kRowsOf; ++k) {
        const int r = warp + kAttnWarps * k;
        const float f[4] = {__uint_as_float(x[k].x << 16), __uint_as_float(x[k].x & 0xFFFF0000u), __uint_as_float(x[k].y << 16),
                            __uint_as_float(x[k].y & 0xFFFF0000u)};
        // the largest exponent (of finite numbers' bits the order is that of the numbers)
        const uint32_t most = __reduce_max_sync(kAll, max(max(x[k].x << 16 & 0x7F800000u, x[k].x & 0x7F800000u),
                                                          max(x[k].y << 16 & 0x7F800000u, x[k].y & 0x7F800000u)));
        // into [2^14, 2^15)
        const int e = min(max(static_cast<int>(most >> 23), 27), 254);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 + 127 - e) << 23);
        const __half2 lo = __floats2half2_rn(f[0] * up, f[1] * up), hi = __floats2half2_rn(f[2] * up, f[3] * up);
        *reinterpret_cast<uint2*>(q_at(turn, r) + 8 * lane) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
        if (lane == 0) factors[r] = a.scale * __uint_as_float(static_cast<uint32_t>(e - 14) << 23) * (kCap ? 1.0f : kLog2e);
      }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < NR; ++r) {
#pragma unroll
        for (int c = 0; c < 4; ++c) qb[r][c] = q_part(turn, r, c);
      }
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        sum[r] = both(0.0f);
#pragma unroll
        for (int c = 0; c < 4; ++c) o[0][r][c] = o[1][r][c] = 0.0f;
      }
    }

    ok = ok && mbar_wait(smem_u32(&full[tile % kTilesAhead]), tile / kTilesAhead & 1, ctx, 91);
    // Whether all rows see all of the warp's block.  Elsewhere what a row does not
    // see gets no weight; a block that is not there is gone through all the same, as
    // whatever finite codes stand in its place.
    bool here[kOf], all_seen = true;
#pragma unroll
    for (int k = 0; k < kOf; ++k) {
      here[k] = ok && (on_page >> (tile % kTilesAhead * kOf + k) & 1u);
      const int j = j0 + 16 * (warp + kAttnWarps * k);
      all_seen = all_seen && here[k] && j >= seen_from && j + 16 <= seen_to;
    }

    // ---- scores times log2(e)
    f32x2 x[kOf][NR][2];
    float2 vs[kOf];
    {
      const uint8_t* keys[kOf];
      float s[kOf][NR][4];
#pragma unroll
      for (int k = 0; k < kOf; ++k) {
        keys[k] = smem + (slot + warp + kAttnWarps * k) * kCacheBlock;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
#pragma unroll
          for (int c = 0; c < 4; ++c) s[k][r][c] = 0.0f;
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int k = 0; k < kOf; ++k) {
          const uint4 ka = *reinterpret_cast<const uint4*>(keys[k] + tok * kHeadDim + 16 * ((q + 4 * c) ^ k_turn));
          const uint4 kb = *reinterpret_cast<const uint4*>(keys[k] + (tok + 1) * kHeadDim + 16 * ((q + 4 * c) ^ k_turn));
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
          for (int r = 0; r < NR; ++r) {
            const uint4 b0 = qb[r][2 * c], b1 = qb[r][2 * c + 1];
            mma(s[k][r], fa[0], b0.x, b0.y);
            mma(s[k][r], fa[1], b0.z, b0.w);
            mma(s[k][r], fa[2], b1.x, b1.y);
            mma(s[k][r], fa[3], b1.z, b1.w);
          }
        }
      }
      float2 ks[kOf];
#pragma unroll
      for (int k = 0; k < kOf; ++k) {
        ks[k] = *reinterpret_cast<const float2*>(keys[k] + kKScales + 4 * tok);
        // (an infinite one gives NaN: its scores would be infinite, of weight 0, or at a cap)
        ks[k] = make_float2(__fmaf_rn(ks[k].x, 0.0f, ks[k].x), __fmaf_rn(ks[k].y, 0.0f, ks[k].y));
        vs[k] = *reinterpret_cast<const float2*>(keys[k] + kVScales + 4 * tok);
      }
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float2 f = *reinterpret_cast<const float2*>(factors + 8 * r + 2 * q);
#pragma unroll
        for (int k = 0; k < kOf; ++k) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
            x[k][r][c] = mul2(mul2(pack2(s[k][r][2 * c], s[k][r][2 * c + 1]), pack2(f.x, f.y)), both(c == 0 ? ks[k].x : ks[k].y));
          if constexpr (kCap) {
            float v[4];
            unpack2(x[k][r][0], v[0], v[1]);
            unpack2(x[k][r][1], v[2], v[3]);
            cap_scores(v, p.cap, p.per_cap);
            x[k][r][0] = pack2(v[0], v[1]);
            x[k][r][1] = pack2(v[2], v[3]);
          }
        }
      }
    }
    if (!all_seen) {
#pragma unroll
      for (int k = 0; k < kOf; ++k) {
        if (!here[k]) vs[k] = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const int2 lo = *reinterpret_cast<const int2*>(lows + odd * S::kRows + 8 * r + 2 * q);
          const int2 hi = *reinterpret_cast<const int2*>(highs + odd * S::kRows + 8 * r + 2 * q);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int at = j0 + 16 * (warp + kAttnWarps * k) + tok + c;
            float v0, v1;
            unpack2(x[k][r][c], v0, v1);
            x[k][r][c] = pack2(here[k] && at >= lo.x && at < hi.x ? v0 : -INFINITY, here[k] && at >= lo.y && at < hi.y ? v1 : -INFINITY);
          }
        }
      }
    }
    // ---- weights, as if the references held
    uint8_t* const weights = ps + turn * (S::kRows * kPStride);
    f32x2 more[kOf][2], part[NR];
    {
      const uint32_t moved = __brev(tile) >> 25 << 16;
#pragma unroll
      for (int k = 0; k < kOf; ++k) {
#pragma unroll
        for (int c = 0; c < 2; ++c) more[k][c] = both(__uint_as_float(jitter + (k << 16) ^ moved ^ c << 22) - kJitterMid);
      }
    }
    for (bool raised = false;; raised = true) {
      // (a piece's first tile has no references yet)
      if (raised || !begins) {
        float most = 0.0f;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const ulonglong2 ref = *reinterpret_cast<const ulonglong2*>(refs + 4 * r + q);
#pragma unroll
          for (int k = 0; k < kOf; ++k) {
            float w[4];
            unpack2(add2(x[k][r][0], ref.x), w[0], w[1]);
            unpack2(add2(x[k][r][1], ref.x), w[2], w[3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = ex2(w[e]);
            const f32x2 p0 = pack2(w[0], w[1]), p1 = pack2(w[2], w[3]);
            part[r] = k == 0 ? add2(p0, p1) : add2(part[r], add2(p0, p1));
            // (2^-c last: no product with a finite scale is then NaN)
            unpack2(fma2(mul2(p0, both(vs[k].x)), ref.y, more[k][0]), w[0], w[1]);
            unpack2(fma2(mul2(p1, both(vs[k].y)), ref.y, more[k][1]), w[2], w[3]);
            if (!all_seen) {      // hidden weights 0, whatever the scale holds
              float v[4];
              unpack2(x[k][r][0], v[0], v[1]);
              unpack2(x[k][r][1], v[2], v[3]);
#pragma unroll
              for (int e = 0; e < 4; ++e) w[e] = v[e] == -INFINITY ? 0.0f : w[e];
            }
            most = fmaxf(most, fmaxf(fmaxf(fabsf(w[0]), fabsf(w[1])), fmaxf(fabsf(w[2]), fabsf(w[3]))));
            uint8_t* const to = weights + (8 * r + 2 * q) * kPStride + 2 * (16 * (warp + kAttnWarps * k) + tok);
            *reinterpret_cast<__half2*>(to) = __floats2half2_rn(w[0], w[2]);
            *reinterpret_cast<__half2*>(to + kPStride) = __floats2half2_rn(w[1], w[3]);
          }
          float p0, p1;
          unpack2(part[r], p0, p1);
          most = fmaxf(most, fmaxf(p0, p1));
        }
        // (behind this barrier all warps are done with the tile before this one)
        const bool raise = __syncthreads_or(most > kMostWeight) != 0;
        if (raised || !raise) break;
      }
      // References of the rows concerned up, what stands under them down.  Each
      // warp's largest score and, over that, weight times scale of a row; then the
      // warps', lane by row.
      float lv[kOf][2];
#pragma unroll
      for (int k = 0; k < kOf; ++k) lv[k][0] = log2_above(vs[k].x), lv[k][1] = log2_above(vs[k].y);
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        float v[kOf][4];
#pragma unroll
        for (int k = 0; k < kOf; ++k) unpack2(x[k][r][0], v[k][0], v[k][1]), unpack2(x[k][r][1], v[k][2], v[k][3]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = -INFINITY, over = -INFINITY;
#pragma unroll
          for (int k = 0; k < kOf; ++k) top = fmaxf(top, fmaxf(v[k][e], v[k][2 + e]));
          top = max_over_g(top);
          if (top == -INFINITY) top = kNone;
#pragma unroll
          for (int k = 0; k < kOf; ++k) over = fmaxf(over, fmaxf(v[k][e] - top + lv[k][0], v[k][2 + e] - top + lv[k][1]));
          over = max_over_g(over);
          if (g == 0) pairs[warp * S::kRows + 8 * r + 2 * q + e] = make_float2(top, over);
        }
      }
      __syncthreads();
      float most = kNone, over = -INFINITY;
      if (lane < S::kRows) {
        float2 of[kAttnWarps];
#pragma unroll
        for (int w = 0; w < kAttnWarps; ++w) {
          of[w] = pairs[w * S::kRows + lane];
          most = fmaxf(most, of[w].x);
        }
#pragma unroll
        for (int w = 0; w < kAttnWarps; ++w) over = fmaxf(over, (of[w].x - most) + of[w].y);
      }
      float* const ref = reinterpret_cast<float*>(refs + (lane >> 1)) + (lane & 1);
      if (begins) {      // (each warp writes the same; nothing stands under them)
        if (lane < S::kRows) {
          ref[0] = -most;
          ref[2] = over == -INFINITY ? 1.0f : power_of_two(fminf(fmaxf(kNewWeight - ceilf(over), -kMostScale), kMostScale));
        }
        __syncwarp();
        continue;
      }
      if (warp == 0 && lane < S::kRows) {
        const float m = -ref[0], c = -log2_of(ref[2]);
        // m up wherever it is below a score, so that no weight passes 1: by a whole number,
        // which c, where no product is larger than before, goes down by (a little more or
        // less, where fp32 rounded m, does not round it up), so that products stay where they
        // are however often m goes up; or, where nothing is left of what was, to the score
        const bool up = most > m || (most - m) + over - c > kLiftWeight;
        float2 keep = make_float2(1.0f, 1.0f);
        if (up) {
          const float rise = most - m;
          const float to = !(rise > 0.0f) ? m : rise < 0x1p20f ? m + ceilf(rise) : most, down = m - to;
          const float c_to = fminf(fmaxf(fmaxf(ceilf(over + (most - to)) - kNewWeight, ceilf(c + down - 0x1p-6f)), -kMostScale), kMostScale);
          keep = make_float2(ex2(down), ex2(down + (c - c_to)));
          ref[0] = -to;
          ref[2] = power_of_two(-c_to);
        }
        keeps[lane] = keep;
      }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float4 keep = *reinterpret_cast<const float4*>(keeps + 8 * r + 2 * q);
        sum[r] = mul2(sum[r], pack2(keep.x, keep.z));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          o[0][r][k] *= (k & 1) ? keep.w : keep.y;
          o[1][r][k] *= (k & 1) ? keep.w : keep.y;
        }
      }
    }
    // (the tile before this one is done with its weights)
    if (i + kTileBlocks >= n && !piece.final) {
      __syncwarp();
      const Piece& behind = pieces[(get + 1) % kPieces];
      to_next = place(behind.seg, behind.fresh, token_next);
      bring_q(behind.b, to_next, turn ^ 1);
    }
    fence_proxy_async_smem();
    send(tile);
#pragma unroll
    for (int r = 0; r < NR; ++r) sum[r] = add2(sum[r], part[r]);
    // ---- outputs
#pragma unroll
    for (int k = 0; k < kTileBlocks; ++k) {
      const uint8_t* const v = smem + (slot + k) * kCacheBlock + kVCodes + 4 * q * kHeadDim + 32 * (warp ^ q) + 4 * g;
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
        const uint2 b = *reinterpret_cast<const uint2*>(weights + (8 * r + g) * kPStride + 32 * k + 8 * q);
        mma(o[0][r], fa[0], b.x, b.y);
        mma(o[1][r], fa[1], b.x, b.y);
      }
    }
    turn ^= 1;
    i += kTileBlocks;
    j0 += kTile;

    if (i >= n) {
      // ---- the piece is done: sums over the warps, outputs
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        float l[2];
        unpack2(sum[r], l[0], l[1]);
#pragma unroll
        for (int d = 4; d <= 16; d <<= 1) {
          l[0] += __shfl_xor_sync(kAll, l[0], d);
          l[1] += __shfl_xor_sync(kAll, l[1], d);
        }
        if (g == 0) *reinterpret_cast<float4*>(pairs + warp * S::kRows + 8 * r + 2 * q) = make_float4(l[0], 0.0f, l[1], 0.0f);
      }
      __syncthreads();
      const bool whole = piece.whole;
      float l = 0.0f;       // lane by row
      if (lane < S::kRows) {
#pragma unroll
        for (int w = 0; w < kAttnWarps; ++w) l += pairs[w * S::kRows + lane].x;
      }
      const int64_t part = (2LL * blockIdx.x + (piece.cut > 0 ? 0 : 1)) * S::kRows;
      const float* const ref = reinterpret_cast<const float*>(refs + (lane >> 1)) + (lane & 1);
      const float c_of = lane < S::kRows ? -log2_of(ref[2]) : 0.0f;
      if (!whole && warp == 0 && lane < S::kRows) p.part_share[part + lane] = Share{-ref[0], c_of, l, 0.0f};
      // (two factors: their product may be past fp32's range)
      const float back = !whole ? 1.0f : l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);      // 0: no token seen
      const float scale = whole ? power_of_two(c_of) : 1.0f;
      uint16_t* const out = a.out + piece.b * a.T * a.q_heads * kHeadDim + 32 * warp + 4 * g;
      float* const part_o = p.part_o + part * kHeadDim + 32 * warp + 4 * g;
#pragma unroll
      for (int r = 0; r < NR; ++r) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int in_tile = 8 * r + 2 * q + c, to = tos[odd * S::kRows + in_tile];
          const float f = __shfl_sync(kAll, back, in_tile), u = __shfl_sync(kAll, scale, in_tile);
          const float4 sums = make_float4(o[0][r][c] * f * u, o[0][r][2 + c] * f * u, o[1][r][c] * f * u, o[1][r][2 + c] * f * u);
          if (to >= 0 && whole)
            *reinterpret_cast<uint2*>(out + static_cast<int64_t>(to) * kHeadDim) =
                make_uint2(bf16x2_rn(sums.x, sums.y), bf16x2_rn(sums.z, sums.w));
          if (to >= 0 && !whole) *reinterpret_cast<float4*>(part_o + in_tile * kHeadDim) = sums;
        }
      }
      if (piece.final) break;
      get = (get + 1) % kPieces;
    }
    ++tile;
    slot += kTileBlocks;
    if (slot >= kSlots) slot -= kSlots;
  }
  if (!ok) {      // what copies are still on their way land before the block ends
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < kWaitLimitNs / 100) {
    }
  }
}

// A row's parts under common references.
struct Joined {
  Share all{kNone, -200.0f, 0.0f, 0.0f};      // below every part's
  float4 o = make_float4(0, 0, 0, 0);         // components 4 lane .. + 3

  __device__ __forceinline__ void add(const Share& s, const float4& v) {
    const float m = fmaxf(all.m, s.m), was_m = all.m - m, is_m = s.m - m;
    const float was = was_m + all.c, is = is_m + s.c, c = fmaxf(was, is);
    const float f = ex2(was - c), g = ex2(is - c);
    all = Share{m, c, all.l * ex2(was_m) + s.l * ex2(is_m), 0.0f};
    o = make_float4(o.x * f + v.x * g, o.y * f + v.y * g, o.z * f + v.z * g, o.w * f + v.w * g);
  }
  // parts k, k + step, .. of those that shares first .. first + parts - 1 left
  __device__ __forceinline__ void add_parts(const AttnParams& p, int64_t first, int parts, int k, int step, int tile_rows, int in_tile,
                                            int lane) {
    constexpr int kAhead = 5;
    for (; k < parts; k += kAhead * step) {
      float4 part[kAhead], v[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int at = k + i * step;
        if (at >= parts) break;
        const int64_t slot = at == 0 ? 2 * first + 1 : 2 * (first + at);
        part[i] = __ldcg(reinterpret_cast<const float4*>(p.part_share + slot * tile_rows + in_tile));
        v[i] = __ldcg(reinterpret_cast<const float4*>(p.part_o + (slot * tile_rows + in_tile) * kHeadDim) + lane);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (k + i * step < parts) add(Share{part[i].x, part[i].y, part[i].z, 0.0f}, v[i]);
    }
  }
  __device__ __forceinline__ void store(const AttnParams& p, int64_t b, int seg, int row, int t, int lane) const {
    const float back = all.l == 0.0f ? 0.0f : __fdiv_rn(1.0f, all.l), u = ex2(all.c);
    const int64_t to = ((b * p.a.T + t) * p.a.q_heads + seg / p.row_tiles * p.G + (row - t * p.G)) * kHeadDim + 4 * lane;
    *reinterpret_cast<uint2*>(p.a.out + to) = make_uint2(bf16x2_rn(o.x * back * u, o.y * back * u), bf16x2_rn(o.z * back * u, o.w * back * u));
  }
};

// The parts of the cut segment that share x + 1 announces, a warp a row: rows 8 y to
// 8 y + 7.
__global__ void __launch_bounds__(256) join_cuts_kernel(const AttnParams p, int tile_rows) {
  const int lane = threadIdx.x & 31, in_tile = 8 * blockIdx.y + (threadIdx.x >> 5);
  grid_dep_wait();
  grid_dep_launch();
  const int4 cut = __ldcg(reinterpret_cast<const int4*>(p.cuts + 8 * (blockIdx.x + 1)));
  const int fresh = __ldcg(p.cuts + 8 * (blockIdx.x + 1) + 4);
  if (cut.x < 0) return;
  const int row = cut.x % p.row_tiles * tile_rows + in_tile, t = row / p.G;
  if (row >= static_cast<int>(p.a.T) * p.G || t >= fresh) return;
  Joined j;
  j.add_parts(p, cut.y, cut.z - cut.y + 1, 0, 1, tile_rows, in_tile, lane);
  j.store(p, cut.w, cut.x, row, t, lane);
}

// The same where there are few segments, of eight parts and more: a block takes
// row y of segment x, its warps parts.
constexpr int kJoinWarps = 8;
__global__ void __launch_bounds__(32 * kJoinWarps) join_segments_kernel(const AttnParams p, int tile_rows, int grid) {
  __shared__ float4 acc[kJoinWarps][32];
  __shared__ Share of[kJoinWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const PagedAttnArgs& a = p.a;
  // The lengths are older than the kernel in front, which starts this one when
  // its own predecessors are done.
  const Plan plan(p, grid, lane);
  const int segs = p.row_tiles * static_cast<int>(a.c.kv_heads);
  const int b = blockIdx.x / segs, seg = blockIdx.x % segs, in_tile = blockIdx.y;
  const int n = __shfl_sync(kAll, plan.parts, b), first = __shfl_sync(kAll, plan.before, b) * segs + seg * n;
  const int row = seg % p.row_tiles * tile_rows + in_tile, t = row / p.G;
  const bool none = n <= 1 || row >= static_cast<int>(a.T) * p.G || t >= seq_len(a.c, b, a.T).fresh;      // one part: written already
  grid_dep_wait();
  grid_dep_launch();
  if (none) return;
  Joined j;
  j.add_parts(p, first, n, warp, kJoinWarps, tile_rows, in_tile, lane);
  acc[warp][lane] = j.o;
  if (lane == 0) of[warp] = j.all;
  __syncthreads();
  if (warp != 0) return;
#pragma unroll
  for (int w = 1; w < kJoinWarps; ++w) j.add(of[w], acc[w][lane]);
  j.store(p, b, seg, row, t, lane);
}

// 8-row groups of a tile for `rows` rows: as few tiles of 32 rows as hold them, and as
// small ones (each reads the segment's blocks again).  12 sequences at 8192: 24 rows
// 50.9 us, 56.5 in a tile of 32; 40 rows in two of 24 81.4, in two of 32 93.3.
int row_groups(int64_t rows) {
  const int64_t tiles = (rows + 31) / 32;
  return static_cast<int>(((rows + tiles - 1) / tiles + 7) / 8);
}

// Whether three thread blocks an SM, with rings of two tiles, do better with 8 rows than
// two with rings of three: where pieces are short, so that their beginnings and ends
// overlap, as far as the host can tell from what tables have room for and the window.
// `blocks` a segment and `share` a thread block (of two an SM), us with three and two:
//   32 and 81 (96 x 1 at 512) 24.8 and 27.7;  63 and 159 (96 x 1 at 1000) 36.9 and 39.0;
//   13 and 87 (256 x 1 at 200) 33.6 and 39.6;  129 and 41 (12 x 1 in a window of 2048)
//   14.5 and 15.2;  63 and 10 (6 x 1 at 1000) 7.4 and 10.0;  250 and 53 (8 x 1 at 4000)
//   15.2 and 15.6;  125 and 316 (96 x 1 at 2000) 59.9 and 59.5;  512 and 162 (12 x 1 at 8192)
//   35.6 and 34.2.
// Few segments are joined from fewer parts (1 x 8192 10.4 and 8.9).
bool short_contexts(int64_t segments, int64_t blocks, int64_t grid) {
  if (few_segments(segments, grid) || blocks >= 400) return false;
  const int64_t share = segments < grid * 400 ? segments * blocks / grid : 400;
  return blocks + 2 * share < 400;
}

template <int NR, bool kCap, int kPerSm>
cudaError_t launch_groups(const AttnParams& p, int grid, cudaStream_t stream) {
  const auto kernel = attn_kernel<NR, kCap, kPerSm>;
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<NR, kPerSm>::kBytes);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_release);
  }
  e = launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(kAttnThreads), Shape<NR, kPerSm>::kBytes, stream, p);
  if (e != cudaSuccess) return e;
  const int64_t rows = p.a.T * p.G, segments = p.a.c.B * p.row_tiles * p.a.c.kv_heads;
  // Segments of many parts are joined by a block for each of their rows, until those
  // are more than run at once beside what is left of the attention (us so and by cuts:
  // 1 x 8192 8.8 and 15.0, 8 x 8192 13.3 and 20.5, 5 x 3 at 1000, 450 blocks, 8.65 and 9.25;
  // 4 x 4 at 1000, 512 blocks, 10.1 and 9.3, 4 x 8, 1024 blocks, 13.5 and 11.6).
  const int64_t in_tile = std::min<int64_t>(rows, 8 * NR);
  if (p.planned && few_segments(segments, grid) && segments * in_tile <= 480)
    return launch_pdl(join_segments_kernel, dim3(static_cast<unsigned>(segments), static_cast<unsigned>(in_tile)),
                      dim3(32 * kJoinWarps), 0, stream, p, 8 * NR, grid);
  return launch_pdl(join_cuts_kernel, dim3(static_cast<unsigned>(grid - 1), NR), dim3(256), 0, stream, p, 8 * NR);
}

template <int NR, int kPerSm>
cudaError_t launch_cap(const AttnParams& p, int grid, cudaStream_t stream) {
  // (a cap past 2^100 changes no score below 2^87 that fp32 can tell from its neighbour, and would overflow)
  return p.a.softcap > 0.0f && p.a.softcap < 0x1p100f ? launch_groups<NR, true, kPerSm>(p, grid, stream)
                                                         : launch_groups<NR, false, kPerSm>(p, grid, stream);
}

}  // namespace

size_t paged_attn_workspace_bytes(int64_t, int64_t T, int64_t q_heads, int64_t kv_heads, int sm_count) {
  const int groups = row_groups(T * (q_heads / kv_heads));
  const size_t grid = (groups == 1 ? 3 : 2) * static_cast<size_t>(sm_count);
  return grid * 32 + 2 * grid * 8 * groups * (sizeof(Share) + kHeadDim * sizeof(float));
}

cudaError_t launch_paged_attn(const PagedAttnArgs& a, int* err, int sm_count, cudaStream_t stream) {
  AttnParams p{};
  p.a = a;
  p.G = static_cast<int>(a.q_heads / a.c.kv_heads);
  const int groups = row_groups(a.T * p.G);
  const int64_t tiles = (a.T * p.G + 8 * groups - 1) / (8 * groups);
  if (a.T * a.q_heads > 0x7FFFFFFFLL || tiles * a.c.kv_heads > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
  p.row_tiles = static_cast<int>(tiles);
  p.err = err;
  p.a.window = std::min<int64_t>(a.window, 1LL << 40);      // (further than any token)
  p.cap = a.softcap * kLog2e;
  p.per_cap = std::min(1.0f / a.softcap, FLT_MAX);
  const int64_t segments = a.c.B * tiles * a.c.kv_heads, longest = a.c.max_pages * (a.c.page_size / 16);
  const bool three = groups == 1 && short_contexts(segments, std::min(longest, p.a.window > 0 ? (p.a.window + a.T) / 16 + 2 : longest), 2 * sm_count);
  const int grid = (three ? 3 : 2) * sm_count;
  p.planned = a.c.B <= 32 && segments <= ((1LL << 31) - 1 - 2 * kTile * grid) / longest;
  p.each = static_cast<int>(grid / segments);
  p.per_grid = ((1ULL << 40) + grid - 1) / grid;
  if (p.each > 0) p.per_each = ((1ULL << 36) + p.each - 1) / p.each;      // (of less than 2^27)
  p.per_group = ((1ULL << 40) + p.G - 1) / p.G;
  const uint64_t in_page = static_cast<uint64_t>(a.c.page_size / 16);
  p.per_page = ((1ULL << 38) + in_page - 1) / in_page;      // (2^12 blocks at most, of 2^26)
  uint8_t* const ws = static_cast<uint8_t*>(a.workspace);
  p.cuts = reinterpret_cast<int32_t*>(ws);
  p.part_o = reinterpret_cast<float*>(ws + static_cast<size_t>(grid) * 32);
  p.part_share = reinterpret_cast<Share*>(p.part_o + 2 * static_cast<size_t>(grid) * 8 * groups * kHeadDim);
  switch (groups) {
    case 1: return three ? launch_cap<1, 3>(p, grid, stream) : launch_cap<1, 2>(p, grid, stream);
    case 2: return launch_cap<2, 2>(p, grid, stream);
    case 3: return launch_cap<3, 2>(p, grid, stream);
    default: return launch_cap<4, 2>(p, grid, stream);
  }
}

}  // namespace qlin
