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
constexpr int kMinShare = kAttnWarps;   // blocks
constexpr int kQStride = 272;       // bytes of a row of q: rows 16 bytes apart mod 128
constexpr int kMeetStride = 36;     // floats of a row's 32 components where the warps meet: 16 bytes apart mod 128
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr float kNone = -1e30f;     // reference of a row that has seen nothing
// Logarithms of the weights that a row's reference may let through, and of its
// largest where it is set: 11 apart, so that few blocks set one (4 apart, a third
// of the blocks of 32 rows did).
constexpr float kMostWeight = 15.0f;
constexpr float kNewWeight = 4.0f;

template <int NR>
struct Shape {
  static constexpr int kRows = 8 * NR;
  static constexpr int kSlots = NR <= 2 ? 2 : 3;         // of a warp
  static constexpr int kPerSm = NR <= 2 ? 2 : 1;
  static constexpr int kRounds = NR == 1 ? 1 : 2;        // in which the outputs meet
  // shared memory, in order
  static constexpr int kRing = kAttnWarps * kSlots * kCacheBlock;
  static constexpr int kQ = kRing;
  static constexpr int kMeet = kQ + kRows * kQStride;    // fp32 [4 / rounds][warps][rows][kMeetStride]
  static constexpr int kShare = kMeet + 4 / kRounds * kAttnWarps * kRows * kMeetStride * 4;   // Share [warps][rows]
  static constexpr int kFactor = kShare + kAttnWarps * kRows * 16;    // fp32 [rows]
  static constexpr int kLow = kFactor + kRows * 4;       // int32 [rows]: first token seen
  static constexpr int kHigh = kLow + kRows * 4;         // and the one behind the last
  static constexpr int kBytes = kHigh + kRows * 4;
};

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

// An 8 x 8 matrix of fp16, row lane / 4 and columns 2 (lane % 4) and the next one a lane, transposed.
__device__ __forceinline__ uint32_t transpose(uint32_t v) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
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
__global__ void __launch_bounds__(kAttnThreads, Shape<NR>::kPerSm) attn_kernel(const AttnParams p) {
  using S = Shape<NR>;
  constexpr int kSlots = S::kSlots;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kAttnWarps][kSlots];
  __shared__ int abort_flag;
  __shared__ int64_t warp_sums[kAttnWarps];
  __shared__ Walk start;
  __shared__ int64_t before_b;
  const PagedAttnArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int kv_heads = static_cast<int>(a.c.kv_heads);
  const int segs = p.row_tiles * kv_heads;

  if (tid == 0) {
    abort_flag = 0;
    for (int w = 0; w < kAttnWarps; ++w)
      for (int i = 0; i < kSlots; ++i) mbar_init(smem_u32(&full[w][i]), 1);
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
  int64_t share = (total + gridDim.x - 1) / gridDim.x;
  if (share < kMinShare) share = kMinShare;
  const int64_t at = blockIdx.x * share;
  if (at >= total) {
    if (tid == 0) p.cuts[4 * blockIdx.x] = -1;
    return;
  }
  for (int64_t b0 = 0, before = 0;; b0 += kAttnThreads) {
    if (b0 > 0) chunk(b0, n0, incl, all);
    const int64_t from = (before + incl - n0) * segs;
    if (n0 > 0 && from <= at && at < from + static_cast<int64_t>(n0) * segs) {
      start.b = b0 + tid;
      start.segs = segs;
      start.seg = static_cast<int>((at - from) / n0);
      start.off = static_cast<int>((at - from) % n0);
      start.left = total - at < share ? total - at : share;
      start.load(a);
      before_b = from;
    }
    before += all;
    if (before * segs > at) break;
  }
  __syncthreads();
  Walk walk = start;
  if (tid == 0) {
    // the first boundary inside a segment announces it
    const int64_t s0 = before_b + static_cast<int64_t>(walk.seg) * walk.span.count;
    const int64_t first = s0 / share, last = (s0 + walk.span.count - 1) / share;
    const bool cut = walk.off > 0 && first == blockIdx.x - 1;
    *reinterpret_cast<int4*>(p.cuts + 4 * blockIdx.x) =
        make_int4(cut ? walk.seg : -1, static_cast<int>(first), static_cast<int>(last), static_cast<int>(walk.b));
  }

  const WaitCtx ctx{p.err, &abort_flag, kWaitLimitNs};
  const int g = lane >> 2, q = lane & 3;
  // Tokens of a block that a lane's scores are of: tok and tok + 2.  Taken so that
  // neither the reads of keys (8 lanes: g = 2 u and 2 u + 1, 4 chunks each) nor
  // those of values (tokens by q) meet in a bank.
  const int u = g >> 1;
  const int tok = (g & 1) ? 4 * (u ^ 2) + 1 : 4 * u;
  const int k_turn = 2 * ((tok >> 2) & 3);
  uint8_t* const qs = smem + S::kQ;
  float* const meet = reinterpret_cast<float*>(smem + S::kMeet);
  Share* const shares = reinterpret_cast<Share*>(smem + S::kShare);
  float* const factors = reinterpret_cast<float*>(smem + S::kFactor);
  int* const lows = reinterpret_cast<int*>(smem + S::kLow);
  int* const highs = reinterpret_cast<int*>(smem + S::kHigh);
  const int rows = static_cast<int>(a.T) * p.G;
  uint8_t* const ring = smem + warp * kSlots * kCacheBlock;
  const uint32_t ring_at = smem_u32(ring), full_at = smem_u32(full[warp]);

  // ---- copies: this warp's blocks, through all pieces, ahead of their use
  Walk ahead = walk;
  int ahead_i = warp;                // of the piece
  int ahead_page = -1, ahead_in_page = 0;
  const uint8_t* ahead_head = nullptr;
  bool ahead_more = true;
  const int per_page = static_cast<int>(a.c.page_size) >> 4;
  const int page_step = kAttnWarps / per_page, in_page_step = kAttnWarps % per_page;
  const int64_t head_bytes = static_cast<int64_t>(per_page) * kCacheBlock, page_bytes = head_bytes * a.c.kv_heads;
  const int32_t* table = nullptr;    // of the sequence, at the block's page
  int in_page = 0;
  const uint8_t* head_at = nullptr;  // of page 0
  auto enter = [&]() {               // the piece's first block
    const int n = ahead.span.first + ahead.off + warp, page = n / per_page;
    in_page = n - page * per_page;
    table = a.c.block_table + ahead.b * a.c.max_pages + page;
    head_at = a.c.cache + ahead.seg / p.row_tiles * head_bytes;
    ahead_i = warp;
  };
  auto look = [&]() {                // the next block's page: read long before it is needed
    while (ahead_i >= ahead.piece()) {
      ahead.next(a);
      if (ahead.left == 0) {
        ahead_more = false;
        return;
      }
      enter();
    }
    ahead_page = __ldg(table);       // (looked at in fetch: nothing waits for it here)
    ahead_in_page = in_page;
    ahead_head = head_at;
    ahead_i += kAttnWarps;
    table += page_step;
    in_page += in_page_step;
    if (in_page >= per_page) {
      in_page -= per_page;
      ++table;
    }
  };
  uint32_t there = 0;                // bit i: the block in slot i is on a page
  auto fetch = [&](int slot) {
    if (!ahead_more) return;
    const bool real = ahead_page >= 0 && ahead_page < a.c.pages;
    there = (there & ~(1u << slot)) | (real ? 1u << slot : 0u);
    if (lane == 0) {
      const uint32_t bar = full_at + 8 * slot;
      mbar_arrive_expect_tx(bar, real ? kCacheBlock : 0);
      if (real) bulk_load(ring_at + slot * kCacheBlock, ahead_head + ahead_page * page_bytes + ahead_in_page * kCacheBlock, kCacheBlock, bar);
    }
    look();
  };
  enter();
  look();
#pragma unroll
  for (int i = 0; i < kSlots; ++i) fetch(i);
  int slot = 0, phase = 0;
  bool ok = true;

  while (walk.left > 0) {
    const int n = walk.piece();
    const int h = walk.seg / p.row_tiles;
    const int row0 = (walk.seg - h * p.row_tiles) * S::kRows;
    const int64_t q_row = walk.b * a.T;
    // q of the tile's rows, what they see
    for (int r = warp; r < S::kRows; r += kAttnWarps) {
      const int row = row0 + r, t = row / p.G;
      const bool real = row < rows && t < walk.seq.fresh;
      uint2 x = make_uint2(0, 0);
      if (real)
        x = __ldg(reinterpret_cast<const uint2*>(a.q + ((q_row + t) * a.q_heads + h * p.G + (row - t * p.G)) * kHeadDim) + lane);
      const float f[4] = {__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xFFFF0000u), __uint_as_float(x.y << 16),
                          __uint_as_float(x.y & 0xFFFF0000u)};
      float top = fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3])));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
      // into [2^14, 2^15)
      const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23), 27), 254);
      const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 + 127 - e) << 23);
      const __half2 lo = __floats2half2_rn(f[0] * up, f[1] * up), hi = __floats2half2_rn(f[2] * up, f[3] * up);
      *reinterpret_cast<uint2*>(qs + r * kQStride + 8 * lane) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      if (lane == 0) {
        factors[r] = a.scale * __uint_as_float(static_cast<uint32_t>(e - 14) << 23) * (kCap ? 1.0f : kLog2e);
        const int i = walk.seq.len - walk.seq.fresh + t;
        const int64_t w = a.window > 0 ? a.window : 1LL << 40;
        lows[r] = i - w + 1 > 0 ? static_cast<int>(i - w + 1) : 0;
        highs[r] = a.causal ? i + 1 : i + w < walk.seq.len ? static_cast<int>(i + w) : walk.seq.len;
        if (!real) highs[r] = 0;
      }
    }
    __syncthreads();
    // tokens that all rows see
    const int last_row = min(min(S::kRows, rows - row0), walk.seq.fresh * p.G - row0) - 1;   // of the tile, < 0: none
    const int seen_from = last_row < 0 ? 0 : lows[last_row], seen_to = last_row < 0 ? 0 : highs[0];

    // q as operand B: in registers for one group of rows, else read again for every block
    uint4 qb[NR == 1 ? 4 : 1];
    auto q_part = [&](int r, int c) {      // components 16 (q + 4 (c / 2)) + 8 (c % 2) .. + 7
      return *reinterpret_cast<const uint4*>(qs + (8 * r + g) * kQStride + 32 * (q + 4 * (c >> 1)) + 16 * (c & 1));
    };
    if constexpr (NR == 1) {
#pragma unroll
      for (int c = 0; c < 4; ++c) qb[c] = q_part(0, c);
    }
    // Of rows 8 r + 2 q and the next one.  The reference is a score (top, its
    // negative) plus a small number (low), so that large scores do not swallow the
    // logarithm of the value scale in it.
    f32x2 factor[NR], top[NR], low[NR], sum[NR];
    float o[8][NR][4];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const float2 f = *reinterpret_cast<const float2*>(factors + 8 * r + 2 * q);
      factor[r] = pack2(f.x, f.y);
      top[r] = both(-kNone);
      low[r] = both(0.0f);
      sum[r] = both(0.0f);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
#pragma unroll
        for (int c = 0; c < 4; ++c) o[j][r][c] = 0.0f;
      }
    }

    for (int i = warp; i < n; i += kAttnWarps) {
      ok = __all_sync(kAll, mbar_wait(full_at + 8 * slot, phase, ctx, 91)) && ok;
      const uint8_t* const blk = ring + slot * kCacheBlock;
      if (ok && (there >> slot & 1u)) {
        // ---- scores
        float s[NR][4];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
#pragma unroll
          for (int c = 0; c < 4; ++c) s[r][c] = 0.0f;
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint4 ka = *reinterpret_cast<const uint4*>(blk + tok * kHeadDim + 16 * ((q + 4 * c) ^ k_turn));
          const uint4 kb = *reinterpret_cast<const uint4*>(blk + (tok + 2) * kHeadDim + 16 * ((q + 4 * c) ^ k_turn));
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
            const uint4 b0 = NR == 1 ? qb[NR == 1 ? 2 * c : 0] : q_part(r, 2 * c);
            const uint4 b1 = NR == 1 ? qb[NR == 1 ? 2 * c + 1 : 0] : q_part(r, 2 * c + 1);
            mma(s[r], fa[0], b0.x, b0.y);
            mma(s[r], fa[1], b0.z, b0.w);
            mma(s[r], fa[2], b1.x, b1.y);
            mma(s[r], fa[3], b1.z, b1.w);
          }
        }
        const float* const scales = reinterpret_cast<const float*>(blk + kKScales);
        const float ks0 = scales[tok], ks1 = scales[tok + 2];
        const float vs0 = scales[16 + tok], vs1 = scales[16 + tok + 2];
        const float lv0 = log2_above(vs0), lv1 = log2_above(vs1);
        const int j0 = 16 * (walk.span.first + walk.off + i);     // first token of the block
        const bool all_seen = j0 >= seen_from && j0 + 16 <= seen_to;
        // scores times log2(e), of tokens tok + 2 c and rows 8 r + 2 q, + 1
        f32x2 x[NR][2];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            x[r][c] = mul2(mul2(pack2(s[r][2 * c], s[r][2 * c + 1]), factor[r]), both(c == 0 ? ks0 : ks1));
            if constexpr (kCap) {
              // tanh(y) = 1 - 2 / (1 + e^2y), with an error of about 2^-23
              float v[2];
              unpack2(x[r][c], v[0], v[1]);
#pragma unroll
              for (int k = 0; k < 2; ++k)
                v[k] = a.softcap * kLog2e * (1.0f - __fdividef(2.0f, 1.0f + ex2(v[k] * (2.0f * kLog2e / a.softcap))));
              x[r][c] = pack2(v[0], v[1]);
            }
          }
        }
        if (!all_seen) {
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            const int2 lo = *reinterpret_cast<const int2*>(lows + 8 * r + 2 * q), hi = *reinterpret_cast<const int2*>(highs + 8 * r + 2 * q);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int j = j0 + tok + 2 * c;
              float v0, v1;
              unpack2(x[r][c], v0, v1);
              x[r][c] = pack2(j >= lo.x && j < hi.x ? v0 : -INFINITY, j >= lo.y && j < hi.y ? v1 : -INFINITY);
            }
          }
        }
        auto under = [&](int r, int c) { return sub2(add2(x[r][c], top[r]), low[r]); };   // less the reference
        float far[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int r = 0; r < NR; ++r) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float v0, v1;
            unpack2(under(r, c), v0, v1);
            far[c] = fmaxf(far[c], fmaxf(v0, v1));
          }
        }
        if (__any_sync(kAll, fmaxf(far[0] + lv0, far[1] + lv1) > kMostWeight)) {
          // references of the rows concerned up, what stands under them down
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            float w[4], m[2], c[2], keep[2];
            bool up[2];
            unpack2(add2(under(r, 0), both(lv0)), w[0], w[1]);
            unpack2(add2(under(r, 1), both(lv1)), w[2], w[3]);
            up[0] = fmaxf(w[0], w[2]) > kMostWeight;
            up[1] = fmaxf(w[1], w[3]) > kMostWeight;
            if (!__any_sync(kAll, up[0] || up[1])) continue;
            unpack2(x[r][0], w[0], w[1]);
            unpack2(x[r][1], w[2], w[3]);
            unpack2(top[r], m[0], m[1]);
            unpack2(low[r], c[0], c[1]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              up[k] = max_over_g(up[k] ? 1.0f : 0.0f) > 0.0f;
              const float next = max_over_g(fmaxf(w[k], w[2 + k]));
              const float over = max_over_g(fmaxf(w[k] - next + lv0, w[2 + k] - next + lv1)) - kNewWeight;
              keep[k] = up[k] ? ex2((-m[k] - next) + (c[k] - over)) : 1.0f;
              m[k] = up[k] ? -next : m[k];
              c[k] = up[k] ? over : c[k];
            }
            top[r] = pack2(m[0], m[1]);
            low[r] = pack2(c[0], c[1]);
            sum[r] = mul2(sum[r], pack2(keep[0], keep[1]));
#pragma unroll
            for (int j = 0; j < 8; ++j) {
#pragma unroll
              for (int k = 0; k < 4; ++k) o[j][r][k] *= keep[k & 1];
            }
          }
        }
        // ---- weights
        uint32_t b0[NR], b1[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          float w[4];
          unpack2(under(r, 0), w[0], w[1]);
          unpack2(under(r, 1), w[2], w[3]);
#pragma unroll
          for (int k = 0; k < 4; ++k) w[k] = ex2(w[k]);
          const f32x2 p0 = pack2(w[0], w[1]), p1 = pack2(w[2], w[3]);
          sum[r] = add2(sum[r], add2(p0, p1));
          unpack2(mul2(p0, both(vs0)), w[0], w[1]);
          unpack2(mul2(p1, both(vs1)), w[2], w[3]);
          const __half2 w0 = __floats2half2_rn(w[0], w[1]), w1 = __floats2half2_rn(w[2], w[3]);
          b0[r] = *reinterpret_cast<const uint32_t*>(&w0);
          b1[r] = *reinterpret_cast<const uint32_t*>(&w1);
        }
        if (!all_seen) {      // hidden weights 0, whatever the scale holds
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            float v[4];
            unpack2(x[r][0], v[0], v[1]);
            unpack2(x[r][1], v[2], v[3]);
            b0[r] &= (v[0] == -INFINITY ? 0u : 0xFFFFu) | (v[1] == -INFINITY ? 0u : 0xFFFF0000u);
            b1[r] &= (v[2] == -INFINITY ? 0u : 0xFFFFu) | (v[3] == -INFINITY ? 0u : 0xFFFF0000u);
          }
        }
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          b0[r] = transpose(b0[r]);
          b1[r] = transpose(b1[r]);
        }
        // ---- outputs: components 16 g + 4 w + 0 .. 3, tokens by q
        const uint8_t* const v = blk + kVCodes;
        const int other = 4 * (q ^ 2) + 1;
        const uint4 va = *reinterpret_cast<const uint4*>(v + 4 * q * kHeadDim + 16 * (g ^ (2 * q)));
        const uint4 vb = *reinterpret_cast<const uint4*>(v + other * kHeadDim + 16 * (g ^ (2 * (q ^ 2))));
        const uint4 vc = *reinterpret_cast<const uint4*>(v + (4 * q + 2) * kHeadDim + 16 * (g ^ (2 * q)));
        const uint4 vd = *reinterpret_cast<const uint4*>(v + (other + 2) * kHeadDim + 16 * (g ^ (2 * (q ^ 2))));
        const uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wb[4] = {vb.x, vb.y, vb.z, vb.w};
        const uint32_t wc[4] = {vc.x, vc.y, vc.z, vc.w}, wd[4] = {vd.x, vd.y, vd.z, vd.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t fa[2][4];
          biased_u8x4_to_f16x4(prmt(wa[w], wb[w], 0x5140u), fa[0][0], fa[0][1]);
          biased_u8x4_to_f16x4(prmt(wc[w], wd[w], 0x5140u), fa[0][2], fa[0][3]);
          biased_u8x4_to_f16x4(prmt(wa[w], wb[w], 0x7362u), fa[1][0], fa[1][1]);
          biased_u8x4_to_f16x4(prmt(wc[w], wd[w], 0x7362u), fa[1][2], fa[1][3]);
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            mma(o[2 * w][r], fa[0], b0[r], b1[r]);
            mma(o[2 * w + 1][r], fa[1], b0[r], b1[r]);
          }
        }
      }
      // the slot is read: the next block into it
      fence_proxy_async_smem();
      __syncwarp();
      if (ok) fetch(slot);
      if (++slot == kSlots) {
        slot = 0;
        phase ^= 1;
      }
    }

    // ---- the piece is done: the warps' sums meet
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      float s0, s1;
      unpack2(sum[r], s0, s1);
#pragma unroll
      for (int d = 4; d <= 16; d <<= 1) {
        s0 += __shfl_xor_sync(kAll, s0, d);
        s1 += __shfl_xor_sync(kAll, s1, d);
      }
      if (g == 0) {
        float m0, m1, c0, c1;
        unpack2(top[r], m0, m1);
        unpack2(low[r], c0, c1);
        Share* const to = shares + warp * S::kRows + 8 * r + 2 * q;
        to[0] = Share{-m0, c0, s0, 0.0f};
        to[1] = Share{-m1, c1, s1, 0.0f};
      }
    }
    const bool done = n == walk.span.count;
    const int64_t part = (2LL * blockIdx.x + (walk.off > 0 ? 0 : 1)) * S::kRows;
    constexpr int kWords = 4 / S::kRounds;
#pragma unroll
    for (int round = 0; round < S::kRounds; ++round) {
      if (round > 0) __syncthreads();
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        const int j = 2 * (round * kWords + w);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
            *reinterpret_cast<float4*>(meet + ((w * kAttnWarps + warp) * S::kRows + 8 * r + 2 * q + c) * kMeetStride + 4 * g) =
                make_float4(o[j][r][c], o[j][r][2 + c], o[j + 1][r][c], o[j + 1][r][2 + c]);
        }
      }
      __syncthreads();
      // a thread joins 4 components of a row
      for (int item = tid; item < S::kRows * 8 * kWords; item += kAttnThreads) {
        const int gg = item & 7, w = item >> 3 & (kWords - 1), in_tile = item / (8 * kWords);
        const int row = row0 + in_tile, t = row / p.G;
        if (row >= rows || t >= walk.seq.fresh) continue;
        Share all{kNone, -INFINITY, 0.0f, 0.0f};
        Share of[kAttnWarps];
#pragma unroll
        for (int k = 0; k < kAttnWarps; ++k) {
          of[k] = shares[k * S::kRows + in_tile];
          all.m = fmaxf(all.m, of[k].m);
        }
#pragma unroll
        for (int k = 0; k < kAttnWarps; ++k) all.c = fmaxf(all.c, of[k].over(all.m));
        float4 v = make_float4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < kAttnWarps; ++k) {
          const float f = ex2(of[k].over(all.m) - all.c);
          const float4 x = *reinterpret_cast<const float4*>(meet + ((w * kAttnWarps + k) * S::kRows + in_tile) * kMeetStride + 4 * gg);
          all.l += f * of[k].l;
          v = make_float4(v.x + f * x.x, v.y + f * x.y, v.z + f * x.z, v.w + f * x.w);
        }
        const int d = 16 * gg + 4 * (round * kWords + w);
        if (done) {
          const float back = all.l == 0.0f ? 0.0f : __fdiv_rn(1.0f, all.l);      // 0: no token seen
          *reinterpret_cast<uint2*>(a.out + ((q_row + t) * a.q_heads + h * p.G + (row - t * p.G)) * kHeadDim + d) =
              make_uint2(bf16x2_rn(v.x * back, v.y * back), bf16x2_rn(v.z * back, v.w * back));
        } else {
          *reinterpret_cast<float4*>(p.part_o + (part + in_tile) * kHeadDim + d) = v;
          if (d == 0) p.part_share[part + in_tile] = all;
        }
      }
    }
    walk.next(a);
    if (walk.left > 0) __syncthreads();     // what the rows' q and the meeting stood in is read
  }
  if (!ok) {      // the copies land before the block ends
    int never = 0;
    const WaitCtx drain{p.err, &never, kWaitLimitNs};
    for (int i = 0; i < kSlots; ++i) {
      if (--slot < 0) {
        slot = kSlots - 1;
        phase ^= 1;
      }
      (void)mbar_wait(full_at + 8 * slot, phase, drain, 92);
    }
  }
}

// The parts of a cut segment joined: block x announces it, a warp takes one row
// (or, `wide`, the block's four one row).
__global__ void __launch_bounds__(128) join_kernel(const AttnParams p, int tile_rows, int wide) {
  __shared__ float4 acc[4][32];
  __shared__ Share of[4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dep_launch();
  grid_dep_wait();
  const PagedAttnArgs& a = p.a;
  const int4 cut = __ldg(reinterpret_cast<const int4*>(p.cuts + 4 * (blockIdx.x + 1)));
  if (cut.x < 0) return;
  const SeqLen seq = seq_len(a.c, cut.w, a.T);
  const int h = cut.x / p.row_tiles;
  const int in_tile = wide ? blockIdx.y : 4 * blockIdx.y + warp;
  const int row = (cut.x - h * p.row_tiles) * tile_rows + in_tile, t = row / p.G;
  if (in_tile >= tile_rows || row >= static_cast<int>(a.T) * p.G || t >= seq.fresh) return;
  const int parts = cut.z - cut.y + 1, step = wide ? 4 : 1;
  Share all{kNone, -200.0f, 0.0f, 0.0f};      // reference below every part's
  float4 o = make_float4(0, 0, 0, 0);
  // all and o with another part
  auto add = [&](const Share& s, const float4& v) {
    const float m = fmaxf(all.m, s.m);
    const float was = all.over(m), is = s.over(m), c = fmaxf(was, is);
    const float f = ex2(was - c), g = ex2(is - c);
    all = Share{m, c, all.l * f + s.l * g, 0.0f};
    o = make_float4(o.x * f + v.x * g, o.y * f + v.y * g, o.z * f + v.z * g, o.w * f + v.w * g);
  };
  constexpr int kAhead = 4;
  for (int k0 = wide ? warp : 0; k0 < parts; k0 += kAhead * step) {
    float4 part[kAhead], v[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = k0 + k * step;
      if (i >= parts) break;
      const int64_t slot = i == 0 ? 2LL * cut.y + 1 : 2LL * (cut.y + i);
      part[k] = __ldg(reinterpret_cast<const float4*>(p.part_share + slot * tile_rows + in_tile));
      v[k] = __ldg(reinterpret_cast<const float4*>(p.part_o + (slot * tile_rows + in_tile) * kHeadDim) + lane);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (k0 + k * step < parts) add(Share{part[k].x, part[k].y, part[k].z, 0.0f}, v[k]);
  }
  if (wide) {
    acc[warp][lane] = o;
    if (lane == 0) of[warp] = all;
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int w = 1; w < 4; ++w) add(of[w], acc[w][lane]);
  }
  const float back = all.l == 0.0f ? 0.0f : __fdiv_rn(1.0f, all.l);
  const int64_t to = ((static_cast<int64_t>(cut.w) * a.T + t) * a.q_heads + h * p.G + (row - t * p.G)) * kHeadDim + 4 * lane;
  *reinterpret_cast<uint2*>(a.out + to) = make_uint2(bf16x2_rn(o.x * back, o.y * back), bf16x2_rn(o.z * back, o.w * back));
}

// 8-row groups of a tile for `rows` rows: as few as hold them, four at most.
int row_groups(int64_t rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : 4; }

int grid_of(int groups, int sm_count) { return sm_count * (groups <= 2 ? 2 : 1); }

template <int NR, bool kCap>
cudaError_t launch_groups(const AttnParams& p, int grid, cudaStream_t stream) {
  const auto kernel = attn_kernel<NR, kCap>;
  // per call: a device's first costs nothing more, and no state is kept
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<NR>::kBytes);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(kAttnThreads), Shape<NR>::kBytes, stream, p);
  if (e != cudaSuccess) return e;
  // Long rows of parts for few segments: four warps a row.
  const int64_t segments = p.a.c.B * p.row_tiles * p.a.c.kv_heads;
  const int wide = grid >= 8 * segments ? 1 : 0;
  const int rows = static_cast<int>(p.a.T * p.G < 8 * NR ? p.a.T * p.G : 8 * NR);
  return launch_pdl(join_kernel, dim3(static_cast<unsigned>(grid - 1), static_cast<unsigned>(wide ? rows : (rows + 3) / 4)), dim3(128), 0,
                    stream, p, 8 * NR, wide);
}

template <int NR>
cudaError_t launch_cap(const AttnParams& p, int grid, cudaStream_t stream) {
  return p.a.softcap > 0.0f ? launch_groups<NR, true>(p, grid, stream) : launch_groups<NR, false>(p, grid, stream);
}

}  // namespace

size_t paged_attn_workspace_bytes(int64_t, int64_t T, int64_t q_heads, int64_t kv_heads, int sm_count) {
  const int groups = row_groups(T * (q_heads / kv_heads));
  const size_t grid = static_cast<size_t>(grid_of(groups, sm_count));
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
  const int grid = grid_of(groups, sm_count);
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
