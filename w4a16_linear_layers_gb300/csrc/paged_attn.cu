// paged_attn.cu -- attention of the new tokens over the paged INT8 cache.
//
// For a row (token i of a sequence, query head h) over the tokens j it sees:
//   x_j = scale ks_j (q . kc_j)  (softcap tanh(x_j / softcap)),
//   out = sum_j exp(x_j) vs_j vc_j / sum_j exp(x_j),
// kc, vc the codes and ks, vs their scales.  One pass over the cache with a
// running maximum m of x_j log2(e), so exp(x_j) = 2^(x_j log2(e) - m).
//
// What bounds it: HBM, 264 bytes a token and key/value head, which its rows (T
// new tokens times G query heads of the group) share.
//
// The work is the list of blocks of 16 tokens of all (sequence, row tile,
// key/value head) segments, in order, cut into equal shares: a thread block
// takes one, whatever the sequences' lengths.  It goes through its share 128
// tokens at a time; the parts of a segment that shares cut meet in a second
// kernel, segments inside one are finished at once.
//
// A tile of 128 tokens: a producer warp brings its eight blocks of 4224 bytes
// into a ring in shared memory by one bulk copy each.  Scores are formed
// transposed, tokens x rows, warp w those of block w: the codes are operand A
// (m16 = the block's tokens), widened to fp16 on the way, and q, as fp16 times a
// power of two of its row, operand B (n8 = rows).  So a batch of 1 to 8 rows
// costs half of what rows as operand A would, and no code is widened twice.
// The warps exchange their rows' maxima, write weights 2^(x - m) vs as fp16 to
// shared memory, and form the output transposed too, components x rows: warp w
// takes the 32 components w % 4 of the half w / 4 of the tokens, again with codes
// as operand A.  Output, maximum and sum stay in registers.
//
// mma.sync, not tcgen05: its operands come from registers, where the codes are
// widened; a tensor-memory A would need them written there, and the tile's rows,
// mostly 4 to 32, fill a fraction of a tcgen05 tile.
//
// Precision.  Codes are exact in fp16, and so is q up to 2^-39 of its row's
// largest component.  Weights are rounded to fp16 relative to R, a power of two
// over the row's largest vs so far: 11 bits down to 2^-29 of that.  Scores, sums
// and outputs are fp32.
#include <cuda_fp16.h>

#include "kv_cache.cuh"

namespace qlin {
namespace {

constexpr int kTile = 128;          // tokens
constexpr int kTileBlocks = kTile / 16;
constexpr int kConsumers = 256;
constexpr int kAttnThreads = kConsumers + 32;
constexpr int kMinShare = kTileBlocks;
constexpr int kQStride = 272;       // bytes of a row of q: rows 16 bytes apart mod 128
constexpr int kPStride = 288;       // bytes of a row of weights: rows 32 bytes apart mod 128
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kAll = 0xFFFFFFFFu;

template <int NR>
struct Shape {
  static constexpr int kRows = 8 * NR;
  static constexpr int kStages = NR == 1 ? 3 : 2;
  static constexpr int kPerSm = NR <= 4 ? 2 : 1;
  // shared memory, in order
  static constexpr int kRing = kStages * kTileBlocks * kCacheBlock;
  static constexpr int kQ = kRing;
  static constexpr int kP = kQ + kRows * kQStride;
  static constexpr int kO = kP + kRows * kPStride;       // fp32 [rows][128]
  static constexpr int kTop = kO + kRows * 512;          // fp32 [rows][8 warps]
  static constexpr int kVTop = kTop + kRows * 32;        // the same, of value scales
  static constexpr int kSum = kVTop + kRows * 32;
  static constexpr int kFactor = kSum + kRows * 32;      // fp32 [rows]
  static constexpr int kLow = kFactor + kRows * 4;       // int32 [rows]: first token seen
  static constexpr int kHigh = kLow + kRows * 4;         // and the one behind the last
  static constexpr int kBytes = kHigh + kRows * 4;
};

struct AttnParams {
  PagedAttnArgs a;
  int G;               // query heads of a key/value head
  int row_tiles;       // of a sequence's T * G rows
  int* err;
  // workspace: where the cut segments are, then their parts
  int32_t* cuts;       // [grid][4]: segment, its first and last share, sequence; segment -1: none
  float2* part_ml;     // [2 grid][rows]: maximum and sum
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
  int seg, segs;       // segment of the sequence, and how many it has
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

// max over the 8 lanes that share lane & 3
__device__ __forceinline__ float max_over_g(float v) {
  v = fmaxf(v, __shfl_xor_sync(kAll, v, 4));
  v = fmaxf(v, __shfl_xor_sync(kAll, v, 8));
  return fmaxf(v, __shfl_xor_sync(kAll, v, 16));
}

// 2^15 over the power of two above v (v below 2^-100 taken as that)
__device__ __forceinline__ float weight_factor(float v) {
  const int e = min(max(static_cast<int>(__float_as_uint(v) >> 23), 27), 253);
  return __uint_as_float(static_cast<uint32_t>(127 + 15 + 126 - e) << 23);
}

template <int NR, bool kCap>
__global__ void __launch_bounds__(kAttnThreads, Shape<NR>::kPerSm) attn_kernel(const AttnParams p) {
  using S = Shape<NR>;
  constexpr int kStages = S::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kStages], empty[kStages];
  __shared__ uint32_t on_page[kStages];      // bit i: block i of the tile is there
  __shared__ int abort_flag;
  __shared__ int warp_sum[9];
  __shared__ Walk start;
  __shared__ int64_t total_blocks, before_b;
  const PagedAttnArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int segs = p.row_tiles * static_cast<int>(a.c.kv_heads);

  if (tid == 0) {
    abort_flag = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), kConsumers / 32);
    }
    fence_barrier_init();
  }
  grid_dep_launch();
  grid_dep_wait();

  // ---- this block's share
  int64_t total;
  {
    int64_t sum = 0;
    for (int64_t b = tid; b < a.c.B; b += kAttnThreads) sum += span_of(a, seq_len(a.c, b, a.T)).count;
    if (tid == 0) total_blocks = 0;
    __syncthreads();
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    if (lane == 0 && sum != 0) atomicAdd(reinterpret_cast<unsigned long long*>(&total_blocks), static_cast<unsigned long long>(sum));
    __syncthreads();
    total = total_blocks * segs;
  }
  int64_t share = (total + gridDim.x - 1) / gridDim.x;
  if (share < kMinShare) share = kMinShare;
  const int64_t at = blockIdx.x * share;
  if (at >= total) {
    if (tid == 0) p.cuts[4 * blockIdx.x] = -1;
    return;
  }
  {
    // the sequence that holds block `at`: its place among 288 at a time
    int64_t before = 0;
    for (int64_t b0 = 0;; b0 += kAttnThreads) {
      const int64_t b = b0 + tid;
      const int n = b < a.c.B ? span_of(a, seq_len(a.c, b, a.T)).count : 0;
      int64_t incl = n;
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(kAll, incl, o);
        if (lane >= o) incl += v;
      }
      __shared__ int64_t sums[9];
      if (lane == 31) sums[warp] = incl;
      __syncthreads();
      int64_t all = 0;
      for (int w = 0; w < 9; ++w) {
        if (w < warp) incl += sums[w];
        all += sums[w];
      }
      incl += before;
      if (n > 0 && (incl - n) * segs <= at && at < incl * segs) {
        const int64_t in_b = at - (incl - n) * segs;
        start.b = b;
        start.segs = segs;
        start.seg = static_cast<int>(in_b / n);
        start.off = static_cast<int>(in_b - static_cast<int64_t>(start.seg) * n);
        start.left = total - at < share ? total - at : share;
        start.load(a);
        before_b = incl - n;
      }
      before += all;
      const bool found = before * segs > at;
      __syncthreads();
      if (found) break;
    }
  }
  Walk walk = start;
  (void)warp_sum;
  if (tid == 0) {
    // the first boundary inside a segment announces it
    const int64_t s0 = before_b * segs + static_cast<int64_t>(walk.seg) * walk.span.count;
    const int64_t first = s0 / share, last = (s0 + walk.span.count - 1) / share;
    const bool cut = walk.off > 0 && first == blockIdx.x - 1;
    int4 c;
    c.x = cut ? walk.seg : -1;
    c.y = static_cast<int>(first);
    c.z = static_cast<int>(last);
    c.w = static_cast<int>(walk.b);
    *reinterpret_cast<int4*>(p.cuts + 4 * blockIdx.x) = c;
  }

  const WaitCtx ctx{p.err, &abort_flag, kWaitLimitNs};
  if (warp == kConsumers / 32) {
    // ---- producer: one block of 16 tokens a lane
    int issued = 0;
    bool ok = true;
    while (ok && walk.left > 0) {
      const int n = walk.piece();
      const int h = walk.seg % static_cast<int>(a.c.kv_heads);
      const int first = walk.span.first + walk.off;
      auto block_at = [&](int i) -> const uint8_t* {
        return lane < kTileBlocks && i + lane < n ? cache_block(a.c, walk.b, h, first + i + lane) : nullptr;
      };
      const uint8_t* next = block_at(0);
      for (int i = 0; i < n; i += kTileBlocks) {
        const uint8_t* const from = next;
        if (i + kTileBlocks < n) next = block_at(i + kTileBlocks);
        const int stage = issued % kStages;
        if (issued >= kStages) ok = mbar_wait(smem_u32(&empty[stage]), (issued / kStages - 1) & 1, ctx, 91);
        if (!__all_sync(kAll, ok)) {
          ok = false;
          break;
        }
        const uint32_t there = __ballot_sync(kAll, from != nullptr);
        if (lane == 0) {
          on_page[stage] = there;
          mbar_arrive_expect_tx(smem_u32(&full[stage]), __popc(there) * kCacheBlock);
        }
        __syncwarp();
        if (from != nullptr)
          bulk_load(smem_u32(smem) + (stage * kTileBlocks + lane) * kCacheBlock, from, kCacheBlock, smem_u32(&full[stage]));
        ++issued;
      }
      if (ok) walk.next(a);
    }
    if (!ok) {      // the copies land before the block ends
      int never = 0;
      const WaitCtx drain{p.err, &never, kWaitLimitNs};
      for (int i = issued < kStages ? 0 : issued - kStages; i < issued; ++i)
        (void)mbar_wait(smem_u32(&full[i % kStages]), (i / kStages) & 1, drain, 92);
    }
    return;
  }

  // ---- consumers
  const int g = lane >> 2, q = lane & 3;
  const int tokA = 2 * (g >> 1) + 8 * (g & 1);    // of a block; the other is tokA + 1
  const int quarter = warp & 3, half = warp >> 2;
  uint8_t* const qs = smem + S::kQ;
  uint8_t* const ps = smem + S::kP;
  float* const os = reinterpret_cast<float*>(smem + S::kO);
  float* const tops = reinterpret_cast<float*>(smem + S::kTop);
  float* const vtops = reinterpret_cast<float*>(smem + S::kVTop);
  float* const sums = reinterpret_cast<float*>(smem + S::kSum);
  float* const factors = reinterpret_cast<float*>(smem + S::kFactor);
  int* const lows = reinterpret_cast<int*>(smem + S::kLow);
  int* const highs = reinterpret_cast<int*>(smem + S::kHigh);
  const int rows = static_cast<int>(a.T) * p.G;
  int taken = 0;

  while (walk.left > 0) {
    const int n = walk.piece();
    const int h = walk.seg % static_cast<int>(a.c.kv_heads);
    const int row0 = walk.seg / static_cast<int>(a.c.kv_heads) * S::kRows;
    const int64_t q_row = walk.b * a.T;
    // q of the tile's rows, what they see
    for (int r = warp; r < S::kRows; r += kConsumers / 32) {
      const int row = row0 + r, t = row / p.G;
      const bool there = row < rows && t < walk.seq.fresh;
      uint2 x = make_uint2(0, 0);
      if (there)
        x = __ldg(reinterpret_cast<const uint2*>(a.q + ((q_row + t) * a.q_heads + h * p.G + (row - t * p.G)) * kHeadDim) + lane);
      float f[4] = {__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xFFFF0000u), __uint_as_float(x.y << 16),
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
        if (!there) highs[r] = 0;
      }
    }
    named_bar_sync(1, kConsumers);
    // tokens that all rows see, and that any does
    const int last_row = min(min(S::kRows, rows - row0), walk.seq.fresh * p.G - row0) - 1;   // of the tile, < 0: none
    const int seen_from = last_row < 0 ? 0 : lows[last_row], seen_to = last_row < 0 ? 0 : highs[0];

    float m[NR][2], l[NR][2], vf[NR][2];
    float o[2][NR][4];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      m[i][0] = m[i][1] = -INFINITY;
      l[i][0] = l[i][1] = 0.0f;
      vf[i][0] = vf[i][1] = weight_factor(0.0f);
#pragma unroll
      for (int j = 0; j < 4; ++j) o[0][i][j] = o[1][i][j] = 0.0f;
    }

    for (int i = 0; i < n; i += kTileBlocks, ++taken) {
      const int stage = taken % kStages;
      bool ok = mbar_wait(smem_u32(&full[stage]), (taken / kStages) & 1, ctx, 93);
      ok = __all_sync(kAll, ok);
      const uint32_t there = ok ? on_page[stage] : 0u;
      const uint8_t* const tile = smem + stage * kTileBlocks * kCacheBlock;
      const int j0 = 16 * (walk.span.first + walk.off + i);       // first token of the tile
      const bool all_seen = j0 >= seen_from && j0 + 16 * min(kTileBlocks, n - i) <= seen_to;

      // scores of this warp's block
      float s[NR][4];
      float vs[2] = {0.0f, 0.0f};
#pragma unroll
      for (int r = 0; r < NR; ++r) {
#pragma unroll
        for (int c = 0; c < 4; ++c) s[r][c] = 0.0f;
      }
      const bool mine = (there >> warp) & 1u;
      if (mine) {
        const uint8_t* const blk = tile + warp * kCacheBlock;
        const int turn = 2 * ((tokA >> 2) & 3);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint4 ka = *reinterpret_cast<const uint4*>(blk + tokA * kHeadDim + 16 * ((q + 4 * c) ^ turn));
          const uint4 kb = *reinterpret_cast<const uint4*>(blk + (tokA + 1) * kHeadDim + 16 * ((q + 4 * c) ^ turn));
          uint32_t fa[4][4];
          biased_u8x4_to_f16x4(ka.x, fa[0][0], fa[0][2]);
          biased_u8x4_to_f16x4(ka.y, fa[1][0], fa[1][2]);
          biased_u8x4_to_f16x4(ka.z, fa[2][0], fa[2][2]);
          biased_u8x4_to_f16x4(ka.w, fa[3][0], fa[3][2]);
          biased_u8x4_to_f16x4(kb.x, fa[0][1], fa[0][3]);
          biased_u8x4_to_f16x4(kb.y, fa[1][1], fa[1][3]);
          biased_u8x4_to_f16x4(kb.z, fa[2][1], fa[2][3]);
          biased_u8x4_to_f16x4(kb.w, fa[3][1], fa[3][3]);
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            const uint8_t* const from = qs + (8 * r + g) * kQStride + 32 * (q + 4 * c);
            const uint4 b0 = *reinterpret_cast<const uint4*>(from);
            const uint4 b1 = *reinterpret_cast<const uint4*>(from + 16);
            mma(s[r], fa[0], b0.x, b0.y);
            mma(s[r], fa[1], b0.z, b0.w);
            mma(s[r], fa[2], b1.x, b1.y);
            mma(s[r], fa[3], b1.z, b1.w);
          }
        }
        const float2 ks = *reinterpret_cast<const float2*>(blk + kKScales + 4 * tokA);
        const float2 v2 = *reinterpret_cast<const float2*>(blk + kVScales + 4 * tokA);
        vs[0] = v2.x;
        vs[1] = v2.y;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const float2 f = *reinterpret_cast<const float2*>(factors + 8 * r + 2 * q);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float x = s[r][c] * ((c & 1) ? f.y : f.x) * (c < 2 ? ks.x : ks.y);
            if (kCap) {
              // tanh(y) = 1 - 2 / (1 + e^2y), with an error of about 2^-23
              const float e = ex2(x * (2.0f * kLog2e / a.softcap));
              x = a.softcap * kLog2e * (1.0f - __fdividef(2.0f, 1.0f + e));
            }
            s[r][c] = x;
          }
        }
      }
      if (!mine || !all_seen) {
        const int jA = j0 + 16 * warp + tokA;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int lo = lows[8 * r + 2 * q + c], hi = highs[8 * r + 2 * q + c];
            if (!mine || jA < lo || jA >= hi) s[r][c] = -INFINITY;
            if (!mine || jA + 1 < lo || jA + 1 >= hi) s[r][2 + c] = -INFINITY;
          }
        }
      }
      // maxima of the scores and of the value scales that a row sees
#pragma unroll
      for (int r = 0; r < NR; ++r) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float top = max_over_g(fmaxf(s[r][c], s[r][2 + c]));
          if (g == 0) tops[(8 * r + 2 * q + c) * 8 + warp] = top;
        }
      }
      if (all_seen) {
        const float top = max_over_g(fmaxf(fabsf(vs[0]), fabsf(vs[1])));
        if (lane == 0) vtops[warp] = top;
      } else {
#pragma unroll
        for (int r = 0; r < NR; ++r) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float top = max_over_g(fmaxf(s[r][c] == -INFINITY ? 0.0f : fabsf(vs[0]), s[r][2 + c] == -INFINITY ? 0.0f : fabsf(vs[1])));
            if (g == 0) vtops[(8 * r + 2 * q + c) * 8 + warp] = top;
          }
        }
      }
      if (!named_bar_and(1, kConsumers, ok)) return;      // a wait ran out, in every warp alike

      auto top_of = [](const float* v) {
        const float4 x = *reinterpret_cast<const float4*>(v), y = *reinterpret_cast<const float4*>(v + 4);
        return fmaxf(fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)), fmaxf(fmaxf(y.x, y.y), fmaxf(y.z, y.w)));
      };
      const float vtop = all_seen ? top_of(vtops) : 0.0f;
      bool same = true;
      float keep[NR][2];
#pragma unroll
      for (int r = 0; r < NR; ++r) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int row = 8 * r + 2 * q + c;
          const float next = fmaxf(m[r][c], top_of(tops + row * 8));
          const float base = next == -INFINITY ? 0.0f : next;
          const float alpha = ex2(m[r][c] - base);
          const float f = fminf(vf[r][c], weight_factor(all_seen ? vtop : top_of(vtops + row * 8)));
          m[r][c] = next;
          // o is in units of 1 / vf: 1 / vf of a power of two by its exponent
          keep[r][c] = alpha * (f * __uint_as_float(0x7F000000u - __float_as_uint(vf[r][c])));
          vf[r][c] = f;
          same = same && keep[r][c] == 1.0f;
          const float p0 = ex2(s[r][c] - base), p1 = ex2(s[r][2 + c] - base);
          l[r][c] = l[r][c] * alpha + (p0 + p1);
          float w0 = p0 * (vs[0] * f), w1 = p1 * (vs[1] * f);
          if (!all_seen) {
            if (s[r][c] == -INFINITY) w0 = 0.0f;
            if (s[r][2 + c] == -INFINITY) w1 = 0.0f;
          }
          const __half2 w = __floats2half2_rn(w0, w1);
          if (mine) *reinterpret_cast<__half2*>(ps + row * kPStride + 2 * (16 * warp + tokA)) = w;
        }
      }
      named_bar_sync(1, kConsumers);
      if (!__all_sync(kAll, same)) {
#pragma unroll
        for (int r = 0; r < NR; ++r) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            o[0][r][c] *= keep[r][c & 1];
            o[1][r][c] *= keep[r][c & 1];
          }
        }
      }
      // outputs: four blocks of tokens, 32 components
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int in_tile = 4 * half + k;
        if (!((there >> in_tile) & 1u)) continue;
        const uint8_t* const v = tile + in_tile * kCacheBlock + kVCodes + 4 * q * kHeadDim + 32 * (quarter ^ q) + 4 * g;
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
          const uint2 b = *reinterpret_cast<const uint2*>(ps + (8 * r + g) * kPStride + 32 * in_tile + 8 * q);
          mma(o[0][r], fa[0], b.x, b.y);
          mma(o[1][r], fa[1], b.x, b.y);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&empty[stage]));
    }

    // ---- the piece is done: sums over the warps, outputs of the two halves
#pragma unroll
    for (int r = 0; r < NR; ++r) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float v = l[r][c];
        v += __shfl_xor_sync(kAll, v, 4);
        v += __shfl_xor_sync(kAll, v, 8);
        v += __shfl_xor_sync(kAll, v, 16);
        if (g == 0) sums[(8 * r + 2 * q + c) * 8 + warp] = v;
        if (half == 1)
          *reinterpret_cast<float4*>(os + (8 * r + 2 * q + c) * kHeadDim + 32 * quarter + 4 * g) =
              make_float4(o[0][r][c], o[0][r][2 + c], o[1][r][c], o[1][r][2 + c]);
      }
    }
    named_bar_sync(1, kConsumers);
    if (half == 0) {
      const bool done = n == walk.span.count;
      const int64_t slot = 2LL * blockIdx.x + (walk.off > 0 ? 0 : 1);
#pragma unroll
      for (int r = 0; r < NR; ++r) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int in_tile = 8 * r + 2 * q + c, row = row0 + in_tile, t = row / p.G;
          if (row >= rows || t >= walk.seq.fresh) continue;
          const float4 other = *reinterpret_cast<const float4*>(os + in_tile * kHeadDim + 32 * quarter + 4 * g);
          const float4 x = *reinterpret_cast<const float4*>(sums + in_tile * 8), y = *reinterpret_cast<const float4*>(sums + in_tile * 8 + 4);
          const float sum = ((x.x + x.y) + (x.z + x.w)) + ((y.x + y.y) + (y.z + y.w));
          float back = __uint_as_float(0x7F000000u - __float_as_uint(vf[r][c]));
          float4 v = make_float4(o[0][r][c] + other.x, o[0][r][2 + c] + other.y, o[1][r][c] + other.z, o[1][r][2 + c] + other.w);
          if (done) {
            back = sum == 0.0f ? 0.0f : __fdiv_rn(back, sum);      // 0: no token seen
            const int64_t to = ((q_row + t) * a.q_heads + h * p.G + (row - t * p.G)) * kHeadDim + 32 * quarter + 4 * g;
            *reinterpret_cast<uint2*>(a.out + to) = make_uint2(bf16x2_rn(v.x * back, v.y * back), bf16x2_rn(v.z * back, v.w * back));
          } else {
            v = make_float4(v.x * back, v.y * back, v.z * back, v.w * back);
            *reinterpret_cast<float4*>(p.part_o + (slot * S::kRows + in_tile) * kHeadDim + 32 * quarter + 4 * g) = v;
            if (quarter == 0 && g == 0) p.part_ml[slot * S::kRows + in_tile] = make_float2(m[r][c], sum);
          }
        }
      }
    }
    walk.next(a);
  }
}

// The parts of a cut segment joined: block x announces it, a warp takes one row
// (or, `wide`, the block's four one row).
__global__ void __launch_bounds__(128) join_kernel(const AttnParams p, int tile_rows, int wide) {
  __shared__ float4 acc[4][32];
  __shared__ float2 ml[4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dep_launch();
  grid_dep_wait();
  const PagedAttnArgs& a = p.a;
  const int4 cut = __ldg(reinterpret_cast<const int4*>(p.cuts + 4 * (blockIdx.x + 1)));
  if (cut.x < 0) return;
  const SeqLen seq = seq_len(a.c, cut.w, a.T);
  const int kv_heads = static_cast<int>(a.c.kv_heads);
  const int h = cut.x % kv_heads;
  const int in_tile = wide ? blockIdx.y : 4 * blockIdx.y + warp;
  const int row = cut.x / kv_heads * tile_rows + in_tile, t = row / p.G;
  if (in_tile >= tile_rows || row >= static_cast<int>(a.T) * p.G || t >= seq.fresh) return;
  const int parts = cut.z - cut.y + 1, step = wide ? 4 : 1;
  float m = -INFINITY, l = 0.0f;
  float4 o = make_float4(0, 0, 0, 0);
  constexpr int kAhead = 4;
  for (int k0 = wide ? warp : 0; k0 < parts; k0 += kAhead * step) {
    float2 part[kAhead];
    float4 v[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = k0 + k * step;
      part[k] = make_float2(-INFINITY, 0.0f);
      v[k] = make_float4(0, 0, 0, 0);
      if (i < parts) {
        const int64_t slot = i == 0 ? 2LL * cut.y + 1 : 2LL * (cut.y + i);
        part[k] = __ldg(p.part_ml + slot * tile_rows + in_tile);
        v[k] = __ldg(reinterpret_cast<const float4*>(p.part_o + (slot * tile_rows + in_tile) * kHeadDim) + lane);
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const float next = fmaxf(m, part[k].x);
      const float base = next == -INFINITY ? 0.0f : next;
      const float old = ex2(m - base), now = ex2(part[k].x - base);
      m = next;
      l = l * old + part[k].y * now;
      o = make_float4(o.x * old + v[k].x * now, o.y * old + v[k].y * now, o.z * old + v[k].z * now, o.w * old + v[k].w * now);
    }
  }
  if (wide) {
    acc[warp][lane] = o;
    if (lane == 0) ml[warp] = make_float2(m, l);
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int w = 1; w < 4; ++w) {
      const float next = fmaxf(m, ml[w].x);
      const float base = next == -INFINITY ? 0.0f : next;
      const float old = ex2(m - base), now = ex2(ml[w].x - base);
      const float4 v = acc[w][lane];
      m = next;
      l = l * old + ml[w].y * now;
      o = make_float4(o.x * old + v.x * now, o.y * old + v.y * now, o.z * old + v.z * now, o.w * old + v.w * now);
    }
  }
  const float back = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
  const int64_t to = ((static_cast<int64_t>(cut.w) * a.T + t) * a.q_heads + h * p.G + (row - t * p.G)) * kHeadDim + 4 * lane;
  *reinterpret_cast<uint2*>(a.out + to) = make_uint2(bf16x2_rn(o.x * back, o.y * back), bf16x2_rn(o.z * back, o.w * back));
}

// 8-row groups of a tile for `rows` rows: as few as hold them, eight at most.
int row_groups(int64_t rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 32 ? 4 : 8; }

int grid_of(int groups, int sm_count) { return sm_count * (groups <= 4 ? 2 : 1); }

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
  return grid * 16 + 2 * grid * 8 * groups * (sizeof(float2) + kHeadDim * sizeof(float));
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
  p.part_ml = reinterpret_cast<float2*>(p.part_o + 2 * static_cast<size_t>(grid) * 8 * groups * kHeadDim);
  switch (groups) {
    case 1: return launch_cap<1>(p, grid, stream);
    case 2: return launch_cap<2>(p, grid, stream);
    case 4: return launch_cap<4>(p, grid, stream);
    default: return launch_cap<8>(p, grid, stream);
  }
}

}  // namespace qlin
