// gemm_channel_pair.cuh -- device side of the per-channel W8A8 linear on
// tcgen05 for batches above the streaming kernel's: one persistent pair of
// thread blocks (two SMs, tcgen05 cta_group::2) per tile of 256 output channels
// x T tokens.
//
//   * The MMA runs with the weights as operand A (256 rows, 128 from each
//     block, widened by threads straight into tensor memory) and the tokens as
//     operand B (T columns, fp16 codes, 128-byte swizzled).  Each block loads
//     its own 128 channels' words and half of the tokens: the pair reads every
//     operand byte once, where two single blocks would read the tokens twice.
//     Per 128-wide K step and SM that is 16 KB of words and T * 128 bytes of
//     codes against 4 T cycles of MMA: 48 bytes a cycle at T = 256.
//   * An accumulator takes at most 1024 of K (exact below 2^24); the
//     epilogue adds each such chunk to int32 registers.
//   * Work: whole tiles go round the pairs in bands of token tiles, so the
//     pairs running at one time share a few channel tiles and one band's
//     tokens in L2.  The tiles that do not fill a last round are cut along
//     K instead, evenly between the pairs, and come first: a block publishes
//     its int32 partial of such a tile, and the last one to arrive on the
//     tile's counter adds the others' to its own.  Integer sums: the result
//     does not depend on who is last.
//   * Roles of a block's 20 warps: 0 streams words and 2 tokens by TMA, 1
//     issues the MMAs (first block of the pair), 4-11 widen weights (two
//     groups taking alternate steps), 12-19 drain and write.
//
// Every wait is bounded; a wait that runs out records an error, aborts the
// block's roles, and the block still drains its copies and frees its TMEM.
#pragma once

#include <cuda_bf16.h>

#include "qlin_device.cuh"
#include "qlin_internal.h"

namespace qlin {
namespace pair {

constexpr int kF = 128;                 // channels of one block
constexpr int kChunk = 8;               // K steps of 128 per accumulator
constexpr int kBufs = 4;                // A buffers in TMEM and token slots in shared memory
constexpr uint32_t kWBytes = 32 * kF * 4;
constexpr int kThreads = 640;
constexpr int kEpiThreads = 256;
constexpr uint32_t kCtrl = 1024;
constexpr uint32_t kSmemMax = 232448;
constexpr int kMaxW = 6;                // even: a slot stays with one widening group

template <int T>
struct Cfg {
  static constexpr int kHalf = T / 2;                         // tokens of one block
  static constexpr uint32_t kXBytes = kHalf * 256u;           // one step's codes of one block
  static constexpr int kND = T <= 128 ? 2 : 1;                // accumulators
  static constexpr int kCols = T / 2;                         // accumulator columns of an epilogue thread
  static constexpr uint32_t kColD = 64 * kBufs;
  static constexpr int kWSlotsFit = static_cast<int>((kSmemMax - 1024 - kCtrl - kBufs * kXBytes) / kWBytes);
  static constexpr int kWSlots = kWSlotsFit < kMaxW ? kWSlotsFit : kMaxW;
  static constexpr uint32_t kSmem = 1024 + kCtrl + kBufs * kXBytes + kWSlots * kWBytes;
  static_assert(T % 32 == 0 && T >= 64 && T <= 256, "token tile");
  static_assert(kColD + kND * T <= 512, "TMEM budget");
  static_assert(kWSlots >= 4 && kWSlots % 2 == 0 && kSmem <= kSmemMax, "shared memory");
};

struct Ctrl {
  uint64_t wfull[kMaxW], wempty[kMaxW];
  uint64_t xfull[kBufs];      // first block: both halves' codes landed
  uint64_t a_full[kBufs];     // first block: both blocks' weights are in TMEM
  uint64_t consumed[kBufs];   // the MMAs of the step completed: A buffer and token slot are free
  uint64_t d_full[2];
  uint64_t d_empty[2];        // first block: both blocks drained the accumulator
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort_flag;
  int last_flag;
};
static_assert(sizeof(Ctrl) <= kCtrl, "control block");

struct Params {
  const float* s_a;
  const float* s_w;
  uint16_t* y;
  int64_t M, N;
  int64_t G;          // K / 128
  int64_t F2, TT;     // tiles of 256 channels, of T tokens
  int64_t band;       // token tiles of a band
  int64_t pairs;
  int64_t sk_tiles;   // tiles cut along K: the last ones of the order
  int64_t sk_pairs;   // pairs that share them
  int* counters;      // [sk_tiles][2]
  int32_t* part;      // [pairs][2][2][T][128]
  int* err;
  uint64_t limit_ns;
};

// The pair's work: segments (tile, [g0, g1)), first its share of the tiles cut
// along K, then its whole tiles.
struct Work {
  const Params& p;
  int64_t pr, whole;          // pair index; whole tiles of all pairs
  int64_t s, s1;              // share of the cut tiles' steps
  int64_t s_first;            // tile (of the cut ones) in which the share starts
  int64_t q;                  // next whole tile
  int64_t tile, f, t, g0, g1;
  bool cut;
  __device__ __forceinline__ Work(const Params& p_, int64_t pair) : p(p_), pr(pair) {
    const int64_t steps = p.sk_tiles * p.G;
    whole = p.F2 * p.TT - p.sk_tiles;
    s = pr < p.sk_pairs ? pr * steps / p.sk_pairs : 0;
    s1 = pr < p.sk_pairs ? (pr + 1) * steps / p.sk_pairs : 0;
    s_first = s / p.G;
    q = pr;
  }
  __device__ __forceinline__ bool next() {
    if (s < s1) {
      tile = s / p.G;
      g0 = s - tile * p.G;
      g1 = p.G < g0 + (s1 - s) ? p.G : g0 + (s1 - s);
      s += g1 - g0;
      cut = g1 - g0 != p.G;
      place(whole + tile);
      return true;
    }
    if (q >= whole) return false;
    cut = false;
    g0 = 0;
    g1 = p.G;
    place(q);
    q += p.pairs;
    return true;
  }
  __device__ __forceinline__ void place(int64_t i) {
    const int64_t b = i / (p.band * p.F2);
    const int64_t r = i - b * p.band * p.F2;
    const int64_t rows = p.TT - b * p.band < p.band ? p.TT - b * p.band : p.band;
    f = r / rows;
    t = b * p.band + (r - f * rows);
  }
};

// The pair whose share holds step i of the cut tiles.
__device__ __forceinline__ int64_t pair_of_step(int64_t i, const Params& p) {
  const int64_t W = p.sk_tiles * p.G;
  return ((i + 1) * p.sk_pairs + W - 1) / W - 1;
}

__device__ __forceinline__ uint32_t map_to_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

// Arrives on a barrier of either block of the pair.  Block-scope release is
// enough, and all that is ordered: tensor-memory accesses that have completed
// (tcgen05.wait) and are fenced (tcgen05.fence::before_thread_sync).  No data
// passes between the blocks through generic memory here.  With cluster scope
// every arrival waited for the block's outstanding stores, and a K step took
// 0.95 us for any T up to 128.
__device__ __forceinline__ void arrive_cluster(uint32_t remote_bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(remote_bar) : "memory");
}

// Tokens: a box of the 3D code map into this block's shared memory, its bytes
// counted on the first block's barrier.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x,
                                              int32_t y, int32_t z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(policy)
      : "memory");
}

__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrives once on `bar` in both blocks when this thread's MMAs so far completed.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  tmem_ld16(taddr, r);
  tmem_ld16(taddr + 16, r + 16);
}

template <int T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    pair_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x, const Params p) {
  using C = Cfg<T>;
  constexpr int NW = C::kWSlots;
  constexpr int ND = C::kND;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  constexpr uint32_t x_off = NW * kWBytes;
  Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem + x_off + kBufs * C::kXBytes);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = blockIdx.x & 1u;     // the cluster is two consecutive blocks
  const int64_t pr = blockIdx.x >> 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NW; ++i) {
      mbar_init(smem_u32(&ctrl->wfull[i]), 1);
      mbar_init(smem_u32(&ctrl->wempty[i]), 4);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(smem_u32(&ctrl->xfull[i]), 1);
      mbar_init(smem_u32(&ctrl->a_full[i]), 8);
      mbar_init(smem_u32(&ctrl->consumed[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&ctrl->d_full[i]), 1);
      mbar_init(smem_u32(&ctrl->d_empty[i]), 16);
    }
    mbar_init(smem_u32(&ctrl->mma_done), 1);
    ctrl->abort_flag = 0;
    ctrl->last_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&tm_w);
    prefetch_tmap(&tm_x);
  }
  __syncwarp();
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ctrl->tmem_base)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();      // both blocks' barriers are initialised
  tc_fence_after();
  grid_dep_launch();
  const uint32_t tmem = ctrl->tmem_base;
  const WaitCtx ctx{p.err, &ctrl->abort_flag, p.limit_ns};
  int never_abort = 0;
  const WaitCtx drain_ctx{p.err, &never_abort, p.limit_ns};

  if (warp < 4) {
    reg_dec<32>();
    if (warp == 0 && lane == 0) {
      // -------------------------------------------------------- words
      // read once when one token tile takes them, else shared by a band
      const uint64_t pol = p.TT == 1 ? policy_evict_first() : policy_evict_normal();
      Work w(p, pr);
      int issued = 0;
      bool ok = true;
      while (ok && w.next()) {
        const int32_t x = static_cast<int32_t>(w.f * 256 + rank * kF);
        for (int64_t g = w.g0; g < w.g1; ++g) {
          const int slot = issued % NW;
          if (!mbar_wait(smem_u32(&ctrl->wempty[slot]), (static_cast<uint32_t>(issued / NW) & 1u) ^ 1u, ctx, 60)) {
            ok = false;
            break;
          }
          const uint32_t full = smem_u32(&ctrl->wfull[slot]);
          mbar_arrive_expect_tx(full, kWBytes);
          tma_load_2d(sbase + slot * kWBytes, &tm_w, full, x, static_cast<int32_t>(g * 32), pol);
          ++issued;
        }
      }
      // every copy lands before the block ends
      for (int j = issued > NW ? issued - NW : 0; j < issued; ++j)
        (void)mbar_wait(smem_u32(&ctrl->wfull[j % NW]), static_cast<uint32_t>(j / NW) & 1u, drain_ctx, 61);
    } else if (warp == 2 && lane == 0) {
      // -------------------------------------------------------- tokens
      grid_dep_wait();   // the codes come from the previous kernel
      const uint64_t pol = policy_evict_last();
      Work w(p, pr);
      int j = 0;
      bool ok = true;
      while (ok && w.next()) {
        const int32_t row = static_cast<int32_t>(w.t * T + rank * C::kHalf);
        for (int64_t g = w.g0; g < w.g1; ++g, ++j) {
          const int slot = j % kBufs;
          if (!mbar_wait(smem_u32(&ctrl->consumed[slot]), (static_cast<uint32_t>(j / kBufs) & 1u) ^ 1u, ctx, 62)) {
            ok = false;
            break;
          }
          const uint32_t full = smem_u32(&ctrl->xfull[slot]);
          if (rank == 0) mbar_arrive_expect_tx(full, 2 * C::kXBytes);
          tma_load_pair(sbase + x_off + slot * C::kXBytes, &tm_x, map_to_rank(full, 0), 0, row,
                        static_cast<int32_t>(2 * g), pol);
        }
      }
      // the first block sees both blocks' last copies land; the second one
      // leaves only after it (the closing cluster barrier)
      if (rank == 0)
        for (int i = j > kBufs ? j - kBufs : 0; i < j; ++i)
          (void)mbar_wait(smem_u32(&ctrl->xfull[i % kBufs]), static_cast<uint32_t>(i / kBufs) & 1u, drain_ctx, 63);
      if (!ok) {
        // given up: the blocks may have issued different numbers of copies, so
        // allow those in flight a millisecond to land
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000u) __nanosleep(1000);
      }
    } else if (warp == 1 && lane == 0 && rank == 0) {
      // ---------------------------------------------------------- MMAs
      constexpr uint32_t idesc = idesc_f16(256, T, false);
      Work w(p, pr);
      int j = 0, d = 0;
      bool ok = true;
      while (ok && w.next()) {
        for (int64_t g = w.g0; ok && g < w.g1; g += kChunk, ++d) {
          const int n = static_cast<int>(w.g1 - g < kChunk ? w.g1 - g : kChunk);
          const int db = d % ND;
          const uint32_t dcol = tmem + C::kColD + db * T;
          if (!mbar_wait(smem_u32(&ctrl->d_empty[db]), (static_cast<uint32_t>(d / ND) & 1u) ^ 1u, ctx, 64)) {
            ok = false;
            break;
          }
          for (int i = 0; i < n; ++i, ++j) {
            const int slot = j % kBufs;
            const uint32_t ph = static_cast<uint32_t>(j / kBufs) & 1u;
            if (!mbar_wait(smem_u32(&ctrl->xfull[slot]), ph, ctx, 65) ||
                !mbar_wait(smem_u32(&ctrl->a_full[slot]), ph, ctx, 66)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t b0 = smem_desc(sbase + x_off + slot * C::kXBytes, 16u, 1024u, 2u);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
              const uint32_t off = static_cast<uint32_t>(ks >> 2) * (C::kHalf * 128u) + static_cast<uint32_t>(ks & 3) * 32u;
              mma_pair(dcol, tmem + slot * 64 + ks * 8, b0 + (off >> 4), idesc, (i > 0 || ks > 0) ? 1u : 0u);
            }
            commit_pair(smem_u32(&ctrl->consumed[slot]));
          }
          if (ok) commit_pair(smem_u32(&ctrl->d_full[db]));
        }
      }
      asm volatile(
          "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(&ctrl->mma_done))
          : "memory");
      (void)mbar_wait(smem_u32(&ctrl->mma_done), 0u, drain_ctx, 67);
    }
    __syncwarp();
  } else if (warp < 12) {
    // ---------------------------------------------------------- widening
    reg_dec<64>();
    const int ct = threadIdx.x - 128;
    const int grp = ct >> 7;
    const int r = ct & 127;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    Work w(p, pr);
    int j = 0;
    bool ok = true;
    while (ok && w.next()) {
      for (int64_t g = w.g0; g < w.g1; ++g, ++j) {
        if ((j & 1) != grp) continue;
        const int ws = j % NW;
        const int ab = j % kBufs;
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&ctrl->wfull[ws]), static_cast<uint32_t>(j / NW) & 1u, ctx, 68));
        if (!ok) break;
        const uint32_t* src = reinterpret_cast<const uint32_t*>(smem + ws * kWBytes);
        uint32_t word[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) word[i] = src[i * kF + r];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctrl->wempty[ws]));
        // buffer ab was last used by step j - 4, this group's as well
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&ctrl->consumed[ab]),
                                                  (static_cast<uint32_t>(j / kBufs) & 1u) ^ 1u, ctx, 69));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          uint32_t v[16];
#pragma unroll
          for (int i = 0; i < 8; ++i) biased_u8x4_to_f16x4(word[8 * h + i], v[2 * i], v[2 * i + 1]);
          tmem_st16(tmem + lane_off + ab * 64 + h * 16, v);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(map_to_rank(smem_u32(&ctrl->a_full[ab]), 0));
      }
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------- epilogue
    reg_inc<160>();
    grid_dep_wait();   // outputs and workspace may still be in use upstream
    constexpr int E = C::kCols;
    const int et = threadIdx.x - 384;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int col0 = ((warp - 12) >> 2) * E;
    int32_t acc[E];
    Work w(p, pr);
    int d = 0;
    bool ok = true;
    while (ok && w.next()) {
      for (int64_t g = w.g0; g < w.g1; g += kChunk, ++d) {
        const int db = d % ND;
        ok = __all_sync(0xFFFFFFFFu,
                        mbar_wait(smem_u32(&ctrl->d_full[db]), static_cast<uint32_t>(d / ND) & 1u, ctx, 70));
        if (!ok) break;
        tc_fence_after();
        const uint32_t dcol = tmem + lane_off + C::kColD + db * T + col0;
#pragma unroll
        for (int c = 0; c < E; c += 16) {
          uint32_t v[16];
          tmem_ld16(dcol + c, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int32_t x = __float2int_rn(__uint_as_float(v[i]));
            acc[c + i] = g == w.g0 ? x : acc[c + i] + x;
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(map_to_rank(smem_u32(&ctrl->d_empty[db]), 0));
      }
      if (!named_bar_and(1, kEpiThreads, ok)) break;
      bool finish = true;
      if (w.cut) {
        // the contributors of this tile, and this block's place among them
        const int64_t c0 = pair_of_step(w.tile * p.G, p);
        const int64_t c1 = pair_of_step(w.tile * p.G + p.G - 1, p);
        int* counter = p.counters + w.tile * 2 + rank;
        const int others = static_cast<int>(c1 - c0);
        // if all the others have arrived, this block's sums stay in registers
        if (et == 0) ctrl->last_flag = ld_acquire_gpu(counter) == others ? 1 : 0;
        named_bar_sync(1, kEpiThreads);
        finish = ctrl->last_flag != 0;
        named_bar_sync(1, kEpiThreads);
        if (!finish) {
          const int mine = w.tile == w.s_first ? 0 : 1;
          int32_t* dst = p.part + ((pr * 2 + mine) * 2 + rank) * static_cast<int64_t>(T * kF) + col0 * kF + r;
#pragma unroll
          for (int c = 0; c < E; ++c) dst[c * kF] = acc[c];
          named_bar_sync(1, kEpiThreads);
          if (et == 0) ctrl->last_flag = atomic_add_acq_rel_gpu(counter, 1) == others ? 1 : 0;
          named_bar_sync(1, kEpiThreads);
          finish = ctrl->last_flag != 0;
          named_bar_sync(1, kEpiThreads);
        }
        if (finish) {
          for (int64_t c = c0; c <= c1; ++c) {
            if (c == pr) continue;
            const int64_t start = c * (p.sk_tiles * p.G) / p.sk_pairs;
            const int theirs = start / p.G == w.tile ? 0 : 1;
            const int32_t* src = p.part + ((c * 2 + theirs) * 2 + rank) * static_cast<int64_t>(T * kF) + col0 * kF + r;
#pragma unroll
            for (int i = 0; i < E; i += 16) {
              int32_t v[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) v[k] = src[(i + k) * kF];
#pragma unroll
              for (int k = 0; k < 16; ++k) acc[i + k] += v[k];
            }
          }
        }
      }
      if (finish) {
        const int64_t n = w.f * 256 + rank * kF + r;
        const int64_t m0 = w.t * T + col0;
        if (n < p.N && m0 < p.M) {
          const float sw = __ldg(p.s_w + n);
          uint16_t* dst = p.y + m0 * p.N + n;
#pragma unroll
          for (int c = 0; c < E; ++c) {
            if (m0 + c < p.M)
              dst[c * p.N] = __bfloat16_as_ushort(__float2bfloat16_rn(
                  __fmul_rn(__fmul_rn(__int2float_rn(acc[c]), sw), __ldg(p.s_a + m0 + c))));
          }
        }
      }
    }
    __syncwarp();
  }

  // ------------------------------------------------------------- teardown
  // The cluster barrier keeps each block's shared and tensor memory until the
  // other one has stopped arriving on it, and the first block's MMAs are done.
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

}  // namespace pair
}  // namespace qlin
