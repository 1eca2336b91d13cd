// gemm_channel_pair.cuh -- device side of the per-channel W8A8 linear on
// tcgen05 for batches above the streaming kernel's: one persistent pair of
// thread blocks (two SMs, tcgen05 cta_group::2) per tile of 256 output channels
// x T tokens.
//
//   * The MMA runs with the weights as operand A (widened by threads straight
//     into tensor memory, 128 channels a block) and the tokens as operand B
//     (T columns, fp16 codes, 128-byte swizzled).  Each block loads its own
//     words and half of the tokens, and one cta_group::2 MMA of 256 x T, issued
//     by the first block, reads both halves where they lie: the pair reads every
//     operand byte once, and an SM takes in 16 KB of words and T x 128 B of codes
//     a K step.  (MMAs of 128 x T of each block's own need all T tokens in both:
//     96 x 5120 x 248320 209 us in this form, 236 with every block loading them
//     all; 128 x 5120 x 5120 12.7 and 13.7.)
//   * An accumulator takes at most 1024 of K (exact below 2^24); the
//     epilogue adds each such chunk to int32 registers, under the next chunk's
//     MMAs: tensor memory holds two accumulators.  (T = 256 has room for one,
//     and the tensor pipe idled for 2000 of every 12,000 cycles.)  At T = 192
//     that leaves room for 256 of K as operand A, cut into units of 64 instead
//     of 128 to keep four of them on the way.
//   * Work: whole tiles go round the pairs in bands of token tiles, so the
//     pairs running at one time share a few channel tiles and one band's
//     tokens in L2.  The tiles that do not fill a last round are cut along
//     K instead, evenly between the pairs, and come first: a block publishes
//     its int32 partial of such a tile, and the last one to arrive on the
//     tile's counter adds the others' to its own.  Integer sums: the result
//     does not depend on who is last.
//   * Few tiles: the two to four pairs of a cluster share a tile, each with its
//     part of K.  Their sums meet in shared memory, where each block finishes
//     its share of the tokens: no workspace, no counters, 2 us instead of 6.
//   * Roles of a block's 20 warps: 0 streams words and 2 tokens by TMA, 1
//     issues the MMAs, 4-11 widen weights (two groups taking alternate steps),
//     12-19 drain and write.
//
// What bounds it: at thousands of tokens the MMAs under the power limit (8192 x
// 5120 x 34816 1.58 to 1.81 ms, 1610 to 1850 TF/s); at 64 to a few hundred, HBM and
// the words and codes on their way from L2 to the SMs, 10 to 12 TB/s (64 x 5120 x
// 248320 194 us, 6.7 TB/s of HBM; 96 tokens 209, 6.3); with little of K the way out
// of tensor memory (836 x 256 x 95952 80 us).
//
// Every wait is bounded; a wait that runs out records an error, aborts the
// block's roles, and the block still drains its copies and frees its TMEM.
#pragma once

#include <cuda_bf16.h>

#include "channel_plan.h"
#include "qlin_device.cuh"
#include "qlin_internal.h"

namespace qlin {
namespace pair {

constexpr int kF = 128;                 // channels of one block
constexpr int kChunkK = 1024;           // K of an accumulator
constexpr int kND = 2;                  // accumulators
constexpr int kA = 4;                   // operand A buffers in TMEM, one unit of K each
constexpr uint32_t kWBytes = 32 * kF * 4;
constexpr int kThreads = 640;
constexpr int kEpiThreads = 256;
constexpr uint32_t kCtrl = 2048;
constexpr uint32_t kSmemMax = 232448;
constexpr int kMaxW = 8;
constexpr int kMaxU = 8;

template <int T>
struct Cfg {
  static constexpr int kHalf = T / 2;                         // tokens that one block loads
  static constexpr int kUnit = T == 192 ? 64 : 128;           // K of a unit: one A buffer, one token slot
  static constexpr int kPerStep = 128 / kUnit;                // units of a K step
  static constexpr int kChunk = kChunkK / kUnit;              // units of an accumulator
  static constexpr int kACols = kUnit / 2;
  static constexpr uint32_t kXBytes = kHalf * kUnit * 2u;     // a unit's codes in one block
  static constexpr int kX = T == 192 ? 8 : 4;                 // token slots
  static constexpr int kE = T / 2;                            // sums of an epilogue thread
  static constexpr uint32_t kColD = kA * kACols;
  static constexpr int kWSlotsFit = static_cast<int>((kSmemMax - 1024 - kCtrl - kX * kXBytes) / kWBytes) & ~1;
  static constexpr int kWSlots = kWSlotsFit < kMaxW ? kWSlotsFit : kMaxW;   // even: a slot stays with one widening group
  static constexpr uint32_t kSmem = 1024 + kCtrl + kX * kXBytes + kWSlots * kWBytes;
  // Registers a thread: the block is launched with 96 and the roles trade them
  // within that.  (Spills are dear: the rings leave no L1 to speak of.)
  static constexpr int kRegsCtl = 48;
  static constexpr int kRegsConv = T > 128 ? 64 : 72;
  static constexpr int kRegsEpi = T > 128 ? 152 : 144;
  static constexpr int kRegsSum = 128 * kRegsCtl + 256 * kRegsConv + 256 * kRegsEpi;
  static_assert(kRegsSum <= 96 * kThreads, "setmaxnreg draws on what the block was launched with");
  static_assert(T % 32 == 0 && T >= 64 && T <= 192, "token tile");
  static_assert(kColD + kND * T <= 512 && kE % 16 == 0, "TMEM budget");
  static_assert(kX >= kA && kX <= kMaxU && kX % 2 == 0, "token slots");
  static_assert(kWSlots >= 4 && kWSlots % 2 == 0 && kSmem <= kSmemMax, "shared memory");
};

struct Ctrl {
  uint64_t wfull[kMaxW], wempty[kMaxW];
  // of a unit; the first block's `ready` and d_empty count both blocks, the
  // second's are not used
  uint64_t ready[kMaxU];      // its weights are in TMEM and its codes landed
  uint64_t consumed[kMaxU];   // the MMAs that read them completed
  uint64_t d_full[2];
  uint64_t d_empty[2];        // the accumulator is drained
  uint64_t mma_done;
  uint64_t part_here;         // partials of a cut tile landed
  alignas(16) float s_a[192]; // of the tile's tokens
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
  int G;              // K / 128
  int F2, TT;         // tiles of 256 channels, of T tokens
  int band;           // token tiles of a band
  int pairs;
  int sk_tiles;       // tiles cut along K: the last ones of the order
  int sk_pairs;       // pairs that share them
  int parts;          // pairs of a cluster, which then are those that share a tile
  int* counters;      // [sk_tiles][2]
  int32_t* part;      // [pairs][2][2][T][128]
  int* err;
  uint64_t limit_ns;
};

// The pair's work: segments (tile, [g0, g1)), first its share of the tiles cut
// along K, then its whole tiles.
struct Work {
  const Params& p;
  int s, s1;              // share of the cut tiles' steps
  int q;                  // next whole tile
  int tile, f, t, g0, g1;
  bool cut;
  __device__ __forceinline__ Work(const Params& p_, int pair) : p(p_), s(0), s1(0), q(pair) {
    if (pair < p.sk_pairs) {
      s = pair * (p.sk_tiles * p.G) / p.sk_pairs;
      s1 = (pair + 1) * (p.sk_tiles * p.G) / p.sk_pairs;
    }
  }
  __device__ __forceinline__ int whole() const { return p.F2 * p.TT - p.sk_tiles; }   // of all pairs
  __device__ __forceinline__ bool next() {
    if (s < s1) {
      tile = s / p.G;
      g0 = s - tile * p.G;
      g1 = min(p.G, g0 + (s1 - s));
      s += g1 - g0;
      cut = g1 - g0 != p.G;
      place(whole() + tile);
      return true;
    }
    if (q >= whole()) return false;
    cut = false;
    g0 = 0;
    g1 = p.G;
    place(q);
    q += p.pairs;
    return true;
  }
  __device__ __forceinline__ bool last() const { return s >= s1 && q >= whole(); }   // nothing after this segment
  __device__ __forceinline__ void place(int i) {
    const int b = i / (p.band * p.F2);
    const int r = i - b * p.band * p.F2;
    const int rows = min(p.TT - b * p.band, p.band);
    f = r / rows;
    t = b * p.band + (r - f * rows);
  }
};

// The pair whose share holds step i of the cut tiles.
__device__ __forceinline__ int pair_of_step(int i, const Params& p) {
  const int W = p.sk_tiles * p.G;
  return ((i + 1) * p.sk_pairs + W - 1) / W - 1;
}

__device__ __forceinline__ uint32_t map_to_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

// Arrives on the first block's barrier at this offset.
// Block-scope release is enough for it too, and all that is ordered: tensor-
// memory accesses that have completed (tcgen05.wait) and are fenced
// (tcgen05.fence::before_thread_sync).  No data passes between the blocks
// through generic memory here.  With cluster scope every arrival waited for
// the block's outstanding stores, and a K step took 0.95 us for any T up to 128.
__device__ __forceinline__ void arrive(uint32_t bar, uint32_t first) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(map_to_rank(bar, first)) : "memory");
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

// Arrives once on `bar`, of this block or (kBoth) of both, when this thread's
// MMAs so far have completed.
template <bool kBoth>
__device__ __forceinline__ void commit(uint32_t bar, uint16_t both) {
  if constexpr (kBoth)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(both)
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t cluster_rank_of_block() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ int4 ld_cluster_int4(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

// Adds the integers that two fp32 words hold (magnitude up to 2^24) to a0 and
// a1, each with kIntegerBias on top, modulo 2^32.  The conversion instruction
// runs at a quarter of the additions' rate here (a drain of 256 x 128 took
// 2000 cycles with it), so: x + 1.5 * 2^35 keeps round(x / 4096) in the low
// bits of its significand, what remains of x is at most 2048, and that plus
// 1.5 * 2^23 is an integer in the low bits of its significand.
constexpr uint32_t kBigMagic = 0x51400000u;     // 1.5 * 2^35
constexpr uint32_t kSmallMagic = 0x4B400000u;   // 1.5 * 2^23
constexpr uint32_t kIntegerBias = (kBigMagic << 12) + kSmallMagic;
__device__ __forceinline__ void add_integers(uint32_t x0, uint32_t x1, int32_t& a0, int32_t& a1) {
  uint32_t h0, h1, l0, l1;
  asm("{\n\t.reg .b64 x, h, l, m, n;\n\t"
      "mov.b64 x, {%4, %5};\n\t"
      "mov.b64 m, {%6, %6};\n\t"
      "mov.b64 n, {%7, %7};\n\t"
      "add.rn.f32x2 h, x, m;\n\t"
      "mov.b64 {%0, %1}, h;\n\t"
      "mov.b64 m, {%8, %8};\n\t"
      "add.rn.f32x2 h, h, m;\n\t"          // round(x / 4096) * 4096, exact
      "mov.b64 m, {%9, %9};\n\t"
      "fma.rn.f32x2 l, h, m, x;\n\t"       // x less that, exact
      "add.rn.f32x2 l, l, n;\n\t"
      "mov.b64 {%2, %3}, l;\n\t}"
      : "=r"(h0), "=r"(h1), "=r"(l0), "=r"(l1)
      : "r"(x0), "r"(x1), "r"(kBigMagic), "r"(kSmallMagic), "r"(kBigMagic | 0x80000000u), "r"(0xBF800000u));
  a0 = static_cast<int32_t>(static_cast<uint32_t>(a0) + (h0 << 12) + l0);
  a1 = static_cast<int32_t>(static_cast<uint32_t>(a1) + (h1 << 12) + l1);
}

template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

template <int T>
__global__ void __launch_bounds__(kThreads, 1)
    pair_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x, const Params p) {
  using C = Cfg<T>;
  constexpr int NW = C::kWSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  constexpr uint32_t x_off = NW * kWBytes;
  Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem + x_off + C::kX * C::kXBytes);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = blockIdx.x & 1u;     // in the pair, two consecutive blocks
  const uint32_t first = cluster_rank_of_block() & ~1u;      // the pair's place in its cluster
  const uint16_t both = static_cast<uint16_t>(3u << first);  // its blocks
  const int pr = static_cast<int>(blockIdx.x >> 1);

  if (threadIdx.x == 0) {
    for (int i = 0; i < NW; ++i) {
      mbar_init(smem_u32(&ctrl->wfull[i]), 1);
      mbar_init(smem_u32(&ctrl->wempty[i]), 4);
    }
    for (int i = 0; i < C::kX; ++i) {
      mbar_init(smem_u32(&ctrl->ready[i]), 9);      // both blocks' widening warps, and the token copies' issuer
      mbar_init(smem_u32(&ctrl->consumed[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&ctrl->d_full[i]), 1);
      mbar_init(smem_u32(&ctrl->d_empty[i]), 16);
    }
    mbar_init(smem_u32(&ctrl->mma_done), 1);
    mbar_init(smem_u32(&ctrl->part_here), 1);
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
  cluster_sync();      // the cluster's barriers are initialised
  tc_fence_after();
  grid_dep_launch();
  const uint32_t tmem = 0;      // the block holds all 512 columns, so they start at 0
  const WaitCtx ctx{p.err, &ctrl->abort_flag, p.limit_ns};
  int never_abort = 0;
  const WaitCtx drain_ctx{p.err, &never_abort, p.limit_ns};

  if (warp < 4) {
    reg_dec<C::kRegsCtl>();
    if (warp == 0 && lane == 0) {
      // -------------------------------------------------------- words
      // read once when one token tile takes them, else shared by a band
      const uint64_t pol = p.TT == 1 ? policy_evict_first() : policy_evict_normal();
      Work w(p, pr);
      int issued = 0;
      bool ok = true;
      while (ok && w.next()) {
        const int32_t x = w.f * 256 + static_cast<int>(rank) * kF;
        for (int g = w.g0; g < w.g1; ++g) {
          const int slot = issued % NW;
          if (!mbar_wait(smem_u32(&ctrl->wempty[slot]), (static_cast<uint32_t>(issued / NW) & 1u) ^ 1u, ctx, 60)) {
            ok = false;
            break;
          }
          const uint32_t full = smem_u32(&ctrl->wfull[slot]);
          mbar_arrive_expect_tx(full, kWBytes);
          tma_load_2d(sbase + slot * kWBytes, &tm_w, full, x, g * 32, pol);
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
        const int32_t row = w.t * T + static_cast<int>(rank) * C::kHalf;
        for (int u = w.g0 * C::kPerStep; u < w.g1 * C::kPerStep; ++u, ++j) {
          const int slot = j % C::kX;
          if (!mbar_wait(smem_u32(&ctrl->consumed[slot]), (static_cast<uint32_t>(j / C::kX) & 1u) ^ 1u, ctx, 62)) {
            ok = false;
            break;
          }
          const uint32_t full = smem_u32(&ctrl->ready[slot]);
          const uint32_t dst = sbase + x_off + slot * C::kXBytes;
          if (rank == 0) mbar_arrive_expect_tx(full, 2 * C::kXBytes);
#pragma unroll
          for (int h = 0; h < C::kUnit / 64; ++h)    // each 64 of K is kHalf rows x 128 B
            tma_load_pair(dst + h * (C::kHalf * 128u), &tm_x, map_to_rank(full, first), 0, row,
                          u * (C::kUnit / 64) + h, pol);
        }
      }
      // the last units' MMAs completed: both blocks' copies landed, and no
      // arrival is on its way here when the block ends
      if (ok)
        for (int i = j > C::kX ? j - C::kX : 0; i < j; ++i)
          (void)mbar_wait(smem_u32(&ctrl->consumed[i % C::kX]), static_cast<uint32_t>(i / C::kX) & 1u, drain_ctx, 63);
      if (!ok) {
        // given up: the blocks may have issued different numbers of copies, so
        // allow those in flight a millisecond to land
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000u) __nanosleep(1000);
      }
    } else if (warp == 1 && rank == 0) {
      // ---------------------------------------------------------- MMAs
      // The whole warp goes through the loop, on values that the compiler can
      // see to be uniform (no branch on a lane's own wait, TMEM from column 0),
      // and one lane issues: the MMA's operands are uniform registers, and filling
      // them from a single lane's made an issue take 60 cycles.
      constexpr uint32_t idesc = idesc_f16(256, T, false);
      const bool leader = elect_one();
      Work w(p, pr);
      int slot = 0, ab = 0, db = 0;
      uint32_t slot_par = 0u, d_par = 1u;
      bool ok = true;
      while (ok && w.next()) {
        const int n = (w.g1 - w.g0) * C::kPerStep;
        for (int i = 0; i < n; ++i) {
          const int ci = i % C::kChunk;
          if (ci == 0) ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&ctrl->d_empty[db]), d_par, ctx, 64));
          if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&ctrl->ready[slot]), slot_par, ctx, 65));
          if (!ok) break;
          tc_fence_after();
          const uint64_t b0 = smem_desc(sbase + x_off + slot * C::kXBytes, 16u, 1024u, 2u);
          const uint32_t a0 = static_cast<uint32_t>(ab * C::kACols);
          const uint32_t dcol = static_cast<uint32_t>(C::kColD + db * T);
          const bool ends = ci == C::kChunk - 1 || i == n - 1;
          if (leader) {
#pragma unroll
            for (int ks = 0; ks < C::kUnit / 16; ++ks) {
              const uint32_t off = static_cast<uint32_t>(ks >> 2) * (C::kHalf * 128u) + static_cast<uint32_t>(ks & 3) * 32u;
              mma_pair(dcol, a0 + ks * 8, b0 + (off >> 4), idesc, (ci > 0 || ks > 0) ? 1u : 0u);
            }
            commit<true>(smem_u32(&ctrl->consumed[slot]), both);
            if (ends) commit<true>(smem_u32(&ctrl->d_full[db]), both);
          }
          __syncwarp();
          if (++slot == C::kX) {
            slot = 0;
            slot_par ^= 1u;
          }
          if (++ab == kA) ab = 0;
          if (ends && ++db == kND) {
            db = 0;
            d_par ^= 1u;
          }
        }
      }
      if (leader) commit<false>(smem_u32(&ctrl->mma_done), both);
      __syncwarp();
      (void)mbar_wait(smem_u32(&ctrl->mma_done), 0u, drain_ctx, 67);
    }
    __syncwarp();
  } else if (warp < 12) {
    // ---------------------------------------------------------- widening
    reg_dec<C::kRegsConv>();
    const int ct = threadIdx.x - 128;
    const int grp = ct >> 7;
    const int r = ct & 127;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    Work w(p, pr);
    int j = 0;
    bool ok = true;
    while (ok && w.next()) {
      for (int g = w.g0; g < w.g1; ++g, ++j) {
        if ((j & 1) != grp) continue;
        const int ws = j % NW;
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&ctrl->wfull[ws]), static_cast<uint32_t>(j / NW) & 1u, ctx, 68));
        if (!ok) break;
        const uint32_t* src = reinterpret_cast<const uint32_t*>(smem + ws * kWBytes);
        uint32_t word[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) word[i] = src[i * kF + r];
#pragma unroll
        for (int part = 0; part < C::kPerStep; ++part) {
          const int u = j * C::kPerStep + part;
          // The A buffer was last used by unit u - kA.  Its barrier's next phase
          // is of unit u - kA + kX, whose weights come after these.
          if (u >= kA)
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&ctrl->consumed[(u - kA) % C::kX]),
                                                   static_cast<uint32_t>((u - kA) / C::kX) & 1u, ctx, 69));
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int h = 0; h < C::kUnit / 32; ++h) {
            uint32_t v[16];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              biased_u8x4_to_f16x4(word[part * (C::kUnit / 4) + 8 * h + i], v[2 * i], v[2 * i + 1]);
            tmem_st16(tmem + lane_off + u % kA * C::kACols + h * 16, v);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            arrive(smem_u32(&ctrl->ready[u % C::kX]), first);
            // The slot is free when the words are in tensor memory, not before: an
            // arrival ahead of that does not keep the compiler from loading the last
            // words behind it, where they can be those of a later step.
            if (part == C::kPerStep - 1) mbar_arrive(smem_u32(&ctrl->wempty[ws]));
          }
        }
        if (!ok) break;
      }
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------- epilogue
    reg_inc<C::kRegsEpi>();
    grid_dep_wait();   // outputs and workspace may still be in use upstream
    constexpr int E = C::kE;
    const int et = threadIdx.x - 384;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int col0 = ((warp - 12) >> 2) * E;
    int32_t acc[E];
    Work w(p, pr);
    int d = 0;
    uint32_t part_par = 0u;
    bool ok = true, summed = false;
    while (ok && w.next()) {
      named_bar_sync(1, kEpiThreads);     // the previous tile's scales are read
      if (et < T) {
        const int64_t m = static_cast<int64_t>(w.t) * T + et;
        ctrl->s_a[et] = m < p.M ? __ldg(p.s_a + m) : 0.0f;
      }
      // Two neighbouring lanes (channels) exchange a value of each two tokens,
      // so that a lane writes both channels of one: 4 bytes, and half the stores.
      const int odd = lane & 1;
      auto write2 = [&](int c, float p0, float p1, float sw, uint16_t* dst, int rows) {   // the sums of tokens c and c + 1
        const float2 sa = *reinterpret_cast<const float2*>(ctrl->s_a + col0 + c);
        const uint32_t mine = bf16x2_rn(__fmul_rn(__fmul_rn(p0, sw), sa.x), __fmul_rn(__fmul_rn(p1, sw), sa.y));
        const uint32_t theirs = __shfl_xor_sync(0xFFFFFFFFu, mine, 1);
        // {theirs.hi, mine.hi} or {mine.lo, theirs.lo}
        if (c < rows) *reinterpret_cast<uint32_t*>(dst) = prmt(mine, theirs, odd ? 0x3276u : 0x5410u);
      };
      auto output = [&](int& rows, float& sw) {   // of token `odd`; rows: that this lane writes
        const int64_t n = static_cast<int64_t>(w.f) * 256 + rank * kF + r;
        sw = n < p.N ? __ldg(p.s_w + n) : 0.0f;
        const int64_t m0 = static_cast<int64_t>(w.t) * T + col0;
        rows = n < p.N ? static_cast<int>(p.M - m0 < E ? p.M - m0 : E) - odd : 0;
        return p.y + (m0 + odd) * p.N + (n - odd);
      };
      if (!w.cut && w.g1 - w.g0 <= kChunkK / 128) {
        // One accumulator holds the whole sum, exact in fp32 as it is (4286 x 384 x
        // 48584 193 us; through the integers 284).
        const int db = d % kND;
        int rows;
        float sw;
        uint16_t* dst = output(rows, sw);
        ok = __all_sync(0xFFFFFFFFu,
                        mbar_wait(smem_u32(&ctrl->d_full[db]), static_cast<uint32_t>(d / kND) & 1u, ctx, 70));
        if (!named_bar_and(1, kEpiThreads, ok)) break;
        tc_fence_after();
        const uint32_t dcol = tmem + lane_off + C::kColD + db * T + col0;
        uint32_t v[2][16];
        tmem_ld16(dcol, v[0]);
#pragma unroll
        for (int c = 0; c < E; c += 16) {
          tmem_wait_ld();
          if (c + 16 < E) tmem_ld16(dcol + c + 16, v[(c / 16 + 1) & 1]);
#pragma unroll
          for (int i = 0; i < 16; i += 2, dst += 2 * p.N)
            write2(c + i, __uint_as_float(v[c / 16 & 1][i]), __uint_as_float(v[c / 16 & 1][i + 1]), sw, dst, rows);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive(smem_u32(&ctrl->d_empty[db]), first);
        ++d;
        continue;
      }
#pragma unroll
      for (int c = 0; c < E; ++c) acc[c] = 0;
      uint32_t chunks = 0;
      for (int g = w.g0; g < w.g1; g += kChunkK / 128, ++d) {
        const int db = d % kND;
        ok = __all_sync(0xFFFFFFFFu,
                        mbar_wait(smem_u32(&ctrl->d_full[db]), static_cast<uint32_t>(d / kND) & 1u, ctx, 70));
        if (!ok) break;
        tc_fence_after();
        const uint32_t dcol = tmem + lane_off + C::kColD + db * T + col0;
        constexpr int kCols = E == 32 ? 32 : 16;   // of one batch of TMEM loads
#pragma unroll
        for (int c = 0; c < E; c += kCols) {
          uint32_t v[kCols];
#pragma unroll
          for (int k = 0; k + 16 <= kCols; k += 16) tmem_ld16(dcol + c + k, v + k);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < kCols; i += 2) add_integers(v[i], v[i + 1], acc[c + i], acc[c + i + 1]);
        }
        ++chunks;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive(smem_u32(&ctrl->d_empty[db]), first);
      }
#pragma unroll
      for (int c = 0; c < E; ++c) acc[c] = static_cast<int32_t>(static_cast<uint32_t>(acc[c]) - chunks * kIntegerBias);
      if (!named_bar_and(1, kEpiThreads, ok)) break;
      if (p.parts > 1) {
        summed = true;
        break;
      }
      bool finish = true;
      if (w.cut) {
        // the contributors of this tile, and this block's place among them
        const int c0 = pair_of_step(w.tile * p.G, p);
        const int c1 = pair_of_step(w.tile * p.G + p.G - 1, p);
        int* counter = p.counters + w.tile * 2 + rank;
        const int others = c1 - c0;
        auto slot_of = [&](int c) {   // a pair's partials: of the tile its share starts in, and of its last one
          const int first = c * (p.sk_tiles * p.G) / p.sk_pairs / p.G;
          return p.part + static_cast<int64_t>((c * 2 + (first == w.tile ? 0 : 1)) * 2 + static_cast<int>(rank)) * (T * kF);
        };
        // if all the others have arrived, this block's sums stay in registers
        if (et == 0) ctrl->last_flag = ld_acquire_gpu(counter) == others ? 1 : 0;
        named_bar_sync(1, kEpiThreads);
        finish = ctrl->last_flag != 0;
        named_bar_sync(1, kEpiThreads);
        if (!finish) {
          int32_t* dst = slot_of(pr) + col0 * kF + r;
#pragma unroll
          for (int c = 0; c < E; ++c) dst[c * kF] = acc[c];
          named_bar_sync(1, kEpiThreads);
          if (et == 0) ctrl->last_flag = atomic_add_acq_rel_gpu(counter, 1) == others ? 1 : 0;
          named_bar_sync(1, kEpiThreads);
          finish = ctrl->last_flag != 0;
          named_bar_sync(1, kEpiThreads);
        }
        if (finish && w.last()) {
          // The pair's last segment: its rings are idle, and the others' partials
          // come into them by bulk copies, as many at a time as there is room for
          // (through registers a partial takes a round trip for every 32 tokens).
          constexpr uint32_t kPart = T * kF * 4u;
          constexpr int kRoom = static_cast<int>((NW * kWBytes + C::kX * C::kXBytes) / kPart);
          int c = c0;
          while (c <= c1) {
            if (et == 0) {
              // the rings were read, and the partials written, by generic accesses
              fence_proxy_async_smem();
              fence_proxy_async_global();
            }
            int n = 0, next = c;
            for (; next <= c1 && n < kRoom; ++next) {
              if (next == pr) continue;
              if (et == 0) {
                mbar_expect_tx(smem_u32(&ctrl->part_here), kPart);
                bulk_load(sbase + n * kPart, slot_of(next), kPart, smem_u32(&ctrl->part_here));
              }
              ++n;
            }
            if (et == 0) mbar_arrive(smem_u32(&ctrl->part_here));
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&ctrl->part_here), part_par, drain_ctx, 73));
            part_par ^= 1u;
            if (!named_bar_and(2, kEpiThreads, ok)) break;
            for (int i = 0; i < n; ++i) {
              const int32_t* src = reinterpret_cast<const int32_t*>(smem + i * kPart) + col0 * kF + r;
#pragma unroll
              for (int k = 0; k < E; ++k) acc[k] += src[k * kF];
            }
            named_bar_sync(1, kEpiThreads);
            c = next;
          }
          finish = ok;
        } else if (finish) {
          for (int c = c0; c <= c1; ++c) {
            if (c == pr) continue;
            const int32_t* src = slot_of(c) + col0 * kF + r;
            constexpr int kBatch = E <= 48 ? E : 32;   // loads in flight, as the registers allow
#pragma unroll
            for (int i = 0; i < E; i += kBatch) {
              int32_t v[kBatch];
#pragma unroll
              for (int k = 0; k < kBatch; ++k) v[k] = src[(i + k) * kF];
#pragma unroll
              for (int k = 0; k < kBatch; ++k) acc[i + k] += v[k];
            }
          }
        }
      }
      if (finish) {
        int rows;
        float sw;
        uint16_t* dst = output(rows, sw);
#pragma unroll
        for (int c = 0; c < E; c += 2, dst += 2 * p.N)
          write2(c, __int2float_rn(acc[c]), __int2float_rn(acc[c + 1]), sw, dst, rows);
      }
    }
    if (p.parts > 1) {
      // The cluster's pairs hold sums of one tile, each over its part of K.
      // Each block leaves its own in shared memory, in its idle rings, and
      // finishes its share of the tokens.
      int32_t* mine = reinterpret_cast<int32_t*>(smem);
      if (summed) {
#pragma unroll
        for (int c = 0; c < E; ++c) mine[(col0 + c) * kF + r] = acc[c];
      }
      __syncwarp();
      cluster_sync();
      if (summed) {
        const int share = (T + p.parts - 1) / p.parts;
        const int tok0 = static_cast<int>(first >> 1) * share;
        const int64_t rows = p.M - static_cast<int64_t>(w.t) * T;    // of the tile
        const int tok1 = static_cast<int>(min(static_cast<int64_t>(min(T, tok0 + share)), rows));
        const int64_t n = static_cast<int64_t>(w.f) * 256 + rank * kF + 4 * lane;
        const float4 sw = n < p.N ? __ldg(reinterpret_cast<const float4*>(p.s_w + n)) : make_float4(0, 0, 0, 0);
        constexpr int kAhead = 3;     // tokens of a warp on their way
        for (int t0 = tok0 + warp - 12; t0 < tok1; t0 += 8 * kAhead) {
          int4 v[kAhead][kMaxParts];
#pragma unroll
          for (int k = 0; k < kAhead; ++k)
#pragma unroll
            for (int i = 0; i < kMaxParts; ++i)
              v[k][i] = t0 + 8 * k < tok1 && i < p.parts
                            ? ld_cluster_int4(map_to_rank(sbase + ((t0 + 8 * k) * kF + 4 * lane) * 4, 2 * i + rank))
                            : make_int4(0, 0, 0, 0);
#pragma unroll
          for (int k = 0; k < kAhead; ++k) {
            const int t = t0 + 8 * k;
            if (t >= tok1 || n >= p.N) continue;
            int4 sum = v[k][0];
#pragma unroll
            for (int i = 1; i < kMaxParts; ++i) {
              sum.x += v[k][i].x;
              sum.y += v[k][i].y;
              sum.z += v[k][i].z;
              sum.w += v[k][i].w;
            }
            const float sa = ctrl->s_a[t];
            uint2 out;
            out.x = bf16x2_rn(__fmul_rn(__fmul_rn(__int2float_rn(sum.x), sw.x), sa),
                              __fmul_rn(__fmul_rn(__int2float_rn(sum.y), sw.y), sa));
            out.y = bf16x2_rn(__fmul_rn(__fmul_rn(__int2float_rn(sum.z), sw.z), sa),
                              __fmul_rn(__fmul_rn(__int2float_rn(sum.w), sw.w), sa));
            *reinterpret_cast<uint2*>(p.y + (static_cast<int64_t>(w.t) * T + t) * p.N + n) = out;
          }
        }
      }
    }
    __syncwarp();
  }
  if (p.parts > 1 && warp < 12) cluster_sync();   // the epilogue's, above

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
