// logits.cu -- logits adjusted by the penalties for repeated tokens, biases
// and a grammar mask, and the greedy token of the result.
//
// For each row, with n(v) the count of v among the row's generated tokens
// and seen(v) whether v occurs in its prompt or generated tokens, in fp32:
//   x <- x > 0 ? x / repetition : x * repetition       where seen(v)
//   x <- x - (frequency * n(v) + presence)             where n(v) > 0
//   x <- x + bias                                      for the row's bias ids
//   x <- -inf                                          where the mask bit is 0
// rounded once to the logits' type; the greedy token is the index of the
// largest rounded value, the lowest on ties.
//
// What bounds it: HBM, one read and one write of the logits; at one row the
// chain of steps below.  A row's vocabulary is cut between the blocks of a
// cluster.  Without penalties and biases a block streams its slice through
// registers.  With them it brings the slice into shared memory by one bulk
// copy, and while that is on its way looks through the history (4 bytes a
// token, from L2) and the bias ids for tokens of its own slice: each is entered
// once in a hash table, with how often it was generated and the last bias entry
// that names it.  Then, in shared memory, every entry's logit is adjusted, and
// the slice is masked, compared and written out.
// 96 rows of 248,320 bf16 logits with 8192 tokens of history each: 35.5 us,
// against 15 us of traffic (two and a half rounds of blocks, of whose 9.5 us the
// history takes 3 and the way out 2.5; 17 us without rules); one row with 2000
// tokens 5.1 us.  fp32 logits, 96 rows of them: 67.8 us, 28.5 of traffic.  Where a
// slice holds more different tokens than the table, each window of it costs
// another look through the history: 330 rows of 248,320 with 30,000 different
// tokens each 1.23 ms, 50 us of traffic; 6000 with 5000 38 us.  (Counters by each token's rank among bits set in a bit map,
// and lists built from it, took 40.1 and 6.0 us; streaming through registers with
// the touched tokens adjusted in global memory afterwards 43 to 66.)
// Counts and maxima of integers do not depend on the order of the atomics.  The
// blocks' best values meet in the first one's shared memory, so there is no
// workspace.
#include <cuda_bf16.h>

#include <atomic>
#include <mutex>

#include "qlin_device.cuh"
#include "qlin_internal.h"

namespace qlin {
namespace {

constexpr int kLThreads = 512;
constexpr int kLWarps = kLThreads / 32;
constexpr int kMaxSplits = 16;
constexpr int kSliceBytes = 65536;  // of the logits that a block holds in shared memory at a time, at most
constexpr int kMaxSlots = 4096;     // of the hash table: with the slice, two blocks an SM
constexpr int kProbes = 32;         // slots that an entry is tried in
constexpr uint32_t kFree = 0xFFFFFFFFu;

struct LogitParams {
  const void* logits;
  int64_t V;
  int L, B;
  const int32_t* tokens;
  const int32_t* prompt_len;
  const int32_t* total_len;
  const float* repetition;
  const float* presence;
  const float* frequency;
  const int32_t* bias_ids;
  const float* bias;
  const uint8_t* allowed;
  int64_t mask_stride;   // bytes of a mask row
  void* out;
  int32_t* argmax;
  int64_t slice;         // tokens of one block, a multiple of 8
  int part;              // tokens held at a time, a multiple of 8
  int slots;             // of the table, a power of two of at least kLThreads
  int splits;            // blocks of a row = cluster size
  int* err;
};

struct RowRules {
  float rep, pres, freq;
};

__device__ __forceinline__ float penalized(float x, uint32_t n, bool seen, const RowRules& r) {
  if (n != 0u || seen) x = x > 0.0f ? __fdiv_rn(x, r.rep) : __fmul_rn(x, r.rep);
  if (n != 0u) x = __fsub_rn(x, __fadd_rn(__fmul_rn(r.freq, static_cast<float>(n)), r.pres));
  return x;
}

struct Best {
  float v;
  int32_t i;
};

// (v, i) into best: the larger value, the lower index on ties; -inf and NaN never
__device__ __forceinline__ void consider(Best& best, float v, int32_t i) {
  if (v > best.v || (v == best.v && best.i >= 0 && i < best.i)) {
    best.v = v;
    best.i = i;
  }
}

__device__ __forceinline__ void warp_best(Best& best) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float v = __shfl_xor_sync(0xFFFFFFFFu, best.v, o);
    const int32_t i = __shfl_xor_sync(0xFFFFFFFFu, best.i, o);
    consider(best, v, i);
  }
}

// 8 neighbouring logits
template <bool kF32>
struct Vec8 {
  uint4 a, b;   // b: fp32 only
  __device__ __forceinline__ void load(const uint4* in) {
    a = in[0];
    if constexpr (kF32) b = in[1];
  }
  __device__ __forceinline__ void store(uint4* out) const {
    out[0] = a;
    if constexpr (kF32) out[1] = b;
  }
  __device__ __forceinline__ uint32_t word(int i) const {
    return i == 0 ? a.x : i == 1 ? a.y : i == 2 ? a.z : i == 3 ? a.w : i == 4 ? b.x : i == 5 ? b.y : i == 6 ? b.z : b.w;
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (kF32) return __uint_as_float(word(e));
    return __uint_as_float((e & 1) ? word(e >> 1) & 0xFFFF0000u : word(e >> 1) << 16);
  }
  // -inf where bit e of m is 0.  The product puts bits 0..3 of a nibble at the
  // top of bytes 0..3 (its 16 partial products meet nowhere), from where prmt
  // spreads them over their elements.
  __device__ __forceinline__ void keep(uint32_t m) {
    const uint32_t lo = (m & 15u) * 0x10204080u;
    const uint32_t hi = (m >> 4 & 15u) * 0x10204080u;
    auto pick = [](uint32_t w, uint32_t k, uint32_t inf) { return (w & k) | (inf & ~k); };
    if constexpr (kF32) {
      constexpr uint32_t inf = 0xFF800000u;
      a = make_uint4(pick(a.x, prmt(lo, 0, 0x8888u), inf), pick(a.y, prmt(lo, 0, 0x9999u), inf),
                     pick(a.z, prmt(lo, 0, 0xAAAAu), inf), pick(a.w, prmt(lo, 0, 0xBBBBu), inf));
      b = make_uint4(pick(b.x, prmt(hi, 0, 0x8888u), inf), pick(b.y, prmt(hi, 0, 0x9999u), inf),
                     pick(b.z, prmt(hi, 0, 0xAAAAu), inf), pick(b.w, prmt(hi, 0, 0xBBBBu), inf));
    } else {
      constexpr uint32_t inf = 0xFF80FF80u;
      a = make_uint4(pick(a.x, prmt(lo, 0, 0x9988u), inf), pick(a.y, prmt(lo, 0, 0xBBAAu), inf),
                     pick(a.z, prmt(hi, 0, 0x9988u), inf), pick(a.w, prmt(hi, 0, 0xBBAAu), inf));
    }
  }
  // the largest value; of a NaN and a number the number
  __device__ __forceinline__ float top() const {
    if constexpr (kF32) {
      return fmaxf(fmaxf(fmaxf(get(0), get(1)), fmaxf(get(2), get(3))), fmaxf(fmaxf(get(4), get(5)), fmaxf(get(6), get(7))));
    } else {
      auto h = [](const uint32_t& w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
      const __nv_bfloat162 m = __hmax2(__hmax2(h(a.x), h(a.y)), __hmax2(h(a.z), h(a.w)));
      return fmaxf(__low2float(m), __high2float(m));
    }
  }
};

// Shared memory of the rules: the slice, then the table: the tokens, their
// occurrences (2 for each generated one, 1 for all in the prompt) and the last
// bias entries.
__host__ __device__ inline int rule_bytes(int part, int elem, int slots) { return part * elem + slots * 12; }

// (fence_barrier_init has published the barrier, all that this announces)
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

// Brings thread tid's share of [p, p + bytes) into L2, the line of p + 128 tid.
__device__ __forceinline__ void prefetch_share(const void* p, int64_t bytes, int tid) {
  const int64_t at = 128 * static_cast<int64_t>(tid);
  if (at < bytes) asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(p) + at));
}

template <bool kF32, bool kRules, bool kMasked>
__global__ void __launch_bounds__(kLThreads, kRules ? 2 : 3) adjust_logits_kernel(const LogitParams p) {
  constexpr int kAhead = kF32 ? 2 : 4;       // vectors in flight a thread
  constexpr int kE = kF32 ? 2 : 1;           // uint4 of a vector
  extern __shared__ uint4 smem4[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>(smem4);
  uint32_t* const key = reinterpret_cast<uint32_t*>(smem + p.part * (kF32 ? 4 : 2));   // the slice's logits come first
  uint32_t* const occurs = key + p.slots;
  int32_t* const entry = reinterpret_cast<int32_t*>(occurs + p.slots);
  __shared__ Best red[kLWarps];
  __shared__ Best others[kMaxSplits];        // rank 0: the other blocks' best values
  __shared__ uint64_t others_here, slice_here;
  __shared__ int abort_flag;
  __shared__ int too_full;
  const int tid = threadIdx.x;
  const int lane = tid & 31;
  const int64_t m = blockIdx.x / p.splits;
  const int rank = static_cast<int>(blockIdx.x % p.splits);
  const int64_t V = p.V;
  const int64_t s0 = rank * p.slice;
  const int64_t s1 = s0 + p.slice < V ? s0 + p.slice : V;
  const uint8_t* row_in = static_cast<const uint8_t*>(p.logits) + m * V * (kF32 ? 4 : 2);
  uint8_t* row_out = p.out ? static_cast<uint8_t*>(p.out) + m * V * (kF32 ? 4 : 2) : nullptr;
  const uint8_t* mask = kMasked ? p.allowed + m * p.mask_stride : nullptr;
  if (tid == 0) {
    abort_flag = 0;
    too_full = 0;
    mbar_init(smem_u32(&others_here), 1);
    mbar_init(smem_u32(&slice_here), 1);
    fence_barrier_init();
  }
  // rank 0's barrier for the others' values is ready once all have passed the
  // cluster barrier, whose wait comes at the end
  if (p.argmax != nullptr && p.splits > 1) cluster_arrive();
  auto fetch_slice = [&](int64_t v0, uint32_t n) {   // thread 0
    const uint32_t bar = smem_u32(&slice_here);
    mbar_arrive_expect_tx(bar, n * (kF32 ? 4 : 2));
    bulk_load(smem_u32(smem), row_in + v0 * (kF32 ? 4 : 2), n * (kF32 ? 4 : 2), bar);
  };
  auto clear_table = [&]() {
    for (int i = tid; i < p.slots / 4; i += kLThreads) {
      reinterpret_cast<uint4*>(key)[i] = make_uint4(kFree, kFree, kFree, kFree);
      reinterpret_cast<uint4*>(occurs)[i] = make_uint4(0, 0, 0, 0);
      reinterpret_cast<uint4*>(entry)[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
    }
  };
  // What small inputs the block reads comes into L2 while an earlier kernel
  // still runs (their values are read after it).
  if (kMasked && s0 < V) prefetch_share(mask + s0 / 8, (s1 - s0) / 8, tid);
  if constexpr (kRules) {
    if (p.B > 0) {
      prefetch_share(p.bias_ids + m * p.B, 4LL * p.B, tid);
      prefetch_share(p.bias + m * p.B, 4LL * p.B, tid);
    }
    clear_table();
  }
  grid_dep_launch();
  grid_dep_wait();
  int total = 0, prompt = 0;
  RowRules rules{1.0f, 0.0f, 0.0f};
  if (kRules) {
    if (p.L > 0) {
      total = p.total_len ? min(max(__ldg(p.total_len + m), 0), p.L) : p.L;
      prompt = p.prompt_len ? __ldg(p.prompt_len + m) : 0;
    }
    if (p.repetition) rules.rep = __ldg(p.repetition + m);
    if (p.presence) rules.pres = __ldg(p.presence + m);
    if (p.frequency) rules.freq = __ldg(p.frequency + m);
  }

  Best best{-INFINITY, -1};
  const WaitCtx ctx{p.err, &abort_flag, kWaitLimitNs};
  int parts_done = 0;
  for (int64_t v0 = s0; v0 < s1; v0 += p.part, ++parts_done) {
    const uint32_t n = static_cast<uint32_t>(s1 - v0 < p.part ? s1 - v0 : p.part);
    const int nvec = static_cast<int>(n / 8);
    const uint4* in = reinterpret_cast<const uint4*>(row_in) + v0 / 8 * kE;
    uint4* to = row_out ? reinterpret_cast<uint4*>(row_out) + v0 / 8 * kE : nullptr;
    const uint8_t* allow = kMasked ? mask + v0 / 8 : nullptr;

    if constexpr (kRules) {
      if (parts_done > 0) {
        __syncthreads();   // the previous part's slice and table are read
        clear_table();
        if (tid == 0) {
          too_full = 0;
          fence_proxy_async_smem();
        }
      }
      if (tid == 0) fetch_slice(v0, n);
      __syncthreads();
      // f(token's place in the part, whether it is a generated one) for the
      // history's tokens of the part; ids outside it, negative ones too, wrap
      // to n and above
      auto history = [&](auto f) {
        const int32_t* toks = p.tokens + m * p.L;
        for (int i0 = tid; i0 < total; i0 += 8 * kLThreads) {
          uint32_t at[8];
#pragma unroll
          for (int k = 0; k < 8; ++k)
            at[k] = i0 + k * kLThreads < total ? static_cast<uint32_t>(__ldg(toks + i0 + k * kLThreads)) : 0xFFFFFFFFu;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            at[k] -= static_cast<uint32_t>(v0);
            if (at[k] < n) f(at[k], i0 + k * kLThreads >= prompt);
          }
        }
      };
      auto bias_place = [&](int j) {   // of entry j, n or more where it is not in the part
        return static_cast<uint32_t>(__ldg(p.bias_ids + m * p.B + j)) - static_cast<uint32_t>(v0);
      };
      auto logit = [&](uint32_t at) {
        return kF32 ? reinterpret_cast<const float*>(smem)[at]
                    : __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(smem)[at]) << 16);
      };
      auto put = [&](uint32_t at, float x) {
        if constexpr (kF32) reinterpret_cast<float*>(smem)[at] = x;
        else reinterpret_cast<uint16_t*>(smem)[at] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
      };
      // The table takes the tokens at lo .. lo + span of the part: all of them
      // at first, hashed; if they are too many for it, as many as it has slots
      // at a time, each in its own.
      uint32_t lo = 0, span = n;
      const int shift = 32 - __ffs(p.slots) + 1;
      bool hashed = true;
      auto slot_of = [&](uint32_t at) {
        uint32_t slot = hashed ? (at * 0x9E3779B1u) >> shift : at - lo;   // 2^32 / golden ratio
        for (int i = 0; i < kProbes; ++i) {
          const uint32_t was = atomicCAS(key + slot, kFree, at);
          if (was == kFree || was == at) return static_cast<int>(slot);
          slot = (slot + 1u) & static_cast<uint32_t>(p.slots - 1);
        }
        too_full = 1;
        return -1;
      };
      const uint32_t first_bias = tid < p.B ? bias_place(tid) : n;   // on its way beside the history
      for (;;) {
        history([&](uint32_t at, bool made) {
          if (at - lo >= span) return;
          const int slot = slot_of(at);
          if (slot < 0) return;
          if (made) atomicAdd(occurs + slot, 2u);
          else atomicOr(occurs + slot, 1u);
        });
        for (int i = tid; i < p.B; i += kLThreads) {
          const uint32_t at = i == tid ? first_bias : bias_place(i);
          if (at >= n || at - lo >= span) continue;
          const int slot = slot_of(at);
          if (slot >= 0) atomicMax(entry + slot, i);
        }
        if (lo == 0 && span == n && !mbar_wait(smem_u32(&slice_here), parts_done & 1, ctx, 81)) abort_flag = 1;
        __syncthreads();
        const bool again = hashed && too_full != 0;
        if (!again) {
          uint32_t mine = 0;   // this thread's slots that hold a token
#pragma unroll
          for (int k = 0; k < kMaxSlots / kLThreads; ++k)
            if (k * kLThreads < p.slots && key[k * kLThreads + tid] != kFree) mine |= 1u << k;
          for (; mine != 0u; mine &= mine - 1u) {
            const int slot = (__ffs(mine) - 1) * kLThreads + tid;
            const uint32_t at = key[slot];
            const uint32_t n_seen = occurs[slot];
            const int j = entry[slot];
            float x = penalized(logit(at), n_seen >> 1, n_seen != 0u, rules);
            if (j >= 0) x = __fadd_rn(x, __ldg(p.bias + m * p.B + j));
            put(at, x);
          }
          if (hashed || lo + span >= n) break;
          lo += span;
        }
        hashed = false;
        span = min(static_cast<uint32_t>(p.slots), n - lo);
        __syncthreads();   // the table is read
        clear_table();
        __syncthreads();
      }
      __syncthreads();
      if (abort_flag) break;   // the slice did not arrive; the error word says so
      in = smem4;
    }

    for (int j0 = tid; j0 < nvec; j0 += kAhead * kLThreads) {
      Vec8<kF32> x[kAhead];
      uint32_t ok[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (j0 + k * kLThreads < nvec) {
          x[k].load(in + (j0 + k * kLThreads) * static_cast<int64_t>(kE));
          if (kMasked) ok[k] = __ldg(allow + j0 + k * kLThreads);
        }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int j = j0 + k * kLThreads;
        if (j >= nvec) break;
        if constexpr (kMasked) x[k].keep(ok[k]);
        if (to) x[k].store(to + j * static_cast<int64_t>(kE));
        const float top = x[k].top();
        if (top > best.v) {   // ascending vectors: the first of equal values stays
          best.v = top;
          uint32_t at = 0;
#pragma unroll
          for (int e = 7; e >= 0; --e)
            if (x[k].get(e) == top) at = e;
          best.i = static_cast<int32_t>(v0) + 8 * j + static_cast<int32_t>(at);
        }
      }
    }
  }
  if (kRules && abort_flag) {   // the copy lands before the block ends
    int never = 0;
    if (tid == 0) (void)mbar_wait(smem_u32(&slice_here), parts_done & 1, WaitCtx{p.err, &never, kWaitLimitNs}, 82);
  }
  if (p.argmax == nullptr) return;

  warp_best(best);
  if (lane == 0) red[tid >> 5] = best;
  __syncthreads();
  if (p.splits > 1) cluster_wait();
  if (tid >= 32) return;
  best = tid < kLWarps ? red[tid] : Best{-INFINITY, -1};
  warp_best(best);
  if (p.splits > 1) {
    const uint32_t bar = smem_u32(&others_here);
    if (rank != 0) {
      // into rank 0's shared memory, counted on its barrier: no second cluster
      // barrier, which would wait for this block's global stores
      if (tid == 0) {
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(
                         map_rank(smem_u32(&others[rank]), 0)),
                     "r"(__float_as_uint(best.v)), "r"(best.i), "r"(map_rank(bar, 0))
                     : "memory");
      }
      return;
    }
    if (tid == 0) mbar_arrive_expect_tx(bar, 8u * (p.splits - 1));
    __syncwarp();
    if (!__all_sync(0xFFFFFFFFu, mbar_wait(bar, 0, ctx, 80))) return;
    if (tid > 0) best = tid < p.splits ? others[tid] : Best{-INFINITY, -1};
    warp_best(best);
  }
  if (tid == 0) p.argmax[m] = best.i;
}

template <bool kF32, bool kRules, bool kMasked>
cudaError_t prepare_kind() {
  const auto kernel = adjust_logits_kernel<kF32, kRules, kMasked>;
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    if (kRules) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           rule_bytes(kSliceBytes / (kF32 ? 4 : 2), kF32 ? 4 : 2, kMaxSlots));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_release);
  }
  return cudaSuccess;
}

// Rows that run at one time on the current device in clusters of 16 blocks.
template <bool kF32>
int rows_in_16(int sm_count) {
  static int rows[64];
  static std::once_flag once[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) dev = 0;
  dev &= 63;
  std::call_once(once[dev], [&] {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kMaxSplits);
    cfg.blockDim = dim3(kLThreads);
    cfg.dynamicSmemBytes = rule_bytes(kSliceBytes / (kF32 ? 4 : 2), kF32 ? 4 : 2, kMaxSlots);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = kMaxSplits;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (prepare_kind<kF32, true, true>() == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&n, adjust_logits_kernel<kF32, true, true>, &cfg) == cudaSuccess) {
      rows[dev] = n;
    } else {
      (void)cudaGetLastError();
      rows[dev] = sm_count / 2 / kMaxSplits;
    }
  });
  return rows[dev];
}

template <bool kF32, bool kRules, bool kMasked>
cudaError_t launch_kind(const LogitParams& p, int64_t M, cudaStream_t stream) {
  const auto kernel = adjust_logits_kernel<kF32, kRules, kMasked>;
  const cudaError_t e = prepare_kind<kF32, kRules, kMasked>();
  if (e != cudaSuccess) return e;
  return launch_cluster_pdl(kernel, dim3(static_cast<unsigned>(M * p.splits)), dim3(kLThreads),
                            kRules ? rule_bytes(p.part, kF32 ? 4 : 2, p.slots) : 0, p.splits, stream, p);
}

template <bool kF32>
cudaError_t launch_type(const LogitParams& p, int64_t M, cudaStream_t stream) {
  const bool masked = p.allowed != nullptr;
  if (p.L > 0 || p.B > 0)
    return masked ? launch_kind<kF32, true, true>(p, M, stream) : launch_kind<kF32, true, false>(p, M, stream);
  return masked ? launch_kind<kF32, false, true>(p, M, stream) : launch_kind<kF32, false, false>(p, M, stream);
}

}  // namespace

cudaError_t launch_adjust_logits(const LogitArgs& a, int* err, int sm_count, cudaStream_t stream) {
  // a history that no penalty looks at is left unread
  const bool penalties = a.repetition != nullptr || a.presence != nullptr || a.frequency != nullptr;
  LogitParams p{a.logits, a.V, penalties ? static_cast<int>(a.L) : 0, static_cast<int>(a.B), a.tokens, a.prompt_len,
                a.total_len, a.repetition, a.presence, a.frequency, a.bias_ids, a.bias,
                reinterpret_cast<const uint8_t*>(a.allowed), (a.V + 31) / 32 * 4, a.out, a.argmax, 0, 0, kLThreads, 1, err};
  const bool rules = p.L > 0 || p.B > 0;
  const int64_t most = rules ? kSliceBytes / (a.f32 ? 4 : 2) : a.V;
  // In clusters of 16 while all rows run at one time (14 on 152 SMs): 7 rows of
  // 248,320 fp32 logits 7.4 us, with 8 blocks a row 12.8; 14 rows 10.9 and 16.1.
  // Beyond that they cost a second round: 33 rows of 50,264 12.6 and 5.6.
  const int in_16 = a.f32 ? rows_in_16<true>(sm_count) : rows_in_16<false>(sm_count);
  const int cap = a.M <= in_16 ? kMaxSplits : 8;
  while (p.splits < cap && (a.M * p.splits < 2 * sm_count || a.V > most * p.splits) && a.V >= 4096 * p.splits)
    p.splits *= 2;
  p.slice = ((a.V + p.splits - 1) / p.splits + 7) / 8 * 8;
  p.part = static_cast<int>(p.slice < most ? p.slice : most);
  // twice the entries where it can have that
  while (p.slots < kMaxSlots && p.slots < 2 * (static_cast<int64_t>(p.L) + p.B)) p.slots *= 2;
  return a.f32 ? launch_type<true>(p, a.M, stream) : launch_type<false>(p, a.M, stream);
}

}  // namespace qlin
