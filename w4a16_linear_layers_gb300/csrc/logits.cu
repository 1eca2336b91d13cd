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
// What bounds it: HBM, one read and one write of the logits.  The counts
// never leave the chip: a row's vocabulary is cut between the blocks of a
// cluster, each block counts the history's tokens of its own part in shared
// memory (one word a token; every block reads the whole history, 4 bytes a
// token, from L2) and then streams its logits once.  Integer counts and a
// maximum do not depend on the order of the atomics.  Biased tokens are few:
// the stream leaves them as they are and a last step recomputes them, the
// last entry of an id winning.  The cluster's blocks compare their best
// values through distributed shared memory, so there is no workspace.
#include <cuda_bf16.h>

#include "qlin_device.cuh"
#include "qlin_internal.h"

namespace qlin {
namespace {

constexpr int kLThreads = 512;
constexpr int kLMaxPart = 24576;           // tokens counted at a time: 96 KB of words
constexpr uint32_t kSeen = 0x80000000u;    // in the prompt
constexpr uint32_t kBiased = 0x40000000u;
constexpr uint32_t kDone = 0xFFFFFFFFu;
constexpr uint32_t kCount = 0x3FFFFFFFu;   // occurrences among the generated tokens

struct LogitParams {
  const void* logits;
  int64_t V, L, B;
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
  int part;              // tokens counted at a time, a multiple of 8
  int splits;            // blocks of a row = cluster size
};

struct RowRules {
  float rep, pres, freq;
};

__device__ __forceinline__ float penalized(float x, uint32_t word, const RowRules& r) {
  const uint32_t n = word & kCount;
  if (n | (word & kSeen)) x = x > 0.0f ? __fdiv_rn(x, r.rep) : __fmul_rn(x, r.rep);
  if (n) x = __fsub_rn(x, __fadd_rn(__fmul_rn(r.freq, static_cast<float>(n)), r.pres));
  return x;
}

template <bool kF32>
__device__ __forceinline__ float rounded(float x) {
  return kF32 ? x : __bfloat162float(__float2bfloat16_rn(x));
}

struct Best {
  float v = -INFINITY;
  int32_t i = -1;
};

template <bool kF32>
__global__ void __launch_bounds__(kLThreads) adjust_logits_kernel(const LogitParams p) {
  extern __shared__ uint32_t words[];
  __shared__ Best red[kLThreads / 32];
  __shared__ Best block_best;
  grid_dep_wait();
  grid_dep_launch();
  const int tid = threadIdx.x;
  const int64_t m = blockIdx.x / p.splits;
  const int rank = static_cast<int>(blockIdx.x % p.splits);
  const int64_t V = p.V;
  const int64_t s0 = rank * p.slice;
  const int64_t s1 = s0 + p.slice < V ? s0 + p.slice : V;
  const bool counting = p.L > 0 || p.B > 0;
  const uint8_t* row_in = static_cast<const uint8_t*>(p.logits) + m * V * (kF32 ? 4 : 2);
  uint8_t* row_out = p.out ? static_cast<uint8_t*>(p.out) + m * V * (kF32 ? 4 : 2) : nullptr;
  const uint8_t* mask = p.allowed ? p.allowed + m * p.mask_stride : nullptr;
  const RowRules rules{p.repetition ? p.repetition[m] : 1.0f, p.presence ? p.presence[m] : 0.0f,
                       p.frequency ? p.frequency[m] : 0.0f};
  int64_t total = 0, prompt = 0;
  if (p.L > 0) {
    total = p.total_len ? p.total_len[m] : p.L;
    total = total < 0 ? 0 : total > p.L ? p.L : total;
    prompt = p.prompt_len ? p.prompt_len[m] : 0;
  }
  const int32_t* toks = p.L > 0 ? p.tokens + m * p.L : nullptr;
  const int32_t* bids = p.B > 0 ? p.bias_ids + m * p.B : nullptr;

  Best best;
  for (int64_t v0 = s0; v0 < s1; v0 += p.part) {
    const int n = static_cast<int>(s1 - v0 < p.part ? s1 - v0 : p.part);
    if (counting) {
      __syncthreads();   // the previous part's words are read
      for (int i = tid; i < n / 4; i += kLThreads) reinterpret_cast<uint4*>(words)[i] = make_uint4(0, 0, 0, 0);
      __syncthreads();
      for (int64_t i = tid; i < total; i += kLThreads) {
        const int64_t at = static_cast<int64_t>(__ldg(toks + i)) - v0;
        if (at >= 0 && at < n) {
          if (i < prompt) atomicOr(&words[at], kSeen);
          else atomicAdd(&words[at], 1u);
        }
      }
      for (int64_t i = tid; i < p.B; i += kLThreads) {
        const int64_t at = static_cast<int64_t>(__ldg(bids + i)) - v0;
        if (at >= 0 && at < n) atomicOr(&words[at], kBiased);
      }
      __syncthreads();
    }
    for (int j = tid; j < n / 8; j += kLThreads) {
      const int64_t v = v0 + 8 * j;
      float x[8];
      if constexpr (kF32) {
        const float4 a = reinterpret_cast<const float4*>(row_in)[v / 4];
        const float4 b = reinterpret_cast<const float4*>(row_in)[v / 4 + 1];
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
      } else {
        const uint4 a = reinterpret_cast<const uint4*>(row_in)[v / 8];
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[2 * e] = __uint_as_float(w[e] << 16);
          x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
        }
      }
      const uint32_t ok = mask ? __ldg(mask + v / 8) : 0xFFu;
      uint32_t skip = 0;   // biased: written unchanged here, recomputed below
      if (counting) {
        const uint4 a = reinterpret_cast<const uint4*>(words)[2 * j];
        const uint4 b = reinterpret_cast<const uint4*>(words)[2 * j + 1];
        if (a.x | a.y | a.z | a.w | b.x | b.y | b.z | b.w) {
          const uint32_t c[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (c[e] & kBiased) skip |= 1u << e;
            else if (c[e]) x[e] = rounded<kF32>(penalized(x[e], c[e], rules));
          }
        }
      }
      if (ok != 0xFFu) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (!((ok | skip) >> e & 1u)) x[e] = -INFINITY;
      }
      if (row_out) {
        if constexpr (kF32) {
          reinterpret_cast<float4*>(row_out)[v / 4] = make_float4(x[0], x[1], x[2], x[3]);
          reinterpret_cast<float4*>(row_out)[v / 4 + 1] = make_float4(x[4], x[5], x[6], x[7]);
        } else {
          reinterpret_cast<uint4*>(row_out)[v / 8] =
              make_uint4(bf16x2_rn(x[0], x[1]), bf16x2_rn(x[2], x[3]), bf16x2_rn(x[4], x[5]),
                         bf16x2_rn(x[6], x[7]));
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (x[e] > best.v && !(skip >> e & 1u)) {   // ascending e: the first of equals stays
          best.v = x[e];
          best.i = static_cast<int32_t>(v + e);
        }
      }
    }
    // Biased tokens, from the last entries to the first: of the entries with
    // one id the highest index takes it.
    for (int64_t c1 = p.B; c1 > 0; c1 -= kLThreads) {
      const int64_t j = c1 - kLThreads + tid;
      int64_t at = -1;
      if (j >= 0) at = static_cast<int64_t>(__ldg(bids + j)) - v0;
      if (at >= n) at = -1;
      __syncthreads();
      uint32_t word = kDone;
      if (at >= 0) word = words[at];
      __syncthreads();
      if (word != kDone) words[at] = 0u;
      __syncthreads();
      if (word != kDone) atomicMax(&words[at], static_cast<uint32_t>(tid) + 1u);
      __syncthreads();
      const bool mine = word != kDone && words[at] == static_cast<uint32_t>(tid) + 1u;
      __syncthreads();
      if (mine) {
        words[at] = kDone;
        const int64_t v = v0 + at;
        float x = kF32 ? reinterpret_cast<const float*>(row_in)[v]
                       : __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(row_in)[v]) << 16);
        x = __fadd_rn(penalized(x, word & ~kBiased, rules), __ldg(p.bias + m * p.B + j));
        if (mask && !(__ldg(mask + v / 8) >> (v & 7) & 1)) x = -INFINITY;
        x = rounded<kF32>(x);
        if (row_out) {
          if constexpr (kF32) reinterpret_cast<float*>(row_out)[v] = x;
          else reinterpret_cast<uint16_t*>(row_out)[v] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
        }
        if (x > best.v || (x == best.v && best.i >= 0 && v < best.i)) {
          best.v = x;
          best.i = static_cast<int32_t>(v);
        }
      }
    }
  }
  if (p.argmax == nullptr) return;

  auto take = [](Best& a, float v, int32_t i) {
    if (i >= 0 && (a.i < 0 || v > a.v || (v == a.v && i < a.i))) {
      a.v = v;
      a.i = i;
    }
  };
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float v = __shfl_xor_sync(0xFFFFFFFFu, best.v, o);
    const int32_t i = __shfl_xor_sync(0xFFFFFFFFu, best.i, o);
    take(best, v, i);
  }
  if ((tid & 31) == 0) red[tid >> 5] = best;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kLThreads / 32; ++w) take(best, red[w].v, red[w].i);
    block_best = best;
  }
  if (p.splits > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (rank == 0 && tid == 0) {
      const uint32_t local = smem_u32(&block_best);
      for (int r = 1; r < p.splits; ++r) {
        uint32_t remote, bits;
        int32_t i;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(r));
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(bits) : "r"(remote) : "memory");
        asm volatile("ld.shared::cluster.s32 %0, [%1 + 4];" : "=r"(i) : "r"(remote) : "memory");
        take(best, __uint_as_float(bits), i);
      }
    }
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  if (rank == 0 && tid == 0) p.argmax[m] = best.i;
}

template <bool kF32>
cudaError_t launch_type(const LogitParams& p, int64_t M, size_t smem, cudaStream_t stream) {
  static const cudaError_t attr =
      cudaFuncSetAttribute(adjust_logits_kernel<kF32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kLMaxPart * 4);
  if (attr != cudaSuccess) return attr;
  return launch_cluster_pdl(adjust_logits_kernel<kF32>, dim3(static_cast<unsigned>(M * p.splits)),
                            dim3(kLThreads), smem, p.splits, stream, p);
}

}  // namespace

cudaError_t launch_adjust_logits(const LogitArgs& a, int sm_count, cudaStream_t stream) {
  LogitParams p{a.logits, a.V, a.L, a.B, a.tokens, a.prompt_len, a.total_len, a.repetition,
                a.presence, a.frequency, a.bias_ids, a.bias,
                reinterpret_cast<const uint8_t*>(a.allowed), (a.V + 31) / 32 * 4, a.out, a.argmax,
                0, 0, 1};
  // Split a row while the blocks do not fill the machine twice or their parts
  // would be counted in several rounds, down to parts of 2048 tokens.
  while (p.splits < 8 && (a.M * p.splits < 2 * sm_count || a.V > static_cast<int64_t>(kLMaxPart) * p.splits) &&
         a.V >= 4096 * p.splits)
    p.splits *= 2;
  p.slice = ((a.V + p.splits - 1) / p.splits + 7) / 8 * 8;
  p.part = static_cast<int>(p.slice < kLMaxPart ? p.slice : kLMaxPart);
  const size_t smem = a.L > 0 || a.B > 0 ? static_cast<size_t>(p.part) * 4 : 0;
  return a.f32 ? launch_type<true>(p, a.M, smem, stream) : launch_type<false>(p, a.M, smem, stream);
}

}  // namespace qlin
