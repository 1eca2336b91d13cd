// gemm_channel.cu -- the INT8 x INT8 linear with one scale per token and one
// per output channel:
//
//   P[m,n] = sum_k q_a[m,k] * q_w[k,n]   (an exact integer),
//   y[m,n] = bf16( (float(P) * s_w[n]) * s_a[m] ).
//
// P is exact whatever the tiling and the split of K: codes are exact in fp16,
// products and sums of up to 1024 of them stay within 2^24 and so are exact in
// an fp32 accumulator, and the sums of each 1024 are added as int32.  y
// therefore does not depend on M, on the split or on the device.
//
// Small batches (streaming kernel).  The weights pass once and HBM is the
// bound.  Every warp streams its own weights from global memory straight into
// registers (16-byte loads, two 64-wide K blocks on their way), widens them to
// fp16 in place and multiplies them with mma.sync: there is no shared-memory
// ring, no barrier and no tensor-memory hand-off on the way, so nothing but the
// loads themselves paces the stream.  The legacy tensor path does one m16n8k16
// per 2 cycles and SM (measured), 256 weight bytes x 8 tokens; HBM delivers 256
// bytes per 11 cycles and SM, so for 8 tokens it has room to spare.  (The int8
// form, m16n8k32, takes 16 cycles here.)  Measured at 8 x 5120 x 34816: 32.4 us,
// 5.5 TB/s, 0.81 of the copy rate; 1 x 5120 x 248320: 208 us, 0.90.
//   * A block's 8 warps share 32 or 64 output channels and interleave the 64-
//     wide K blocks between them; a cluster of up to 8 blocks splits K further
//     where the channels alone do not fill the machine.  Partials are integers:
//     they meet in shared memory by atomic addition, and across the cluster
//     through distributed shared memory, in any order with one result.
//   * K inside a block is permuted so that a thread's 16 codes of a token are
//     16 contiguous bytes, and its weights are the words of 4 neighbouring
//     channels: all loads are 16 bytes.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <mutex>

#include "channel_plan.h"
#include "gemm_channel_pair.cuh"
#include "qlin_device.cuh"
#include "qlin_internal.h"

namespace qlin {
namespace {

constexpr int kSThreads = 32 * kSWarps;
constexpr int kExactBlocks = 1024 / kKB;   // steps whose fp32 sums stay exact

struct ChannelParams {
  const void* act;          // int8 or fp16 codes [M, K]
  const float* s_a;         // [M]
  const uint32_t* w;        // 8-bit GPTQ words [K/4, N]
  const float* s_w;         // [N]
  uint16_t* y;              // bf16 [M, N]
  int64_t M, N, K;
};

__device__ __forceinline__ void mma_f16(float* d, uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ld_stream(const uint32_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

__device__ __forceinline__ int2 ld_cluster_int2(uint32_t local_addr, uint32_t rank) {
  uint32_t remote;
  int2 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local_addr), "r"(rank));
  asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(remote) : "memory");
  return v;
}

__device__ __forceinline__ uint16_t channel_out(int p, float sw, float sa) {
  return __bfloat16_as_ushort(__float2bfloat16_rn(__fmul_rn(__fmul_rn(__int2float_rn(p), sw), sa)));
}

// kHalves x 32 output channels and kTiles x 8 tokens a block.
template <int kHalves, int kTiles, bool kC16>
__global__ void __launch_bounds__(kSThreads, kHalves * kTiles == 1 ? 3 : 2)
    stream_kernel(const ChannelParams p, int splits) {
  constexpr int F = 32 * kHalves;
  constexpr int T = 8 * kTiles;
  constexpr int kCodes = kC16 ? 2 : 1;         // uint4 of 16 codes
  constexpr int kPad = F + 4;                  // words of one token's row of partials
  __shared__ __align__(16) int part[T * kPad];
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int g = lane >> 2;                     // channel group of 4, and token of a tile of 8
  const int t = lane & 3;                      // quarter of the 64-wide K block
  const uint32_t rank = splits > 1 ? cluster_rank() : 0u;
  const int64_t f0 = static_cast<int64_t>(blockIdx.x / splits) * F;
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * T;
  const int64_t N = p.N, K = p.K;
  const int nkb = static_cast<int>(K / kKB);
  const int stride = kSWarps * splits;
  const int first = static_cast<int>(rank) * kSWarps + warp;

  for (int i = threadIdx.x; i < T * kPad; i += kSThreads) part[i] = 0;

  // this thread's words: rows 4t .. 4t+3 of each K block's 16, channels 4g .. 4g+3 of each 32
  const uint32_t* wbase = p.w + static_cast<int64_t>(4 * t) * N + f0 + 4 * g;
  bool have[kHalves];
#pragma unroll
  for (int hf = 0; hf < kHalves; ++hf) have[hf] = f0 + 32 * hf + 4 * g < N;   // N is a multiple of 8
  uint4 w[2][4 * kHalves];
  auto load_w = [&](uint4 (&to)[4 * kHalves], int kb) {
    const uint32_t* src = wbase + static_cast<int64_t>(kb) * 16 * N;
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int hf = 0; hf < kHalves; ++hf)
        to[s * kHalves + hf] = have[hf] ? ld_stream(src + s * N + 32 * hf) : make_uint4(0, 0, 0, 0);
  };
  // two steps of weights on their way; they depend on no earlier kernel
  if (first < nkb) load_w(w[0], first);
  if (first + stride < nkb) load_w(w[1], first + stride);
  grid_dep_launch();
  grid_dep_wait();
  __syncthreads();

  // this thread's tokens, one of each tile of 8 (the last one again past it:
  // computed and not written)
  const char* abase[kTiles];
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
    const int64_t mine = m0 + 8 * i + g < p.M ? m0 + 8 * i + g : p.M - 1;
    abase[i] = static_cast<const char*>(p.act) + (mine * K + 16 * t) * (kC16 ? 2 : 1);
  }
  uint4 a[2][kTiles * kCodes];
  auto load_a = [&](uint4 (&to)[kTiles * kCodes], int kb) {
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      const uint4* src = reinterpret_cast<const uint4*>(abase[i] + static_cast<int64_t>(kb) * kKB * (kC16 ? 2 : 1));
#pragma unroll
      for (int c = 0; c < kCodes; ++c) to[i * kCodes + c] = src[c];
    }
  };
  if (first < nkb) load_a(a[0], first);

  float acc[kTiles][2 * kHalves][4];
#pragma unroll
  for (int i = 0; i < kTiles; ++i)
#pragma unroll
    for (int j = 0; j < 2 * kHalves; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.0f;
  auto flush = [&]() {
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int j = 0; j < 2 * kHalves; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // row of the 16 x 8 result: channel 4g + 2 (j & 1) + (e >> 1); column: token 2t + (e & 1)
          const int ch = 32 * (j >> 1) + 4 * g + 2 * (j & 1) + (e >> 1);
          atomicAdd(&part[(8 * i + 2 * t + (e & 1)) * kPad + ch], __float2int_rn(acc[i][j][e]));
          acc[i][j][e] = 0.0f;
        }
  };

  int done = 0;
  auto step = [&](uint4 (&wc)[4 * kHalves], uint4 (&ac)[kTiles * kCodes], uint4 (&an)[kTiles * kCodes], int kb) {
    uint32_t b[kTiles][4][2];          // the tokens' codes, 4 of K for each product
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      if constexpr (kC16) {
        const uint4 lo = ac[2 * i], hi = ac[2 * i + 1];
        const uint32_t c[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          b[i][s][0] = c[2 * s];
          b[i][s][1] = c[2 * s + 1];
        }
      } else {
        const uint32_t c[4] = {ac[i].x, ac[i].y, ac[i].z, ac[i].w};
#pragma unroll
        for (int s = 0; s < 4; ++s) biased_u8x4_to_f16x4(c[s] ^ 0x80808080u, b[i][s][0], b[i][s][1]);
      }
    }
    if (kb + stride < nkb) load_a(an, kb + stride);
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int hf = 0; hf < kHalves; ++hf) {
        const uint4 v = wc[s * kHalves + hf];
        uint32_t c0[2], c1[2], c2[2], c3[2];
        biased_u8x4_to_f16x4(v.x, c0[0], c0[1]);
        biased_u8x4_to_f16x4(v.y, c1[0], c1[1]);
        biased_u8x4_to_f16x4(v.z, c2[0], c2[1]);
        biased_u8x4_to_f16x4(v.w, c3[0], c3[1]);
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
          mma_f16(acc[i][2 * hf], c0[0], c1[0], c0[1], c1[1], b[i][s][0], b[i][s][1]);
          mma_f16(acc[i][2 * hf + 1], c2[0], c3[0], c2[1], c3[1], b[i][s][0], b[i][s][1]);
        }
      }
    if (kb + 2 * stride < nkb) load_w(wc, kb + 2 * stride);
    if (++done == kExactBlocks) {
      flush();
      done = 0;
    }
  };
  for (int kb = first; kb < nkb; kb += 2 * stride) {
    step(w[0], a[0], a[1], kb);
    if (kb + stride < nkb) step(w[1], a[1], a[0], kb + stride);
  }
  if (done) flush();

  // each block of the cluster finishes its share of the tile's outputs
  if (splits > 1) cluster_sync_all();
  else __syncthreads();
  const uint32_t pbase = smem_u32(part);
  constexpr int kPairs = T * F / 2;            // two neighbouring channels at a time
  for (int o = static_cast<int>(rank) * kSThreads + threadIdx.x; o < kPairs; o += kSThreads * splits) {
    const int tok = o / (F / 2);
    const int ch = 2 * (o - tok * (F / 2));
    const int64_t m = m0 + tok;
    const int64_t n = f0 + ch;
    if (m >= p.M || n >= N) continue;
    int v0 = 0, v1 = 0;
    const int at = tok * kPad + ch;
    if (splits > 1) {
      int2 v[kMaxSplits];        // all on their way before the first is added
#pragma unroll
      for (int r = 0; r < kMaxSplits; ++r)
        v[r] = r < splits ? ld_cluster_int2(pbase + 4u * at, r) : make_int2(0, 0);
#pragma unroll
      for (int r = 0; r < kMaxSplits; ++r) {
        v0 += v[r].x;
        v1 += v[r].y;
      }
    } else {
      v0 = part[at];
      v1 = part[at + 1];
    }
    const float sa = __ldg(p.s_a + m);
    const uint32_t out = static_cast<uint32_t>(channel_out(v0, __ldg(p.s_w + n), sa)) |
                         (static_cast<uint32_t>(channel_out(v1, __ldg(p.s_w + n + 1), sa)) << 16);
    *reinterpret_cast<uint32_t*>(p.y + m * N + n) = out;
  }
  if (splits > 1) cluster_sync_all();   // no block leaves while another reads its partials
}

template <int kHalves, int kTiles, bool kC16>
cudaError_t launch_stream(const ChannelParams& p, int splits, cudaStream_t stream) {
  const int64_t ftiles = (p.N + 32 * kHalves - 1) / (32 * kHalves);
  const int64_t ttiles = (p.M + 8 * kTiles - 1) / (8 * kTiles);
  return launch_cluster_pdl(stream_kernel<kHalves, kTiles, kC16>,
                            dim3(static_cast<unsigned>(ftiles * splits), static_cast<unsigned>(ttiles)),
                            dim3(kSThreads), 0, splits, stream, p, splits);
}

template <typename Kernel>
int clusters_at_once(Kernel kernel, int threads, size_t smem, int size, int blocks_per_sm, int sm_count) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(size));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(size);
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess && n > 0) return n;
  (void)cudaGetLastError();
  return blocks_per_sm * sm_count / size;
}

// Of the current device.
const Room& room_of_device(int sm_count) {
  static Room rooms[64];
  static std::once_flag once[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) dev = 0;
  dev &= 63;
  std::call_once(once[dev], [&] {
    Room& r = rooms[dev];
    r.sm_count = sm_count;
    (void)cudaFuncSetAttribute(pair::pair_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(pair::Cfg<128>::kSmem));
    for (int c = 1; c <= kMaxParts; ++c)
      r.pairs[c] = clusters_at_once(pair::pair_kernel<128>, pair::kThreads, pair::Cfg<128>::kSmem, 2 * c, 1, sm_count);
    for (int c = 1; c <= kMaxSplits; ++c) {
      r.narrow[c] = clusters_at_once(stream_kernel<1, 1, false>, kSThreads, 0, c, 3, sm_count);
      r.wide[c] = clusters_at_once(stream_kernel<2, 1, false>, kSThreads, 0, c, 2, sm_count);
      r.tokens16[c] = clusters_at_once(stream_kernel<1, 2, false>, kSThreads, 0, c, 2, sm_count);
    }
  });
  return rooms[dev];
}

template <bool kC16>
cudaError_t launch_c(const ChannelParams& p, const Room& room, cudaStream_t stream) {
  const StreamPlan pl = plan_stream(p.M, p.N, p.K, room);
  if (pl.tokens == 16) return launch_stream<1, 2, kC16>(p, pl.splits, stream);
  if (pl.channels == 64) return launch_stream<2, 1, kC16>(p, pl.splits, stream);
  return launch_stream<1, 1, kC16>(p, pl.splits, stream);
}

// ------------------------------------------------------- larger batches

// Before the pair kernel: the counters to zero and int8 codes as fp16 (16 a
// thread).
__global__ void __launch_bounds__(256) pair_prepare_kernel(int* counters, const int8_t* __restrict__ q,
                                                           uint16_t* __restrict__ image, int64_t n16) {
  grid_dep_launch();  // the pairs' blocks may take the SMs that come free, and load words
  grid_dep_wait();    // the workspace may still be in use, and the codes come from the previous kernel
  if (blockIdx.x == 0 && counters != nullptr) counters[threadIdx.x] = 0;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(256) + threadIdx.x; i < n16;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const uint4 raw = __ldg(reinterpret_cast<const uint4*>(q) + i);
    uint4 lo, hi;
    biased_u8x4_to_f16x4(raw.x ^ 0x80808080u, lo.x, lo.y);
    biased_u8x4_to_f16x4(raw.y ^ 0x80808080u, lo.z, lo.w);
    biased_u8x4_to_f16x4(raw.z ^ 0x80808080u, hi.x, hi.y);
    biased_u8x4_to_f16x4(raw.w ^ 0x80808080u, hi.z, hi.w);
    reinterpret_cast<uint4*>(image)[2 * i] = lo;
    reinterpret_cast<uint4*>(image)[2 * i + 1] = hi;
  }
}
static_assert(kCounterBytes == 256 * sizeof(int), "one counter a thread");

template <int T>
cudaError_t launch_pair_t(const CUtensorMap& tw, const CUtensorMap& tx, const pair::Params& p, cudaStream_t stream) {
  // The kernel's warps trade registers (setmaxnreg) within what the block was
  // launched with.  A build that gave the block less would wait for them
  // forever, so it is refused here.
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, pair::pair_kernel<T>);
    if (e != cudaSuccess) return e;
    if (fa.numRegs * pair::kThreads < pair::Cfg<T>::kRegsSum) return cudaErrorLaunchOutOfResources;
    e = cudaFuncSetAttribute(pair::pair_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(pair::Cfg<T>::kSmem));
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_release);
  }
  return launch_cluster_pdl(pair::pair_kernel<T>, dim3(static_cast<unsigned>(2 * p.pairs)), dim3(pair::kThreads),
                            pair::Cfg<T>::kSmem, 2 * p.parts, stream, tw, tx, p);
}

cudaError_t launch_pair(const ChannelGemmArgs& a, int* err, const Room& room, cudaStream_t stream) {
  const PairPlan pl = plan_pair(a.M, a.N, a.K, room);
  if (pl.TT * pl.F2 > (1LL << 30)) return cudaErrorInvalidValue;   // y would not fit any memory
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  const void* codes = a.act;
  int* counters = nullptr;
  size_t at = 0;
  if (pl.cut) {
    counters = reinterpret_cast<int*>(ws);
    at = kCounterBytes + pl.part_bytes;
  }
  if (pl.cut || !a.act_c16) {
    const int8_t* q = a.act_c16 ? nullptr : static_cast<const int8_t*>(a.act);
    const int64_t n16 = a.act_c16 ? 0 : a.M * a.K / 16;
    uint16_t* image = a.act_c16 ? nullptr : reinterpret_cast<uint16_t*>(ws + at);
    int64_t blocks = (n16 + 255) / 256;
    blocks = blocks < 1 ? 1 : blocks > 4096 ? 4096 : blocks;
    const cudaError_t e = launch_pdl(pair_prepare_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream,
                                     counters, q, image, n16);
    if (e != cudaSuccess) return e;
    if (!a.act_c16) codes = image;
  }
  CUtensorMap tw, tx;
  if (!make_map_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_INT32, a.qweight, a.N, a.K / 4, static_cast<uint64_t>(a.N) * 4, 128,
                   32, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !make_act_map(&tx, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, codes, a.M, a.K, static_cast<uint32_t>(pl.T / 2), 1))
    return cudaErrorInvalidValue;
  pair::Params p;
  p.s_a = a.s_a;
  p.s_w = a.s_w;
  p.y = a.y;
  p.M = a.M;
  p.N = a.N;
  p.G = static_cast<int>(pl.G);
  p.F2 = static_cast<int>(pl.F2);
  p.TT = static_cast<int>(pl.TT);
  p.band = static_cast<int>(pl.band);
  p.pairs = static_cast<int>(pl.pairs);
  p.sk_tiles = static_cast<int>(pl.sk_tiles);
  p.sk_pairs = pl.sk_pairs > 0 ? static_cast<int>(pl.sk_pairs) : 1;
  p.parts = static_cast<int>(pl.parts);
  p.counters = counters;
  p.part = pl.cut ? reinterpret_cast<int32_t*>(ws + kCounterBytes) : nullptr;
  p.err = err;
  p.limit_ns = kWaitLimitNs;
  switch (pl.T) {
    case 64: return launch_pair_t<64>(tw, tx, p, stream);
    case 96: return launch_pair_t<96>(tw, tx, p, stream);
    case 128: return launch_pair_t<128>(tw, tx, p, stream);
    default: return launch_pair_t<192>(tw, tx, p, stream);
  }
}

}  // namespace

size_t channel_workspace_bytes(int64_t M, int64_t N, int64_t K, bool c16, int sm_count) {
  return plan_workspace_bytes(M, N, K, c16, room_of_device(sm_count));
}

cudaError_t launch_gemm_channel(const ChannelGemmArgs& a, int* err, int sm_count, cudaStream_t stream) {
  const Room& room = room_of_device(sm_count);
  if (!streams(a.M, a.N, a.K, room)) return launch_pair(a, err, room, stream);
  const ChannelParams p{a.act, a.s_a, reinterpret_cast<const uint32_t*>(a.qweight), a.s_w, a.y, a.M, a.N, a.K};
  return a.act_c16 ? launch_c<true>(p, room, stream) : launch_c<false>(p, room, stream);
}

}  // namespace qlin
