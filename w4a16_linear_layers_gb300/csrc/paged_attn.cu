// paged_attn.cu -- attention of the new tokens over the paged INT8 cache.
//
// For a row (token i of a sequence, query head h) over the tokens j it sees:
//   x_j = scale q . K_j (softcap tanh(x_j / softcap)),
//   out = sum_j exp(x_j) V_j / sum_j exp(x_j).
// One block of 128 threads a row, 128 tokens at a time: a thread forms one
// token's score, then one component of the output, under the running maximum.
#include "kv_cache.cuh"

namespace qlin {
namespace {

__device__ __forceinline__ float bf16_float(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

__global__ void __launch_bounds__(128) simple_attn_kernel(const PagedAttnArgs a) {
  __shared__ float qs[kHeadDim], weight[kHeadDim], red[4];
  __shared__ const uint8_t* blocks[8];
  const int tid = threadIdx.x;
  grid_dep_launch();
  grid_dep_wait();
  const int64_t row = blockIdx.x / a.q_heads;
  const int head = static_cast<int>(blockIdx.x % a.q_heads);
  const int64_t b = row / a.T;
  const SeqLen seq = seq_len(a.c, b, a.T);
  const int t = static_cast<int>(row - b * a.T);
  if (t >= seq.fresh) return;
  const int i = seq.len - seq.fresh + t;
  const int kv = head / static_cast<int>(a.q_heads / a.c.kv_heads);
  qs[tid] = bf16_float(a.q[(row * a.q_heads + head) * kHeadDim + tid]);
  const int64_t w = a.window > 0 ? a.window : 1LL << 40;
  const int lo = i - w + 1 > 0 ? static_cast<int>(i - w + 1) : 0;
  const int hi = a.causal ? i + 1 : (i + w < seq.len ? static_cast<int>(i + w) : seq.len);
  float m = -INFINITY, l = 0.0f, o = 0.0f;
  for (int j0 = lo & ~15; j0 < hi; j0 += 128) {
    __syncthreads();
    if (tid < 8) blocks[tid] = j0 + 16 * tid < hi ? cache_block(a.c, b, kv, j0 / 16 + tid) : nullptr;
    __syncthreads();
    const int j = j0 + tid, r = tid & 15;
    const uint8_t* blk = blocks[tid >> 4];
    const bool seen = j >= lo && j < hi && blk != nullptr;
    float x = -INFINITY, vs = 0.0f;
    if (seen) {
      float dot = 0.0f;
      for (int d = 0; d < kHeadDim; ++d)
        dot = fmaf(qs[d], static_cast<float>(blk[r * kHeadDim + code_place(r, d)]) - 128.0f, dot);
      x = dot * reinterpret_cast<const float*>(blk + kKScales)[r] * a.scale;
      if (a.softcap > 0.0f) x = a.softcap * tanhf(x / a.softcap);
      vs = reinterpret_cast<const float*>(blk + kVScales)[r];
    }
    float top = x;
    for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, s));
    if ((tid & 31) == 0) red[tid >> 5] = top;
    __syncthreads();
    const float next = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float keep = next == -INFINITY ? 1.0f : expf(m - next);
    const float p = seen ? expf(x - next) : 0.0f;
    weight[tid] = seen ? p * vs : 0.0f;
    float sum = p;
    for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, s);
    __syncthreads();
    if ((tid & 31) == 0) red[tid >> 5] = sum;
    __syncthreads();
    l = l * keep + (red[0] + red[1] + red[2] + red[3]);
    o *= keep;
    m = next;
    for (int k = 0; k < 128; ++k) {
      const uint8_t* kb = blocks[k >> 4];
      if (kb == nullptr) continue;
      o = fmaf(weight[k], static_cast<float>(kb[kVCodes + (k & 15) * kHeadDim + code_place(k & 15, tid)]) - 128.0f, o);
    }
  }
  const uint32_t v = bf16x2_rn(l == 0.0f ? 0.0f : o / l, 0.0f);
  a.out[(row * a.q_heads + head) * kHeadDim + tid] = static_cast<uint16_t>(v);
}

}  // namespace

size_t paged_attn_workspace_bytes(int64_t, int64_t, int64_t, int64_t, int) { return 0; }

cudaError_t launch_paged_attn(const PagedAttnArgs& a, int*, int, cudaStream_t stream) {
  const int64_t blocks = a.c.B * a.T * a.q_heads;
  if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
  return launch_pdl(simple_attn_kernel, dim3(static_cast<unsigned>(blocks)), dim3(128), 0, stream, a);
}

}  // namespace qlin
