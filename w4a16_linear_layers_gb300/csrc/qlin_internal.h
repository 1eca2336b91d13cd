// qlin_internal.h -- host-side declarations shared by the translation units
// of libqlin (launchers called from the C ABI in qlin_api.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace qlin {

// Per-device facts cached by the API layer.
struct DeviceInfo {
  int device = -1;
  int sm_count = 0;
  bool supported = false;  // sm_103
  int* err_word = nullptr; // device address of the error word
};

// Returns the cached info of the current device (nullptr if no device).
const DeviceInfo* current_device();

// TMA descriptors (tensor_map.cu); false if the driver refuses the map.
// make_act_map: 16-bit codes or activations [M, K] as boxes of `halves`
// 64-wide K halves x T rows; make_map_2d: a plain row-major matrix.
bool make_act_map(CUtensorMap* map, CUtensorMapDataType dtype, const void* base, uint64_t M,
                  uint64_t K, uint32_t T, uint32_t halves);
bool make_map_2d(CUtensorMap* map, CUtensorMapDataType dtype, const void* base, uint64_t inner,
                 uint64_t outer, uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer,
                 CUtensorMapSwizzle swz);

// The act-quant producers write the codes q as int8, or (c16) as the same
// integers in fp16 [M, K].
cudaError_t launch_act_quant(const uint16_t* x, int64_t M, int64_t K, void* q, bool c16,
                             float* s, cudaStream_t stream);

cudaError_t launch_rmsnorm_quant(const uint16_t* x, const uint16_t* gamma, float eps, int64_t M,
                                 int64_t K, void* q, bool c16, float* s, uint16_t* y, int* err,
                                 int sm_count, cudaStream_t stream);

cudaError_t launch_silu_mul_quant(const uint16_t* gate_up, int64_t M, int64_t I, void* q,
                                  bool c16, float* s, uint16_t* y, int* err, int sm_count,
                                  cudaStream_t stream);

// Residual addition + RMSNorm + act-quant; h (the sum) may be x or r.
cudaError_t launch_add_rmsnorm_quant(const uint16_t* x, const uint16_t* r, const uint16_t* gamma,
                                     float eps, int64_t M, int64_t K, uint16_t* h, void* q,
                                     bool c16, float* s, uint16_t* y, int sm_count,
                                     cudaStream_t stream);

// The W8A8 linear with one scale per token and one per output channel.
struct ChannelGemmArgs {
  const void* act;        // int8 or (act_c16) fp16 codes [M, K]
  bool act_c16;
  const float* s_a;       // [M]
  const int32_t* qweight; // [K/4, N]
  const float* s_w;       // [N]
  uint16_t* y;            // bf16 [M, N]
  int64_t M, N, K;
  void* workspace;        // channel_workspace_bytes(M, N, K, act_c16, sm_count) bytes
};
// Sums of 130944 products of two int8 values stay below 2^31.
constexpr int64_t kChannelMaxK = 130944;
size_t channel_workspace_bytes(int64_t M, int64_t N, int64_t K, bool c16, int sm_count);
cudaError_t launch_gemm_channel(const ChannelGemmArgs& a, int* err, int sm_count,
                                cudaStream_t stream);

// Penalties, biases and the grammar mask on logits (f32 or bf16).
struct LogitArgs {
  const void* logits;
  bool f32;
  int64_t M, V;
  const int32_t* tokens;      // [M, L] or nullptr
  int64_t L;
  const int32_t* prompt_len;  // [M] or nullptr
  const int32_t* total_len;   // [M] or nullptr
  const float* repetition;    // [M] or nullptr
  const float* presence;
  const float* frequency;
  const int32_t* bias_ids;    // [M, B] or nullptr
  const float* bias;
  int64_t B;
  const int32_t* allowed;     // [M, ceil(V / 32)] or nullptr
  void* out;                  // the logits' type, or nullptr
  int32_t* argmax;            // [M] or nullptr
};
cudaError_t launch_adjust_logits(const LogitArgs& a, int* err, int sm_count, cudaStream_t stream);

// The paged INT8 key/value cache and where its sequences' tokens are.
constexpr int kCacheBlock = 4224;   // bytes of 16 tokens of a head
struct CacheArgs {
  uint8_t* cache;
  int64_t pages, kv_heads, page_size;
  const int32_t* block_table;   // [B, max_pages]
  int64_t B, max_pages;
  const int32_t* total_len;     // [B]
  const int32_t* new_len;       // [B] or nullptr
};

struct KvWriteArgs {
  CacheArgs c;
  const uint16_t* qkv;          // [B T, q_heads + 2 kv_heads, 128]
  int64_t T, q_heads;
  const uint16_t* q_gamma;      // [128] or nullptr
  const uint16_t* k_gamma;
  float eps;
  const float* cos_sin;         // [P, R] or nullptr
  int64_t P, R;
  const int32_t* positions;     // [A, B T] or nullptr
  int64_t A;
  const uint8_t* axes;          // [R / 2] or nullptr
  uint16_t* q;                  // [B T, q_heads, 128]
};
cudaError_t launch_kv_write(const KvWriteArgs& a, int sm_count, cudaStream_t stream);

// k, v: bf16 [B, L, kv_heads, 128], either may be nullptr
cudaError_t launch_kv_read(const CacheArgs& c, const int32_t* start, int64_t L, uint16_t* k, uint16_t* v,
                           cudaStream_t stream);

struct PagedAttnArgs {
  CacheArgs c;
  const uint16_t* q;            // [B T, q_heads, 128]
  int64_t T, q_heads;
  float scale, softcap;
  int64_t window;
  bool causal;
  uint16_t* out;                // as q
  void* workspace;
};
size_t paged_attn_workspace_bytes(int64_t B, int64_t T, int64_t q_heads, int64_t kv_heads, int sm_count);
cudaError_t launch_paged_attn(const PagedAttnArgs& a, int* err, int sm_count, cudaStream_t stream);

cudaError_t launch_pack(const int8_t* q, int64_t K, int64_t N, int bits, int32_t* qweight,
                        int32_t* qzeros, int* err, cudaStream_t stream);

cudaError_t launch_wait_timeout(int64_t limit_ns, int* err, cudaStream_t stream);

cudaError_t launch_ingest_nk(const int32_t* packed_nk, const uint16_t* scales_ng, int64_t K,
                             int64_t N, int bits, int32_t* qweight, uint16_t* scales,
                             cudaStream_t stream);

// Bytes of the tile layout of a [K*bits/32, N] GPTQ weight matrix, and the
// repack into it (see tiles_kernel in pack.cu).
size_t tiles_bytes(int64_t K, int64_t N, int bits);
cudaError_t launch_pack_tiles(const int32_t* qweight, int64_t K, int64_t N, int bits,
                              int32_t* tiles, cudaStream_t stream);

// GEMM problem description passed from the API to the launcher.
enum class GemmMode : int { kW8A8 = 0, kW8A8Partials = 1, kW4A16 = 2, kW8A16 = 3 };

struct GemmArgs {
  GemmMode mode;
  const void* act;        // int8 q_a [M,K] (W8A8) or bf16 x [M,K] (W4A16)
  const float* s_a;       // W8A8 only
  const int32_t* qweight; // [K/4,N] or [K/8,N]
  const uint16_t* scales; // fp16 (W8A8) or bf16 (W4A16) [K/128,N]
  void* out;              // bf16 y [M,N] or int32 P [K/128,M,N]
  int64_t M, N, K;
  void* workspace;
  size_t workspace_bytes;
  // Greedy-argmax variant: instead of writing y, reduce every output row to
  // a 64-bit key (order-preserving bf16 bits << 32 | ~n) with atomicMax; the
  // largest key is the largest value, lowest n on ties.  nullptr = write y.
  unsigned long long* amax_keys = nullptr;
  // W8A16: K-width of a scale group (32 or 128), or 0 for one scale per column
  int group_size = 128;
  // Weights in the tile layout (qweight is then unused), else nullptr.
  const int32_t* wtiles = nullptr;
  // W8A8: act holds the codes as fp16 [M,K] (integers in [-127, 127])
  // instead of int8.
  bool act_c16 = false;
};

// Offset of the argmax keys (one per row, M <= 96) inside the fixed counter
// region at the start of the workspace.
constexpr size_t kArgmaxKeysOffset = 4096;
constexpr int64_t kArgmaxMaxRows = 96;

// idx[m] = the column index encoded in keys[m] (-1 if no key).  Programmatic
// dependent launch: waits for the GEMM that produced the keys.
cudaError_t launch_argmax_finalize(const unsigned long long* keys, int64_t M, int32_t* idx,
                                   cudaStream_t stream);

// Tiling plan for one GEMM call.
struct GemmPlan {
  int T;           // token tile (MMA N): 16, 32, 64 or 96
  int64_t F;       // feature tiles of 128
  int64_t TT;      // token tiles
  int64_t G;       // groups of 128 along K
  int64_t steps;   // TT * F * G
  int64_t ctas;    // grid size
  int64_t band;    // banded whole-tile schedule: token tiles per band (0: stream-K)
  size_t counter_bytes;
  size_t act_offset;     // W8A8 activations in the other code width: the fp16
                         // image of int8 codes (token tiles >= 64) or the int8
                         // codes of fp16 ones (token tiles <= 32)
  size_t workspace_bytes;
};

GemmPlan plan_gemm(int64_t M, int64_t N, int64_t K, int sm_count);

cudaError_t launch_gemm(const GemmArgs& a, const GemmPlan& p, int* err, cudaStream_t stream);

// Launches `kernel` with programmatic stream serialization: it may start
// before the previous kernel on the stream has finished, and must call
// griddepcontrol.wait before it touches memory that kernel produces or uses.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// launch_pdl in clusters of `cluster` blocks along x (grid.x a multiple of it).
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                               int cluster, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

}  // namespace qlin
