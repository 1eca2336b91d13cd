// kv_cache.cu -- new tokens into the paged INT8 key/value cache, and tokens
// out of it.
//
// kv_write: for each head x of 128 of a row of the fused q/k/v linear,
//   u = gamma x,  y = u rotated in pairs,  rho = 1 / sqrt(mean x^2 + eps),
//   query: bf16(y rho);  key, value: a = max|y|, code = rint(127 y / a),
//   scale = a rho / 127
// in one pass: the head is read once, and nothing is written but q, codes and
// scales.  rho is a factor of the whole head, so codes do not depend on it.
//
// Codes are those of exact arithmetic.  The fp32 quotient t = y (127 / a) is
// less than 2^-13 off (y by 2.42 half steps of a, as the products of a rotation
// are at most sqrt(2) a, a by as much, 127 / a by one, the product by one:
// 127 * 6.9 * 2^-24 = 2^-14.2).  Where t is further than that from a
// half-integer, its rounding is the exact one's; elsewhere (one element in
// 4096, and every x = a / 2 of a value head) y and a are formed again as
// unevaluated pairs of fp32 values (two-product and two-sum, error about 2^-46)
// and 254 |y| is compared with the odd multiple of a.
//
// A half warp holds a head, 8 components a lane, so that a rotation's partner
// is R/16 lanes away and reductions take four shuffles; a warp goes through
// heads of one row two at a time, with the rotation's factors in registers.
#include "f32x2.cuh"
#include "kv_cache.cuh"

namespace qlin {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr uint32_t kAll = 0xFFFFFFFFu;

// the larger of |a| and b; NaN where either is
__device__ __forceinline__ float max_abs(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(fabsf(a)), "f"(b));
  return d;
}

// reductions over a head's 16 lanes
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ float head_max(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = max_abs(__shfl_xor_sync(kAll, v, o), v);
  return v;
}

// a lane's 8 components, two at a time
struct Part {
  f32x2 v[4];
  __device__ __forceinline__ void fill(float x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pack2(x, x);
  }
  __device__ __forceinline__ void widen(const uint4& w) {
    v[0] = widen2(w.x);
    v[1] = widen2(w.y);
    v[2] = widen2(w.z);
    v[3] = widen2(w.w);
  }
  __device__ __forceinline__ void times(const Part& o) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], o.v[i]);
  }
  __device__ __forceinline__ void times(float x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], pack2(x, x));
  }
  __device__ __forceinline__ float square_sum() const {
    f32x2 s = mul2(v[0], v[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) s = fma2(v[i], v[i], s);
    float lo, hi;
    unpack2(s, lo, hi);
    return lo + hi;
  }
  __device__ __forceinline__ float top() const {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      unpack2(v[i], lo, hi);
      m = max_abs(lo, max_abs(hi, m));
    }
    return m;
  }
  __device__ __forceinline__ float get(int e) const {
    float lo, hi;
    unpack2(v[e >> 1], lo, hi);
    return (e & 1) ? hi : lo;
  }
};

// Factors of a lane's components in the rotation: y = u * own + partner * other.
struct Turn {
  Part own, other;
  __device__ __forceinline__ Part apply(const Part& u, const Part& partner) const {
    Part y;
#pragma unroll
    for (int i = 0; i < 4; ++i) y.v[i] = fma2(partner.v[i], other.v[i], mul2(u.v[i], own.v[i]));
    return y;
  }
};

__device__ __forceinline__ Turn load_turn(const KvWriteArgs& a, int64_t row, int pos, int i) {
  Turn t;
  t.own.fill(1.0f);
  t.other.fill(0.0f);
  const int R = static_cast<int>(a.R);
  if (8 * i >= R) return t;
  const int half = R / 2;
  const bool second = 8 * i >= half;
  const int pair0 = second ? 8 * i - half : 8 * i;
  const int last = static_cast<int>(a.P) - 1;
  float c[8], s[8];
  if (a.A <= 1 || a.positions == nullptr) {
    const int at = min(max(a.positions == nullptr ? pos : __ldg(a.positions + row), 0), last);
    const float4* const p = reinterpret_cast<const float4*>(a.cos_sin + static_cast<int64_t>(at) * R + pair0);
    const float4 c0 = __ldg(p), c1 = __ldg(p + 1), s0 = __ldg(p + half / 4), s1 = __ldg(p + half / 4 + 1);
    c[0] = c0.x, c[1] = c0.y, c[2] = c0.z, c[3] = c0.w, c[4] = c1.x, c[5] = c1.y, c[6] = c1.z, c[7] = c1.w;
    s[0] = s0.x, s[1] = s0.y, s[2] = s0.z, s[3] = s0.w, s[4] = s1.x, s[5] = s1.y, s[6] = s1.z, s[7] = s1.w;
  } else {
    const int64_t rows = a.c.B * a.T;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int axis = min(static_cast<int>(__ldg(a.axes + pair0 + e)), static_cast<int>(a.A) - 1);
      const int at = min(max(__ldg(a.positions + axis * rows + row), 0), last);
      const float* const p = a.cos_sin + static_cast<int64_t>(at) * R + pair0 + e;
      c[e] = __ldg(p);
      s[e] = __ldg(p + half);
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    t.own.v[e] = pack2(c[2 * e], c[2 * e + 1]);
    t.other.v[e] = second ? pack2(s[2 * e], s[2 * e + 1]) : pack2(-s[2 * e], -s[2 * e + 1]);
  }
  return t;
}

struct Pair {
  float hi, lo;
};

// u c + p s as an unevaluated pair
__device__ __forceinline__ Pair exact_turn(float u, float c, float p, float s) {
  const float q = __fmul_rn(u, c), qe = __fmaf_rn(u, c, -q);
  const float r = __fmul_rn(p, s), re = __fmaf_rn(p, s, -r);
  const float h = __fadd_rn(q, r);
  const float b = __fsub_rn(h, q);
  const float l = __fadd_rn(__fadd_rn(__fsub_rn(q, __fsub_rn(h, b)), __fsub_rn(r, b)), __fadd_rn(qe, re));
  const float hi = __fadd_rn(h, l);
  return {hi, __fsub_rn(l, __fsub_rn(hi, h))};
}

// The 8 codes of a lane, decided exactly (all lanes of the warp take part).
__device__ void exact_codes(const Part& u, const Part& partner, const Turn& turn, int code[8]) {
  Pair y[8];
  float top = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    y[e] = exact_turn(u.get(e), turn.own.get(e), partner.get(e), turn.other.get(e));
    if (y[e].hi < 0.0f) y[e].lo = -y[e].lo;      // of |y| from here on
    top = fmaxf(top, fabsf(y[e].hi));
  }
  top = head_max(top);
  float low = -INFINITY;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (fabsf(y[e].hi) == top) low = fmaxf(low, y[e].lo);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) low = fmaxf(low, __shfl_xor_sync(kAll, low, o));
  const float r = __fdiv_rn(127.0f, top);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float h = fabsf(y[e].hi);
    const float t = __fmul_rn(h, r);
    const float below = floorf(t);
    float n = rintf(t);
    if (fabsf(t - below - 0.5f) < 0x1p-12f) {
      const float odd = __fmaf_rn(2.0f, below, 1.0f);
      const float p = __fmul_rn(254.0f, h), pe = __fmaf_rn(254.0f, h, -p);
      const float q = __fmul_rn(odd, top), qe = __fmaf_rn(odd, top, -q);
      const float d = __fadd_rn(__fsub_rn(p, q), __fadd_rn(__fsub_rn(pe, qe), __fsub_rn(__fmul_rn(254.0f, y[e].lo), __fmul_rn(odd, low))));
      n = d > 0.0f ? below + 1.0f : d < 0.0f ? below : 2.0f * rintf(0.5f * (below + 0.5f));
    }
    code[e] = static_cast<int>(y[e].hi < 0.0f ? -n : n);
  }
}

// One unit of a warp: `per` pairs of heads of a row, of the row's `chunks` such.
// Query, key and value heads are paired among themselves.
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const KvWriteArgs a, int chunks, int per) {
  const int lane = threadIdx.x & 31;
  const int i = lane & 15;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  grid_dep_launch();
  grid_dep_wait();
  const int64_t row = unit / chunks;
  if (row >= a.c.B * a.T) return;
  const int64_t b = row / a.T;
  const int t = static_cast<int>(row - b * a.T);
  const int q_heads = static_cast<int>(a.q_heads), kv_heads = static_cast<int>(a.c.kv_heads);
  const int q_pairs = (q_heads + 1) / 2, kv_pairs = (kv_heads + 1) / 2;
  const SeqLen seq = seq_len(a.c, b, a.T);
  if (t >= seq.fresh) return;
  const int pos = seq.len - seq.fresh + t;
  const int first = static_cast<int>(unit - row * chunks) * per;
  const int last = min(first + per, q_pairs + 2 * kv_pairs);
  const uint16_t* const in = a.qkv + row * (q_heads + 2 * kv_heads) * kHeadDim + 8 * i;

  // where a pair's head of this half warp is: its kind, number and place in the row
  struct Head {
    int kind, at;
    bool there;
  };
  auto head_of = [&](int pair) {
    Head h;
    h.kind = pair < q_pairs ? 0 : pair < q_pairs + kv_pairs ? 1 : 2;
    h.at = 2 * (pair - (h.kind == 0 ? 0 : h.kind == 1 ? q_pairs : q_pairs + kv_pairs)) + (lane >> 4);
    h.there = h.at < (h.kind == 0 ? q_heads : kv_heads);
    return h;
  };
  auto load = [&](const Head& h) {
    if (!h.there) return make_uint4(0, 0, 0, 0);
    return __ldg(reinterpret_cast<const uint4*>(in + (h.at + (h.kind == 0 ? 0 : h.kind == 1 ? q_heads : q_heads + kv_heads)) * kHeadDim));
  };

  Head head = head_of(first);
  uint4 next = load(head);
  uint8_t* block = nullptr;       // of head 0
  if (last > q_pairs) block = cache_block(a.c, b, 0, pos >> 4);
  const int64_t head_step = (a.c.page_size >> 4) * kCacheBlock;
  const bool turned = a.R != 0;
  const Turn turn = load_turn(a, row, pos, i);
  const int step = static_cast<int>(a.R) >> 4;
  const int partner_lane = i < step ? lane + step : i < 2 * step ? lane - step : lane;
  Part gain, partner_gain;
  int gained = -1;                // the kind that the gains are of

  for (int pair = first; pair < last; ++pair) {
    const Head h = head;
    const uint4 x = next;
    if (pair + 1 < last) {
      head = head_of(pair + 1);
      next = load(head);
    }
    const uint16_t* const gamma = h.kind == 0 ? a.q_gamma : h.kind == 1 ? a.k_gamma : nullptr;
    if (gamma != nullptr && gained != h.kind) {
      gained = h.kind;
      gain.widen(__ldg(reinterpret_cast<const uint4*>(gamma) + i));
      partner_gain.widen(__ldg(reinterpret_cast<const uint4*>(gamma) + (partner_lane & 15)));
    }
    Part u;
    u.widen(x);
    float rho = 1.0f;
    if (gamma != nullptr) {
      const float sum = head_sum(u.square_sum());
      // a head of zeros stays one with eps = 0; a sum past fp32's range gives NaN
      rho = sum == 0.0f ? 0.0f : sum < INFINITY ? __frsqrt_rn(__fmaf_rn(sum, 1.0f / kHeadDim, a.eps)) : NAN;
      u.times(gain);
    }
    Part partner = u;
    Part y = u;
    if (turned && h.kind != 2) {
      uint4 w;
      w.x = __shfl_sync(kAll, x.x, partner_lane);
      w.y = __shfl_sync(kAll, x.y, partner_lane);
      w.z = __shfl_sync(kAll, x.z, partner_lane);
      w.w = __shfl_sync(kAll, x.w, partner_lane);
      partner.widen(w);
      if (gamma != nullptr) partner.times(partner_gain);
      y = turn.apply(u, partner);
    }
    if (h.kind == 0) {
      if (gamma != nullptr) y.times(rho);
      if (h.there)
        *reinterpret_cast<uint4*>(a.q + (row * q_heads + h.at) * kHeadDim + 8 * i) =
            make_uint4(narrow2(y.v[0]), narrow2(y.v[1]), narrow2(y.v[2]), narrow2(y.v[3]));
      continue;
    }

    float top = head_max(y.top());
    float scaled = 1.0f;
    if (__any_sync(kAll, (top > 0.0f && top < 0x1p-60f) || (top > 0x1p100f && top < INFINITY))) {
      // where 127 / a or the pairs' remainders would leave fp32's range
      scaled = top < 0x1p-60f ? 0x1p60f : top > 0x1p100f ? 0x1p-30f : 1.0f;
      u.times(scaled);
      partner.times(scaled);
      y = u;
      if (turned && h.kind != 2) y = turn.apply(u, partner);
      top = head_max(y.top());
    }
    const bool good = top > 0.0f && top < INFINITY;
    const float r = good ? __fdiv_rn(127.0f, top) : 0.0f;
    const f32x2 r2 = pack2(r, r);
    constexpr float kMagic = 12582912.0f + 128.0f;   // its low byte becomes code + 128
    const f32x2 magic = pack2(kMagic, kMagic);
    uint32_t m[8];
    float far = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const f32x2 n = fma2(y.v[e], r2, magic);
      const f32x2 back = sub2(n, magic);
      const f32x2 d = fma2(y.v[e], r2, mul2(back, pack2(-1.0f, -1.0f)));
      float lo, hi;
      unpack2(d, lo, hi);
      far = fmaxf(far, fmaxf(fabsf(lo), fabsf(hi)));
      unpack2(n, lo, hi);
      m[2 * e] = __float_as_uint(lo);
      m[2 * e + 1] = __float_as_uint(hi);
    }
    if (__any_sync(kAll, good && far > 0.5f - 0x1p-13f)) {
      Turn none;
      none.own.fill(1.0f);
      none.other.fill(0.0f);
      int code[8];
      exact_codes(u, partner, turned && h.kind != 2 ? turn : none, code);
      if (good) {
#pragma unroll
        for (int e = 0; e < 8; ++e) m[e] = static_cast<uint32_t>(code[e] + 128);
      }
    }
    if (!h.there || block == nullptr) continue;
    uint8_t* const to = block + h.at * head_step;
    const int place = pos & 15;
    const uint32_t lo = prmt(prmt(m[0], m[1], 0x0040u), prmt(m[2], m[3], 0x0040u), 0x5410u);
    const uint32_t hi = prmt(prmt(m[4], m[5], 0x0040u), prmt(m[6], m[7], 0x0040u), 0x5410u);
    *reinterpret_cast<uint2*>(to + (h.kind == 1 ? 0 : kVCodes) + place * kHeadDim + code_place(place, 8 * i)) = make_uint2(lo, hi);
    if (i == 0) {
      const float s = __fdiv_rn(__fmul_rn(top, rho), 127.0f) * (1.0f / scaled);
      reinterpret_cast<float*>(to + (h.kind == 1 ? kKScales : kVScales))[place] =
          top == 0.0f ? 0.0f : good && s < INFINITY ? s : NAN;
    }
  }
}

// A warp takes one block of 16 tokens of a head: 4 vectors of codes a lane and
// tensor, all in flight at once.
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const CacheArgs c, const int32_t* start, int64_t L, int spans,
                                                           uint16_t* k, uint16_t* v) {
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  grid_dep_launch();
  grid_dep_wait();
  const int kv_heads = static_cast<int>(c.kv_heads);
  const int64_t span = unit / kv_heads;
  const int h = static_cast<int>(unit - span * kv_heads);
  const int64_t b = span / spans;
  if (b >= c.B) return;
  const int len = seq_len(c, b, 1).len;
  const int first = start == nullptr ? 0 : min(max(__ldg(start + b), 0), len);
  const int n = first / 16 + static_cast<int>(span - b * spans);
  const int tok0 = 16 * n;
  const uint8_t* const block = tok0 < len ? cache_block(c, b, h, n) : nullptr;
  const int chunk = lane & 7;
  uint4 code[2][4];
  float scale[2][4];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = 4 * j + (lane >> 3);
      code[w][j] = make_uint4(0, 0, 0, 0);
      scale[w][j] = 0.0f;
      if (block != nullptr && tok0 + r < len && (w == 0 ? k : v) != nullptr) {
        code[w][j] = __ldg(reinterpret_cast<const uint4*>(block + w * kVCodes + r * kHeadDim + code_place(r, 16 * chunk)));
        scale[w][j] = __ldg(reinterpret_cast<const float*>(block + (w == 0 ? kKScales : kVScales)) + r);
      }
    }
  }
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    uint16_t* const out = w == 0 ? k : v;
    if (out == nullptr) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = 4 * j + (lane >> 3);
      const int64_t at = static_cast<int64_t>(tok0) + r - first;
      if (at < 0 || at >= L) continue;
      const bool there = block != nullptr && tok0 + r < len;
      const uint32_t words[4] = {code[w][j].x, code[w][j].y, code[w][j].z, code[w][j].w};
      uint32_t o[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // 2^23 + u for each byte u, less 2^23 + 128
        float f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          f[i] = (__uint_as_float(prmt(words[e], 0x4B000000u, 0x7440u + i)) - 8388736.0f) * scale[w][j];
        o[2 * e] = there ? bf16x2_rn(f[0], f[1]) : 0u;
        o[2 * e + 1] = there ? bf16x2_rn(f[2], f[3]) : 0u;
      }
      uint4* const to = reinterpret_cast<uint4*>(out + ((b * L + at) * kv_heads + h) * kHeadDim + 16 * chunk);
      to[0] = make_uint4(o[0], o[1], o[2], o[3]);
      to[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

}  // namespace

cudaError_t launch_kv_write(const KvWriteArgs& a, int sm_count, cudaStream_t stream) {
  const int64_t rows = a.c.B * a.T;
  const int64_t pairs = (a.q_heads + 1) / 2 + 2 * ((a.c.kv_heads + 1) / 2);
  // A warp takes one pair of heads until that fills the SMs' warps, then more
  // of a row, which share the rotation's factors.
  int per = 1;
  while (per < 8 && rows * ((pairs + per - 1) / per) > 2LL * 48 * sm_count) per *= 2;
  const int64_t chunks = (pairs + per - 1) / per;
  const int64_t blocks = (rows * chunks + kWarps - 1) / kWarps;
  if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
  return launch_pdl(kv_write_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, stream, a, static_cast<int>(chunks), per);
}

cudaError_t launch_kv_read(const CacheArgs& c, const int32_t* start, int64_t L, uint16_t* k, uint16_t* v,
                           cudaStream_t stream) {
  // blocks of 16 that L tokens from any start on may touch
  const int64_t spans = start == nullptr ? (L + 15) / 16 : (L + 30) / 16;
  const int64_t blocks = (c.B * spans * c.kv_heads + kWarps - 1) / kWarps;
  if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
  return launch_pdl(kv_read_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, stream, c, start, L,
                    static_cast<int>(spans), k, v);
}

}  // namespace qlin
