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
// less than 2^-14 off (y by 2.42 half steps of a, as the products of a rotation
// are at most sqrt(2) a, a by as much, 127 / a by three: 127 * 7.84 * 2^-24 =
// 2^-14.04).  Where t is further than that from a half-integer, its rounding is
// the exact one's; for the rest (one element in 8192) y and a are formed again
// as unevaluated pairs of fp32 values (two-product and two-sum, error about
// 2^-46) and 254 |y| is compared with the odd multiple of a.  A head that is
// neither normalised nor rotated is bf16: there a half-integer is met exactly
// (every x = a / 2) or missed by 2^-17 of t, and t from 127 / a as a pair of
// fp32 values rounds as the exact one does.
//
// A quarter warp holds a head, 16 components a lane in two vectors of 8, which
// are each other's partners in the rotation: nothing passes between lanes but
// three steps of a reduction.  A warp goes through heads of one row four at a
// time, the next four on their way, with the rotation's factors in registers.
//
// Long calls wait for their loads: 8192 rows of 32 + 16 heads take 39.8 us, 4.6 TB/s of
// what has to move and 3.7 TB/s of DRAM traffic (what is written last stays in L2), 36.4 us
// where nothing is normalised or turned.  Memory is not full, nor is issue (53%): 20 warps
// an SM with one group each on its way, in 2.7 rounds of blocks.  With a half warp a head,
// partners R/16 lanes away and whole heads decided again where one code was near a
// half-integer it took 98.6.  Warps that stay and take rows in turn took 42 to 46 us, two
// or three groups ahead 46 to 48; 16 warps an SM 46, 24 with spilled registers 46 to 49.
// Short calls are a chain of loads (length, angles or page, the head) and take 3.6 us, 1.5
// of them above an empty launch.
#include <algorithm>
#include <type_traits>

#include "f32x2.cuh"
#include "kv_cache.cuh"

namespace qlin {
namespace {

// Warps have nothing to do with one another, and small blocks start and end by
// themselves: writes in blocks of one warp (12 x 8 rows 4.2 us, 4.6 in blocks of two or
// four; 8192 rows 39.7, 40.3, 40.5), reads of two (515 tokens 2.5 us, 2.8 in four;
// 12 x 8192 in blocks of one 93.1, of two 90.6).
//
// What kernels of this library write (rows of qkv, the cache) is read past L1: a kernel
// may start before the one in front of it, which writes them, and beside the one in front
// of that, whose reads could leave older lines in the L1 that they share.
constexpr int kReadWarps = 2;
constexpr int64_t kWritesAtOnce = 20;     // blocks of a write on an SM, which is what 96 registers allow
constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr float kSure = 0.5f - 0x1p-14f;   // quotients this near their codes round as the exact ones

// the largest of |a|, |b| and |c|; NaN where one is
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// reductions over a head's 8 lanes
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ float head_max(float v) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v = max_abs(__shfl_xor_sync(kAll, v, o), v, v);
  return v;
}

// 8 components, two at a time
struct Part {
  f32x2 v[4];
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
  __device__ __forceinline__ float top() const {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack2(v[i], f[2 * i], f[2 * i + 1]);
    return max_abs(max_abs(f[0], f[1], f[2]), max_abs(f[3], f[4], f[5]), max_abs(f[6], f[7], f[7]));
  }
};

// A lane's two vectors of a head's 16: with the first R/2 components turned
// against the next R/2, lanes below R/16 hold partners, the others neighbours
// of the rest.
struct Place {
  int at[2];            // vectors of 8 components
  bool turned;
  __device__ __forceinline__ Place(int R, int lane) {
    const int l = lane & 7, half = R >> 4;
    turned = l < half;
    at[0] = turned ? l : 2 * l;
    at[1] = turned ? l + half : 2 * l + 1;
  }
};

// cosines and sines of a turned lane's first vector: y0 = u0 c - u1 s, y1 = u1 c + u0 s
struct Turn {
  Part c, s;
};

__device__ __forceinline__ Turn load_turn(const KvWriteArgs& a, int64_t row, int pos, const Place& place) {
  Turn t;
  const int R = static_cast<int>(a.R), half = R / 2;
  const int pair0 = 8 * place.at[0];
  const int last = static_cast<int>(a.P) - 1;
  if (a.A <= 1 || a.positions == nullptr) {
    const int at = min(max(a.positions == nullptr ? pos : __ldg(a.positions + row), 0), last);
    const float4* const p = reinterpret_cast<const float4*>(a.cos_sin + static_cast<int64_t>(at) * R + pair0);
    const float4 c0 = __ldg(p), c1 = __ldg(p + 1), s0 = __ldg(p + half / 4), s1 = __ldg(p + half / 4 + 1);
    t.c.v[0] = pack2(c0.x, c0.y), t.c.v[1] = pack2(c0.z, c0.w), t.c.v[2] = pack2(c1.x, c1.y), t.c.v[3] = pack2(c1.z, c1.w);
    t.s.v[0] = pack2(s0.x, s0.y), t.s.v[1] = pack2(s0.z, s0.w), t.s.v[2] = pack2(s1.x, s1.y), t.s.v[3] = pack2(s1.z, s1.w);
  } else {
    const int64_t rows = a.c.B * a.T;
    float c[8], s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int axis = min(static_cast<int>(__ldg(a.axes + pair0 + e)), static_cast<int>(a.A) - 1);
      const int at = min(max(__ldg(a.positions + axis * rows + row), 0), last);
      const float* const p = a.cos_sin + static_cast<int64_t>(at) * R + pair0 + e;
      c[e] = __ldg(p);
      s[e] = __ldg(p + half);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      t.c.v[e] = pack2(c[2 * e], c[2 * e + 1]);
      t.s.v[e] = pack2(s[2 * e], s[2 * e + 1]);
    }
  }
  return t;
}

__device__ __forceinline__ void load_gain(const uint16_t* gamma, const Place& place, Part gain[2]) {
#pragma unroll
  for (int w = 0; w < 2; ++w) gain[w].widen(__ldg(reinterpret_cast<const uint4*>(gamma) + place.at[w]));
}

// u0 c - u1 s and u1 c + u0 s
__device__ __forceinline__ void turn_heads(const Part u[2], const Turn& t, Part y[2]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float u_lo, u_hi, s_lo, s_hi, q_lo, q_hi;
    unpack2(u[1].v[i], u_lo, u_hi);
    unpack2(t.s.v[i], s_lo, s_hi);
    unpack2(mul2(u[0].v[i], t.c.v[i]), q_lo, q_hi);
    const f32x2 second = fma2(u[0].v[i], t.s.v[i], mul2(u[1].v[i], t.c.v[i]));
    y[0].v[i] = pack2(__fmaf_rn(-u_lo, s_lo, q_lo), __fmaf_rn(-u_hi, s_hi, q_hi));   // (only these have a sign for free)
    y[1].v[i] = second;
  }
}

// four low bytes
__device__ __forceinline__ uint32_t low_bytes(const float m[4]) {
  return prmt(prmt(__float_as_uint(m[0]), __float_as_uint(m[1]), 0x0040u), prmt(__float_as_uint(m[2]), __float_as_uint(m[3]), 0x0040u),
              0x5410u);
}

// 1 / x, two half steps off at most for what is above 2^-100
__device__ __forceinline__ float rcp(float x) {
  float d;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(x));
  return d;
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

__device__ __forceinline__ float bf16_value(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

// Component e of a lane's 16 of the head at x, times `scaled`, as an
// unevaluated pair; formed again from memory, as few are asked for.
__device__ __forceinline__ Pair exact_component(const KvWriteArgs& a, uint32_t row, int pos, const uint16_t* x, const uint16_t* gamma,
                                                bool turned, const Place& place, int e, float scaled) {
  const int i = e & 7, d0 = 8 * place.at[0] + i, d1 = 8 * place.at[1] + i;
  // (the scaling first: a subnormal product would lose bits)
  float u0 = bf16_value(__ldcg(x + d0)) * scaled, u1 = bf16_value(__ldcg(x + d1)) * scaled;
  if (gamma != nullptr) u0 *= bf16_value(__ldg(gamma + d0)), u1 *= bf16_value(__ldg(gamma + d1));
  if (!turned) return {e < 8 ? u0 : u1, 0.0f};
  const int R = static_cast<int>(a.R);
  int at = pos;
  if (a.positions != nullptr) {
    const int axis = a.A <= 1 ? 0 : min(static_cast<int>(__ldg(a.axes + d0)), static_cast<int>(a.A) - 1);
    at = __ldg(a.positions + axis * (a.c.B * a.T) + row);
  }
  at = min(max(at, 0), static_cast<int>(a.P) - 1);
  const float* const p = a.cos_sin + static_cast<int64_t>(at) * R + d0;
  const float c = __ldg(p), s = __ldg(p + R / 2);
  return e < 8 ? exact_turn(u0, c, u1, -s) : exact_turn(u1, c, u0, s);
}

// A unit of a warp is `per` groups of four heads of row x, the y-th such.  Query,
// key and value heads are grouped among themselves.
struct Split {
  uint32_t per, q_groups, kv_groups;
};

__global__ void __launch_bounds__(32, kWritesAtOnce) kv_write_kernel(const __grid_constant__ KvWriteArgs a, const Split split) {
  const int lane = threadIdx.x;
  const uint32_t row = blockIdx.x;
  grid_dep_launch();
  grid_dep_wait();
  const int q_heads = static_cast<int>(a.q_heads), kv_heads = static_cast<int>(a.c.kv_heads);
  const int q_groups = split.q_groups, k_end = q_groups + split.kv_groups, groups = k_end + split.kv_groups;
  const int first = static_cast<int>(blockIdx.y * split.per);
  const int last = min(first + static_cast<int>(split.per), groups);
  const Place place(static_cast<int>(a.R), lane);

  // this quarter warp's head of the group whose components come next
  int at;                         // its number among the heads of its kind
  const uint16_t* x;
  uint4 next[2];
  auto load = [&](int heads) {
#pragma unroll
    for (int w = 0; w < 2; ++w) next[w] = at < heads ? __ldcg(reinterpret_cast<const uint4*>(x) + place.at[w]) : make_uint4(0, 0, 0, 0);
  };
  auto enter = [&](int group) {
    const bool query = group < q_groups, value = group >= k_end;
    at = 4 * (group - (query ? 0 : value ? k_end : q_groups)) + (lane >> 3);
    x = a.qkv + (static_cast<int64_t>(row) * (q_heads + 2 * kv_heads) + at + (query ? 0 : value ? q_heads + kv_heads : q_heads)) * kHeadDim;
    load(query ? q_heads : kv_heads);
  };

  enter(first);                   // (of rows of padding too: they are in the buffer)
  const uint32_t b = a.T == 1 ? row : row / static_cast<uint32_t>(a.T);
  const int t = static_cast<int>(row - b * static_cast<uint32_t>(a.T));
  const SeqLen seq = seq_len(a.c, b, a.T);
  if (t >= seq.fresh) return;
  const int pos = seq.len - seq.fresh + t;
  const bool turned = a.R != 0;
  Turn turn;
  if (place.turned) turn = load_turn(a, row, pos, place);
  const int place_of = pos & 15;
  const int64_t head_step = (a.c.page_size >> 4) * kCacheBlock;
  uint8_t* block = nullptr;       // of head 0
  if (last > q_groups) block = cache_block(a.c, b, 0, pos >> 4);

  auto run = [&](auto kind_of) {
    constexpr int kKind = decltype(kind_of)::value;
    const int from = max(first, kKind == 0 ? 0 : kKind == 1 ? q_groups : k_end);
    const int end = min(last, kKind == 0 ? q_groups : kKind == 1 ? k_end : groups);
    if (from >= end) return;
    const uint16_t* const gamma = kKind == 0 ? a.q_gamma : kKind == 1 ? a.k_gamma : nullptr;
    Part gain[2];
    if (gamma != nullptr) load_gain(gamma, place, gain);
    // the head's place in q or in the cache (where that has one)
    const bool placed = kKind == 0 || block != nullptr;
    uint8_t* to = kKind == 0 ? reinterpret_cast<uint8_t*>(a.q + (static_cast<int64_t>(row) * q_heads + at) * kHeadDim)
                             : (placed ? block : a.c.cache) + at * head_step + place_of * kHeadDim + (kKind == 1 ? 0 : kVCodes);
    const int64_t step = kKind == 0 ? 4 * kHeadDim * 2 : 4 * head_step;
    const int to_place[2] = {kKind == 0 ? 16 * place.at[0] : code_place(place_of, 8 * place.at[0]),
                             kKind == 0 ? 16 * place.at[1] : code_place(place_of, 8 * place.at[1])};
    const int heads = kKind == 0 ? q_heads : kv_heads;
    for (int group = from; group < end; ++group, to += step) {
      const uint4 x0 = next[0], x1 = next[1];
      const bool there = at < heads;
      const uint16_t* const head = x;
      if (group + 1 < end) {
        at += 4;
        x += 4 * kHeadDim;
        load(heads);
      } else if (kKind < 2 && end < last) {
        enter(end);
      }
      Part y[2];
      y[0].widen(x0);
      y[1].widen(x1);
      float rho = 1.0f;
      if (gamma != nullptr) {
        f32x2 two = mul2(y[0].v[0], y[0].v[0]);
#pragma unroll
        for (int e = 1; e < 8; ++e) two = fma2(y[e >> 2].v[e & 3], y[e >> 2].v[e & 3], two);
        float lo, hi;
        unpack2(two, lo, hi);
        const float sum = head_sum(lo + hi);
        // a head of zeros stays one with eps = 0; a sum past fp32's range gives NaN
        const float mean = __fmaf_rn(sum, 1.0f / kHeadDim, a.eps);
        rho = mean == 0.0f ? 0.0f : mean < INFINITY ? rsqrtf(mean) : NAN;
        y[0].times(gain[0]);
        y[1].times(gain[1]);
      }
      if (place.turned && kKind != 2) {      // (the others' would be u1 * 0 off: NaN beside an infinity)
        const Part u[2] = {y[0], y[1]};
        turn_heads(u, turn, y);
      }
      if constexpr (kKind == 0) {
        if (gamma != nullptr) {
          y[0].times(rho);
          y[1].times(rho);
        }
#pragma unroll
        for (int w = 0; w < 2; ++w)
          if (there)
            *reinterpret_cast<uint4*>(to + to_place[w]) =
                make_uint4(narrow2(y[w].v[0]), narrow2(y[w].v[1]), narrow2(y[w].v[2]), narrow2(y[w].v[3]));
        continue;
      }
      float top = head_max(max_abs(y[0].top(), y[1].top(), 0.0f));
      const bool good = top > 0.0f && top < INFINITY;
      const float inverse = rcp(top);
      const float r = good ? 127.0f * inverse : 0.0f;
      constexpr float kMagic = 12582912.0f + 128.0f;   // its low byte becomes code + 128
      const f32x2 magic = pack2(kMagic, kMagic), minus = pack2(-1.0f, -1.0f), r2 = pack2(r, r);
      uint32_t codes[4];
      const bool out_of_range = good && (top < 0x1p-60f || top > 0x1p100f);
      float far = 0.0f;               // the largest distance of a quotient from its code
      if (gamma == nullptr && !(turned && kKind == 1)) {
        const float rest = good ? __fmul_rn(__fmaf_rn(-top, r, 127.0f), inverse) : 0.0f;
        const f32x2 rest2 = pack2(rest, rest);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          float m[4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const f32x2 v = y[w >> 1].v[2 * (w & 1) + i];
            unpack2(add2(fma2(v, r2, mul2(v, rest2)), magic), m[2 * i], m[2 * i + 1]);
          }
          codes[w] = low_bytes(m);
        }
      } else {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          float m[4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const f32x2 v = y[w >> 1].v[2 * (w & 1) + i];
            const f32x2 n = fma2(v, r2, magic);
            // v r - (n - magic), rounded once: the sum in brackets is exact
            const f32x2 d = fma2(v, r2, fma2(n, minus, magic));
            float lo, hi;
            unpack2(d, lo, hi);
            far = max_abs(far, lo, hi);
            unpack2(n, m[2 * i], m[2 * i + 1]);
          }
          codes[w] = low_bytes(m);
        }
      }
      float back = 1.0f;
      if (__any_sync(kAll, good && (far > kSure || out_of_range))) {
        // Elements to decide (bits 0..15), and those that may be the largest: all of
        // a head where 127 / a or the pairs' remainders would leave fp32's range.
        const float scaled = !out_of_range ? 1.0f : top < 1.0f ? 0x1p60f : 0x1p-30f;
        uint32_t unsure = 0, tops = 0;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float lo, hi;
          unpack2(y[e >> 3].v[(e & 7) >> 1], lo, hi);
          const float v = fabsf((e & 1) ? hi : lo);
          const float n = __fmaf_rn(v, r, kMagic);
          if (out_of_range || fabsf(__fmaf_rn(v, r, kMagic - n)) > kSure) unsure |= 1u << e;
          if (out_of_range || v >= top * (1.0f - 0x1p-20f)) tops |= 1u << e;
        }
        const float head_far = head_max(far);
        if (!good || !(head_far > kSure || out_of_range)) unsure = tops = 0;
        const bool rotated = place.turned && kKind == 1;
        Pair most{0.0f, -INFINITY};   // of the head, as a pair
        for (; __any_sync(kAll, tops != 0); tops &= tops - 1) {
          if (tops == 0) continue;
          Pair v = exact_component(a, row, pos, head, gamma, rotated, place, __ffs(tops) - 1, scaled);
          if (v.hi < 0.0f) v.lo = -v.lo, v.hi = -v.hi;
          if (v.hi > most.hi || (v.hi == most.hi && v.lo > most.lo)) most = v;
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) {
          const Pair v{__shfl_xor_sync(kAll, most.hi, o), __shfl_xor_sync(kAll, most.lo, o)};
          if (v.hi > most.hi || (v.hi == most.hi && v.lo > most.lo)) most = v;
        }
        const float per_top = __fdiv_rn(127.0f, most.hi);
        for (; __any_sync(kAll, unsure != 0); unsure &= unsure - 1) {
          if (unsure == 0) continue;
          const int e = __ffs(unsure) - 1;
          Pair v = exact_component(a, row, pos, head, gamma, rotated, place, e, scaled);
          const bool negative = v.hi < 0.0f;
          if (negative) v.lo = -v.lo, v.hi = -v.hi;
          const float t = __fmul_rn(v.hi, per_top);
          const float below = floorf(t);
          float n = rintf(t);
          if (fabsf(t - below - 0.5f) < 0x1p-12f) {
            const float odd = __fmaf_rn(2.0f, below, 1.0f);
            const float p = __fmul_rn(254.0f, v.hi), pe = __fmaf_rn(254.0f, v.hi, -p);
            const float q = __fmul_rn(odd, most.hi), qe = __fmaf_rn(odd, most.hi, -q);
            const float d = __fadd_rn(__fsub_rn(p, q), __fadd_rn(__fsub_rn(pe, qe), __fsub_rn(__fmul_rn(254.0f, v.lo), __fmul_rn(odd, most.lo))));
            n = d > 0.0f ? below + 1.0f : d < 0.0f ? below : 2.0f * rintf(0.5f * (below + 0.5f));
          }
          const uint32_t code = static_cast<uint32_t>(static_cast<int>(negative ? -n : n) + 128);
          const int shift = 8 * (e & 3);
#pragma unroll
          for (int w = 0; w < 4; ++w)
            if (e >> 2 == w) codes[w] = (codes[w] & ~(0xFFu << shift)) | code << shift;
        }
        if (out_of_range) {
          top = most.hi;
          back = 1.0f / scaled;
        }
      }
      if (!there || !placed) continue;
#pragma unroll
      for (int w = 0; w < 2; ++w) *reinterpret_cast<uint2*>(to + to_place[w]) = make_uint2(codes[2 * w], codes[2 * w + 1]);
      if ((lane & 7) == 0) {
        const float s = __fmul_rn(__fmul_rn(top, rho), 1.0f / 127.0f) * back;
        // from the token's codes to its scale
        const int to_scale = (kKind == 1 ? kKScales : kVScales - kVCodes) + place_of * (4 - kHeadDim);
        *reinterpret_cast<float*>(to + to_scale) = top == 0.0f ? 0.0f : good && s < INFINITY ? s : NAN;
      }
      }
    };
  run(std::integral_constant<int, 0>());
  run(std::integral_constant<int, 1>());
  run(std::integral_constant<int, 2>());
}

// A warp takes one block of 16 tokens of a head: 4 vectors of codes a lane and
// tensor, all in flight at once.
__global__ void __launch_bounds__(32 * kReadWarps) kv_read_kernel(const CacheArgs c, const int32_t* start, int64_t L, uint32_t spans,
                                                           uint16_t* k, uint16_t* v) {
  const int lane = threadIdx.x & 31;
  const uint32_t unit = blockIdx.x * kReadWarps + (threadIdx.x >> 5);
  grid_dep_launch();
  grid_dep_wait();
  const uint32_t kv_heads = static_cast<uint32_t>(c.kv_heads);
  const uint32_t span = unit / kv_heads;
  const int h = static_cast<int>(unit - span * kv_heads);
  const uint32_t b = span / spans;
  if (b >= c.B) return;
  // Lengths, starts and, where no start shifts it, the page are on their way together
  // (an entry past the sequence's length is not used).
  const int total = __ldcg(c.total_len + b), from = start == nullptr ? 0 : __ldg(start + b);
  const int per_page = static_cast<int>(c.page_size) >> 4;
  const int32_t* const table = c.block_table + b * c.max_pages;
  int n = static_cast<int>(span - b * spans);
  int of_table = per_page == 1 ? n : n / per_page;
  int page = start == nullptr && of_table < c.max_pages ? __ldg(table + of_table) : -1;
  const int len = seq_of(c, 1, total, 0).len;
  const int first = min(max(from, 0), len);
  if (start != nullptr) {
    n += first >> 4;
    of_table = per_page == 1 ? n : n / per_page;
    if (16LL * n < len) page = __ldg(table + of_table);
  }
  const int64_t tok0 = 16LL * n;
  const uint8_t* const block =
      tok0 < len && page >= 0 && page < c.pages
          ? c.cache + ((static_cast<int64_t>(page) * kv_heads + h) * per_page + (n - of_table * per_page)) * kCacheBlock
          : nullptr;
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
        code[w][j] = __ldcg(reinterpret_cast<const uint4*>(block + w * kVCodes + r * kHeadDim + code_place(r, 16 * chunk)));
        scale[w][j] = __ldcg(reinterpret_cast<const float*>(block + (w == 0 ? kKScales : kVScales)) + r);
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
      const int64_t at = tok0 + r - first;
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
  const int64_t q_groups = (a.q_heads + 3) / 4, kv_groups = (a.c.kv_heads + 3) / 4, groups = q_groups + 2 * kv_groups;
  // Rows are cut into as many parts as run at one time, whose groups share the
  // rotation's factors (1545 ragged rows of 9 groups of three axes: whole 7.5 us, in
  // parts for two rounds 8.8, for three 10.3; 700 rows of 12 groups: in four 6.0, in
  // eight 7.3).
  const int64_t parts = std::min(std::max<int64_t>(kWritesAtOnce * sm_count / rows, 1), groups);
  const int64_t per = (groups + parts - 1) / parts;
  const int64_t chunks = (groups + per - 1) / per;
  const Split split{static_cast<uint32_t>(per), static_cast<uint32_t>(q_groups), static_cast<uint32_t>(kv_groups)};
  return launch_pdl(kv_write_kernel, dim3(static_cast<unsigned>(rows), static_cast<unsigned>(chunks)), dim3(32), 0, stream, a, split);
}

cudaError_t launch_kv_read(const CacheArgs& c, const int32_t* start, int64_t L, uint16_t* k, uint16_t* v,
                           cudaStream_t stream) {
  // blocks of 16 that L tokens from any start on may touch
  const int64_t spans = start == nullptr ? (L + 15) / 16 : (L + 30) / 16;
  if (c.B > 0x7FFFFFFFLL / (spans * c.kv_heads)) return cudaErrorInvalidConfiguration;    // (outputs of 2^43 bytes)
  const int64_t blocks = (c.B * spans * c.kv_heads + kReadWarps - 1) / kReadWarps;
  return launch_pdl(kv_read_kernel, dim3(static_cast<unsigned>(blocks)), dim3(32 * kReadWarps), 0, stream, c, start, L,
                    static_cast<uint32_t>(spans), k, v);
}

}  // namespace qlin
