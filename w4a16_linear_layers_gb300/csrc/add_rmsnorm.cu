// add_rmsnorm.cu -- the residual addition fused with RMSNorm and the dynamic
// per-token INT8 activation quantization.
//
// For each row:  h = bf16(x + r),  t = bf16(h / sqrt(mean h^2 + eps)),
// z = bf16(gamma * t),  s = max|z| / 127,  q = rint(z / s): one read of x and
// r, one write of h and of the codes, instead of an elementwise addition, a
// second read of its result by the norm and a third by the quantizer.
//
// Exactness.  h, t, z, s and q are the values that the definition gives in
// exact arithmetic with its roundings (h, t, z to bf16; s and z / s to fp32):
//   * x + r and gamma * t are one bf16 instruction each, rounded once;
//   * the squares of bf16 values are exact in fp32 and are added with TwoSum
//     (Knuth), the dropped parts kept in a second sum;
//   * rstd is an unevaluated pair of fp32 values (relative error about 2^-44,
//     by a Newton-Raphson step on rsqrtf's result).  h * rstd is rounded to
//     bf16 from two fp32 products, one with a slightly larger and one with a
//     slightly smaller factor: rounding is monotonic, so where both give the same
//     bf16 value it is the exact product's, and elsewhere (one element in
//     8192) the side is decided with the product's remainder;
//   * codes come from the row's reciprocal scale in the same way, and next to
//     a half-integer from the IEEE divide.
// No binary64 arithmetic: this part runs it at 1/64 of the fp32 rate.
//
// What bounds it: HBM at many rows (7 or 8 bytes an element), with instruction
// issue close behind, which the two-element instructions (f32x2, bf16x2) are
// for (27 warp instructions for 32 elements); two block-wide reductions and
// the launch at few.  8192 x 5120: 55.1 us with fp16 codes, 6.09 TB/s, 0.90 of
// the copy rate (39 instructions took 62.7); 50.9 with int8 codes, 5.77 TB/s.  (A ring of rows filled ahead by
// bulk copies was slower, 74 us against 62 then: many small blocks already
// overlap one row's loads with another's reductions.)
#include <cuda_bf16.h>

#include "f32x2.cuh"
#include "qlin_device.cuh"
#include "qlin_internal.h"

namespace qlin {
namespace {

// (s, c) += h * h, c collecting what each addition to s drops (TwoSum, with
// the exact square inside the multiply-adds)
__device__ __forceinline__ void add_square2(f32x2& s, f32x2& c, f32x2 h) {
  const f32x2 t = fma2(h, h, s);
  const f32x2 nb = sub2(s, t);                 // -(t - s)
  const f32x2 ds = sub2(s, add2(t, nb));
  const f32x2 dv = fma2(h, h, nb);
  c = add2(c, add2(ds, dv));
  s = t;
}
// (s, c) += v
__device__ __forceinline__ void twosum1(float& s, float& c, float v) {
  const float t = __fadd_rn(s, v);
  const float bp = __fsub_rn(t, s);
  const float ap = __fsub_rn(t, bp);
  c = __fadd_rn(c, __fadd_rn(__fsub_rn(s, ap), __fsub_rn(v, bp)));
  s = t;
}

struct Rstd {
  float hi, lo;
};

// 1 / sqrt((s + c) / K + eps) as hi + lo; 1 / K as ki + kl.  y0 is rsqrtf's
// approximation; with r = 1 - v y0^2 (formed exactly to about 2^-45),
// 1 / sqrt(v) = y0 (1 - r)^(-1/2) = y0 + y0 (r / 2 + 3 r^2 / 8 + ...).
// v above 2^60 or below 2^-60 is brought nearer to 1 by a power of 4: from 2^105
// and 2^-104 on the products' remainders would be subnormal, and rounded.
// A row of zeros with eps = 0 gives 0; a sum that is not finite gives NaN (its
// c is NaN, from the difference of two infinities).
__device__ __forceinline__ Rstd row_rstd(float s, float c, float ki, float kl, float eps) {
  const float about = __fmaf_rn(s, ki, eps);
  const float back = about > 0x1p60f ? 0x1p-50f : about < 0x1p-60f ? 0x1p50f : 1.0f;
  const float scale = __fmul_rn(back, back);
  s = __fmul_rn(s, scale);
  float vh = __fmul_rn(s, ki);
  float vl = __fadd_rn(__fmaf_rn(s, ki, -vh), __fmaf_rn(s, kl, __fmul_rn(__fmul_rn(c, scale), ki)));
  twosum1(vh, vl, __fmul_rn(eps, scale));
  const float t = __fadd_rn(vh, vl);
  vl = __fsub_rn(vl, __fsub_rn(t, vh));
  vh = t;
  if (vh == 0.0f) return Rstd{0.0f, 0.0f};
  const float y0 = rsqrtf(vh);
  const float a = __fmul_rn(y0, y0);
  const float ae = __fmaf_rn(y0, y0, -a);
  const float p = __fmul_rn(vh, a);
  const float pe = __fadd_rn(__fmaf_rn(vh, a, -p), __fmaf_rn(vh, ae, __fmul_rn(vl, a)));
  const float r = __fsub_rn(__fsub_rn(1.0f, p), pe);
  const float corr = __fmul_rn(y0, __fmul_rn(r, __fmaf_rn(0.375f, r, 0.5f)));
  const float hi = __fadd_rn(y0, corr);
  return Rstd{__fmul_rn(hi, back), __fmul_rn(__fsub_rn(corr, __fsub_rn(hi, y0)), back)};
}

// bf16 bits of x * (hi + lo), rounded once: p + e is the product with its
// remainder, and p's distance from the bf16 halfway point of its binade step
// plus e decides the side.
__device__ __noinline__ uint32_t norm_border(float x, Rstd rs) {
  const float p = __fmul_rn(x, rs.hi);
  const float e = __fmaf_rn(x, rs.lo, __fmaf_rn(x, rs.hi, -p));
  const uint32_t u = __float_as_uint(p);
  const uint32_t low = u & 0xFFFFu;
  if (low - 0x7FFCu > 8u) return __bfloat16_as_ushort(__float2bfloat16_rn(p));
  const float half = __uint_as_float((u & 0x7FFF0000u) | 0x8000u);
  const float d = __fadd_rn(__fsub_rn(fabsf(p), half), (u >> 31) ? -e : e);
  const uint32_t base = u >> 16;
  if (d > 0.0f) return (base + 1u) & 0xFFFFu;
  if (d < 0.0f) return base;
  return (base + (base & 1u)) & 0xFFFFu;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// t of one bf16x2 word of h, with the products' remainders
__device__ __noinline__ uint32_t norm_pair_slow(uint32_t h, Rstd rs) {
  const uint32_t t0 = norm_border(__uint_as_float(h << 16), rs);
  const uint32_t t1 = norm_border(__uint_as_float(h & 0xFFFF0000u), rs);
  return t0 | (t1 << 16);
}

// A factor and its bounds 1 +- 2^-22: the fp32 rounding of the factor and of a
// product with it stay inside.
struct Bracket {
  f32x2 up, down;
  __device__ __forceinline__ explicit Bracket(float f) {
    const float u = __fmul_rn(f, 1.0f + 0x1p-22f), d = __fmul_rn(f, 1.0f - 0x1p-22f);
    up = pack2(u, u);
    down = pack2(d, d);
  }
};

__device__ __forceinline__ uint4 norm8(uint4 h, uint4 g, Rstd rs, const Bracket& b) {
  const uint32_t hw[4] = {h.x, h.y, h.z, h.w};
  const uint32_t gw[4] = {g.x, g.y, g.z, g.w};
  uint32_t t[4];
  uint32_t differ = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x2 f = widen2(hw[i]);
    t[i] = narrow2(mul2(f, b.up));
    differ |= t[i] ^ narrow2(mul2(f, b.down));
  }
  if (differ) {
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = norm_pair_slow(hw[i], rs);
  }
  return make_uint4(mul_bf16x2(t[0], gw[0]), mul_bf16x2(t[1], gw[1]), mul_bf16x2(t[2], gw[2]), mul_bf16x2(t[3], gw[3]));
}

// magnitudes of the larger ones (signs to be ignored); of a NaN and a number the number
__device__ __forceinline__ uint32_t absmax2(uint32_t m, uint32_t v) {
  uint32_t d;
  asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(m), "r"(v));
  return d;
}

constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23: t + kMagic rounds t to an integer

// Codes of 8 elements by IEEE divides.
__device__ __noinline__ void quant8_div(uint4 z, float s, float* r) {
  const uint32_t w[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[2 * i] = rintf(__fdiv_rn(__uint_as_float(w[i] << 16), s));
    r[2 * i + 1] = rintf(__fdiv_rn(__uint_as_float(w[i] & 0xFFFF0000u), s));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = fminf(fmaxf(r[i], -127.0f), 127.0f);
}

// Stores 8 codes: z / s rounded to an integer by adding kMagic, with the
// bounds of 1 / s; where they disagree (next to a half-integer) by the divide.
// `divide` takes it always (scales whose reciprocal overflows).
template <bool kC16>
__device__ __forceinline__ void quant_store8(uint4 z, float s, const Bracket& inv, bool divide, void* qrow,
                                             int64_t v) {
  const uint32_t w[4] = {z.x, z.y, z.z, z.w};
  const f32x2 magic2 = pack2(kMagic, kMagic);
  float m[8];       // r + kMagic
  f32x2 differ = divide ? 1ull : 0ull;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x2 f = widen2(w[i]);
    const f32x2 up = fma2(f, inv.up, magic2);
    differ |= up ^ fma2(f, inv.down, magic2);
    unpack2(up, m[2 * i], m[2 * i + 1]);
  }
  if (differ) {
    float r[8];
    quant8_div(z, s, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = r[i] + kMagic;
  }
  if constexpr (kC16) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float r0, r1;
      unpack2(add2(pack2(m[2 * i], m[2 * i + 1]), pack2(-kMagic, -kMagic)), r0, r1);   // -0 has become +0
      asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(o[i]) : "f"(r1), "f"(r0));
    }
    reinterpret_cast<uint4*>(qrow)[v] = make_uint4(o[0], o[1], o[2], o[3]);
  } else {
    // the low byte of r + kMagic's bits is r in two's complement
    uint32_t o[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t a = prmt(__float_as_uint(m[4 * i]), __float_as_uint(m[4 * i + 1]), 0x0040u);
      const uint32_t b = prmt(__float_as_uint(m[4 * i + 2]), __float_as_uint(m[4 * i + 3]), 0x0040u);
      o[i] = prmt(a, b, 0x5410u);
    }
    reinterpret_cast<uint2*>(qrow)[v] = make_uint2(o[0], o[1]);
  }
}

__device__ __forceinline__ uint4 add8(uint4 x, uint4 r) {
  return make_uint4(add_bf16x2(x.x, r.x), add_bf16x2(x.y, r.y), add_bf16x2(x.z, r.z), add_bf16x2(x.w, r.w));
}

__device__ __forceinline__ void sumsq8(uint4 h, f32x2& s, f32x2& c) {
  const uint32_t w[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) add_square2(s, c, widen2(w[i]));
}

struct AddNormParams {
  const uint16_t* x;
  const uint16_t* r;
  const uint16_t* gamma;
  uint16_t* h;
  void* q;
  float* s;
  uint16_t* y;
  int64_t K;
  float eps, ki, kl;   // 1 / K = ki + kl
};

__device__ __forceinline__ uint32_t map_block(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void row_sync() {   // all threads of the row's blocks
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The block's place among the kParts of its row.
template <int kParts>
__device__ __forceinline__ int block_of_row() {
  return static_cast<int>(blockIdx.x % kParts);
}

// The sums of squares of the block's threads -> rstd, in every thread.  Each
// warp's pair goes through shared memory and every warp adds all of them in
// the same order, so all threads hold the same rstd after one barrier.
// The kParts blocks of a row, a cluster, send them to one another, with a
// cluster barrier in the block's place.
template <int kParts>
__device__ __forceinline__ Rstd block_rstd(f32x2 s2, f32x2 c2, float2* red, const AddNormParams& p) {
  float s, s1, c, c1;
  unpack2(s2, s, s1);
  unpack2(c2, c, c1);
  c = __fadd_rn(c, c1);
  twosum1(s, c, s1);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float so = __shfl_xor_sync(0xFFFFFFFFu, s, o);
    const float co = __shfl_xor_sync(0xFFFFFFFFu, c, o);
    c = __fadd_rn(c, co);
    twosum1(s, c, so);
  }
  const int lane = threadIdx.x & 31;
  int nw = blockDim.x >> 5;
  if constexpr (kParts > 1) {
    if (lane < kParts)
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(
                       map_block(smem_u32(red + block_of_row<kParts>() * nw + (threadIdx.x >> 5)), lane)),
                   "f"(s), "f"(c)
                   : "memory");
    row_sync();
    nw *= kParts;
  } else if (nw > 1) {
    if (lane == 0) red[threadIdx.x >> 5] = make_float2(s, c);
    __syncthreads();
  }
  if (nw > 1) {
    const float2 mine = lane < nw ? red[lane] : make_float2(0.0f, 0.0f);
    s = mine.x;
    c = mine.y;
    for (int i = lane + 32; kParts > 1 && i < nw; i += 32) {
      c = __fadd_rn(c, red[i].y);
      twosum1(s, c, red[i].x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float so = __shfl_xor_sync(0xFFFFFFFFu, s, o);
      const float co = __shfl_xor_sync(0xFFFFFFFFu, c, o);
      c = __fadd_rn(c, co);
      twosum1(s, c, so);
    }
  }
  return row_rstd(s, c, p.ki, p.kl, p.eps);
}

template <int kParts>
__device__ __forceinline__ float block_absmax(uint32_t m2, uint32_t* red) {
  uint32_t m = max(m2 & 0x7FFFu, m2 >> 16 & 0x7FFFu);   // non-negative bf16 bits order as integers
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  const int lane = threadIdx.x & 31;
  int nw = blockDim.x >> 5;
  if constexpr (kParts > 1) {
    if (lane < kParts)
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(
                       map_block(smem_u32(red + block_of_row<kParts>() * nw + (threadIdx.x >> 5)), lane)),
                   "r"(m)
                   : "memory");
    row_sync();
    nw *= kParts;
  } else if (nw > 1) {
    if (lane == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
  }
  if (nw > 1) {
    m = lane < nw ? red[lane] : 0u;
    for (int i = lane + 32; kParts > 1 && i < nw; i += 32) m = max(m, red[i]);
    m = __reduce_max_sync(0xFFFFFFFFu, m);
  }
  return __uint_as_float(m << 16);
}

// NaN where the row has no finite norm: its z are all NaN, which the maximum leaves out.
__device__ __forceinline__ float row_scale(float amax, Rstd rs) {
  return rs.hi == rs.hi ? __fdiv_rn(amax, 127.0f) : __int_as_float(0x7FFFFFFF);
}

// kParts blocks (a cluster) per row, kVec vectors of 8 elements a thread
// (kParts * blockDim * kVec >= K / 8): the row stays in registers from its one
// read to the codes.
template <int kVec, int kParts, int kMaxThreads, int kMinBlocks, bool kC16>
__global__ void __launch_bounds__(kMaxThreads, kMinBlocks) add_rmsnorm_kernel(const AddNormParams p) {
  __shared__ float2 red[32 * kParts];
  __shared__ uint32_t redm[32 * kParts];
  if constexpr (kParts > 1) {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  }
  grid_dep_wait();     // x and r come from earlier kernels, which may still read h or q
  grid_dep_launch();
  const int nvec = static_cast<int>(p.K / 8);
  const int64_t row = blockIdx.x / kParts;
  const int64_t base = row * p.K;
  // h may be x or r itself: plain loads, every element read before its thread writes it
  const uint4* xr = reinterpret_cast<const uint4*>(p.x + base);
  const uint4* rr = reinterpret_cast<const uint4*>(p.r + base);
  const uint4* gr = reinterpret_cast<const uint4*>(p.gamma);
  uint4* hr = reinterpret_cast<uint4*>(p.h + base);
  uint4* yr = p.y ? reinterpret_cast<uint4*>(p.y + base) : nullptr;
  void* qr = kC16 ? static_cast<void*>(static_cast<uint16_t*>(p.q) + base)
                  : static_cast<void*>(static_cast<int8_t*>(p.q) + base);
  const int step = blockDim.x * kParts;
  const int tid = block_of_row<kParts>() * blockDim.x + threadIdx.x;   // among the row's threads

  uint4 h[kVec];
  {
    uint4 r[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int v = tid + i * step;
      h[i] = v < nvec ? xr[v] : make_uint4(0u, 0u, 0u, 0u);
      r[i] = v < nvec ? rr[v] : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) h[i] = add8(h[i], r[i]);
  }
  f32x2 s2 = 0ull, c2 = 0ull;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int v = tid + i * step;
    if (v < nvec) hr[v] = h[i];
    sumsq8(h[i], s2, c2);
  }
  if constexpr (kParts > 1) {   // the row's blocks have all started: their shared memory can be written
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  const Rstd rs = block_rstd<kParts>(s2, c2, red, p);
  const Bracket norm(rs.hi);
  uint32_t m2 = 0;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int v = tid + i * step;
    if (v < nvec) {
      h[i] = norm8(h[i], __ldg(gr + v), rs, norm);
      m2 = absmax2(absmax2(absmax2(absmax2(m2, h[i].x), h[i].y), h[i].z), h[i].w);
      if (yr) yr[v] = h[i];
    }
  }
  const float amax = block_absmax<kParts>(m2, redm);
  const float s = row_scale(amax, rs);
  if (tid == 0) p.s[row] = s;
  const bool zero = s == 0.0f;
  const Bracket inv(zero ? 0.0f : __frcp_rn(s));
  const bool divide = !zero && !(s >= 0x1p-120f);
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int v = tid + i * step;
    if (v < nvec) quant_store8<kC16>(h[i], s, inv, divide, qr, v);
  }
}

// Rows of more than 32768 elements: the same steps, h read back (from L2)
// for the norm, and the norm formed a second time for the codes.
template <bool kC16>
__global__ void __launch_bounds__(1024) add_rmsnorm_long_kernel(const AddNormParams p) {
  __shared__ float2 red[32];
  __shared__ uint32_t redm[32];
  grid_dep_wait();
  grid_dep_launch();
  const int64_t nvec = p.K / 8;
  const int64_t base = static_cast<int64_t>(blockIdx.x) * p.K;
  const uint4* xr = reinterpret_cast<const uint4*>(p.x + base);
  const uint4* rr = reinterpret_cast<const uint4*>(p.r + base);
  const uint4* gr = reinterpret_cast<const uint4*>(p.gamma);
  uint4* hr = reinterpret_cast<uint4*>(p.h + base);
  uint4* yr = p.y ? reinterpret_cast<uint4*>(p.y + base) : nullptr;
  void* qr = kC16 ? static_cast<void*>(static_cast<uint16_t*>(p.q) + base)
                  : static_cast<void*>(static_cast<int8_t*>(p.q) + base);
  f32x2 s2 = 0ull, c2 = 0ull;
  for (int64_t v = threadIdx.x; v < nvec; v += blockDim.x) {
    const uint4 h = add8(xr[v], rr[v]);
    hr[v] = h;
    sumsq8(h, s2, c2);
  }
  const Rstd rs = block_rstd<1>(s2, c2, red, p);
  const Bracket norm(rs.hi);
  uint32_t m2 = 0;
  for (int64_t v = threadIdx.x; v < nvec; v += blockDim.x) {
    const uint4 z = norm8(hr[v], __ldg(gr + v), rs, norm);   // this thread's own store
    m2 = absmax2(absmax2(absmax2(absmax2(m2, z.x), z.y), z.z), z.w);
    if (yr) yr[v] = z;
  }
  const float amax = block_absmax<1>(m2, redm);
  const float s = row_scale(amax, rs);
  if (threadIdx.x == 0) p.s[blockIdx.x] = s;
  const bool zero = s == 0.0f;
  const Bracket inv(zero ? 0.0f : __frcp_rn(s));
  const bool divide = !zero && !(s >= 0x1p-120f);
  for (int64_t v = threadIdx.x; v < nvec; v += blockDim.x)
    quant_store8<kC16>(norm8(hr[v], __ldg(gr + v), rs, norm), s, inv, divide, qr, v);
}

template <bool kC16>
cudaError_t launch_rows(const AddNormParams& p, int64_t M, int sm_count, cudaStream_t stream) {
  const int64_t nvec = p.K / 8;
  const dim3 grid(static_cast<unsigned>(M));
  if (nvec > 4096)
    return launch_pdl(add_rmsnorm_long_kernel<kC16>, grid, dim3(1024), 0, stream, p);
  auto threads = [&](int vec) {   // of a block with nvec / vec of them, in whole warps
    return dim3(static_cast<unsigned>((((nvec + vec - 1) / vec) + 31) / 32 * 32));
  };
  auto launch = [&](auto kernel, int vec) { return launch_pdl(kernel, grid, threads(vec), 0, stream, p); };
  auto launch_parts = [&](auto kernel, int vec, int parts) {
    return launch_cluster_pdl(kernel, dim3(static_cast<unsigned>(M * parts)), threads(vec * parts), 0, parts, stream,
                              p);
  };
  // As few vectors a thread as the row's threads allow while all rows run at
  // one time (the row's latency is the call's), those of long rows in several
  // blocks: 8 x 17408 3.7 us in four blocks a row and 5.9 in one, 152 x 17408 8.6
  // in two and 10.2 in one.  In four while half the SMs, or for blocks of which
  // two fit one all of them, take the clusters (38 x 17408 5.5 us, in one block
  // 7.9; 38 x 32768 10.1 and 9.3); in two above 16384 (152 x 12288 7.4 us, in one
  // block 6.9) and up to 18432.
  if (M <= sm_count && nvec <= 1024) return launch(add_rmsnorm_kernel<1, 1, 1024, 1, kC16>, 1);
  if (M * 8 <= sm_count || (M * 4 <= sm_count && nvec <= 2304))
    return launch_parts(add_rmsnorm_kernel<1, 4, 1024, 1, kC16>, 1, 4);
  if (M <= sm_count && nvec <= 2048) return launch(add_rmsnorm_kernel<2, 1, 1024, 1, kC16>, 2);
  if (M <= sm_count && nvec <= 2304) return launch_parts(add_rmsnorm_kernel<2, 2, 576, 2, kC16>, 2, 2);
  // Two while all rows' blocks run at one time (512 x 5120: 7.6 us, with four
  // 9.8) and for short rows (8192 x 2048: 24.9 and 26.6); else four, which
  // share the reductions' instructions (8192 x 5120: 55.4, with two 57.6).
  if (nvec <= 320 || (nvec <= 640 && M <= 4 * static_cast<int64_t>(sm_count)))
    return launch(add_rmsnorm_kernel<2, 1, 320, 4, kC16>, 2);
  // Blocks of 288 to 576 threads within 56 registers a thread, so that two
  // share an SM: 4096 x 17408 99.6 us, one an SM 120.7; shorter rows are faster
  // with 64 registers.
  if (nvec > 1152 && nvec <= 2304) return launch(add_rmsnorm_kernel<4, 1, 576, 2, kC16>, 4);
  return launch(add_rmsnorm_kernel<4, 1, 1024, 1, kC16>, 4);
}

}  // namespace

cudaError_t launch_add_rmsnorm_quant(const uint16_t* x, const uint16_t* r, const uint16_t* gamma,
                                     float eps, int64_t M, int64_t K, uint16_t* h, void* q,
                                     bool c16, float* s, uint16_t* y, int sm_count,
                                     cudaStream_t stream) {
  AddNormParams p{x, r, gamma, h, q, s, y, K, eps, 0.0f, 0.0f};
  const double inv = 1.0 / static_cast<double>(K);
  p.ki = static_cast<float>(inv);
  p.kl = static_cast<float>(inv - static_cast<double>(p.ki));
  return c16 ? launch_rows<true>(p, M, sm_count, stream) : launch_rows<false>(p, M, sm_count, stream);
}

}  // namespace qlin
