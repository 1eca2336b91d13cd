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
//   * x + r in fp32 rounds to the bf16 value nearest the exact sum: two bf16
//     values whose exponents differ by 16 or less add exactly in fp32, and
//     with a larger difference the sum is far from a bf16 halfway point;
//   * the squares of bf16 values are exact in fp32 and are added with TwoSum
//     (Knuth), the dropped parts kept in a second sum;
//   * rstd is an unevaluated pair of fp32 values (relative error about 2^-44,
//     by a Newton-Raphson step on rsqrtf's result): x * rstd is formed in fp32
//     and, where that value lies within 4 fp32 ulps of a bf16 halfway point
//     (it is within 2 of the exact one), the side is decided with the
//     product's remainder;
//   * codes come from the row's reciprocal scale and, next to a half-integer,
//     from the IEEE divide.
// No binary64 arithmetic: this part runs it at 1/64 of the fp32 rate.
//
// What bounds it: HBM at many rows (7 or 8 bytes an element); two block-wide
// reductions and the launch at few.  The elementwise arithmetic runs two
// elements to an instruction (add / mul.rn.f32x2), without which instruction
// issue would bind before HBM.
#include <cuda_bf16.h>

#include "qlin_device.cuh"
#include "qlin_internal.h"

namespace qlin {
namespace {

using f32x2 = unsigned long long;   // two fp32 values, the lower-indexed one low

__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
  f32x2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void unpack2(f32x2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 neg2(f32x2 a) { return a ^ 0x8000000080000000ull; }
__device__ __forceinline__ f32x2 sub2(f32x2 a, f32x2 b) { return add2(a, neg2(b)); }

// bf16x2 word -> its two values in fp32
__device__ __forceinline__ f32x2 widen2(uint32_t w) {
  return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t narrow2(f32x2 v) {
  float lo, hi;
  unpack2(v, lo, hi);
  return bf16x2_rn(lo, hi);
}

// (s, c) += v, c collecting what each addition to s drops (TwoSum)
__device__ __forceinline__ void twosum2(f32x2& s, f32x2& c, f32x2 v) {
  const f32x2 t = add2(s, v);
  const f32x2 bp = sub2(t, s);
  const f32x2 ap = sub2(t, bp);
  c = add2(c, add2(sub2(s, ap), sub2(v, bp)));
  s = t;
}
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

// 1 / sqrt((s + c) / K + eps) as hi + lo; inv_k = 1 / K as ki + kl.  y0 is
// rsqrtf's approximation; with r = 1 - v y0^2 (formed exactly to about 2^-45),
// 1 / sqrt(v) = y0 (1 - r)^(-1/2) = y0 + y0 (r / 2 + 3 r^2 / 8 + ...).
// A row of zeros with eps = 0 gives 0.
__device__ __forceinline__ Rstd row_rstd(float s, float c, float ki, float kl, float eps) {
  float vh = __fmul_rn(s, ki);
  float vl = __fadd_rn(__fmaf_rn(s, ki, -vh), __fmaf_rn(s, kl, __fmul_rn(c, ki)));
  twosum1(vh, vl, eps);
  const float t = __fadd_rn(vh, vl);
  vl = __fsub_rn(vl, __fsub_rn(t, vh));
  vh = t;
  if (!(vh > 0.0f)) return Rstd{0.0f, 0.0f};
  const float y0 = rsqrtf(vh);
  const float a = __fmul_rn(y0, y0);
  const float ae = __fmaf_rn(y0, y0, -a);
  const float p = __fmul_rn(vh, a);
  const float pe = __fadd_rn(__fmaf_rn(vh, a, -p), __fmaf_rn(vh, ae, __fmul_rn(vl, a)));
  const float r = __fsub_rn(__fsub_rn(1.0f, p), pe);
  const float corr = __fmul_rn(y0, __fmul_rn(r, __fmaf_rn(0.375f, r, 0.5f)));
  const float hi = __fadd_rn(y0, corr);
  return Rstd{hi, __fsub_rn(corr, __fsub_rn(hi, y0))};
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

// Non-zero when either fp32 value of the pair may lie within 4 ulps of a bf16
// halfway point (low 16 bits 0x7FFC .. 0x8003; a carry between the halves
// moves the upper window by one, which stays wider than the 2 ulps needed).
__device__ __forceinline__ uint32_t near_half2(f32x2 v) {
  float lo, hi;
  unpack2(v, lo, hi);
  const uint32_t w = prmt(__float_as_uint(lo), __float_as_uint(hi), 0x5410u) + 0x00040004u;
  const uint32_t y = (w & 0xFFF8FFF8u) ^ 0x80008000u;
  return (y - 0x00010001u) & ~y & 0x80008000u;
}

// z of one bf16x2 word of h
__device__ __noinline__ uint32_t norm_pair_slow(uint32_t h, uint32_t g, Rstd rs) {
  const uint32_t t0 = norm_border(__uint_as_float(h << 16), rs);
  const uint32_t t1 = norm_border(__uint_as_float(h & 0xFFFF0000u), rs);
  return narrow2(mul2(widen2(t0 | (t1 << 16)), widen2(g)));
}

__device__ __forceinline__ uint4 norm8(uint4 h, uint4 g, Rstd rs, f32x2 hi2) {
  const uint32_t hw[4] = {h.x, h.y, h.z, h.w};
  const uint32_t gw[4] = {g.x, g.y, g.z, g.w};
  uint32_t z[4];
  uint32_t border = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x2 t = mul2(widen2(hw[i]), hi2);
    border |= near_half2(t);
    // the product of two bf16 values is exact in fp32: one rounding
    z[i] = narrow2(mul2(widen2(narrow2(t)), widen2(gw[i])));
  }
  if (border) {
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] = norm_pair_slow(hw[i], gw[i], rs);
  }
  return make_uint4(z[0], z[1], z[2], z[3]);
}

__device__ __forceinline__ uint32_t absmax2(uint32_t m, uint32_t v) {
  const __nv_bfloat162 a = *reinterpret_cast<const __nv_bfloat162*>(&m);
  const uint32_t av = v & 0x7FFF7FFFu;
  const __nv_bfloat162 b = *reinterpret_cast<const __nv_bfloat162*>(&av);
  const __nv_bfloat162 r = __hmax2(a, b);
  return *reinterpret_cast<const uint32_t*>(&r);
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

// Stores 8 codes.  inv = 1 / s: t = z * inv is within 2^-16 of z / s (|t| <=
// 127), so further than 2^-15 from a half-integer t rounds as the IEEE
// quotient does; nearer, the divide is taken.  `divide` takes it always
// (scales whose reciprocal overflows).
template <bool kC16>
__device__ __forceinline__ void quant_store8(uint4 z, float s, float inv, bool divide, void* qrow,
                                             int64_t v) {
  const uint32_t w[4] = {z.x, z.y, z.z, z.w};
  const f32x2 inv2 = pack2(inv, inv);
  const f32x2 magic2 = pack2(kMagic, kMagic);
  float m[8];       // r + kMagic
  float far = 0.0f; // largest |t - r|
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x2 t = mul2(widen2(w[i]), inv2);
    const f32x2 mm = add2(t, magic2);
    const f32x2 d = sub2(t, sub2(mm, magic2));
    float d0, d1;
    unpack2(d, d0, d1);
    far = fmaxf(far, fmaxf(fabsf(d0), fabsf(d1)));
    unpack2(mm, m[2 * i], m[2 * i + 1]);
  }
  if (divide || far > 0.5f - 0x1p-15f) {
    float r[8];
    quant8_div(z, s, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = r[i] + kMagic;
  }
  if constexpr (kC16) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float r0 = m[2 * i] - kMagic, r1 = m[2 * i + 1] - kMagic;   // -0 becomes +0
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
  return make_uint4(narrow2(add2(widen2(x.x), widen2(r.x))), narrow2(add2(widen2(x.y), widen2(r.y))),
                    narrow2(add2(widen2(x.z), widen2(r.z))), narrow2(add2(widen2(x.w), widen2(r.w))));
}

__device__ __forceinline__ void sumsq8(uint4 h, f32x2& s, f32x2& c) {
  const uint32_t w[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x2 f = widen2(w[i]);
    twosum2(s, c, mul2(f, f));
  }
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

// The sums of squares of the block's threads -> rstd, in every thread.  Each
// warp's pair goes through shared memory and every warp adds all of them in
// the same order, so all threads hold the same rstd after one barrier.
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
  const int nw = blockDim.x >> 5;
  if (nw > 1) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(s, c);
    __syncthreads();
    const int lane = threadIdx.x & 31;
    const float2 mine = lane < nw ? red[lane] : make_float2(0.0f, 0.0f);
    s = mine.x;
    c = mine.y;
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

__device__ __forceinline__ float block_absmax(uint32_t m2, uint32_t* red) {
  uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);   // non-negative bf16 bits order as integers
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  const int nw = blockDim.x >> 5;
  if (nw > 1) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    m = __reduce_max_sync(0xFFFFFFFFu, lane < nw ? red[lane] : 0u);
  }
  return __uint_as_float(m << 16);
}

// One block per row, kVec vectors of 8 elements a thread (blockDim * kVec >=
// K / 8): the row stays in registers from its one read to the codes.
template <int kVec, bool kC16>
__global__ void __launch_bounds__(1024) add_rmsnorm_kernel(const AddNormParams p) {
  __shared__ float2 red[32];
  __shared__ uint32_t redm[32];
  grid_dep_wait();     // x and r come from earlier kernels, which may still read h or q
  grid_dep_launch();
  const int nvec = static_cast<int>(p.K / 8);
  const int64_t base = static_cast<int64_t>(blockIdx.x) * p.K;
  // h may be x or r itself: plain loads, every element read before its thread writes it
  const uint4* xr = reinterpret_cast<const uint4*>(p.x + base);
  const uint4* rr = reinterpret_cast<const uint4*>(p.r + base);
  const uint4* gr = reinterpret_cast<const uint4*>(p.gamma);
  uint4* hr = reinterpret_cast<uint4*>(p.h + base);
  uint4* yr = p.y ? reinterpret_cast<uint4*>(p.y + base) : nullptr;
  void* qr = kC16 ? static_cast<void*>(static_cast<uint16_t*>(p.q) + base)
                  : static_cast<void*>(static_cast<int8_t*>(p.q) + base);
  const int tid = threadIdx.x;
  const int step = blockDim.x;

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
  const Rstd rs = block_rstd(s2, c2, red, p);
  const f32x2 hi2 = pack2(rs.hi, rs.hi);
  uint32_t m2 = 0;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int v = tid + i * step;
    if (v < nvec) {
      h[i] = norm8(h[i], __ldg(gr + v), rs, hi2);
      m2 = absmax2(absmax2(absmax2(absmax2(m2, h[i].x), h[i].y), h[i].z), h[i].w);
      if (yr) yr[v] = h[i];
    }
  }
  const float amax = block_absmax(m2, redm);
  const float s = __fdiv_rn(amax, 127.0f);
  if (tid == 0) p.s[blockIdx.x] = s;
  const bool zero = amax == 0.0f;
  const float inv = zero ? 0.0f : __frcp_rn(s);
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
  const Rstd rs = block_rstd(s2, c2, red, p);
  const f32x2 hi2 = pack2(rs.hi, rs.hi);
  uint32_t m2 = 0;
  for (int64_t v = threadIdx.x; v < nvec; v += blockDim.x) {
    const uint4 z = norm8(hr[v], __ldg(gr + v), rs, hi2);   // this thread's own store
    m2 = absmax2(absmax2(absmax2(absmax2(m2, z.x), z.y), z.z), z.w);
    if (yr) yr[v] = z;
  }
  const float amax = block_absmax(m2, redm);
  const float s = __fdiv_rn(amax, 127.0f);
  if (threadIdx.x == 0) p.s[blockIdx.x] = s;
  const bool zero = amax == 0.0f;
  const float inv = zero ? 0.0f : __frcp_rn(s);
  const bool divide = !zero && !(s >= 0x1p-120f);
  for (int64_t v = threadIdx.x; v < nvec; v += blockDim.x)
    quant_store8<kC16>(norm8(hr[v], __ldg(gr + v), rs, hi2), s, inv, divide, qr, v);
}

template <bool kC16>
cudaError_t launch_rows(const AddNormParams& p, int64_t M, int sm_count, cudaStream_t stream) {
  const int64_t nvec = p.K / 8;
  const dim3 grid(static_cast<unsigned>(M));
  if (nvec > 4096)
    return launch_pdl(add_rmsnorm_long_kernel<kC16>, grid, dim3(1024), 0, stream, p);
  auto threads = [&](int vec) {
    return dim3(static_cast<unsigned>((((nvec + vec - 1) / vec) + 31) / 32 * 32));
  };
  // One vector a thread while every row has an SM of its own (the row's
  // latency is the call's) and the row fits 1024 threads; else four, whose
  // blocks are small enough for several rows to share an SM.
  if (M <= sm_count && nvec <= 1024)
    return launch_pdl(add_rmsnorm_kernel<1, kC16>, grid, threads(1), 0, stream, p);
  if (M <= sm_count && nvec <= 2048)
    return launch_pdl(add_rmsnorm_kernel<2, kC16>, grid, threads(2), 0, stream, p);
  return launch_pdl(add_rmsnorm_kernel<4, kC16>, grid, threads(4), 0, stream, p);
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
