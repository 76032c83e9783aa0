// cfc_trunk.cuh -- device helpers of the trunk operators (layer norm, dropout, causal
// convolution, selective scan): 8-column loads and stores of fp32 or bf16 activations, the
// activations' functions, and the counter-based generator.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "cfc_ptx.cuh"

namespace cfc {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// Eight consecutive activations as they are stored: 32 bytes of fp32 or 16 bytes of bf16, one
// load each (p aligned to that size), or element by element.
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
  float v[8];
  __device__ __forceinline__ void load(const float* p) {
    asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
                   "=f"(v[6]), "=f"(v[7])
                 : "l"(p));
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
  }
  __device__ __forceinline__ void set(int j, float x) { v[j] = x; }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = v[j];
  }
  // To and from shared memory, in pieces of 16 bytes `stride` of them apart.
  __device__ __forceinline__ void put(uint4* p, int stride) const {
    float4* const to = reinterpret_cast<float4*>(p);
    to[0] = make_float4(v[0], v[1], v[2], v[3]);
    to[stride] = make_float4(v[4], v[5], v[6], v[7]);
  }
  __device__ __forceinline__ void pick(const uint4* p, int stride) {
    const float4* const from = reinterpret_cast<const float4*>(p);
    const float4 lo = from[0], hi = from[stride];
    v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
    v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
  }
};
template <>
struct Raw8<__nv_bfloat16> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 r = *reinterpret_cast<const uint4*>(p);
    w[0] = r.x; w[1] = r.y; w[2] = r.z; w[3] = r.w;
  }
  __device__ __forceinline__ void clear() { w[0] = w[1] = w[2] = w[3] = 0u; }
  // Into a cleared place.
  __device__ __forceinline__ void set(int j, __nv_bfloat16 x) {
    w[j / 2] |= static_cast<uint32_t>(__bfloat16_as_ushort(x)) << (16 * (j % 2));
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_lo_f32(w[i]);
      f[2 * i + 1] = bf16_hi_f32(w[i]);
    }
  }
  __device__ __forceinline__ void put(uint4* p, int) const { *p = make_uint4(w[0], w[1], w[2], w[3]); }
  __device__ __forceinline__ void pick(const uint4* p, int) {
    const uint4 r = *p;
    w[0] = r.x; w[1] = r.y; w[2] = r.z; w[3] = r.w;
  }
};
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]),
               "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint4 r;
  r.x = bf16x2_rn(v[0], v[1]);
  r.y = bf16x2_rn(v[2], v[3]);
  r.z = bf16x2_rn(v[4], v[5]);
  r.w = bf16x2_rn(v[6], v[7]);
  *reinterpret_cast<uint4*>(p) = r;
}

// Sixteen bytes to shared memory, in the background.
__device__ __forceinline__ void cp_async_16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src)
               : "memory");
}

// 2^v, a few ulp, 0 for v below the normal range.
__device__ __forceinline__ float exp2_f(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// A log2 e, finite unless A is not a number: a step that does not count has d = 0, and 0 times an
// infinity would not be 0.  (Rates from 2.4e38 on decay to 0 in any step that counts all the same.)
__device__ __forceinline__ float rate_f(float A) {
  constexpr float kMost = 3.402823466e38f;
  const float v = A * 1.4426950408889634f;
  return v < -kMost ? -kMost : v > kMost ? kMost : v;
}

// 2^(d A2), the factor by which a state goes on; 1 where d is 0.  The hardware's 2^v is too small on
// average, by 2e-8 for v in (-1, -0.003) and 6e-9 nearer to 0, and a recurrence adds that up over all
// the steps that a state remembers.  What is added to the exponent, in the product's own multiply-add,
// takes most of that back (1e-8 either way is left, 1.6e-8 at most).  64 x 512 steps x 1024 channels x
// 16 states, errors against 64 bits (2-norm): dA 1.6e-6 without and 8.2e-7 with it, dh0 1.8e-6 and
// 9.1e-7, in the same time (step by step with expf they are 8e-7 and 1.4e-6).  2^2e-8 rounds to 1.
constexpr float kDecayBias = 2e-8f;
__device__ __forceinline__ float decay_f(float d, float A2) { return exp2_f(fmaf(d, A2, kDecayBias)); }
__device__ __forceinline__ float2 decay2_f(float d, float2 A2) {
  const float2 m = fma2(make_float2(d, d), A2, make_float2(kDecayBias, kDecayBias));
  return make_float2(exp2_f(m.x), exp2_f(m.y));
}

// 1 / v, one ulp, and the logistic function from it.  The flush-to-zero forms of the hardware's
// exponential and reciprocal: their subnormal results and arguments (here below 2^-126 of 1)
// would take three more instructions each.
__device__ __forceinline__ float rcp_f(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float sigmoid_f(float v) {
  return rcp_f(1.f + exp2_f(-1.4426950408889634f * v));
}

// ln(1 + e^v) = max(v, 0) + ln(1 + t), t = e^-|v| in (0, 1].  ln(1 + t) = 2 artanh(s) with
// s = t / (2 + t) <= 1/3, which keeps full relative precision for small t, where 1 + t would lose
// it.  artanh(s) / s is a polynomial in s^2 of degree 4, interpolated at the Chebyshev nodes of
// [0, 1/9] (relative error 8e-9, below fp32's rounding; the power series would take degree 7).
// Two values at a time: the polynomial runs in packed pairs.
__device__ __forceinline__ float2 softplus2_f(float2 v) {
  constexpr float kLog2e = 1.4426950408889634f;
  const float2 t = make_float2(exp2_f(-kLog2e * fabsf(v.x)), exp2_f(-kLog2e * fabsf(v.y)));
  const float2 s = __fmul2_rn(t, make_float2(rcp_f(2.f + t.x), rcp_f(2.f + t.y)));
  const float2 q = __fmul2_rn(s, s);
  float2 p = make_float2(0.14078889787197113f, 0.14078889787197113f);
  p = fma2(p, q, make_float2(0.13982579112052917f, 0.13982579112052917f));
  p = fma2(p, q, make_float2(0.20012298226356506f, 0.20012298226356506f));
  p = fma2(p, q, make_float2(0.3333316147327423f, 0.3333316147327423f));
  p = fma2(p, q, make_float2(1.f, 1.f));
  return fma2(__fmul2_rn(s, p), make_float2(2.f, 2.f), make_float2(fmaxf(v.x, 0.f), fmaxf(v.y, 0.f)));
}
__device__ __forceinline__ float softplus_f(float v) { return softplus2_f(make_float2(v, v)).x; }

// Philox 4x32, ten rounds (Salmon, Moraes, Dror, Shaw: "Parallel random numbers: as easy as
// 1, 2, 3", 2011): 128 random bits from a 128-bit counter and a 64-bit key.
__device__ __forceinline__ uint4 philox4x32(uint4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint32_t h0 = __umulhi(c.x, 0xD2511F53u), l0 = c.x * 0xD2511F53u;
    const uint32_t h1 = __umulhi(c.z, 0xCD9E8D57u), l1 = c.z * 0xCD9E8D57u;
    c = make_uint4(h1 ^ c.y ^ k0, l1, h0 ^ c.w ^ k1, l0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return c;
}

// Key and offset of a dropout call, read from its device-side {seed, offset} pair.
struct DropKey {
  uint32_t k0, k1, o0, o1;
};
__device__ __forceinline__ DropKey drop_key(const unsigned long long* rng) {
  const unsigned long long s = rng[0], o = rng[1];
  return {static_cast<uint32_t>(s), static_cast<uint32_t>(s >> 32), static_cast<uint32_t>(o),
          static_cast<uint32_t>(o >> 32)};
}

// Which of the eight columns 8 * group .. 8 * group + 7 of `row` are kept: k[j] where the j-th
// 16-bit piece of the generator's output, lowest first, is >= cut.  Sixteen bits an element hold
// the drop probability to 2^-17 and cost one generator call for eight elements; the scale uses
// the held probability, so the expectation is exact.
__device__ __forceinline__ void keep8(const DropKey& key, uint32_t row, uint32_t group,
                                      uint32_t cut, bool (&k)[8]) {
  const uint4 r = philox4x32(make_uint4(group, row, key.o0, key.o1), key.k0, key.k1);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  const uint32_t high = cut << 16;   // compared against whole words: the low half cannot decide
  const bool any = cut < 65536u;     // everything is dropped otherwise
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    k[2 * i] = any && (w[i] << 16) >= high;
    k[2 * i + 1] = any && w[i] >= high;
  }
}

// f(true or false as a constant): a uniform condition decided once for straight-line code.
template <typename F>
__device__ __forceinline__ void decide(bool c, F&& f) {
  if (c) f(std::true_type{});
  else f(std::false_type{});
}

}  // namespace cfc
