// cfc_held8.cuh -- values held in 8 bits: e4m3 codes in blocks of 32 columns of a row, each block
// with a power-of-two scale in one byte (e8m0: 2^(byte - 127)), the layout of the OCP microscaling
// formats.  The scale is the smallest power of two that brings the block's largest magnitude to
// 448, e4m3's largest, or below, so that nothing is cut off and every value is off by at most half
// a step of e4m3 (2^-4 of it, or 2^-10 of the scale where it is small).  A power of two costs no
// rounding of its own: v / 2^k and code * 2^k are exact, and what is held fits bf16 as well.  A
// block with an infinity or a NaN is held as NaN throughout (byte 255).
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "cfc_ptx.cuh"
#include "cfc_trunk.cuh"

namespace cfc {

constexpr int kHeldBlock = 32;
__host__ __device__ constexpr int held_blocks(int n) { return (n + kHeldBlock - 1) / kHeldBlock; }

// |v| as an integer: ordered as the magnitudes are, infinity and NaN above every number.
__device__ __forceinline__ uint32_t magnitude_bits(float v) {
  return __float_as_uint(v) & 0x7fffffffu;
}

// The scale's byte from a block's largest magnitude (its bits): max |v| = m 2^e with m in [1, 2)
// and 448 = 1.75 * 2^8, so k is e - 8 for m <= 1.75 and e - 7 above; adding 0x1fffff to the bits
// carries into the exponent exactly there.  At least 1 (2^-126), so that 2^-k is finite; 255 for
// infinities and NaN.
__device__ __forceinline__ uint32_t held_scale_byte(uint32_t most) {
  const int k = static_cast<int>((most + 0x1fffffu) >> 23) - 8;
  return most >= 0x7f800000u ? 255u : static_cast<uint32_t>(max(k, 1));
}
// 2^-k, which the values are multiplied with before they are rounded (NaN for byte 255).
__device__ __forceinline__ float held_down(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7fffffffu : (254u - byte) << 23);
}
// 2^k, which the codes are multiplied with (NaN for byte 255; byte 0, which is never written
// here, is 2^-127).
__device__ __forceinline__ float held_up(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7fffffffu : byte == 0u ? 0x00400000u : byte << 23);
}

// Two scaled values to codes, the first one in the low byte; rounded to nearest even.
__device__ __forceinline__ uint32_t held_codes2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
// Two codes (low byte first) as fp32; exact.
__device__ __forceinline__ float2 held_values2(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes)));
  float2 v;
  asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %2;\ncvt.f32.f16 %0, lo;\ncvt.f32.f16 %1, hi;\n}"
      : "=f"(v.x), "=f"(v.y)
      : "r"(h));
  return v;
}

// Eight columns of a block by each of four neighbouring lanes (all of the warp call): codes and,
// in every one of the four, the scale's byte.  Columns that do not exist hold 0.
__device__ __forceinline__ uint2 held_pack8(const float (&v)[8], uint32_t& byte) {
  uint32_t most = 0u;
#pragma unroll
  for (int j = 0; j < 8; ++j) most = max(most, magnitude_bits(v[j]));
  most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
  most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
  byte = held_scale_byte(most);
  const float down = held_down(byte);
  uint2 r;
  r.x = held_codes2(v[0] * down, v[1] * down) | held_codes2(v[2] * down, v[3] * down) << 16;
  r.y = held_codes2(v[4] * down, v[5] * down) | held_codes2(v[6] * down, v[7] * down) << 16;
  return r;
}
// One column of a block by each lane of a warp.
__device__ __forceinline__ uint32_t held_pack1(float v, uint32_t& byte) {
  byte = held_scale_byte(__reduce_max_sync(0xffffffffu, magnitude_bits(v)));
  return held_codes2(v * held_down(byte), 0.f) & 0xffu;
}

__device__ __forceinline__ void held_unpack8(uint2 codes, uint32_t byte, float (&v)[8]) {
  const float up = held_up(byte);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t w = j < 2 ? codes.x : codes.y;
    const float2 p = held_values2((w >> (16 * (j % 2))) & 0xffffu);
    v[2 * j] = p.x * up;
    v[2 * j + 1] = p.y * up;
  }
}

}  // namespace cfc
