// cfc_gated.cuh -- what the passes of the gated linear recurrence share.
//
//   f_t = sigmoid(f_t + bias),   h_t = f_t h_{t-1} + (1 - f_t) x_t,   y_t = h_t silu(z_t)
//
// A warp takes kGatedPeriod steps of 32 V neighbouring channels (V = 2, or 1 where channels are not
// aligned in pairs) of one sequence.  A composition of steps is again one: over a run of them
// h_out = A h_in + H with A = prod f and H the state that the run reaches from 0.  So the warps of
// a cluster take runs one after another in time, each forms its A and H at once, and what enters a
// run is folded from those of the runs before it: K / (steps of a cluster) rounds with an exchange
// each take the place of K steps one after another, and every input is read once.
#pragma once
#include "cfc_gated_kernels.h"
#include "cfc_held8.cuh"
#include "cfc_launch.cuh"
#include "cfc_trunk.cuh"

namespace cfc {

constexpr int kGS = kGatedPeriod;      // steps of a run
constexpr int kGatedWarps = 16;        // most runs of a CTA

// f = sigmoid(v) and i = 1 - f = sigmoid(-v), both to full relative precision: with e = e^-|v| the
// smaller of the two is e / (1 + e) and the larger is 1 minus it, which is rounded to nearest, so
// that a long product of f does not drift with an error of the reciprocal.
__device__ __forceinline__ void gates_f(float v, float& f, float& i) {
  const float e = exp2_f(-1.4426950408889634f * fabsf(v));
  const float small = e * rcp_f(1.f + e), large = 1.f - small;
  f = v < 0.f ? small : large;
  i = v < 0.f ? large : small;
}

// V channels of one step as they are stored.
template <typename T, int V>
struct RawV;
template <>
struct RawV<float, 1> {
  float v;
  __device__ __forceinline__ void load(const float* p) { v = *p; }
  __device__ __forceinline__ void clear() { v = 0.f; }
  __device__ __forceinline__ void get(float (&o)[1]) const { o[0] = v; }
};
template <>
struct RawV<float, 2> {
  float2 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float2*>(p); }
  __device__ __forceinline__ void clear() { v = make_float2(0.f, 0.f); }
  __device__ __forceinline__ void get(float (&o)[2]) const { o[0] = v.x; o[1] = v.y; }
};
template <>
struct RawV<__nv_bfloat16, 1> {
  unsigned short v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    v = *reinterpret_cast<const unsigned short*>(p);
  }
  __device__ __forceinline__ void clear() { v = 0; }
  __device__ __forceinline__ void get(float (&o)[1]) const {
    o[0] = __uint_as_float(static_cast<uint32_t>(v) << 16);
  }
};
template <>
struct RawV<__nv_bfloat16, 2> {
  uint32_t v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    v = *reinterpret_cast<const uint32_t*>(p);
  }
  __device__ __forceinline__ void clear() { v = 0u; }
  __device__ __forceinline__ void get(float (&o)[2]) const {
    o[0] = bf16_lo_f32(v);
    o[1] = bf16_hi_f32(v);
  }
};
__device__ __forceinline__ void store_v(float* p, const float (&v)[1]) { *p = v[0]; }
__device__ __forceinline__ void store_v(float* p, const float (&v)[2]) {
  *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
}
__device__ __forceinline__ void store_v(__nv_bfloat16* p, const float (&v)[1]) {
  *p = __float2bfloat16_rn(v[0]);
}
__device__ __forceinline__ void store_v(__nv_bfloat16* p, const float (&v)[2]) {
  *reinterpret_cast<uint32_t*>(p) = bf16x2_rn(v[0], v[1]);
}

// A lane's place: its channels and which of them exist.
template <int V>
struct Channels {
  int d;       // first channel
  bool in;     // it exists (V = 2: D is even, so both do)
  __device__ __forceinline__ Channels(int tile, int D)
      : d((tile * 32 + static_cast<int>(threadIdx.x) % 32) * V), in(d < D) {}
};

template <int V>
__device__ __forceinline__ void load_par_v(const float* p, const Channels<V>& c, float (&v)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = p && c.in ? __ldg(p + c.d + j) : 0.f;
}

// Where the element (step, sequence, channel) of an [K][B][D] tensor held in 8 bits lies.
struct HeldAt {
  size_t code, scale;
};
template <int V>
__device__ __forceinline__ HeldAt held_at(const GatedCall& q, int t, int b, int d) {
  const size_t row = static_cast<size_t>(t) * q.B + b;
  return {row * q.D + d, row * held_blocks(q.D) + d / kHeldBlock};
}
// V channels a lane to 8 bits: a block is 32 / V lanes.
template <int V>
__device__ __forceinline__ void store_held_v(const Held8& h, const HeldAt& at, const float (&v)[V],
                                             bool in) {
  uint32_t byte, codes;
  if constexpr (V == 1) {
    codes = held_pack1(v[0], byte);
    if (in) h.codes[at.code] = static_cast<uint8_t>(codes);
  } else {
    uint32_t most = max(magnitude_bits(v[0]), magnitude_bits(v[1]));
#pragma unroll
    for (int d = 1; d < 16; d *= 2) most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
    byte = held_scale_byte(most);
    const float down = held_down(byte);
    codes = held_codes2(v[0] * down, v[1] * down);
    if (in) *reinterpret_cast<uint16_t*>(h.codes + at.code) = static_cast<uint16_t>(codes);
  }
  if (in && threadIdx.x % (32 / V) == 0) h.scales[at.scale] = static_cast<uint8_t>(byte);
}

// V channels of one step in 8 bits, as they are stored.
template <int V>
struct RawHeldV {
  uint16_t codes;
  uint8_t byte;
  __device__ __forceinline__ void load(const Held8& h, const HeldAt& at) {
    codes = V == 1 ? h.codes[at.code] : *reinterpret_cast<const uint16_t*>(h.codes + at.code);
    byte = h.scales[at.scale];
  }
  __device__ __forceinline__ void clear() { codes = 0; byte = 1; }
  __device__ __forceinline__ void get(float (&o)[V]) const {
    const float2 p = held_values2(codes);
    const float up = held_up(byte);
    o[0] = p.x * up;
    if constexpr (V == 2) o[1] = p.y * up;
  }
};

}  // namespace cfc
