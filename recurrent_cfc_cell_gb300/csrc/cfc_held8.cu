// cfc_held8.cu -- activations to 8 bits and back (the form is described in cfc_held8.cuh): what a
// training step keeps for its backward pass, and what an 8-bit row stands for.
//
// Bound by memory: 1 + 1 / 32 bytes an element on one side and the activation on the other.  Eight
// columns to a thread where everything is aligned, otherwise one, so that a warp's accesses are
// consecutive whatever the rows' alignment.
#include "cfc_gated_kernels.h"
#include "cfc_held8.cuh"
#include "cfc_launch.cuh"
#include "cfc_trunk.cuh"

namespace cfc {
namespace {

constexpr int kThreads = 256;

// Pieces of a row, rounded up to whole blocks: a block's lanes are always of one row.
template <bool VEC>
__host__ __device__ constexpr int pieces(int n) {
  return held_blocks(n) * (VEC ? 4 : kHeldBlock);
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) pack8_kernel(const Held8Call q) {
  const int n = q.n, per = pieces<VEC>(n);
  const long long total = static_cast<long long>(per) * q.rows;
  const long long step = static_cast<long long>(gridDim.x) * kThreads;
  // Whole warps stay together: `total` may end inside one.
  for (long long at = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
       at - threadIdx.x % 32 < total; at += step) {
    const long long row = at / per;
    const int c = static_cast<int>(at - row * per) * (VEC ? 8 : 1);
    const bool in = at < total && c < n;
    const T* const x = static_cast<const T*>(q.x) + row * q.ldx + c;
    uint8_t* const codes = q.held.codes + row * n + c;
    uint32_t byte;
    if constexpr (VEC) {
      Raw8<T> raw;
      if (in) raw.load(x);
      else raw.clear();
      float v[8];
      raw.get(v);
      const uint2 r = held_pack8(v, byte);
      if (in) *reinterpret_cast<uint2*>(codes) = r;
    } else {
      const uint32_t r = held_pack1(in ? to_f32(*x) : 0.f, byte);
      if (in) *codes = static_cast<uint8_t>(r);
    }
    if (in && c % kHeldBlock == 0)
      q.held.scales[row * held_blocks(n) + c / kHeldBlock] = static_cast<uint8_t>(byte);
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) unpack8_kernel(const Held8Call q) {
  const int n = q.n, per = pieces<VEC>(n);
  const long long total = static_cast<long long>(per) * q.rows;
  for (long long at = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; at < total;
       at += static_cast<long long>(gridDim.x) * kThreads) {
    const long long row = at / per;
    const int c = static_cast<int>(at - row * per) * (VEC ? 8 : 1);
    if (c >= n) continue;
    const uint8_t* const codes = q.held.codes + row * n + c;
    const uint32_t byte = q.held.scales[row * held_blocks(n) + c / kHeldBlock];
    T* const y = static_cast<T*>(q.y) + row * q.ldy + c;
    if constexpr (VEC) {
      float v[8];
      held_unpack8(*reinterpret_cast<const uint2*>(codes), byte, v);
      store8(y, v);
    } else {
      *y = from_f32<T>(held_values2(*codes).x * held_up(byte));
    }
  }
}

bool vectors(const Held8Call& q, const void* p, long long ld) {
  return q.n % 8 == 0 && ld % 8 == 0 && reinterpret_cast<uintptr_t>(q.held.codes) % 8 == 0 &&
         reinterpret_cast<uintptr_t>(p) % (q.bf16 ? 16 : 32) == 0;
}

LaunchCfg shape(const Held8Call& q, bool vec, cudaStream_t s) {
  const long long total =
      static_cast<long long>(vec ? pieces<true>(q.n) : pieces<false>(q.n)) * q.rows;
  const long long need = (total + kThreads - 1) / kThreads, most = 152 * 8 * 8;
  LaunchCfg c;
  c.grid = dim3(static_cast<unsigned>(need < most ? need : most));
  c.block = dim3(kThreads);
  c.stream = s;
  return c;
}

}  // namespace

cudaError_t pack8_launch(const Held8Call& q, cudaStream_t s) {
  const bool vec = vectors(q, q.x, q.ldx);
  const LaunchCfg c = shape(q, vec, s);
  if (q.bf16)
    return vec ? launch(c, pack8_kernel<__nv_bfloat16, true>, q)
               : launch(c, pack8_kernel<__nv_bfloat16, false>, q);
  return vec ? launch(c, pack8_kernel<float, true>, q) : launch(c, pack8_kernel<float, false>, q);
}
cudaError_t unpack8_launch(const Held8Call& q, cudaStream_t s) {
  const bool vec = vectors(q, q.y, q.ldy);
  const LaunchCfg c = shape(q, vec, s);
  if (q.bf16)
    return vec ? launch(c, unpack8_kernel<__nv_bfloat16, true>, q)
               : launch(c, unpack8_kernel<__nv_bfloat16, false>, q);
  return vec ? launch(c, unpack8_kernel<float, true>, q)
             : launch(c, unpack8_kernel<float, false>, q);
}

}  // namespace cfc
