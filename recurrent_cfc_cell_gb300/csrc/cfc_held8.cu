// cfc_held8.cu -- activations to 8 bits and back (the form is described in cfc_held8.cuh): what a
// training step keeps for its backward pass, and what an 8-bit row stands for.
//
// Bound by memory: 1 + 1 / 32 bytes an element on one side and the activation on the other.  Eight
// columns to a thread where everything is aligned, otherwise one, so that a warp's accesses are
// consecutive whatever the rows' alignment.  16384 x 2048 bf16: to 8 bits 22.5 us (4.5 TB/s), back
// 18.5 us (5.5 TB/s).
#include "cfc_gated_kernels.h"
#include "cfc_held8.cuh"
#include "cfc_launch.cuh"
#include "cfc_trunk.cuh"

#include <type_traits>

namespace cfc {
namespace {

constexpr int kThreads = 256, kPieces = 4;  // pieces a thread, whose loads are in flight together
constexpr int kTile = kThreads * kPieces;

// Pieces of a row, rounded up to whole blocks: a block's lanes are always of one row.
template <bool VEC>
__host__ __device__ constexpr int pieces(int n) {
  return held_blocks(n) * (VEC ? 4 : kHeldBlock);
}

// Where a thread's pieces of a CTA's tile lie: one 64-bit division a tile, 32-bit ones a piece.
template <bool VEC>
struct Place {
  long long row[kPieces];
  int col[kPieces];
  bool in[kPieces];
  __device__ __forceinline__ Place(const Held8Call& q, long long tile) {
    const unsigned per = pieces<VEC>(q.n);
    const long long base = tile * kTile, row0 = base / per;
    const unsigned from = static_cast<unsigned>(base - row0 * per) + threadIdx.x;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const unsigned at = from + i * kThreads, r = at / per;
      row[i] = row0 + r;
      col[i] = static_cast<int>(at - r * per) * (VEC ? 8 : 1);
      in[i] = row[i] < q.rows && col[i] < q.n;
    }
  }
};

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) pack8_kernel(const Held8Call q, long long tiles) {
  const int n = q.n;
  for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const Place<VEC> at(q, tile);
    std::conditional_t<VEC, Raw8<T>, T> raw[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const T* const x = static_cast<const T*>(q.x) + at.row[i] * q.ldx + at.col[i];
      if constexpr (VEC) {
        if (at.in[i]) raw[i].load(x);
        else raw[i].clear();
      } else {
        raw[i] = at.in[i] ? *x : from_f32<T>(0.f);
      }
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      uint8_t* const codes = q.held.codes + at.row[i] * n + at.col[i];
      uint32_t byte;
      if constexpr (VEC) {
        float v[8];
        raw[i].get(v);
        const uint2 r = held_pack8(v, byte);
        if (at.in[i]) *reinterpret_cast<uint2*>(codes) = r;
      } else {
        const uint32_t r = held_pack1(to_f32(raw[i]), byte);
        if (at.in[i]) *codes = static_cast<uint8_t>(r);
      }
      if (at.in[i] && at.col[i] % kHeldBlock == 0)
        q.held.scales[at.row[i] * held_blocks(n) + at.col[i] / kHeldBlock] =
            static_cast<uint8_t>(byte);
    }
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) unpack8_kernel(const Held8Call q, long long tiles) {
  const int n = q.n;
  for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const Place<VEC> at(q, tile);
    std::conditional_t<VEC, uint2, uint8_t> codes[kPieces];
    uint32_t byte[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      if (!at.in[i]) continue;
      codes[i] = *reinterpret_cast<const decltype(&codes[0])>(q.held.codes + at.row[i] * n +
                                                              at.col[i]);
      byte[i] = q.held.scales[at.row[i] * held_blocks(n) + at.col[i] / kHeldBlock];
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      if (!at.in[i]) continue;
      T* const y = static_cast<T*>(q.y) + at.row[i] * q.ldy + at.col[i];
      if constexpr (VEC) {
        float v[8];
        held_unpack8(codes[i], byte[i], v);
        store8(y, v);
      } else {
        *y = from_f32<T>(held_values2(codes[i]).x * held_up(byte[i]));
      }
    }
  }
}

bool vectors(const Held8Call& q, const void* p, long long ld) {
  return q.n % 8 == 0 && ld % 8 == 0 && reinterpret_cast<uintptr_t>(q.held.codes) % 8 == 0 &&
         reinterpret_cast<uintptr_t>(p) % (q.bf16 ? 16 : 32) == 0;
}

long long tiles_of(const Held8Call& q, bool vec) {
  const long long total =
      static_cast<long long>(vec ? pieces<true>(q.n) : pieces<false>(q.n)) * q.rows;
  return (total - 1) / kTile + 1;
}
LaunchCfg shape(long long tiles, cudaStream_t s) {
  const long long most = 152 * 64;
  LaunchCfg c;
  c.grid = dim3(static_cast<unsigned>(tiles < most ? tiles : most));
  c.block = dim3(kThreads);
  c.stream = s;
  return c;
}

}  // namespace

cudaError_t pack8_launch(const Held8Call& q, cudaStream_t s) {
  const bool vec = vectors(q, q.x, q.ldx);
  const long long tiles = tiles_of(q, vec);
  const LaunchCfg c = shape(tiles, s);
  if (q.bf16)
    return vec ? launch(c, pack8_kernel<__nv_bfloat16, true>, q, tiles)
               : launch(c, pack8_kernel<__nv_bfloat16, false>, q, tiles);
  return vec ? launch(c, pack8_kernel<float, true>, q, tiles) : launch(c, pack8_kernel<float, false>, q, tiles);
}
cudaError_t unpack8_launch(const Held8Call& q, cudaStream_t s) {
  const bool vec = vectors(q, q.y, q.ldy);
  const long long tiles = tiles_of(q, vec);
  const LaunchCfg c = shape(tiles, s);
  if (q.bf16)
    return vec ? launch(c, unpack8_kernel<__nv_bfloat16, true>, q, tiles)
               : launch(c, unpack8_kernel<__nv_bfloat16, false>, q, tiles);
  return vec ? launch(c, unpack8_kernel<float, true>, q, tiles)
             : launch(c, unpack8_kernel<float, false>, q, tiles);
}

}  // namespace cfc
