// cfc_merge.cu -- the sum of a few hundred rows of partial sums, in a fixed order: what ends the
// parameter gradients of the gated block's operators.
//
// A CTA takes 32 columns and gives each warp every 32nd row, up to eight loads in flight a lane, so
// that the merge is two trips to memory long and not one for every few rows: 456 rows x 256 columns
// 2.9 us behind the kernel that wrote them, reduce_axis0 5.9 us.  More rows than kMergeRows are
// reduce_axis0's, which spreads them over a cluster.
#include "cfc_gated_kernels.h"
#include "cfc_kernels.h"
#include "cfc_launch.cuh"
#include "cfc_ptx.cuh"

namespace cfc {
namespace {

constexpr int kMergeRows = 2048;

__global__ void __launch_bounds__(1024) merge_kernel(const float* in, int rows, int n, float* out) {
  __shared__ float part[32][33];
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
  grid_dep_wait();
  float v = 0.f;
  if (c < n) {
    const float* p = in + static_cast<size_t>(w) * n + c;
    const size_t step = static_cast<size_t>(32) * n;
    int r = w;
    for (; r + 7 * 32 < rows; r += 8 * 32, p += 8 * step) {
      float a[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = p[i * step];
#pragma unroll
      for (int i = 0; i < 8; ++i) v += a[i];
    }
    float a[8];
#pragma unroll
    for (int i = 0; i < 7; ++i) a[i] = r + i * 32 < rows ? p[i * step] : 0.f;
#pragma unroll
    for (int i = 0; i < 7; ++i) v += a[i];
  }
  part[w][lane] = v;
  __syncthreads();
  v = part[lane][w];  // column w of the tile, row group `lane`
#pragma unroll
  for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xffffffffu, v, d);
  if (lane == 0 && blockIdx.x * 32 + w < n) out[blockIdx.x * 32 + w] = v;
}

}  // namespace

cudaError_t merge_launch(const float* in, int rows, int n, float* out, cudaStream_t s, bool pdl) {
  if (rows > kMergeRows) return reduce_axis0_launch(in, rows, n, out, s, pdl);
  LaunchCfg c;
  c.grid = dim3((n + 31) / 32);
  c.block = dim3(1024);
  c.stream = s;
  c.pdl = pdl;
  return launch(c, merge_kernel, in, rows, n, out);
}

}  // namespace cfc
