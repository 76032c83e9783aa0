// cfc_gated_kernels.h -- launchers of the gated block's operators: root-mean-square norm
// (cfc_rmsnorm.cu), values held in 8 bits (cfc_held8.cu), the gated linear recurrence
// (cfc_gated_fwd.cu, cfc_gated_bwd.cu) and products with 4-bit weights (cfc_weights4.cu).  The
// entry points that check their arguments are in cfc_gated_abi.cu.
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace cfc {

// Activations are fp32 or bf16 (`bf16`); pointers to them are untyped.

// Rows held in 8 bits: codes [rows][n], scales [rows][ceil(n / 32)].
struct Held8 {
  uint8_t *codes, *scales;
};

// out[n] <- the sum of `rows` rows of n partial sums (cfc_merge.cu); `pdl`: as a dependent launch.
cudaError_t merge_launch(const float* in, int rows, int n, float* out, cudaStream_t s, bool pdl);

struct RmsCall {
  const void *x, *residual, *dy, *ds;  // backward: x is the stream s (null: s8 is read)
  long long ldx, ldr, lddy, ldds;
  const float* w;
  float eps;
  int rows, n;
  bool bf16;
  void *s, *y, *dx;                    // backward: y is formed again (or null)
  long long lds, ldy, lddx;
  Held8 y8, s8;
  float* rstd;                         // [rows]
};
size_t rms_ws_floats(int rows, int n);
cudaError_t rms_fwd_launch(const RmsCall& q, cudaStream_t s);
cudaError_t rms_bwd_launch(const RmsCall& q, float* dw, float* ws, cudaStream_t s);

struct Held8Call {
  const void* x;
  void* y;
  long long ldx, ldy;
  int rows, n;
  bool bf16;
  Held8 held;
};
cudaError_t pack8_launch(const Held8Call& q, cudaStream_t s);
cudaError_t unpack8_launch(const Held8Call& q, cudaStream_t s);

constexpr int kGatedPeriod = 8;        // steps between the states that a training forward keeps
struct GatedCall {
  int B, K, D;
  bool bf16, has_z, keep;
  const int* lengths;                  // [B] or null
  const void *x, *f, *z, *dy;
  long long x_t, x_b, f_t, f_b, z_t, z_b, dy_t, dy_b;
  const float *bias, *h0, *dh_last;
  Held8 x8, f8, z8;                    // `keep`: written by the forward, read by the backward pass
  // forward; y also the backward pass's (formed again, or null)
  void* y;
  long long y_t, y_b;
  float *h_last, *states;              // states: [ceil(K / kGatedPeriod)][B][D]
  // backward
  void *dx, *df, *dz;
  long long dx_t, dx_b, df_t, df_b, dz_t, dz_b;
  float *dbias, *dh0, *ws;
};
// Workspace: what the launches over segments share (forward and backward), and behind it the partial
// sums of dbias (backward).
size_t gated_segments_floats(int B, int K, int D, bool backward);
size_t gated_partials_floats(int B, int K, int D);
cudaError_t gated_fwd_launch(const GatedCall& q, cudaStream_t s);
cudaError_t gated_bwd_launch(const GatedCall& q, cudaStream_t s);
cudaError_t gated_step_launch(const GatedCall& q, cudaStream_t s);

struct Weights4Call {
  int M, N, K, group;
  bool bf16;
  const void* x;                       // activations [M][K], or the weights to quantize [N][K]
  long long ldx, ldy;
  const uint8_t* codes;                // [N][ceil(K / 2)]
  const uint16_t* scales;              // [N][ceil(K / group)] bf16
  uint8_t* codes_out;
  uint16_t* scales_out;
  uint8_t* laid_out;
  const uint8_t* weights;              // laid out
  void* y;                             // [M][N]
};
size_t weights4_bytes(int N, int K, int group);
cudaError_t weights4_quantize_launch(const Weights4Call& q, cudaStream_t s);
cudaError_t weights4_lay_out_launch(const Weights4Call& q, cudaStream_t s);
cudaError_t weights4_matvec_launch(const Weights4Call& q, cudaStream_t s);

}  // namespace cfc
