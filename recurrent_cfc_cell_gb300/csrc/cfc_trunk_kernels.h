// cfc_trunk_kernels.h -- launchers of the trunk operators: layer norm and dropout (cfc_norm.cu), the
// causal convolution (cfc_conv.cu) and the selective scan (cfc_scan_fwd.cu, cfc_scan_bwd.cu).  The
// entry points that check their arguments are in cfc_trunk_abi.cu.
#pragma once
#include <cuda_runtime.h>

#include <cstddef>

namespace cfc {

// Activations are fp32 or bf16 (`bf16`); pointers to them are untyped.

// Layer norm over rows of n columns, with dropout and the residual sum in front of it when `rng`
// is set (x is then the dropped input and s the stream that the norm reads); dropout alone uses
// x, residual and s.
struct NormCall {
  const void *x, *residual, *dy, *ds;
  long long ldx, ldr, lddy, ldds;  // row strides (elements)
  const float *w, *b;
  const unsigned long long* rng;   // {seed, offset}
  unsigned cut;                    // 65536 p, rounded
  float scale, eps;
  int rows, n;
  bool bf16;
  void *s, *y, *dx, *dres;
  long long lds, ldy, lddx, lddr;
  float* stats;                    // [rows][2] mean, rstd
};
size_t norm_ws_floats(int rows, int n);
cudaError_t norm_fwd_launch(const NormCall& q, cudaStream_t s);
cudaError_t norm_bwd_launch(const NormCall& q, float* dw, float* db, float* ws, cudaStream_t s);
cudaError_t dropout_launch(const NormCall& q, cudaStream_t s);

// Causal convolution of W taps (2 to 4); the single-token form uses x (stride x_b), x0 as the
// state, last as the new state, and u.
struct ConvCall {
  int B, K, D, W;
  bool bf16, silu;
  const int* lengths;              // [B] or null
  const void *x, *x0, *du;
  const float *w, *bias;
  void *u, *last, *dx, *dx0;
  long long x_t, x_b, u_t, u_b, du_t, du_b, dx_t, dx_b;  // step and sequence strides (elements)
};
int conv_partials(int B, int K, int D, bool bf16);
cudaError_t conv_fwd_launch(const ConvCall& q, cudaStream_t s);
cudaError_t conv_bwd_launch(const ConvCall& q, float* dw, float* db, float* ws, cudaStream_t s);
cudaError_t conv_step_launch(const ConvCall& q, cudaStream_t s);

// Selective scan.
constexpr int kScanMaxStates = 128;
constexpr int kScanPeriod = 8;     // steps between the states that a training forward keeps
struct ScanCall {
  int B, K, D, N, G;
  bool bf16, softplus;
  const int* lengths;              // [B] or null
  const void *x, *dt, *z, *Bm, *Cm, *dy;
  long long x_t, x_b, dt_t, dt_b, z_t, z_b, Bm_t, Bm_b, Cm_t, Cm_b, dy_t, dy_b;
  const float *A, *skip, *dt_bias, *h0, *dh_last;
  // forward
  void* y;
  long long y_t, y_b;
  float *h_last, *states;          // states: [ceil(K / kScanPeriod)][B][D][N]
  // backward
  void *dx, *ddt, *dz, *dB, *dC;
  long long dx_t, dx_b, ddt_t, ddt_b, dz_t, dz_b;
  float *dA, *dskip, *ddt_bias, *dh0;
  float* ws;
};
size_t scan_fwd_ws_floats(const ScanCall& q);
size_t scan_bwd_ws_floats(const ScanCall& q);
cudaError_t scan_fwd_launch(const ScanCall& q, cudaStream_t s);
cudaError_t scan_bwd_launch(const ScanCall& q, cudaStream_t s);
cudaError_t scan_step_launch(const ScanCall& q, cudaStream_t s);
// Splits of the steps over CTAs (1: none) for a recurrence that takes `ctas` CTAs unsplit, so that
// about `slots` run: at least `least_steps` steps each, and none with fewer than `least_total` steps
// or three splits, which would not pay for the pass that carries the state (or its gradient) over
// the splits.  On return of that pass carry [splits][B][D][N] holds what enters each split.
struct ScanSplit {
  int splits, steps;               // steps per split, a multiple of 2 kScanPeriod
};
ScanSplit scan_split(int K, long long ctas, int slots, int least_steps, int least_total);
size_t scan_carry_floats(const ScanCall& q, const ScanSplit& sp);
cudaError_t scan_carry_launch(const ScanCall& q, const ScanSplit& sp, bool reverse, float* carry,
                              cudaStream_t s);

}  // namespace cfc
