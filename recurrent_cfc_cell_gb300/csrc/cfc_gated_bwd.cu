// cfc_gated_bwd.cu -- the gradients of the gated linear recurrence (cfc_gated.cuh says how the steps
// are divided; here the runs follow one another backwards in time).
//
//   g_t = dL/dh_t = dy_t silu(z_t) + f_{t+1} g_{t+1}
//   dx_t = g_t (1 - f_t),   df_t = g_t (h_{t-1} - x_t) f_t (1 - f_t)   (of the logit)
//   dz_t = dy_t h_t silu'(z_t),   dbias = sum df,   dh0 = f_0 g_0
//
// h is formed again within each run from the state that the forward pass kept at its start.
#include "cfc_gated.cuh"
#include "cfc_kernels.h"

namespace cfc {
namespace {

template <typename T, int V, bool KEEP>
struct Input {  // an activation that the backward pass reads as it is, or in 8 bits
  RawV<T, V> raw[kGS];
  __device__ __forceinline__ void load(int k, const T* p, const Held8&, const HeldAt&) {
    raw[k].load(p);
  }
};
template <typename T, int V>
struct Input<T, V, true> {
  RawHeldV<V> raw[kGS];
  __device__ __forceinline__ void load(int k, const T*, const Held8& h, const HeldAt& at) {
    raw[k].load(h, at);
  }
};

template <typename T, int V, bool Z, bool KEEP>
__global__ void __launch_bounds__(32 * kGatedWarps) gated_bwd_kernel(const GatedCall q,
                                                                     float* dbias) {
  __shared__ float2 run[2][kGatedWarps][32 * V];
  const int warps = blockDim.x / 32, w = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int b = blockIdx.y, K = q.K;
  const Channels<V> ch(blockIdx.x, q.D);
  const int len = q.lengths ? min(max(q.lengths[b], 0), K) : K;
  const T* const xp = KEEP ? nullptr : static_cast<const T*>(q.x) + b * q.x_b + ch.d;
  const T* const fp = KEEP ? nullptr : static_cast<const T*>(q.f) + b * q.f_b + ch.d;
  const T* const zp = KEEP || !Z ? nullptr : static_cast<const T*>(q.z) + b * q.z_b + ch.d;
  const T* const dyp = static_cast<const T*>(q.dy) + b * q.dy_b + ch.d;
  T* const dxp = static_cast<T*>(q.dx) + b * q.dx_b + ch.d;
  T* const dfp = static_cast<T*>(q.df) + b * q.df_b + ch.d;
  T* const dzp = Z ? static_cast<T*>(q.dz) + b * q.dz_b + ch.d : nullptr;
  T* const yp = q.y ? static_cast<T*>(q.y) + b * q.y_b + ch.d : nullptr;
  float bias[V], carry[V], dsum[V] = {};
  load_par_v<V>(q.bias, ch, bias);
  load_par_v<V>(q.dh_last ? q.dh_last + static_cast<size_t>(b) * q.D : nullptr, ch, carry);
  const float zero[V] = {};

  int turn = 0;
  const int round = warps * kGS;
  for (int base = (K - 1) / round * round; base >= 0; base -= round, turn ^= 1) {
    const int t0 = base + w * kGS;
    if (base >= len) {
#pragma unroll
      for (int k = 0; k < kGS; ++k) {
        const long long t = t0 + k;
        if (t >= K || !ch.in) continue;
        store_v(dxp + t * q.dx_t, zero);
        store_v(dfp + t * q.df_t, zero);
        if (Z) store_v(dzp + t * q.dz_t, zero);
        if (yp) store_v(yp + t * q.y_t, zero);
      }
      continue;
    }
    Input<T, V, KEEP> x, f, z;
    RawV<T, V> dy[kGS];
    RawV<float, V> start;
#pragma unroll
    for (int k = 0; k < kGS; ++k) {
      const long long t = t0 + k;
      if (t < len && ch.in) {
        const HeldAt at = held_at<V>(q, t0 + k, b, ch.d);
        x.load(k, xp + t * q.x_t, q.x8, at);
        f.load(k, fp + t * q.f_t, q.f8, at);
        if (Z) z.load(k, zp + t * q.z_t, q.z8, at);
        dy[k].load(dyp + t * q.dy_t);
      } else {
        x.raw[k].clear();
        f.raw[k].clear();
        if (Z) z.raw[k].clear();
        dy[k].clear();
      }
    }
    if (t0 < len && ch.in)
      start.load(q.states + (static_cast<size_t>(t0 / kGS) * q.B + b) * q.D + ch.d);
    else
      start.clear();
    float h[V];
    start.get(h);
    float a[kGS][V], i[kGS][V], u[kGS][V], dh[kGS][V];
#pragma unroll
    for (int k = 0; k < kGS; ++k) {
      const bool on = t0 + k < len;
      float xv[V], fv[V], zv[V], dyv[V], dz[V], y[V];
      x.raw[k].get(xv);
      f.raw[k].get(fv);
      if (Z) z.raw[k].get(zv);
      dy[k].get(dyv);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        gates_f(fv[j] + bias[j], a[k][j], i[k][j]);
        u[k][j] = (h[j] - xv[j]) * a[k][j] * i[k][j];
        h[j] = fmaf(a[k][j], h[j], i[k][j] * xv[j]);
        if constexpr (Z) {
          const float sg = sigmoid_f(zv[j]), gate = zv[j] * sg;
          dh[k][j] = dyv[j] * gate;
          dz[j] = dyv[j] * h[j] * fmaf(gate, 1.f - sg, sg);
          y[j] = h[j] * gate;
        } else {
          dh[k][j] = dyv[j];
          y[j] = h[j];
        }
        if (!on) {
          a[k][j] = 1.f;
          i[k][j] = u[k][j] = dh[k][j] = dz[j] = y[j] = 0.f;
        }
      }
      if (t0 + k < K && ch.in) {
        if (Z) store_v(dzp + static_cast<long long>(t0 + k) * q.dz_t, dz);
        if (yp) store_v(yp + static_cast<long long>(t0 + k) * q.y_t, y);
      }
    }
    // What leaves a run backwards: A carry + H, with carry = f_t g_t of the step after it.
    float A[V], H[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      A[j] = 1.f, H[j] = 0.f;
#pragma unroll
      for (int k = kGS - 1; k >= 0; --k) {
        H[j] = a[k][j] * (dh[k][j] + H[j]);
        A[j] *= a[k][j];
      }
      run[turn][w][lane * V + j] = make_float2(A[j], H[j]);
    }
    __syncthreads();
    float g[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float v = carry[j];
      for (int n = warps - 1; n >= 0; --n) {
        if (n == w) g[j] = v;
        const float2 r = run[turn][n][lane * V + j];
        v = fmaf(r.x, v, r.y);
      }
      carry[j] = v;
    }
#pragma unroll
    for (int k = kGS - 1; k >= 0; --k) {
      float dx[V], df[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        g[j] += dh[k][j];
        dx[j] = g[j] * i[k][j];
        df[j] = g[j] * u[k][j];
        dsum[j] += df[j];
        g[j] *= a[k][j];
      }
      if (t0 + k < K && ch.in) {
        store_v(dxp + static_cast<long long>(t0 + k) * q.dx_t, dx);
        store_v(dfp + static_cast<long long>(t0 + k) * q.df_t, df);
      }
    }
  }
  if (q.dh0 && w == 0 && ch.in) store_v(q.dh0 + static_cast<size_t>(b) * q.D + ch.d, carry);
  if (!dbias) return;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < V; ++j) run[0][w][lane * V + j].x = dsum[j];
  __syncthreads();
  if (w == 0 && ch.in) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float v = 0.f;
      for (int n = 0; n < warps; ++n) v += run[0][n][lane * V + j].x;
      dbias[static_cast<size_t>(b) * q.D + ch.d + j] = v;
    }
  }
}

bool pair(const void* p, long long t, long long b, bool bf16) {
  return !p || (reinterpret_cast<uintptr_t>(p) % (bf16 ? 4 : 8) == 0 && t % 2 == 0 && b % 2 == 0);
}
bool pair32(const float* p) { return reinterpret_cast<uintptr_t>(p) % 8 == 0; }
bool pair8(const Held8& h) { return reinterpret_cast<uintptr_t>(h.codes) % 2 == 0; }
bool pairs(const GatedCall& q) {
  return q.D % 2 == 0 && pair(q.x, q.x_t, q.x_b, q.bf16) && pair(q.f, q.f_t, q.f_b, q.bf16) &&
         pair(q.z, q.z_t, q.z_b, q.bf16) && pair(q.y, q.y_t, q.y_b, q.bf16) &&
         pair(q.dy, q.dy_t, q.dy_b, q.bf16) && pair(q.dx, q.dx_t, q.dx_b, q.bf16) &&
         pair(q.df, q.df_t, q.df_b, q.bf16) && pair(q.dz, q.dz_t, q.dz_b, q.bf16) &&
         pair32(q.states) && pair32(q.dh0) && pair8(q.x8) && pair8(q.f8) && pair8(q.z8);
}

template <typename T, int V, bool Z, bool KEEP>
cudaError_t bwd(const GatedCall& q, cudaStream_t s) {
  const int runs = (q.K + kGS - 1) / kGS;
  LaunchCfg c;
  c.grid = dim3((q.D + 32 * V - 1) / (32 * V), q.B);
  c.block = dim3(32 * (runs < kGatedWarps ? runs : kGatedWarps));
  c.stream = s;
  float* const first = q.dbias && q.B > 1 ? q.ws : q.dbias;
  const cudaError_t e = launch(c, gated_bwd_kernel<T, V, Z, KEEP>, q, first);
  if (e != cudaSuccess || first == q.dbias) return e;
  return reduce_axis0_launch(q.ws, q.B, q.D, q.dbias, s, false);
}
template <typename T, int V>
cudaError_t bwd_v(const GatedCall& q, cudaStream_t s) {
  if (q.keep)
    return q.has_z ? bwd<T, V, true, true>(q, s) : bwd<T, V, false, true>(q, s);
  return q.has_z ? bwd<T, V, true, false>(q, s) : bwd<T, V, false, false>(q, s);
}
template <typename T>
cudaError_t bwd_t(const GatedCall& q, cudaStream_t s) {
  return pairs(q) ? bwd_v<T, 2>(q, s) : bwd_v<T, 1>(q, s);
}

}  // namespace

size_t gated_ws_floats(int B, int, int D, bool) {
  return B > 1 ? static_cast<size_t>(B) * D : 0;
}
cudaError_t gated_bwd_launch(const GatedCall& q, cudaStream_t s) {
  return q.bf16 ? bwd_t<__nv_bfloat16>(q, s) : bwd_t<float>(q, s);
}

}  // namespace cfc
