// cfc_gated_fwd.cu -- the gated linear recurrence, forward and for single tokens (cfc_gated.cuh says
// how the steps are divided).
#include "cfc_gated.cuh"

namespace cfc {
namespace {

// A CTA: up to kGatedWarps runs of one sequence's steps, 32 V channels.  Grid (tiles, B).
template <typename T, int V, bool Z, bool KEEP>
__global__ void __launch_bounds__(32 * kGatedWarps) gated_fwd_kernel(const GatedCall q) {
  // Each run's A and H, two rounds in turn.
  __shared__ float2 run[2][kGatedWarps][32 * V];
  const int warps = blockDim.x / 32, w = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int b = blockIdx.y, K = q.K;
  const Channels<V> ch(blockIdx.x, q.D);
  const int len = q.lengths ? min(max(q.lengths[b], 0), K) : K;
  const T* const xp = static_cast<const T*>(q.x) + b * q.x_b + ch.d;
  const T* const fp = static_cast<const T*>(q.f) + b * q.f_b + ch.d;
  const T* const zp = Z ? static_cast<const T*>(q.z) + b * q.z_b + ch.d : nullptr;
  T* const yp = static_cast<T*>(q.y) + b * q.y_b + ch.d;
  float bias[V], h_in[V];
  load_par_v<V>(q.bias, ch, bias);
  load_par_v<V>(q.h0 ? q.h0 + static_cast<size_t>(b) * q.D : nullptr, ch, h_in);
  const float zero[V] = {};

  int turn = 0;
  for (int base = 0; base < K; base += warps * kGS, turn ^= 1) {
    const int t0 = base + w * kGS;
    if (base >= len) {  // the sequence has ended, for the whole CTA
#pragma unroll
      for (int k = 0; k < kGS; ++k)
        if (t0 + k < K && ch.in) store_v(yp + (t0 + k) * q.y_t, zero);
      continue;
    }
    RawV<T, V> x[kGS], f[kGS], z[kGS];
#pragma unroll
    for (int k = 0; k < kGS; ++k) {
      const long long t = t0 + k;
      const bool on = t < len && ch.in;
      if (on) {
        x[k].load(xp + t * q.x_t);
        f[k].load(fp + t * q.f_t);
        if (Z) z[k].load(zp + t * q.z_t);
      } else {
        x[k].clear();
        f[k].clear();
        if (Z) z[k].clear();
      }
    }
    float a[kGS][V], c[kGS][V], A[V], H[V];
#pragma unroll
    for (int j = 0; j < V; ++j) A[j] = 1.f, H[j] = 0.f;
#pragma unroll
    for (int k = 0; k < kGS; ++k) {
      const bool on = t0 + k < len;
      float xv[V], fv[V];
      x[k].get(xv);
      f[k].get(fv);
      if constexpr (KEEP) {
        if (on) {
          const HeldAt at = held_at<V>(q, t0 + k, b, ch.d);
          store_held_v<V>(q.x8, at, xv, ch.in);
          store_held_v<V>(q.f8, at, fv, ch.in);
          if (Z) {
            float zv[V];
            z[k].get(zv);
            store_held_v<V>(q.z8, at, zv, ch.in);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float i;
        gates_f(fv[j] + bias[j], a[k][j], i);
        c[k][j] = i * xv[j];
        if (!on) a[k][j] = 1.f, c[k][j] = 0.f;
        H[j] = fmaf(a[k][j], H[j], c[k][j]);
        A[j] *= a[k][j];
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) run[turn][w][lane * V + j] = make_float2(A[j], H[j]);
    __syncthreads();
    float h[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float v = h_in[j];
      for (int i = 0; i < warps; ++i) {
        if (i == w) h[j] = v;
        const float2 r = run[turn][i][lane * V + j];
        v = fmaf(r.x, v, r.y);
      }
      h_in[j] = v;
    }
    if (q.states && t0 < K && ch.in)
      store_v(q.states + (static_cast<size_t>(t0 / kGS) * q.B + b) * q.D + ch.d, h);
#pragma unroll
    for (int k = 0; k < kGS; ++k) {
      float zv[V], y[V];
      if (Z) z[k].get(zv);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        h[j] = fmaf(a[k][j], h[j], c[k][j]);
        y[j] = Z ? h[j] * (zv[j] * sigmoid_f(zv[j])) : h[j];
        if (t0 + k >= len) y[j] = 0.f;
      }
      if (t0 + k < K && ch.in) store_v(yp + (t0 + k) * q.y_t, y);
    }
  }
  if (q.h_last && w == 0 && ch.in) store_v(q.h_last + static_cast<size_t>(b) * q.D + ch.d, h_in);
}

// One step for every sequence, V channels a thread.
template <typename T, int V>
__global__ void __launch_bounds__(256) gated_step_kernel(const GatedCall q) {
  const int per = q.D / V;
  const long long at = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  const long long b = at / per;
  if (b >= q.B) return;
  const int d = static_cast<int>(at - b * per) * V;
  RawV<T, V> rx, rf, rz;
  RawV<float, V> rh;
  rx.load(static_cast<const T*>(q.x) + b * q.x_b + d);
  rf.load(static_cast<const T*>(q.f) + b * q.f_b + d);
  if (q.z) rz.load(static_cast<const T*>(q.z) + b * q.z_b + d);
  rh.load(q.h0 + b * q.D + d);
  float x[V], f[V], z[V], h[V], y[V];
  rx.get(x);
  rf.get(f);
  rh.get(h);
  if (q.z) rz.get(z);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    float a, i;
    gates_f(f[j] + (q.bias ? __ldg(q.bias + d + j) : 0.f), a, i);
    h[j] = fmaf(a, h[j], i * x[j]);
    y[j] = q.z ? h[j] * (z[j] * sigmoid_f(z[j])) : h[j];
  }
  store_v(q.h_last + b * q.D + d, h);
  store_v(static_cast<T*>(q.y) + b * q.y_b + d, y);
}

bool pair(const void* p, long long t, long long b, bool bf16) {
  return !p || (reinterpret_cast<uintptr_t>(p) % (bf16 ? 4 : 8) == 0 && t % 2 == 0 && b % 2 == 0);
}
bool pair32(const float* p) { return reinterpret_cast<uintptr_t>(p) % 8 == 0; }
bool pair8(const Held8& h) { return reinterpret_cast<uintptr_t>(h.codes) % 2 == 0; }
// Channels of all tensors are aligned in pairs.
bool pairs(const GatedCall& q) {
  return q.D % 2 == 0 && pair(q.x, q.x_t, q.x_b, q.bf16) && pair(q.f, q.f_t, q.f_b, q.bf16) &&
         pair(q.z, q.z_t, q.z_b, q.bf16) && pair(q.y, q.y_t, q.y_b, q.bf16) && pair32(q.h0) &&
         pair32(q.h_last) && pair32(q.states) && pair8(q.x8) && pair8(q.f8) && pair8(q.z8);
}

template <typename T, int V, bool Z, bool KEEP>
cudaError_t fwd(const GatedCall& q, cudaStream_t s) {
  const int runs = (q.K + kGS - 1) / kGS;
  LaunchCfg c;
  c.grid = dim3((q.D + 32 * V - 1) / (32 * V), q.B);
  c.block = dim3(32 * (runs < kGatedWarps ? runs : kGatedWarps));
  c.stream = s;
  return launch(c, gated_fwd_kernel<T, V, Z, KEEP>, q);
}
template <typename T, int V>
cudaError_t fwd_v(const GatedCall& q, cudaStream_t s) {
  if (q.keep)
    return q.has_z ? fwd<T, V, true, true>(q, s) : fwd<T, V, false, true>(q, s);
  return q.has_z ? fwd<T, V, true, false>(q, s) : fwd<T, V, false, false>(q, s);
}
template <typename T>
cudaError_t fwd_t(const GatedCall& q, cudaStream_t s) {
  return pairs(q) ? fwd_v<T, 2>(q, s) : fwd_v<T, 1>(q, s);
}
template <typename T>
cudaError_t step_t(const GatedCall& q, cudaStream_t s) {
  LaunchCfg c;
  const bool two = pairs(q);
  const long long total = static_cast<long long>(q.B) * (q.D / (two ? 2 : 1));
  c.grid = dim3(static_cast<unsigned>((total + 255) / 256));
  c.block = dim3(256);
  c.stream = s;
  return two ? launch(c, gated_step_kernel<T, 2>, q) : launch(c, gated_step_kernel<T, 1>, q);
}

}  // namespace

cudaError_t gated_fwd_launch(const GatedCall& q, cudaStream_t s) {
  return q.bf16 ? fwd_t<__nv_bfloat16>(q, s) : fwd_t<float>(q, s);
}
cudaError_t gated_step_launch(const GatedCall& q, cudaStream_t s) {
  return q.bf16 ? step_t<__nv_bfloat16>(q, s) : step_t<float>(q, s);
}

}  // namespace cfc
