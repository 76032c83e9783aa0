// cfc_conv.cu -- the short causal convolution in front of the selective scan: one filter of W
// taps per channel over the steps of each sequence, a bias and (optionally) SiLU.
//
//   forward   p_t = bias + sum_j w[j] x_{t-(W-1)+j},  u_t = p_t sigmoid(p_t)
//   backward  g_t = du_t s (1 + p_t (1 - s)), s = sigmoid(p_t)   (p_t formed again from x)
//             dx_t = sum_j w[j] g_{t+(W-1)-j},  dw[j] = sum_{t,b} g_t x_{t-(W-1)+j},
//             dbias = sum_{t,b} g_t
//
// x before the sequence's first step comes from a carried history of W-1 inputs (zero without
// one); a sequence of length L < K ends at L, its later outputs and gradients are 0 and its
// last history is the one before L.
//
// Bound by memory: x is read and u written once (backward: x and du read, dx written), up to
// W - 1 steps read again where two runs of steps meet.  A thread holds neighbouring channels
// (8 bytes of them; with 16 the backward pass's windows and sums would not fit in registers) and
// walks a run of steps with the last W inputs in registers; runs are short where there are few
// channels and sequences, so that the GPU is full, and long otherwise.  The parameter gradients are
// summed in registers over the run, over the CTA's eight runs in shared memory and over the CTAs by
// reduce_axis0.
//
// Measured on GB300: 64 sequences of up to 1023 steps, 1536 channels, bf16, 4 taps, lengths spread
// evenly over 0 .. 1023, so that half the steps are read and all are written: forward 66 us (4.6 TB/s),
// which waits for memory, backward 121 us (3.3 TB/s), whose first stall is the barrier before its sums
// (2.0 of 7 cycles an instruction; memory 1.1, DRAM 38% busy): a CTA's runs are eight in a row of one
// sequence, and those past its end hold their registers until the longest is done.  Four steps' loads
// go out while the four before them are computed (backward 123 us; without, 144 us).  One token of
// 1024 sequences of 2048 channels 10.4 us for 33.5 MB (5 us): each lane reads its taps, once for four
// sequences, one by one (36 us with a read for every sequence).
#include "cfc_kernels.h"
#include "cfc_launch.cuh"
#include "cfc_trunk.cuh"
#include "cfc_trunk_kernels.h"

namespace cfc {
namespace {

constexpr int kLanes = 32;  // channel vectors of a CTA
constexpr int kRuns = 8;    // runs of steps of a CTA
constexpr int kTokens = 4;  // sequences of a thread in the single-token form

// V neighbouring channels: 8 bytes of them (bf16 V = 4, fp32 V = 2), or one.
template <typename T, int V>
struct Raw;
template <typename T>
struct Raw<T, 1> {
  T v;
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = to_f32(v); }
};
template <>
struct Raw<float, 2> {
  float2 v;
  __device__ __forceinline__ void get(float (&f)[2]) const { f[0] = v.x; f[1] = v.y; }
};
template <>
struct Raw<__nv_bfloat16, 4> {
  uint2 v;
  __device__ __forceinline__ void get(float (&f)[4]) const {
    f[0] = bf16_lo_f32(v.x); f[1] = bf16_hi_f32(v.x);
    f[2] = bf16_lo_f32(v.y); f[3] = bf16_hi_f32(v.y);
  }
};
template <typename T, int V>
__device__ __forceinline__ void store_v(T* p, const float (&v)[V]) {
  if constexpr (V == 1) {
    *p = from_f32<T>(v[0]);
  } else if constexpr (V == 2) {
    *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
  } else {
    *reinterpret_cast<uint2*>(p) = make_uint2(bf16x2_rn(v[0], v[1]), bf16x2_rn(v[2], v[3]));
  }
}

struct ConvArgs {
  ConvCall q;
  int run;   // steps of a run
  float *pw, *pb;
};

// The taps and bias of channels c .. c + V - 1.
template <int V, int W>
struct Taps {
  float w[W][V], bias[V];
  __device__ __forceinline__ Taps(const ConvCall& q, int c) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      bias[v] = q.bias ? q.bias[c + v] : 0.f;
#pragma unroll
      for (int j = 0; j < W; ++j) w[j][v] = q.w[static_cast<long long>(c + v) * W + j];
    }
  }
  __device__ __forceinline__ float pre(const float (&x)[W][V], int v) const {
    float p = bias[v];
#pragma unroll
    for (int j = 0; j < W; ++j) p = fmaf(w[j][v], x[j][v], p);
    return p;
  }
};

template <int V, int W>
__device__ __forceinline__ void shift(float (&x)[W][V]) {
#pragma unroll
  for (int j = 0; j + 1 < W; ++j)
#pragma unroll
    for (int v = 0; v < V; ++v) x[j][v] = x[j + 1][v];
}

// x_t of sequence b before step 0 (the history), channels c .. c + V - 1, or of step t.
template <typename T, int V, int W>
__device__ __forceinline__ void load_x(const ConvCall& q, int t, int b, int c, float (&v)[V]) {
  Raw<T, V> r{};
  if (t >= 0)
    r = *reinterpret_cast<const Raw<T, V>*>(static_cast<const T*>(q.x) + t * q.x_t + b * q.x_b + c);
  else if (q.x0 != nullptr && t >= -(W - 1))
    r = *reinterpret_cast<const Raw<T, V>*>(
        static_cast<const T*>(q.x0) + (static_cast<long long>(b) * (W - 1) + t + W - 1) * q.D + c);
  r.get(v);
}

constexpr int kU = 4;  // steps whose loads are issued together

template <typename T, int V, int W>
__global__ void __launch_bounds__(kLanes * kRuns, 4) conv_fwd_kernel(const ConvArgs a) {
  const ConvCall& q = a.q;
  const int c = (blockIdx.x * kLanes + threadIdx.x % kLanes) * V;
  if (c >= q.D) return;
  const int b = blockIdx.y;
  const int len = q.lengths ? min(max(q.lengths[b], 0), q.K) : q.K;
  const int t0 = (blockIdx.z * kRuns + threadIdx.x / kLanes) * a.run;
  const int t1 = min(q.K, t0 + a.run);
  if (t0 == 0 && q.last != nullptr) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      float h[V];
      load_x<T, V, W>(q, len - (W - 1) + j, b, c, h);
      store_v<T, V>(static_cast<T*>(q.last) + (static_cast<long long>(b) * (W - 1) + j) * q.D + c, h);
    }
  }
  if (t0 >= q.K) return;
  T* u = static_cast<T*>(q.u) + b * q.u_b + c;
  const int te = min(t1, len);
  if (t0 < te) {
    const T* x = static_cast<const T*>(q.x) + b * q.x_b + c;
    const Taps<V, W> taps(q, c);
    float win[W][V];  // the last W inputs
#pragma unroll
    for (int j = 0; j + 1 < W; ++j) load_x<T, V, W>(q, t0 - (W - 1) + j, b, c, win[j]);
    auto step = [&](int t, const Raw<T, V>& r) {
      float o[V];
      r.get(win[W - 1]);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float p = taps.pre(win, v);
        o[v] = q.silu ? p * sigmoid_f(p) : p;
      }
      store_v<T, V>(u + t * q.u_t, o);
      shift(win);
    };
    // Whole blocks of kU steps, the next block's loads on their way while one is computed.
    Raw<T, V> nx[kU], ny[kU];
    auto block = [&](int tb, Raw<T, V> (&r)[kU]) {
      const T* xb = x + tb * q.x_t;
#pragma unroll
      for (int i = 0; i < kU; ++i) r[i] = *reinterpret_cast<const Raw<T, V>*>(xb + i * q.x_t);
    };
    int t = t0;
    if (t + kU <= te) block(t, nx);
    for (; t + kU <= te; t += kU) {
      if (t + 2 * kU <= te) block(t + kU, ny);
#pragma unroll
      for (int i = 0; i < kU; ++i) step(t + i, nx[i]);
#pragma unroll
      for (int i = 0; i < kU; ++i) nx[i] = ny[i];
    }
    if (t < te) {
#pragma unroll
      for (int i = 0; i < kU; ++i)
        if (t + i < te) nx[i] = *reinterpret_cast<const Raw<T, V>*>(x + (t + i) * q.x_t);
#pragma unroll
      for (int i = 0; i < kU; ++i)
        if (t + i < te) step(t + i, nx[i]);
    }
  }
  const float zero[V] = {};
  for (int t = max(t0, te); t < t1; ++t) store_v<T, V>(u + t * q.u_t, zero);
}

template <typename T, int V, int W>
__global__ void __launch_bounds__(kLanes * kRuns, 2) conv_bwd_kernel(const ConvArgs a) {
  __shared__ float part[kRuns][(W + 1) * V][kLanes];
  grid_dep_launch_dependents();
  const ConvCall& q = a.q;
  const int lane = threadIdx.x % kLanes, run = threadIdx.x / kLanes;
  const int c = (blockIdx.x * kLanes + lane) * V;
  const int b = blockIdx.y;
  const int len = q.lengths ? min(max(q.lengths[b], 0), q.K) : q.K;
  const int t0 = (blockIdx.z * kRuns + run) * a.run;
  const int t1 = min(q.K, t0 + a.run);
  float dw[W][V], db[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    db[v] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][v] = 0.f;
  }
  if (c < q.D && t0 < t1) {
    const Taps<V, W> taps(q, c);
    const T* x = static_cast<const T*>(q.x) + b * q.x_b + c;
    const T* du = static_cast<const T*>(q.du) + b * q.du_b + c;
    T* dx = static_cast<T*>(q.dx) + b * q.dx_b + c;
    T* dx0 = q.dx0 ? static_cast<T*>(q.dx0) + static_cast<long long>(b) * (W - 1) * q.D + c : nullptr;
    float win[W][V], g[W][V];  // the last W inputs, and the last W gradients of p
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) g[j][v] = 0.f;
    const int te = min(t1, len);
    if (t0 < te) {
#pragma unroll
      for (int j = 0; j + 1 < W; ++j) load_x<T, V, W>(q, t0 - (W - 1) + j, b, c, win[j]);
    }
    // Step t forms g_t and with it completes dx at t - (W - 1), which takes g there .. g_t.
    // `own`: the step is the run's own and counts in the parameters' sums (the W - 1 steps after
    // the run only complete its dx).
    auto gradient = [&](const Raw<T, V>& rx, const Raw<T, V>& rd, bool own) {
      float d[V];
      rx.get(win[W - 1]);
      rd.get(d);
      shift(g);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float gv = d[v];
        if (q.silu) {
          const float p = taps.pre(win, v), s = sigmoid_f(p);
          gv *= s * fmaf(p, 1.f - s, 1.f);
        }
        g[W - 1][v] = gv;
        if (own) {
          db[v] += gv;
#pragma unroll
          for (int j = 0; j < W; ++j) dw[j][v] = fmaf(gv, win[j][v], dw[j][v]);
        }
      }
      shift(win);
    };
    auto finish = [&](int td) {
      float o[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        o[v] = 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) o[v] = fmaf(taps.w[W - 1 - k][v], g[k][v], o[v]);
      }
      if (td >= t0) store_v<T, V>(dx + td * q.dx_t, o);
      else if (td < 0 && dx0) store_v<T, V>(dx0 + static_cast<long long>(td + W - 1) * q.D, o);
    };
    const int tl = min(t1 + W - 1, len);  // steps with a gradient that the run needs
    Raw<T, V> nx[kU], nd[kU], px[kU], pd[kU];
    auto block = [&](int tb, Raw<T, V> (&rx)[kU], Raw<T, V> (&rd)[kU]) {
      const T *xb = x + tb * q.x_t, *db_ = du + tb * q.du_t;
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        rx[i] = *reinterpret_cast<const Raw<T, V>*>(xb + i * q.x_t);
        rd[i] = *reinterpret_cast<const Raw<T, V>*>(db_ + i * q.du_t);
      }
    };
    int t = t0;
    if (t + kU <= te) block(t, nx, nd);
    for (; t + kU <= te; t += kU) {
      if (t + 2 * kU <= te) block(t + kU, px, pd);
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        gradient(nx[i], nd[i], true);
        finish(t + i - (W - 1));
      }
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        nx[i] = px[i];
        nd[i] = pd[i];
      }
    }
    for (; t < tl; ++t) {
      gradient(*reinterpret_cast<const Raw<T, V>*>(x + t * q.x_t),
               *reinterpret_cast<const Raw<T, V>*>(du + t * q.du_t), t < te);
      finish(t - (W - 1));
    }
    // Past the sequence's end the gradients are zero, and W - 1 steps on so is dx.
    for (; t < min(t1, max(t0, len)) + W - 1; ++t) {
      shift(g);
#pragma unroll
      for (int v = 0; v < V; ++v) g[W - 1][v] = 0.f;
      finish(t - (W - 1));
    }
    const float zero[V] = {};
    for (int td = t - (W - 1); td < t1; ++td) store_v<T, V>(dx + td * q.dx_t, zero);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int j = 0; j < W; ++j) part[run][v * W + j][lane] = dw[j][v];
    part[run][V * W + v][lane] = db[v];
  }
  __syncthreads();
  // Sums over the CTA's runs, in run order.
  const size_t row = static_cast<size_t>(blockIdx.z) * gridDim.y + blockIdx.y;
  for (int e = threadIdx.x; e < (W + 1) * V * kLanes; e += kLanes * kRuns) {
    const int l = e % kLanes, k = e / kLanes;
    const int ch = (blockIdx.x * kLanes + l) * V + (k < V * W ? k / W : k - V * W);
    if (ch >= q.D) continue;
    float s = 0.f;
#pragma unroll
    for (int r = 0; r < kRuns; ++r) s += part[r][k][l];
    if (k < V * W) a.pw[(row * q.D + ch) * W + k % W] = s;
    else a.pb[row * q.D + ch] = s;
  }
}

// One token: u = silu(bias + w . [state ; x]), and the state moves on by one input.  A thread
// holds V channels of kTokens sequences, so their taps are read once for them.  The state may be
// the new state's own memory: a thread reads what it writes before it writes it.
template <typename T, int V, int W>
__global__ void __launch_bounds__(128) conv_step_kernel(const ConvCall q) {
  const int c = (blockIdx.x * 128 + threadIdx.x) * V;
  if (c >= q.D) return;
  const int b0 = blockIdx.y * kTokens;
  using R = Raw<T, V>;
  R r[kTokens][W];
#pragma unroll
  for (int k = 0; k < kTokens; ++k) {
    const int b = min(b0 + k, q.B - 1);
    const T* st = static_cast<const T*>(q.x0) + static_cast<long long>(b) * (W - 1) * q.D + c;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) r[k][j] = *reinterpret_cast<const R*>(st + static_cast<long long>(j) * q.D);
    r[k][W - 1] = *reinterpret_cast<const R*>(static_cast<const T*>(q.x) + b * q.x_b + c);
  }
  const Taps<V, W> taps(q, c);
#pragma unroll
  for (int k = 0; k < kTokens; ++k) {
    const int b = b0 + k;
    if (b >= q.B) break;
    float x[W][V], o[V];
#pragma unroll
    for (int j = 0; j < W; ++j) r[k][j].get(x[j]);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float p = taps.pre(x, v);
      o[v] = q.silu ? p * sigmoid_f(p) : p;
    }
    T* ns = static_cast<T*>(q.last) + static_cast<long long>(b) * (W - 1) * q.D + c;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) *reinterpret_cast<R*>(ns + static_cast<long long>(j) * q.D) = r[k][j + 1];
    store_v<T, V>(static_cast<T*>(q.u) + b * q.u_b + c, o);
  }
}

// ---- host side ----

bool al8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

// Vector width: 8 bytes of channels where every row starts on 8 bytes, else one channel.
bool conv_vec(const ConvCall& q) {
  const long long v = q.bf16 ? 4 : 2;
  return q.D % v == 0 && al8(q.x) && al8(q.u) && al8(q.x0) && al8(q.last) && al8(q.du) &&
         al8(q.dx) && al8(q.dx0) && q.x_t % v == 0 && q.x_b % v == 0 && q.u_t % v == 0 &&
         q.u_b % v == 0 && q.du_t % v == 0 && q.du_b % v == 0 && q.dx_t % v == 0 &&
         q.dx_b % v == 0;
}

// Steps of a run and CTAs along the steps, from the sizes alone (so the order of the parameter
// sums does not change with alignment).
int conv_run(int B, int K, int D, bool bf16, int halo) {
  const int v = bf16 ? 4 : 2;
  const long long threads = static_cast<long long>(B) * ((D + v - 1) / v);
  int run = 64;
  while (run > (halo ? 8 : 4) && threads * ((K + run - 1) / run) < 152LL * 1024) run /= 2;
  return run;
}
int conv_ctas_t(int K, int run) { return (K + run * kRuns - 1) / (run * kRuns); }

template <typename F>
cudaError_t by_taps(int W, F&& f) {
  switch (W) {
    case 2: return f(std::integral_constant<int, 2>{});
    case 3: return f(std::integral_constant<int, 3>{});
    default: return f(std::integral_constant<int, 4>{});
  }
}

template <typename T, int V>
cudaError_t conv_fwd(const ConvArgs& a, cudaStream_t s) {
  LaunchCfg c;
  c.grid = dim3((a.q.D + kLanes * V - 1) / (kLanes * V), a.q.B, conv_ctas_t(a.q.K, a.run));
  c.block = dim3(kLanes * kRuns);
  c.stream = s;
  return by_taps(a.q.W, [&](auto w) { return launch(c, conv_fwd_kernel<T, V, decltype(w)::value>, a); });
}

template <typename T, int V>
cudaError_t conv_bwd(const ConvArgs& a, cudaStream_t s) {
  LaunchCfg c;
  c.grid = dim3((a.q.D + kLanes * V - 1) / (kLanes * V), a.q.B, conv_ctas_t(a.q.K, a.run));
  c.block = dim3(kLanes * kRuns);
  c.stream = s;
  return by_taps(a.q.W, [&](auto w) { return launch(c, conv_bwd_kernel<T, V, decltype(w)::value>, a); });
}

template <typename T, int V>
cudaError_t conv_step(const ConvCall& q, cudaStream_t s) {
  LaunchCfg c;
  c.grid = dim3((q.D + 128 * V - 1) / (128 * V), (q.B + kTokens - 1) / kTokens);
  c.block = dim3(128);
  c.stream = s;
  return by_taps(q.W, [&](auto w) { return launch(c, conv_step_kernel<T, V, decltype(w)::value>, q); });
}

}  // namespace

int conv_partials(int B, int K, int D, bool bf16) {
  return B * conv_ctas_t(K, conv_run(B, K, D, bf16, 1));
}

cudaError_t conv_fwd_launch(const ConvCall& q, cudaStream_t s) {
  const ConvArgs a{q, conv_run(q.B, q.K, q.D, q.bf16, 0), nullptr, nullptr};
  if (q.bf16) return conv_vec(q) ? conv_fwd<__nv_bfloat16, 4>(a, s) : conv_fwd<__nv_bfloat16, 1>(a, s);
  return conv_vec(q) ? conv_fwd<float, 2>(a, s) : conv_fwd<float, 1>(a, s);
}

cudaError_t conv_bwd_launch(const ConvCall& q, float* dw, float* db, float* ws, cudaStream_t s) {
  ConvArgs a{q, conv_run(q.B, q.K, q.D, q.bf16, 1), nullptr, nullptr};
  const int P = conv_partials(q.B, q.K, q.D, q.bf16);
  a.pw = P == 1 ? dw : ws;
  a.pb = P == 1 ? db : ws + static_cast<size_t>(P) * q.D * q.W;
  cudaError_t e;
  if (q.bf16) e = conv_vec(q) ? conv_bwd<__nv_bfloat16, 4>(a, s) : conv_bwd<__nv_bfloat16, 1>(a, s);
  else e = conv_vec(q) ? conv_bwd<float, 2>(a, s) : conv_bwd<float, 1>(a, s);
  if (e != cudaSuccess || P == 1) return e;
  return reduce_axis0_pair_launch(a.pw, P, q.D * q.W, 0, 0, dw, nullptr, a.pb, P, q.D, db, s, true);
}

cudaError_t conv_step_launch(const ConvCall& q, cudaStream_t s) {
  if (q.bf16) return conv_vec(q) ? conv_step<__nv_bfloat16, 4>(q, s) : conv_step<__nv_bfloat16, 1>(q, s);
  return conv_vec(q) ? conv_step<float, 2>(q, s) : conv_step<float, 1>(q, s);
}

}  // namespace cfc
