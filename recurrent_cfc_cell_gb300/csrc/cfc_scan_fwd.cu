// cfc_scan_fwd.cu -- the selective state space scan: prompts (and training's forward pass), the
// carry over splits of a long axis, and the single-token step.
//
//   d_t = softplus(dt_t + dt_bias)            (or dt_t + dt_bias)
//   h_t[n] = exp(d_t A[n]) h_{t-1}[n] + d_t B_t[n] x_t
//   y_t = (sum_n C_t[n] h_t[n] + skip x_t) z_t sigmoid(z_t)
//
// per channel, with N states; B and C are shared by the channels of a group.  A sequence of
// length L < K ends at L: its state stays and its later outputs are 0.
//
// A lane holds S states of one channel in registers and LPC lanes share a channel, so a warp
// covers 32 / LPC neighbouring channels and its loads of x, dt and z are consecutive.  exp is
// 2^(d A log2 e), and the state arithmetic runs in pairs of states (packed FMA).  B and C of a
// chunk of steps sit in shared memory as fp32 and are read by broadcast; the next chunk's
// inputs are in registers while this one is computed.  With few channels and many steps the
// steps are split over CTAs: a first pass runs every split from a zero state, the splits'
// end states are folded in order, and the second pass starts each split from its true state.
#include "cfc_kernels.h"
#include "cfc_launch.cuh"
#include "cfc_trunk.cuh"

namespace cfc {
namespace {

constexpr int kThreads = 128;
constexpr int kTC = 8;  // steps of a chunk
static_assert(kScanPeriod % kTC == 0 || kTC % kScanPeriod == 0, "chunks and kept states line up");
constexpr float kLog2e = 1.4426950408889634f;

// What a lane group's tile is: channels of one group of B / C.
struct Tile {
  int tiles_per_group, per_group;  // per_group: channels D / G
};

// MODE 0: outputs.  MODE 1: the end state of each split from a zero state (forward), and the sum
// of its steps.  MODE 2: the same for the gradient, running the steps backwards.
template <typename T, int S, int LPC, int MODE>
__global__ void __launch_bounds__(kThreads) scan_fwd_kernel(const ScanCall q, const Tile tl,
                                                            const int steps, float* carry,
                                                            float* dsum) {
  constexpr int NP = S * LPC;            // padded states
  constexpr int CH = kThreads / LPC;     // channels of a CTA
  constexpr int kPer = (kTC * NP + kThreads - 1) / kThreads;  // staged values per thread and array
  __shared__ __align__(16) float sB[kTC][NP];
  __shared__ __align__(16) float sC[MODE == 1 ? 1 : kTC][MODE == 1 ? 4 : NP];
  const int tid = threadIdx.x;
  const int group = blockIdx.x / tl.tiles_per_group;
  const int in_group = (blockIdx.x % tl.tiles_per_group) * CH + tid / LPC;
  const bool live = in_group < tl.per_group;
  const int d = group * tl.per_group + (live ? in_group : 0);
  const int b = blockIdx.y, split = blockIdx.z;
  const int n0 = (tid % LPC) * S;
  const int len = q.lengths ? min(max(q.lengths[b], 0), q.K) : q.K;
  const int lo = split * steps;
  const int hi = min(q.K, lo + steps);
  const int end = min(hi, len);  // steps [lo, end) count
  const size_t cn = (static_cast<size_t>(b) * q.D + d) * q.N + n0;  // this lane's states
  const size_t plane = static_cast<size_t>(q.B) * q.D * q.N;

  float2 A2[S / 2], h[S / 2];
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const bool in = live && n0 + i < q.N;
    const float av = in ? q.A[static_cast<size_t>(d) * q.N + n0 + i] * kLog2e : 0.f;
    float hv = 0.f;
    if (MODE == 0 && in) {
      if (carry) hv = carry[split * plane + cn + i];
      else if (q.h0) hv = q.h0[cn + i];
    }
    if (i & 1) {
      A2[i / 2].y = av;
      h[i / 2].y = hv;
    } else {
      A2[i / 2].x = av;
      h[i / 2].x = hv;
    }
  }
  const float bias = q.dt_bias ? q.dt_bias[d] : 0.f;
  const float skip = q.skip ? q.skip[d] : 0.f;
  const T* xp = static_cast<const T*>(MODE == 2 ? q.dy : q.x) + (MODE == 2 ? b * q.dy_b : b * q.x_b) + d;
  const T* tp = static_cast<const T*>(q.dt) + b * q.dt_b + d;
  const T* zp = (q.z && MODE != 1) ? static_cast<const T*>(q.z) + b * q.z_b + d : nullptr;
  const long long x_t = MODE == 2 ? q.dy_t : q.x_t;
  const T* Bp = static_cast<const T*>(q.Bm) + b * q.Bm_b + static_cast<long long>(group) * q.N;
  const T* Cp = static_cast<const T*>(q.Cm) + b * q.Cm_b + static_cast<long long>(group) * q.N;
  T* yp = static_cast<T*>(q.y) + b * q.y_b + d;

  // Chunks of kTC steps, forwards or backwards; chunk c covers steps lo + c kTC ...
  const int chunks = end > lo ? (end - lo + kTC - 1) / kTC : 0;
  // The next chunk's inputs, as they are stored (converted when their chunk begins, so that
  // nothing waits for the loads before that).
  T rx[kTC], rt[kTC], rz[kTC], rB[kPer], rC[kPer];
  const T none = from_f32<T>(0.f);
  auto fetch = [&](int c) {
    const int t0 = lo + c * kTC;
#pragma unroll
    for (int i = 0; i < kTC; ++i) {
      const bool in = t0 + i < end;
      rx[i] = in ? xp[(t0 + i) * x_t] : none;
      rt[i] = in ? tp[(t0 + i) * q.dt_t] : none;
      rz[i] = (in && zp) ? zp[(t0 + i) * q.z_t] : none;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = tid + i * kThreads, t = e / NP, n = e % NP;
      const bool in = t < kTC && t0 + t < end && n < q.N;
      if (MODE != 2) rB[i] = in ? Bp[(t0 + t) * q.Bm_t + n] : none;
      if (MODE != 1) rC[i] = in ? Cp[(t0 + t) * q.Cm_t + n] : none;
    }
  };
  float total = 0.f;  // sum of the split's steps
  if (chunks > 0) fetch(MODE == 2 ? chunks - 1 : 0);
  for (int cc = 0; cc < chunks; ++cc) {
    const int c = MODE == 2 ? chunks - 1 - cc : cc;
    const int t0 = lo + c * kTC;
    float x[kTC], dt[kTC], z[kTC];
#pragma unroll
    for (int i = 0; i < kTC; ++i) {
      x[i] = to_f32(rx[i]);
      dt[i] = to_f32(rt[i]) + bias;
      z[i] = to_f32(rz[i]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = tid + i * kThreads;
      if (e < kTC * NP) {
        if (MODE != 2) (&sB[0][0])[e] = to_f32(rB[i]);
        if (MODE != 1) (&sC[0][0])[e] = to_f32(rC[i]);
      }
    }
    __syncthreads();
    if (cc + 1 < chunks) fetch(MODE == 2 ? c - 1 : c + 1);
    if (MODE == 0 && q.states != nullptr && t0 % kScanPeriod == 0 && live) {
      float* st = q.states + (t0 / kScanPeriod) * plane + cn;
      if (q.N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < S / 4; ++i)
          if (n0 + 4 * i < q.N)
            reinterpret_cast<float4*>(st)[i] =
                make_float4(h[2 * i].x, h[2 * i].y, h[2 * i + 1].x, h[2 * i + 1].y);
      } else {
#pragma unroll
        for (int i = 0; i < S; ++i)
          if (n0 + i < q.N) st[i] = (i & 1) ? h[i / 2].y : h[i / 2].x;
      }
    }
#pragma unroll
    for (int ii = 0; ii < kTC; ++ii) {
      const int i = MODE == 2 ? kTC - 1 - ii : ii;
      if (t0 + i < end) {
        const float dv = q.softplus ? softplus_f(dt[i]) : dt[i];
        if (MODE != 0) total += dv;
        const float2 d2 = make_float2(dv, dv);
        if constexpr (MODE != 2) {
          const float2 dx2 = make_float2(dv * x[i], dv * x[i]);
          float2 y2 = make_float2(0.f, 0.f);
#pragma unroll
          for (int s = 0; s < S / 2; ++s) {
            const float2 e = __fmul2_rn(d2, A2[s]);
            const float2 a = make_float2(exp2_f(e.x), exp2_f(e.y));
            const float2 Bv = reinterpret_cast<const float2*>(&sB[i][n0])[s];
            h[s] = fma2(a, h[s], __fmul2_rn(dx2, Bv));
            if constexpr (MODE == 0)
              y2 = fma2(h[s], reinterpret_cast<const float2*>(&sC[i][n0])[s], y2);
          }
          if constexpr (MODE == 0) {
            float y = y2.x + y2.y;
#pragma unroll
            for (int m = LPC / 2; m > 0; m >>= 1) y += __shfl_xor_sync(0xffffffffu, y, m);
            y = fmaf(skip, x[i], y);
            if (zp) y *= z[i] * sigmoid_fast(z[i]);
            if (live && tid % LPC == 0) yp[(t0 + i) * q.y_t] = from_f32<T>(y);
          }
        } else {
          // c <- a_t (c + C_t g_t), g_t the gradient of y_t before the gate
          float g = x[i];
          if (zp) g *= z[i] * sigmoid_fast(z[i]);
          const float2 g2 = make_float2(g, g);
#pragma unroll
          for (int s = 0; s < S / 2; ++s) {
            const float2 e = __fmul2_rn(d2, A2[s]);
            const float2 a = make_float2(exp2_f(e.x), exp2_f(e.y));
            h[s] = __fmul2_rn(a, fma2(g2, reinterpret_cast<const float2*>(&sC[i][n0])[s], h[s]));
          }
        }
      }
    }
  }
  if (!live) return;
  if constexpr (MODE == 0) {
    // The end of the sequence, where this split holds it.
    const bool last = (len > lo && len <= hi) || (len == 0 && split == 0);
    if (q.h_last != nullptr && last) {
#pragma unroll
      for (int i = 0; i < S; ++i)
        if (n0 + i < q.N) q.h_last[cn + i] = (i & 1) ? h[i / 2].y : h[i / 2].x;
    }
    if (tid % LPC == 0)
      for (int t = max(lo, end); t < hi; ++t) yp[t * q.y_t] = from_f32<T>(0.f);
  } else {
#pragma unroll
    for (int i = 0; i < S; ++i)
      if (n0 + i < q.N) carry[split * plane + cn + i] = (i & 1) ? h[i / 2].y : h[i / 2].x;
    if (tid % LPC == 0) dsum[(static_cast<size_t>(split) * q.B + b) * q.D + d] = total;
  }
}

// Folds the splits' own end states into what enters each split, in place: a thread a state.
__global__ void __launch_bounds__(256) scan_fold_kernel(const ScanCall q, int splits, bool reverse,
                                                        float* carry, const float* dsum) {
  grid_dep_wait();
  const size_t plane = static_cast<size_t>(q.B) * q.D * q.N;
  const size_t e = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (e >= plane) return;
  const size_t bd = e / q.N;
  const float A2 = q.A[(bd % q.D) * q.N + e % q.N] * kLog2e;
  const float* start = reverse ? q.dh_last : q.h0;
  float h = start ? start[e] : 0.f;
  for (int i = 0; i < splits; ++i) {
    const int s = reverse ? splits - 1 - i : i;
    const float own = carry[s * plane + e];
    const float a = exp2_f(A2 * dsum[s * (plane / q.N) + bd]);
    carry[s * plane + e] = h;
    h = fmaf(a, h, own);
  }
}

// One token: a lane holds four states of a channel and walks over kSeqs sequences, so A and the
// channel's parameters are read once for them.  The state may be the new state's own memory.
constexpr int kSeqs = 4;
template <typename T, int LPC, bool VEC>
__global__ void __launch_bounds__(256) scan_step_kernel(const ScanCall q) {
  const int lane = threadIdx.x % LPC;
  const int d_raw = blockIdx.x * (256 / LPC) + threadIdx.x / LPC;
  const bool live = d_raw < q.D;
  const int d = live ? d_raw : q.D - 1;
  const int group = d / (q.D / q.G);
  const float bias = q.dt_bias ? q.dt_bias[d] : 0.f, skip = q.skip ? q.skip[d] : 0.f;
  const int b0 = blockIdx.y * kSeqs;
  float yv[kSeqs] = {};
  float dv[kSeqs], xv[kSeqs];
#pragma unroll
  for (int k = 0; k < kSeqs; ++k) {
    const int b = min(b0 + k, q.B - 1);
    xv[k] = to_f32(static_cast<const T*>(q.x)[b * q.x_b + d]);
    const float raw = to_f32(static_cast<const T*>(q.dt)[b * q.dt_b + d]) + bias;
    dv[k] = q.softplus ? softplus_f(raw) : raw;
  }
  for (int n = lane * 4; n < q.N; n += LPC * 4) {
    float A2[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      A2[i] = n + i < q.N ? q.A[static_cast<size_t>(d) * q.N + n + i] * kLog2e : 0.f;
    float h[kSeqs][4];
#pragma unroll
    for (int k = 0; k < kSeqs; ++k) {
      const float* hp = q.h0 + (static_cast<size_t>(min(b0 + k, q.B - 1)) * q.D + d) * q.N + n;
      if constexpr (VEC) {
        const float4 r = *reinterpret_cast<const float4*>(hp);
        h[k][0] = r.x; h[k][1] = r.y; h[k][2] = r.z; h[k][3] = r.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) h[k][i] = n + i < q.N ? hp[i] : 0.f;
      }
    }
#pragma unroll
    for (int k = 0; k < kSeqs; ++k) {
      const int b = min(b0 + k, q.B - 1);
      const T* Bp = static_cast<const T*>(q.Bm) + b * q.Bm_b + static_cast<long long>(group) * q.N + n;
      const T* Cp = static_cast<const T*>(q.Cm) + b * q.Cm_b + static_cast<long long>(group) * q.N + n;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool in = VEC || n + i < q.N;
        const float bv = in ? to_f32(Bp[i]) : 0.f, cv = in ? to_f32(Cp[i]) : 0.f;
        h[k][i] = fmaf(exp2_f(dv[k] * A2[i]), h[k][i], dv[k] * xv[k] * bv);
        yv[k] = fmaf(h[k][i], cv, yv[k]);
      }
      if (live && b0 + k < q.B) {
        float* np = q.h_last + (static_cast<size_t>(b) * q.D + d) * q.N + n;
        if constexpr (VEC) {
          *reinterpret_cast<float4*>(np) = make_float4(h[k][0], h[k][1], h[k][2], h[k][3]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (n + i < q.N) np[i] = h[k][i];
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kSeqs; ++k) {
#pragma unroll
    for (int m = LPC / 2; m > 0; m >>= 1) yv[k] += __shfl_xor_sync(0xffffffffu, yv[k], m);
    if (live && lane == 0 && b0 + k < q.B) {
      const int b = b0 + k;
      float y = fmaf(skip, xv[k], yv[k]);
      if (q.z) {
        const float z = to_f32(static_cast<const T*>(q.z)[b * q.z_b + d]);
        y *= z * sigmoid_fast(z);
      }
      static_cast<T*>(q.y)[b * q.y_b + d] = from_f32<T>(y);
    }
  }
}

// ---- host side ----

// States per lane and lanes per channel: f(S, LPC).  `few`: there are few channels, so that the
// step's latency counts and the states are spread over more lanes.
template <typename F>
cudaError_t by_states(int N, bool few, F&& f) {
  using std::integral_constant;
#define CFC_SCAN_CASE(S, L) return f(integral_constant<int, S>{}, integral_constant<int, L>{})
  if (N <= 4) CFC_SCAN_CASE(4, 1);
  if (few) {
    if (N <= 8) CFC_SCAN_CASE(4, 2);
    if (N <= 16) CFC_SCAN_CASE(4, 4);
    if (N <= 32) CFC_SCAN_CASE(4, 8);
    if (N <= 64) CFC_SCAN_CASE(4, 16);
  }
  if (N <= 8) CFC_SCAN_CASE(8, 1);
  if (N <= 16) CFC_SCAN_CASE(16, 1);
  if (N <= 32) CFC_SCAN_CASE(16, 2);
  if (N <= 64) CFC_SCAN_CASE(16, 4);
  CFC_SCAN_CASE(16, 8);
#undef CFC_SCAN_CASE
}

// Fewer channels than this leave SMs without a warp when a lane holds sixteen states.
bool scan_few(const ScanCall& q) {
  return static_cast<long long>(q.B) * q.D * ((q.N + 15) / 16) < 152LL * 4 * 32 * 2;
}

int lanes_for(const ScanCall& q) {
  int l = 1;
  (void)by_states(q.N, scan_few(q), [&](auto, auto L) {
    l = decltype(L)::value;
    return cudaSuccess;
  });
  return l;
}

template <typename T, int MODE>
cudaError_t run_scan(const ScanCall& q, const ScanSplit& sp, float* carry, float* dsum, bool pdl,
                     cudaStream_t s) {
  (void)pdl;
  return by_states(q.N, scan_few(q), [&](auto S, auto L) {
    constexpr int CH = kThreads / decltype(L)::value;
    Tile tl;
    tl.per_group = q.D / q.G;
    tl.tiles_per_group = (tl.per_group + CH - 1) / CH;
    LaunchCfg c;
    c.grid = dim3(tl.tiles_per_group * q.G, q.B, sp.splits);
    c.block = dim3(kThreads);
    c.stream = s;
    return launch(c, scan_fwd_kernel<T, decltype(S)::value, decltype(L)::value, MODE>, q, tl,
                  sp.steps, carry, dsum);
  });
}

}  // namespace

ScanSplit scan_split(const ScanCall& q, int channels_per_warp, int warps_wanted) {
  const long long warps =
      static_cast<long long>(q.B) * q.G * ((q.D / q.G + channels_per_warp - 1) / channels_per_warp);
  const int unit = 2 * kScanPeriod;
  ScanSplit sp{1, q.K};
  if (warps * 2 > warps_wanted || q.K < 16 * unit) return sp;
  long long splits = (warps_wanted + warps - 1) / warps;
  const long long most = q.K / (4 * unit);
  if (splits > most) splits = most;
  sp.steps = static_cast<int>(((q.K + splits - 1) / splits + unit - 1) / unit * unit);
  sp.splits = (q.K + sp.steps - 1) / sp.steps;
  return sp;
}

size_t scan_carry_floats(const ScanCall& q, const ScanSplit& sp) {
  if (sp.splits == 1) return 0;
  return static_cast<size_t>(sp.splits) * q.B * q.D * (q.N + 1);
}

cudaError_t scan_carry_launch(const ScanCall& q, const ScanSplit& sp, bool reverse, float* carry,
                              cudaStream_t s) {
  const size_t plane = static_cast<size_t>(q.B) * q.D * q.N;
  float* dsum = carry + sp.splits * plane;
  cudaError_t e;
  if (q.bf16)
    e = reverse ? run_scan<__nv_bfloat16, 2>(q, sp, carry, dsum, false, s)
                : run_scan<__nv_bfloat16, 1>(q, sp, carry, dsum, false, s);
  else
    e = reverse ? run_scan<float, 2>(q, sp, carry, dsum, false, s)
                : run_scan<float, 1>(q, sp, carry, dsum, false, s);
  if (e != cudaSuccess) return e;
  LaunchCfg c;
  c.grid = dim3(static_cast<unsigned>((plane + 255) / 256));
  c.block = dim3(256);
  c.stream = s;
  c.pdl = true;
  return launch(c, scan_fold_kernel, q, sp.splits, reverse, carry, static_cast<const float*>(dsum));
}

namespace {
ScanSplit fwd_split(const ScanCall& q) { return scan_split(q, 32 / lanes_for(q), 152 * 12); }
}  // namespace

size_t scan_fwd_ws_floats(const ScanCall& q) { return scan_carry_floats(q, fwd_split(q)); }

cudaError_t scan_fwd_launch(const ScanCall& q, cudaStream_t s) {
  const ScanSplit sp = fwd_split(q);
  float* carry = nullptr;
  if (sp.splits > 1) {
    carry = q.ws;
    const cudaError_t e = scan_carry_launch(q, sp, false, carry, s);
    if (e != cudaSuccess) return e;
  }
  return q.bf16 ? run_scan<__nv_bfloat16, 0>(q, sp, carry, nullptr, false, s)
                : run_scan<float, 0>(q, sp, carry, nullptr, false, s);
}

cudaError_t scan_step_launch(const ScanCall& q, cudaStream_t s) {
  const bool vec = q.N % 4 == 0 && (reinterpret_cast<uintptr_t>(q.h0) & 15u) == 0 &&
                   (reinterpret_cast<uintptr_t>(q.h_last) & 15u) == 0;
  int lpc = 1;
  while (lpc * 4 < q.N && lpc < 32) lpc *= 2;
  LaunchCfg c;
  c.block = dim3(256);
  c.stream = s;
  c.grid = dim3((q.D + 256 / lpc - 1) / (256 / lpc), (q.B + kSeqs - 1) / kSeqs);
  auto go = [&](auto L) {
    constexpr int l = decltype(L)::value;
    if (q.bf16)
      return vec ? launch(c, scan_step_kernel<__nv_bfloat16, l, true>, q)
                 : launch(c, scan_step_kernel<__nv_bfloat16, l, false>, q);
    return vec ? launch(c, scan_step_kernel<float, l, true>, q)
               : launch(c, scan_step_kernel<float, l, false>, q);
  };
  switch (lpc) {
    case 1: return go(std::integral_constant<int, 1>{});
    case 2: return go(std::integral_constant<int, 2>{});
    case 4: return go(std::integral_constant<int, 4>{});
    case 8: return go(std::integral_constant<int, 8>{});
    case 16: return go(std::integral_constant<int, 16>{});
    default: return go(std::integral_constant<int, 32>{});
  }
}

}  // namespace cfc
