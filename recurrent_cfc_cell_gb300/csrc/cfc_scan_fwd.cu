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
// A warp holds 32 neighbouring channels times S (4, 8 or 16) states, a channel to a lane, its
// states in registers; NT warps side by side hold up to 16 NT states, CW warps 32 CW channels.
// exp is 2^(d A log2 e), and the state arithmetic runs in pairs of states (packed FMA).  The steps
// go in chunks: what a step needs per channel (d and d x) is formed once, a thread a value, and
// put in shared memory with the chunk's B and C as fp32 (read by broadcast); the warps then run
// the recurrence over the chunk, and the sums over states come back through shared memory to the
// threads that formed the values, which hold x and z for the skip and the gate.  The next
// chunk's inputs are loaded meanwhile.
//
// Bound by arithmetic at 16 states: a state's step takes one exponential, two multiplications
// and two multiply-adds, so both the exponential unit (32 a clock and SM) and the FMA pipe (128)
// allow 32 states a clock and SM.  With few channels and many steps the steps are split over
// CTAs: a first pass runs every split from a zero state, the splits' end states are folded in
// order, and the second pass starts each split from its true state.
//
// Measured on GB300, 16 states: 64 x 512 steps x 1024 channels, bf16, keeping states, 204 us (2.6e12
// state steps a second, a quarter of the exponential unit's rate; 130 instructions for 512 of them
// and what their 32 channels need, issued at 0.6 a clock and scheduler: 13 warps an SM is all there
// are).  Prompts 2 x 8191 x 1024: 135 us, of which the first pass over the split steps 45.  Tried:
// states spread over more lanes (four each, 279 us), one warp for sixteen states (302 us), chunks of
// eight steps (242 us), more CTAs an SM at fewer registers (273 us with five).
#include "cfc_launch.cuh"
#include "cfc_trunk.cuh"
#include "cfc_trunk_kernels.h"

namespace cfc {
namespace {

constexpr int kT = 2 * kScanPeriod;  // steps of a chunk

struct Tile {
  int tiles_per_group, per_group;  // channel tiles and channels of a group of B / C
};

// MODE 0: outputs.  MODE 1: the end state of each split from a zero state, and the sum of its
// steps.  MODE 2: the same for the gradient carried backwards, c <- a_t (c + C_t r_t) with r_t the
// gradient of y_t before the gate (it reads dy in the place of x).
template <typename T, int S, int CW, int NT, int MODE>
__global__ void __launch_bounds__(32 * CW * NT, CW * NT <= 4 ? 4 : 1) scan_fwd_kernel(const ScanCall q, const Tile tl,
                                                                const int steps, float* carry,
                                                                float* dsum) {
  constexpr int kThreads = 32 * CW * NT, CH = 32 * CW, NP = S * NT;
  constexpr int kEl = kT / NT;                                 // per-channel values of a thread
  constexpr int kEl2 = (kEl + 1) / 2;
  constexpr int kBC = (kT * NP + kThreads - 1) / kThreads;     // B (or C) values of a thread
  constexpr bool kGate = MODE != 1;
  __shared__ __align__(16) float2 sDU[kT][CH];
  __shared__ __align__(16) float sB[kT][NP];
  __shared__ __align__(16) float sC[MODE == 0 ? kT : 1][NP];
  __shared__ float sY[MODE == 0 ? NT : 1][MODE == 0 ? kT : 1][CH];
  if (MODE != 0) grid_dep_launch_dependents();
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int nt = warp % NT, cw = warp / NT;
  const int group = blockIdx.x / tl.tiles_per_group;
  const int t_base = (blockIdx.x % tl.tiles_per_group) * CH;
  const int b = blockIdx.y, split = blockIdx.z;
  const int len = q.lengths ? min(max(q.lengths[b], 0), q.K) : q.K;
  const int lo = split * steps;
  const int hi = min(q.K, lo + steps);
  const int end = min(hi, len);  // steps [lo, end) count
  const size_t plane = static_cast<size_t>(q.B) * q.D * q.N;

  // This lane's channel and states in the recurrence.
  const int ch = cw * 32 + lane, n0 = nt * S;
  const bool live = t_base + ch < tl.per_group;
  const int d = group * tl.per_group + (live ? t_base + ch : 0);
  const size_t cn = (static_cast<size_t>(b) * q.D + d) * q.N + n0;
  float2 A2[S / 2], h[S / 2];
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const bool in = live && n0 + i < q.N;
    const float av = in ? rate_f(q.A[static_cast<size_t>(d) * q.N + n0 + i]) : 0.f;
    float hv = 0.f;
    if (MODE == 0 && in) {
      if (carry) hv = carry[split * plane + cn + i];
      else if (q.h0) hv = q.h0[cn + i];
    }
    (i & 1 ? A2[i / 2].y : A2[i / 2].x) = av;
    (i & 1 ? h[i / 2].y : h[i / 2].x) = hv;
  }
  const bool octet = q.N % 8 == 0;
  auto put_state = [&](float* p) {
    if (!live) return;
    if (S >= 8 && octet && (reinterpret_cast<uintptr_t>(p) & 31u) == 0) {
#pragma unroll
      for (int i = 0; i < S / 8; ++i)
        if (n0 + 8 * i < q.N) {
          const float v[8] = {h[4 * i].x, h[4 * i].y, h[4 * i + 1].x, h[4 * i + 1].y,
                              h[4 * i + 2].x, h[4 * i + 2].y, h[4 * i + 3].x, h[4 * i + 3].y};
          store8(p + 8 * i, v);
        }
    } else {
#pragma unroll
      for (int i = 0; i < S; ++i)
        if (n0 + i < q.N) p[i] = (i & 1) ? h[i / 2].y : h[i / 2].x;
    }
  };

  // This thread's channel in the per-channel phases, and its steps tf, tf + NT, ...  Addresses
  // are a uniform base (sequence, tile, step) plus the thread's own offset, so that a load costs
  // no address arithmetic of the thread's.
  const int chf = NT == 1 ? tid : tid % CH, tf = NT == 1 ? 0 : tid / CH;
  const bool livef = t_base + chf < tl.per_group;
  const unsigned at = livef ? chf : 0;
  const int d0 = group * tl.per_group + t_base;
  const float bias = q.dt_bias ? q.dt_bias[d0 + at] : 0.f;
  const float skip = q.skip ? q.skip[d0 + at] : 0.f;
  const bool gated = kGate && q.z != nullptr;
  const long long x_t = MODE == 2 ? q.dy_t : q.x_t;
  const T* xp = (MODE == 2 ? static_cast<const T*>(q.dy) + b * q.dy_b
                           : static_cast<const T*>(q.x) + b * q.x_b) + d0;
  const T* tp = static_cast<const T*>(q.dt) + b * q.dt_b + d0;
  const T* zp = gated ? static_cast<const T*>(q.z) + b * q.z_b + d0 : nullptr;
  const size_t xo = at + tf * x_t, to = at + tf * q.dt_t, zo = at + tf * q.z_t;
  // MODE 2 reads C in the place of B.
  const long long B_t = MODE == 2 ? q.Cm_t : q.Bm_t;
  const T* Bp = (MODE == 2 ? static_cast<const T*>(q.Cm) + b * q.Cm_b
                           : static_cast<const T*>(q.Bm) + b * q.Bm_b) +
                static_cast<long long>(group) * q.N;
  const T* Cp = static_cast<const T*>(q.Cm) + b * q.Cm_b + static_cast<long long>(group) * q.N;
  T* yp = static_cast<T*>(q.y) + b * q.y_b + d0;
  const size_t yo = at + tf * q.y_t;
  // Offset of thread-dependent steps: at NT == 1 there are none and it stays 32 bits wide.
  auto pick = [&](const T* base, size_t off) -> const T* {
    if constexpr (NT == 1) return base + at;
    return base + off;
  };

  // This thread's values of a chunk's B and C: step kb + i kStepBC, state nb (NP divides the
  // threads, or the threads NP).
  constexpr int kPerStep = NP < kThreads ? NP : kThreads;      // threads on one step
  constexpr int kStepBC = kThreads / kPerStep;                 // steps apart
  constexpr int kWide = NP / kPerStep;                         // values of one step
  constexpr int kStepsBC = kT / kStepBC;
  static_assert(kBC == kStepsBC * kWide && kT % kStepBC == 0, "B and C spread evenly");
  const int nb = tid % kPerStep, kb0 = tid / kPerStep;
  const size_t bo = nb + kb0 * B_t, co = nb + kb0 * q.Cm_t;

  // The next chunk's inputs, as they are stored (converted when their chunk begins, so that
  // nothing waits for the loads before that).
  T rx[kEl], rt[kEl], rz[kEl], rB[kBC], rC[kBC];
  const T none = from_f32<T>(0.f);
  auto fetch_as = [&](int t0, auto whole) {
    constexpr bool kWhole = decltype(whole)::value;  // every step of the chunk counts
    const T* x0 = xp + t0 * x_t;
    const T* dt0 = tp + t0 * q.dt_t;
    const T* z0 = gated ? zp + t0 * q.z_t : nullptr;
#pragma unroll
    for (int i = 0; i < kEl; ++i) {
      const bool in = kWhole || t0 + tf + i * NT < end;
      rx[i] = in ? *pick(x0 + i * NT * x_t, xo) : none;
      rt[i] = in ? *pick(dt0 + i * NT * q.dt_t, to) : none;
    }
    if (gated) {
#pragma unroll
      for (int i = 0; i < kEl; ++i)
        rz[i] = kWhole || t0 + tf + i * NT < end ? *pick(z0 + i * NT * q.z_t, zo) : none;
    }
    const T* b0 = Bp + t0 * B_t;
    const T* c0 = Cp + t0 * q.Cm_t;
#pragma unroll
    for (int i = 0; i < kStepsBC; ++i)
#pragma unroll
      for (int w = 0; w < kWide; ++w) {
        const bool in = (kWhole || t0 + kb0 + i * kStepBC < end) && nb + w * kPerStep < q.N;
        rB[i * kWide + w] = in ? (b0 + i * kStepBC * B_t)[bo + w * kPerStep] : none;
        if (MODE == 0)
          rC[i * kWide + w] = in ? (c0 + i * kStepBC * q.Cm_t)[co + w * kPerStep] : none;
      }
  };
  auto fetch = [&](int t0) {
    if (t0 + kT <= end) fetch_as(t0, std::true_type{});
    else fetch_as(t0, std::false_type{});
  };
  static_assert(kT % NT == 0, "every thread has the same number of steps");

  float total = 0.f;  // sum of this thread's steps d
  const int chunks = end > lo ? (end - lo + kT - 1) / kT : 0;
  if (chunks > 0) fetch(lo + (MODE == 2 ? chunks - 1 : 0) * kT);
  for (int cc = 0; cc < chunks; ++cc) {
    const int t0 = lo + (MODE == 2 ? chunks - 1 - cc : cc) * kT;
    const bool whole = t0 + kT <= end;
    // ---- per channel and step: d and d x (MODE 2: d and r)
    float x[kEl], z[kEl];
    decide(gated, [&](auto gate) {
#pragma unroll
      for (int i = 0; i < kEl; ++i) {
        x[i] = to_f32(rx[i]);
        z[i] = decltype(gate)::value ? to_f32(rz[i]) : 0.f;
      }
    });
    decide(q.softplus, [&](auto sp) {
#pragma unroll
      for (int j = 0; j < kEl2; ++j) {
        const int i0 = 2 * j, i1 = 2 * j + 1 < kEl ? 2 * j + 1 : 2 * j;
        float2 dv = make_float2(to_f32(rt[i0]) + bias, to_f32(rt[i1]) + bias);
        if constexpr (decltype(sp)::value) dv = softplus2_f(dv);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const int i = 2 * j + m;
          if (i >= kEl) break;
          const int k = tf + i * NT;
          // Steps past the end leave the state alone: d = 0, so a = 1 and nothing is added.
          const float dd = whole || t0 + k < end ? (m ? dv.y : dv.x) : 0.f;
          float u = dd * x[i];
          if (MODE == 2) {
            u = x[i];
            if (gated) u *= z[i] * sigmoid_f(z[i]);
          }
          sDU[k][chf] = make_float2(dd, u);
          if (MODE != 0) total += dd;
        }
      }
    });
#pragma unroll
    for (int i = 0; i < kStepsBC; ++i)
#pragma unroll
      for (int w = 0; w < kWide; ++w) {
        sB[kb0 + i * kStepBC][nb + w * kPerStep] = to_f32(rB[i * kWide + w]);
        if (MODE == 0) sC[kb0 + i * kStepBC][nb + w * kPerStep] = to_f32(rC[i * kWide + w]);
      }
    __syncthreads();
    if (cc + 1 < chunks) fetch(MODE == 2 ? t0 - kT : t0 + kT);

    // ---- the recurrence
    float* const kept = MODE == 0 && q.states != nullptr
                            ? q.states + (t0 / kScanPeriod) * plane + cn : nullptr;
    // Blocks of kU steps: their decays do not depend on the state, so all of a block's
    // exponentials are on their way before its first update.
    constexpr int kU = S > 8 ? 2 : 4;
#pragma unroll
    for (int kb = 0; kb < kT; kb += kU) {
      if (MODE == 0 && kept && kb % kScanPeriod == 0 && (kb == 0 || t0 + kb < end))
        put_state(kept + (kb / kScanPeriod) * plane);
      float2 a[kU][S / 2], u2[kU];
#pragma unroll
      for (int j = 0; j < kU; ++j) {
        const float2 du = sDU[MODE == 2 ? kT - 1 - kb - j : kb + j][ch];
        u2[j] = make_float2(du.y, du.y);
#pragma unroll
        for (int s = 0; s < S / 2; ++s) a[j][s] = decay2_f(du.x, A2[s]);
      }
#pragma unroll
      for (int j = 0; j < kU; ++j) {
        const int k = MODE == 2 ? kT - 1 - kb - j : kb + j;
        float2 y2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int s = 0; s < S / 4; ++s) {
          const float4 bv = reinterpret_cast<const float4*>(&sB[k][n0])[s];
          const float2 B2[2] = {make_float2(bv.x, bv.y), make_float2(bv.z, bv.w)};
          float2 C2[2] = {};
          if constexpr (MODE == 0) {
            const float4 cv = reinterpret_cast<const float4*>(&sC[k][n0])[s];
            C2[0] = make_float2(cv.x, cv.y);
            C2[1] = make_float2(cv.z, cv.w);
          }
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            float2& hs = h[2 * s + m];
            const float2 am = a[j][2 * s + m];
            if constexpr (MODE == 2) {
              hs = __fmul2_rn(am, fma2(u2[j], B2[m], hs));
            } else {
              hs = fma2(am, hs, __fmul2_rn(u2[j], B2[m]));
              if constexpr (MODE == 0) y2 = fma2(hs, C2[m], y2);
            }
          }
        }
        if constexpr (MODE == 0) sY[nt][k][ch] = y2.x + y2.y;
      }
    }
    __syncthreads();

    // ---- per channel and step: the skip, the gate, the output
    if constexpr (MODE == 0) {
      T* y0 = yp + t0 * q.y_t;
      decide(gated, [&](auto gate) {
        float y[kEl];
#pragma unroll
        for (int i = 0; i < kEl; ++i) {
          const int k = tf + i * NT;
          y[i] = sY[0][k][chf];
#pragma unroll
          for (int m = 1; m < NT; ++m) y[i] += sY[m][k][chf];
          y[i] = fmaf(skip, x[i], y[i]);
          if (decltype(gate)::value) y[i] *= z[i] * sigmoid_f(z[i]);
        }
        if (!livef) return;
        decide(whole, [&](auto all) {
#pragma unroll
          for (int i = 0; i < kEl; ++i) {
            const int t = t0 + tf + i * NT;
            if (decltype(all)::value || t < hi)
              *const_cast<T*>(pick(y0 + i * NT * q.y_t, yo)) =
                  decltype(all)::value || t < end ? from_f32<T>(y[i]) : none;
          }
        });
      });
    }
  }

  if constexpr (MODE == 0) {
    if (livef)
      for (int t = lo + chunks * kT + tf; t < hi; t += NT) yp[t * q.y_t + at] = none;
    // The end of the sequence, where this split holds it.
    const bool last = (len > lo && len <= hi) || (len == 0 && split == 0);
    if (q.h_last != nullptr && last) put_state(q.h_last + cn);
  } else {
    put_state(carry + split * plane + cn);
    // The NT threads of a channel, in order.
    float* sum = reinterpret_cast<float*>(&sDU[0][0]);
    static_assert(kThreads <= 2 * kT * CH, "the sums fit the staged values");
    sum[tid] = total;
    __syncthreads();
    if (tid < CH && livef) {
#pragma unroll
      for (int m = 1; m < NT; ++m) total += sum[tid + m * CH];
      dsum[(static_cast<size_t>(split) * q.B + b) * q.D + d0 + chf] = total;
    }
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
  const float A2 = rate_f(q.A[(bd % q.D) * q.N + e % q.N]);
  const float* start = reverse ? q.dh_last : q.h0;
  float h = start ? start[e] : 0.f;
  // Eight splits at a time: their loads are in flight together.
  constexpr int U = 8;
  for (int i0 = 0; i0 < splits; i0 += U) {
    float own[U], a[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int i = min(i0 + j, splits - 1), s = reverse ? splits - 1 - i : i;
      own[j] = carry[s * plane + e];
      a[j] = dsum[s * (plane / q.N) + bd];
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int i = i0 + j, s = reverse ? splits - 1 - i : i;
      if (i >= splits) break;
      carry[s * plane + e] = h;
      h = fmaf(decay_f(a[j], A2), h, own[j]);
    }
  }
}

// One token: a lane holds four states of a channel, LPC lanes a channel, for kSeqs sequences, so
// that A is read once for them.  What a sequence needs per channel (d and d x, later the gate) is
// formed by one lane of the channel and handed round.  The state may be the new state's own
// memory: a thread reads what it writes before it writes it.  1024 x 2048 x 64 states 198 us (5.5
// TB/s).  Tried: the state as what L2 evicts first (203 us among other passes, 81 against 79 us at 16
// states with the convolution's token, 60 against 63 us at a quarter of the sequences), four CTAs an
// SM (215 us, spilling).
constexpr int kSeqs = 4;

__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
  const float4 r = *reinterpret_cast<const float4*>(p);
  v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&v)[4]) {
  const uint2 r = *reinterpret_cast<const uint2*>(p);
  v[0] = bf16_lo_f32(r.x); v[1] = bf16_hi_f32(r.x);
  v[2] = bf16_lo_f32(r.y); v[3] = bf16_hi_f32(r.y);
}

// VEC: groups of four states are whole and aligned, in the states (16 bytes) and in B and C.  A
// CTA takes `seqs` sequences, kSeqs at a time; LPC lanes hold all states (4 LPC >= N).
template <typename T, int LPC, bool VEC>
__global__ void __launch_bounds__(256) scan_step_kernel(const ScanCall q, const int per_group,
                                                        const int seqs) {
  constexpr int kOwn = LPC >= kSeqs ? 1 : kSeqs / LPC;  // sequences whose values a lane forms
  const int lane = threadIdx.x % LPC;
  const int d_raw = blockIdx.x * (256 / LPC) + threadIdx.x / LPC;
  const int d = min(d_raw, q.D - 1);
  const int group = q.G == 1 ? 0 : d / per_group;
  const int n = lane * 4;
  const bool in = n < q.N, live = d_raw < q.D;
  const float bias = q.dt_bias ? q.dt_bias[d] : 0.f, skip = q.skip ? q.skip[d] : 0.f;
  const size_t row = static_cast<size_t>(q.D) * q.N;  // states of a sequence
  const size_t ho = static_cast<size_t>(d) * q.N + n, go = static_cast<size_t>(group) * q.N + n;
  float A2[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) A2[i] = n + i < q.N ? rate_f(q.A[ho + i]) : 0.f;
  const int b_end = min(q.B, (static_cast<int>(blockIdx.y) + 1) * seqs);
  for (int b0 = blockIdx.y * seqs; b0 < b_end; b0 += kSeqs) {
    // Uniform bases of the sequences (the last one again where there are fewer than kSeqs).
    const float* hp = q.h0 + b0 * row;
    const T* Bp = static_cast<const T*>(q.Bm) + b0 * q.Bm_b;
    const T* Cp = static_cast<const T*>(q.Cm) + b0 * q.Cm_b;
    const int last = b_end - 1 - b0;
    float h[kSeqs][4] = {}, Bv[kSeqs][4] = {}, Cv[kSeqs][4] = {};
#pragma unroll
    for (int k = 0; k < kSeqs; ++k) {
      const int kk = min(k, last);
      if constexpr (VEC) {
        if (in) {
          load4(hp + kk * row + ho, h[k]);
          load4(Bp + kk * q.Bm_b + go, Bv[k]);
          load4(Cp + kk * q.Cm_b + go, Cv[k]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n + i < q.N) {
            h[k][i] = hp[kk * row + ho + i];
            Bv[k][i] = to_f32(Bp[kk * q.Bm_b + go + i]);
            Cv[k][i] = to_f32(Cp[kk * q.Cm_b + go + i]);
          }
      }
    }
    float own_d[kOwn], own_x[kOwn], own_z[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int b = b0 + min(lane % kSeqs + i * LPC, last);
      own_x[i] = to_f32(static_cast<const T*>(q.x)[b * q.x_b + d]);
      own_z[i] = q.z ? to_f32(static_cast<const T*>(q.z)[b * q.z_b + d]) : 0.f;
      const float raw = to_f32(static_cast<const T*>(q.dt)[b * q.dt_b + d]) + bias;
      own_d[i] = q.softplus ? softplus_f(raw) : raw;
    }
    float yv[kSeqs];
#pragma unroll
    for (int k = 0; k < kSeqs; ++k) {
      const float dv = __shfl_sync(0xffffffffu, own_d[k / LPC % kOwn], k % LPC, LPC);
      const float uv = dv * __shfl_sync(0xffffffffu, own_x[k / LPC % kOwn], k % LPC, LPC);
      yv[k] = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[k][i] = fmaf(decay_f(dv, A2[i]), h[k][i], uv * Bv[k][i]);
        yv[k] = fmaf(h[k][i], Cv[k][i], yv[k]);
      }
      if (live && in && k <= last) {
        float* np = q.h_last + (b0 + k) * row + ho;
        if constexpr (VEC) {
          *reinterpret_cast<float4*>(np) = make_float4(h[k][0], h[k][1], h[k][2], h[k][3]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (n + i < q.N) np[i] = h[k][i];
        }
      }
    }
#pragma unroll
    for (int m = LPC / 2; m > 0; m >>= 1)
#pragma unroll
      for (int k = 0; k < kSeqs; ++k) yv[k] += __shfl_xor_sync(0xffffffffu, yv[k], m);
#pragma unroll
    for (int k = 0; k < kSeqs; ++k) {
      if (!live || lane != k % LPC || k > last) continue;
      const float z = own_z[k / LPC % kOwn];
      float y = fmaf(skip, own_x[k / LPC % kOwn], yv[k]);
      if (q.z) y *= z * sigmoid_f(z);
      static_cast<T*>(q.y)[(b0 + k) * q.y_b + d] = from_f32<T>(y);
    }
  }
}

// ---- host side ----

// States of a warp and warps side by side: f(S, CW, NT).
template <typename F>
cudaError_t by_states(int N, F&& f) {
  using std::integral_constant;
#define CFC_SCAN_CASE(S, C, L) \
  return f(integral_constant<int, S>{}, integral_constant<int, C>{}, integral_constant<int, L>{})
  if (N <= 4) CFC_SCAN_CASE(4, 2, 1);
  if (N <= 8) CFC_SCAN_CASE(8, 2, 1);
  if (N <= 16) CFC_SCAN_CASE(8, 2, 2);
  if (N <= 32) CFC_SCAN_CASE(8, 1, 4);
  if (N <= 64) CFC_SCAN_CASE(8, 1, 8);
  CFC_SCAN_CASE(16, 1, 8);
#undef CFC_SCAN_CASE
}

template <typename T, int MODE>
cudaError_t run_scan(const ScanCall& q, const ScanSplit& sp, float* carry, float* dsum,
                     cudaStream_t s) {
  return by_states(q.N, [&](auto S, auto C, auto L) {
    constexpr int CW = decltype(C)::value, NT = decltype(L)::value;
    Tile tl;
    tl.per_group = q.D / q.G;
    tl.tiles_per_group = (tl.per_group + 32 * CW - 1) / (32 * CW);
    LaunchCfg c;
    c.grid = dim3(tl.tiles_per_group * q.G, q.B, sp.splits);
    c.block = dim3(32 * CW * NT);
    c.stream = s;
    return launch(c, scan_fwd_kernel<T, decltype(S)::value, CW, NT, MODE>, q, tl, sp.steps, carry,
                  dsum);
  });
}

}  // namespace

ScanSplit scan_split(int K, long long ctas, int slots, int least_steps, int least_total) {
  const int unit = 2 * kScanPeriod;
  ScanSplit sp{1, K};
  long long splits = slots / ctas;
  if (splits > K / least_steps) splits = K / least_steps;
  if (splits < 3 || K < least_total) return sp;
  sp.steps = static_cast<int>(((K + splits - 1) / splits + unit - 1) / unit * unit);
  sp.splits = (K + sp.steps - 1) / sp.steps;
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
    e = reverse ? run_scan<__nv_bfloat16, 2>(q, sp, carry, dsum, s)
                : run_scan<__nv_bfloat16, 1>(q, sp, carry, dsum, s);
  else
    e = reverse ? run_scan<float, 2>(q, sp, carry, dsum, s)
                : run_scan<float, 1>(q, sp, carry, dsum, s);
  if (e != cudaSuccess) return e;
  LaunchCfg c;
  c.grid = dim3(static_cast<unsigned>((plane + 255) / 256));
  c.block = dim3(256);
  c.stream = s;
  c.pdl = true;
  return launch(c, scan_fold_kernel, q, sp.splits, reverse, carry, static_cast<const float*>(dsum));
}

namespace {
// Six CTAs an SM: 2 x 8191 x 1024 x 16 133 us with 28 splits, 145 us with 18, 138 and 135 us with 37
// and 55.  A second pass over the steps pays from about 256 of them.
ScanSplit fwd_split(const ScanCall& q) {
  long long ctas = 1;
  (void)by_states(q.N, [&](auto, auto C, auto) {
    constexpr int ch = 32 * decltype(C)::value;
    ctas = static_cast<long long>(q.B) * q.G * ((q.D / q.G + ch - 1) / ch);
    return cudaSuccess;
  });
  return scan_split(q.K, ctas, 152 * 6, 64, 256);
}
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
  return q.bf16 ? run_scan<__nv_bfloat16, 0>(q, sp, carry, nullptr, s)
                : run_scan<float, 0>(q, sp, carry, nullptr, s);
}

cudaError_t scan_step_launch(const ScanCall& q, cudaStream_t s) {
  const uintptr_t e = q.bf16 ? 8 : 16;  // bytes of four values of B or C
  const bool vec = q.N % 4 == 0 && reinterpret_cast<uintptr_t>(q.h0) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(q.h_last) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(q.Bm) % e == 0 && q.Bm_b % 4 == 0 &&
                   reinterpret_cast<uintptr_t>(q.Cm) % e == 0 && q.Cm_b % 4 == 0;
  int lpc = 1;
  while (lpc * 4 < q.N) lpc *= 2;
  LaunchCfg c;
  c.block = dim3(256);
  c.stream = s;
  // Sixteen sequences a CTA where that still leaves several CTAs an SM (A and the channel's
  // parameters are then read once for them), else four.
  const int tiles = (q.D + 256 / lpc - 1) / (256 / lpc);
  const int seqs = static_cast<long long>(tiles) * ((q.B + 15) / 16) >= 152 * 8 ? 16 : kSeqs;
  const int per_group = q.D / q.G;
  c.grid = dim3(tiles, (q.B + seqs - 1) / seqs);
  auto go = [&](auto L) {
    constexpr int l = decltype(L)::value;
    if (q.bf16)
      return vec ? launch(c, scan_step_kernel<__nv_bfloat16, l, true>, q, per_group, seqs)
                 : launch(c, scan_step_kernel<__nv_bfloat16, l, false>, q, per_group, seqs);
    return vec ? launch(c, scan_step_kernel<float, l, true>, q, per_group, seqs)
               : launch(c, scan_step_kernel<float, l, false>, q, per_group, seqs);
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
