// cfc_scan_bwd.cu -- the selective scan's backward pass.  With a_t = exp(d_t A), q_t = a_t h_{t-1},
// r_t = dL/d(y_t before the gate) and e_t = dL/dh_t:
//
//   e_t = r_t C_t + a_{t+1} e_{t+1}
//   dC_t = sum_d r_t h_t,  dB_t = sum_d e_t d_t x_t          (over the channels of a group)
//   dA = sum_{t,b} e_t q_t d_t
//   dx_t = d_t sum_n e_t B_t + skip r_t,  dd_t = sum_n e_t (A q_t + x_t B_t)
//   ddt_t = dd_t sigmoid(dt_t + dt_bias),  dskip = sum r_t x_t,  ddt_bias = sum ddt_t
//   dz_t = dy_t (y_t before the gate) silu'(z_t),  dh0 = a_0 e_0
//
// The forward pass kept the state before every kScanPeriod-th step, so the pass walks chunks of
// that many steps from the last: forwards through the chunk from its kept state (the sums with
// h_t: y, dC), leaving q_t in shared memory, then backwards (everything with e_t).
//
// A lane holds a pair of channels (its arithmetic is packed) times four states, and a warp 16
// channels times 16 states: the sums over states (y, e B, e A q) then cross four lanes and the
// sums over channels (dB, dC) eight, each by exchanging halves.  What a step
// needs per channel (d, x, r and the gate's and softplus's derivatives) is formed once per
// chunk, a thread a value, and read back four channels at a time.  NT warps side by side hold up
// to 16 NT states, CW warps 16 CW channels.  Sums over warps, channel tiles, sequences and
// splits are added in a fixed order (shared memory, then a merge), without atomics.
#include "cfc_kernels.h"
#include "cfc_launch.cuh"
#include "cfc_trunk.cuh"

namespace cfc {
namespace {

constexpr int T8 = kScanPeriod;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

constexpr int kCL = 2;       // channels of a lane, a packed pair
constexpr int kWC = 8 * kCL;  // channels of a warp

template <int CW, int NT>
struct Shape {
  static constexpr int kWarps = CW * NT, kThreads = 32 * kWarps, CH = kWC * CW, NP = 16 * NT;
  static constexpr int kPer = T8 * CH;  // one value per (step, channel)
  static constexpr int kRows = kThreads / CH;  // threads of a channel in the per-channel phases
  static constexpr int kHist = T8 * 4 * kCL * 32;  // q_t of a warp
  // Dynamic shared memory, in floats: q_t as [warp][step][2][lane][4], then what only the
  // per-channel phases use: x, dy silu'(z), sigmoid(dt + bias), and at NT = 8 the sums W.
  static constexpr int oQ = 0, oX = kWarps * kHist, oZ = oX + kPer, oS = oZ + kPer;
  static constexpr int oW = oS + kPer;
  static constexpr bool kSpill = NT == 8;  // W does not fit the 48 KB of static shared memory
  static constexpr int kFloats = oW + (kSpill ? NT * kPer : 0);
};

// Sum of a pair over the four state lanes (lane bits 0, 1): the lane keeps the first value where
// bit 1 is clear and the second where it is set.
__device__ __forceinline__ float sum_states(float2 v, int lane) {
  const bool hi = lane & 2;
  const float a = (hi ? v.y : v.x) + __shfl_xor_sync(0xffffffffu, hi ? v.x : v.y, 2);
  return a + __shfl_xor_sync(0xffffffffu, a, 1);
}

// Sum of v[0..3] over the eight channel lanes (lane bits 2..4): the lane keeps v[lane >> 3].
__device__ __forceinline__ float sum_channels(const float (&v)[4], int lane) {
  const bool hi = lane & 16;
  const float k0 = hi ? v[2] : v[0], k1 = hi ? v[3] : v[1];
  const float s0 = hi ? v[0] : v[2], s1 = hi ? v[1] : v[3];
  const float a = k0 + __shfl_xor_sync(0xffffffffu, s0, 16);
  const float b = k1 + __shfl_xor_sync(0xffffffffu, s1, 16);
  const bool lo = lane & 8;
  const float c = (lo ? b : a) + __shfl_xor_sync(0xffffffffu, lo ? a : b, 8);
  return c + __shfl_xor_sync(0xffffffffu, c, 4);
}

struct BwdPlan {
  int per_group, tiles_per_group, steps;
  const float* carry;   // [splits][B][D][N] or null
  float* params;        // [splits * B][D][N + 2]
  float *pB, *pC;       // [tiles_per_group][K][B][G][N], or null: straight to dB / dC
};

template <typename T, int CW, int NT>
__global__ void __launch_bounds__(32 * CW * NT) scan_bwd_kernel(const ScanCall q, const BwdPlan pl) {
  using Sh = Shape<CW, NT>;
  // Arrays of their own for what the walks read and what they write, so that a step's loads can
  // be issued before the last step's stores.
  extern __shared__ __align__(16) float sm[];
  __shared__ __align__(16) float sD[Sh::kPer], sU[Sh::kPer], sR[Sh::kPer];  // d, d x, r
  __shared__ __align__(16) float sB[2 * T8 * Sh::NP], sC[2 * T8 * Sh::NP];  // every value twice
  __shared__ float sY[NT * Sh::kPer], sV[NT * Sh::kPer], sWs[Sh::kSpill ? 1 : NT * Sh::kPer];
  __shared__ float sDB[CW * T8 * Sh::NP], sDC[CW * T8 * Sh::NP];
  float* const sW = Sh::kSpill ? sm + Sh::oW : sWs;
  grid_dep_launch_dependents();
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int nt = warp % NT, cw = warp / NT;
  const int group = blockIdx.x / pl.tiles_per_group, tile = blockIdx.x % pl.tiles_per_group;
  const int b = blockIdx.y, split = blockIdx.z;
  const int len = q.lengths ? min(max(q.lengths[b], 0), q.K) : q.K;
  const int lo = split * pl.steps, hi = min(q.K, lo + pl.steps), end = min(hi, len);
  const size_t plane = static_cast<size_t>(q.B) * q.D * q.N;
  const int d_base = group * pl.per_group;   // the group's first channel
  const int t_base = tile * Sh::CH;          // the tile's first channel in its group

  // This thread's channel in the per-channel phases, and its steps tf, tf + kRows, ...  Addresses
  // are a uniform base (sequence, tile, step) plus the thread's own offset.
  constexpr int NR = Sh::kRows;
  const bool busy = NR <= T8 || tid / Sh::CH < T8;  // threads beyond the chunk's steps rest
  const int chf = tid % Sh::CH, tf = busy ? tid / Sh::CH : 0;
  const bool livef = busy && t_base + chf < pl.per_group;
  const unsigned own = livef ? chf : 0;
  const int d0 = d_base + t_base;
  const float bias = q.dt_bias ? q.dt_bias[d0 + own] : 0.f, skip = q.skip ? q.skip[d0 + own] : 0.f;
  const T* xp = static_cast<const T*>(q.x) + b * q.x_b + d0;
  const T* tp = static_cast<const T*>(q.dt) + b * q.dt_b + d0;
  const T* zp = q.z ? static_cast<const T*>(q.z) + b * q.z_b + d0 : nullptr;
  const T* gp = static_cast<const T*>(q.dy) + b * q.dy_b + d0;
  T* dxp = static_cast<T*>(q.dx) + b * q.dx_b + d0;
  T* dtp = static_cast<T*>(q.ddt) + b * q.ddt_b + d0;
  T* dzp = q.dz ? static_cast<T*>(q.dz) + b * q.dz_b + d0 : nullptr;
  // The thread's element of the steps from `base` on.
  auto pick = [&](auto* base, long long stride) { return base + (own + tf * stride); };
  const T* Bp = static_cast<const T*>(q.Bm) + b * q.Bm_b + static_cast<long long>(group) * q.N;
  const T* Cp = static_cast<const T*>(q.Cm) + b * q.Cm_b + static_cast<long long>(group) * q.N;

  // This lane's states: channels c0 and c0 + 1 of the tile (a pair), states n0 .. n0 + 3.
  const int c0 = cw * kWC + (lane >> 2) * kCL, n0 = nt * 16 + (lane & 3) * 4;
  float2 A2[4], e[4], dA[4], h[4];
  auto in_state = [&](int c, int s) { return t_base + c0 + c < pl.per_group && n0 + s < q.N; };
  auto state_at = [&](int c) {  // offset of state n0 of channel c in a [B][D][N] plane
    return (static_cast<size_t>(b) * q.D + d_base + t_base + c0 + c) * q.N + n0;
  };
  // The lane's states of a plane, zero outside.
  const bool quad = q.N % 4 == 0;
  const size_t s_at = state_at(0);
  auto load_states = [&](const float* p, float2 (&v)[4]) {
    float r[2][4] = {};
    if (p != nullptr) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (!in_state(c, 0)) continue;
        const float* at = p + s_at + c * q.N;
        if (quad) {
          const float4 f = *reinterpret_cast<const float4*>(at);
          r[c][0] = f.x; r[c][1] = f.y; r[c][2] = f.z; r[c][3] = f.w;
        } else {
#pragma unroll
          for (int s = 0; s < 4; ++s)
            if (n0 + s < q.N) r[c][s] = at[s];
        }
      }
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) v[s] = make_float2(r[0][s], r[1][s]);
  };
  load_states(pl.carry ? pl.carry + split * plane : q.dh_last, e);
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const float* at = q.A + static_cast<size_t>(d_base + t_base + c0) * q.N + n0 + s;
    A2[s] = make_float2(in_state(0, s) ? at[0] * kLog2e : 0.f, in_state(1, s) ? at[q.N] * kLog2e : 0.f);
    dA[s] = make_float2(0.f, 0.f);
  }
  float dskip = 0.f, dbias = 0.f;
  float* const hist = sm + Sh::oQ + warp * Sh::kHist + lane * 4;

  // dB / dC of this tile: partial sums, or the outputs themselves.
  auto put_bc = [&](int t, int n, float vb, float vc) {
    const size_t row = (static_cast<size_t>(t) * q.B + b) * q.G + group;
    if (pl.pB) {
      const size_t at = (static_cast<size_t>(tile) * q.K * q.B * q.G + row) * q.N + n;
      pl.pB[at] = vb;
      pl.pC[at] = vc;
    } else {
      static_cast<T*>(q.dB)[row * q.N + n] = from_f32<T>(vb);
      static_cast<T*>(q.dC)[row * q.N + n] = from_f32<T>(vc);
    }
  };

  const int chunks = end > lo ? (end - lo + T8 - 1) / T8 : 0;
  // Steps after the sequence's end: zeros.
  for (int t = lo + chunks * T8 + tf; livef && t < hi; t += NR < T8 ? NR : T8) {
    dxp[t * q.dx_t + own] = from_f32<T>(0.f);
    dtp[t * q.ddt_t + own] = from_f32<T>(0.f);
    if (dzp) dzp[t * q.dz_t + own] = from_f32<T>(0.f);
  }
  for (int t = lo + chunks * T8; t < hi; ++t)
    for (int n = tid; n < q.N; n += Sh::kThreads) put_bc(t, n, 0.f, 0.f);

  // The next chunk's inputs, as they are stored.
  constexpr int kEl = NR < T8 ? T8 / NR : 1, kBC = (T8 * Sh::NP + Sh::kThreads - 1) / Sh::kThreads;
  static_assert(T8 % NR == 0 || NR % T8 == 0, "every thread has the same number of steps");
  T rx[kEl], rt[kEl], rz[kEl], rg[kEl], rB[kBC], rC[kBC];
  const T none = from_f32<T>(0.f);
  auto fetch_as = [&](int t0, auto all) {
    constexpr bool kAll = decltype(all)::value;  // every step of the chunk counts
    const T* x0 = xp + t0 * q.x_t;
    const T* dt0 = tp + t0 * q.dt_t;
    const T* g0 = gp + t0 * q.dy_t;
    const T* z0 = zp ? zp + t0 * q.z_t : nullptr;
#pragma unroll
    for (int i = 0; i < kEl; ++i) {
      const bool in = kAll || t0 + tf + i * NR < end;
      rx[i] = in ? *pick(x0 + i * NR * q.x_t, q.x_t) : none;
      rt[i] = in ? *pick(dt0 + i * NR * q.dt_t, q.dt_t) : none;
      rg[i] = in ? *pick(g0 + i * NR * q.dy_t, q.dy_t) : none;
    }
    if (zp) {
#pragma unroll
      for (int i = 0; i < kEl; ++i)
        rz[i] = kAll || t0 + tf + i * NR < end ? *pick(z0 + i * NR * q.z_t, q.z_t) : none;
    }
#pragma unroll
    for (int i = 0; i < kBC; ++i) {
      const int at = tid + i * Sh::kThreads, k = at / Sh::NP, n = at % Sh::NP;
      const bool in = k < T8 && (kAll || t0 + k < end) && n < q.N;
      rB[i] = in ? Bp[(t0 + k) * q.Bm_t + n] : none;
      rC[i] = in ? Cp[(t0 + k) * q.Cm_t + n] : none;
    }
  };
  auto fetch = [&](int t0) {
    if (t0 + T8 <= end) fetch_as(t0, std::true_type{});
    else fetch_as(t0, std::false_type{});
  };
  if (chunks > 0) {
    fetch(lo + (chunks - 1) * T8);
    load_states(q.states + ((lo + (chunks - 1) * T8) / T8) * plane, h);
  }

  for (int ck = chunks - 1; ck >= 0; --ck) {
    const int t0 = lo + ck * T8;
    // ---- per channel and step: d, d x, r, and for the end x, dy silu'(z), sigmoid(dt + bias)
#pragma unroll
    for (int j = 0; j < (kEl + 1) / 2; ++j) {
      const int i1 = 2 * j + 1 < kEl ? 2 * j + 1 : 2 * j;
      const float2 raw = make_float2(to_f32(rt[2 * j]) + bias, to_f32(rt[i1]) + bias);
      const float2 d2 = q.softplus ? softplus2_f(raw) : raw;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int i = 2 * j + m, k = tf + i * NR;
        if (i < kEl && busy) {
          // Steps past the end and channels past the group's leave the state, its gradient and the
          // sums over channels alone: d = 0, x = 0, r = 0.
          const bool in = livef && t0 + k < end;
          const float dv = in ? (m ? d2.y : d2.x) : 0.f, xv = in ? to_f32(rx[i]) : 0.f;
          float rv = in ? to_f32(rg[i]) : 0.f, zf = 0.f;
          if (zp) {
            const float z = in ? to_f32(rz[i]) : 0.f, s = sigmoid_f(z), gs = rv * s;
            rv = gs * z;
            zf = gs * fmaf(z, 1.f - s, 1.f);
          }
          const int at = k * Sh::CH + chf;
          sD[at] = dv;
          sU[at] = dv * xv;
          sR[at] = rv;
          sm[Sh::oX + at] = xv;
          sm[Sh::oZ + at] = zf;
          sm[Sh::oS + at] = !in ? 0.f : q.softplus ? sigmoid_f(m ? raw.y : raw.x) : 1.f;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kBC; ++i) {
      const int at = tid + i * Sh::kThreads;
      if (at < T8 * Sh::NP) {
        const float bv = to_f32(rB[i]), cv = to_f32(rC[i]);
        reinterpret_cast<float2*>(sB)[at] = make_float2(bv, bv);
        reinterpret_cast<float2*>(sC)[at] = make_float2(cv, cv);
      }
    }
    __syncthreads();
    if (ck > 0) fetch(t0 - T8);

    // What both directions read of a step: d, d x and r of the lane's four channels in pairs, B
    // and C of its four states, each twice.
    float2 d2, u2, r2, B2[4], C2[4];
    auto read = [&](int k) {
      d2 = *reinterpret_cast<const float2*>(&sD[k * Sh::CH + c0]);
      u2 = *reinterpret_cast<const float2*>(&sU[k * Sh::CH + c0]);
      r2 = *reinterpret_cast<const float2*>(&sR[k * Sh::CH + c0]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 bv = *reinterpret_cast<const float4*>(&sB[2 * (k * Sh::NP + n0) + 4 * i]);
        const float4 cv = *reinterpret_cast<const float4*>(&sC[2 * (k * Sh::NP + n0) + 4 * i]);
        B2[2 * i] = make_float2(bv.x, bv.y); B2[2 * i + 1] = make_float2(bv.z, bv.w);
        C2[2 * i] = make_float2(cv.x, cv.y); C2[2 * i + 1] = make_float2(cv.z, cv.w);
      }
    };
    const bool even = !(lane & 1);
    const int y_at = nt * Sh::kPer + cw * kWC + (lane >> 1);  // of a sum over states

    // ---- forwards through the chunk
#pragma unroll 2
    for (int k = 0; k < T8; ++k) {
      read(k);
      float2 y2, qq[4];
      float dc[4];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const float2 m = __fmul2_rn(d2, A2[s]);
        qq[s] = __fmul2_rn(make_float2(exp2_f(m.x), exp2_f(m.y)), h[s]);
        h[s] = fma2(u2, B2[s], qq[s]);
        y2 = s == 0 ? __fmul2_rn(h[s], C2[s]) : fma2(h[s], C2[s], y2);
        dc[s] = fmaf(r2.y, h[s].y, r2.x * h[s].x);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        *reinterpret_cast<float4*>(hist + (k * 2 + i) * 128) =
            make_float4(qq[2 * i].x, qq[2 * i].y, qq[2 * i + 1].x, qq[2 * i + 1].y);
      const float y = sum_states(y2, lane);
      if (even) sY[y_at + k * Sh::CH] = y;
      const float sc = sum_channels(dc, lane);
      if (!(lane & 4)) sDC[(cw * T8 + k) * Sh::NP + n0 + (lane >> 3)] = sc;
    }
    // The next chunk's kept state, on its way during the walk back.
    if (ck > 0) load_states(q.states + (t0 / T8 - 1) * plane, h);
    // ---- and back
#pragma unroll 2
    for (int k = T8 - 1; k >= 0; --k) {
      read(k);
      float2 v2, w2;
      float db[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 q4 = *reinterpret_cast<const float4*>(hist + (k * 2 + i) * 128);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int s = 2 * i + j;
          const float2 qq = j ? make_float2(q4.z, q4.w) : make_float2(q4.x, q4.y);
          const float2 m = __fmul2_rn(d2, A2[s]);
          const float2 a = make_float2(exp2_f(m.x), exp2_f(m.y));
          const float2 et = fma2(r2, C2[s], e[s]);
          const float2 eq = __fmul2_rn(et, qq);
          dA[s] = fma2(eq, d2, dA[s]);
          w2 = s == 0 ? __fmul2_rn(eq, A2[s]) : fma2(eq, A2[s], w2);
          v2 = s == 0 ? __fmul2_rn(et, B2[s]) : fma2(et, B2[s], v2);
          db[s] = fmaf(et.y, u2.y, et.x * u2.x);
          e[s] = __fmul2_rn(a, et);
        }
      }
      const float v = sum_states(v2, lane), w = sum_states(w2, lane);
      if (even) {
        sV[y_at + k * Sh::CH] = v;
        sW[y_at + k * Sh::CH] = w;
      }
      const float sb = sum_channels(db, lane);
      if (!(lane & 4)) sDB[(cw * T8 + k) * Sh::NP + n0 + (lane >> 3)] = sb;
    }
    __syncthreads();

    // ---- per channel and step: the gradients of the inputs
    T* const dx0 = dxp + t0 * q.dx_t;
    T* const dt0 = dtp + t0 * q.ddt_t;
    T* const dz0 = dzp ? dzp + t0 * q.dz_t : nullptr;
    const bool all = t0 + T8 <= hi;
#pragma unroll
    for (int i = 0; i < kEl; ++i) {
      const int k = tf + i * NR;
      if (!busy || (!all && t0 + k >= hi)) break;
      const int at = k * Sh::CH + chf;
      float y = sY[at], v = sV[at], w = sW[at];
#pragma unroll
      for (int m = 1; m < NT; ++m) {
        y += sY[m * Sh::kPer + at];
        v += sV[m * Sh::kPer + at];
        w += sW[m * Sh::kPer + at];
      }
      const float xv = sm[Sh::oX + at], rv = sR[at];
      const float ddt = sm[Sh::oS + at] * fmaf(w, kLn2, xv * v);
      dskip = fmaf(rv, xv, dskip);
      dbias += ddt;
      if (livef) {
        *pick(dx0 + i * NR * q.dx_t, q.dx_t) = from_f32<T>(fmaf(sD[at], v, skip * rv));
        *pick(dt0 + i * NR * q.ddt_t, q.ddt_t) = from_f32<T>(ddt);
        if (dzp) *pick(dz0 + i * NR * q.dz_t, q.dz_t) = from_f32<T>(sm[Sh::oZ + at] * fmaf(skip, xv, y));
      }
    }
    for (int i = tid; i < T8 * Sh::NP; i += Sh::kThreads) {
      const int k = i / Sh::NP, n = i % Sh::NP;
      if (t0 + k >= hi || n >= q.N) continue;
      float vb = 0.f, vc = 0.f;
#pragma unroll
      for (int m = 0; m < CW; ++m) {
        vb += sDB[m * T8 * Sh::NP + i];
        vc += sDC[m * T8 * Sh::NP + i];
      }
      put_bc(t0 + k, n, vb, vc);
    }
    __syncthreads();
  }

  // ---- what leaves the split
  float* params = pl.params + (static_cast<size_t>(split) * q.B + b) * q.D * (q.N + 2);
#pragma unroll
  for (int c = 0; c < kCL; ++c) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (!in_state(c, s)) continue;
      if (split == 0 && q.dh0) q.dh0[s_at + c * q.N + s] = c ? e[s].y : e[s].x;
      params[static_cast<size_t>(d_base + t_base + c0 + c) * (q.N + 2) + n0 + s] = c ? dA[s].y : dA[s].x;
    }
  }
  // The threads of a channel, in order (the chunk loop ended with a barrier).
  if (busy) {
    sD[tid] = dskip;
    sU[tid] = dbias;
  }
  __syncthreads();
  if (tid < Sh::CH && livef) {
    float sk = 0.f, bi = 0.f;
#pragma unroll
    for (int m = 0; m < (NR < T8 ? NR : T8); ++m) {
      sk += sD[tid + m * Sh::CH];
      bi += sU[tid + m * Sh::CH];
    }
    params[static_cast<size_t>(d0 + tid) * (q.N + 2) + q.N] = sk;
    params[static_cast<size_t>(d0 + tid) * (q.N + 2) + q.N + 1] = bi;
  }
}

// dB and dC: the channel tiles' partial sums added in tile order, rounded once.
template <typename T>
__global__ void __launch_bounds__(256) scan_bc_kernel(const float* pB, const float* pC, int tiles,
                                                      size_t count, T* dB, T* dC) {
  grid_dep_launch_dependents();
  grid_dep_wait();
  const float* p = blockIdx.y ? pC : pB;
  T* out = blockIdx.y ? dC : dB;
  for (size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x; i < count;
       i += static_cast<size_t>(gridDim.x) * 256) {
    float s = p[i];
    for (int k = 1; k < tiles; ++k) s += p[k * count + i];
    out[i] = from_f32<T>(s);
  }
}

// ---- host side ----

template <typename F>
cudaError_t by_tiles(int N, F&& f) {
  using std::integral_constant;
  if (N <= 16) return f(integral_constant<int, 4>{}, integral_constant<int, 1>{});
  if (N <= 32) return f(integral_constant<int, 2>{}, integral_constant<int, 2>{});
  if (N <= 64) return f(integral_constant<int, 1>{}, integral_constant<int, 4>{});
  return f(integral_constant<int, 1>{}, integral_constant<int, 8>{});
}

struct BwdLayout {
  ScanSplit sp;
  int tiles;          // channel tiles per group
  size_t params, bc, carry, total;  // offsets in floats
};

BwdLayout bwd_layout(const ScanCall& q) {
  BwdLayout L{};
  int ch = 32;
  (void)by_tiles(q.N, [&](auto CW, auto NT) {
    ch = Shape<decltype(CW)::value, decltype(NT)::value>::CH;
    return cudaSuccess;
  });
  L.sp = scan_split(q, 152 * 8);  // eight warps an SM fill it
  L.tiles = (q.D / q.G + ch - 1) / ch;
  auto up = [](size_t v) { return (v + 3) & ~static_cast<size_t>(3); };
  L.params = 0;
  L.bc = up(static_cast<size_t>(L.sp.splits) * q.B * q.D * (q.N + 2));
  const size_t bc = static_cast<size_t>(L.tiles) * q.K * q.B * q.G * q.N;
  L.carry = L.bc + (L.tiles > 1 ? 2 * up(bc) : 0);
  L.total = L.carry + scan_carry_floats(q, L.sp);
  return L;
}

template <typename T, int CW, int NT>
cudaError_t run_bwd(const ScanCall& q, const BwdLayout& L, cudaStream_t s) {
  using Sh = Shape<CW, NT>;
  static_assert(Sh::kRows <= T8 ? Sh::kThreads <= Sh::kPer : true, "the last sums fit the per-channel values");
  constexpr size_t smem = Sh::kFloats * sizeof(float);
  const cudaError_t e = cudaFuncSetAttribute(scan_bwd_kernel<T, CW, NT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  BwdPlan pl{};
  pl.per_group = q.D / q.G;
  pl.tiles_per_group = L.tiles;
  pl.steps = L.sp.steps;
  pl.carry = L.sp.splits > 1 ? q.ws + L.carry : nullptr;
  pl.params = q.ws + L.params;
  const size_t bc = static_cast<size_t>(L.tiles) * q.K * q.B * q.G * q.N;
  if (L.tiles > 1) {
    pl.pB = q.ws + L.bc;
    pl.pC = pl.pB + ((bc + 3) & ~static_cast<size_t>(3));
  }
  LaunchCfg c;
  c.grid = dim3(L.tiles * q.G, q.B, L.sp.splits);
  c.block = dim3(Sh::kThreads);
  c.smem = smem;
  c.stream = s;
  return launch(c, scan_bwd_kernel<T, CW, NT>, q, pl);
}

template <typename T>
cudaError_t bwd_all(const ScanCall& q, cudaStream_t s) {
  const BwdLayout L = bwd_layout(q);
  cudaError_t e = cudaSuccess;
  if (L.sp.splits > 1) e = scan_carry_launch(q, L.sp, true, q.ws + L.carry, s);
  if (e == cudaSuccess)
    e = by_tiles(q.N, [&](auto CW, auto NT) {
      return run_bwd<T, decltype(CW)::value, decltype(NT)::value>(q, L, s);
    });
  if (e == cudaSuccess && L.tiles > 1) {
    const size_t count = static_cast<size_t>(q.K) * q.B * q.G * q.N;
    const size_t bc = static_cast<size_t>(L.tiles) * count;
    const float* pB = q.ws + L.bc;
    const float* pC = pB + ((bc + 3) & ~static_cast<size_t>(3));
    LaunchCfg c;
    const size_t blocks = (count + 255) / 256;
    c.grid = dim3(static_cast<unsigned>(blocks < 152 * 16 ? blocks : 152 * 16), 2);
    c.block = dim3(256);
    c.stream = s;
    c.pdl = true;
    e = launch(c, scan_bc_kernel<T>, pB, pC, L.tiles, count, static_cast<T*>(q.dB),
               static_cast<T*>(q.dC));
  }
  if (e == cudaSuccess)
    e = reduce_axis0_rows_launch(q.ws + L.params, L.sp.splits * q.B, q.D * (q.N + 2), q.N + 2, q.N,
                                 q.dA, q.dskip, s, true, q.ddt_bias);
  return e;
}

}  // namespace

size_t scan_bwd_ws_floats(const ScanCall& q) { return bwd_layout(q).total; }

cudaError_t scan_bwd_launch(const ScanCall& q, cudaStream_t s) {
  return q.bf16 ? bwd_all<__nv_bfloat16>(q, s) : bwd_all<float>(q, s);
}

}  // namespace cfc
