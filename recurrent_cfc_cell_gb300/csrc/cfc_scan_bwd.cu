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
// The forward pass kept the state before every kScanPeriod-th (8th) step; the pass walks chunks of
// that many steps from the last, and a chunk in two halves of four steps, the later one first.  A
// lane holds one channel's four states (its arithmetic in packed pairs) and goes forwards through
// the half (the sums with h_t: y, dC), keeping a_t and q_t of its four steps in registers, and then
// backwards (everything with e_t); the later half's first state is formed again from the chunk's
// kept one.  Four lanes hold a channel's 16 states and a warp eight channels at a time; it walks
// over IT such groups for each half, with the half's B and C and the sums dB and dC in registers, so
// that the sums over channels cross lanes only once per half.  The sums over states (y, e B, e A q)
// cross four lanes, three shuffles each for four steps of eight channels.  e and dA of a channel
// wait in shared memory between its halves (so dA is added four steps at a time).
//
// What a step needs per channel (d, x, r and the gate's and softplus's derivatives) is formed once
// per chunk, a thread up to eight steps of a channel.  NT warps side by side hold up to 16 NT states,
// CW warps 8 IT CW channels.  Sums over warps, channel tiles, sequences and splits are added in a
// fixed order (shared memory, then a merge), without atomics.
//
// Bound by instruction issue: a state's step takes 12 multiply-adds and an exponential and a half, and
// 512 of them with what their 32 channels need are 399 instructions, issued at 0.55 a clock and
// scheduler with eight warps an SM (254 registers a thread; 168 or 146 spill, and cost more than the
// warps they allow bring: 933 and 945 us).  Measured on GB300 at 64 x 512 steps x 1024 channels x 16
// states, bf16: 766 us (393 us for 38 sequences, which fill the SMs evenly; 64 leave a half-empty
// second wave).  History: 2008 us with four channels times four states a lane and q_t of a chunk in
// shared memory; 920 us with packed arithmetic and loads in flight; 834 us with half that tile;
// 823 us in this form, whose sums over channels and shared-memory traffic are a third; 766 us with
// the uniform choices (gate, softplus, whole chunks) made once per chunk.
#include "cfc_kernels.h"
#include "cfc_launch.cuh"
#include "cfc_trunk.cuh"
#include "cfc_trunk_kernels.h"

namespace cfc {
namespace {

constexpr int T8 = kScanPeriod;
constexpr float kLn2 = 0.6931471805599453f;

constexpr int kHalf = T8 / 2;

// Place of a half (four steps) of a channel among [channel][step] values: the halves of every other
// four channels change places, so that eight channels' sixteen bytes fall in different banks.
__device__ __forceinline__ int half_at(int ch, int half) {
  return ch * T8 + ((half ^ (ch >> 2 & 1)) << 2);
}

template <int CW, int NT, int IT>
struct Shape {
  static constexpr int kWarps = CW * NT, kThreads = 32 * kWarps, CH = 8 * IT * CW, NP = 16 * NT;
  static constexpr int kSt = NT * CH * 16;       // one value per (channel, state)
  static constexpr int kRow = CH * T8;           // one value per (channel, step)
  // Dynamic shared memory, in floats.
  static constexpr int oE = 0, oDA = oE + kSt, oZ = oDA + kSt, oS = oZ + kRow;
  static constexpr int oY = oS + kRow, oV = oY + NT * kRow, oW = oV + NT * kRow;
  static constexpr int oDB = oW + NT * kRow, oDC = oDB + CW * T8 * NP;
  static constexpr int kFloats = oDC + CW * T8 * NP;
};

// Sum of v[0..3] over the four state lanes (lane bits 0, 1): lane nl keeps v[nl].
__device__ __forceinline__ float sum_states(const float (&v)[4], int lane) {
  const bool hi = lane & 2;
  const float a = (hi ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[2], 2);
  const float b = (hi ? v[3] : v[1]) + __shfl_xor_sync(0xffffffffu, hi ? v[1] : v[3], 2);
  const bool lo = lane & 1;
  return (lo ? b : a) + __shfl_xor_sync(0xffffffffu, lo ? a : b, 1);
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
  float* pA;            // [splits * B][D][N]: dA
  float* pD;            // [splits * B][D][2]: dskip, ddt_bias
  float *pB, *pC;       // [tiles_per_group][K][B][G][N], or null: straight to dB / dC
};

template <typename T, int CW, int NT, int IT>
__global__ void __launch_bounds__(32 * CW * NT) scan_bwd_kernel(const ScanCall q, const BwdPlan pl) {
  using Sh = Shape<CW, NT, IT>;
  extern __shared__ __align__(16) float sm[];
  __shared__ __align__(16) float sD[Sh::kRow], sX[Sh::kRow], sR[Sh::kRow];  // [channel][step]
  __shared__ __align__(16) float sA[Sh::kSt];                               // [nt][channel][16]
  __shared__ __align__(16) float sB[T8 * Sh::NP], sC[T8 * Sh::NP];
  grid_dep_launch_dependents();
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int nt = warp % NT, cw = warp / NT, nl = lane & 3, dl = lane >> 2;
  const int group = blockIdx.x / pl.tiles_per_group, tile = blockIdx.x % pl.tiles_per_group;
  const int b = blockIdx.y, split = blockIdx.z;
  const int len = q.lengths ? min(max(q.lengths[b], 0), q.K) : q.K;
  const int lo = split * pl.steps, hi = min(q.K, lo + pl.steps), end = min(hi, len);
  const size_t plane = static_cast<size_t>(q.B) * q.D * q.N;
  const int d0 = group * pl.per_group + tile * Sh::CH;        // the tile's first channel
  const int count = min(Sh::CH, pl.per_group - tile * Sh::CH);  // its channels

  const T* Bp = static_cast<const T*>(q.Bm) + b * q.Bm_b + static_cast<long long>(group) * q.N;
  const T* Cp = static_cast<const T*>(q.Cm) + b * q.Cm_b + static_cast<long long>(group) * q.N;
  const size_t tile_at = (static_cast<size_t>(b) * q.D + d0) * q.N;  // of the tile in a plane

  // A, e and dA of the tile's channels, zero outside; shared memory [nt][channel][16].
  const float* c_in = pl.carry ? pl.carry + split * plane : q.dh_last;
  for (int i = tid; i < Sh::kSt; i += Sh::kThreads) {
    const int ch = i / 16 % Sh::CH, n = i / (16 * Sh::CH) * 16 + i % 16;
    const bool in = ch < count && n < q.N;
    sA[i] = in ? rate_f(q.A[static_cast<size_t>(d0 + ch) * q.N + n]) : 0.f;
    sm[Sh::oE + i] = in && c_in ? c_in[tile_at + static_cast<size_t>(ch) * q.N + n] : 0.f;
    sm[Sh::oDA + i] = 0.f;
  }

  // The lane's four states of channel ch in the kept plane of the chunk, zero outside.
  const int n0 = nt * 16 + nl * 4;
  const bool quad = q.N % 4 == 0;
  auto kept = [&](const float* p, int ch) {
    float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
    if (ch < count && n0 < q.N) {
      const float* at = p + tile_at + static_cast<size_t>(ch) * q.N + n0;
      if (quad) {
        r = *reinterpret_cast<const float4*>(at);
      } else {
        r.x = at[0];
        if (n0 + 1 < q.N) r.y = at[1];
        if (n0 + 2 < q.N) r.z = at[2];
        if (n0 + 3 < q.N) r.w = at[3];
      }
    }
    return r;
  };

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

  // The per-channel phases: a thread takes PS consecutive steps of one channel, from step k0 of the
  // chunk on.
  constexpr int PS = T8 * Sh::CH / Sh::kThreads;
  static_assert(T8 % PS == 0 && T8 / PS * Sh::CH == Sh::kThreads, "a piece a thread");
  const int ch = Sh::kThreads == Sh::CH ? tid : tid % Sh::CH;
  const int k0 = Sh::kThreads == Sh::CH ? 0 : tid / Sh::CH * PS;
  const bool live = ch < count;
  const float bias = q.dt_bias && live ? q.dt_bias[d0 + ch] : 0.f;
  const float skip = q.skip && live ? q.skip[d0 + ch] : 0.f;
  float dskip = 0.f, dbias = 0.f;
  const T* xr = static_cast<const T*>(q.x) + b * q.x_b + d0;
  const T* tr = static_cast<const T*>(q.dt) + b * q.dt_b + d0;
  const T* zr = q.z ? static_cast<const T*>(q.z) + b * q.z_b + d0 : nullptr;
  const T* gr = static_cast<const T*>(q.dy) + b * q.dy_b + d0;
  T* dxr = static_cast<T*>(q.dx) + b * q.dx_b + d0;
  T* dtr = static_cast<T*>(q.ddt) + b * q.ddt_b + d0;
  T* dzr = q.dz ? static_cast<T*>(q.dz) + b * q.dz_b + d0 : nullptr;

  const int chunks = end > lo ? (end - lo + T8 - 1) / T8 : 0;
  // Steps after the sequence's end: zeros.
  for (int t = lo + chunks * T8; t < hi; ++t) {
    for (int c = tid; c < count; c += Sh::kThreads) {
      dxr[t * q.dx_t + c] = from_f32<T>(0.f);
      dtr[t * q.ddt_t + c] = from_f32<T>(0.f);
      if (dzr) dzr[t * q.dz_t + c] = from_f32<T>(0.f);
    }
    for (int n = tid; n < q.N; n += Sh::kThreads) put_bc(t, n, 0.f, 0.f);
  }

  // A chunk's inputs as they are stored: read while the chunk after it (the one before in this
  // walk) is finished, from the second-level cache, where they were sent for when its sums began.
  // Addresses are a uniform base (sequence, tile, step) plus the thread's own offset.
  constexpr int kBC = (T8 * Sh::NP + Sh::kThreads - 1) / Sh::kThreads;
  const T none = from_f32<T>(0.f);
  const unsigned own = live ? ch : 0;
  const int k0s = live ? k0 : 0;
  auto pick = [&](auto* base, long long stride) {
    if constexpr (Sh::kThreads == Sh::CH) return base + own;
    return base + (own + k0s * stride);
  };
  T rx[PS], rt[PS], rz[PS], rg[PS], rB[kBC], rC[kBC];
  auto fetch_as = [&](int t0, auto all) {
    constexpr bool kAll = decltype(all)::value;  // every step of the chunk and channel counts
    const T *x0 = xr + t0 * q.x_t, *dt0 = tr + t0 * q.dt_t, *g0 = gr + t0 * q.dy_t;
    const T* z0 = zr ? zr + t0 * q.z_t : nullptr;
#pragma unroll
    for (int j = 0; j < PS; ++j) {
      const bool in = kAll || (live && t0 + k0 + j < end);
      rx[j] = in ? *pick(x0 + j * q.x_t, q.x_t) : none;
      rt[j] = in ? *pick(dt0 + j * q.dt_t, q.dt_t) : none;
      rg[j] = in ? *pick(g0 + j * q.dy_t, q.dy_t) : none;
    }
    if (zr) {
#pragma unroll
      for (int j = 0; j < PS; ++j)
        rz[j] = kAll || (live && t0 + k0 + j < end) ? *pick(z0 + j * q.z_t, q.z_t) : none;
    }
#pragma unroll
    for (int i = 0; i < kBC; ++i) {
      const int at = tid + i * Sh::kThreads, k = at / Sh::NP, n = at % Sh::NP;
      const bool in = k < T8 && (kAll || t0 + k < end) && n < q.N;
      rB[i] = in ? (Bp + (t0 + k) * q.Bm_t)[n] : none;
      rC[i] = in ? (Cp + (t0 + k) * q.Cm_t)[n] : none;
    }
  };
  auto whole = [&](int t0) { return count == Sh::CH && t0 + T8 <= end; };
  auto fetch = [&](int t0) {
    if (whole(t0)) fetch_as(t0, std::true_type{});
    else fetch_as(t0, std::false_type{});
  };
  auto send_for = [&](int t0) {
    constexpr int kLine = 128 / sizeof(T), kLines = (Sh::CH + kLine - 1) / kLine;  // of a row
    for (int i = tid; i < 4 * T8 * kLines; i += Sh::kThreads) {
      const int which = i / T8 % 4, at = i / (4 * T8) * kLine;
      const long long t = t0 + i % T8;
      const T* row = which == 0 ? xr + t * q.x_t : which == 1 ? tr + t * q.dt_t
                   : which == 2 ? gr + t * q.dy_t : zr ? zr + t * q.z_t : nullptr;
      if (row != nullptr && at < count) prefetch_l2(row + at);
    }
    const float* p = q.states + (t0 / T8) * plane + tile_at;
    for (int i = tid * 32; i < count * q.N; i += Sh::kThreads * 32) prefetch_l2(p + i);
  };
  // The thread's steps of its channel in a [channel][step] array, FS (up to four) at a time from
  // step k of the chunk on.
  constexpr int FS = PS < kHalf ? PS : kHalf;
  auto put = [&](float* p, int k, const float (&f)[FS]) {
    if constexpr (FS == kHalf) {
      *reinterpret_cast<float4*>(p + half_at(ch, k / kHalf)) = make_float4(f[0], f[1], f[2], f[3]);
    } else {
#pragma unroll
      for (int j = 0; j < FS; ++j) p[half_at(ch, k / kHalf) + k % kHalf + j] = f[j];
    }
  };
  auto get = [&](const float* p, int k, float (&f)[FS]) {
    if constexpr (FS == kHalf) {
      const float4 r = *reinterpret_cast<const float4*>(p + half_at(ch, k / kHalf));
      f[0] = r.x; f[1] = r.y; f[2] = r.z; f[3] = r.w;
    } else {
#pragma unroll
      for (int j = 0; j < FS; ++j) f[j] = p[half_at(ch, k / kHalf) + k % kHalf + j];
    }
  };
  if (chunks > 0) fetch(lo + (chunks - 1) * T8);

  for (int ck = chunks - 1; ck >= 0; --ck) {
    const int t0 = lo + ck * T8;
    const float* const plane_in = q.states + (t0 / T8) * plane;
    const int c_first = cw * IT * 8 + dl;
    float4 next = kept(plane_in, c_first);
    // ---- per channel: d, x, r, and for the end dy silu'(z) and sigmoid(dt + bias)
#pragma unroll
    for (int f = 0; f < PS; f += FS) {
      float dv[FS], xv[FS], rv[FS], zf[FS], sg[FS];
      decide(q.softplus, [&](auto sp) {
#pragma unroll
        for (int j = 0; j < FS; j += 2) {
          const int j1 = j + 1 < FS ? j + 1 : j;
          const float2 raw = make_float2(to_f32(rt[f + j]) + bias, to_f32(rt[f + j1]) + bias);
          float2 d2 = raw;
          if constexpr (decltype(sp)::value) d2 = softplus2_f(raw);
          dv[j1] = d2.y;
          dv[j] = d2.x;
          sg[j1] = decltype(sp)::value ? sigmoid_f(raw.y) : 1.f;
          sg[j] = decltype(sp)::value ? sigmoid_f(raw.x) : 1.f;
        }
      });
      decide(zr != nullptr, [&](auto gate) {
#pragma unroll
        for (int j = 0; j < FS; ++j) {
          xv[j] = to_f32(rx[f + j]);
          rv[j] = to_f32(rg[f + j]);
          zf[j] = 0.f;
          if (decltype(gate)::value) {
            const float z = to_f32(rz[f + j]), s = sigmoid_f(z), gs = rv[j] * s;
            rv[j] = gs * z;
            zf[j] = gs * fmaf(z, 1.f - s, 1.f);
          }
        }
      });
      if (!whole(t0)) {
        // Steps past the end and channels past the group's leave the state, its gradient and the
        // sums alone: d = 0 (x and r were read as 0).
#pragma unroll
        for (int j = 0; j < FS; ++j)
          if (!live || t0 + k0 + f + j >= end) dv[j] = sg[j] = 0.f;
      }
      put(sD, k0 + f, dv);
      put(sX, k0 + f, xv);
      put(sR, k0 + f, rv);
      put(&sm[Sh::oZ], k0 + f, zf);
      put(&sm[Sh::oS], k0 + f, sg);
    }
#pragma unroll
    for (int i = 0; i < kBC; ++i) {
      const int at = tid + i * Sh::kThreads;
      if (at < T8 * Sh::NP) {
        sB[at] = to_f32(rB[i]);
        sC[at] = to_f32(rC[i]);
      }
    }
    if (ck > 0) send_for(t0 - T8);
    __syncthreads();

    // ---- the two halves
#pragma unroll
    for (int half = 1; half >= 0; --half) {
      float2 db[kHalf][2], dc[kHalf][2];
#pragma unroll
      for (int j = 0; j < kHalf; ++j)
#pragma unroll
        for (int p = 0; p < 2; ++p) db[j][p] = dc[j][p] = make_float2(0.f, 0.f);
      // B or C of the lane's states at step k of the chunk (a broadcast: one cycle of shared
      // memory, and registers free for another warp).
      auto bc = [&](const float* p, int k, float2 (&f)[2]) {
        const float4 r = *reinterpret_cast<const float4*>(p + k * Sh::NP + n0);
        f[0] = make_float2(r.x, r.y);
        f[1] = make_float2(r.z, r.w);
      };
#pragma unroll 1
      for (int it = 0; it < IT; ++it) {
        const int cl = c_first + it * 8;  // the lane's channel
        const int st = (nt * Sh::CH + cl) * 16 + nl * 4;
        float2 h[2] = {make_float2(next.x, next.y), make_float2(next.z, next.w)};
        // The next group's kept state (after the later half's last, the earlier half's first).
        if (it + 1 < IT || half) next = kept(plane_in, it + 1 < IT ? cl + 8 : c_first);
        const float4 a4 = *reinterpret_cast<const float4*>(&sA[st]);
        const float2 A2[2] = {make_float2(a4.x, a4.y), make_float2(a4.z, a4.w)};
        if (half) {
          const float4 d4 = *reinterpret_cast<const float4*>(&sD[half_at(cl, 0)]);
          const float4 x4 = *reinterpret_cast<const float4*>(&sX[half_at(cl, 0)]);
          const float dv[4] = {d4.x, d4.y, d4.z, d4.w}, xv[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
          for (int j = 0; j < kHalf; ++j) {
            const float u = dv[j] * xv[j];
            float2 B0[2];
            bc(sB, j, B0);
#pragma unroll
            for (int p = 0; p < 2; ++p)
              h[p] = fma2(decay2_f(dv[j], A2[p]), h[p], __fmul2_rn(make_float2(u, u), B0[p]));
          }
        }
        const int at = half_at(cl, half);
        const float4 d4 = *reinterpret_cast<const float4*>(&sD[at]);
        const float4 x4 = *reinterpret_cast<const float4*>(&sX[at]);
        const float4 r4 = *reinterpret_cast<const float4*>(&sR[at]);
        const float4 e4 = *reinterpret_cast<const float4*>(&sm[Sh::oE + st]);
        const float4 da4 = *reinterpret_cast<const float4*>(&sm[Sh::oDA + st]);
        const float dv[4] = {d4.x, d4.y, d4.z, d4.w}, rv[4] = {r4.x, r4.y, r4.z, r4.w};
        const float uv[4] = {d4.x * x4.x, d4.y * x4.y, d4.z * x4.z, d4.w * x4.w};
        // Forwards.
        float2 a[kHalf][2], qq[kHalf][2];
        float y[4], v[4], w[4];
#pragma unroll
        for (int j = 0; j < kHalf; ++j) {
          const float2 u2 = make_float2(uv[j], uv[j]);
          const float2 r2 = make_float2(rv[j], rv[j]);
          float2 y2, Bv[2], Cv[2];
          bc(sB, half * kHalf + j, Bv);
          bc(sC, half * kHalf + j, Cv);
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            a[j][p] = decay2_f(dv[j], A2[p]);
            qq[j][p] = __fmul2_rn(a[j][p], h[p]);
            h[p] = fma2(u2, Bv[p], qq[j][p]);
            y2 = p ? fma2(h[p], Cv[p], y2) : __fmul2_rn(h[p], Cv[p]);
            dc[j][p] = fma2(r2, h[p], dc[j][p]);
          }
          y[j] = y2.x + y2.y;
        }
        const float ys = sum_states(y, lane);
        // And back.
        float2 e[2] = {make_float2(e4.x, e4.y), make_float2(e4.z, e4.w)};
        float2 dA[2];
#pragma unroll
        for (int j = kHalf - 1; j >= 0; --j) {
          const float2 d2 = make_float2(dv[j], dv[j]), u2 = make_float2(uv[j], uv[j]);
          const float2 r2 = make_float2(rv[j], rv[j]);
          float2 v2, w2, Bv[2], Cv[2];
          bc(sB, half * kHalf + j, Bv);
          bc(sC, half * kHalf + j, Cv);
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const float2 et = fma2(r2, Cv[p], e[p]);
            const float2 eq = __fmul2_rn(et, qq[j][p]);
            dA[p] = j == kHalf - 1 ? __fmul2_rn(eq, d2) : fma2(eq, d2, dA[p]);
            w2 = p ? fma2(eq, A2[p], w2) : __fmul2_rn(eq, A2[p]);
            v2 = p ? fma2(et, Bv[p], v2) : __fmul2_rn(et, Bv[p]);
            db[j][p] = fma2(et, u2, db[j][p]);
            e[p] = __fmul2_rn(a[j][p], et);
          }
          v[j] = v2.x + v2.y;
          w[j] = w2.x + w2.y;
        }
        *reinterpret_cast<float4*>(&sm[Sh::oE + st]) = make_float4(e[0].x, e[0].y, e[1].x, e[1].y);
        *reinterpret_cast<float4*>(&sm[Sh::oDA + st]) =
            make_float4(da4.x + dA[0].x, da4.y + dA[0].y, da4.z + dA[1].x, da4.w + dA[1].y);
        const int out = nt * Sh::kRow + at + nl;
        sm[Sh::oY + out] = ys;
        sm[Sh::oV + out] = sum_states(v, lane);
        sm[Sh::oW + out] = sum_states(w, lane);
      }
      // The half's dB and dC over the warp's channels.
#pragma unroll
      for (int j = 0; j < kHalf; ++j) {
        const float vb[4] = {db[j][0].x, db[j][0].y, db[j][1].x, db[j][1].y};
        const float vc[4] = {dc[j][0].x, dc[j][0].y, dc[j][1].x, dc[j][1].y};
        const float sb = sum_channels(vb, lane), sc = sum_channels(vc, lane);
        if (!(lane & 4)) {
          const int at = (cw * T8 + half * kHalf + j) * Sh::NP + n0 + (lane >> 3);
          sm[Sh::oDB + at] = sb;
          sm[Sh::oDC + at] = sc;
        }
      }
    }
    __syncthreads();
    if (ck > 0) fetch(t0 - T8);

    // ---- per channel and step: the gradients of the inputs.  (A thread reads back what it formed
    // itself, and the sums; the next chunk's values may follow without a barrier.)
    const bool all_out = count == Sh::CH && t0 + T8 <= hi;
#pragma unroll 1
    for (int f = 0; f < PS; f += FS) {
      const int k = k0 + f;
      float y[FS], v[FS], w[FS], dv[FS], xv[FS], rv[FS], zf[FS], sg[FS];
      get(&sm[Sh::oY], k, y);
      get(&sm[Sh::oV], k, v);
      get(&sm[Sh::oW], k, w);
#pragma unroll
      for (int m = 1; m < NT; ++m) {
        float o[FS];
        get(&sm[Sh::oY + m * Sh::kRow], k, o);
#pragma unroll
        for (int j = 0; j < FS; ++j) y[j] += o[j];
        get(&sm[Sh::oV + m * Sh::kRow], k, o);
#pragma unroll
        for (int j = 0; j < FS; ++j) v[j] += o[j];
        get(&sm[Sh::oW + m * Sh::kRow], k, o);
#pragma unroll
        for (int j = 0; j < FS; ++j) w[j] += o[j];
      }
      get(sD, k, dv);
      get(sX, k, xv);
      get(sR, k, rv);
      get(&sm[Sh::oZ], k, zf);
      get(&sm[Sh::oS], k, sg);
      T *dx0 = dxr + (t0 + f) * q.dx_t, *dt0 = dtr + (t0 + f) * q.ddt_t;
      T* dz0 = dzr ? dzr + (t0 + f) * q.dz_t : nullptr;
      float ddt[FS];
#pragma unroll
      for (int j = 0; j < FS; ++j) {
        ddt[j] = sg[j] * fmaf(w[j], kLn2, xv[j] * v[j]);
        dskip = fmaf(rv[j], xv[j], dskip);
        dbias += ddt[j];
      }
      decide(all_out, [&](auto all) {
        auto each = [&](auto&& f1) {
#pragma unroll
          for (int j = 0; j < FS; ++j)
            if (decltype(all)::value || (live && t0 + k + j < hi)) f1(j);
        };
        each([&](int j) {
          *pick(dx0 + j * q.dx_t, q.dx_t) = from_f32<T>(fmaf(dv[j], v[j], skip * rv[j]));
          *pick(dt0 + j * q.ddt_t, q.ddt_t) = from_f32<T>(ddt[j]);
        });
        if (dzr)
          each([&](int j) {
            *pick(dz0 + j * q.dz_t, q.dz_t) = from_f32<T>(zf[j] * fmaf(skip, xv[j], y[j]));
          });
      });
    }
    for (int i = tid; i < T8 * Sh::NP; i += Sh::kThreads) {
      const int k = i / Sh::NP, n = i % Sh::NP;
      if (t0 + k >= hi || n >= q.N) continue;
      float vb = 0.f, vc = 0.f;
#pragma unroll
      for (int m = 0; m < CW; ++m) {
        vb += sm[Sh::oDB + m * T8 * Sh::NP + i];
        vc += sm[Sh::oDC + m * T8 * Sh::NP + i];
      }
      put_bc(t0 + k, n, vb, vc);
    }
  }

  // ---- what leaves the split
  const size_t part = static_cast<size_t>(split) * q.B + b;
  float* pA = pl.pA + part * q.D * q.N;
  float* pD = pl.pD + (part * q.D + d0) * 2;
  __syncthreads();
  for (int i = tid; i < Sh::kSt; i += Sh::kThreads) {
    const int ch = i / 16 % Sh::CH, n = i / (16 * Sh::CH) * 16 + i % 16;
    if (ch >= count || n >= q.N) continue;
    if (split == 0 && q.dh0) q.dh0[tile_at + static_cast<size_t>(ch) * q.N + n] = sm[Sh::oE + i];
    pA[static_cast<size_t>(d0 + ch) * q.N + n] = sm[Sh::oDA + i];
  }
  // The pieces of a channel, in order.
  sD[tid] = dskip;
  sX[tid] = dbias;
  __syncthreads();
  if (tid < count) {
    float sk = 0.f, bi = 0.f;
#pragma unroll
    for (int m = 0; m < T8 / PS; ++m) {
      sk += sD[tid + m * Sh::CH];
      bi += sX[tid + m * Sh::CH];
    }
    pD[2 * tid] = sk;
    pD[2 * tid + 1] = bi;
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

// f(shape): warps along channels and states, groups of eight channels a warp.  With many channels a
// warp takes four groups, so that the sums over channels, B and C serve more (32 x 128 steps x 1024
// channels x 16 states: 112 us, 130 us with two); with fewer two, so that there are more warps
// (16 x 128 x 1024 x 16: 68 us, 83 us with four; 32 x 64 x 256 x 32: 40 and 44 us); and one where
// even the split steps leave SMs idle, so that a step takes less (4 x 128 x 256 x 16: 22.8 us, 24.9 us
// with two; 4 x 1024 x 256 x 16: 61.7 and 57.4 us).
template <typename F>
cudaError_t by_tiles(const ScanCall& q, F&& f) {
  const long long groups = static_cast<long long>(q.B) * q.G * ((q.D / q.G + 7) / 8) * ((q.N + 15) / 16);
  const bool few = groups < 152LL * 12 * 2, very_few = groups * q.K < 152LL * 256;
  if (q.N <= 16)
    return very_few ? f(Shape<4, 1, 1>{}) : few ? f(Shape<4, 1, 2>{}) : f(Shape<4, 1, 4>{});
  if (q.N <= 32)
    return very_few ? f(Shape<2, 2, 1>{}) : few ? f(Shape<2, 2, 2>{}) : f(Shape<2, 2, 4>{});
  if (q.N <= 64) return few ? f(Shape<1, 4, 2>{}) : f(Shape<1, 4, 4>{});
  return f(Shape<1, 8, 4>{});
}
template <int CW, int NT, int IT>
constexpr int tile_channels(Shape<CW, NT, IT>) { return Shape<CW, NT, IT>::CH; }

struct BwdLayout {
  ScanSplit sp;
  int tiles;          // channel tiles per group
  size_t pA, pD, spare, bc, carry, total;  // offsets in floats
};

BwdLayout bwd_layout(const ScanCall& q) {
  BwdLayout L{};
  int ch = 32;
  (void)by_tiles(q, [&](auto sh) {
    ch = tile_channels(sh);
    return cudaSuccess;
  });
  L.tiles = (q.D / q.G + ch - 1) / ch;
  // 4 x 128 x 256 x 16: 25 us in eight splits of 16 steps, 50 us unsplit; 15 x 209 x 28 x 4: 26 and
  // 85 us; 4 x 64 x 908 x 24: 39 and 34 us.
  L.sp = scan_split(q.K, static_cast<long long>(q.B) * q.G * L.tiles, 152 * 4, 16, 96);
  auto up = [](size_t v) { return (v + 3) & ~static_cast<size_t>(3); };
  const size_t parts = static_cast<size_t>(L.sp.splits) * q.B;
  L.pA = 0;
  L.pD = up(parts * q.D * q.N);
  L.spare = L.pD + up(parts * q.D * 2);  // for dskip and ddt_bias where they are not wanted
  L.bc = L.spare + up(static_cast<size_t>(q.D) * 2);
  const size_t bc = static_cast<size_t>(L.tiles) * q.K * q.B * q.G * q.N;
  L.carry = L.bc + (L.tiles > 1 ? 2 * up(bc) : 0);
  L.total = L.carry + scan_carry_floats(q, L.sp);
  return L;
}

template <typename T, int CW, int NT, int IT>
cudaError_t run_bwd(const ScanCall& q, const BwdLayout& L, Shape<CW, NT, IT>, cudaStream_t s) {
  using Sh = Shape<CW, NT, IT>;
  constexpr size_t smem = Sh::kFloats * sizeof(float);
  cudaError_t e = cudaFuncSetAttribute(scan_bwd_kernel<T, CW, NT, IT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(scan_bwd_kernel<T, CW, NT, IT>,
                             cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
  if (e != cudaSuccess) return e;
  BwdPlan pl{};
  pl.per_group = q.D / q.G;
  pl.tiles_per_group = L.tiles;
  pl.steps = L.sp.steps;
  pl.carry = L.sp.splits > 1 ? q.ws + L.carry : nullptr;
  pl.pA = q.ws + L.pA;
  pl.pD = q.ws + L.pD;
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
  return launch(c, scan_bwd_kernel<T, CW, NT, IT>, q, pl);
}

template <typename T>
cudaError_t bwd_all(const ScanCall& q, cudaStream_t s) {
  const BwdLayout L = bwd_layout(q);
  cudaError_t e = cudaSuccess;
  if (L.sp.splits > 1) e = scan_carry_launch(q, L.sp, true, q.ws + L.carry, s);
  if (e == cudaSuccess)
    e = by_tiles(q, [&](auto sh) { return run_bwd<T>(q, L, sh, s); });
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
    e = reduce_axis0_pair_launch(q.ws + L.pD, L.sp.splits * q.B, q.D * 2, 2, 1,
                                 q.dskip ? q.dskip : q.ws + L.spare,
                                 q.ddt_bias ? q.ddt_bias : q.ws + L.spare + q.D, q.ws + L.pA,
                                 L.sp.splits * q.B, q.D * q.N, q.dA, s, true);
  return e;
}

}  // namespace

size_t scan_bwd_ws_floats(const ScanCall& q) { return bwd_layout(q).total; }

cudaError_t scan_bwd_launch(const ScanCall& q, cudaStream_t s) {
  return q.bf16 ? bwd_all<__nv_bfloat16>(q, s) : bwd_all<float>(q, s);
}

}  // namespace cfc
