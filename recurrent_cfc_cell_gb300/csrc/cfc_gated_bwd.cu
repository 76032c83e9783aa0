// cfc_gated_bwd.cu -- the gradients of the gated linear recurrence (cfc_gated.cuh says how the steps
// are divided; here the runs follow one another backwards in time).
//
//   g_t = dL/dh_t = dy_t silu(z_t) + f_{t+1} g_{t+1}
//   dx_t = g_t (1 - f_t),   df_t = g_t (h_{t-1} - x_t) f_t (1 - f_t)   (of the logit)
//   dz_t = dy_t h_t silu'(z_t),   dbias = sum df,   dh0 = f_0 g_0
//
// h is formed again within each run from the state that the forward pass kept at its start.
//
// Rounds are bound by memory: 64 x 1024 steps x 1536 channels bf16 249 us (5.9 TB/s), 64 x 512 x 1024
// fp32 151 us (6.3 TB/s).  What is kept in 8 bits is bound by the instructions and their latency (131 a
// warp for a step of 64 channels, 107 for inputs as they are; 2.5 of 4 a cycle from 3.3 warps a
// scheduler): 16 x 2048 x 2048 bf16 203 us with y formed again.  128 registers hold a run's factors
// between the two ways through it (gather, finish), so that nothing is computed twice.
#include "cfc_gated.cuh"

namespace cfc {
namespace {

template <typename T, int V, bool KEEP>
struct Input {  // a run of an activation that the backward pass reads as it is, or in 8 bits
  RawV<T, V> raw[kGS];
  __device__ __forceinline__ void load(int k, const T* p, const Held8&, const HeldAt&) {
    raw[k].load(p);
  }
};
template <typename T, int V>
struct Input<T, V, true> {
  RawHeld2 raw[kGS];
  __device__ __forceinline__ void load(int k, const T*, const Held8& h, const HeldAt& at) {
    raw[k].load(h, at);
  }
};
// One channel a lane: a warp's channels are one block, whose scales lanes hold for each other.
template <typename T>
struct Input<T, 1, true> {
  struct Code {
    uint8_t v;
    __device__ __forceinline__ void clear() { v = 0; }
  } raw[kGS];
  __device__ __forceinline__ void load(int k, const T*, const Held8& h, const HeldAt& at) {
    raw[k].v = h.codes[at.code];
  }
  __device__ __forceinline__ Fv<1> get(int k, float up) const {
    return Fv<1>(held_values2(raw[k].v).x * __shfl_sync(0xffffffffu, up, k));
  }
};

// Rounds on their way to shared memory, and the one being worked on, of a warp: dy, and x, f and z where
// IN, the first ones as kept where they are.
template <typename T, bool Z, bool KEEP, GatedPath PATH>
struct Ring {
  static constexpr bool IN = !KEEP || PATH == kSixteens;
  using Run = RingRun<sizeof(T), PATH == kSixteens ? 16 : 2 * sizeof(T)>;
  using In = std::conditional_t<KEEP, RingRun<1, 8>, Run>;
  static constexpr int kStages = sizeof(T) == 2 ? 3 : 2;
  static constexpr int kInput = In::kBytes;
  static constexpr int kStage = Run::kBytes + (IN ? (Z ? 3 : 2) * kInput : 0), kWarp = kStages * kStage;
};

// The scales of a run of 32 V channels in 8 bits: lane V k + i holds the one of step k's block i.
template <int V>
__device__ __forceinline__ uint32_t run_scales(const Held8& h, const GatedCall& q, int b, int tile,
                                               int t0, int len) {
  const int lane = threadIdx.x % 32, t = t0 + lane / V, block = V * tile + lane % V;
  const bool in = lane < V * kGS && t < len && block < held_blocks(q.D);
  return in ? h.scales[(static_cast<size_t>(t) * q.B + b) * held_blocks(q.D) + block] : 1u;
}
__device__ __forceinline__ Fv<2> ring_get_held(const char* run, int k, float up) {
  const int lane = threadIdx.x % 32;
  Fv<2> v;
  v.v = held_values2(reinterpret_cast<const uint16_t*>(run + k * 64)[lane]);
  return v * Fv<2>(__shfl_sync(0xffffffffu, up, 2 * k + lane / 16));
}

// kRounds: grid (tiles, B), CTAs of any number of warps.  kSummary and kSegments: grid (tiles x CTAs of
// segments, B), kGatedWarps warps.
template <typename T, bool Z, bool KEEP, GatedPath PATH, GatedMode MODE>
__global__ void __launch_bounds__(32 * kGatedWarps, 2)
    gated_bwd_kernel(const GatedCall q, const GatedShape sh, float* dbias) {
  extern __shared__ __align__(128) char shared[];  // the rounds on their way, the exchange
  constexpr bool RING = PATH != kSingles;
  constexpr int V = path_v(PATH);
  using Rg = Ring<T, Z, KEEP, PATH>;
  constexpr bool IN = RING && Rg::IN;        // x, f and z come through the ring
  constexpr bool AHEAD = !RING;              // everything comes to registers, a run ahead
  constexpr bool SCALES = KEEP && (IN || !RING);  // scales come a run ahead, a lane one of them
  grid_dep_launch_dependents();
  const int warps = blockDim.x / 32, w = threadIdx.x / 32;
  const Exchange<V> ex{shared + (RING ? warps * Rg::kWarp : 0), warps};
  const int ctas = MODE == kRounds ? 1 : sh.ctas;
  const int b = blockIdx.y, K = q.K, tile = blockIdx.x / ctas, cta = blockIdx.x % ctas;
  const Channels<V> ch(tile, q.D);
  const int len = q.lengths ? min(max(q.lengths[b], 0), K) : K;
  const int from = RING ? tile * 64 : ch.d;
  const T* const xp = KEEP ? nullptr : static_cast<const T*>(q.x) + b * q.x_b + from;
  const T* const fp = KEEP ? nullptr : static_cast<const T*>(q.f) + b * q.f_b + from;
  const T* const zp = KEEP || !Z ? nullptr : static_cast<const T*>(q.z) + b * q.z_b + from;
  const T* const dyp = static_cast<const T*>(q.dy) + b * q.dy_b + from;
  T* const dxp = static_cast<T*>(q.dx) + b * q.dx_b + ch.d;
  T* const dfp = static_cast<T*>(q.df) + b * q.df_b + ch.d;
  T* const dzp = Z ? static_cast<T*>(q.dz) + b * q.dz_b + ch.d : nullptr;
  T* const yp = q.y ? static_cast<T*>(q.y) + b * q.y_b + ch.d : nullptr;
  const Fv<V> bias2 = load_par_v<V>(q.bias, ch) * Fv<V>(kLog2e);
  Fv<V> dsum(0.f);
  // The warp's steps, `round` of them from a run to its next one; where its first one begins, and the
  // run that it takes first, the last one.
  const int round = MODE == kRounds ? warps * kGS : kGS;
  const int first = MODE == kRounds ? w * kGS : (cta * kGatedWarps + w) * sh.steps;
  const int end = MODE == kRounds ? K : min(first + sh.steps, K);
  // Rounds are taken from the last to the first; a segment that there is not has none.
  const int last = MODE == kRounds ? (K - 1) / round : first < end ? (end - first - 1) / round : -1;
  const Segments<V> seg(q.ws, MODE == kRounds ? 0 : gridDim.x / ctas, tile, b, ctas);

  char* const mine = shared + w * Rg::kWarp;
  RawV<float, V> start_next;
  uint32_t sx_next = 1u, sf_next = 1u, sz_next = 1u;
  typename Rg::Run rdy;
  typename Rg::In rx, rf, rz;
  const int left = q.D - tile * 64;
  int fetched = last * round + first;  // the first step of the run that is fetched next
  const long long kept_t = static_cast<long long>(q.B) * q.D;
  const long long xs = KEEP ? kept_t : q.x_t, fs = KEEP ? kept_t : q.f_t, zs = KEEP ? kept_t : q.z_t;
  if constexpr (RING) {
    rdy.start(dyp, q.dy_t, first, left);
  }
  if constexpr (IN) {
    const size_t at = static_cast<size_t>(b) * q.D + tile * 64;
    rx.start(KEEP ? static_cast<const void*>(q.x8.codes + at) : xp, xs, first, left);
    rf.start(KEEP ? static_cast<const void*>(q.f8.codes + at) : fp, fs, first, left);
    if constexpr (Z) rz.start(KEEP ? static_cast<const void*>(q.z8.codes + at) : zp, zs, first, left);
  }
  uint32_t filled = 0;  // the stage that is filled next
  auto fetch = [&]() {
    const int on = fetched >= first ? len - fetched : 0;
    if (on > 0) {
      const uint32_t to = smem_addr(mine) + filled, in = to + Rg::Run::kBytes;
      const long long ahead = fetched - first;
      const long long inputs = ahead * (KEEP ? 1 : static_cast<int>(sizeof(T)));
      rdy.copy(to, ahead * static_cast<int>(sizeof(T)) * q.dy_t, q.dy_t, on, left);
      if constexpr (IN) {
        if constexpr (MODE != kSummary) rx.copy(in, inputs * xs, xs, on, left);
        rf.copy(in + Rg::kInput, inputs * fs, fs, on, left);
        if constexpr (Z) rz.copy(in + 2 * Rg::kInput, inputs * zs, zs, on, left);
      }
    }
    fetched -= round;
    filled = filled == (Rg::kStages - 1) * Rg::kStage ? 0 : filled + Rg::kStage;
    cp_async_commit();
  };
  // What is not copied but loaded, a round ahead: the state before the run, the scales.
  auto fetch_next = [&](int n) {
    const int t0 = (last - n) * round + first;
    const bool on = n <= last && t0 < len;
    if (MODE != kSummary && on && ch.in)
      start_next.load(q.states + (static_cast<size_t>(t0 / kGS) * q.B + b) * q.D + ch.d);
    else
      start_next.clear();
    if constexpr (SCALES) {
      if (on) {
        if constexpr (MODE != kSummary) sx_next = run_scales<V>(q.x8, q, b, tile, t0, len);
        sf_next = run_scales<V>(q.f8, q, b, tile, t0, len);
        if constexpr (Z) sz_next = run_scales<V>(q.z8, q, b, tile, t0, len);
      }
    }
  };
  // What does not come through the ring: without one the next run's loads are on their way to
  // registers; what is kept and aligned in pairs only is loaded for the run at hand.
  struct Inputs {
    Input<T, V, KEEP> x, f, z;
    RawV<T, V> dy[kGS];
  };
  Inputs in_next;
  auto load = [&](Inputs& to, int t0) {
#pragma unroll
    for (int k = 0; k < kGS; ++k) {
      const long long t = t0 + k;
      if (t0 >= first && t < len && ch.in) {
        const HeldAt at = held_at<V>(q, t0 + k, b, ch.d);
        if constexpr (MODE != kSummary) to.x.load(k, xp + t * q.x_t, q.x8, at);
        to.f.load(k, fp + t * q.f_t, q.f8, at);
        if (Z) to.z.load(k, zp + t * q.z_t, q.z8, at);
        if constexpr (!RING) to.dy[k].load(dyp + t * q.dy_t);
      } else {
        if constexpr (MODE != kSummary) to.x.raw[k].clear();
        to.f.raw[k].clear();
        if (Z) to.z.raw[k].clear();
        if constexpr (!RING) to.dy[k].clear();
      }
    }
  };
  if constexpr (RING) {
#pragma unroll
    for (int n = 0; n < Rg::kStages - 1; ++n) fetch();
  }
  if constexpr (AHEAD) load(in_next, last * round + first);
  fetch_next(0);
  // What comes back into the warp's last run; kSummary: 0, and A of the runs so far.
  Fv<V> carry(0.f), through_all(1.f);
  if constexpr (MODE != kSummary)
    carry = load_par_v<V>(q.dh_last ? q.dh_last + static_cast<size_t>(b) * q.D : nullptr, ch);
  if constexpr (MODE == kSegments) {
    grid_dep_wait();
    carry = seg.template enter<true>(carry, cta, w);
  }

  int done = 0;  // rounds that had steps
  for (int n = 0; n <= last; ++n) {
    const int base = (last - n) * round, t0 = base + first;
    T* const dxr = dxp + t0 * q.dx_t;
    T* const dfr = dfp + t0 * q.df_t;
    T* const dzr = Z ? dzp + t0 * q.dz_t : nullptr;
    T* const yr = yp ? yp + t0 * q.y_t : nullptr;
    if ((MODE == kRounds ? base : t0) >= len) {
      if constexpr (RING) fetch();
      if constexpr (AHEAD) load(in_next, t0 - round);
      fetch_next(n + 1);
      if constexpr (MODE == kSummary) continue;
#pragma unroll
      for (int k = 0; k < kGS; ++k) {
        if (t0 + k >= K || !ch.in) continue;
        store_v(dxr + k * q.dx_t, Fv<V>(0.f));
        store_v(dfr + k * q.df_t, Fv<V>(0.f));
        if (Z) store_v(dzr + k * q.dz_t, Fv<V>(0.f));
        if (yr) store_v(yr + k * q.y_t, Fv<V>(0.f));
      }
      continue;
    }
    Inputs in;
    const char* const stage = mine + n % Rg::kStages * Rg::kStage;
    Fv<V> h = start_next.get();
    float ux = 0.f, uf = 0.f, uz = 0.f;  // the scales' values
    if constexpr (SCALES) ux = held_up(sx_next), uf = held_up(sf_next), uz = held_up(sz_next);
    if constexpr (AHEAD) {
      in = in_next;
      load(in_next, t0 - round);
    } else if constexpr (!IN) {
      load(in, t0);
    }
    if constexpr (RING) {
      __syncwarp();  // the stage that is filled next has been read by all lanes
      fetch();
    }
    fetch_next(n + 1);
    if constexpr (RING) {
      cp_async_wait<Rg::kStages - 1>();
      __syncwarp();
    }
    Fv<V> a[kGS], i[kGS], u[kGS], dh[kGS];
    auto gather = [&](auto whole) {
      T *to_z = dzr, *to_y = yr;
#pragma unroll
      for (int k = 0; k < kGS; ++k) {
        Fv<V> xv(0.f), fv, zv, dyv, dz(0.f), y;
        if constexpr (RING) dyv = ring_get<T>(stage, k);
        else dyv = in.dy[k].get();
        [[maybe_unused]] const char* const runs = stage + Rg::Run::kBytes;
        if constexpr (IN && KEEP) {
          if constexpr (MODE != kSummary) xv = ring_get_held(runs, k, ux);
          fv = ring_get_held(runs + Rg::kInput, k, uf);
          if constexpr (Z) zv = ring_get_held(runs + 2 * Rg::kInput, k, uz);
        } else if constexpr (IN) {
          if constexpr (MODE != kSummary) xv = ring_get<T>(runs, k);
          fv = ring_get<T>(runs + Rg::kInput, k);
          if constexpr (Z) zv = ring_get<T>(runs + 2 * Rg::kInput, k);
        } else if constexpr (KEEP && !RING) {
          if constexpr (MODE != kSummary) xv = in.x.get(k, ux);
          fv = in.f.get(k, uf);
          if constexpr (Z) zv = in.z.get(k, uz);
        } else {
          if constexpr (MODE != kSummary) xv = in.x.raw[k].get();
          fv = in.f.raw[k].get();
          if constexpr (Z) zv = in.z.raw[k].get();
        }
        gates<V>(fv, bias2, a[k], i[k]);
        u[k] = fma(xv, Fv<V>(-1.f), h) * (a[k] * i[k]);
        h = fma(a[k], h, i[k] * xv);
        if constexpr (Z) {
          const Fv<V> sg = logistic<V>(zv), gate = zv * sg;
          dh[k] = dyv * gate;
          dz = dyv * h * fma(gate, fma(sg, Fv<V>(-1.f), Fv<V>(1.f)), sg);
          y = h * gate;
        } else {
          dh[k] = dyv;
          y = h;
        }
        const bool on = decltype(whole)::value || t0 + k < len;
        if (!on) {
          a[k] = Fv<V>(1.f);
          i[k] = u[k] = dh[k] = dz = y = Fv<V>(0.f);
        }
        if (MODE != kSummary && (decltype(whole)::value || t0 + k < K) && ch.in) {
          if (Z) store_v(to_z, dz);
          if (yr) store_v(to_y, y);
        }
        if (Z) to_z += q.dz_t;
        to_y += q.y_t;
      }
    };
    const bool whole = t0 + kGS <= len;
    decide(whole, gather);
    // What leaves a run backwards: A carry + H, with carry = f_t g_t of the step after it.
    Fv<V> A(1.f), H(0.f);
#pragma unroll
    for (int k = kGS - 1; k >= 0; --k) {
      H = a[k] * (dh[k] + H);
      A = A * a[k];
    }
    if constexpr (MODE == kSummary) {
      carry = fma(A, carry, H);
      through_all = through_all * A;
      continue;
    }
    Fv<V> g = carry;
    if constexpr (MODE == kRounds) g = enter<V, true>(ex, done++, w, A, H, carry);
    auto finish = [&](auto whole) {
      T *to_x = dxr + (kGS - 1) * q.dx_t, *to_f = dfr + (kGS - 1) * q.df_t;
#pragma unroll
      for (int k = kGS - 1; k >= 0; --k, to_x -= q.dx_t, to_f -= q.df_t) {
        g = g + dh[k];
        Fv<V> dx = g * i[k], df = g * u[k];
        // Behind the end g may be an infinity or a NaN that dh_last brought.
        if (!decltype(whole)::value && t0 + k >= len) dx = df = Fv<V>(0.f);
        dsum = dsum + df;
        g = g * a[k];
        if ((decltype(whole)::value || t0 + k < K) && ch.in) {
          store_v(to_x, dx);
          store_v(to_f, df);
        }
      }
    };
    decide(whole, finish);
    if (MODE == kSegments) carry = g;
  }
  if constexpr (RING) cp_async_wait<0>();
  if constexpr (MODE == kSummary) {
    seg.template put<true>(ex, cta, w, through_all, carry);
    return;
  }
  // In rounds every warp ends with it.
  if (q.dh0 && cta == 0 && w == 0 && ch.in)
    store_v(q.dh0 + static_cast<size_t>(b) * q.D + ch.d, carry);
  if (!dbias) return;
  __syncthreads();
  put_ah(ex.run(0, w), dsum, dsum);
  __syncthreads();
  if (w == 0 && ch.in) {
    Fv<V> v(0.f);
    for (int n = 0; n < warps; ++n) {
      Fv<V> part, same;
      get_ah(ex.run(0, n), part, same);
      v = v + part;
    }
    store_v(dbias + (static_cast<size_t>(b) * ctas + cta) * q.D + ch.d, v);
  }
}

// Channels of all tensors are aligned in pairs.
bool pairs(const GatedCall& q) {
  const int e = q.bf16 ? 4 : 8;
  return q.D % 2 == 0 && group_aligned(q.x, q.x_t, q.x_b, e, 2) &&
         group_aligned(q.f, q.f_t, q.f_b, e, 2) && group_aligned(q.z, q.z_t, q.z_b, e, 2) &&
         group_aligned(q.y, q.y_t, q.y_b, e, 2) && group_aligned(q.dy, q.dy_t, q.dy_b, e, 2) &&
         group_aligned(q.dx, q.dx_t, q.dx_b, e, 2) && group_aligned(q.df, q.df_t, q.df_b, e, 2) &&
         group_aligned(q.dz, q.dz_t, q.dz_b, e, 2) && group_aligned(q.states, 0, 0, 8, 2) &&
         group_aligned(q.dh0, 0, 0, 8, 2) && group_aligned(q.dbias, 0, 0, 8, 2) && group_aligned(q.x8.codes, 0, 0, 2, 2) &&
         group_aligned(q.f8.codes, 0, 0, 2, 2) && group_aligned(q.z8.codes, 0, 0, 2, 2);
}
// And the inputs in pieces of 16 bytes (8 of what is kept).
bool sixteens(const GatedCall& q) {
  const int per = q.bf16 ? 8 : 4;
  if (q.D % per || !group_aligned(q.dy, q.dy_t, q.dy_b, 16, per)) return false;
  if (q.keep)
    return q.D % 8 == 0 && group_aligned(q.x8.codes, 0, 0, 8, 8) &&
           group_aligned(q.f8.codes, 0, 0, 8, 8) && group_aligned(q.z8.codes, 0, 0, 8, 8);
  return group_aligned(q.x, q.x_t, q.x_b, 16, per) && group_aligned(q.f, q.f_t, q.f_b, 16, per) &&
         group_aligned(q.z, q.z_t, q.z_b, 16, per);
}

template <typename T, bool Z, bool KEEP, GatedPath PATH, GatedMode MODE>
cudaError_t bwd_mode(const GatedCall& q, const GatedShape& sh, int tiles, float* dbias,
                     cudaStream_t s) {
  auto* const kern = gated_bwd_kernel<T, Z, KEEP, PATH, MODE>;
  LaunchCfg c;
  c.grid = dim3(MODE == kRounds ? tiles : tiles * sh.ctas, q.B);
  c.block = dim3(32 * sh.warps);
  c.stream = s;
  c.pdl = MODE == kSegments;
  constexpr size_t ring = PATH == kSingles ? 0 : Ring<T, Z, KEEP, PATH>::kWarp;
  c.smem = gated_smem<path_v(PATH)>(sh.warps, ring);
  const cudaError_t e = allow_smem(kern, c.smem, gated_smem<path_v(PATH)>(kGatedWarps, ring));
  return e == cudaSuccess ? launch(c, kern, q, sh, dbias) : e;
}
template <typename T, bool Z, bool KEEP, GatedPath PATH>
cudaError_t bwd(const GatedCall& q, cudaStream_t s) {
  const int tiles = (q.D - 1) / (32 * path_v(PATH)) + 1;
  const GatedShape sh = gated_shape(q.B, q.K, tiles, kBwdSlots);
  const int P = q.B * (sh.ctas ? sh.ctas : 1);
  // Partial sums of dbias behind what the launches over segments share.
  float* const parts = q.ws + gated_segments_floats(q.B, q.K, q.D, true);
  float* const first = q.dbias && P > 1 ? parts : q.dbias;
  cudaError_t e;
  if (sh.ctas == 0) {
    e = bwd_mode<T, Z, KEEP, PATH, kRounds>(q, sh, tiles, first, s);
  } else {
    e = bwd_mode<T, Z, KEEP, PATH, kSummary>(q, sh, tiles, nullptr, s);
    if (e == cudaSuccess) e = bwd_mode<T, Z, KEEP, PATH, kSegments>(q, sh, tiles, first, s);
  }
  if (e != cudaSuccess || first == q.dbias) return e;
  return merge_launch(parts, P, q.D, q.dbias, s, true);
}
template <typename T, GatedPath PATH>
cudaError_t bwd_path(const GatedCall& q, cudaStream_t s) {
  if (q.keep) return q.has_z ? bwd<T, true, true, PATH>(q, s) : bwd<T, false, true, PATH>(q, s);
  return q.has_z ? bwd<T, true, false, PATH>(q, s) : bwd<T, false, false, PATH>(q, s);
}
template <typename T>
cudaError_t bwd_t(const GatedCall& q, cudaStream_t s) {
  if (!pairs(q)) return bwd_path<T, kSingles>(q, s);
  return sixteens(q) ? bwd_path<T, kSixteens>(q, s) : bwd_path<T, kPairs>(q, s);
}

}  // namespace

size_t gated_partials_floats(int B, int K, int D) {
  int most = 1;
  for (int V = 1; V <= 2; ++V) {
    const int ctas = gated_shape(B, K, (D - 1) / (32 * V) + 1, kBwdSlots).ctas;
    most = ctas > most ? ctas : most;
  }
  return static_cast<size_t>(B) * most * D;
}
cudaError_t gated_bwd_launch(const GatedCall& q, cudaStream_t s) {
  return q.bf16 ? bwd_t<__nv_bfloat16>(q, s) : bwd_t<float>(q, s);
}

}  // namespace cfc
