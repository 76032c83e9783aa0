// cfc_gated_bwd.cu -- the gradients of the gated linear recurrence (cfc_gated.cuh says how the steps
// are divided; here the runs follow one another backwards in time).
//
//   g_t = dL/dh_t = dy_t silu(z_t) + f_{t+1} g_{t+1}
//   dx_t = g_t (1 - f_t),   df_t = g_t (h_{t-1} - x_t) f_t (1 - f_t)   (of the logit)
//   dz_t = dy_t h_t silu'(z_t),   dbias = sum df,   dh0 = f_0 g_0
//
// h is formed again within each run from the state that the forward pass kept at its start.
#include "cfc_gated.cuh"

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

// Rounds on their way to shared memory, and the one being worked on, of a warp: x, f and dy, and z,
// the first ones as kept where they are.
template <typename T, bool Z, bool KEEP>
struct Ring {
  using Run = RingRun<sizeof(T), 16>;
  using Codes = RingRun<1, 8>;
  static constexpr int kStages = sizeof(T) == 2 ? 3 : 2;
  using In = std::conditional_t<KEEP, Codes, Run>;
  static constexpr int kInput = KEEP ? Codes::kBytes : Run::kBytes;
  static constexpr int kStage = Run::kBytes + (Z ? 3 : 2) * kInput, kWarp = kStages * kStage;
};

// The scales of a run of 64 channels in 8 bits: lane 2 k + i holds the one of step k's block i.
__device__ __forceinline__ uint32_t run_scales(const Held8& h, const GatedCall& q, int b, int tile,
                                               int t0, int len) {
  const int lane = threadIdx.x % 32, t = t0 + lane / 2, block = 2 * tile + lane % 2;
  const bool in = lane < 2 * kGS && t < len && block < held_blocks(q.D);
  return in ? h.scales[(static_cast<size_t>(t) * q.B + b) * held_blocks(q.D) + block] : 1u;
}
__device__ __forceinline__ Fv<2> ring_get_held(const char* run, int k, float up) {
  const int lane = threadIdx.x % 32;
  Fv<2> v;
  v.v = held_values2(reinterpret_cast<const uint16_t*>(run + k * 64)[lane]);
  return v * Fv<2>(__shfl_sync(0xffffffffu, up, 2 * k + lane / 16));
}

template <typename T, int V, bool Z, bool KEEP, bool RING>
__global__ void __launch_bounds__(32 * kGatedWarps, 2)
    gated_bwd_kernel(const GatedCall q, int ctas, float* dbias, int* status) {
  grid_dep_launch_dependents();
  extern __shared__ __align__(128) char shared[];  // the rounds on their way, the exchange
  __shared__ uint64_t bars[2];
  using Rg = Ring<T, Z, KEEP>;
  const int warps = blockDim.x / 32;
  const Exchange<V> ex{shared + (RING ? warps * Rg::kWarp : 0), warps, ctas, smem_addr(bars),
                       status};
  const int w = threadIdx.x / 32;
  const int b = blockIdx.y, K = q.K, tile = blockIdx.x / ctas, rank = blockIdx.x % ctas;
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
  Fv<V> carry = load_par_v<V>(q.dh_last ? q.dh_last + static_cast<size_t>(b) * q.D : nullptr, ch);
  const int round = ctas * warps * kGS, first = (rank * warps + w) * kGS;
  const int last = (K - 1) / round;  // rounds are taken from the last to the first

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
    const size_t at = static_cast<size_t>(b) * q.D + tile * 64;
    rdy.start(dyp, q.dy_t, first, left);
    rx.start(KEEP ? static_cast<const void*>(q.x8.codes + at) : xp, xs, first, left);
    rf.start(KEEP ? static_cast<const void*>(q.f8.codes + at) : fp, fs, first, left);
    if constexpr (Z) rz.start(KEEP ? static_cast<const void*>(q.z8.codes + at) : zp, zs, first, left);
  }
  uint32_t filled = 0;  // the stage that is filled next
  auto fetch = [&]() {
    const int on = fetched >= 0 ? len - fetched : 0;
    if (on > 0) {
      const uint32_t to = smem_addr(mine) + filled, in = to + Rg::Run::kBytes;
      const long long ahead = fetched - first;
      const long long inputs = ahead * (KEEP ? 1 : static_cast<int>(sizeof(T)));
      rdy.copy(to, ahead * static_cast<int>(sizeof(T)) * q.dy_t, q.dy_t, on, left);
      rx.copy(in, inputs * xs, xs, on, left);
      rf.copy(in + Rg::kInput, inputs * fs, fs, on, left);
      if constexpr (Z) rz.copy(in + 2 * Rg::kInput, inputs * zs, zs, on, left);
    }
    fetched -= round;
    filled = filled == (Rg::kStages - 1) * Rg::kStage ? 0 : filled + Rg::kStage;
    cp_async_commit();
  };
  // What is not copied but loaded, a round ahead: the state before the run, the scales.
  auto fetch_next = [&](int n) {
    const int t0 = (last - n) * round + first;
    const bool on = n <= last && t0 < len;
    if (on && ch.in)
      start_next.load(q.states + (static_cast<size_t>(t0 / kGS) * q.B + b) * q.D + ch.d);
    else
      start_next.clear();
    if constexpr (KEEP && RING) {
      if (on) {
        sx_next = run_scales(q.x8, q, b, tile, t0, len);
        sf_next = run_scales(q.f8, q, b, tile, t0, len);
        if constexpr (Z) sz_next = run_scales(q.z8, q, b, tile, t0, len);
      }
    }
  };
  if constexpr (RING) {
#pragma unroll
    for (int n = 0; n < Rg::kStages - 1; ++n) fetch();
  }
  fetch_next(0);
  ex.start();

  int done = 0;  // rounds that had steps
  for (int n = 0; n <= last; ++n) {
    const int base = (last - n) * round, t0 = base + first;
    T* const dxr = dxp + t0 * q.dx_t;
    T* const dfr = dfp + t0 * q.df_t;
    T* const dzr = Z ? dzp + t0 * q.dz_t : nullptr;
    T* const yr = yp ? yp + t0 * q.y_t : nullptr;
    if (base >= len) {
      if constexpr (RING) fetch();
      fetch_next(n + 1);
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
    Input<T, V, KEEP> x, f, z;
    RawV<T, V> dy[kGS];
    const char* const stage = mine + n % Rg::kStages * Rg::kStage;
    Fv<V> h = start_next.get();
    float ux = 0.f, uf = 0.f, uz = 0.f;  // the scales' values
    if constexpr (RING) {
      if constexpr (KEEP) ux = held_up(sx_next), uf = held_up(sf_next), uz = held_up(sz_next);
      __syncwarp();  // the stage that is filled next has been read by all lanes
      fetch();
      fetch_next(n + 1);
      cp_async_wait<Rg::kStages - 1>();
      __syncwarp();
    } else {
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
      fetch_next(n + 1);
    }
    Fv<V> a[kGS], i[kGS], u[kGS], dh[kGS];
    auto gather = [&](auto whole) {
      T *to_z = dzr, *to_y = yr;
#pragma unroll
      for (int k = 0; k < kGS; ++k) {
        Fv<V> xv, fv, zv, dyv, dz(0.f), y;
        if constexpr (RING) {
          const char* const in = stage + Rg::Run::kBytes;
          dyv = ring_get<T>(stage, k);
          if constexpr (KEEP) {
            xv = ring_get_held(in, k, ux);
            fv = ring_get_held(in + Rg::kInput, k, uf);
            if constexpr (Z) zv = ring_get_held(in + 2 * Rg::kInput, k, uz);
          } else {
            xv = ring_get<T>(in, k);
            fv = ring_get<T>(in + Rg::kInput, k);
            if constexpr (Z) zv = ring_get<T>(in + 2 * Rg::kInput, k);
          }
        } else {
          xv = x.raw[k].get();
          fv = f.raw[k].get();
          if constexpr (Z) zv = z.raw[k].get();
          dyv = dy[k].get();
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
        if ((decltype(whole)::value || t0 + k < K) && ch.in) {
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
    Fv<V> g = enter<V, true>(ex, done++, w, rank, A, H, carry);
    auto finish = [&](auto whole) {
      T *to_x = dxr + (kGS - 1) * q.dx_t, *to_f = dfr + (kGS - 1) * q.df_t;
#pragma unroll
      for (int k = kGS - 1; k >= 0; --k, to_x -= q.dx_t, to_f -= q.df_t) {
        g = g + dh[k];
        const Fv<V> dx = g * i[k], df = g * u[k];
        dsum = dsum + df;
        g = g * a[k];
        if ((decltype(whole)::value || t0 + k < K) && ch.in) {
          store_v(to_x, dx);
          store_v(to_f, df);
        }
      }
    };
    decide(whole, finish);
  }
  if constexpr (RING) cp_async_wait<0>();
  if (q.dh0 && rank == 0 && w == 0 && ch.in)
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
    store_v(dbias + (static_cast<size_t>(b) * ctas + rank) * q.D + ch.d, v);
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

template <typename T, int V, bool Z, bool KEEP, bool RING>
cudaError_t bwd(const GatedCall& q, cudaStream_t s) {
  auto* const kern = gated_bwd_kernel<T, V, Z, KEEP, RING>;
  const int tiles = (q.D - 1) / (32 * V) + 1;
  const GatedShape sh = gated_shape(q, tiles);
  LaunchCfg c;
  c.grid = dim3(tiles * sh.ctas, q.B);
  c.block = dim3(32 * sh.warps);
  c.stream = s;
  if (sh.ctas > 1) c.cluster = dim3(sh.ctas, 1, 1);
  c.smem = Exchange<V>::bytes(sh.warps, sh.ctas);
  if (RING) c.smem += static_cast<size_t>(sh.warps) * Ring<T, Z, KEEP>::kWarp;
  cudaError_t e = gated_attributes(kern, c.smem, sh.ctas);
  const int P = q.B * sh.ctas;
  float* const first = q.dbias && P > 1 ? q.ws : q.dbias;
  if (e == cudaSuccess) e = launch(c, kern, q, sh.ctas, first, q.status);
  if (e != cudaSuccess || first == q.dbias) return e;
  return merge_launch(q.ws, P, q.D, q.dbias, s, true);
}
template <typename T, int V, bool RING>
cudaError_t bwd_v(const GatedCall& q, cudaStream_t s) {
  if (q.keep)
    return q.has_z ? bwd<T, V, true, true, RING>(q, s) : bwd<T, V, false, true, RING>(q, s);
  return q.has_z ? bwd<T, V, true, false, RING>(q, s) : bwd<T, V, false, false, RING>(q, s);
}
template <typename T>
cudaError_t bwd_t(const GatedCall& q, cudaStream_t s) {
  if (!pairs(q)) return bwd_v<T, 1, false>(q, s);
  return sixteens(q) ? bwd_v<T, 2, true>(q, s) : bwd_v<T, 2, false>(q, s);
}

}  // namespace

size_t gated_ws_floats(int B, int, int D, bool) {
  return static_cast<size_t>(B) * kGatedCluster * D;
}
cudaError_t gated_bwd_launch(const GatedCall& q, cudaStream_t s) {
  return q.bf16 ? bwd_t<__nv_bfloat16>(q, s) : bwd_t<float>(q, s);
}

}  // namespace cfc
