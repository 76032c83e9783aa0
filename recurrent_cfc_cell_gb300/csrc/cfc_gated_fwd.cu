// cfc_gated_fwd.cu -- the gated linear recurrence, forward and for single tokens (cfc_gated.cuh says
// how the steps are divided).
#include "cfc_gated.cuh"

namespace cfc {
namespace {

// Rounds on their way to shared memory, and the one being worked on, of a warp.
template <typename T, bool Z>
struct Ring {
  using Run = RingRun<sizeof(T), 16>;
  static constexpr int kStages = 2, kTensors = Z ? 3 : 2;
  static constexpr int kStage = kTensors * Run::kBytes, kWarp = kStages * kStage;
};

// The largest magnitude's bits of eight values as they are stored.
__device__ __forceinline__ uint32_t most8(const Raw8<float>& r) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, magnitude_bits(r.v[i]));
  return m;
}
__device__ __forceinline__ uint32_t most8(const Raw8<__nv_bfloat16>& r) {
  uint32_t m = r.w[0] & 0x7fff7fffu;
#pragma unroll
  for (int i = 1; i < 4; ++i) m = __vmaxu2(m, r.w[i] & 0x7fff7fffu);
  return max(m << 16, m & 0xffff0000u);
}

// A run of a tensor, kGS steps x 64 channels in shared memory, to 8 bits: eight channels of a step to a
// lane, a block to four lanes, so that shared memory is read and codes are written whole rows at a
// time.  `code`, `scale`: where the first of the lane's steps (lane / 8 and that plus 4) goes; `on` of
// the run's steps are there.
template <typename T>
__device__ __forceinline__ void keep_run(const char* run, const Held8& h, size_t code, size_t scale,
                                         size_t code_step, size_t scale_step, int on, bool in) {
  const int lane = threadIdx.x % 32;
  Raw8<T> r[2];
  uint32_t most[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const T* const p = reinterpret_cast<const T*>(run) + (4 * i + lane / 8) * 64 + lane % 8 * 8;
    r[i].pick(reinterpret_cast<const uint4*>(p), 1);
    most[i] = most8(r[i]);
  }
#pragma unroll
  for (int d = 1; d < 4; d *= 2)
#pragma unroll
    for (int i = 0; i < 2; ++i) most[i] = max(most[i], __shfl_xor_sync(0xffffffffu, most[i], d));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t byte = held_scale_byte(most[i]);
    const Fv<2> down(held_down(byte));
    float v[8];
    r[i].get(v);
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      Fv<2> p;
      p.v = make_float2(v[2 * j], v[2 * j + 1]);
      p = p * down;
      c[j] = held_codes2(p[0], p[1]);
    }
    if (in && 4 * i + lane / 8 < on) {
      *reinterpret_cast<uint2*>(h.codes + code + i * code_step) =
          make_uint2(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410));
      if (lane % 4 == 0) h.scales[scale + i * scale_step] = static_cast<uint8_t>(byte);
    }
  }
}

// A cluster: up to kGatedCluster x kGatedWarps runs of one sequence's steps, 32 V channels.
// Grid (tiles x CTAs of a cluster, B).
template <typename T, int V, bool Z, bool KEEP, bool RING>
__global__ void __launch_bounds__(32 * kGatedWarps, 3)
    gated_fwd_kernel(const GatedCall q, int ctas, int* status) {
  extern __shared__ __align__(128) char shared[];  // the rounds on their way, the exchange
  __shared__ uint64_t bars[2];
  using Rg = Ring<T, Z>;
  const int warps = blockDim.x / 32;
  const Exchange<V> ex{shared + (RING ? warps * Rg::kWarp : 0), warps, ctas, smem_addr(bars),
                       status};
  const int w = threadIdx.x / 32;
  const int b = blockIdx.y, K = q.K, tile = blockIdx.x / ctas, rank = blockIdx.x % ctas;
  const Channels<V> ch(tile, q.D);
  const int len = q.lengths ? min(max(q.lengths[b], 0), K) : K;
  const T* const xp = static_cast<const T*>(q.x) + b * q.x_b + (RING ? tile * 64 : ch.d);
  const T* const fp = static_cast<const T*>(q.f) + b * q.f_b + (RING ? tile * 64 : ch.d);
  const T* const zp = Z ? static_cast<const T*>(q.z) + b * q.z_b + (RING ? tile * 64 : ch.d) : nullptr;
  T* const yp = static_cast<T*>(q.y) + b * q.y_b + ch.d;
  const Fv<V> bias2 = load_par_v<V>(q.bias, ch) * Fv<V>(kLog2e);
  Fv<V> carry = load_par_v<V>(q.h0 ? q.h0 + static_cast<size_t>(b) * q.D : nullptr, ch);
  const int round = ctas * warps * kGS, first = (rank * warps + w) * kGS;

  char* const mine = shared + w * Rg::kWarp;
  const int left = q.D - tile * 64;
  typename Rg::Run rx, rf, rz;
  if constexpr (RING) {
    rx.start(xp, q.x_t, first, left);
    rf.start(fp, q.f_t, first, left);
    if constexpr (Z) rz.start(zp, q.z_t, first, left);
  }
  uint32_t filled = 0;  // the stage that is filled next
  int fetched = first;  // the first step of the run that comes there
  auto fetch = [&]() {
    const int on = len - fetched;
    if (on > 0) {
      const uint32_t to = smem_addr(mine) + filled;
      const long long ahead = static_cast<long long>(fetched - first) * static_cast<int>(sizeof(T));
      rx.copy(to, ahead * q.x_t, q.x_t, on, left);
      rf.copy(to + Rg::Run::kBytes, ahead * q.f_t, q.f_t, on, left);
      if constexpr (Z) rz.copy(to + 2 * Rg::Run::kBytes, ahead * q.z_t, q.z_t, on, left);
    }
    fetched += round;
    filled = filled == (Rg::kStages - 1) * Rg::kStage ? 0 : filled + Rg::kStage;
    cp_async_commit();
  };
  // Where the lane's first step of a run goes in what is kept.
  size_t code = 0, scale = 0;
  const int kept_d = tile * 64 + static_cast<int>(threadIdx.x) % 8 * 8;
  const size_t code_t = static_cast<size_t>(q.B) * q.D, scale_t = static_cast<size_t>(q.B) * held_blocks(q.D);
  if constexpr (KEEP && RING) {
    const size_t row = static_cast<size_t>(first + static_cast<int>(threadIdx.x) % 32 / 8) * q.B + b;
    code = row * q.D + kept_d;
    scale = row * held_blocks(q.D) + kept_d / kHeldBlock;
  }
  if constexpr (RING) {
#pragma unroll
    for (int n = 0; n < Rg::kStages - 1; ++n) fetch();
  }
  ex.start();

  for (int base = 0, n = 0; base < K; base += round, ++n) {
    const int t0 = base + first;
    T* const yr = yp + t0 * q.y_t;
    if (base >= len) {  // the sequence has ended, for the whole cluster
#pragma unroll
      for (int k = 0; k < kGS; ++k)
        if (t0 + k < K && ch.in) store_v(yr + k * q.y_t, Fv<V>(0.f));
      continue;
    }
    RawV<T, V> x[kGS], f[kGS], z[kGS];
    const char* const stage = mine + n % Rg::kStages * Rg::kStage;
    if constexpr (RING) {
      __syncwarp();  // the stage that is filled next has been read by all lanes
      fetch();
      cp_async_wait<Rg::kStages - 1>();
      __syncwarp();
      if constexpr (KEEP) {
        const bool in = kept_d < q.D;
        const int on = len - t0;
        if (on > 0) {
          keep_run<T>(stage, q.x8, code, scale, 4 * code_t, 4 * scale_t, on, in);
          keep_run<T>(stage + Rg::Run::kBytes, q.f8, code, scale, 4 * code_t, 4 * scale_t, on, in);
          if constexpr (Z)
            keep_run<T>(stage + 2 * Rg::Run::kBytes, q.z8, code, scale, 4 * code_t, 4 * scale_t, on,
                        in);
        }
        code += round * code_t;
        scale += round * scale_t;
      }
    } else {
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
    }
    Fv<V> a[kGS], c[kGS], A(1.f), H(0.f);
    // `whole`: no step of the run is behind the sequence's end.
    auto gather = [&](auto whole) {
#pragma unroll
      for (int k = 0; k < kGS; ++k) {
        const Fv<V> xv = [&] {
          if constexpr (RING) return ring_get<T>(stage, k);
          else return x[k].get();
        }();
        const Fv<V> fv = [&] {
          if constexpr (RING) return ring_get<T>(stage + Rg::Run::kBytes, k);
          else return f[k].get();
        }();
        if constexpr (KEEP && !RING) {
          if (t0 + k < len) {
            const HeldAt at = held_at<V>(q, t0 + k, b, ch.d);
            store_held_v<V>(q.x8, at, xv, ch.in);
            store_held_v<V>(q.f8, at, fv, ch.in);
            if constexpr (Z) store_held_v<V>(q.z8, at, z[k].get(), ch.in);
          }
        }
        Fv<V> i;
        gates<V>(fv, bias2, a[k], i);
        c[k] = i * xv;
        if (!decltype(whole)::value && t0 + k >= len) {
          a[k] = Fv<V>(1.f);
          c[k] = Fv<V>(0.f);
        }
        H = fma(a[k], H, c[k]);
        A = A * a[k];
      }
    };
    const bool whole = t0 + kGS <= len;
    decide(whole, gather);
    Fv<V> h = enter<V, false>(ex, n, w, rank, A, H, carry);
    if (q.states && t0 < K && ch.in)
      store_v(q.states + (static_cast<size_t>(t0 / kGS) * q.B + b) * q.D + ch.d, h);
    auto finish = [&](auto whole) {
      T* to = yr;
#pragma unroll
      for (int k = 0; k < kGS; ++k, to += q.y_t) {
        h = fma(a[k], h, c[k]);
        Fv<V> y = h;
        if constexpr (Z) {
          const Fv<V> zv = [&] {
            if constexpr (RING) return ring_get<T>(stage + 2 * Rg::Run::kBytes, k);
            else return z[k].get();
          }();
          y = h * (zv * logistic<V>(zv));
        }
        if (decltype(whole)::value) {
          if (ch.in) store_v(to, y);
        } else {
          if (t0 + k < K && ch.in) store_v(to, t0 + k < len ? y : Fv<V>(0.f));
        }
      }
    };
    decide(whole, finish);
  }
  if constexpr (RING) cp_async_wait<0>();
  if (q.h_last && rank == 0 && w == 0 && ch.in)
    store_v(q.h_last + static_cast<size_t>(b) * q.D + ch.d, carry);
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
  Fv<V> bias2(0.f), a, i;
  if (q.bias) {
#pragma unroll
    for (int j = 0; j < V; ++j) bias2[j] = __ldg(q.bias + d + j) * kLog2e;
  }
  gates<V>(rf.get(), bias2, a, i);
  const Fv<V> h = fma(a, rh.get(), i * rx.get());
  store_v(q.h_last + b * q.D + d, h);
  Fv<V> y = h;
  if (q.z) {
    const Fv<V> z = rz.get();
    y = h * (z * logistic<V>(z));
  }
  store_v(static_cast<T*>(q.y) + b * q.y_b + d, y);
}

// Channels of all tensors are aligned in pairs.
bool pairs(const GatedCall& q) {
  const int e = q.bf16 ? 4 : 8;
  return q.D % 2 == 0 && group_aligned(q.x, q.x_t, q.x_b, e, 2) &&
         group_aligned(q.f, q.f_t, q.f_b, e, 2) && group_aligned(q.z, q.z_t, q.z_b, e, 2) &&
         group_aligned(q.y, q.y_t, q.y_b, e, 2) && group_aligned(q.h0, 0, 0, 8, 2) &&
         group_aligned(q.h_last, 0, 0, 8, 2) && group_aligned(q.states, 0, 0, 8, 2) &&
         group_aligned(q.x8.codes, 0, 0, 2, 2) && group_aligned(q.f8.codes, 0, 0, 2, 2) &&
         group_aligned(q.z8.codes, 0, 0, 2, 2);
}
// And the inputs in pieces of 16 bytes.
bool sixteens(const GatedCall& q) {
  const int per = q.bf16 ? 8 : 4;
  return q.D % per == 0 && group_aligned(q.x, q.x_t, q.x_b, 16, per) &&
         group_aligned(q.f, q.f_t, q.f_b, 16, per) && group_aligned(q.z, q.z_t, q.z_b, 16, per) &&
         (!q.keep || (q.D % 8 == 0 && group_aligned(q.x8.codes, 0, 0, 8, 8) &&
                      group_aligned(q.f8.codes, 0, 0, 8, 8) && group_aligned(q.z8.codes, 0, 0, 8, 8)));
}

template <typename T, int V, bool Z, bool KEEP, bool RING>
cudaError_t fwd(const GatedCall& q, cudaStream_t s) {
  auto* const kern = gated_fwd_kernel<T, V, Z, KEEP, RING>;
  const GatedShape sh = gated_shape(q, (q.D - 1) / (32 * V) + 1);
  LaunchCfg c;
  c.grid = dim3(((q.D - 1) / (32 * V) + 1) * sh.ctas, q.B);
  c.block = dim3(32 * sh.warps);
  c.stream = s;
  if (sh.ctas > 1) c.cluster = dim3(sh.ctas, 1, 1);
  c.smem = Exchange<V>::bytes(sh.warps, sh.ctas);
  if (RING) c.smem += static_cast<size_t>(sh.warps) * Ring<T, Z>::kWarp;
  const cudaError_t e = gated_attributes(kern, c.smem, sh.ctas);
  return e == cudaSuccess ? launch(c, kern, q, sh.ctas, q.status) : e;
}
template <typename T, int V, bool RING>
cudaError_t fwd_v(const GatedCall& q, cudaStream_t s) {
  if (q.keep)
    return q.has_z ? fwd<T, V, true, true, RING>(q, s) : fwd<T, V, false, true, RING>(q, s);
  return q.has_z ? fwd<T, V, true, false, RING>(q, s) : fwd<T, V, false, false, RING>(q, s);
}
template <typename T>
cudaError_t fwd_t(const GatedCall& q, cudaStream_t s) {
  if (!pairs(q)) return fwd_v<T, 1, false>(q, s);
  return sixteens(q) ? fwd_v<T, 2, true>(q, s) : fwd_v<T, 2, false>(q, s);
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
