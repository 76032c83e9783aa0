// cfc_gated_fwd.cu -- the gated linear recurrence, forward and for single tokens (cfc_gated.cuh says
// how the steps are divided).
//
// Rounds are bound by memory, segments and what is kept in 8 bits by the instructions and their latency
// (65 a warp for a step of 64 channels with z, 115 with all three inputs kept, four a channel of them
// exponentials and reciprocals; 2.4 and 2.8 of 4 a cycle).  64 x 1024 steps x 1536 channels bf16 with
// states: 135 us (6.3 TB/s); 64 x 512 x 1024 fp32 82 us (6.7 TB/s); 32768 steps of one sequence of 1024
// channels bf16 70 us in segments, of which the summary, that reads x and f once more, is a third; 16 x
// 2048 x 2048 bf16 in 8 bits 169 us.  A token of 1024 sequences of 2048 channels in bf16 8 us.
#include "cfc_gated.cuh"

namespace cfc {
namespace {

// Rounds on their way to shared memory, and the one being worked on, of a warp.
template <typename T, bool Z, GatedPath PATH>
struct Ring {
  using Run = RingRun<sizeof(T), PATH == kSixteens ? 16 : 2 * sizeof(T)>;
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
// the run's steps are there, and `left` of the lane's channels.  `WHOLE`: D is a multiple of 8 and
// codes are aligned for eight at once, otherwise (D is even) for two.
template <typename T, bool WHOLE>
__device__ __forceinline__ void keep_run(const char* run, const Held8& h, size_t code, size_t scale,
                                         size_t code_step, size_t scale_step, int on, int left) {
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
    if (left > 0 && 4 * i + lane / 8 < on) {
      uint8_t* const to = h.codes + code + i * code_step;
      if constexpr (WHOLE) {
        *reinterpret_cast<uint2*>(to) =
            make_uint2(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410));
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (2 * j < left) reinterpret_cast<uint16_t*>(to)[j] = static_cast<uint16_t>(c[j]);
      }
      if (lane % 4 == 0) h.scales[scale + i * scale_step] = static_cast<uint8_t>(byte);
    }
  }
}

// A run of one channel a lane, kGS steps x the 32 of a block, to 8 bits: lane k finds the scale of step k.
// `code`, `scale`: where the first step's go.
template <typename T>
__device__ __forceinline__ void keep_singles(const RawV<T, 1> (&v)[kGS], const Held8& h, size_t code,
                                             size_t scale, size_t code_t, size_t scale_t, int on, bool in) {
  const int lane = threadIdx.x % 32;
  uint32_t most = 0u;
#pragma unroll
  for (int k = 0; k < kGS; ++k) {
    const uint32_t m = __reduce_max_sync(0xffffffffu, magnitude_bits(v[k].get()[0]));
    if (lane == k) most = m;
  }
  const uint32_t byte = held_scale_byte(most);
  if (lane < kGS && lane < on) h.scales[scale + lane * scale_t] = static_cast<uint8_t>(byte);
  const float down = held_down(byte);
  uint8_t* to = h.codes + code;
#pragma unroll
  for (int k = 0; k < kGS; ++k, to += code_t) {
    const float s = __shfl_sync(0xffffffffu, down, k);
    if (in && k < on) *to = static_cast<uint8_t>(held_codes2(v[k].get()[0] * s, 0.f));
  }
}

// kRounds: grid (tiles, B), CTAs of any number of warps.  kSummary and kSegments: grid (tiles x CTAs of
// segments, B), kGatedWarps warps.  Two of them an SM where channels are kept singly, which three spill
// (32 x 1024 steps x 1537 channels bf16 393 us, two 216 us).
template <typename T, bool Z, bool KEEP, GatedPath PATH, GatedMode MODE>
__global__ void __launch_bounds__(32 * kGatedWarps, KEEP && PATH == kSingles ? 2 : 3)
    gated_fwd_kernel(const GatedCall q, const GatedShape sh) {
  extern __shared__ __align__(128) char shared[];  // the rounds on their way, the exchange
  constexpr bool RING = PATH != kSingles;
  constexpr int V = path_v(PATH);
  using Rg = Ring<T, Z, PATH>;
  if (MODE == kSummary) grid_dep_launch_dependents();
  const int warps = blockDim.x / 32, w = threadIdx.x / 32;
  const Exchange<V> ex{shared + (RING ? warps * Rg::kWarp : 0), warps};
  const int ctas = MODE == kRounds ? 1 : sh.ctas;
  const int b = blockIdx.y, K = q.K, tile = blockIdx.x / ctas, cta = blockIdx.x % ctas;
  const Channels<V> ch(tile, q.D);
  const int len = q.lengths ? min(max(q.lengths[b], 0), K) : K;
  const T* const xp = static_cast<const T*>(q.x) + b * q.x_b + (RING ? tile * 64 : ch.d);
  const T* const fp = static_cast<const T*>(q.f) + b * q.f_b + (RING ? tile * 64 : ch.d);
  const T* const zp = Z ? static_cast<const T*>(q.z) + b * q.z_b + (RING ? tile * 64 : ch.d) : nullptr;
  T* const yp = static_cast<T*>(q.y) + b * q.y_b + ch.d;
  const Fv<V> bias2 = load_par_v<V>(q.bias, ch) * Fv<V>(kLog2e);
  // The warp's first step, the steps from a run to its next one, and where its steps (and those that
  // count) end.
  const int round = MODE == kRounds ? warps * kGS : kGS;
  const int first = MODE == kRounds ? w * kGS : (cta * kGatedWarps + w) * sh.steps;
  const int last = MODE == kRounds ? K : min(first + sh.steps, K);
  const int stop = min(len, last);
  const Segments<V> seg(q.ws, MODE == kRounds ? 0 : gridDim.x / ctas, tile, b, ctas);

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
    const int on = stop - fetched;
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
  // Without a ring the next run's loads are on their way to registers.
  struct Raws {
    RawV<T, V> v[kGS];
  };
  Raws x_next, f_next, z_next;
  auto load = [&](int t0) {
#pragma unroll
    for (int k = 0; k < kGS; ++k) {
      const long long t = t0 + k;
      if (t < stop && ch.in) {
        x_next.v[k].load(xp + t * q.x_t);
        f_next.v[k].load(fp + t * q.f_t);
        if (Z) z_next.v[k].load(zp + t * q.z_t);
      } else {
        x_next.v[k].clear();
        f_next.v[k].clear();
        if (Z) z_next.v[k].clear();
      }
    }
  };
  if constexpr (RING) {
#pragma unroll
    for (int n = 0; n < Rg::kStages - 1; ++n) fetch();
  } else {
    load(first);
  }
  // What enters the warp's first run; kSummary: 0, and A of the runs so far.
  Fv<V> carry(0.f), through_all(1.f);
  if constexpr (MODE == kSegments) {
    grid_dep_wait();
    Fv<V> start, same;
    get_ah(seg.start(), start, same);
    carry = seg.template enter<false>(start, cta, w);
  } else {
    const Fv<V> start = load_par_v<V>(q.h0 ? q.h0 + static_cast<size_t>(b) * q.D : nullptr, ch);
    if (MODE == kRounds) carry = start;
    else if (cta == 0 && w == 0) put_ah(seg.start(), start, start);  // h_last may be in h0's place
  }

  for (int t0 = first, n = 0; MODE == kRounds ? t0 - first < K : t0 < last; t0 += round, ++n) {
    T* const yr = yp + t0 * q.y_t;
    if ((MODE == kRounds ? t0 - first : t0) >= len) {  // the sequence has ended, for the whole CTA (or warp)
      if constexpr (MODE == kSummary) break;
#pragma unroll
      for (int k = 0; k < kGS; ++k)
        if (t0 + k < K && ch.in) store_v(yr + k * q.y_t, Fv<V>(0.f));
      continue;
    }
    Raws x, f, z;
    const char* const stage = mine + n % Rg::kStages * Rg::kStage;
    if constexpr (RING) {
      __syncwarp();  // the stage that is filled next has been read by all lanes
      fetch();
      cp_async_wait<Rg::kStages - 1>();
      __syncwarp();
      if constexpr (KEEP) {
        const int on = stop - t0, of = q.D - kept_d;
        constexpr bool WHOLE = PATH == kSixteens;
        if (on > 0) {
          keep_run<T, WHOLE>(stage, q.x8, code, scale, 4 * code_t, 4 * scale_t, on, of);
          keep_run<T, WHOLE>(stage + Rg::Run::kBytes, q.f8, code, scale, 4 * code_t, 4 * scale_t, on,
                             of);
          if constexpr (Z)
            keep_run<T, WHOLE>(stage + 2 * Rg::Run::kBytes, q.z8, code, scale, 4 * code_t,
                               4 * scale_t, on, of);
        }
        code += round * code_t;
        scale += round * scale_t;
      }
    } else {
      x = x_next, f = f_next;
      if (Z) z = z_next;
      load(t0 + round);
      if constexpr (KEEP) {
        const int on = stop - t0;
        if (on > 0) {
          const HeldAt at = held_at<V>(q, t0, b, ch.d);
          keep_singles<T>(x.v, q.x8, at.code, at.scale, code_t, scale_t, on, ch.in);
          keep_singles<T>(f.v, q.f8, at.code, at.scale, code_t, scale_t, on, ch.in);
          if constexpr (Z) keep_singles<T>(z.v, q.z8, at.code, at.scale, code_t, scale_t, on, ch.in);
        }
      }
    }
    auto gate = [&](int k) {
      if constexpr (RING) return ring_get<T>(stage + 2 * Rg::Run::kBytes, k);
      else return z.v[k].get();
    };
    Fv<V> a[kGS], c[kGS], A(1.f), H(0.f);
    // `whole`: no step of the run is behind the sequence's end.
    auto gather = [&](auto whole) {
#pragma unroll
      for (int k = 0; k < kGS; ++k) {
        const Fv<V> xv = [&] {
          if constexpr (RING) return ring_get<T>(stage, k);
          else return x.v[k].get();
        }();
        const Fv<V> fv = [&] {
          if constexpr (RING) return ring_get<T>(stage + Rg::Run::kBytes, k);
          else return f.v[k].get();
        }();
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
    if constexpr (MODE == kSummary) {
      carry = fma(A, carry, H);
      through_all = through_all * A;
      continue;
    }
    Fv<V> h = carry;
    if constexpr (MODE == kRounds) h = enter<V, false>(ex, n, w, A, H, carry);
    if (q.states && t0 < K && ch.in)
      store_v(q.states + (static_cast<size_t>(t0 / kGS) * q.B + b) * q.D + ch.d, h);
    auto finish = [&](auto whole) {
      T* to = yr;
#pragma unroll
      for (int k = 0; k < kGS; ++k, to += q.y_t) {
        h = fma(a[k], h, c[k]);
        Fv<V> y = h;
        if constexpr (Z) {
          const Fv<V> zv = gate(k);
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
    if (MODE == kSegments) carry = h;
  }
  if constexpr (RING) cp_async_wait<0>();
  if constexpr (MODE == kSummary) {
    seg.template put<false>(ex, cta, w, through_all, carry);
    return;
  }
  // Rounds end with the last state in every warp, segments in the last one's.
  if (q.h_last && ch.in && (MODE == kRounds ? w == 0 : w == kGatedWarps - 1 && cta == ctas - 1))
    store_v(q.h_last + static_cast<size_t>(b) * q.D + ch.d, carry);
}

// One step for every sequence, W channels a thread: eight where everything is aligned for them, or one.
template <typename T, int W>
__global__ void __launch_bounds__(256) gated_step_kernel(const GatedCall q) {
  constexpr int V = W == 8 ? 2 : 1;
  const int per = q.D / W;
  const long long at = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  const long long b = at / per;
  if (b >= q.B) return;
  const int d = static_cast<int>(at - b * per) * W;
  const T* const xp = static_cast<const T*>(q.x) + b * q.x_b + d;
  const T* const fp = static_cast<const T*>(q.f) + b * q.f_b + d;
  const T* const zp = q.z ? static_cast<const T*>(q.z) + b * q.z_b + d : nullptr;
  const float* const hp = q.h0 + b * q.D + d;
  float x[W], f[W], z[W], h[W], bias[W], y[W];
  if constexpr (W == 8) {
    Raw8<T> rx, rf, rz;
    Raw8<float> rh, rb;
    rx.load(xp);
    rf.load(fp);
    if (zp) rz.load(zp);
    rh.load(hp);
    if (q.bias) rb.load(q.bias + d);
    else rb.clear();
    rx.get(x);
    rf.get(f);
    if (zp) rz.get(z);
    rh.get(h);
    rb.get(bias);
  } else {
    x[0] = to_f32(*xp), f[0] = to_f32(*fp), h[0] = *hp;
    if (zp) z[0] = to_f32(*zp);
    bias[0] = q.bias ? __ldg(q.bias + d) : 0.f;
  }
#pragma unroll
  for (int j = 0; j < W; j += V) {
    Fv<V> xv, fv, zv, hv, bv, a, i;
#pragma unroll
    for (int k = 0; k < V; ++k) xv[k] = x[j + k], fv[k] = f[j + k], hv[k] = h[j + k], bv[k] = bias[j + k];
    gates<V>(fv, bv * Fv<V>(kLog2e), a, i);
    hv = fma(a, hv, i * xv);
    Fv<V> yv = hv;
    if (zp) {
#pragma unroll
      for (int k = 0; k < V; ++k) zv[k] = z[j + k];
      yv = hv * (zv * logistic<V>(zv));
    }
#pragma unroll
    for (int k = 0; k < V; ++k) h[j + k] = hv[k], y[j + k] = yv[k];
  }
  float* const ho = q.h_last + b * q.D + d;
  T* const yo = static_cast<T*>(q.y) + b * q.y_b + d;
  if constexpr (W == 8) {
    store8(ho, h);
    store8(yo, y);
  } else {
    *ho = h[0];
    *yo = from_f32<T>(y[0]);
  }
}
bool eights(const GatedCall& q) {
  const int e = q.bf16 ? 16 : 32;
  return q.D % 8 == 0 && group_aligned(q.x, 0, q.x_b, e, 8) && group_aligned(q.f, 0, q.f_b, e, 8) &&
         group_aligned(q.z, 0, q.z_b, e, 8) && group_aligned(q.y, 0, q.y_b, e, 8) &&
         group_aligned(q.h0, 0, 0, 32, 8) && group_aligned(q.h_last, 0, 0, 32, 8) &&
         group_aligned(q.bias, 0, 0, 32, 8);
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

template <typename T, bool Z, bool KEEP, GatedPath PATH, GatedMode MODE>
cudaError_t fwd_mode(const GatedCall& q, const GatedShape& sh, int tiles, cudaStream_t s) {
  auto* const kern = gated_fwd_kernel<T, Z, KEEP, PATH, MODE>;
  LaunchCfg c;
  c.grid = dim3(MODE == kRounds ? tiles : tiles * sh.ctas, q.B);
  c.block = dim3(32 * sh.warps);
  c.stream = s;
  c.pdl = MODE == kSegments;
  constexpr size_t ring = PATH == kSingles ? 0 : Ring<T, Z, PATH>::kWarp;
  c.smem = gated_smem<path_v(PATH)>(sh.warps, ring);
  const cudaError_t e = allow_smem(kern, c.smem, gated_smem<path_v(PATH)>(kGatedWarps, ring));
  return e == cudaSuccess ? launch(c, kern, q, sh) : e;
}
template <typename T, bool Z, bool KEEP, GatedPath PATH>
cudaError_t fwd(const GatedCall& q, cudaStream_t s) {
  const int tiles = (q.D - 1) / (32 * path_v(PATH)) + 1;
  const GatedShape sh = gated_shape(q.B, q.K, tiles, kFwdSlots);
  if (sh.ctas == 0) return fwd_mode<T, Z, KEEP, PATH, kRounds>(q, sh, tiles, s);
  const cudaError_t e = fwd_mode<T, false, false, PATH, kSummary>(q, sh, tiles, s);
  return e == cudaSuccess ? fwd_mode<T, Z, KEEP, PATH, kSegments>(q, sh, tiles, s) : e;
}
template <typename T, GatedPath PATH>
cudaError_t fwd_path(const GatedCall& q, cudaStream_t s) {
  if (q.keep) return q.has_z ? fwd<T, true, true, PATH>(q, s) : fwd<T, false, true, PATH>(q, s);
  return q.has_z ? fwd<T, true, false, PATH>(q, s) : fwd<T, false, false, PATH>(q, s);
}
template <typename T>
cudaError_t fwd_t(const GatedCall& q, cudaStream_t s) {
  if (!pairs(q)) return fwd_path<T, kSingles>(q, s);
  return sixteens(q) ? fwd_path<T, kSixteens>(q, s) : fwd_path<T, kPairs>(q, s);
}
template <typename T>
cudaError_t step_t(const GatedCall& q, cudaStream_t s) {
  LaunchCfg c;
  const bool eight = eights(q);
  const long long total = static_cast<long long>(q.B) * (q.D / (eight ? 8 : 1));
  c.grid = dim3(static_cast<unsigned>((total + 255) / 256));
  c.block = dim3(256);
  c.stream = s;
  return eight ? launch(c, gated_step_kernel<T, 8>, q) : launch(c, gated_step_kernel<T, 1>, q);
}

}  // namespace

size_t gated_segments_floats(int B, int K, int D, bool backward) {
  // Whether channels come in pairs depends on the tensors, which the sizing calls do not have.
  size_t most = 0;
  for (int V = 1; V <= 2; ++V) {
    const int tiles = (D - 1) / (32 * V) + 1;
    const GatedShape sh = gated_shape(B, K, tiles, backward ? kBwdSlots : kFwdSlots);
    if (sh.ctas == 0) continue;
    const size_t each = V == 1 ? Segments<1>::floats(sh.ctas) : Segments<2>::floats(sh.ctas);
    const size_t all = each * tiles * B;
    most = all > most ? all : most;
  }
  return most;
}
cudaError_t gated_fwd_launch(const GatedCall& q, cudaStream_t s) {
  return q.bf16 ? fwd_t<__nv_bfloat16>(q, s) : fwd_t<float>(q, s);
}
cudaError_t gated_step_launch(const GatedCall& q, cudaStream_t s) {
  return q.bf16 ? step_t<__nv_bfloat16>(q, s) : step_t<float>(q, s);
}

}  // namespace cfc
