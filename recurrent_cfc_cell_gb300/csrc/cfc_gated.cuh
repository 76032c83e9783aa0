// cfc_gated.cuh -- what the passes of the gated linear recurrence share.
//
//   f_t = sigmoid(f_t + bias),   h_t = f_t h_{t-1} + (1 - f_t) x_t,   y_t = h_t silu(z_t)
//
// A warp takes kGatedPeriod steps of 32 V neighbouring channels (V = 2, or 1 where channels are not
// aligned in pairs) of one sequence.  A composition of steps is again one: over a run of them
// h_out = A h_in + H with A = prod f and H the state that the run reaches from 0.  So the warps of
// a cluster take runs one after another in time, each forms its A and H at once, and what enters a
// run is folded from those of the runs before it: K / (steps of a cluster) rounds with an exchange
// each take the place of K steps one after another, and every input is read once.
#pragma once
#include "cfc_gated_kernels.h"
#include "cfc_held8.cuh"
#include "cfc_launch.cuh"
#include "cfc_trunk.cuh"

namespace cfc {

constexpr int kGS = kGatedPeriod;      // steps of a run
constexpr int kGatedWarps = 8;         // most runs of a CTA
constexpr int kGatedCluster = 16;      // most CTAs of a cluster

// V channels in a lane's registers: a float, or a pair that the packed fp32 instructions take.
template <int V>
struct Fv;
template <>
struct Fv<1> {
  float v;
  __device__ __forceinline__ Fv() {}
  __device__ __forceinline__ explicit Fv(float x) : v(x) {}
  __device__ __forceinline__ float operator[](int) const { return v; }
  __device__ __forceinline__ float& operator[](int) { return v; }
};
template <>
struct Fv<2> {
  float2 v;
  __device__ __forceinline__ Fv() {}
  __device__ __forceinline__ explicit Fv(float x) : v(make_float2(x, x)) {}
  __device__ __forceinline__ float operator[](int j) const { return j ? v.y : v.x; }
  __device__ __forceinline__ float& operator[](int j) { return j ? v.y : v.x; }
};
__device__ __forceinline__ Fv<1> operator*(Fv<1> a, Fv<1> b) { return Fv<1>(a.v * b.v); }
__device__ __forceinline__ Fv<1> operator+(Fv<1> a, Fv<1> b) { return Fv<1>(a.v + b.v); }
__device__ __forceinline__ Fv<1> fma(Fv<1> a, Fv<1> b, Fv<1> c) { return Fv<1>(fmaf(a.v, b.v, c.v)); }
__device__ __forceinline__ Fv<2> operator*(Fv<2> a, Fv<2> b) {
  a.v = __fmul2_rn(a.v, b.v);
  return a;
}
__device__ __forceinline__ Fv<2> operator+(Fv<2> a, Fv<2> b) {
  a.v = __fadd2_rn(a.v, b.v);
  return a;
}
__device__ __forceinline__ Fv<2> fma(Fv<2> a, Fv<2> b, Fv<2> c) {
  a.v = fma2(a.v, b.v, c.v);
  return a;
}

constexpr float kLog2e = 1.4426950408889634f;

// f = sigmoid(logit + bias) and i = 1 - f, both to full relative precision, from t = (logit + bias)
// log2 e: i = 1 / (1 + 2^t), and f = 2^t i where that is the smaller one, else 1 - i, which is
// rounded to nearest, so that a long product of f does not drift with an error of the reciprocal.
// `bias2` is bias log2 e.  2^t may be infinite: i is 0 then and f 1.
template <int V>
__device__ __forceinline__ void gates(Fv<V> logit, Fv<V> bias2, Fv<V>& f, Fv<V>& i) {
  const Fv<V> t = fma(logit, Fv<V>(kLog2e), bias2);
  Fv<V> e;
#pragma unroll
  for (int j = 0; j < V; ++j) e[j] = exp2_f(t[j]);
  const Fv<V> d = e + Fv<V>(1.f);
#pragma unroll
  for (int j = 0; j < V; ++j) i[j] = rcp_f(d[j]);
  const Fv<V> small = e * i, large = fma(i, Fv<V>(-1.f), Fv<V>(1.f));
#pragma unroll
  for (int j = 0; j < V; ++j) f[j] = t[j] < 0.f ? small[j] : large[j];
}

// sigmoid(z).
template <int V>
__device__ __forceinline__ Fv<V> logistic(Fv<V> z) {
  Fv<V> t = z * Fv<V>(-kLog2e);
#pragma unroll
  for (int j = 0; j < V; ++j) t[j] = exp2_f(t[j]);
  t = t + Fv<V>(1.f);
#pragma unroll
  for (int j = 0; j < V; ++j) t[j] = rcp_f(t[j]);
  return t;
}

// V channels of one step as they are stored.
template <typename T, int V>
struct RawV;
template <>
struct RawV<float, 1> {
  float v;
  __device__ __forceinline__ void load(const float* p) { v = *p; }
  __device__ __forceinline__ void clear() { v = 0.f; }
  __device__ __forceinline__ Fv<1> get() const { return Fv<1>(v); }
};
template <>
struct RawV<float, 2> {
  float2 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float2*>(p); }
  __device__ __forceinline__ void clear() { v = make_float2(0.f, 0.f); }
  __device__ __forceinline__ Fv<2> get() const {
    Fv<2> o;
    o.v = v;
    return o;
  }
};
template <>
struct RawV<__nv_bfloat16, 1> {
  unsigned short v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    v = *reinterpret_cast<const unsigned short*>(p);
  }
  __device__ __forceinline__ void clear() { v = 0; }
  __device__ __forceinline__ Fv<1> get() const {
    return Fv<1>(__uint_as_float(static_cast<uint32_t>(v) << 16));
  }
};
template <>
struct RawV<__nv_bfloat16, 2> {
  uint32_t v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    v = *reinterpret_cast<const uint32_t*>(p);
  }
  __device__ __forceinline__ void clear() { v = 0u; }
  __device__ __forceinline__ Fv<2> get() const {
    Fv<2> o;
    o.v = make_float2(bf16_lo_f32(v), bf16_hi_f32(v));
    return o;
  }
};
__device__ __forceinline__ void store_v(float* p, Fv<1> v) { *p = v.v; }
__device__ __forceinline__ void store_v(float* p, Fv<2> v) { *reinterpret_cast<float2*>(p) = v.v; }
__device__ __forceinline__ void store_v(__nv_bfloat16* p, Fv<1> v) { *p = __float2bfloat16_rn(v.v); }
__device__ __forceinline__ void store_v(__nv_bfloat16* p, Fv<2> v) {
  *reinterpret_cast<uint32_t*>(p) = bf16x2_rn(v.v.x, v.v.y);
}

// A lane's place: its channels and which of them exist.
template <int V>
struct Channels {
  int d;       // first channel
  bool in;     // it exists (V = 2: D is even, so both do)
  __device__ __forceinline__ Channels(int tile, int D)
      : d((tile * 32 + static_cast<int>(threadIdx.x) % 32) * V), in(d < D) {}
};

template <int V>
__device__ __forceinline__ Fv<V> load_par_v(const float* p, const Channels<V>& c) {
  Fv<V> v(0.f);
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (p && c.in) v[j] = __ldg(p + c.d + j);
  return v;
}

// Where the element (step, sequence, channel) of an [K][B][D] tensor held in 8 bits lies.
struct HeldAt {
  size_t code, scale;
};
template <int V>
__device__ __forceinline__ HeldAt held_at(const GatedCall& q, int t, int b, int d) {
  const size_t row = static_cast<size_t>(t) * q.B + b;
  return {row * q.D + d, row * held_blocks(q.D) + d / kHeldBlock};
}
// V channels a lane to 8 bits: a block is 32 / V lanes.
template <int V>
__device__ __forceinline__ void store_held_v(const Held8& h, const HeldAt& at, Fv<V> v, bool in) {
  uint32_t byte, codes;
  if constexpr (V == 1) {
    codes = held_pack1(v[0], byte);
    if (in) h.codes[at.code] = static_cast<uint8_t>(codes);
  } else {
    uint32_t most = max(magnitude_bits(v[0]), magnitude_bits(v[1]));
#pragma unroll
    for (int d = 1; d < 16; d *= 2) most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
    byte = held_scale_byte(most);
    const float down = held_down(byte);
    codes = held_codes2(v[0] * down, v[1] * down);
    if (in) *reinterpret_cast<uint16_t*>(h.codes + at.code) = static_cast<uint16_t>(codes);
  }
  if (in && threadIdx.x % (32 / V) == 0) h.scales[at.scale] = static_cast<uint8_t>(byte);
}

// V channels of one step in 8 bits, as they are stored.
template <int V>
struct RawHeldV {
  uint16_t codes;
  uint8_t byte;
  __device__ __forceinline__ void load(const Held8& h, const HeldAt& at) {
    codes = V == 1 ? h.codes[at.code] : *reinterpret_cast<const uint16_t*>(h.codes + at.code);
    byte = h.scales[at.scale];
  }
  __device__ __forceinline__ void clear() { codes = 0; byte = 1; }
  __device__ __forceinline__ Fv<V> get() const {
    const float2 p = held_values2(codes);
    Fv<V> o;
    o[0] = p.x;
    if constexpr (V == 2) o[1] = p.y;
    return o * Fv<V>(held_up(byte));
  }
};

// ---- what enters a run ----

// A and H of every run of a round and, in a cluster, of every CTA's runs together; two rounds in
// turn, so that one barrier a round is enough: a round's values are written over two rounds later,
// behind a barrier that every reader has passed in between (of other CTAs' values: behind this CTA's
// own values of the round in between, which the others wait for).  In dynamic shared memory.
template <int V>
struct Exchange {
  static constexpr int kBytes = 32 * V * 2 * sizeof(float);  // a run's values
  char* base;
  int warps, ctas;
  uint32_t bars;   // two barriers: the values of all CTAs have arrived
  int* status;     // where a wait that ran out is reported
  static size_t bytes(int warps, int ctas) {
    return static_cast<size_t>(2 * kBytes) * (warps + (ctas > 1 ? ctas : 0));
  }
  __device__ __forceinline__ char* run(int turn, int i) const {
    return base + (turn * warps + i) * kBytes + threadIdx.x % 32 * (V * 8);
  }
  __device__ __forceinline__ char* cta(int turn, int i) const {
    return base + (2 * warps + turn * ctas + i) * kBytes + threadIdx.x % 32 * (V * 8);
  }
  // All threads call, before the first round.  Behind it other CTAs may write to this one.
  __device__ __forceinline__ void start() const {
    if (ctas == 1) return;
    if (threadIdx.x == 0) {
      mbar_init(bars, 1);
      mbar_init(bars + 8, 1);
      fence_mbar_init_cluster();
      mbar_arrive_expect_tx(bars, ctas * kBytes);
      mbar_arrive_expect_tx(bars + 8, ctas * kBytes);
    }
    cluster_sync_all();
  }
};

__device__ __forceinline__ void put_ah(char* p, Fv<1> a, Fv<1> h) {
  *reinterpret_cast<float2*>(p) = make_float2(a.v, h.v);
}
__device__ __forceinline__ void put_ah(char* p, Fv<2> a, Fv<2> h) {
  *reinterpret_cast<float4*>(p) = make_float4(a.v.x, a.v.y, h.v.x, h.v.y);
}
__device__ __forceinline__ void get_ah(const char* p, Fv<1>& a, Fv<1>& h) {
  const float2 r = *reinterpret_cast<const float2*>(p);
  a.v = r.x;
  h.v = r.y;
}
__device__ __forceinline__ void get_ah(const char* p, Fv<2>& a, Fv<2>& h) {
  const float4 r = *reinterpret_cast<const float4*>(p);
  a.v = make_float2(r.x, r.y);
  h.v = make_float2(r.z, r.w);
}
__device__ __forceinline__ void send_ah(uint32_t at, Fv<1> a, Fv<1> h, uint32_t bar) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(at),
      "r"(__float_as_uint(a.v)), "r"(__float_as_uint(h.v)), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void send_ah(uint32_t at, Fv<2> a, Fv<2> h, uint32_t bar) {
  st_async_v4(at, a.v.x, a.v.y, h.v.x, h.v.y, bar);
}

// v through the compositions at p, p + step, ...; most of the time there are N of them.
template <int V, int N>
__device__ __forceinline__ Fv<V> through(Fv<V> v, const char* p, int step, int count) {
  if (count == N) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      Fv<V> a, h;
      get_ah(p + i * step, a, h);
      v = fma(a, v, h);
    }
    return v;
  }
#pragma unroll 1
  for (; count > 0; --count, p += step) {
    Fv<V> a, h;
    get_ah(p, a, h);
    v = fma(a, v, h);
  }
  return v;
}

// From what entered the round (`carry`) to what enters run w of CTA `rank` (the result), and on to
// what leaves the round (`carry`), folded in the order of the runs; `REV`: from the last to the
// first.  `n` counts the rounds.  All threads of the cluster call.
template <int V, bool REV>
__device__ __forceinline__ Fv<V> enter(const Exchange<V>& ex, int n, int w, int rank, Fv<V> A,
                                       Fv<V> H, Fv<V>& carry) {
  const int warps = ex.warps, ctas = ex.ctas, turn = n & 1;
  constexpr int kStep = REV ? -Exchange<V>::kBytes : Exchange<V>::kBytes;
  put_ah(ex.run(turn, w), A, H);
  __syncthreads();
  const char* const runs = ex.run(turn, REV ? warps - 1 : 0);
  const int before = REV ? warps - 1 - w : w;
  if (ctas == 1) {
    const Fv<V> in = through<V, 0>(carry, runs, kStep, before);
    carry = through<V, 4>(carry, runs, kStep, warps);
    return in;
  }
  const uint32_t bar = ex.bars + 8 * turn;
  // Each warp sends the CTA's A and H to the CTAs w, w + warps, ...
  if (w < ctas) {
    Fv<V> a(1.f), h(0.f);
#pragma unroll
    for (int i = 0; i < kGatedWarps; ++i) {
      if (i >= warps) break;
      Fv<V> ra, rh;
      get_ah(runs + i * kStep, ra, rh);
      h = fma(ra, h, rh);
      a = a * ra;
    }
    const uint32_t mine = smem_addr(ex.cta(turn, rank));
    for (int to = w; to < ctas; to += warps)
      send_ah(map_to_rank(mine, to), a, h, map_to_rank(bar, to));
  }
  __syncwarp();
  (void)mbar_wait_bounded_cluster(bar, (n >> 1) & 1, ex.status);
  if (threadIdx.x == 0) mbar_arrive_expect_tx(bar, ctas * Exchange<V>::kBytes);  // for n + 2
  const char* const all = ex.cta(turn, REV ? ctas - 1 : 0);
  const Fv<V> in = through<V, 0>(carry, all, kStep, REV ? ctas - 1 - rank : rank);
  carry = through<V, kGatedCluster>(carry, all, kStep, ctas);
  return through<V, 0>(in, runs, kStep, before);
}

// ---- runs on their way ----

// One tensor's runs of kGS steps x 64 channels on their way to shared memory, copied in the background
// 8 or 16 bytes (CB) a lane.  A warp copies and reads its own runs only, so no barrier is needed but
// the warp's.
template <int ES, int CB>  // bytes of an element, of a copy
struct RingRun {
  static constexpr int kRow = 64 * ES, kBytes = kGS * kRow;
  static constexpr int kLanes = kRow / CB, kRows = 32 / kLanes;  // lanes a row, rows a copy
  // What this lane copies first of the first run.
  const char* from;
  static __device__ __forceinline__ void copy_one(uint32_t to, const char* p, int bytes) {
    if constexpr (CB == 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(p), "r"(bytes)
                   : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(p), "r"(bytes)
                   : "memory");
  }
  // `base`: the tensor at step 0 and the tile's first channel, `stride` elements a step; t0: the
  // first run's first step.  Of the tile's channels `left` exist.
  __device__ __forceinline__ void start(const void* base, long long stride, int t0, int left) {
    const int lane = threadIdx.x % 32, c = lane % kLanes * CB;
    from = static_cast<const char*>(base) + (c < left * ES ? c : 0) +
           (t0 + lane / kLanes) * stride * ES;
  }
  // The run `ahead` bytes further to `dst`: zeros for its steps from `on` on and for channels that do not exist, neither of
  // which is read.
  __device__ __forceinline__ void copy(uint32_t dst, long long ahead, long long stride, int on,
                                       int left) const {
    const int lane = threadIdx.x % 32;
    const uint32_t to = dst + lane / kLanes * kRow + lane % kLanes * CB;
    const int bytes = lane % kLanes * CB < left * ES ? CB : 0;
    const long long step = stride * (kRows * ES);
    // One form for runs that are there as a whole and others: with a branch between the two the
    // backward pass of 64 x 1024 steps x 1536 channels took 284 us, without it 249.
#pragma unroll
    for (int i = 0; i < kGS / kRows; ++i) {
      const bool there = i * kRows + lane / kLanes < on;
      copy_one(to + i * kRows * kRow,
               there ? from + ahead + i * step : from + ahead - lane / kLanes * (stride * ES),
               there ? bytes : 0);
    }
  }
};
template <typename T>
__device__ __forceinline__ Fv<2> ring_get(const char* run, int k) {
  RawV<T, 2> r;
  r.load(reinterpret_cast<const T*>(run + k * 64 * sizeof(T)) + 2 * (threadIdx.x % 32));
  return r.get();
}

// ---- launches ----

// Channels of a tensor are aligned in groups of `bytes`, `per` of them.
inline bool group_aligned(const void* p, long long t, long long b, int bytes, int per) {
  return !p || (reinterpret_cast<uintptr_t>(p) % bytes == 0 && t % per == 0 && b % per == 0);
}

// How the runs of a sequence are spread: warps of a CTA, CTAs of a cluster.
struct GatedShape {
  int warps, ctas;
};
// A CTA of four warps where there are columns enough for two CTAs an SM: its barrier waits least
// (64 x 1024 steps x 1536 channels, bf16: forward 148 us, backward 247; eight warps 163 and 259, two
// 167 and 305).  Fewer columns take longer rounds, and at last clusters.
inline GatedShape gated_shape(const GatedCall& q, int tiles) {
  const int runs = (q.K - 1) / kGS + 1;
  const long long columns = static_cast<long long>(tiles) * q.B;
  GatedShape s{columns >= 2 * 152 ? 4 : kGatedWarps, 1};
  if (runs < s.warps) s.warps = runs;
  while (s.ctas < kGatedCluster && columns * s.ctas < 152 && runs > s.warps * s.ctas) s.ctas *= 2;
  return s;
}
template <typename F>
cudaError_t gated_attributes(F* kern, size_t smem, int ctas) {
  cudaError_t e = cudaSuccess;
  if (smem > 16 * 1024)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem));
  if (e == cudaSuccess && ctas > 8)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  return e;
}

}  // namespace cfc
