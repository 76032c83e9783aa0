// cfc_gated.cuh -- what the passes of the gated linear recurrence share.
//
//   f_t = sigmoid(f_t + bias),   h_t = f_t h_{t-1} + (1 - f_t) x_t,   y_t = h_t silu(z_t)
//
// A warp takes kGatedPeriod steps, a run, of 32 V neighbouring channels (V = 2, or 1 where channels are
// not aligned in pairs) of one sequence at a time.  A composition of steps is again one: over any number
// of them h_out = A h_in + H with A = prod f and H the state that they reach from 0.  Two ways to go
// along the steps from that:
//
//   rounds    the warps of a CTA take runs one after another in time, each forms its A and H at once, and
//             what enters a run is folded from those of the runs before it: a barrier for every 32 or 64
//             steps, and every input is read once.  For as many sequences and channels as fill the GPU.
//   segments  every warp has a stretch of the steps of its own.  A first launch (the summary) forms A and
//             H of each, the second one folds what enters a stretch from those before it and goes through
//             it without a barrier.  For few sequences and channels and many steps: x and f are read
//             twice, but any number of warps takes part.
#pragma once
#include "cfc_gated_kernels.h"
#include "cfc_held8.cuh"
#include "cfc_launch.cuh"
#include "cfc_trunk.cuh"

namespace cfc {

constexpr int kGS = kGatedPeriod;      // steps of a run
constexpr int kGatedWarps = 8;         // most runs of a CTA
constexpr int kMostSplits = 32;        // most CTAs of segments along a sequence
enum GatedMode { kRounds, kSummary, kSegments };
// How a warp reads its runs, by how the tensors are aligned: in pieces of 16 bytes or in pairs of
// channels, both on their way through shared memory (V = 2), or channel by channel into registers.
enum GatedPath { kSixteens, kPairs, kSingles };
__host__ __device__ constexpr int path_v(GatedPath p) { return p == kSingles ? 1 : 2; }

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

// f = sigmoid(logit + bias) and i = 1 - f from t = (logit + bias) log2 e: i = 1 / (1 + 2^t), and
// f = 2^t i where that is the smaller one, else 1 - i, which is rounded to nearest, so that a long
// product of f does not drift with an error of the reciprocal.  Both have fp32's relative precision
// for their t, which is off by 2^-24 of itself and of bias log2 e (a bias is a few units).
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
// Two channels of one step in 8 bits, as they are stored.
struct RawHeld2 {
  uint16_t codes;
  uint8_t byte;
  __device__ __forceinline__ void load(const Held8& h, const HeldAt& at) {
    codes = *reinterpret_cast<const uint16_t*>(h.codes + at.code);
    byte = h.scales[at.scale];
  }
  __device__ __forceinline__ void clear() { codes = 0; byte = 1; }
  __device__ __forceinline__ Fv<2> get() const {
    Fv<2> o;
    o.v = held_values2(codes);
    return o * Fv<2>(held_up(byte));
  }
};

// ---- what enters a run ----

__host__ __device__ constexpr int ah_bytes(int V) { return 32 * V * 2 * static_cast<int>(sizeof(float)); }

// A and H of every run of a round; two rounds in turn, so that one barrier a round is enough: a round's
// values are written over two rounds later, behind a barrier that every reader has passed in between.
// In dynamic shared memory.
template <int V>
struct Exchange {
  static constexpr int kBytes = ah_bytes(V);
  char* base;
  int warps;
  static size_t bytes(int warps) { return static_cast<size_t>(2 * kBytes) * warps; }
  __device__ __forceinline__ char* run(int turn, int i) const {
    return base + (turn * warps + i) * kBytes + threadIdx.x % 32 * (V * 8);
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

// From what entered the round (`carry`) to what enters run w (the result), and on to what leaves the
// round (`carry`), folded in the order of the runs; `REV`: from the last to the first.  `n` counts the
// rounds.  All threads of the CTA call.
template <int V, bool REV>
__device__ __forceinline__ Fv<V> enter(const Exchange<V>& ex, int n, int w, Fv<V> A, Fv<V> H,
                                       Fv<V>& carry) {
  const int warps = ex.warps, turn = n & 1;
  constexpr int kStep = REV ? -Exchange<V>::kBytes : Exchange<V>::kBytes;
  put_ah(ex.run(turn, w), A, H);
  __syncthreads();
  const char* const runs = ex.run(turn, REV ? warps - 1 : 0);
  const Fv<V> in = through<V, 0>(carry, runs, kStep, REV ? warps - 1 - w : w);
  carry = through<V, 4>(carry, runs, kStep, warps);
  return in;
}

// What the two launches over segments share, for one sequence and tile of channels: A and H of every
// warp's segment, of every CTA's segments together, and the state before the first step.
template <int V>
struct Segments {
  static constexpr int kBytes = ah_bytes(V);
  char* base;
  int ctas;
  // Floats of one sequence and tile.
  static size_t floats(int ctas) {
    return static_cast<size_t>(kBytes / sizeof(float)) * (ctas * (kGatedWarps + 1) + 1);
  }
  __device__ __forceinline__ Segments(float* ws, int tiles, int tile, int b, int ctas_)
      : base(reinterpret_cast<char*>(ws + (static_cast<size_t>(b) * tiles + tile) * (kBytes / sizeof(float)) *
                                              (ctas_ * (kGatedWarps + 1) + 1)) +
             threadIdx.x % 32 * (V * 8)),
        ctas(ctas_) {}
  __device__ __forceinline__ char* warp(int c, int w) const {
    return base + (c * kGatedWarps + w) * kBytes;
  }
  __device__ __forceinline__ char* cta(int c) const { return base + (ctas * kGatedWarps + c) * kBytes; }
  __device__ __forceinline__ char* start() const { return base + ctas * (kGatedWarps + 1) * kBytes; }

  // A warp's A and H, and its CTA's.  All threads of the CTA call; `ex` lies in shared memory.
  template <bool REV>
  __device__ __forceinline__ void put(const Exchange<V>& ex, int c, int w, Fv<V> A, Fv<V> H) const {
    put_ah(ex.run(0, w), A, H);
    put_ah(warp(c, w), A, H);
    __syncthreads();
    if (w > 0) return;
    Fv<V> a(1.f), h(0.f);
#pragma unroll
    for (int i = 0; i < kGatedWarps; ++i) {
      Fv<V> ra, rh;
      get_ah(ex.run(0, REV ? kGatedWarps - 1 - i : i), ra, rh);
      h = fma(ra, h, rh);
      a = a * ra;
    }
    put_ah(cta(c), a, h);
  }
  // What enters warp w's segment of CTA c: v through those before it, `REV`: behind it.
  template <bool REV>
  __device__ __forceinline__ Fv<V> enter(Fv<V> v, int c, int w) const {
    constexpr int kStep = REV ? -kBytes : kBytes;
    v = batches(v, cta(REV ? ctas - 1 : 0), kStep, REV ? ctas - 1 - c : c);
    return batches(v, warp(c, REV ? kGatedWarps - 1 : 0), kStep, REV ? kGatedWarps - 1 - w : w);
  }
  // Eight values on their way from L2 at a time.
  static __device__ __forceinline__ Fv<V> batches(Fv<V> v, const char* p, int step, int count) {
    for (int i = 0; i < count; i += 8) {
      Fv<V> a[8], h[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i + j < count) get_ah(p + (i + j) * step, a[j], h[j]);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i + j < count) v = fma(a[j], v, h[j]);
    }
    return v;
  }
};

// ---- runs on their way ----

// One tensor's runs of kGS steps x 64 channels on their way to shared memory, copied in the background
// 4, 8 or 16 bytes (CB) a lane.  A warp copies and reads its own runs only, so no barrier is needed but
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
    else if constexpr (CB == 8)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(p), "r"(bytes)
                   : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(p), "r"(bytes)
                   : "memory");
  }
  // `base`: the tensor at step 0 and the tile's first channel, `stride` elements a step; t0: the
  // first run's first step.  Of the tile's channels `left` exist.
  __device__ __forceinline__ void start(const void* base, long long stride, int t0, int left) {
    const int lane = threadIdx.x % 32, c = lane % kLanes * CB;
    from = static_cast<const char*>(base) + (c < left * ES ? c : 0) +
           (t0 + lane / kLanes) * stride * ES;
  }
  // The run `ahead` bytes further to `dst`: zeros for its steps from `on` on and for channels that do
  // not exist, neither of which is read.
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

// How the steps of a sequence are gone along: by CTAs of `warps` warps in rounds (ctas = 0), or by `ctas`
// CTAs of kGatedWarps segments of `steps` steps.
struct GatedShape {
  int warps, ctas, steps;
};
// `slots`: CTAs of segments that the GPU holds.
inline GatedShape gated_shape(int B, int K, int tiles, int slots) {
  const int runs = (K - 1) / kGS + 1;
  const long long columns = static_cast<long long>(tiles) * B;
  // Rounds of four warps where there are columns enough for two CTAs an SM: their barrier waits least
  // (64 x 1024 steps x 1536 channels, bf16: forward 133 us, backward 249; eight warps 143 and 312, two
  // 167 and 305).
  GatedShape s{columns >= 2 * 152 ? 4 : kGatedWarps, 0, 0};
  if (runs < s.warps) s.warps = runs;
  // Segments from 448 steps and below 100 columns: with 64 columns of 4096 steps they take 41 us forward
  // and 74 backward (rounds 82 and 109), with 128 of 2048 steps 41 and 73 (43 and 60), with 64 of 512
  // steps 10 and 16 (13 and 19), with 128 of 256 steps 10 and 16 (8 and 12).
  if (columns >= 100 || K < 448) return s;
  // Full waves of them, two or one.
  long long ctas = 2 * slots / columns;
  if (ctas > kMostSplits) ctas = slots / columns;
  if (ctas > kMostSplits) ctas = kMostSplits;
  if (ctas > runs / (2 * kGatedWarps)) ctas = runs / (2 * kGatedWarps);
  if (ctas < 1) return s;
  const int segments = static_cast<int>(ctas) * kGatedWarps;
  s.steps = ((runs - 1) / segments + 1) * kGS;
  s.ctas = (K - 1) / (s.steps * kGatedWarps) + 1;
  s.warps = kGatedWarps;
  return s;
}
constexpr int kFwdSlots = 3 * 152, kBwdSlots = 2 * 152;
// Dynamic shared memory of a CTA: `ring` bytes a warp (0: without one) and the exchange.
template <int V>
size_t gated_smem(int warps, size_t ring) {
  return Exchange<V>::bytes(warps) + warps * ring;
}

}  // namespace cfc
