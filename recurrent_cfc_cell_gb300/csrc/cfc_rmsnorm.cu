// cfc_rmsnorm.cu -- root-mean-square norm over rows with the residual's addition, forward and
// backward, its results and its stream in the activations' type or held in 8 bits.
//
//   forward   s = x + residual                        (rounded to its type; s = x without)
//             rstd = (sum s^2 / n + eps)^-1/2,  y = s rstd w
//   backward  hat = s rstd,  g = dy w
//             dx = rstd (g - hat sum(g hat) / n) + ds,  dw = sum_rows dy hat
//
// Every pass is bound by memory: a row stays in registers between its sum and its results.  A row
// belongs to a team: 4 to 32 lanes of a warp up to 256 columns, a CTA of up to 1024 threads up to 8192.
// Longer rows are read twice (the second time from L2) and element by element, a CTA a row (16384 x 12288
// bf16 625 us forward, 2.6 TB/s, and 896 backward).  Lanes load and store eight columns at once;
// where rows start anywhere (an odd width) their groups of eight follow the memory's alignment, and
// the row's two ends are stored element by element.  Tensors that are aligned differently from one
// another, and odd widths in 8 bits, whose blocks begin with the row, are done element by element:
// neighbouring lanes have neighbouring columns, and a warp holds a block.
//
// 262144 x 256 rows with a residual: bf16 85 us forward (6.3 TB/s) and 95 backward with dw's second
// launch (5.7), fp32 162 and 162 (6.6), with the stream kept in 8 bits 171 and 176.  9001 x 1537 bf16
// takes 25 and 33 us (4.5 and 3.3 TB/s): the rows' ends, stored one by one, and a barrier a row cost
// as many instructions as the rest of them.
//
// dw is summed in each lane's registers over the rows of its team, over the CTA's teams in shared
// memory, and over the CTAs by a second launch: no atomics, an order that depends on the sizes and on
// the rows' alignment.
#include "cfc_gated_kernels.h"
#include "cfc_held8.cuh"
#include "cfc_launch.cuh"
#include "cfc_trunk.cuh"

#include <type_traits>

namespace cfc {
namespace {

constexpr int kSms = 152;
constexpr int kLongRow = 8192;   // columns from which rows are read twice

// How rows lie.  kScalar: anyhow; a thread's columns are a team apart, so that a warp's accesses are
// consecutive.  kAligned: every row of every tensor starts on a group of eight columns.  kShifted:
// row r of every tensor starts at the same place within a group of eight (an odd width, say): a
// thread's groups follow the memory's alignment, and what of a group lies in the rows before and
// after is left out.
enum Layout { kScalar, kAligned, kShifted };

// A team of up to TPR threads a row, SLOTS pieces a thread; a piece is eight columns, or one
// (kScalar).  Teams of a warp's lanes have TPR of them; the others are a whole CTA, of as many warps
// as the row needs.
template <int TPR_, int SLOTS_, Layout LY_>
struct Team {
  static constexpr int TPR = TPR_, SLOTS = SLOTS_;
  static constexpr Layout LY = LY_;
  static constexpr bool VEC = LY != kScalar, kWarp = TPR <= 32;
  static constexpr int W = VEC ? 8 : 1;            // columns of a piece
  static constexpr int E = SLOTS * W;              // columns of a thread
  static constexpr int kThreads = kWarp ? 256 : TPR;
  static constexpr int kTeams = kThreads / TPR;
  static constexpr int kCols = TPR * E;
  static __device__ __forceinline__ int team() { return kWarp ? threadIdx.x / TPR : 0; }
};

// A thread's columns.
template <typename TM>
struct At {
  int n, rows, first, step;  // first: its first column, step: from a piece's to the next one's
  // `row0`: the team's first row of a tensor (kShifted: all its rows start at the same place).
  template <typename T>
  __device__ __forceinline__ At(int n_, int rows_, const T* row0) : n(n_), rows(rows_) {
    const int lane = TM::kWarp ? threadIdx.x % TM::TPR : threadIdx.x;
    first = lane * TM::W;
    step = (TM::kWarp ? TM::TPR : static_cast<int>(blockDim.x)) * TM::W;
    if constexpr (TM::LY == kShifted)
      first -= static_cast<int>(reinterpret_cast<uintptr_t>(row0) / sizeof(T) % 8);
  }
  __device__ __forceinline__ int col(int slot) const { return first + slot * step; }
  // Column i of a piece is in the row.
  __device__ __forceinline__ bool in(int slot, int i) const {
    return static_cast<unsigned>(col(slot) + i) < static_cast<unsigned>(n);
  }
  // Some of the piece is in the row; all of it is.
  __device__ __forceinline__ bool some(int slot) const {
    return col(slot) < n && (TM::LY != kShifted || col(slot) > -8);
  }
  __device__ __forceinline__ bool whole(int slot) const {
    return TM::LY != kShifted || (col(slot) >= 0 && col(slot) + 8 <= n);
  }
};

__device__ __forceinline__ void add8(Raw8<float>& a, const Raw8<float>& b) {
#pragma unroll
  for (int j = 0; j < 8; ++j) a.v[j] += b.v[j];
}
__device__ __forceinline__ void add8(Raw8<__nv_bfloat16>& a, const Raw8<__nv_bfloat16>& b) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    a.w[j] = bf16x2_rn(bf16_lo_f32(a.w[j]) + bf16_lo_f32(b.w[j]),
                       bf16_hi_f32(a.w[j]) + bf16_hi_f32(b.w[j]));
}
__device__ __forceinline__ void store_raw(float* p, const Raw8<float>& r) { store8(p, r.v); }
__device__ __forceinline__ void store_raw(__nv_bfloat16* p, const Raw8<__nv_bfloat16>& r) {
  *reinterpret_cast<uint4*>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
}

// A thread's columns of row `row` as they are stored; columns that are not in the row come out as 0.
template <typename T, typename TM>
struct Piece {
  std::conditional_t<TM::VEC, Raw8<T>, T> raw[TM::SLOTS];
  __device__ __forceinline__ void load(const At<TM>& at, const T* p, long long row, bool ok) {
#pragma unroll
    for (int j = 0; j < TM::SLOTS; ++j) {
      const int c = at.col(j);
      if constexpr (!TM::VEC) {
        raw[j] = ok && c < at.n ? p[c] : from_f32<T>(0.f);
      } else if (!(ok && at.some(j))) {
        raw[j].clear();
      } else if (TM::LY == kAligned || ((c >= 0 || row > 0) && (c + 8 <= at.n || row + 1 < at.rows))) {
        // At its row's ends a group reaches into the rows before and after, but for the tensor's
        // first and last one.
        raw[j].load(p + c);
      } else {
        raw[j].clear();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (at.in(j, i)) raw[j].set(i, p[c + i]);
      }
    }
  }
  __device__ __forceinline__ void get(const At<TM>& at, float (&v)[TM::E]) const {
#pragma unroll
    for (int j = 0; j < TM::SLOTS; ++j) {
      if constexpr (!TM::VEC) {
        v[j] = to_f32(raw[j]);
      } else {
        float p[8];
        raw[j].get(p);
        if (!at.whole(j)) {
#pragma unroll
          for (int i = 0; i < 8; ++i) p[i] = at.in(j, i) ? p[i] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[8 * j + i] = p[i];
      }
    }
  }
  // The sum with another row's, rounded to T.
  __device__ __forceinline__ void add(const Piece& r) {
#pragma unroll
    for (int j = 0; j < TM::SLOTS; ++j) {
      if constexpr (TM::VEC) add8(raw[j], r.raw[j]);
      else raw[j] = from_f32<T>(to_f32(raw[j]) + to_f32(r.raw[j]));
    }
  }
};

template <typename TM, typename T>
__device__ __forceinline__ void store_row(const At<TM>& at, T* row, const float (&v)[TM::E], bool ok) {
#pragma unroll
  for (int j = 0; j < TM::SLOTS; ++j) {
    if (!(ok && at.some(j))) continue;
    if constexpr (TM::VEC) {
      if (at.whole(j)) {
        float p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = v[8 * j + i];
        store8(row + at.col(j), p);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (at.in(j, i)) row[at.col(j) + i] = from_f32<T>(v[8 * j + i]);
      }
    } else {
      row[at.col(j)] = from_f32<T>(v[j]);
    }
  }
}
// The same of values that are held as T already.
template <typename TM, typename T>
__device__ __forceinline__ void store_row(const At<TM>& at, T* row, const Piece<T, TM>& x,
                                          const float (&v)[TM::E], bool ok) {
#pragma unroll
  for (int j = 0; j < TM::SLOTS; ++j) {
    if (!(ok && at.some(j))) continue;
    if constexpr (TM::VEC) {
      if (at.whole(j)) {
        store_raw(row + at.col(j), x.raw[j]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (at.in(j, i)) row[at.col(j) + i] = from_f32<T>(v[8 * j + i]);
      }
    } else {
      row[at.col(j)] = x.raw[j];
    }
  }
}

template <typename TM>
__device__ __forceinline__ void load_par(const At<TM>& at, const float* p, float (&v)[TM::E]) {
#pragma unroll
  for (int j = 0; j < TM::SLOTS; ++j)
#pragma unroll
    for (int i = 0; i < TM::W; ++i)
      v[j * TM::W + i] = at.in(j, i) ? __ldg(p + at.col(j) + i) : 0.f;
}

// A row to 8 bits (all lanes of every warp call; columns that do not exist hold 0).
template <typename TM>
__device__ __forceinline__ void store_held(const At<TM>& at, const Held8& h, long long row,
                                           const float (&v)[TM::E], bool ok) {
  uint8_t* const codes = h.codes + row * at.n;
  uint8_t* const scales = h.scales + row * held_blocks(at.n);
#pragma unroll
  for (int j = 0; j < TM::SLOTS; ++j) {
    const int c = at.col(j);
    const bool in = ok && c < at.n;
    uint32_t byte;
    if constexpr (TM::VEC) {
      float p[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = v[8 * j + i];
      const uint2 r = held_pack8(p, byte);
      if (in) *reinterpret_cast<uint2*>(codes + c) = r;
    } else {
      const uint32_t r = held_pack1(v[j], byte);
      if (in) codes[c] = static_cast<uint8_t>(r);
    }
    if (in && c % kHeldBlock == 0) scales[c / kHeldBlock] = static_cast<uint8_t>(byte);
  }
}
// A thread's columns of a row in 8 bits, as they are held.
template <typename TM>
struct HeldPiece {
  using C = std::conditional_t<TM::VEC, uint2, uint8_t>;
  C codes[TM::SLOTS];
  uint8_t byte[TM::SLOTS];
  __device__ __forceinline__ void load(const At<TM>& at, const Held8& h, long long row, bool ok) {
#pragma unroll
    for (int j = 0; j < TM::SLOTS; ++j) {
      const int c = at.col(j);
      const bool in = ok && c < at.n;
      codes[j] = in ? *reinterpret_cast<const C*>(h.codes + row * at.n + c) : C{};
      byte[j] = in ? h.scales[row * held_blocks(at.n) + c / kHeldBlock] : uint8_t(1);
    }
  }
  __device__ __forceinline__ void get(float (&v)[TM::E]) const {
#pragma unroll
    for (int j = 0; j < TM::SLOTS; ++j) {
      if constexpr (TM::VEC) {
        float p[8];
        held_unpack8(codes[j], byte[j], p);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[8 * j + i] = p[i];
      } else {
        v[j] = held_values2(codes[j]).x * held_up(byte[j]);
      }
    }
  }
};

// The sum over a row's team, in every thread.  `part` holds two rows' partial sums in turn, so that
// one barrier a row is enough.
template <typename TM>
__device__ __forceinline__ float team_sum(float v, float (*part)[32], int turn) {
  constexpr int kLanes = TM::kWarp ? TM::TPR : 32;
#pragma unroll
  for (int d = kLanes / 2; d > 0; d /= 2) v += __shfl_xor_sync(0xffffffffu, v, d);
  if constexpr (!TM::kWarp) {
    float* const p = part[turn & 1];
    const int lane = threadIdx.x % 32;
    if (lane == 0) p[threadIdx.x / 32] = v;
    __syncthreads();
    v = lane < static_cast<int>(blockDim.x) / 32 ? p[lane] : 0.f;
    constexpr int kMost = TM::TPR / 32;  // a power of two
#pragma unroll
    for (int d = kMost / 2; d > 0; d /= 2) v += __shfl_xor_sync(0xffffffffu, v, d);
    v = __shfl_sync(0xffffffffu, v, 0);
  }
  return v;
}

// (sum / n + eps)^-1/2: the hardware's estimate and one step of Newton's iteration.  An estimate
// of 0 or infinity stays as it is.
__device__ __forceinline__ float rstd_of(float sum, int n, float eps) {
  const float m = sum / static_cast<float>(n) + eps;
  const float r = rsqrtf(m);
  const float better = r * fmaf(-0.5f * m * r, r, 1.5f);
  return r > 0.f && r < 1e18f && m < 1e38f ? better : r;
}

// s rstd w rounded once: the product s rstd, n^1/2 at most, is kept in two parts.  (s w could be beyond
// fp32 where y is not.)
__device__ __forceinline__ float normed(float s, float w, float rstd) {
  const float p = __fmul_rn(s, rstd);
  const float low = fmaf(s, rstd, -p);
  return fmaf(p, w, low * w);
}

// ---- y to 8 bits ----
//
// Next to a border between two codes an error in the last place of y decides which one it becomes, and
// a code is 2^-3 of the value.  So y is formed in two fp32 parts, from a sum of squares in two parts
// (relative error below 1e-12), and rounded to fp32 to odd: where something is left behind the last
// place, that place is set, so that a value beside a border stays on its side of it in the rounding to
// three bits that follows.  16384 x 2048 bf16: 70 us, bound by instructions (47 us with sums and products
// in fp32, whose codes differ beside borders).

struct Two {  // hi + lo, |lo| at most half a place of hi
  float hi, lo;
};
// a + b where |a| >= |b| or a is 0; Dekker's sum.
__device__ __forceinline__ Two fast_two(float a, float b) {
  const float s = a + b;
  return {s, b - (s - a)};
}
// a + b of two sums; Knuth's sum of the high parts, whose rest joins the low ones, which nothing but
// sums of theirs follows: they are put right at the end.
__device__ __forceinline__ Two plus(Two a, Two b) {
  const float s = a.hi + b.hi, t = s - a.hi;
  const float rest = (a.hi - (s - t)) + (b.hi - t);
  return {s, a.lo + b.lo + rest};
}

// The same for the two columns of a pair, in packed arithmetic.
struct Pair {
  float2 hi, lo;
};
__device__ __forceinline__ float2 neg2(float2 a) { return make_float2(-a.x, -a.y); }
// v + a^2.  `EXACT`: the squares of bf16 values are exact in fp32.
template <bool EXACT>
__device__ __forceinline__ Pair plus_square(Pair v, float2 a) {
  const float2 p = __fmul2_rn(a, a);
  const float2 s = __fadd2_rn(v.hi, p), t = __fadd2_rn(s, neg2(v.hi));
  float2 rest = __fadd2_rn(__fadd2_rn(v.hi, neg2(__fadd2_rn(s, neg2(t)))), __fadd2_rn(p, neg2(t)));
  if (!EXACT) rest = __fadd2_rn(rest, fma2(a, a, neg2(p)));
  return {s, __fadd2_rn(v.lo, rest)};
}
__device__ __forceinline__ Two both(Pair v) {
  return plus(Two{v.hi.x, v.lo.x}, Two{v.hi.y, v.lo.y});
}
// (sum / n + eps)^-1/2 in two parts.  r = m^-1/2 (1 - e / 2 + ...) with e = m r^2 - 1.  Products whose
// rests are formed are rounded by their own (__fmul_rn): with one of them inside a multiply-add its rest
// would count twice.
__device__ __forceinline__ Two rstd_two(Two sum, float nf, float over_n, float eps) {
  const float q = __fmul_rn(sum.hi, over_n);  // within a place of the quotient: its rest is exact
  const Two m = plus(Two{q, (fmaf(-q, nf, sum.hi) + sum.lo) * over_n}, Two{eps, 0.f});
  const float r = rsqrtf(m.hi);
  const float rr = __fmul_rn(r, r), rr_low = fmaf(r, r, -rr);
  const float p = __fmul_rn(m.hi, rr);  // near 1
  const float e = (p - 1.f) + (fmaf(m.hi, rr, -p) + (m.hi * rr_low + m.lo * rr));
  const float low = r * e * fmaf(0.375f, e, -0.5f);
  return r > 0.f && r < 1e18f && m.hi < 1e38f ? fast_two(r, low) : Two{r, 0.f};
}
// s rstd w in two parts.
__device__ __forceinline__ Pair normed_two(float2 s, float2 w, Two rstd) {
  const float2 hi = make_float2(rstd.hi, rstd.hi), lo = make_float2(rstd.lo, rstd.lo);
  const float2 p = __fmul2_rn(s, hi), p_low = fma2(s, lo, fma2(s, hi, neg2(p)));
  const float2 y = __fmul2_rn(p, w);
  const float2 low = fma2(p_low, w, fma2(p, w, neg2(y)));
  const float2 sum = __fadd2_rn(y, low);
  return {sum, __fadd2_rn(low, neg2(__fadd2_rn(sum, neg2(y))))};
}
// The same of one column.
__device__ __forceinline__ Two normed_two(float s, float w, Two rstd) {
  const float p = __fmul_rn(s, rstd.hi), p_low = fmaf(s, rstd.lo, fmaf(s, rstd.hi, -p));
  const float y = __fmul_rn(p, w);
  return fast_two(y, fmaf(p_low, w, fmaf(p, w, -y)));
}
// To odd: a last place of 0 becomes 1, upwards or downwards to where the rest lies.
__device__ __forceinline__ float to_odd(float hi, float lo) {
  const uint32_t bits = __float_as_uint(hi), some = fabsf(lo) > 0.f ? 1u : 0u;
  const uint32_t less = ((bits ^ __float_as_uint(lo)) >> 31) & some;  // the rest points to 0
  return __uint_as_float((bits - less) | some);
}

// The sum over a row's team in two parts, in the order of team_sum.
template <typename TM>
__device__ __forceinline__ Two team_sum_two(Two v, Two (*part)[32], int turn) {
  constexpr int kLanes = TM::kWarp ? TM::TPR : 32;
  auto add = [&](int d) {
    const Two o{__shfl_xor_sync(0xffffffffu, v.hi, d), __shfl_xor_sync(0xffffffffu, v.lo, d)};
    v = plus(v, o);
  };
#pragma unroll
  for (int d = kLanes / 2; d > 0; d /= 2) add(d);
  if constexpr (!TM::kWarp) {
    Two* const p = part[turn & 1];
    const int lane = threadIdx.x % 32;
    if (lane == 0) p[threadIdx.x / 32] = v;
    __syncthreads();
    v = lane < static_cast<int>(blockDim.x) / 32 ? p[lane] : Two{0.f, 0.f};
#pragma unroll
    for (int d = TM::TPR / 64; d > 0; d /= 2) add(d);
    v.hi = __shfl_sync(0xffffffffu, v.hi, 0);
    v.lo = __shfl_sync(0xffffffffu, v.lo, 0);
  }
  return v;
}

// The next row's loads are on their way while a row is worked on.  Teams' rows are a multiple of
// eight apart, so that a team's rows start at the same place within a group of eight.
// OUT8: y is held in 8 bits.
template <typename T, typename TM, bool OUT8>
__global__ void __launch_bounds__(TM::kThreads) rms_fwd_kernel(const RmsCall q) {
  __shared__ std::conditional_t<OUT8, Two, float> part[2][32];
  const long long step = static_cast<long long>(gridDim.x) * TM::kTeams;
  long long row = static_cast<long long>(blockIdx.x) * TM::kTeams + TM::team();
  const At<TM> at(q.n, q.rows, static_cast<const T*>(q.x) + row * q.ldx);
  float w[TM::E];
  load_par<TM>(at, q.w, w);
  const float nf = static_cast<float>(q.n), over_n = 1.f / nf;  // n, at most 2^24, is exact
  Piece<T, TM> x_next, res_next;
  auto fetch = [&](long long row) {
    const bool ok = row < q.rows;
    x_next.load(at, static_cast<const T*>(q.x) + row * q.ldx, row, ok);
    if (q.residual)
      res_next.load(at, static_cast<const T*>(q.residual) + row * q.ldr, row, ok);
  };
  fetch(row);
  int turn = 0;
  // Warps stay together: `row` is the first of its CTA's teams' where the loop ends.
  for (; row - TM::team() < q.rows; row += step, ++turn) {
    const bool ok = row < q.rows;
    Piece<T, TM> x = x_next;
    if (q.residual) x.add(res_next);
    if (row - TM::team() + step < q.rows) fetch(row + step);
    float s[TM::E];
    x.get(at, s);
    if (q.s) store_row<TM>(at, static_cast<T*>(q.s) + row * q.lds, x, s, ok);
    if constexpr (OUT8) {
      constexpr bool EXACT = sizeof(T) == 2;
      Pair sum{make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int i = 0; i < TM::E; i += 2)
        sum = plus_square<EXACT>(sum, make_float2(s[i], i + 1 < TM::E ? s[i + 1] : 0.f));
      const Two rstd = rstd_two(team_sum_two<TM>(both(sum), part, turn), nf, over_n, q.eps);
      if (ok && q.rstd && threadIdx.x % TM::TPR == 0) q.rstd[row] = rstd.hi;
      if (q.s8.codes) store_held<TM>(at, q.s8, row, s, ok);
      float y[TM::E];
      if constexpr (TM::E == 1) {
        const Two v = normed_two(s[0], w[0], rstd);
        y[0] = v.hi;
        s[0] = to_odd(v.hi, v.lo);
      } else {
#pragma unroll
        for (int i = 0; i < TM::E; i += 2) {
          const Pair v = normed_two(make_float2(s[i], s[i + 1]), make_float2(w[i], w[i + 1]), rstd);
          y[i] = v.hi.x, y[i + 1] = v.hi.y;
          s[i] = to_odd(v.hi.x, v.lo.x);
          s[i + 1] = to_odd(v.hi.y, v.lo.y);
        }
      }
      if (q.y) store_row<TM>(at, static_cast<T*>(q.y) + row * q.ldy, y, ok);
      store_held<TM>(at, q.y8, row, s, ok);
    } else {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < TM::E; ++i) sum = fmaf(s[i], s[i], sum);
      const float rstd = rstd_of(team_sum<TM>(sum, part, turn), q.n, q.eps);
      if (ok && q.rstd && threadIdx.x % TM::TPR == 0) q.rstd[row] = rstd;
      if constexpr (TM::LY != kShifted) {
        if (q.s8.codes) store_held<TM>(at, q.s8, row, s, ok);
      }
      if (!q.y) continue;
#pragma unroll
      for (int i = 0; i < TM::E; ++i) s[i] = normed(s[i], w[i], rstd);
      store_row<TM>(at, static_cast<T*>(q.y) + row * q.ldy, s, ok);
    }
  }
}

// CTAs of the backward pass that an SM holds, which sets their registers and the number of partial
// sums of dw: 1024 threads of an SM in bf16 (16384 x 2048 54 us; 768 threads 59 us; 131072 x 512 94 and
// 102 us), 768 where a warp has a row or rows are shifted (262144 x 256 95 us; 1024 threads 105 us;
// 9001 x 1537 33 and 35 us), 512 in fp32, whose rows take twice the registers.
template <typename T, typename TM>
constexpr int bwd_per_sm() {
  const int threads = sizeof(T) == 4 || !TM::VEC ? 512 : TM::TPR == 32 || TM::LY == kShifted ? 768 : 1024;
  return threads > TM::kThreads ? threads / TM::kThreads : 1;
}

template <typename T, typename TM, bool KEPT>
__global__ void __launch_bounds__(TM::kThreads, bwd_per_sm<T, TM>()) rms_bwd_kernel(const RmsCall q, float* dw) {
  __shared__ float part[2][32];
  extern __shared__ float sums[];  // [teams][kCols], teams of a warp only
  grid_dep_launch_dependents();
  const int n = q.n;
  const long long step = static_cast<long long>(gridDim.x) * TM::kTeams;
  long long row = static_cast<long long>(blockIdx.x) * TM::kTeams + TM::team();
  const At<TM> at(n, q.rows, static_cast<const T*>(q.dy) + row * q.lddy);
  float w[TM::E], acc[TM::E];
  load_par<TM>(at, q.w, w);
#pragma unroll
  for (int i = 0; i < TM::E; ++i) acc[i] = 0.f;
  Piece<T, TM> dy_next, s_next;
  HeldPiece<TM> held_next;
  float rstd_next = 0.f;
  auto fetch = [&](long long row) {
    const bool ok = row < q.rows;
    dy_next.load(at, static_cast<const T*>(q.dy) + row * q.lddy, row, ok);
    if constexpr (KEPT) held_next.load(at, q.s8, row, ok);
    else s_next.load(at, static_cast<const T*>(q.x) + row * q.ldx, row, ok);
    rstd_next = ok ? q.rstd[row] : 0.f;
  };
  fetch(row);
  int turn = 0;
  for (; row - TM::team() < q.rows; row += step, ++turn) {
    const bool ok = row < q.rows;
    const float rstd = rstd_next;
    float s[TM::E], dy[TM::E];
    if constexpr (KEPT) held_next.get(s);
    else s_next.get(at, s);
    dy_next.get(at, dy);
    Piece<T, TM> ds;  // wanted last
    if (q.ds) ds.load(at, static_cast<const T*>(q.ds) + row * q.ldds, row, ok);
    if (row - TM::team() + step < q.rows) fetch(row + step);
    if (q.y) {
      float y[TM::E];
#pragma unroll
      for (int i = 0; i < TM::E; ++i) y[i] = normed(s[i], w[i], rstd);
      store_row<TM>(at, static_cast<T*>(q.y) + row * q.ldy, y, ok);
    }
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < TM::E; ++i) {
      s[i] *= rstd;  // hat
      acc[i] = fmaf(dy[i], s[i], acc[i]);
      dy[i] *= w[i];  // g
      dot = fmaf(dy[i], s[i], dot);
    }
    const float mean = team_sum<TM>(dot, part, turn) / static_cast<float>(n);
#pragma unroll
    for (int i = 0; i < TM::E; ++i) s[i] = rstd * fmaf(-mean, s[i], dy[i]);
    if (q.ds) {
      ds.get(at, dy);
#pragma unroll
      for (int i = 0; i < TM::E; ++i) s[i] += dy[i];
    }
    store_row<TM>(at, static_cast<T*>(q.dx) + row * q.lddx, s, ok);
  }
  float* const out = dw + static_cast<size_t>(blockIdx.x) * n;
  if constexpr (TM::kWarp) {
    float* const mine = sums + TM::team() * TM::kCols;
#pragma unroll
    for (int j = 0; j < TM::SLOTS; ++j)
#pragma unroll
      for (int i = 0; i < TM::W; ++i)
        if (at.in(j, i)) mine[at.col(j) + i] = acc[j * TM::W + i];
    __syncthreads();
    for (int c = threadIdx.x; c < n; c += TM::kThreads) {
      float v = sums[c];
#pragma unroll 8
      for (int i = 1; i < TM::kTeams; ++i) v += sums[i * TM::kCols + c];
      out[c] = v;
    }
  } else {
#pragma unroll
    for (int j = 0; j < TM::SLOTS; ++j)
#pragma unroll
      for (int i = 0; i < TM::W; ++i)
        if (at.in(j, i)) out[at.col(j) + i] = acc[j * TM::W + i];
  }
}

// ---- rows of more than kLongRow columns: a CTA a row, each column by the same thread in both
// passes ----

constexpr int kLongThreads = 512;
using LongTeam = Team<kLongThreads, 1, kScalar>;

template <typename T, bool OUT8>
__global__ void __launch_bounds__(kLongThreads) rms_long_fwd_kernel(const RmsCall q) {
  __shared__ std::conditional_t<OUT8, Two, float> part[2][32];
  const int n = q.n, whole = held_blocks(n) * kHeldBlock;
  int turn = 0;
  // Columns past n (to a whole block) hold 0, so that whole warps pack.
  auto hold = [&](const Held8& h, long long row, int c, float v) {
    uint32_t byte;
    const uint32_t r = held_pack1(v, byte);
    if (c < n) h.codes[row * n + c] = static_cast<uint8_t>(r);
    if (c % kHeldBlock == 0)
      h.scales[row * held_blocks(n) + c / kHeldBlock] = static_cast<uint8_t>(byte);
  };
  for (long long row = blockIdx.x; row < q.rows; row += gridDim.x, ++turn) {
    const T* const x = static_cast<const T*>(q.x) + row * q.ldx;
    const T* const res = q.residual ? static_cast<const T*>(q.residual) + row * q.ldr : nullptr;
    T* const so = q.s ? static_cast<T*>(q.s) + row * q.lds : nullptr;
    Two sum{0.f, 0.f};
    [[maybe_unused]] Pair squares{make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    for (int c = threadIdx.x; c < whole; c += kLongThreads) {
      float v = 0.f;
      if (c < n) {
        v = to_f32(x[c]);
        if (res) v = to_f32(from_f32<T>(v + to_f32(res[c])));
        if (so) so[c] = from_f32<T>(v);
      }
      if constexpr (OUT8) squares = plus_square<false>(squares, make_float2(v, 0.f));
      else sum.hi = fmaf(v, v, sum.hi);
      if (q.s8.codes) hold(q.s8, row, c, v);
    }
    Two rstd{0.f, 0.f};
    if constexpr (OUT8)
      rstd = rstd_two(team_sum_two<LongTeam>(both(squares), part, turn), static_cast<float>(n),
                      1.f / static_cast<float>(n), q.eps);
    else
      rstd.hi = rstd_of(team_sum<LongTeam>(sum.hi, part, turn), n, q.eps);
    if (q.rstd && threadIdx.x == 0) q.rstd[row] = rstd.hi;
    if (!q.y && !OUT8) continue;
    for (int c = threadIdx.x; c < whole; c += kLongThreads) {
      Two y{0.f, 0.f};
      if (c < n) {
        // s where it was written: x and the residual may have been in its place.
        float v = to_f32(so ? so[c] : x[c]);
        if (res && !so) v = to_f32(from_f32<T>(v + to_f32(res[c])));
        if constexpr (OUT8) y = normed_two(v, __ldg(q.w + c), rstd);
        else y.hi = normed(v, __ldg(q.w + c), rstd.hi);
        if (q.y) static_cast<T*>(q.y)[row * q.ldy + c] = from_f32<T>(y.hi);
      }
      if constexpr (OUT8) hold(q.y8, row, c, to_odd(y.hi, y.lo));
    }
  }
}

template <typename T, bool KEPT>
__device__ __forceinline__ float stream_at(const RmsCall& q, long long row, int c) {
  if constexpr (KEPT)
    return held_values2(q.s8.codes[row * q.n + c]).x *
           held_up(q.s8.scales[row * held_blocks(q.n) + c / kHeldBlock]);
  else
    return to_f32(static_cast<const T*>(q.x)[row * q.ldx + c]);
}

// dw of a tile of 256 columns over a run of rows, before dx may overwrite dy.
template <typename T, bool KEPT>
__global__ void __launch_bounds__(256) rms_long_dw_kernel(const RmsCall q, int per, float* dw) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= q.n) return;
  const long long lo = static_cast<long long>(blockIdx.y) * per;
  const long long hi = min(lo + per, static_cast<long long>(q.rows));
  float acc = 0.f;
#pragma unroll 4
  for (long long row = lo; row < hi; ++row)
    acc = fmaf(to_f32(static_cast<const T*>(q.dy)[row * q.lddy + c]),
               stream_at<T, KEPT>(q, row, c) * q.rstd[row], acc);
  dw[static_cast<size_t>(blockIdx.y) * q.n + c] = acc;
}

template <typename T, bool KEPT>
__global__ void __launch_bounds__(kLongThreads) rms_long_bwd_kernel(const RmsCall q) {
  __shared__ float part[2][32];
  const int n = q.n;
  int turn = 0;
  for (long long row = blockIdx.x; row < q.rows; row += gridDim.x, ++turn) {
    const T* const dy = static_cast<const T*>(q.dy) + row * q.lddy;
    const float rstd = q.rstd[row];
    float dot = 0.f;
    for (int c = threadIdx.x; c < n; c += kLongThreads)
      dot = fmaf(to_f32(dy[c]) * __ldg(q.w + c), stream_at<T, KEPT>(q, row, c) * rstd, dot);
    const float mean = team_sum<LongTeam>(dot, part, turn) / static_cast<float>(n);
    for (int c = threadIdx.x; c < n; c += kLongThreads) {
      const float s = stream_at<T, KEPT>(q, row, c), w = __ldg(q.w + c);
      float v = rstd * fmaf(-mean, s * rstd, to_f32(dy[c]) * w);
      if (q.ds) v += to_f32(static_cast<const T*>(q.ds)[row * q.ldds + c]);
      if (q.y) static_cast<T*>(q.y)[row * q.ldy + c] = from_f32<T>(normed(s, w, rstd));
      static_cast<T*>(q.dx)[row * q.lddx + c] = from_f32<T>(v);
    }
  }
}

// ---- launches ----

struct Rows {
  const void* p;
  long long ld;
};
// The layout that all rows there are allow; what is held in 8 bits has blocks that begin with the row.
Layout layout(const RmsCall& q) {
  const Rows r[] = {{q.x, q.ldx}, {q.residual, q.ldr}, {q.dy, q.lddy}, {q.ds, q.ldds},
                    {q.s, q.lds}, {q.y, q.ldy}, {q.dx, q.lddx}};
  const bool held = q.s8.codes || q.y8.codes;
  const uintptr_t e = q.bf16 ? 2 : 4;
  bool aligned = q.n % 8 == 0 && reinterpret_cast<uintptr_t>(q.s8.codes) % 8 == 0 &&
                 reinterpret_cast<uintptr_t>(q.y8.codes) % 8 == 0;
  bool alike = !held && q.n >= 8 && q.n <= kLongRow - 7;
  const Rows* first = nullptr;
  for (const Rows& a : r) {
    if (!a.p) continue;
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.p);
    aligned = aligned && at % (8 * e) == 0 && a.ld % 8 == 0;
    alike = alike && a.ld >= q.n;
    if (first)
      alike = alike && (at - reinterpret_cast<uintptr_t>(first->p)) % (8 * e) == 0 &&
              (a.ld - first->ld) % 8 == 0;
    else
      first = &a;
  }
  return aligned ? kAligned : alike ? kShifted : kScalar;
}

// f of the smallest team that covers n columns and of the threads of its CTA.
template <Layout LY, typename F>
cudaError_t with_vec_team(int n, F&& f) {
  const int span = LY == kShifted ? n + 7 : n, cta = (span + 255) / 256 * 32;
  if (span <= 32) return f(Team<4, 1, LY>{}, 256);
  if (span <= 64) return f(Team<8, 1, LY>{}, 256);
  if (span <= 128) return f(Team<16, 1, LY>{}, 256);
  if (span <= 256) return f(Team<32, 1, LY>{}, 256);
  if (span <= 512) return f(Team<64, 1, LY>{}, cta);
  if (span <= 1024) return f(Team<128, 1, LY>{}, cta);
  if (span <= 2048) return f(Team<256, 1, LY>{}, cta);
  if (span <= 4096) return f(Team<512, 1, LY>{}, cta);
  return f(Team<1024, 1, LY>{}, cta);
}
template <typename F>
cudaError_t with_team(int n, Layout ly, F&& f) {
  if (ly == kAligned) return with_vec_team<kAligned>(n, f);
  if (ly == kShifted) return with_vec_team<kShifted>(n, f);
  const int cta = (n + 255) / 256 * 32;
  if (n <= 32) return f(Team<32, 1, kScalar>{}, 256);
  if (n <= 64) return f(Team<32, 2, kScalar>{}, 256);
  if (n <= 128) return f(Team<32, 4, kScalar>{}, 256);
  if (n <= 256) return f(Team<32, 8, kScalar>{}, 256);
  if (n <= 512) return f(Team<64, 8, kScalar>{}, cta);
  if (n <= 1024) return f(Team<128, 8, kScalar>{}, cta);
  if (n <= 2048) return f(Team<256, 8, kScalar>{}, cta);
  if (n <= 4096) return f(Team<512, 8, kScalar>{}, cta);
  return f(Team<1024, 8, kScalar>{}, cta);
}

// CTAs for `rows`: a multiple of eight (152 is one) where a CTA has one team.
long long in_eights(long long ctas, int teams) {
  return teams % 8 == 0 ? ctas : (ctas - 1) / 8 * 8 + 8;
}
int fwd_ctas(int rows, int teams, int threads) {
  const long long need = in_eights((rows - 1) / teams + 1, teams), most = kSms * (2048 / threads);
  return static_cast<int>(need < most ? need : most);
}
// CTAs of the backward pass, and so rows of the partial sums of dw: a row of them costs 8 bytes a
// column to write and read, so a CTA takes four rows of a team at least once all SMs have one.
template <typename T, typename TM>
int bwd_ctas(int rows) {
  const long long most = kSms * bwd_per_sm<T, TM>();
  const long long need = in_eights((rows - 1) / TM::kTeams + 1, TM::kTeams);
  const long long want = need / 4 > kSms ? in_eights(need / 4, TM::kTeams) : kSms;
  return static_cast<int>(need < want ? need : want < most ? want : most);
}
// CTAs for long rows: one a row, up to what the GPU holds (64 rows x 65536 fp32 forward 771 us with eight
// rows a CTA, 122 us so).
int long_ctas(int rows) {
  const int most = kSms * (2048 / kLongThreads);
  return rows < most ? rows : most;
}
int long_splits(int rows) { return rows < 64 ? 1 : rows / 64 < 64 ? rows / 64 : 64; }
template <typename T>
int partials(int rows, int n, Layout ly) {
  if (n > kLongRow) return long_splits(rows);
  int p = 1;
  (void)with_team(n, ly, [&](auto tm, int) {
    p = rows == 1 ? 1 : bwd_ctas<T, decltype(tm)>(rows);
    return cudaSuccess;
  });
  return p;
}

template <typename T, bool OUT8>
cudaError_t fwd(const RmsCall& q, cudaStream_t s) {
  LaunchCfg c;
  c.stream = s;
  if (q.n > kLongRow) {
    c.grid = dim3(long_ctas(q.rows));
    c.block = dim3(kLongThreads);
    return launch(c, rms_long_fwd_kernel<T, OUT8>, q);
  }
  return with_team(q.n, layout(q), [&](auto tm, int threads) {
    using TM = decltype(tm);
    if constexpr (OUT8 && TM::LY == kShifted) return cudaErrorInvalidValue;  // never chosen
    else {
      c.grid = dim3(fwd_ctas(q.rows, TM::kTeams, threads));
      c.block = dim3(threads);
      return launch(c, rms_fwd_kernel<T, TM, OUT8>, q);
    }
  });
}

template <typename T, bool KEPT>
cudaError_t bwd(const RmsCall& q, float* dw, float* ws, cudaStream_t s) {
  LaunchCfg c;
  c.stream = s;
  const Layout ly = layout(q);
  const int P = partials<T>(q.rows, q.n, ly);
  float* const first = P == 1 ? dw : ws;
  cudaError_t e;
  if (q.n > kLongRow) {
    c.grid = dim3((q.n + 255) / 256, P);
    c.block = dim3(256);
    e = launch(c, rms_long_dw_kernel<T, KEPT>, q, (q.rows - 1) / P + 1, first);
    if (e != cudaSuccess) return e;
    c.grid = dim3(long_ctas(q.rows));
    c.block = dim3(kLongThreads);
    e = launch(c, rms_long_bwd_kernel<T, KEPT>, q);
  } else {
    e = with_team(q.n, ly, [&](auto tm, int threads) {
      using TM = decltype(tm);
      if constexpr (KEPT && TM::LY == kShifted) return cudaErrorInvalidValue;  // never chosen
      else {
        c.grid = dim3(P);
        c.block = dim3(threads);
        c.smem = TM::kWarp ? sizeof(float) * TM::kTeams * TM::kCols : 0;
        return launch(c, rms_bwd_kernel<T, TM, KEPT>, q, first);
      }
    });
  }
  if (e != cudaSuccess || P == 1) return e;
  return merge_launch(ws, P, q.n, dw, s, q.n <= kLongRow);
}

}  // namespace

size_t rms_ws_floats(int rows, int n) {
  // Which layout and type runs depends on the tensors, which the sizing call does not have.
  int p = 1;
  for (const Layout ly : {kScalar, kAligned, kShifted}) {
    if (ly == kShifted && n > kLongRow - 7) continue;
    const int a = partials<float>(rows, n, ly), b = partials<__nv_bfloat16>(rows, n, ly);
    p = a > p ? a : p;
    p = b > p ? b : p;
  }
  return p == 1 ? 0 : static_cast<size_t>(p) * n;
}
cudaError_t rms_fwd_launch(const RmsCall& q, cudaStream_t s) {
  if (q.y8.codes) return q.bf16 ? fwd<__nv_bfloat16, true>(q, s) : fwd<float, true>(q, s);
  return q.bf16 ? fwd<__nv_bfloat16, false>(q, s) : fwd<float, false>(q, s);
}
cudaError_t rms_bwd_launch(const RmsCall& q, float* dw, float* ws, cudaStream_t s) {
  if (q.x)
    return q.bf16 ? bwd<__nv_bfloat16, false>(q, dw, ws, s) : bwd<float, false>(q, dw, ws, s);
  return q.bf16 ? bwd<__nv_bfloat16, true>(q, dw, ws, s) : bwd<float, true>(q, dw, ws, s);
}

}  // namespace cfc
