// cfc_norm.cu -- layer norm over rows, forward and backward, alone or behind dropout and a
// residual sum, and dropout alone.
//
//   forward   s = residual + keep * x * scale        (dropout; s = x without it)
//             mean = sum s / n, var = sum (s - mean)^2 / n, rstd = (var + eps)^-1/2
//             y = (s - mean) rstd w + b
//   backward  g = dy w, hat = (s - mean) rstd
//             d = rstd (g - sum g / n - hat sum(g hat) / n)       (+ the stream's gradient ds)
//             dw = sum_rows dy hat, db = sum_rows dy
//             dres = d, dx = keep * d * scale
//
// Every pass is bound by memory: each element is read once and written once, so a row stays in
// registers between its sums and its results (two sums: the mean, then the squares of what is
// left, so that a large mean costs no precision), and the next row's loads are on their way
// meanwhile.  A row belongs to a team of lanes, eight columns to a lane and piece: 4 to 32 lanes
// of one warp up to 256 columns, 2 or 4 warps up to 1024, a whole CTA of just enough warps up to
// 8192, two pieces a lane (with the rows on their way in shared memory where they would take too many
// registers, see Ring).  Longer rows are read again for each sum (they stay in L2).
//
// Lanes load and store eight columns at once.  Where rows start anywhere (an odd width), the
// lanes' groups of eight follow the memory's alignment instead of the row's start, and the row's
// two ends are done element by element; a team's rows are a multiple of eight apart, so their
// starts are aligned alike and its parameters and sums stay in registers.  Tensors that are
// aligned differently from one another are done element by element throughout.
//
// The parameter gradients stay in each lane's registers over all rows of its team, are added over
// the CTA's teams in shared memory and over the CTAs by reduce_axis0: no atomics, and an order
// that depends on the sizes and the alignment alone.  The dropout mask is never stored: both
// passes draw it again from the counter-based generator, whose counter is the element's place.
//
// Measured on GB300 (copy rate 6.69 TB/s): 262144 x 256 fp32 forward 84 us (6.4 TB/s), backward 125 us
// (6.4 TB/s); the same rows in bf16 with dropout and residual 98 us (5.5 TB/s; a row's generator calls
// are a third of its instructions) and 127 us (5.3 TB/s); 10529 x 3528 fp32 56 and 88 us (5.3 and
// 5.0 TB/s), bf16 31 and 53 us (4.8 and 4.2 TB/s); 6007 x 2501 bf16, rows of every alignment, 20 and
// 32 us (3.0 and 2.8 TB/s).  What bounds wide bf16 rows are instructions and shared memory: 21.5 and
// 29.4 instructions an element at 2501 columns (an aligned fp32 row of 256 takes 15), issued at 2.6 and
// 2.4 a clock of 4, the shared-memory pipe busy to 68% and 44%: w and b are read from it again, in
// fp32, for every row.  The rows' ends, element by element, and a barrier a row come on top.
// Dropout alone with the residual, 262144 x 256: fp32 127 us (6.3 TB/s), bf16 68 us (5.9 TB/s); its
// backward pass 90 us (6.0 TB/s) and 60 us (4.5 TB/s); 24028 x 2501 bf16 121 and 111 us (3.0 and
// 2.2 TB/s).
#include "cfc_kernels.h"
#include "cfc_launch.cuh"
#include "cfc_trunk.cuh"
#include "cfc_trunk_kernels.h"

#include <type_traits>

namespace cfc {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxWarps = 16;
constexpr int kWholeCta = 99;

// How a team of lanes covers a row.  WPR 0: L lanes of a warp (32 / L rows per warp); WPR 1, 2, 4:
// that many warps of a 256-thread CTA; kWholeCta: all warps of the CTA (as many as the row needs).
// I pieces of 8 columns a lane; MAXW: most warps of a whole CTA.
template <int WPR_, int L_, int I_, int MAXW = kThreads / 32>
struct Team {
  static constexpr int WPR = WPR_, L = L_, I = I_;
  static constexpr bool kWhole = WPR == kWholeCta;
  static constexpr int kLanes = WPR > 0 ? 32 : L;  // lanes of one warp's tile
  static constexpr int kTeams = kWhole ? 1 : WPR > 0 ? kThreads / 32 / WPR : kThreads / L;
  static constexpr int kMaxThreads = 32 * MAXW;
  // Columns of a piece.
  static __device__ __forceinline__ int cols() {
    return kWhole ? 8 * static_cast<int>(blockDim.x) : 8 * kLanes * (WPR > 0 ? WPR : 1);
  }
};

// How rows are laid out.  kScalar: anyhow; a lane's columns are kLanes apart, so that a warp's
// element loads are consecutive.  kAligned: every row starts on a group of eight.  kShifted:
// every tensor's row r starts at the same place within a group of eight.
enum Layout { kScalar, kAligned, kShifted };

// A lane's place: which team of the CTA, and its columns.
template <typename TM, Layout LY>
struct Lane {
  int team, lane, base;  // base: first column of this warp's tile in a piece
  int shift = 0;         // kShifted: the row's start within its group of eight
  __device__ __forceinline__ Lane() {
    const int w = threadIdx.x / 32;
    if constexpr (TM::kWhole) {
      team = 0;
      lane = threadIdx.x % 32;
      base = w * 256;
    } else if constexpr (TM::WPR > 0) {
      team = w / TM::WPR;
      lane = threadIdx.x % 32;
      base = (w % TM::WPR) * 256;
    } else {
      team = threadIdx.x / TM::L;
      lane = threadIdx.x % TM::L;
      base = 0;
    }
  }
  template <typename T>
  __device__ __forceinline__ void set_row(const T* row) {
    if constexpr (LY == kShifted)
      shift = static_cast<int>((reinterpret_cast<uintptr_t>(row) / sizeof(T)) % 8);
  }
  __device__ __forceinline__ int col(int piece, int j) const {
    const int c = piece * TM::cols() + base;
    return LY == kScalar ? c + j * TM::kLanes + lane : c + lane * 8 + j - shift;
  }
  __device__ __forceinline__ bool in(int piece, int j, int n) const {
    return static_cast<unsigned>(col(piece, j)) < static_cast<unsigned>(n);
  }
  // All eight columns of the lane are in the row, and aligned.
  __device__ __forceinline__ bool whole(int piece, int n) const {
    if constexpr (LY == kScalar) return false;
    if constexpr (LY == kAligned) return col(piece, 0) < n;
    return col(piece, 0) >= 0 && col(piece, 7) < n;
  }
  // Whether a lane's eight columns of row `row` of a tensor of `rows` rows are read at once.  At the row's ends a group reaches up to seven elements into the rows before and
  // after, which is the tensor's own memory where it has that many: `near` rows before and after
  // the row (7 columns' worth).  Groups at the tensor's ends (and those of rows that lie on one
  // another, ld < n) are read element by element.
  // `first`: the group's first column.
  __device__ __forceinline__ static bool vec(long long ld, long long row, int rows, int first, int n) {
    if constexpr (LY == kScalar) return false;
    if constexpr (LY == kAligned) return first < n;
    const int last = first + 7, near = n >= 7 ? 1 : 7;
    return (first >= 0 && last < n) || (ld >= n && last >= 0 && first < n &&
                                        (first >= 0 || row >= near) && (last < n || row < rows - near));
  }
  // The lane's eight columns as they are stored; clean() drops what is not the row's.
  template <typename T>
  __device__ __forceinline__ void load(const T* p, long long ld, long long row, int rows, int piece,
                                       int n, Raw8<T>& r) const {
    const T* at = p + row * ld;
    if (vec(ld, row, rows, col(piece, 0), n)) {
      r.load(at + col(piece, 0));
      return;
    }
    r.clear();
    if constexpr (LY != kAligned) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (in(piece, j, n)) r.set(j, at[col(piece, j)]);
    }
  }
  template <typename T>
  __device__ __forceinline__ void clean(const Raw8<T>& r, int piece, int n, float (&v)[8]) const {
    r.get(v);
    if constexpr (LY == kShifted)
      if (!whole(piece, n)) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (!in(piece, j, n)) v[j] = 0.f;
      }
  }
  // The same of the parameters (in no particular alignment to the rows).  `buf`: 256 floats of the
  // warp's own; shifted lanes read their eight columns from there, so that the loads from memory
  // are consecutive.  Every lane of the warp takes part.
  __device__ __forceinline__ void params(const float* p, int piece, int n, float* buf,
                                         float (&v)[8]) const {
    if constexpr (LY == kAligned) {
      Raw8<float> r;
      load(p, 0, 0, 1, piece, n, r);
      r.get(v);
    } else if constexpr (LY == kShifted && TM::WPR > 0) {
      const int c = piece * TM::cols() + base - shift;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int at = c + j * 32 + lane;
        buf[j * 32 + lane] = static_cast<unsigned>(at) < static_cast<unsigned>(n) ? p[at] : 0.f;
      }
      __syncwarp();
      const float4 lo = *reinterpret_cast<const float4*>(buf + lane * 8);
      const float4 hi = *reinterpret_cast<const float4*>(buf + lane * 8 + 4);
      v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
      v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
      __syncwarp();
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = in(piece, j, n) ? p[col(piece, j)] : 0.f;
    }
  }
  // The lane's eight columns into a row of fp32 sums (of any alignment), likewise.
  __device__ __forceinline__ void put_sums(float* p, int piece, int n, float* buf,
                                           const float (&v)[8]) const {
    if constexpr (LY != kScalar) {
      *reinterpret_cast<float4*>(buf + lane * 8) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(buf + lane * 8 + 4) = make_float4(v[4], v[5], v[6], v[7]);
      __syncwarp();
      const int c = piece * TM::cols() + base - shift;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int at = c + j * 32 + lane;
        if (static_cast<unsigned>(at) < static_cast<unsigned>(n)) p[at] = buf[j * 32 + lane];
      }
      __syncwarp();
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (in(piece, j, n)) p[col(piece, j)] = v[j];
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(T* row, int piece, int n, const float (&v)[8]) const {
    if (whole(piece, n)) {
      store8(row + col(piece, 0), v);
      return;
    }
    if constexpr (LY != kAligned) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (in(piece, j, n)) row[col(piece, j)] = from_f32<T>(v[j]);
    }
  }
  // Which of the lane's eight columns are kept.  The generator serves eight consecutive columns
  // from a multiple of eight; where a lane's columns are others, each lane draws for its eight of
  // those and the bits change hands inside the warp's tile.  Every lane of the warp takes part.
  __device__ __forceinline__ void keep(const DropKey& key, uint32_t row, int piece, uint32_t cut,
                                       bool (&k)[8]) const {
    const int group = (piece * TM::cols() + base) / 8 + lane;
    keep8(key, row, static_cast<uint32_t>(group), cut, k);
    if constexpr (LY == kAligned) return;
    uint32_t own = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) own |= k[j] ? 1u << j : 0u;
    if constexpr (LY == kScalar) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int at = j * TM::kLanes + lane;
        k[j] = __shfl_sync(0xffffffffu, own, at >> 3, TM::kLanes) >> (at & 7) & 1u;
      }
    } else {
      // Columns 8 group - shift ..: the last `shift` bits of the group before, then the first of
      // this one.
      uint32_t before = __shfl_up_sync(0xffffffffu, own, 1, TM::kLanes);
      if (lane == 0 && group > 0) {
        bool p[8];
        keep8(key, row, static_cast<uint32_t>(group - 1), cut, p);
        before = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) before |= p[j] ? 1u << j : 0u;
      }
      const uint32_t both = (before & 0xffu) | own << 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) k[j] = both >> (8 - shift + j) & 1u;
    }
  }
};

// Sums of N values over the team.  Teams of several warps go through shared memory: `slot` holds
// two sets of a value per warp, used in turn, so one barrier a sum is enough.  (A whole CTA's set
// is added by every warp for itself, a slot a lane; slots without a warp hold zero.)
template <int N>
struct Slots {
  float v[2][N][kMaxWarps];
};
template <typename TM, int N>
__device__ __forceinline__ void clear_slots(Slots<N>& s) {
  if constexpr (TM::kWhole) {
    for (int i = threadIdx.x; i < 2 * N * kMaxWarps; i += blockDim.x) (&s.v[0][0][0])[i] = 0.f;
    __syncthreads();
  }
}
__device__ __forceinline__ void half_warp_sum(float& v) {
#pragma unroll
  for (int d = kMaxWarps / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
}
__device__ __forceinline__ void warp_sum(float& v) {
  v += __shfl_xor_sync(0xffffffffu, v, 16);
  half_warp_sum(v);
}
template <typename TM, int N, int M>
__device__ __forceinline__ void team_sum(float (&v)[N], Slots<M>& slot, int turn, int team) {
  constexpr int kSpan = TM::WPR > 0 ? 32 : TM::L;
#pragma unroll
  for (int d = kSpan / 2; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
  if constexpr (TM::WPR > 1) {
    const int w = threadIdx.x / 32;
    if (threadIdx.x % 32 == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) slot.v[turn][i][w] = v[i];
    }
    if constexpr (TM::kWhole) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = slot.v[turn][i][threadIdx.x % kMaxWarps];
#pragma unroll
      for (int i = 0; i < N; ++i) half_warp_sum(v[i]);
    } else {
      asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(TM::WPR * 32) : "memory");
#pragma unroll
      for (int i = 0; i < N; ++i) {
        v[i] = slot.v[turn][i][team * TM::WPR];
#pragma unroll
        for (int j = 1; j < TM::WPR; ++j) v[i] += slot.v[turn][i][team * TM::WPR + j];
      }
    }
  }
}

// The rows on their way: NT tensors, two rows of each in shared memory, for whole-CTA teams whose
// groups of eight are aligned.  A warp copies its own groups (32 consecutive pieces of 16
// bytes at a time) and reads them itself, so only its own copies are waited for, and the copies need
// no registers meanwhile.
// Shared memory: [row of the ring][tensor][piece][16 bytes of eight columns][thread], then the
// parameters, likewise.
template <typename T, typename TM, Layout LY, int NT>
struct Ring {
  [[maybe_unused]] static constexpr int kDepth = 2;
  static constexpr int kQuads = sizeof(T) / 2;  // 16 bytes each, of eight columns
  static constexpr int kRow = NT * TM::I * kQuads;
  [[maybe_unused]] static constexpr int kParam = TM::I * 2;      // a parameter's, in fp32
  uint4* mine;
  int at = 0;
  __device__ __forceinline__ explicit Ring(uint4* smem) : mine(smem + threadIdx.x) {}
  __device__ __forceinline__ uint4* place(int slot, int t, int piece) const {
    return mine + (slot * kRow + (t * TM::I + piece) * kQuads) * static_cast<int>(blockDim.x);
  }
  __device__ __forceinline__ uint4* param(int which, int piece) const {
    return mine + (kDepth * kRow + which * kParam + piece * 2) * static_cast<int>(blockDim.x);
  }
  __device__ __forceinline__ void put_param(int which, int piece, const float (&v)[8]) const {
    float4* const to = reinterpret_cast<float4*>(param(which, piece));
    to[0] = make_float4(v[0], v[1], v[2], v[3]);
    to[blockDim.x] = make_float4(v[4], v[5], v[6], v[7]);
  }
  __device__ __forceinline__ void get_param(int which, int piece, float (&v)[8]) const {
    const float4* const from = reinterpret_cast<const float4*>(param(which, piece));
    const float4 lo = from[0], hi = from[blockDim.x];
    v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
    v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
  }
  // A group with none of the row's columns is never fetched, and stays zero.
  static __device__ __forceinline__ bool outside(const Lane<TM, LY>& ln, int piece, int n) {
    return ln.col(piece, 7) < 0 || ln.col(piece, 0) >= n;
  }
  __device__ __forceinline__ void clear(const Lane<TM, LY>& ln, int n) const {
    Raw8<T> zero;
    zero.clear();
    for (int slot = 0; slot < kDepth; ++slot)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < TM::I; ++i)
          if (outside(ln, i, n)) zero.put(place(slot, t, i), static_cast<int>(blockDim.x));
  }
  __device__ __forceinline__ void fetch(const Lane<TM, LY>& ln, int slot, int t, const T* p, long long ld,
                                        long long row, int rows, int n) const {
    if constexpr (kQuads > 1) __syncwarp();  // all that its lanes have read
#pragma unroll
    for (int i = 0; i < TM::I; ++i) {
      uint4* const to = place(slot, t, i);
#pragma unroll
      for (int q = 0; q < kQuads; ++q) {
        const int chunk = q * 32 + ln.lane, of = chunk / kQuads, part = chunk % kQuads;
        const int first = ln.col(i, 0) + (of - ln.lane) * 8;
        if (ln.vec(ld, row, rows, first, n))
          cp_async_16(to + (of - ln.lane) + part * static_cast<int>(blockDim.x),
                      p + row * ld + first + part * (16 / static_cast<int>(sizeof(T))));
      }
      if (LY == kShifted && !outside(ln, i, n) && !ln.vec(ld, row, rows, ln.col(i, 0), n)) {
        Raw8<T> r;
        ln.load(p, ld, row, rows, i, n, r);
        r.put(to, static_cast<int>(blockDim.x));
      }
    }
  }
  __device__ __forceinline__ void take(int t, int piece, Raw8<T>& r) const {
    r.pick(place(at, t, piece), static_cast<int>(blockDim.x));
  }
  // The oldest row has arrived (this warp's groups of it).
  __device__ __forceinline__ void wait() const {
    cp_async_wait<kDepth - 1>();
    if constexpr (kQuads > 1) __syncwarp();
  }
  __device__ __forceinline__ void next() { at ^= 1; }
};

// Where the rows on their way take too many registers: the ring.  bf16: all but the backward pass of
// aligned rows without dropout; fp32, whose copies of 16 bytes are twice as many: rows with dropout
// that are shifted, or above 4096 columns in the backward pass.  Measured (us, with the ring and
// without):
//   bf16          10529 x 3528 forward 33, 39; backward 67, 54       3000 x 8185 27 + 45, 29 + 54
//     dropout     10529 x 3528 66 + 83, 75 + 103                     6007 x 2501 46 + 59, 49 + 79
//   fp32          10529 x 3528 86 + 108, 56 + 88                     3000 x 8185 57 + 80, 42 + 74
//     dropout     10529 x 3528 130 + 179, 94 + 147                   6007 x 2501 58 + 83, 79 + 114
template <typename T, typename TM, Layout LY, bool DROP>
__host__ __device__ constexpr bool fwd_ring() {
  return TM::kWhole && LY != kScalar && (sizeof(T) == 2 || (DROP && LY == kShifted));
}
template <typename T, typename TM, Layout LY, bool DROP>
__host__ __device__ constexpr bool bwd_ring() {
  if (!TM::kWhole || LY == kScalar) return false;
  if (sizeof(T) == 2) return DROP || LY == kShifted;
  return DROP && (LY == kShifted || TM::kMaxThreads > kThreads);
}
// CTAs of the most threads that an SM's registers must hold (0: as the compiler finds).  Forward,
// 256 threads: four (64 registers; 262144 x 256 bf16 with dropout 99 us, 105 us with the three that
// the registers taken freely allow, 125 us with five), but two of shifted rows with dropout, which
// spill at 64 (28467 x 319 bf16 48 us, 56 us with three); whole CTAs: 128 registers, 64 with a ring
// that holds the rows without dropout.  Backward: shifted rows three, with dropout two, as the grid
// has (28467 x 319: bf16 37 us, 50 us freely; fp32 with dropout 73 and 93 us); whole CTAs with shifted
// rows or a ring 128 registers (6007 x 2501 fp32 49 us, 68 us freely); aligned rows with the loads in
// registers as the compiler finds (262144 x 256 fp32 125 us; asked for one CTA, it spends the
// registers on an order of loads that takes 158 us).  Where a figure is bf16's alone, fp32 has not
// been timed apart; it spills there: 36 to 48 bytes a thread forwards (aligned rows with dropout), 40
// to 104 backwards (shifted rows without).
template <typename T, typename TM, Layout LY, bool DROP>
__host__ __device__ constexpr int fwd_ctas() {
  if (!TM::kWhole) return LY == kShifted && DROP ? 2 : 4;
  return (fwd_ring<T, TM, LY, DROP>() && !DROP ? 1024 : 512) / TM::kMaxThreads;
}
template <typename T, typename TM, Layout LY, bool DROP>
__host__ __device__ constexpr int bwd_ctas() {
  if (!TM::kWhole) return LY != kShifted ? 0 : DROP ? 2 : 3;
  return LY != kShifted && !bwd_ring<T, TM, LY, DROP>() ? 0 : 512 / TM::kMaxThreads;
}

// Arithmetic goes in pairs of columns, one instruction for two (6007 x 2501 bf16 50.5 us, 51.6 us one
// by one; 28467 x 319 bf16 58 and 61 us).
__device__ __forceinline__ float2 pair(const float (&v)[8], int j) { return make_float2(v[2 * j], v[2 * j + 1]); }
__device__ __forceinline__ void set_pair(float (&v)[8], int j, float2 p) { v[2 * j] = p.x; v[2 * j + 1] = p.y; }
__device__ __forceinline__ float2 twice(float v) { return make_float2(v, v); }

struct NormArgs {
  const void *x, *residual, *dy, *ds;
  long long ldx, ldr, lddy, ldds;
  const float *w, *b;
  const unsigned long long* rng;
  uint32_t cut;
  float scale, eps;
  int rows, n;
  void *s, *y, *dx, *dres;
  long long lds, ldy, lddx, lddr;
  float2* stats;
  float *pw, *pb;  // [gridDim.x][n] sums of dw and db
};

// The rows of a team: the first, the distance to the next, and how many turns every team takes
// (teams of one warp share its shuffles, so they take the same number).
struct Turns {
  long long first, step;
  int count;
};
template <typename TM>
__device__ __forceinline__ Turns turns_of(int rows, int team) {
  const long long step = static_cast<long long>(gridDim.x) * TM::kTeams;
  return {static_cast<long long>(blockIdx.x) * TM::kTeams + team, step,
          static_cast<int>((rows + step - 1) / step)};
}

template <typename T, typename TM, Layout LY, bool DROP>
__global__ void __launch_bounds__(TM::kMaxThreads, fwd_ctas<T, TM, LY, DROP>())
    norm_fwd_kernel(const NormArgs a) {
  __shared__ Slots<2> slot;
  extern __shared__ uint4 smem[];
  using Rg = Ring<T, TM, LY, DROP ? 2 : 1>;
  constexpr bool kRing = fwd_ring<T, TM, LY, DROP>();
  constexpr int kBufs = !kRing && (LY == kShifted || (TM::kWhole && LY != kScalar)) ? TM::kMaxThreads / 32 : 1;
  __shared__ __align__(16) float bufs[kBufs][256];
  clear_slots<TM>(slot);
  // (A ring's first kilobytes, before and after its use.)
  float* const buf = kRing ? reinterpret_cast<float*>(smem) + threadIdx.x / 32 * 256
                           : bufs[kBufs > 1 ? threadIdx.x / 32 : 0];
  Rg ring(smem);
  Lane<TM, LY> at;
  const int n = a.n;
  const float inv_n = 1.f / static_cast<float>(n);
  DropKey key{};
  if constexpr (DROP) key = drop_key(a.rng);
  const Turns tn = turns_of<TM>(a.rows, at.team);
  const T* const xp = static_cast<const T*>(a.x);
  const T* const rp = DROP ? static_cast<const T*>(a.residual) : nullptr;
  Raw8<T> nx[TM::I], nr[TM::I];
  auto fetch = [&](long long row) {
#pragma unroll
    for (int i = 0; i < TM::I; ++i) {
      at.load(xp, a.ldx, row, a.rows, i, n, nx[i]);
      if (DROP && rp) at.load(rp, a.ldr, row, a.rows, i, n, nr[i]);
    }
  };
  auto fetch_ring = [&](long long row, int place) {
    if (row < a.rows) {
      ring.fetch(at, place, 0, xp, a.ldx, row, a.rows, n);
      if (DROP && rp) ring.fetch(at, place, DROP ? 1 : 0, rp, a.ldr, row, a.rows, n);
    }
    cp_async_commit();
  };
  // Aligned parameters are two loads from the first-level cache a row; others stay in registers.
  float w[TM::I][8], b[TM::I][8];
  at.set_row(xp + (tn.first < a.rows ? tn.first : 0) * a.ldx);
  auto params = [&]() {
#pragma unroll
    for (int i = 0; i < TM::I; ++i) {
      at.params(a.w, i, n, buf, w[i]);
      at.params(a.b, i, n, buf, b[i]);
    }
  };
  // Columns of a whole CTA's warp: this one, and (lane % kMaxWarps).
  auto columns = [&](int warp) {
    int sum = 0;
#pragma unroll
    for (int i = 0; i < TM::I; ++i) {
      const int lo = i * TM::cols() + warp * 256 - at.shift;
      sum += max(0, min(n, lo + 256) - max(0, lo));
    }
    return warp < static_cast<int>(blockDim.x) / 32 ? static_cast<float>(sum) : 0.f;
  };
  const float own_n = columns(threadIdx.x / 32), other_n = columns(at.lane % kMaxWarps);
  const float own_inv = own_n > 0.f ? 1.f / own_n : 0.f, other_inv = other_n > 0.f ? 1.f / other_n : 0.f;
  // v less `from`, and the sum of its squares, of the row's columns alone.
  auto spread = [&](float (&v)[TM::I][8], float from, float& sq) {
#pragma unroll
    for (int i = 0; i < TM::I; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) set_pair(v[i], j, __fadd2_rn(pair(v[i], j), twice(-from)));
      if (at.whole(i, n)) {
        float2 two = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < 4; ++j) two = fma2(pair(v[i], j), pair(v[i], j), two);
        sq += two.x + two.y;
      } else if (LY != kAligned) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (at.in(i, j, n)) sq = fmaf(v[i][j], v[i][j], sq);
      }
    }
  };
  if constexpr (kRing) {
#pragma unroll
    for (int i = 0; i < TM::I; ++i) {
      at.params(a.w, i, n, buf, w[i]);
      ring.put_param(0, i, w[i]);
      at.params(a.b, i, n, buf, b[i]);
      ring.put_param(1, i, b[i]);
    }
    __syncthreads();
    ring.clear(at, n);
    for (int i = 0; i < Rg::kDepth; ++i) fetch_ring(tn.first + i * tn.step, i);
  } else {
    if constexpr (LY != kAligned) params();
    if (tn.first < a.rows) fetch(tn.first);
  }
  for (int turn = 0; turn < tn.count; ++turn) {
    const long long row = tn.first + turn * tn.step;
    const bool live = row < a.rows;
    if (TM::WPR > 0 && !live) return;  // the whole team
    float v[TM::I][8];
    if constexpr (kRing) ring.wait();
#pragma unroll
    for (int i = 0; i < TM::I; ++i) {
      if constexpr (kRing) ring.take(0, i, nx[i]);
      at.clean(nx[i], i, n, v[i]);
    }
    if constexpr (DROP) {
      float res[TM::I][8];
      if (rp) {
#pragma unroll
        for (int i = 0; i < TM::I; ++i) {
          if constexpr (kRing) ring.take(1, i, nr[i]);
          at.clean(nr[i], i, n, res[i]);
        }
      }
      if (!kRing && row + tn.step < a.rows) fetch(row + tn.step);
#pragma unroll
      for (int i = 0; i < TM::I; ++i) {
        bool keep[8];
        at.keep(key, static_cast<uint32_t>(row), i, a.cut, keep);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          // Product and sum rounded apart: the same values as dropout followed by the sum.
          float d = keep[j] ? __fmul_rn(v[i][j], a.scale) : 0.f;
          if (rp) d = __fadd_rn(res[i][j], d);
          // The norm reads the stream as it is stored, so that the backward pass, which reads
          // the stored stream, differentiates what the forward pass computed.
          v[i][j] = to_f32(from_f32<T>(d));
        }
        if (live) at.store(static_cast<T*>(a.s) + row * a.lds, i, n, v[i]);
      }
    } else {
      if (!kRing && row + tn.step < a.rows) fetch(row + tn.step);
    }
    float2 two = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < TM::I; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) two = __fadd2_rn(two, pair(v[i], j));
    float sum = two.x + two.y;
    if constexpr (LY == kAligned && !kRing) params();
    float mean, var, left = 0.f;  // left: what is still to be added to v
    if constexpr (TM::kWhole) {
      // Each warp takes its own mean and the squares of what is left; these are put together behind
      // one barrier: sum of squares = sum over warps of (its own + its columns (its mean - mean)^2).
      warp_sum(sum);
      if constexpr (kRing) {  // the warp has read this row
        fetch_ring(row + Rg::kDepth * tn.step, ring.at);
        ring.next();
      }
      const float own = sum * own_inv;
      float sq = 0.f;
      spread(v, own, sq);
      warp_sum(sq);
      const int w = threadIdx.x / 32, side = turn & 1;
      if (at.lane == 0) {
        slot.v[side][0][w] = sum;
        slot.v[side][1][w] = sq;
      }
      __syncthreads();
      const float their = slot.v[side][0][at.lane % kMaxWarps];
      mean = their;
      half_warp_sum(mean);
      mean *= inv_n;
      const float off = their * other_inv - mean;
      var = fmaf(other_n * off, off, slot.v[side][1][at.lane % kMaxWarps]);
      half_warp_sum(var);
      var *= inv_n;
      left = own - mean;
    } else {
      float one[1] = {sum};
      team_sum<TM>(one, slot, 0, at.team);
      mean = one[0] * inv_n;
      one[0] = 0.f;
      spread(v, mean, one[0]);
      team_sum<TM>(one, slot, 1, at.team);
      var = one[0] * inv_n;
    }
    const float rstd = rsqrtf(var + a.eps);
    if (!live) continue;
    T* y = static_cast<T*>(a.y) + row * a.ldy;
#pragma unroll
    for (int i = 0; i < TM::I; ++i) {
      if constexpr (kRing) {
        ring.get_param(0, i, w[i]);
        ring.get_param(1, i, b[i]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 hat = TM::kWhole ? fma2(pair(v[i], j), twice(rstd), twice(left * rstd))
                                      : __fmul2_rn(pair(v[i], j), twice(rstd));
        set_pair(v[i], j, fma2(hat, pair(w[i], j), pair(b[i], j)));
      }
      at.store(y, i, n, v[i]);
    }
    if (at.base == 0 && at.lane == 0) a.stats[row] = make_float2(mean, rstd);
  }
}

template <typename T, typename TM, Layout LY, bool DROP>
__global__ void __launch_bounds__(TM::kMaxThreads, bwd_ctas<T, TM, LY, DROP>())
    norm_bwd_kernel(const NormArgs a) {
  __shared__ Slots<2> slot;
  __shared__ float part[TM::kTeams > 1 ? 2 : 1][TM::kTeams > 1 ? kThreads / 32 : 1][256];
  __shared__ int shifts[TM::kTeams];
  extern __shared__ uint4 smem[];
  using Rg = Ring<T, TM, LY, DROP ? 3 : 2>;
  constexpr bool kRing = bwd_ring<T, TM, LY, DROP>();
  constexpr int kBufs = !kRing && (LY == kShifted || (TM::kWhole && LY != kScalar)) ? TM::kMaxThreads / 32 : 1;
  __shared__ __align__(16) float bufs[kBufs][256];
  grid_dep_launch_dependents();
  clear_slots<TM>(slot);
  float* const buf = kRing ? reinterpret_cast<float*>(smem) + threadIdx.x / 32 * 256
                           : bufs[kBufs > 1 ? threadIdx.x / 32 : 0];
  Rg ring(smem);
  Lane<TM, LY> at;
  const int n = a.n;
  const float inv_n = 1.f / static_cast<float>(n);
  DropKey key{};
  if constexpr (DROP) key = drop_key(a.rng);
  const Turns tn = turns_of<TM>(a.rows, at.team);
  const T* const xp = static_cast<const T*>(a.x);
  const T* const gp = static_cast<const T*>(a.dy);
  const T* const sp = DROP ? static_cast<const T*>(a.ds) : nullptr;
  Raw8<T> nx[TM::I], ng[TM::I], ns[TM::I];
  float2 nst = make_float2(0.f, 0.f);
  auto fetch = [&](long long row) {
#pragma unroll
    for (int i = 0; i < TM::I; ++i) {
      at.load(xp, a.ldx, row, a.rows, i, n, nx[i]);
      at.load(gp, a.lddy, row, a.rows, i, n, ng[i]);
      if (DROP && sp) at.load(sp, a.ldds, row, a.rows, i, n, ns[i]);
    }
    nst = a.stats[row];
  };
  auto fetch_ring = [&](long long row, int place) {
    if (row < a.rows) {
      ring.fetch(at, place, 0, xp, a.ldx, row, a.rows, n);
      ring.fetch(at, place, 1, gp, a.lddy, row, a.rows, n);
      if (DROP && sp) ring.fetch(at, place, DROP ? 2 : 0, sp, a.ldds, row, a.rows, n);
    }
    cp_async_commit();
  };
  // As in the forward pass; with dropout, keeping w in registers was the faster (262144 x 256 bf16:
  // 128 us, and 155 us with w read again).
  constexpr bool kReload = LY == kAligned && !DROP;
  float w[TM::I][8], dw[TM::I][8], db[TM::I][8];
  at.set_row(xp + (tn.first < a.rows ? tn.first : 0) * a.ldx);
#pragma unroll
  for (int i = 0; i < TM::I; ++i) {
    if constexpr (kRing || !kReload) at.params(a.w, i, n, buf, w[i]);
    if constexpr (kRing) ring.put_param(0, i, w[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = db[i][j] = 0.f;
  }
  if constexpr (kRing) {
    __syncthreads();
    ring.clear(at, n);
    for (int i = 0; i < Rg::kDepth; ++i) fetch_ring(tn.first + i * tn.step, i);
    if (tn.first < a.rows) nst = a.stats[tn.first];
  } else {
    if (tn.first < a.rows) fetch(tn.first);
  }
  for (int turn = 0; turn < tn.count; ++turn) {
    const long long row = tn.first + turn * tn.step;
    const bool live = row < a.rows;
    if (TM::WPR > 0 && !live) break;  // the whole team
    const float2 st = nst;
    float hat[TM::I][8], g[TM::I][8], ds[TM::I][8];
    float sum[2];
    float2 two[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    if constexpr (kRing) ring.wait();
#pragma unroll
    for (int i = 0; i < TM::I; ++i) {
      if constexpr (kRing) {
        ring.get_param(0, i, w[i]);
        ring.take(0, i, nx[i]);
        ring.take(1, i, ng[i]);
      } else if constexpr (kReload) {
        at.params(a.w, i, n, buf, w[i]);
      }
      at.clean(nx[i], i, n, hat[i]);
      at.clean(ng[i], i, n, g[i]);
      if (!kRing && DROP && sp) at.clean(ns[i], i, n, ds[i]);
    }
    if constexpr (kRing) {
      if (row + tn.step < a.rows) nst = a.stats[row + tn.step];
    } else {
      if (row + tn.step < a.rows) fetch(row + tn.step);
    }
#pragma unroll
    for (int i = 0; i < TM::I; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // Outside the row dy is zero, and so is all that it enters.
        const float2 d = live ? pair(g[i], j) : make_float2(0.f, 0.f);
        const float2 ht = __fmul2_rn(__fadd2_rn(pair(hat[i], j), twice(-st.x)), twice(st.y));
        if (live) set_pair(dw[i], j, fma2(d, ht, pair(dw[i], j)));
        set_pair(db[i], j, __fadd2_rn(pair(db[i], j), d));
        const float2 gw = __fmul2_rn(d, pair(w[i], j));
        set_pair(hat[i], j, ht);
        set_pair(g[i], j, gw);
        two[0] = __fadd2_rn(two[0], gw);
        two[1] = fma2(gw, ht, two[1]);
      }
    }
    sum[0] = two[0].x + two[0].y;
    sum[1] = two[1].x + two[1].y;
    team_sum<TM>(sum, slot, turn & 1, at.team);
    const float c1 = sum[0] * inv_n, c2 = sum[1] * inv_n;
    // st.y (g - c1 - hat c2)
    auto grad = [&](int i, int j) {
      const float2 left = fma2(pair(hat[i], j), twice(-c2), __fadd2_rn(pair(g[i], j), twice(-c1)));
      return __fmul2_rn(left, twice(st.y));
    };
    if constexpr (kRing) {  // this row has been read, the stream's gradient apart
      if (DROP && sp) {
#pragma unroll
        for (int i = 0; i < TM::I; ++i) {
          ring.take(DROP ? 2 : 0, i, ns[i]);
          at.clean(ns[i], i, n, ds[i]);
        }
      }
    }
    if constexpr (DROP) {
#pragma unroll
      for (int i = 0; i < TM::I; ++i) {
        bool keep[8];
        at.keep(key, static_cast<uint32_t>(row), i, a.cut, keep);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float2 d = grad(i, j);
          if (sp) d = __fadd2_rn(d, pair(ds[i], j));
          set_pair(g[i], j, d);
          d = __fmul2_rn(d, twice(a.scale));
          hat[i][2 * j] = keep[2 * j] ? d.x : 0.f;
          hat[i][2 * j + 1] = keep[2 * j + 1] ? d.y : 0.f;
        }
        if (live) {
          if (a.dres) at.store(static_cast<T*>(a.dres) + row * a.lddr, i, n, g[i]);
          at.store(static_cast<T*>(a.dx) + row * a.lddx, i, n, hat[i]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < TM::I; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) set_pair(g[i], j, grad(i, j));
        if (live) at.store(static_cast<T*>(a.dx) + row * a.lddx, i, n, g[i]);
      }
    }
    if constexpr (kRing) {
      fetch_ring(row + Rg::kDepth * tn.step, ring.at);
      ring.next();
    }
  }
  if constexpr (kRing) __syncthreads();  // before the ring's memory serves the sums
  // The CTA's sums over its teams, in team order.
  float* pw = a.pw + static_cast<size_t>(blockIdx.x) * n;
  float* pb = a.pb + static_cast<size_t>(blockIdx.x) * n;
  if constexpr (TM::kTeams == 1) {
#pragma unroll
    for (int i = 0; i < TM::I; ++i) {
      at.put_sums(pw, i, n, buf, dw[i]);
      at.put_sums(pb, i, n, buf, db[i]);
    }
  } else {
    // A team's columns lie `shift` further on in its part; teams of one warp are shifted alike
    // only if they are aligned or scalar, so shifted ones are added one team at a time.
    const int wp = threadIdx.x / 32;
    if (at.lane == 0 && at.base == 0) shifts[at.team] = at.shift;
    constexpr bool kFold = TM::WPR == 0 && LY != kShifted;  // a warp's teams are added first
    if constexpr (kFold) {
#pragma unroll
      for (int d = TM::L; d < 32; d <<= 1)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          dw[0][j] += __shfl_xor_sync(0xffffffffu, dw[0][j], d);
          db[0][j] += __shfl_xor_sync(0xffffffffu, db[0][j], d);
        }
    }
    // Place of a column of this warp's part: within the tile, after the tiles of the warp's
    // teams before.
    const int tile = TM::WPR == 0 && !kFold ? (threadIdx.x % 32) / TM::L * (8 * TM::L) : 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = (LY == kScalar ? j * TM::kLanes + at.lane : at.lane * 8 + j) + tile;
      if (!kFold || threadIdx.x % 32 < TM::L) {
        part[0][wp][c] = dw[0][j];
        part[1][wp][c] = db[0][j];
      }
    }
    __syncthreads();
    constexpr int kPer = TM::WPR > 0 ? TM::WPR : 1;                   // warps of one set
    constexpr int kSets = kFold ? kThreads / 32 : TM::kTeams;         // sets of the same columns
    for (int c = threadIdx.x; c < n; c += kThreads) {
      float sw = 0.f, sb = 0.f;
      for (int t = 0; t < kSets; ++t) {
        int wt = t * kPer, p = c;
        if constexpr (LY == kShifted) p += shifts[t];
        if constexpr (TM::WPR == 0 && !kFold) {
          constexpr int kIn = 32 / TM::L;  // teams of a warp
          wt = t / kIn;
          p += t % kIn * (8 * TM::L);
        }
        sw += part[0][wt + (TM::WPR > 0 ? p / 256 : 0)][p % 256];
        sb += part[1][wt + (TM::WPR > 0 ? p / 256 : 0)][p % 256];
      }
      pw[c] = sw;
      pb[c] = sb;
    }
  }
}

// Rows longer than a team's registers: one CTA a row, read again for each sum.  Dropout works on
// groups of eight columns, one group a thread at a time.
template <typename T, bool DROP>
__global__ void __launch_bounds__(kThreads) norm_long_fwd_kernel(const NormArgs a) {
  using TM = Team<kWholeCta, 32, 1>;
  __shared__ Slots<1> slot;
  clear_slots<TM>(slot);
  const long long row = blockIdx.x;
  const int n = a.n;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  if constexpr (DROP) {
    const DropKey key = drop_key(a.rng);
    const T* rp = static_cast<const T*>(a.residual);
    T* s = static_cast<T*>(a.s) + row * a.lds;
    for (int g = threadIdx.x; g < (n + 7) / 8; g += kThreads) {
      bool keep[8];
      keep8(key, static_cast<uint32_t>(row), g, a.cut, keep);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = g * 8 + j;
        if (c >= n) break;
        float d = keep[j] ? __fmul_rn(to_f32(x[c]), a.scale) : 0.f;
        if (rp) d = __fadd_rn(to_f32(rp[row * a.ldr + c]), d);
        s[c] = from_f32<T>(d);
      }
    }
    __syncthreads();
    x = s;
  }
  float sum[1] = {0.f};
  for (int c = threadIdx.x; c < n; c += kThreads) sum[0] += to_f32(x[c]);
  team_sum<TM>(sum, slot, 0, 0);
  const float mean = sum[0] / static_cast<float>(n);
  sum[0] = 0.f;
  for (int c = threadIdx.x; c < n; c += kThreads) {
    const float d = to_f32(x[c]) - mean;
    sum[0] = fmaf(d, d, sum[0]);
  }
  team_sum<TM>(sum, slot, 1, 0);
  const float rstd = rsqrtf(sum[0] / static_cast<float>(n) + a.eps);
  T* y = static_cast<T*>(a.y) + row * a.ldy;
  for (int c = threadIdx.x; c < n; c += kThreads)
    y[c] = from_f32<T>(fmaf((to_f32(x[c]) - mean) * rstd, a.w[c], a.b[c]));
  if (threadIdx.x == 0) a.stats[row] = make_float2(mean, rstd);
}

template <typename T, bool DROP>
__global__ void __launch_bounds__(kThreads) norm_long_bwd_kernel(const NormArgs a) {
  using TM = Team<kWholeCta, 32, 1>;
  __shared__ Slots<2> slot;
  clear_slots<TM>(slot);
  const long long row = blockIdx.x;
  const int n = a.n;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
  const float2 st = a.stats[row];
  float sum[2] = {0.f, 0.f};
  for (int c = threadIdx.x; c < n; c += kThreads) {
    const float g = to_f32(dy[c]) * a.w[c];
    sum[0] += g;
    sum[1] = fmaf(g, (to_f32(x[c]) - st.x) * st.y, sum[1]);
  }
  team_sum<TM>(sum, slot, 0, 0);
  const float c1 = sum[0] / static_cast<float>(n), c2 = sum[1] / static_cast<float>(n);
  T* dx = static_cast<T*>(a.dx) + row * a.lddx;
  DropKey key{};
  if constexpr (DROP) key = drop_key(a.rng);
  for (int g = threadIdx.x; g < (n + 7) / 8; g += kThreads) {
    bool keep[8] = {};
    if constexpr (DROP) keep8(key, static_cast<uint32_t>(row), g, a.cut, keep);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = g * 8 + j;
      if (c >= n) break;
      float d = st.y * (to_f32(dy[c]) * a.w[c] - c1 - (to_f32(x[c]) - st.x) * st.y * c2);
      if constexpr (DROP) {
        if (a.ds) d += to_f32(static_cast<const T*>(a.ds)[row * a.ldds + c]);
        if (a.dres) static_cast<T*>(a.dres)[row * a.lddr + c] = from_f32<T>(d);
        d = keep[j] ? d * a.scale : 0.f;
      }
      dx[c] = from_f32<T>(d);
    }
  }
}

// Parameter gradients of long rows: a thread a column, a block of rows a CTA (grid: column
// blocks x row blocks).
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_long_param_kernel(const NormArgs a) {
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= a.n) return;
  float dw = 0.f, db = 0.f;
  for (long long row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const float2 st = a.stats[row];
    const float d = to_f32(static_cast<const T*>(a.dy)[row * a.lddy + c]);
    const float h = (to_f32(static_cast<const T*>(a.x)[row * a.ldx + c]) - st.x) * st.y;
    dw = fmaf(d, h, dw);
    db += d;
  }
  a.pw[static_cast<size_t>(blockIdx.y) * a.n + c] = dw;
  a.pb[static_cast<size_t>(blockIdx.y) * a.n + c] = db;
}

// out = residual + keep * x * scale (a null residual: no sum).  The backward pass is the same
// kernel on the gradient.
template <typename T, typename TM, Layout LY>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const NormArgs a) {
  Lane<TM, LY> at;
  const DropKey key = drop_key(a.rng);
  const int n = a.n;
  const int pieces = (n + (LY == kShifted ? 7 : 0) + TM::cols() - 1) / TM::cols();
  const long long tiles = static_cast<long long>(a.rows) * pieces;
  const long long per = static_cast<long long>(gridDim.x) * TM::kTeams;
  const long long turns = (tiles + per - 1) / per;
  const T* const xp = static_cast<const T*>(a.x);
  const T* const rp = static_cast<const T*>(a.residual);
  for (long long turn = 0; turn < turns; ++turn) {
    const long long t = turn * per + static_cast<long long>(blockIdx.x) * TM::kTeams + at.team;
    const bool live = t < tiles;
    const long long row = live ? t / pieces : a.rows - 1;
    const int piece = live ? static_cast<int>(t % pieces) : 0;
    at.set_row(xp + row * a.ldx);
    Raw8<T> rx, rr;
    float v[8], res[8];
    at.load(xp, a.ldx, row, a.rows, piece, n, rx);
    if (rp) at.load(rp, a.ldr, row, a.rows, piece, n, rr);
    bool keep[8];
    at.keep(key, static_cast<uint32_t>(row), piece, a.cut, keep);
    at.clean(rx, piece, n, v);
    if (rp) at.clean(rr, piece, n, res);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = keep[j] ? __fmul_rn(v[j], a.scale) : 0.f;
      if (rp) v[j] = __fadd_rn(res[j], v[j]);
    }
    if (live) at.store(static_cast<T*>(a.s) + row * a.lds, piece, n, v);
  }
}

// ---- host side ----

constexpr int kLongCols = 8192;  // widest row that a team holds in registers

// How the call's rows are laid out (see Layout); `params`: w and b are read in groups too.
struct Rows {
  const void* p;
  long long ld;
};
Layout layout_of(const NormArgs& a, size_t e) {
  const Rows r[] = {{a.x, a.ldx}, {a.residual, a.ldr}, {a.dy, a.lddy}, {a.ds, a.ldds},
                    {a.s, a.lds}, {a.y, a.ldy}, {a.dx, a.lddx}, {a.dres, a.lddr}};
  const uintptr_t start = reinterpret_cast<uintptr_t>(a.x) % (8 * e);
  const long long ld = a.ldx % 8;
  for (const Rows& q : r)
    if (q.p && (reinterpret_cast<uintptr_t>(q.p) % (8 * e) != start || q.ld % 8 != ld)) return kScalar;
  const bool params = reinterpret_cast<uintptr_t>(a.w) % 32 == 0 && reinterpret_cast<uintptr_t>(a.b) % 32 == 0;
  return start == 0 && ld == 0 && a.n % 8 == 0 && params ? kAligned : kShifted;
}

// f(team, threads of a CTA) for rows of `n` columns (a shifted row may touch one group more).
template <typename F>
cudaError_t by_width(int n, Layout ly, F&& f) {
  const int c = ly == kShifted ? n + 7 : n;
  if (c <= 32) return f(Team<0, 4, 1>{}, kThreads);
  if (c <= 64) return f(Team<0, 8, 1>{}, kThreads);
  if (c <= 128) return f(Team<0, 16, 1>{}, kThreads);
  if (c <= 256) return f(Team<1, 32, 1>{}, kThreads);
  if (c <= 512) return f(Team<2, 32, 1>{}, kThreads);
  if (c <= 1024) return f(Team<4, 32, 1>{}, kThreads);
  if (c <= 4096) return f(Team<kWholeCta, 32, 2>{}, (c + 511) / 512 * 32);
  return f(Team<kWholeCta, 32, 2, kMaxWarps>{}, (c + 511) / 512 * 32);
}
// Widest row: in two pieces of 16 warps.
bool long_row(int n, Layout ly) { return n + (ly == kShifted ? 7 : 0) > kLongCols; }

// CTAs of the backward pass, which is also the number of partial sums: as many as are resident (whole
// CTAs 512 threads an SM; of 256 threads two with dropout, else three; 262144 x 256: fp32 125 us with three an SM, 134 and
// 136 us with two and four; bf16 with dropout 128 us with two, 132 and 155 us with four and three).
// Multiples of eight, where a team takes several rows.
constexpr int kLongParts = 64;
int most_ctas(int n, int threads, bool drop) {
  return 152 * (threads != kThreads || n > 1024 ? 512 / threads : drop && n <= 256 ? 2 : 3);
}
int ctas_for(int rows, int teams, int most) {
  const long long need = (static_cast<long long>(rows) + teams - 1) / teams;
  return need < most ? static_cast<int>(need) : most;
}

template <typename F>
cudaError_t by_layout(Layout ly, F&& f) {
  if (ly == kAligned) return f(std::integral_constant<Layout, kAligned>{});
  if (ly == kShifted) return f(std::integral_constant<Layout, kShifted>{});
  return f(std::integral_constant<Layout, kScalar>{});
}

// Shared memory of a ring of NT tensors and `params` parameters (at most 224 KB: 8192 columns, fp32,
// backward with dropout).
template <bool RING, typename T, typename TM, Layout LY, int NT>
cudaError_t launch_rows(void (*kern)(const NormArgs), LaunchCfg c, const NormArgs& a, int params) {
  if constexpr (RING) {
    using Rg = Ring<T, TM, LY, NT>;
    c.smem = 16 * static_cast<size_t>(c.block.x) * (Rg::kDepth * Rg::kRow + params * Rg::kParam);
    const cudaError_t e = allow_smem(kern, c.smem, 16 * static_cast<size_t>(TM::kMaxThreads) *
                                                       (Rg::kDepth * Rg::kRow + params * Rg::kParam));
    if (e != cudaSuccess) return e;
  }
  return launch(c, kern, a);
}

template <typename T, bool DROP>
cudaError_t fwd(const NormArgs& a, cudaStream_t s) {
  LaunchCfg c;
  c.stream = s;
  const Layout ly = layout_of(a, sizeof(T));
  if (long_row(a.n, ly)) {
    c.block = dim3(kThreads);
    c.grid = dim3(a.rows);
    return launch(c, norm_long_fwd_kernel<T, DROP>, a);
  }
  return by_width(a.n, ly, [&](auto tm, int threads) {
    using TM = decltype(tm);
    c.block = dim3(threads);
    return by_layout(ly, [&](auto layout) {
      constexpr Layout LY = decltype(layout)::value;
      constexpr bool ring = fwd_ring<T, TM, LY, DROP>();
      // As many as are resident where a CTA's first row waits for its parameters (unaligned rows),
      // or for a ring; aligned rows twice that, so that the last ones are evened out.
      const int most = ring             ? (DROP ? 512 : 1024) / threads
                       : LY == kAligned ? 8
                       : TM::kWhole     ? 3
                                        : fwd_ctas<T, TM, LY, DROP>();
      c.grid = dim3(ctas_for(a.rows, TM::kTeams, 152 * most));
      return launch_rows<ring, T, TM, LY, DROP ? 2 : 1>(norm_fwd_kernel<T, TM, LY, DROP>, c, a, 2);
    });
  });
}

template <typename T, bool DROP>
cudaError_t bwd(NormArgs a, float* dw, float* db, float* ws, cudaStream_t s) {
  LaunchCfg c;
  c.stream = s;
  const Layout ly = layout_of(a, sizeof(T));
  int G = 1;
  auto parts = [&](int count) {  // one CTA: its sums are the result
    G = count;
    a.pw = G == 1 ? dw : ws;
    a.pb = G == 1 ? db : ws + static_cast<size_t>(G) * a.n;
  };
  cudaError_t e;
  if (long_row(a.n, ly)) {
    parts(a.rows < kLongParts ? a.rows : kLongParts);
    c.block = dim3(kThreads);
    c.grid = dim3((a.n + kThreads - 1) / kThreads, G);
    e = launch(c, norm_long_param_kernel<T>, a);
    c.grid = dim3(a.rows);
    if (e == cudaSuccess) e = launch(c, norm_long_bwd_kernel<T, DROP>, a);
  } else {
    e = by_width(a.n, ly, [&](auto tm, int threads) {
      using TM = decltype(tm);
      parts(ctas_for(a.rows, TM::kTeams, most_ctas(a.n, threads, DROP)));
      c.block = dim3(threads);
      c.grid = dim3(G);
      return by_layout(ly, [&](auto layout) {
        constexpr Layout LY = decltype(layout)::value;
        return launch_rows<bwd_ring<T, TM, LY, DROP>(), T, TM, LY, DROP ? 3 : 2>(
            norm_bwd_kernel<T, TM, LY, DROP>, c, a, 1);
      });
    });
  }
  if (e != cudaSuccess || G == 1) return e;
  return reduce_axis0_pair_launch(a.pw, G, a.n, 0, 0, dw, nullptr, a.pb, G, a.n, db, s, true);
}

template <typename T>
cudaError_t drop(const NormArgs& a, cudaStream_t s) {
  LaunchCfg c;
  c.stream = s;
  const Layout ly = layout_of(a, sizeof(T));
  const int most = ly == kShifted ? 249 : 256;
  return by_width(a.n < most ? a.n : most, ly, [&](auto tm, int threads) -> cudaError_t {
    using TM = decltype(tm);
    if constexpr (TM::WPR > 1) {
      return cudaErrorInvalidValue;  // not reached: at most one warp a row
    } else {
      constexpr int cols = 8 * TM::kLanes;
      const int shift = ly == kShifted ? 7 : 0;
      const long long tiles = static_cast<long long>(a.rows) * ((a.n + shift + cols - 1) / cols);
      const long long need = (tiles + TM::kTeams - 1) / TM::kTeams;
      c.block = dim3(threads);
      c.grid = dim3(static_cast<unsigned>(need < 152 * 8 ? need : 152 * 8));
      return by_layout(ly, [&](auto layout) {
        return launch(c, dropout_kernel<T, TM, decltype(layout)::value>, a);
      });
    }
  });
}

NormArgs to_args(const NormCall& q) {
  NormArgs a{};
  a.x = q.x; a.ldx = q.ldx;
  a.residual = q.residual; a.ldr = q.ldr;
  a.dy = q.dy; a.lddy = q.lddy;
  a.ds = q.ds; a.ldds = q.ldds;
  a.w = q.w; a.b = q.b;
  a.rng = q.rng;
  a.cut = q.cut; a.scale = q.scale; a.eps = q.eps;
  a.rows = q.rows; a.n = q.n;
  a.s = q.s; a.lds = q.lds;
  a.y = q.y; a.ldy = q.ldy;
  a.dx = q.dx; a.lddx = q.lddx;
  a.dres = q.dres; a.lddr = q.lddr;
  a.stats = reinterpret_cast<float2*>(q.stats);
  return a;
}

}  // namespace

// Enough for every layout: shifted rows may take the next wider team, with fewer teams a CTA and
// so more CTAs.
size_t norm_ws_floats(int rows, int n) {
  int most = 1;
  for (const Layout ly : {kAligned, kShifted}) {
    int G = rows < kLongParts ? rows : kLongParts;
    if (!long_row(n, ly))
      (void)by_width(n, ly, [&](auto tm, int threads) {
        G = ctas_for(rows, decltype(tm)::kTeams, most_ctas(n, threads, false));
        return cudaSuccess;
      });
    if (G > most) most = G;
  }
  return most == 1 ? 0 : 2 * static_cast<size_t>(most) * n;
}

cudaError_t norm_fwd_launch(const NormCall& q, cudaStream_t s) {
  const NormArgs a = to_args(q);
  if (q.bf16) return q.rng ? fwd<__nv_bfloat16, true>(a, s) : fwd<__nv_bfloat16, false>(a, s);
  return q.rng ? fwd<float, true>(a, s) : fwd<float, false>(a, s);
}

cudaError_t norm_bwd_launch(const NormCall& q, float* dw, float* db, float* ws, cudaStream_t s) {
  const NormArgs a = to_args(q);
  if (q.bf16)
    return q.rng ? bwd<__nv_bfloat16, true>(a, dw, db, ws, s)
                 : bwd<__nv_bfloat16, false>(a, dw, db, ws, s);
  return q.rng ? bwd<float, true>(a, dw, db, ws, s) : bwd<float, false>(a, dw, db, ws, s);
}

cudaError_t dropout_launch(const NormCall& q, cudaStream_t s) {
  const NormArgs a = to_args(q);
  return q.bf16 ? drop<__nv_bfloat16>(a, s) : drop<float>(a, s);
}

}  // namespace cfc
