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
// left, so that a large mean costs no precision).  A row belongs to a team of lanes, eight
// columns to a lane: 4 to 32 lanes of one warp up to 256 columns, 2 to 8 warps beyond, with two
// or four pieces of 2048 columns up to 8192.  Longer rows are read again for each sum (they stay
// in L2).  The parameter gradients stay in each lane's registers over all rows of its CTA, are
// added over the CTA's teams in shared memory and over the CTAs by reduce_axis0: no atomics, and
// an order that depends on the sizes alone.  The dropout mask is never stored: both passes draw
// it again from the counter-based generator, whose counter is the element's place.
#include "cfc_kernels.h"
#include "cfc_launch.cuh"
#include "cfc_trunk.cuh"

namespace cfc {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// How a team of lanes covers a row: WPR > 0: WPR warps and I pieces of 256 * WPR columns;
// WPR == 0: L lanes of a warp (32 / L rows per warp), one piece.
template <int WPR_, int L_, int I_>
struct Team {
  static constexpr int WPR = WPR_, L = L_, I = I_;
  static constexpr int kLanes = WPR > 0 ? 32 : L;                    // lanes of one warp's tile
  static constexpr int kTeams = WPR > 0 ? kWarps / WPR : kThreads / L;  // teams per CTA
  static constexpr int kCols = 8 * kLanes * (WPR > 0 ? WPR : 1);     // columns per piece
};

// A lane's place: which team of the CTA, and its first column and column stride in a piece.
// Aligned rows: eight consecutive columns.  Others: columns kLanes apart, so that a warp's
// scalar loads are consecutive.
template <typename TM, bool ALIGNED>
struct Lane {
  int team, lane, base;  // base: first column of this warp's tile in a piece
  __device__ __forceinline__ Lane() {
    if constexpr (TM::WPR > 0) {
      const int w = threadIdx.x / 32;
      team = w / TM::WPR;
      lane = threadIdx.x % 32;
      base = (w % TM::WPR) * 256;
    } else {
      team = threadIdx.x / TM::L;
      lane = threadIdx.x % TM::L;
      base = 0;
    }
  }
  __device__ __forceinline__ int col(int piece, int j) const {
    return piece * TM::kCols + base + (ALIGNED ? lane * 8 + j : j * TM::kLanes + lane);
  }
  // The lane's eight columns of a row piece, `fill` beyond the row's end.
  template <typename T>
  __device__ __forceinline__ void load(const T* row, int piece, int n, float fill,
                                       float (&v)[8]) const {
    if constexpr (ALIGNED) {
      if (col(piece, 0) < n) {
        load8(row + col(piece, 0), v);
        return;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = fill;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = col(piece, j) < n ? to_f32(row[col(piece, j)]) : fill;
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(T* row, int piece, int n, const float (&v)[8]) const {
    if constexpr (ALIGNED) {
      if (col(piece, 0) < n) store8(row + col(piece, 0), v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (col(piece, j) < n) row[col(piece, j)] = from_f32<T>(v[j]);
    }
  }
  // Keep bits of the lane's eight columns.  The generator serves eight consecutive columns; where
  // a lane's columns are not consecutive, each lane draws for its eight consecutive ones and the
  // bits change hands inside the warp's tile.  Every lane of the warp takes part.
  __device__ __forceinline__ uint32_t keep(const DropKey& k, uint32_t row, int piece,
                                           uint32_t cut) const {
    const uint32_t group = static_cast<uint32_t>((piece * TM::kCols + base) / 8 + lane);
    const uint32_t own = keep_mask8(k, row, group, cut);
    if constexpr (ALIGNED) return own;
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int at = j * TM::kLanes + lane;
      const uint32_t from = __shfl_sync(0xffffffffu, own, at >> 3, TM::kLanes);
      m |= ((from >> (at & 7)) & 1u) << j;
    }
    return m;
  }
};

// Sum of (a, b) over the team.  Teams of several warps go through shared memory: `slot` holds
// two sets of two floats per warp, used in turn, so one barrier a sum is enough.
template <typename TM>
__device__ __forceinline__ float2 team_sum(float2 v, float2 (*slot)[kWarps], int turn, int team) {
  constexpr int kSpan = TM::WPR > 0 ? 32 : TM::L;
#pragma unroll
  for (int d = kSpan / 2; d > 0; d >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, d);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, d);
  }
  if constexpr (TM::WPR > 1) {
    const int w = threadIdx.x / 32;
    if (threadIdx.x % 32 == 0) slot[turn][w] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(TM::WPR * 32) : "memory");
    v = slot[turn][team * TM::WPR];
#pragma unroll
    for (int i = 1; i < TM::WPR; ++i) {
      const float2 o = slot[turn][team * TM::WPR + i];
      v.x += o.x;
      v.y += o.y;
    }
  }
  return v;
}

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

template <typename T, typename TM, bool ALIGNED, bool DROP>
__global__ void __launch_bounds__(kThreads) norm_fwd_kernel(const NormArgs a) {
  __shared__ float2 slot[2][kWarps];
  const Lane<TM, ALIGNED> at;
  const int n = a.n;
  const float inv_n = 1.f / static_cast<float>(n);
  DropKey key{};
  if constexpr (DROP) key = drop_key(a.rng);
  // Teams of one warp share its shuffles, so they take the same number of turns.
  const long long per = static_cast<long long>(gridDim.x) * TM::kTeams;
  const int turns = static_cast<int>((a.rows + per - 1) / per);
  for (int turn = 0; turn < turns; ++turn) {
    const long long r = turn * per + static_cast<long long>(blockIdx.x) * TM::kTeams + at.team;
    const bool live = r < a.rows;
    if (TM::WPR > 0 && !live) return;  // the whole team
    const long long row = live ? r : a.rows - 1;
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    float v[TM::I][8];
#pragma unroll
    for (int i = 0; i < TM::I; ++i) at.load(x, i, n, 0.f, v[i]);
    if constexpr (DROP) {
      float res[TM::I][8];
      const T* rp = static_cast<const T*>(a.residual);
      if (rp) {
#pragma unroll
        for (int i = 0; i < TM::I; ++i) at.load(rp + row * a.ldr, i, n, 0.f, res[i]);
      }
#pragma unroll
      for (int i = 0; i < TM::I; ++i) {
        const uint32_t keep = at.keep(key, static_cast<uint32_t>(row), i, a.cut);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          // Product and sum rounded apart: the same values as dropout followed by the sum.
          float d = (keep >> j & 1u) ? __fmul_rn(v[i][j], a.scale) : 0.f;
          if (rp) d = __fadd_rn(res[i][j], d);
          // The norm reads the stream as it is stored, so that the backward pass, which reads
          // the stored stream, differentiates what the forward pass computed.
          v[i][j] = to_f32(from_f32<T>(d));
        }
        if (live) at.store(static_cast<T*>(a.s) + row * a.lds, i, n, v[i]);
      }
      // Beyond the row's end the generator may have kept nothing but zeros; they stay zero.
    }
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < TM::I; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) sum.x += v[i][j];
    const float mean = team_sum<TM>(sum, slot, 0, at.team).x * inv_n;
    sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < TM::I; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float c = at.col(i, j) < n ? v[i][j] - mean : 0.f;
        sum.x = fmaf(c, c, sum.x);
      }
    const float rstd = rsqrtf(team_sum<TM>(sum, slot, 1, at.team).x * inv_n + a.eps);
    if (!live) continue;
    T* y = static_cast<T*>(a.y) + row * a.ldy;
#pragma unroll
    for (int i = 0; i < TM::I; ++i) {
      float w[8], b[8];
      at.load(a.w, i, n, 0.f, w);
      at.load(a.b, i, n, 0.f, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = fmaf((v[i][j] - mean) * rstd, w[j], b[j]);
      at.store(y, i, n, v[i]);
    }
    if (at.base == 0 && at.lane == 0) a.stats[row] = make_float2(mean, rstd);
  }
}

template <typename T, typename TM, bool ALIGNED, bool DROP>
__global__ void __launch_bounds__(kThreads) norm_bwd_kernel(const NormArgs a) {
  __shared__ float2 slot[2][kWarps];
  __shared__ float part[2][kWarps][256];
  grid_dep_launch_dependents();
  const Lane<TM, ALIGNED> at;
  const int n = a.n;
  const float inv_n = 1.f / static_cast<float>(n);
  DropKey key{};
  if constexpr (DROP) key = drop_key(a.rng);
  float dw[TM::I][8], db[TM::I][8];
#pragma unroll
  for (int i = 0; i < TM::I; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = db[i][j] = 0.f;
  const long long per = static_cast<long long>(gridDim.x) * TM::kTeams;
  const int turns = static_cast<int>((a.rows + per - 1) / per);
  for (int turn = 0; turn < turns; ++turn) {
    const long long r = turn * per + static_cast<long long>(blockIdx.x) * TM::kTeams + at.team;
    const bool live = r < a.rows;
    if (TM::WPR > 0 && !live) break;  // the whole team
    const long long row = live ? r : a.rows - 1;
    const float2 st = a.stats[row];
    float hat[TM::I][8], g[TM::I][8];
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < TM::I; ++i) {
      at.load(static_cast<const T*>(a.x) + row * a.ldx, i, n, st.x, hat[i]);
      at.load(static_cast<const T*>(a.dy) + row * a.lddy, i, n, 0.f, g[i]);
    }
#pragma unroll
    for (int i = 0; i < TM::I; ++i) {
      float w[8];
      at.load(a.w, i, n, 0.f, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = live ? g[i][j] : 0.f;
        hat[i][j] = (hat[i][j] - st.x) * st.y;
        if (live) dw[i][j] = fmaf(d, hat[i][j], dw[i][j]);
        db[i][j] += d;
        g[i][j] = d * w[j];
        sum.x += g[i][j];
        sum.y = fmaf(g[i][j], hat[i][j], sum.y);
      }
    }
    sum = team_sum<TM>(sum, slot, turn & 1, at.team);
    const float c1 = sum.x * inv_n, c2 = sum.y * inv_n;
    if constexpr (DROP) {
#pragma unroll
      for (int i = 0; i < TM::I; ++i) {
        float ds[8];
        const T* dsp = static_cast<const T*>(a.ds);
        if (dsp) at.load(dsp + row * a.ldds, i, n, 0.f, ds);
        const uint32_t keep = at.keep(key, static_cast<uint32_t>(row), i, a.cut);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          g[i][j] = st.y * (g[i][j] - c1 - hat[i][j] * c2) + (dsp ? ds[j] : 0.f);
          hat[i][j] = (keep >> j & 1u) ? g[i][j] * a.scale : 0.f;
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
        for (int j = 0; j < 8; ++j) g[i][j] = st.y * (g[i][j] - c1 - hat[i][j] * c2);
        if (live) at.store(static_cast<T*>(a.dx) + row * a.lddx, i, n, g[i]);
      }
    }
  }
  // The CTA's sums over its teams, in team order.
  float* pw = a.pw + static_cast<size_t>(blockIdx.x) * n;
  float* pb = a.pb + static_cast<size_t>(blockIdx.x) * n;
  if constexpr (TM::kTeams == 1) {
#pragma unroll
    for (int i = 0; i < TM::I; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (at.col(i, j) < n) {
          pw[at.col(i, j)] = dw[i][j];
          pb[at.col(i, j)] = db[i][j];
        }
  } else {
    const int w = threadIdx.x / 32;
    if constexpr (TM::WPR == 0) {
#pragma unroll
      for (int d = TM::L; d < 32; d <<= 1)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          dw[0][j] += __shfl_xor_sync(0xffffffffu, dw[0][j], d);
          db[0][j] += __shfl_xor_sync(0xffffffffu, db[0][j], d);
        }
    }
    constexpr int kSets = TM::WPR > 0 ? TM::kTeams : kWarps;  // warps that hold the same columns
    constexpr int kPer = TM::WPR > 0 ? TM::WPR : 1;           // warps of one set
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = at.col(0, j) - at.base;
      if (TM::WPR > 0 || threadIdx.x % 32 < TM::L) {
        part[0][w][c] = dw[0][j];
        part[1][w][c] = db[0][j];
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < TM::kCols && c < n; c += kThreads) {
      float sw = 0.f, sb = 0.f;
#pragma unroll
      for (int t = 0; t < kSets; ++t) {
        sw += part[0][t * kPer + c / 256][c % 256];
        sb += part[1][t * kPer + c / 256][c % 256];
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
  using TM = Team<kWarps, 32, 1>;
  __shared__ float2 slot[2][kWarps];
  const long long row = blockIdx.x;
  const int n = a.n;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  if constexpr (DROP) {
    const DropKey key = drop_key(a.rng);
    const T* rp = static_cast<const T*>(a.residual);
    T* s = static_cast<T*>(a.s) + row * a.lds;
    for (int g = threadIdx.x; g < (n + 7) / 8; g += kThreads) {
      const uint32_t keep = keep_mask8(key, static_cast<uint32_t>(row), g, a.cut);
      for (int j = 0; j < 8 && g * 8 + j < n; ++j) {
        const int c = g * 8 + j;
        float d = (keep >> j & 1u) ? __fmul_rn(to_f32(x[c]), a.scale) : 0.f;
        if (rp) d = __fadd_rn(to_f32(rp[row * a.ldr + c]), d);
        s[c] = from_f32<T>(d);
      }
    }
    __syncthreads();
    x = s;
  }
  float2 sum = make_float2(0.f, 0.f);
  for (int c = threadIdx.x; c < n; c += kThreads) sum.x += to_f32(x[c]);
  const float mean = team_sum<TM>(sum, slot, 0, 0).x / static_cast<float>(n);
  sum = make_float2(0.f, 0.f);
  for (int c = threadIdx.x; c < n; c += kThreads) {
    const float d = to_f32(x[c]) - mean;
    sum.x = fmaf(d, d, sum.x);
  }
  const float rstd = rsqrtf(team_sum<TM>(sum, slot, 1, 0).x / static_cast<float>(n) + a.eps);
  T* y = static_cast<T*>(a.y) + row * a.ldy;
  for (int c = threadIdx.x; c < n; c += kThreads)
    y[c] = from_f32<T>(fmaf((to_f32(x[c]) - mean) * rstd, a.w[c], a.b[c]));
  if (threadIdx.x == 0) a.stats[row] = make_float2(mean, rstd);
}

template <typename T, bool DROP>
__global__ void __launch_bounds__(kThreads) norm_long_bwd_kernel(const NormArgs a) {
  using TM = Team<kWarps, 32, 1>;
  __shared__ float2 slot[2][kWarps];
  const long long row = blockIdx.x;
  const int n = a.n;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
  const float2 st = a.stats[row];
  float2 sum = make_float2(0.f, 0.f);
  for (int c = threadIdx.x; c < n; c += kThreads) {
    const float g = to_f32(dy[c]) * a.w[c];
    sum.x += g;
    sum.y = fmaf(g, (to_f32(x[c]) - st.x) * st.y, sum.y);
  }
  sum = team_sum<TM>(sum, slot, 0, 0);
  const float c1 = sum.x / static_cast<float>(n), c2 = sum.y / static_cast<float>(n);
  T* dx = static_cast<T*>(a.dx) + row * a.lddx;
  DropKey key{};
  if constexpr (DROP) key = drop_key(a.rng);
  for (int g = threadIdx.x; g < (n + 7) / 8; g += kThreads) {
    uint32_t keep = 0xffu;
    if constexpr (DROP) keep = keep_mask8(key, static_cast<uint32_t>(row), g, a.cut);
    for (int j = 0; j < 8 && g * 8 + j < n; ++j) {
      const int c = g * 8 + j;
      float d = st.y * (to_f32(dy[c]) * a.w[c] - c1 - (to_f32(x[c]) - st.x) * st.y * c2);
      if constexpr (DROP) {
        if (a.ds) d += to_f32(static_cast<const T*>(a.ds)[row * a.ldds + c]);
        if (a.dres) static_cast<T*>(a.dres)[row * a.lddr + c] = from_f32<T>(d);
        d = (keep >> j & 1u) ? d * a.scale : 0.f;
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
template <typename T, typename TM, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const NormArgs a) {
  const Lane<TM, ALIGNED> at;
  const DropKey key = drop_key(a.rng);
  const int n = a.n;
  const int pieces = (n + TM::kCols - 1) / TM::kCols;
  const long long tiles = static_cast<long long>(a.rows) * pieces;
  const long long per = static_cast<long long>(gridDim.x) * TM::kTeams;
  const long long turns = (tiles + per - 1) / per;
  for (long long turn = 0; turn < turns; ++turn) {
    const long long t = turn * per + static_cast<long long>(blockIdx.x) * TM::kTeams + at.team;
    const bool live = t < tiles;
    const long long row = live ? t / pieces : a.rows - 1;
    const int piece = live ? static_cast<int>(t % pieces) : 0;
    float v[8], res[8];
    at.load(static_cast<const T*>(a.x) + row * a.ldx, piece, n, 0.f, v);
    const T* rp = static_cast<const T*>(a.residual);
    if (rp) at.load(rp + row * a.ldr, piece, n, 0.f, res);
    const uint32_t keep = at.keep(key, static_cast<uint32_t>(row), piece, a.cut);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = (keep >> j & 1u) ? __fmul_rn(v[j], a.scale) : 0.f;
      if (rp) v[j] = __fadd_rn(res[j], v[j]);
    }
    if (live) at.store(static_cast<T*>(a.s) + row * a.lds, piece, n, v);
  }
}

// ---- host side ----

constexpr int kLongCols = 8192;  // widest row that a team holds in registers
constexpr int kNormCtas = 152 * 4;

bool rows_aligned(const void* p, long long ld, size_t elem) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % (8 * elem) == 0 && ld % 8 == 0);
}

bool norm_aligned(const NormArgs& a, size_t e) {
  return a.n % 8 == 0 && rows_aligned(a.x, a.ldx, e) && rows_aligned(a.residual, a.ldr, e) &&
         rows_aligned(a.dy, a.lddy, e) && rows_aligned(a.ds, a.ldds, e) &&
         rows_aligned(a.s, a.lds, e) && rows_aligned(a.y, a.ldy, e) &&
         rows_aligned(a.dx, a.lddx, e) && rows_aligned(a.dres, a.lddr, e) &&
         rows_aligned(a.w, 0, 4) && rows_aligned(a.b, 0, 4);
}

// Lanes per row of a team (256: one warp tile up to 256 columns, then whole warps).
template <typename F>
cudaError_t by_width(int n, F&& f) {
  if (n <= 32) return f(Team<0, 4, 1>{});
  if (n <= 64) return f(Team<0, 8, 1>{});
  if (n <= 128) return f(Team<0, 16, 1>{});
  if (n <= 256) return f(Team<1, 32, 1>{});
  if (n <= 512) return f(Team<2, 32, 1>{});
  if (n <= 1024) return f(Team<4, 32, 1>{});
  if (n <= 2048) return f(Team<8, 32, 1>{});
  if (n <= 4096) return f(Team<8, 32, 2>{});
  return f(Team<8, 32, 4>{});
}

int teams_per_cta(int n) {
  return n <= 32 ? 64 : n <= 64 ? 32 : n <= 128 ? 16 : n <= 256 ? 8 : n <= 512 ? 4 : n <= 1024 ? 2 : 1;
}

// CTAs of the backward pass, which is also the number of partial sums: from the sizes alone.
int bwd_ctas(int rows, int n) {
  if (n > kLongCols) return rows < 64 ? rows : 64;
  const int need = (rows + teams_per_cta(n) - 1) / teams_per_cta(n);
  return need < kNormCtas ? need : kNormCtas;
}

template <typename T, bool DROP>
cudaError_t fwd(const NormArgs& a, cudaStream_t s) {
  LaunchCfg c;
  c.block = dim3(kThreads);
  c.stream = s;
  if (a.n > kLongCols) {
    c.grid = dim3(a.rows);
    return launch(c, norm_long_fwd_kernel<T, DROP>, a);
  }
  const bool al = norm_aligned(a, sizeof(T));
  return by_width(a.n, [&](auto tm) {
    using TM = decltype(tm);
    const int need = (a.rows + TM::kTeams - 1) / TM::kTeams;
    c.grid = dim3(need < 2 * kNormCtas ? need : 2 * kNormCtas);
    return al ? launch(c, norm_fwd_kernel<T, TM, true, DROP>, a)
              : launch(c, norm_fwd_kernel<T, TM, false, DROP>, a);
  });
}

template <typename T, bool DROP>
cudaError_t bwd(NormArgs a, float* dw, float* db, float* ws, cudaStream_t s) {
  const int G = bwd_ctas(a.rows, a.n);
  // One CTA: its sums are the result.
  a.pw = G == 1 ? dw : ws;
  a.pb = G == 1 ? db : ws + static_cast<size_t>(G) * a.n;
  LaunchCfg c;
  c.block = dim3(kThreads);
  c.stream = s;
  cudaError_t e;
  if (a.n > kLongCols) {
    c.grid = dim3((a.n + kThreads - 1) / kThreads, G);
    e = launch(c, norm_long_param_kernel<T>, a);
    c.grid = dim3(a.rows);
    if (e == cudaSuccess) e = launch(c, norm_long_bwd_kernel<T, DROP>, a);
  } else {
    const bool al = norm_aligned(a, sizeof(T));
    c.grid = dim3(G);
    e = by_width(a.n, [&](auto tm) {
      using TM = decltype(tm);
      return al ? launch(c, norm_bwd_kernel<T, TM, true, DROP>, a)
                : launch(c, norm_bwd_kernel<T, TM, false, DROP>, a);
    });
  }
  if (e != cudaSuccess || G == 1) return e;
  return reduce_axis0_pair_launch(a.pw, G, a.n, 0, 0, dw, nullptr, a.pb, G, a.n, db, s, true);
}

template <typename T>
cudaError_t drop(const NormArgs& a, cudaStream_t s) {
  LaunchCfg c;
  c.block = dim3(kThreads);
  c.stream = s;
  const bool al = norm_aligned(a, sizeof(T));
  return by_width(a.n < 256 ? a.n : 256, [&](auto tm) {
    using TM = decltype(tm);
    const long long tiles = static_cast<long long>(a.rows) * ((a.n + TM::kCols - 1) / TM::kCols);
    const long long need = (tiles + TM::kTeams - 1) / TM::kTeams;
    c.grid = dim3(static_cast<unsigned>(need < 2 * kNormCtas ? need : 2 * kNormCtas));
    return al ? launch(c, dropout_kernel<T, TM, true>, a) : launch(c, dropout_kernel<T, TM, false>, a);
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

size_t norm_ws_floats(int rows, int n) {
  const int G = bwd_ctas(rows, n);
  return G == 1 ? 0 : 2 * static_cast<size_t>(G) * n;
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
