// cfc_rmsnorm.cu -- root-mean-square norm over rows with the residual's addition, forward and
// backward, its results and its stream in the activations' type or held in 8 bits.
//
//   forward   s = x + residual                        (rounded to its type; s = x without)
//             rstd = (sum s^2 / n + eps)^-1/2,  y = s rstd w
//   backward  hat = s rstd,  g = dy w
//             dx = rstd (g - hat sum(g hat) / n) + ds,  dw = sum_rows dy hat
//
// Every pass is bound by memory: a row stays in registers between its sum and its results.  A row
// belongs to a team: 4 to 32 lanes of a warp up to 1024 columns, a CTA of 128 to 512 threads up to
// 8192.  Longer rows are read twice (the second time from L2).  Where all tensors are aligned and n
// is a multiple of 8, a lane loads and stores eight columns at once, and four neighbouring lanes
// hold a block of the 8-bit form; otherwise neighbouring lanes have neighbouring columns, a warp's
// loads are consecutive whatever the rows' alignment, and a warp holds a block.
//
// dw is summed in each lane's registers over the rows of its team, over the CTA's teams in shared
// memory, and over the CTAs by reduce_axis0: no atomics, an order that depends on the sizes and on
// which of the two layouts runs.
#include "cfc_gated_kernels.h"
#include "cfc_held8.cuh"
#include "cfc_kernels.h"
#include "cfc_launch.cuh"
#include "cfc_trunk.cuh"

namespace cfc {
namespace {

constexpr int kSms = 152;
constexpr int kLongRow = 8192;   // columns from which rows are read twice

// A team of TPR threads a row, SLOTS pieces a thread; a piece is eight columns (VEC) or one.
template <int TPR_, int SLOTS_, bool VEC_>
struct Team {
  static constexpr int TPR = TPR_, SLOTS = SLOTS_;
  static constexpr bool VEC = VEC_, kWarp = TPR <= 32;
  static constexpr int W = VEC ? 8 : 1;            // columns of a piece
  static constexpr int E = SLOTS * W;              // columns of a thread
  static constexpr int kThreads = kWarp ? 256 : TPR;
  static constexpr int kTeams = kThreads / TPR;
  static constexpr int kCols = TPR * E;
  static __device__ __forceinline__ int team() { return threadIdx.x / TPR; }
  static __device__ __forceinline__ int col(int slot) {
    return (slot * TPR + static_cast<int>(threadIdx.x) % TPR) * W;
  }
};

// A thread's columns of a row as they are stored; columns that do not exist are 0.
template <typename T, typename TM>
struct Piece;
template <typename T, int TPR, int SLOTS>
struct Piece<T, Team<TPR, SLOTS, true>> {
  using TM = Team<TPR, SLOTS, true>;
  Raw8<T> raw[SLOTS];
  __device__ __forceinline__ void load(const T* row, int n, bool ok) {
#pragma unroll
    for (int j = 0; j < SLOTS; ++j) {
      if (ok && TM::col(j) < n) raw[j].load(row + TM::col(j));
      else raw[j].clear();
    }
  }
  __device__ __forceinline__ void get(float (&v)[TM::E]) const {
#pragma unroll
    for (int j = 0; j < SLOTS; ++j) {
      float p[8];
      raw[j].get(p);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[8 * j + i] = p[i];
    }
  }
};
template <typename T, int TPR, int SLOTS>
struct Piece<T, Team<TPR, SLOTS, false>> {
  using TM = Team<TPR, SLOTS, false>;
  T raw[SLOTS];
  __device__ __forceinline__ void load(const T* row, int n, bool ok) {
#pragma unroll
    for (int j = 0; j < SLOTS; ++j)
      raw[j] = ok && TM::col(j) < n ? row[TM::col(j)] : from_f32<T>(0.f);
  }
  __device__ __forceinline__ void get(float (&v)[TM::E]) const {
#pragma unroll
    for (int j = 0; j < SLOTS; ++j) v[j] = to_f32(raw[j]);
  }
};

template <typename TM, typename T>
__device__ __forceinline__ void store_row(T* row, const float (&v)[TM::E], int n, bool ok) {
#pragma unroll
  for (int j = 0; j < TM::SLOTS; ++j) {
    if (!(ok && TM::col(j) < n)) continue;
    if constexpr (TM::VEC) {
      float p[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = v[8 * j + i];
      store8(row + TM::col(j), p);
    } else {
      row[TM::col(j)] = from_f32<T>(v[j]);
    }
  }
}

template <typename TM>
__device__ __forceinline__ void load_par(const float* p, float (&v)[TM::E], int n) {
#pragma unroll
  for (int j = 0; j < TM::SLOTS; ++j)
#pragma unroll
    for (int i = 0; i < TM::W; ++i) {
      const int c = TM::col(j) + i;
      v[j * TM::W + i] = c < n ? __ldg(p + c) : 0.f;
    }
}

// A row to 8 bits (all lanes of every warp call; columns that do not exist hold 0).
template <typename TM>
__device__ __forceinline__ void store_held(const Held8& h, long long row, const float (&v)[TM::E],
                                           int n, bool ok) {
  uint8_t* const codes = h.codes + row * n;
  uint8_t* const scales = h.scales + row * held_blocks(n);
#pragma unroll
  for (int j = 0; j < TM::SLOTS; ++j) {
    const int c = TM::col(j);
    const bool in = ok && c < n;
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
template <typename TM>
__device__ __forceinline__ void load_held(const Held8& h, long long row, float (&v)[TM::E], int n,
                                          bool ok) {
  const uint8_t* const codes = h.codes + row * n;
  const uint8_t* const scales = h.scales + row * held_blocks(n);
  if constexpr (TM::VEC) {
    uint2 r[TM::SLOTS];
    uint32_t byte[TM::SLOTS];
#pragma unroll
    for (int j = 0; j < TM::SLOTS; ++j) {
      const int c = TM::col(j);
      const bool in = ok && c < n;
      r[j] = in ? *reinterpret_cast<const uint2*>(codes + c) : make_uint2(0u, 0u);
      byte[j] = in ? scales[c / kHeldBlock] : 1u;
    }
#pragma unroll
    for (int j = 0; j < TM::SLOTS; ++j) {
      float p[8];
      held_unpack8(r[j], byte[j], p);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[8 * j + i] = p[i];
    }
  } else {
    uint32_t r[TM::SLOTS], byte[TM::SLOTS];
#pragma unroll
    for (int j = 0; j < TM::SLOTS; ++j) {
      const int c = TM::col(j);
      const bool in = ok && c < n;
      r[j] = in ? codes[c] : 0u;
      byte[j] = in ? scales[c / kHeldBlock] : 1u;
    }
#pragma unroll
    for (int j = 0; j < TM::SLOTS; ++j) v[j] = held_values2(r[j]).x * held_up(byte[j]);
  }
}

// The sum over a row's team, in every thread.  `part` holds two rows' partial sums in turn, so that
// one barrier a row is enough.
template <typename TM>
__device__ __forceinline__ float team_sum(float v, float (*part)[16], int turn) {
  constexpr int kLanes = TM::kWarp ? TM::TPR : 32;
#pragma unroll
  for (int d = kLanes / 2; d > 0; d /= 2) v += __shfl_xor_sync(0xffffffffu, v, d);
  if constexpr (!TM::kWarp) {
    constexpr int kWarps = TM::TPR / 32;
    float* const p = part[turn & 1];
    if (threadIdx.x % 32 == 0) p[threadIdx.x / 32] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) v += p[i];
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

// s w rstd rounded once: the product s w is kept in two parts.
__device__ __forceinline__ float normed(float s, float w, float rstd) {
  const float p = s * w;
  const float low = fmaf(s, w, -p);
  return fmaf(p, rstd, low * rstd);
}

template <typename T, typename TM>
__global__ void __launch_bounds__(TM::kThreads) rms_fwd_kernel(const RmsCall q) {
  __shared__ float part[2][16];
  const int n = q.n;
  float w[TM::E];
  load_par<TM>(q.w, w, n);
  int turn = 0;
  for (long long base = static_cast<long long>(blockIdx.x) * TM::kTeams; base < q.rows;
       base += static_cast<long long>(gridDim.x) * TM::kTeams, ++turn) {
    const long long row = base + TM::team();
    const bool ok = row < q.rows;
    Piece<T, TM> x, res;
    x.load(static_cast<const T*>(q.x) + row * q.ldx, n, ok);
    if (q.residual) res.load(static_cast<const T*>(q.residual) + row * q.ldr, n, ok);
    float s[TM::E];
    x.get(s);
    if (q.residual) {
      float r[TM::E];
      res.get(r);
#pragma unroll
      for (int i = 0; i < TM::E; ++i) s[i] = to_f32(from_f32<T>(s[i] + r[i]));
    }
    if (q.s) store_row<TM>(static_cast<T*>(q.s) + row * q.lds, s, n, ok);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < TM::E; ++i) sum = fmaf(s[i], s[i], sum);
    const float rstd = rstd_of(team_sum<TM>(sum, part, turn), n, q.eps);
    if (ok && q.rstd && threadIdx.x % TM::TPR == 0) q.rstd[row] = rstd;
    if (q.s8.codes) store_held<TM>(q.s8, row, s, n, ok);
    if (!q.y && !q.y8.codes) continue;
#pragma unroll
    for (int i = 0; i < TM::E; ++i) s[i] = normed(s[i], w[i], rstd);
    if (q.y) store_row<TM>(static_cast<T*>(q.y) + row * q.ldy, s, n, ok);
    if (q.y8.codes) store_held<TM>(q.y8, row, s, n, ok);
  }
}

template <typename T, typename TM, bool KEPT>
__global__ void __launch_bounds__(TM::kThreads) rms_bwd_kernel(const RmsCall q, float* dw) {
  __shared__ float part[2][16];
  extern __shared__ float sums[];  // [warps][kCols], teams of a warp only
  const int n = q.n;
  float w[TM::E], acc[TM::E];
  load_par<TM>(q.w, w, n);
#pragma unroll
  for (int i = 0; i < TM::E; ++i) acc[i] = 0.f;
  int turn = 0;
  for (long long base = static_cast<long long>(blockIdx.x) * TM::kTeams; base < q.rows;
       base += static_cast<long long>(gridDim.x) * TM::kTeams, ++turn) {
    const long long row = base + TM::team();
    const bool ok = row < q.rows;
    Piece<T, TM> pdy, ps, pds;
    float s[TM::E], dy[TM::E];
    pdy.load(static_cast<const T*>(q.dy) + row * q.lddy, n, ok);
    if (q.ds) pds.load(static_cast<const T*>(q.ds) + row * q.ldds, n, ok);
    if constexpr (KEPT) {
      load_held<TM>(q.s8, row, s, n, ok);
    } else {
      ps.load(static_cast<const T*>(q.x) + row * q.ldx, n, ok);
      ps.get(s);
    }
    pdy.get(dy);
    const float rstd = ok ? q.rstd[row] : 0.f;
    if (q.y) {
      float y[TM::E];
#pragma unroll
      for (int i = 0; i < TM::E; ++i) y[i] = normed(s[i], w[i], rstd);
      store_row<TM>(static_cast<T*>(q.y) + row * q.ldy, y, n, ok);
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
      pds.get(dy);
#pragma unroll
      for (int i = 0; i < TM::E; ++i) s[i] += dy[i];
    }
    store_row<TM>(static_cast<T*>(q.dx) + row * q.lddx, s, n, ok);
  }
  float* const out = dw + static_cast<size_t>(blockIdx.x) * n;
  if constexpr (TM::kWarp) {
#pragma unroll
    for (int i = 0; i < TM::E; ++i)
#pragma unroll
      for (int d = TM::TPR; d < 32; d *= 2) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], d);
    float* const mine = sums + threadIdx.x / 32 * TM::kCols;
    if (threadIdx.x % 32 < TM::TPR) {
#pragma unroll
      for (int j = 0; j < TM::SLOTS; ++j)
#pragma unroll
        for (int i = 0; i < TM::W; ++i) mine[TM::col(j) + i] = acc[j * TM::W + i];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < n; c += TM::kThreads) {
      float v = sums[c];
#pragma unroll
      for (int i = 1; i < TM::kThreads / 32; ++i) v += sums[i * TM::kCols + c];
      out[c] = v;
    }
  } else {
#pragma unroll
    for (int j = 0; j < TM::SLOTS; ++j)
#pragma unroll
      for (int i = 0; i < TM::W; ++i)
        if (TM::col(j) + i < n) out[TM::col(j) + i] = acc[j * TM::W + i];
  }
}

// ---- rows of more than kLongRow columns: a CTA a row, each column by the same thread in both
// passes ----

constexpr int kLongThreads = 512;
using LongTeam = Team<kLongThreads, 1, false>;

template <typename T>
__global__ void __launch_bounds__(kLongThreads) rms_long_fwd_kernel(const RmsCall q) {
  __shared__ float part[2][16];
  const int n = q.n, whole = held_blocks(n) * kHeldBlock;
  int turn = 0;
  for (long long row = blockIdx.x; row < q.rows; row += gridDim.x, ++turn) {
    const T* const x = static_cast<const T*>(q.x) + row * q.ldx;
    const T* const res = q.residual ? static_cast<const T*>(q.residual) + row * q.ldr : nullptr;
    T* const so = q.s ? static_cast<T*>(q.s) + row * q.lds : nullptr;
    // Columns past n (to a whole block) hold 0, so that whole warps pack.
    float sum = 0.f;
    for (int c = threadIdx.x; c < whole; c += kLongThreads) {
      float v = 0.f;
      if (c < n) {
        v = to_f32(x[c]);
        if (res) v = to_f32(from_f32<T>(v + to_f32(res[c])));
        if (so) so[c] = from_f32<T>(v);
      }
      sum = fmaf(v, v, sum);
      if (q.s8.codes) {
        uint32_t byte;
        const uint32_t r = held_pack1(v, byte);
        if (c < n) q.s8.codes[row * n + c] = static_cast<uint8_t>(r);
        if (c % kHeldBlock == 0)
          q.s8.scales[row * held_blocks(n) + c / kHeldBlock] = static_cast<uint8_t>(byte);
      }
    }
    const float rstd = rstd_of(team_sum<LongTeam>(sum, part, turn), n, q.eps);
    if (q.rstd && threadIdx.x == 0) q.rstd[row] = rstd;
    if (!q.y && !q.y8.codes) continue;
    for (int c = threadIdx.x; c < whole; c += kLongThreads) {
      float v = 0.f;
      if (c < n) {
        // s where it was written: x and the residual may have been in its place.
        v = to_f32(so ? so[c] : x[c]);
        if (res && !so) v = to_f32(from_f32<T>(v + to_f32(res[c])));
        v = normed(v, __ldg(q.w + c), rstd);
        if (q.y) static_cast<T*>(q.y)[row * q.ldy + c] = from_f32<T>(v);
      }
      if (q.y8.codes) {
        uint32_t byte;
        const uint32_t r = held_pack1(v, byte);
        if (c < n) q.y8.codes[row * n + c] = static_cast<uint8_t>(r);
        if (c % kHeldBlock == 0)
          q.y8.scales[row * held_blocks(n) + c / kHeldBlock] = static_cast<uint8_t>(byte);
      }
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
  __shared__ float part[2][16];
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

bool aligned(const void* p, long long ld, bool bf16) {
  return !p || (reinterpret_cast<uintptr_t>(p) % (bf16 ? 16 : 32) == 0 && ld % 8 == 0);
}
bool held_aligned(const Held8& h) { return reinterpret_cast<uintptr_t>(h.codes) % 8 == 0; }
bool vectors(const RmsCall& q) {
  return q.n % 8 == 0 && aligned(q.x, q.ldx, q.bf16) && aligned(q.residual, q.ldr, q.bf16) &&
         aligned(q.dy, q.lddy, q.bf16) && aligned(q.ds, q.ldds, q.bf16) &&
         aligned(q.s, q.lds, q.bf16) && aligned(q.y, q.ldy, q.bf16) &&
         aligned(q.dx, q.lddx, q.bf16) && held_aligned(q.y8) && held_aligned(q.s8);
}

// f of the smallest team that covers n columns.
template <typename F>
cudaError_t with_team(int n, bool vec, F&& f) {
  if (vec) {
    if (n <= 32) return f(Team<4, 1, true>{});
    if (n <= 64) return f(Team<8, 1, true>{});
    if (n <= 128) return f(Team<16, 1, true>{});
    if (n <= 256) return f(Team<32, 1, true>{});
    if (n <= 512) return f(Team<32, 2, true>{});
    if (n <= 1024) return f(Team<128, 1, true>{});
    if (n <= 2048) return f(Team<256, 1, true>{});
    if (n <= 4096) return f(Team<512, 1, true>{});
    return f(Team<512, 2, true>{});
  }
  if (n <= 32) return f(Team<32, 1, false>{});
  if (n <= 64) return f(Team<32, 2, false>{});
  if (n <= 128) return f(Team<32, 4, false>{});
  if (n <= 256) return f(Team<32, 8, false>{});
  if (n <= 512) return f(Team<128, 4, false>{});
  if (n <= 1024) return f(Team<128, 8, false>{});
  if (n <= 2048) return f(Team<256, 8, false>{});
  if (n <= 4096) return f(Team<512, 8, false>{});
  return f(Team<512, 16, false>{});
}

int most_ctas(int threads) { return kSms * (2048 / threads); }
int ctas_of(int rows, int teams, int threads) {
  const int need = (rows - 1) / teams + 1, most = most_ctas(threads);
  return need < most ? need : most;
}
// CTAs of the backward pass, and so rows of the partial sums of dw: a row of them costs 8 bytes a
// column to write and read, so a CTA takes four rows of a team at least once all SMs have one.
int bwd_ctas(int rows, int teams, int threads) {
  const int most = kSms * (1024 / threads), need = (rows - 1) / teams + 1;
  const int want = need / 4 > kSms ? need / 4 : kSms;
  return need < want ? need : want < most ? want : most;
}
int long_splits(int rows) { return rows < 64 ? 1 : rows / 64 < 64 ? rows / 64 : 64; }
int partials(int rows, int n, bool vec) {
  if (n > kLongRow) return long_splits(rows);
  int p = 1;
  (void)with_team(n, vec, [&](auto tm) {
    p = bwd_ctas(rows, decltype(tm)::kTeams, decltype(tm)::kThreads);
    return cudaSuccess;
  });
  return p;
}

template <typename T>
cudaError_t fwd(const RmsCall& q, cudaStream_t s) {
  LaunchCfg c;
  c.stream = s;
  if (q.n > kLongRow) {
    c.grid = dim3(ctas_of(q.rows, 1, kLongThreads));
    c.block = dim3(kLongThreads);
    return launch(c, rms_long_fwd_kernel<T>, q);
  }
  return with_team(q.n, vectors(q), [&](auto tm) {
    using TM = decltype(tm);
    c.grid = dim3(ctas_of(q.rows, TM::kTeams, TM::kThreads));
    c.block = dim3(TM::kThreads);
    return launch(c, rms_fwd_kernel<T, TM>, q);
  });
}

template <typename T, bool KEPT>
cudaError_t bwd(const RmsCall& q, float* dw, float* ws, cudaStream_t s) {
  LaunchCfg c;
  c.stream = s;
  const bool vec = vectors(q);
  const int P = partials(q.rows, q.n, vec);
  float* const first = P == 1 ? dw : ws;
  cudaError_t e;
  if (q.n > kLongRow) {
    c.grid = dim3((q.n + 255) / 256, P);
    c.block = dim3(256);
    e = launch(c, rms_long_dw_kernel<T, KEPT>, q, (q.rows - 1) / P + 1, first);
    if (e != cudaSuccess) return e;
    c.grid = dim3(ctas_of(q.rows, 1, kLongThreads));
    c.block = dim3(kLongThreads);
    e = launch(c, rms_long_bwd_kernel<T, KEPT>, q);
  } else {
    e = with_team(q.n, vec, [&](auto tm) {
      using TM = decltype(tm);
      c.grid = dim3(P);
      c.block = dim3(TM::kThreads);
      c.smem = TM::kWarp ? sizeof(float) * TM::kThreads / 32 * TM::kCols : 0;
      return launch(c, rms_bwd_kernel<T, TM, KEPT>, q, first);
    });
  }
  if (e != cudaSuccess || P == 1) return e;
  return reduce_axis0_launch(ws, P, q.n, dw, s, false);
}

}  // namespace

size_t rms_ws_floats(int rows, int n) {
  // Which layout runs depends on the tensors, which the sizing call does not have.
  const int a = partials(rows, n, true), b = partials(rows, n, false), p = a > b ? a : b;
  return p == 1 ? 0 : static_cast<size_t>(p) * n;
}
cudaError_t rms_fwd_launch(const RmsCall& q, cudaStream_t s) {
  return q.bf16 ? fwd<__nv_bfloat16>(q, s) : fwd<float>(q, s);
}
cudaError_t rms_bwd_launch(const RmsCall& q, float* dw, float* ws, cudaStream_t s) {
  if (q.x)
    return q.bf16 ? bwd<__nv_bfloat16, false>(q, dw, ws, s) : bwd<float, false>(q, dw, ws, s);
  return q.bf16 ? bwd<__nv_bfloat16, true>(q, dw, ws, s) : bwd<float, true>(q, dw, ws, s);
}

}  // namespace cfc
