// cfc_weights4.cu -- products of a few rows with a matrix of 4-bit weights, y = x W^T with
// W[n][k] = (code[n][k] - 8) scale[n][k / group], and what turns a matrix into that form.
//
// For a few rows the weights' bytes are the work: each is read once and has to become numbers at
// the rate at which memory delivers it.  The products run on the tensor cores (m16n8k16, bf16 with
// fp32 sums): 16 rows of W against 8 columns, of which a row of x takes one in bf16 and three in
// fp32, so that one to eight tokens in bf16, and one or two in fp32, cost the same products.  A code
// minus 8 is exact in bf16, so is x where it is bf16; fp32 x is taken in three bf16 terms, which hold
// all of its 24 bits, and the scale multiplies each group's sum in fp32.  Nothing is rounded before
// the sums.
//
// Measured, groups of 128: 1 x 16384 x 4096 12.3 us, bf16 and fp32 (35 MB of weights, 5.2 us at the
// rate of a copy), 8 rows 14 us, 16 rows 24 us, 32 rows 39 us, 1 x 4096 x 16384 14 us, 16 x 8192 x
// 8192 25 us, 1 x 4096 x 4096 6.2 us.  One row is bound by latency, of the launch and of the first
// weights, which a warp's four to eight tiles do not hide, and by instructions: 2.6 for a code, 4.6 us
// at one a cycle and scheduler (it issues 1.9 of 4 a cycle); the tensor cores are busy for 1.8 us of
// it.  32 rows wait for weights, of which 16 warps an SM (their sums take 128 registers) have too few
// on their way, and bring in x anew in every CTA (1.0 of 4 instructions a cycle, 442 for a tile with
// its part of x).
//
// Laid-out weights: tiles of 16 rows x 128 columns of 1024 bytes, one after another along a row of
// tiles.  In a tile lane 4 g + t of a warp owns rows g and g + 8 (one 16-byte load each) and of
// every 32 columns the eight from 8 t on, in one 32-bit word: columns j and j + 4 of the eight are
// 16 bits apart, a pair as the tensor cores take it, and the order of columns within a product is
// free as long as x follows it.  Scales follow the codes, 16 rows of a group together, rows g and g + 8
// side by side.
#include "cfc_gated_kernels.h"
#include "cfc_launch.cuh"
#include "cfc_trunk.cuh"

namespace cfc {
namespace {

constexpr int kTileN = 16, kTileK = 128, kTileBytes = kTileN * kTileK / 2;
// Tiles whose weights a warp has on their way together: two, so that four CTAs fit an SM (16384 x 4096,
// one row of bf16: 12.5 us; four tiles and three CTAs 13.9, four and four 15.5, which spills).
constexpr int kAhead = 2;

// Shared memory for a chunk of x.  The warps' sums, at most 512 threads x 4 of 16 bytes, fit it too.
constexpr int kChunkBytes = 64 * 1024;

struct Shape4 {
  int tn, tk, groups;   // tiles along N and K, groups of a row (padded to whole tiles)
  size_t codes_bytes;
};
__host__ __device__ inline Shape4 shape4(int N, int K, int group) {
  Shape4 s;
  s.tn = (N - 1) / kTileN + 1;
  s.tk = (K - 1) / kTileK + 1;
  s.groups = s.tk * (kTileK / group);
  s.codes_bytes = static_cast<size_t>(s.tn) * s.tk * kTileBytes;
  return s;
}

// ---- to 4 bits: a warp a group of a row ----

template <typename T>
__global__ void __launch_bounds__(256) quantize4_kernel(const Weights4Call q, int groups) {
  const long long at = static_cast<long long>(blockIdx.x) * 8 + threadIdx.x / 32;
  if (at >= static_cast<long long>(q.N) * groups) return;
  const int lane = threadIdx.x % 32, n = static_cast<int>(at / groups);
  const int g = static_cast<int>(at - static_cast<long long>(n) * groups), k0 = g * q.group;
  const T* const row = static_cast<const T*>(q.x) + n * q.ldx;
  uint32_t most = 0u;
  for (int k = k0 + lane; k < min(q.K, k0 + q.group); k += 32)
    most = max(most, __float_as_uint(to_f32(row[k])) & 0x7fffffffu);
  most = __reduce_max_sync(0xffffffffu, most);
  // The largest magnitude becomes 7 steps, up to the scale's rounding; of an infinity NaN, as of a NaN.
  if (most == 0x7f800000u) most = 0x7fffffffu;
  const __nv_bfloat16 held = __float2bfloat16_rn(__uint_as_float(most) / 7.f);
  const float scale = __bfloat162float(held);
  if (lane == 0) q.scales_out[at] = __bfloat16_as_ushort(held);
  const size_t pitch = (static_cast<size_t>(q.K) + 1) / 2;
  for (int k = k0 + 2 * lane; k < min(q.K, k0 + q.group); k += 64) {
    uint32_t byte = 0u;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float c = 0.f;  // the code of a zero weight, also behind the last column
      if (k + j < q.K && scale > 0.f)
        c = fminf(fmaxf(rintf(to_f32(row[k + j]) / scale), -8.f), 7.f);
      byte |= static_cast<uint32_t>(static_cast<int>(c) + 8) << (4 * j);
    }
    q.codes_out[n * pitch + k / 2] = static_cast<uint8_t>(byte);
  }
}

// ---- into the order in which the products read them ----

__global__ void __launch_bounds__(256) lay_out4_kernel(const Weights4Call q) {
  const Shape4 s = shape4(q.N, q.K, q.group);
  const long long at = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  const long long words = static_cast<long long>(s.tn) * s.tk * 64;  // 16-byte words
  const size_t pitch = (static_cast<size_t>(q.K) + 1) / 2;
  if (at < words) {
    const long long tile = at / 64;
    const int in = static_cast<int>(at % 64), r = in / 32, lane = in % 32;
    const int kb = static_cast<int>(tile % s.tk);
    const int n = static_cast<int>(tile / s.tk) * kTileN + lane / 4 + 8 * r;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = kb * kTileK + 32 * j + 8 * (lane % 4);
      w[j] = 0x88888888u;
      if (n >= q.N) continue;
      const uint8_t* const from = q.codes + n * pitch;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int kk = k + 2 * i;
        if (kk >= q.K) continue;
        uint32_t byte = from[kk / 2];
        if (kk + 1 >= q.K) byte = (byte & 15u) | 0x80u;
        w[j] = (w[j] & ~(0xffu << (8 * i))) | byte << (8 * i);
      }
    }
    reinterpret_cast<uint4*>(q.laid_out)[at] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  const long long scales = static_cast<long long>(s.tn) * s.groups * kTileN;
  const int have = (q.K - 1) / q.group + 1;
  uint16_t* const to = reinterpret_cast<uint16_t*>(q.laid_out + s.codes_bytes);
  for (long long i = at; i < scales; i += static_cast<long long>(gridDim.x) * 256) {
    const int in = static_cast<int>(i % kTileN);
    const long long rest = i / kTileN;
    const int g = static_cast<int>(rest % s.groups);
    const int n = static_cast<int>(rest / s.groups) * kTileN + in / 2 + in % 2 * 8;
    to[i] = n < q.N && g < have ? q.scales[static_cast<size_t>(n) * have + g] : uint16_t(0);
  }
}

// ---- the products ----

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same onto sums of 0.
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint4 ld_shared(uint32_t at) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(at));
  return r;
}

// Weights are read once: they do not stay in L1, where x is.
__device__ __forceinline__ uint4 ld_once(const uint4* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

// Codes j and j + 4 of a word, minus 8, as a pair of bf16.  A bf16 number from 128 to 256 has seven bits
// behind the leading one, worth 64 to 1: with a code in the last four of 128's it is 128 + code, and the
// difference from 136 is exact.
template <int J>
__device__ __forceinline__ uint32_t codes_bf16(uint32_t word) {
  constexpr uint32_t kTwo = 0x00010001u;  // in both halves
  constexpr uint32_t kCode = 15u * kTwo, k128 = 0x4300u * kTwo, k136 = 0x4308u * kTwo;
  uint32_t v, r;
  // (word >> 4 J & kCode) | k128 in one instruction behind the shift.
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(v) : "r"(word >> (4 * J)), "r"(kCode), "r"(k128));
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(k136));
  return r;
}

// Eight neighbouring values of a row of x in the order of the codes' pairs (0 4, 1 5, 2 6, 3 7), in
// as many bf16 terms as their type needs.
template <typename T>
struct XPiece;
template <>
struct XPiece<__nv_bfloat16> {
  static constexpr int kTerms = 1;
  static __device__ __forceinline__ void split(const Raw8<__nv_bfloat16>& r, uint4 (&term)[1]) {
    term[0] = make_uint4(__byte_perm(r.w[0], r.w[2], 0x5410), __byte_perm(r.w[0], r.w[2], 0x7632),
                         __byte_perm(r.w[1], r.w[3], 0x5410), __byte_perm(r.w[1], r.w[3], 0x7632));
  }
};
template <>
struct XPiece<float> {
  static constexpr int kTerms = 3;
  // A term is the upper half of what is left, eight bits of it, so that three of them are all 24 and
  // every difference is exact.  Of an infinity nothing is left; of a NaN whose upper half alone would be
  // an infinity the difference is one in every half.
  static __device__ __forceinline__ float rest(float a) {
    const float r = a - __uint_as_float(__float_as_uint(a) & 0xffff0000u);
    return (__float_as_uint(a) & 0x7fffffffu) == 0x7f800000u ? 0.f : r;
  }
  static __device__ __forceinline__ void split(const Raw8<float>& r, uint4 (&term)[3]) {
    float v[8];
    r.get(v);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = __byte_perm(__float_as_uint(v[j]), __float_as_uint(v[j + 4]), 0x7632);
        v[j] = rest(v[j]);
        v[j + 4] = rest(v[j + 4]);
      }
      term[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
};

// How a CTA's warps are spread: over 1 << `rows` tiles of 16 rows of W, and `deep` of them over K.
struct Spread {
  int rows, deep;
  int m;            // rows of x of a CTA, at most
  int chunk;        // tiles along K whose part of x is in shared memory at a time
  bool vec;         // x is read 8 values at a time
};

// A CTA: its tiles of W against up to 8 NT columns of x, a column being a term of a row of x, so that
// two rows of fp32 and eight of bf16 cost the same.  x waits in shared memory, split and in the order
// in which lanes take it (16 bytes for a lane's part of a product), so that the loop over the weights is
// little but turning codes into numbers; what a code becomes serves all columns.  Columns that there are
// not are computed from the last one and dropped.  A warp has kAhead tiles of weights on their way
// together, the first of them while x is brought in.
template <typename T, int GROUP, int NT>
__global__ void __launch_bounds__(512, NT == 1 ? 2 : 1)
    matvec4_kernel(const Weights4Call q, const Spread sp) {
  extern __shared__ uint4 xs[];  // [tiles of a chunk][4][columns][4]; later the warps' sums
  using X = XPiece<T>;
  constexpr int kTerms = X::kTerms, kPer = kTileK / GROUP;  // groups of a tile
  const int tk = (q.K - 1) / kTileK + 1, tn = (q.N - 1) / kTileN + 1;
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32, g = lane / 4, t = lane % 4;
  const int m0 = blockIdx.y * sp.m, mm = min(q.M - m0, sp.m), cols = mm * kTerms;
  const int deep = w >> sp.rows;
  // Beyond the last tile of rows the last one is computed again, and dropped.
  const int row_tile = min((static_cast<int>(blockIdx.x) << sp.rows) + (w & ((1 << sp.rows) - 1)), tn - 1);
  const size_t tile0 = static_cast<size_t>(row_tile) * tk + deep;
  const uint4* codes = reinterpret_cast<const uint4*>(q.weights) + tile0 * 64 + lane;
  const uint32_t* scales = reinterpret_cast<const uint32_t*>(
                               q.weights + static_cast<size_t>(tn) * tk * kTileBytes) +
                           tile0 * (kPer * kTileN / 2) + g;
  const int code_step = sp.deep * 64, scale_step = sp.deep * (kPer * kTileN / 2);
  const uint32_t step = 64 * cols;  // bytes of 32 values of K in xs
  uint32_t from[NT];                // this lane's column
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
    from[nt] = smem_addr(xs) + (min(8 * nt + g, cols - 1) * 4 + t) * 16 + deep * 4 * step;
  float acc[NT][4] = {};
  uint4 lo[kAhead], hi[kAhead];
  uint32_t sc[kAhead][kPer];
  auto fetch = [&](int a) {  // the warp's next tile
    lo[a] = ld_once(codes);
    hi[a] = ld_once(codes + 32);
#pragma unroll
    for (int i = 0; i < kPer; ++i) sc[a][i] = __ldg(scales + i * (kTileN / 2));
    codes += code_step;
    scales += scale_step;
  };
  // Tiles of this warp in a chunk that begins at c0 (a multiple of `deep`, as chunks are).
  auto tiles = [&](int c0) {
    return (min(sp.chunk, tk - c0) - deep + sp.deep - 1) / sp.deep;
  };
  for (int c0 = 0; c0 < tk; c0 += sp.chunk) {
    int left = tiles(c0);
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
      if (a < left) fetch(a);
    if (c0 > 0) __syncthreads();
    // x of the chunk, in pieces of 8 values: 16 threads a row's part of a tile.
    const unsigned count = min(sp.chunk, tk - c0) * mm;
    for (unsigned i = threadIdx.x / 16; i < count; i += blockDim.x / 16) {
      const unsigned kb = mm == 1 ? i : i / mm, m = i - kb * mm, p = threadIdx.x % 16;
      const int k = (c0 + kb) * kTileK + 8 * p;
      const T* const x = static_cast<const T*>(q.x) + static_cast<long long>(m0 + m) * q.ldx + k;
      Raw8<T> raw;
      raw.clear();
      if (sp.vec && k + 8 <= q.K) {
        raw.load(x);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (k + j < q.K) raw.set(j, x[j]);
      }
      uint4 term[kTerms];
      X::split(raw, term);
#pragma unroll
      for (int j = 0; j < kTerms; ++j)
        xs[((4 * kb + p / 4) * cols + m * kTerms + j) * 4 + p % 4] = term[j];
    }
    __syncthreads();
    uint32_t at = 0;
    while (left > 0) {
#pragma unroll
      for (int a = 0; a < kAhead; ++a, at += 4 * sp.deep * step) {
        if (a >= left) break;
        const uint32_t wa[4] = {lo[a].x, lo[a].y, lo[a].z, lo[a].w};
        const uint32_t wb[4] = {hi[a].x, hi[a].y, hi[a].z, hi[a].w};
        float part[NT][4];
        uint32_t xk = at;
#pragma unroll
        for (int s = 0; s < 4; ++s, xk += step) {
          const uint32_t a0[4] = {codes_bf16<0>(wa[s]), codes_bf16<0>(wb[s]), codes_bf16<1>(wa[s]),
                                  codes_bf16<1>(wb[s])};
          const uint32_t a1[4] = {codes_bf16<2>(wa[s]), codes_bf16<2>(wb[s]), codes_bf16<3>(wa[s]),
                                  codes_bf16<3>(wb[s])};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint4 b = ld_shared(from[nt] + xk);
            if (s * 32 % GROUP == 0) mma_first(part[nt], a0, b.x, b.y);
            else mma_bf16(part[nt], a0, b.x, b.y);
            mma_bf16(part[nt], a1, b.z, b.w);
          }
          if ((s + 1) * 32 % GROUP == 0) {
            const uint32_t two = sc[a][s * 32 / GROUP];
            const float s0 = bf16_lo_f32(two), s1 = bf16_hi_f32(two);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              acc[nt][0] = fmaf(part[nt][0], s0, acc[nt][0]);
              acc[nt][1] = fmaf(part[nt][1], s0, acc[nt][1]);
              acc[nt][2] = fmaf(part[nt][2], s1, acc[nt][2]);
              acc[nt][3] = fmaf(part[nt][3], s1, acc[nt][3]);
            }
          }
        }
        if (a + kAhead < left) fetch(a);
      }
      left -= kAhead;
    }
  }
  __syncthreads();
  float4* const sums = reinterpret_cast<float4*>(xs);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
    sums[(w * NT + nt) * 32 + lane] = make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
  __syncthreads();
  // Sum i of lane 4 g + t is row g + 8 (i / 2) of the tile and column 2 t + i % 2.
  const float* const all = reinterpret_cast<const float*>(sums);
  for (int at = threadIdx.x; at < mm << (4 + sp.rows); at += blockDim.x) {
    const int row = at % 16, m = at >> (4 + sp.rows), r = (at >> 4) - (m << sp.rows);
    const int n = ((static_cast<int>(blockIdx.x) << sp.rows) + r) * kTileN + row;
    if (n >= q.N) continue;
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kTerms; ++i) {
      const int col = m * kTerms + i, of = 4 * (row % 8) + col % 8 / 2, j = 2 * (row / 8) + col % 2;
      const float* p = all + ((r * NT + col / 8) * 32 + of) * 4 + j;
#pragma unroll 4
      for (int k = 0; k < sp.deep; ++k, p += (NT * 128) << sp.rows) v += *p;
    }
    static_cast<T*>(q.y)[static_cast<long long>(m0 + m) * q.ldy + n] = from_f32<T>(v);
  }
}

template <typename T, int GROUP>
cudaError_t matvec(const Weights4Call& q, cudaStream_t s) {
  constexpr int kTerms = XPiece<T>::kTerms;
  const Shape4 sh = shape4(q.N, q.K, GROUP);
  const int nt = q.M * kTerms <= 8 ? 1 : q.M * kTerms <= 16 ? 2 : 4;
  Spread sp;
  sp.vec = reinterpret_cast<uintptr_t>(q.x) % (q.bf16 ? 16 : 32) == 0 && q.ldx % 8 == 0;
  sp.m = 8 * nt / kTerms;
  if (q.M < sp.m) sp.m = q.M;
  // More tiles of rows at a time share what a CTA reads of x, as long as half of the SMs have a CTA:
  // with four tiles 16 x 8192 x 8192 takes 25 us (two 37 us, one 53 us) and 8 x 16384 x 4096 14 us (18 and
  // 27 us), with two 8 x 4096 x 4096 8.8 us (four 10.3 us).  One row of x has little to share (1 x 4096
  // x 16384 14.5 us, with two 20 us).
  sp.rows = sp.m * kTerms <= 2 ? 0 : 2;
  while (sp.rows > 0 && sh.tn >> sp.rows < 152 / 2) --sp.rows;
  // Sixteen warps where the GPU holds all CTAs at a time (8 x 16384 x 4096 14 us, eight 17 us), else eight
  // (32 x 16384 x 4096 39 us, sixteen 42.5 us).  In one column of tiles eight, whose parts of x fit shared
  // memory for any number of rows.
  const long long ctas = ((sh.tn - 1ll >> sp.rows) + 1) * ((q.M - 1) / sp.m + 1);
  sp.deep = sp.rows > 0 && ctas <= (nt == 1 ? 304 : 152) ? 16 >> sp.rows : 8 >> sp.rows;
  // Shorter columns of warps where the CTAs are more than the GPU holds at a time, so that a warp has
  // more tiles for what it does once (1 x 12288 x 4096 10.3 us, always eight 11.6 us; 65536 x 1024 12.4
  // and 18.2 us); where they are not, all eight (1 x 8192 x 4096 8.6 us, four 10.2 us).
  while (sp.rows == 0 && sp.deep > 2 && sh.tn > 152 * 32 / sp.deep) sp.deep /= 2;
  if (sh.tk < sp.deep) sp.deep = sh.tk;
  const int bytes = 256 * sp.m * kTerms;  // of x for a tile along K; at most 8 KB,
                                              // so a chunk has eight tiles, and deep is at most 8
  sp.chunk = kChunkBytes / bytes / sp.deep * sp.deep;
  if (sp.chunk > sh.tk) sp.chunk = sh.tk;
  LaunchCfg c;
  c.grid = dim3((sh.tn - 1 >> sp.rows) + 1, (q.M - 1) / sp.m + 1);
  c.block = dim3(32 * (sp.deep << sp.rows));
  const size_t sums = sizeof(float4) * c.block.x * nt, xs = static_cast<size_t>(sp.chunk) * bytes;
  c.smem = sums > xs ? sums : xs;
  c.stream = s;
  auto run = [&](auto* kern) {
    const cudaError_t e = allow_smem(kern, c.smem, kChunkBytes);
    return e == cudaSuccess ? launch(c, kern, q, sp) : e;
  };
  if (nt == 1) return run(matvec4_kernel<T, GROUP, 1>);
  if (nt == 2) return run(matvec4_kernel<T, GROUP, 2>);
  return run(matvec4_kernel<T, GROUP, 4>);
}
template <typename T>
cudaError_t by_group(const Weights4Call& q, cudaStream_t s) {
  if (q.group == 32) return matvec<T, 32>(q, s);
  if (q.group == 64) return matvec<T, 64>(q, s);
  return matvec<T, 128>(q, s);
}

}  // namespace

size_t weights4_bytes(int N, int K, int group) {
  const Shape4 s = shape4(N, K, group);
  return s.codes_bytes + static_cast<size_t>(s.tn) * s.groups * kTileN * 2;
}
cudaError_t weights4_quantize_launch(const Weights4Call& q, cudaStream_t s) {
  const int groups = (q.K - 1) / q.group + 1;
  LaunchCfg c;
  c.grid = dim3(static_cast<unsigned>((static_cast<long long>(q.N) * groups + 7) / 8));
  c.block = dim3(256);
  c.stream = s;
  return q.bf16 ? launch(c, quantize4_kernel<__nv_bfloat16>, q, groups)
                : launch(c, quantize4_kernel<float>, q, groups);
}
cudaError_t weights4_lay_out_launch(const Weights4Call& q, cudaStream_t s) {
  const Shape4 sh = shape4(q.N, q.K, q.group);
  LaunchCfg c;
  c.grid = dim3(static_cast<unsigned>((static_cast<long long>(sh.tn) * sh.tk * 64 + 255) / 256));
  c.block = dim3(256);
  c.stream = s;
  return launch(c, lay_out4_kernel, q);
}
cudaError_t weights4_matvec_launch(const Weights4Call& q, cudaStream_t s) {
  return q.bf16 ? by_group<__nv_bfloat16>(q, s) : by_group<float>(q, s);
}

}  // namespace cfc
