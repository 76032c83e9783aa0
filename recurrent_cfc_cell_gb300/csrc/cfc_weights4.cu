// cfc_weights4.cu -- products of a few rows with a matrix of 4-bit weights, y = x W^T with
// W[n][k] = (code[n][k] - 8) scale[n][k / group], and what turns a matrix into that form.
//
// For a few rows the weights' bytes are the work: each is read once and has to become numbers at
// the rate at which memory delivers it.  The products run on the tensor cores (m16n8k16, bf16 with
// fp32 sums): 16 rows of W against up to 8 rows of x, so that one to eight tokens cost the same.  A
// code minus 8 is exact in bf16, so is x where it is bf16; fp32 x is taken in three bf16 terms,
// which hold all of its 24 bits, and the scale multiplies each group's sum in fp32.  Nothing is
// rounded before the sums.
//
// Laid-out weights: tiles of 16 rows x 128 columns of 1024 bytes, one after another along a row of
// tiles.  In a tile lane 4 g + t of a warp owns rows g and g + 8 (one 16-byte load each) and of
// every 32 columns the eight from 8 t on, in one 32-bit word: columns j and j + 4 of the eight are
// 16 bits apart, a pair as the tensor cores take it, and the order of columns within a product is
// free as long as x follows it.  Scales follow the codes, 16 rows of a group together.
#include "cfc_gated_kernels.h"
#include "cfc_launch.cuh"
#include "cfc_trunk.cuh"

namespace cfc {
namespace {

constexpr int kTileN = 16, kTileK = 128, kTileBytes = kTileN * kTileK / 2;
constexpr int kWarps = 8;

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
  // The largest magnitude becomes 7 steps, up to the scale's rounding.
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
    const int n = static_cast<int>(rest / s.groups) * kTileN + in;
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

// Codes j and j + 4 of a word, minus 8, as a pair of bf16: 0x4300 is 128, whose last place is 1.
template <int J>
__device__ __forceinline__ uint32_t codes_bf16(uint32_t word) {
  const uint32_t v = ((word >> (4 * J)) & 0x000f000fu) | 0x43004300u;
  const __nv_bfloat162 r =
      __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), __float2bfloat162_rn(136.f));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Eight neighbouring values of a row of x in the order of the codes' pairs (0 4, 1 5, 2 6, 3 7), in
// as many bf16 terms as their type needs.  Columns from K on are not read.
template <typename T>
struct XPiece;
template <>
struct XPiece<__nv_bfloat16> {
  static constexpr int kTerms = 1;
  uint32_t term[1][4];
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int left, bool vec, bool in) {
    Raw8<__nv_bfloat16> raw;
    raw.clear();
    if (in && left > 0) {
      if (vec && left >= 8) {
        raw.load(p);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < left) raw.set(j, p[j]);
      }
    }
    term[0][0] = __byte_perm(raw.w[0], raw.w[2], 0x5410);
    term[0][1] = __byte_perm(raw.w[0], raw.w[2], 0x7632);
    term[0][2] = __byte_perm(raw.w[1], raw.w[3], 0x5410);
    term[0][3] = __byte_perm(raw.w[1], raw.w[3], 0x7632);
  }
};
template <>
struct XPiece<float> {
  static constexpr int kTerms = 3;
  uint32_t term[3][4];
  static __device__ __forceinline__ float rest(float a) {
    const float r = a - __uint_as_float(__float_as_uint(a) & 0xffff0000u);
    return r == r ? r : 0.f;
  }
  __device__ __forceinline__ void load(const float* p, int left, bool vec, bool in) {
    Raw8<float> raw;
    raw.clear();
    if (in && left > 0) {
      if (vec && left >= 8) {
        raw.load(p);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < left) raw.set(j, p[j]);
      }
    }
    // A term is the upper half of what is left, eight bits of it, so that three of them are all 24
    // and every difference is exact (of an infinity it is not a number: nothing is left).
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float a = raw.v[j], b = raw.v[j + 4];
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        term[i][j] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
        a = rest(a);
        b = rest(b);
      }
    }
  }
};

// A CTA: 16 rows of W against 8 rows of x; its warps take the tiles along K in turn.
template <typename T, int GROUP>
__global__ void __launch_bounds__(32 * kWarps) matvec4_kernel(const Weights4Call q, bool vec) {
  __shared__ float sums[kWarps][32][4];
  const Shape4 sh = shape4(q.N, q.K, GROUP);
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32, g = lane / 4, t = lane % 4;
  const int m = blockIdx.y * 8 + g;
  const T* const x = static_cast<const T*>(q.x) + static_cast<long long>(m) * q.ldx;
  const size_t tile0 = static_cast<size_t>(blockIdx.x) * sh.tk;
  const uint4* const codes = reinterpret_cast<const uint4*>(q.weights) + tile0 * 64 + lane;
  constexpr int kPer = kTileK / GROUP;  // groups of a tile
  const uint16_t* const scales = reinterpret_cast<const uint16_t*>(q.weights + sh.codes_bytes) +
                                 tile0 * (kPer * kTileN) + g;
  float acc[4] = {};
  for (int kb = w; kb < sh.tk; kb += kWarps) {
    const uint4 lo = __ldg(codes + static_cast<size_t>(kb) * 64);
    const uint4 hi = __ldg(codes + static_cast<size_t>(kb) * 64 + 32);
    const uint32_t wa[4] = {lo.x, lo.y, lo.z, lo.w}, wb[4] = {hi.x, hi.y, hi.z, hi.w};
    float part[4] = {};
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      XPiece<T> xp;
      const int k = kb * kTileK + 32 * s + 8 * t;
      xp.load(x + k, q.K - k, vec, m < q.M);
      const uint32_t a0[4] = {codes_bf16<0>(wa[s]), codes_bf16<0>(wb[s]), codes_bf16<1>(wa[s]),
                              codes_bf16<1>(wb[s])};
      const uint32_t a1[4] = {codes_bf16<2>(wa[s]), codes_bf16<2>(wb[s]), codes_bf16<3>(wa[s]),
                              codes_bf16<3>(wb[s])};
#pragma unroll
      for (int i = 0; i < XPiece<T>::kTerms; ++i) {
        mma_bf16(part, a0, xp.term[i][0], xp.term[i][1]);
        mma_bf16(part, a1, xp.term[i][2], xp.term[i][3]);
      }
      if ((s + 1) * 32 % GROUP == 0) {
        const uint16_t* const sc = scales + (static_cast<size_t>(kb) * kPer + s * 32 / GROUP) * kTileN;
        const float s0 = __uint_as_float(static_cast<uint32_t>(__ldg(sc)) << 16);
        const float s1 = __uint_as_float(static_cast<uint32_t>(__ldg(sc + 8)) << 16);
        acc[0] = fmaf(part[0], s0, acc[0]);
        acc[1] = fmaf(part[1], s0, acc[1]);
        acc[2] = fmaf(part[2], s1, acc[2]);
        acc[3] = fmaf(part[3], s1, acc[3]);
        part[0] = part[1] = part[2] = part[3] = 0.f;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) sums[w][lane][i] = acc[i];
  __syncthreads();
  // Sum i of lane 4 g + t is row g + 8 (i / 2) of the tile and row 2 t + i % 2 of x.
  if (threadIdx.x >= 128) return;
  const int row = threadIdx.x % 16, col = threadIdx.x / 16;
  const int from = 4 * (row % 8) + col / 2, i = 2 * (row / 8) + col % 2;
  float v = 0.f;
#pragma unroll
  for (int k = 0; k < kWarps; ++k) v += sums[k][from][i];
  const int n = blockIdx.x * kTileN + row, mm = blockIdx.y * 8 + col;
  if (n < q.N && mm < q.M)
    static_cast<T*>(q.y)[static_cast<long long>(mm) * q.ldy + n] = from_f32<T>(v);
}

template <typename T>
cudaError_t matvec(const Weights4Call& q, cudaStream_t s) {
  const Shape4 sh = shape4(q.N, q.K, q.group);
  const bool vec = reinterpret_cast<uintptr_t>(q.x) % (q.bf16 ? 16 : 32) == 0 && q.ldx % 8 == 0;
  LaunchCfg c;
  c.grid = dim3(sh.tn, (q.M - 1) / 8 + 1);
  c.block = dim3(32 * kWarps);
  c.stream = s;
  if (q.group == 32) return launch(c, matvec4_kernel<T, 32>, q, vec);
  if (q.group == 64) return launch(c, matvec4_kernel<T, 64>, q, vec);
  return launch(c, matvec4_kernel<T, 128>, q, vec);
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
  return q.bf16 ? matvec<__nv_bfloat16>(q, s) : matvec<float>(q, s);
}

}  // namespace cfc
