// cfc_trunk_checks.h -- argument checks that the entry points of the trunk operators
// (cfc_trunk_abi.cu) and of the gated block (cfc_gated_abi.cu) share.
#pragma once
#include <cuda_runtime.h>

#include <cmath>
#include <cstddef>
#include <cstdint>

#include "cfc.h"

namespace cfc {
int device_ready();  // cfc_abi.cu

namespace checks {

inline int launched(cudaError_t e) {
  if (e == cudaSuccess) return CFC_OK;
  (void)cudaGetLastError();
  return CFC_ERR_LAUNCH_FAILED;
}

inline bool valid_dtype(int t) { return t == CFC_F32 || t == CFC_BF16; }
inline bool off(const void* p, uintptr_t align) { return (reinterpret_cast<uintptr_t>(p) & (align - 1)) != 0; }
// An activation of this type is misaligned for its element.
inline bool off_act(const void* p, int dtype) { return off(p, dtype == CFC_BF16 ? 2 : 4); }

constexpr int kMaxSequences = 65535;   // a grid dimension
constexpr int kMaxSteps = 1 << 24;
constexpr int kMaxWidth = 1 << 24;     // columns of a row, channels

inline int ws_check(const void* ws, size_t have, size_t need) {
  if (need == 0) return CFC_OK;
  if (!ws) return CFC_ERR_NULL_PTR;
  if (off(ws, 16)) return CFC_ERR_MISALIGNED;
  return have < need ? CFC_ERR_WS_TOO_SMALL : CFC_OK;
}

inline int rows_check(int rows, int n, int dtype) {
  if (rows <= 0 || n <= 0 || n > kMaxWidth) return CFC_ERR_INVALID_DIM;
  return valid_dtype(dtype) ? CFC_OK : CFC_ERR_INVALID_ARG;
}
inline bool bad_eps(float eps) { return !(eps >= 0.f) || std::isinf(eps); }

// A tensor that a call reads or writes, or may do without.  What is read may repeat in memory
// (stride 0); what is written may not.
enum Use { kIn, kInOpt, kOut, kOutOpt };
inline bool required(Use u) { return u == kIn || u == kOut; }
inline bool written(Use u) { return u == kOut || u == kOutOpt; }

struct Rows {
  const void* p;
  long long ld;
  Use use;
};
inline int rows_ok(const Rows* r, int count, int n, int dtype) {
  for (int i = 0; i < count; ++i)
    if (!r[i].p && required(r[i].use)) return CFC_ERR_NULL_PTR;
  for (int i = 0; i < count; ++i)
    if (r[i].p && r[i].ld < (written(r[i].use) ? n : 0)) return CFC_ERR_INVALID_DIM;
  for (int i = 0; i < count; ++i)
    if (off_act(r[i].p, dtype)) return CFC_ERR_MISALIGNED;
  return CFC_OK;
}

struct Seq {  // a [K][B][..] activation and its strides
  const void* p;
  long long t, b;
  Use use;
};
inline int seqs_ok(const Seq* r, int count, int dtype, bool steps = true) {
  for (int i = 0; i < count; ++i)
    if (!r[i].p && required(r[i].use)) return CFC_ERR_NULL_PTR;
  for (int i = 0; i < count; ++i) {
    const long long least = written(r[i].use) ? 1 : 0;
    if (r[i].p && ((steps && r[i].t < least) || r[i].b < least)) return CFC_ERR_INVALID_DIM;
  }
  for (int i = 0; i < count; ++i)
    if (off_act(r[i].p, dtype)) return CFC_ERR_MISALIGNED;
  return CFC_OK;
}

}  // namespace checks
}  // namespace cfc
