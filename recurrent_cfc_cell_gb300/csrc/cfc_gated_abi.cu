// cfc_gated_abi.cu -- extern "C" entry points of the gated block's operators (root-mean-square norm,
// values in 8 bits, gated linear recurrence, products with 4-bit weights): argument checks on the
// host, then the launches.  Nothing is allocated, nothing synchronises, and a refused call has
// enqueued nothing.
#include "cfc.h"
#include "cfc_gated_kernels.h"
#include "cfc_held8.cuh"
#include "cfc_trunk_checks.h"

using namespace cfc::checks;

namespace {

cudaStream_t on(cfc_stream_t s) { return static_cast<cudaStream_t>(s); }

cfc::Held8 held(const cfc_held8* h) {
  return h ? cfc::Held8{static_cast<uint8_t*>(h->codes), static_cast<uint8_t*>(h->scales)}
           : cfc::Held8{};
}
int held_ok(const cfc_held8* h) { return h->codes && h->scales ? CFC_OK : CFC_ERR_NULL_PTR; }

int pack_call(const void* act, long long ld, Use use, int rows, int n, int dtype,
              const cfc_held8* h, cfc::Held8Call* q) {
  int rc = rows_check(rows, n, dtype);
  if (rc != CFC_OK) return rc;
  const Rows r[] = {{act, ld, use}};
  rc = rows_ok(r, 1, n, dtype);
  if (rc != CFC_OK) return rc;
  if (!h) return CFC_ERR_NULL_PTR;
  rc = held_ok(h);
  if (rc == CFC_OK) rc = cfc::device_ready();
  if (rc != CFC_OK) return rc;
  q->rows = rows; q->n = n; q->bf16 = dtype == CFC_BF16;
  q->held = held(h);
  return CFC_OK;
}

int gated_check(int B, int K, int D, int dtype, bool steps) {
  if (B <= 0 || B > kMaxSequences || D <= 0 || D > kMaxWidth) return CFC_ERR_INVALID_DIM;
  if (steps && (K <= 0 || K > kMaxSteps)) return CFC_ERR_INVALID_DIM;
  return valid_dtype(dtype) ? CFC_OK : CFC_ERR_INVALID_ARG;
}

// Fills the common part of a call; the argument errors of the struct itself.  `inputs`: x, f and z
// are read.
int gated_call(const cfc_gated_args* a, bool steps, bool inputs, cfc::GatedCall* q) {
  if (!a) return CFC_ERR_NULL_PTR;
  int rc = gated_check(a->B, a->K, a->D, a->dtype, steps);
  if (rc != CFC_OK) return rc;
  if (inputs) {
    const Seq in[] = {{a->x, a->x_t, a->x_b, kIn}, {a->f, a->f_t, a->f_b, kIn},
                      {a->z, a->z_t, a->z_b, kInOpt}};
    rc = seqs_ok(in, 3, a->dtype, steps);
    if (rc != CFC_OK) return rc;
    q->x = a->x; q->x_t = a->x_t; q->x_b = a->x_b;
    q->f = a->f; q->f_t = a->f_t; q->f_b = a->f_b;
    q->z = a->z; q->z_t = a->z_t; q->z_b = a->z_b;
  }
  if (off(a->bias, 4) || off(a->h0, 4) || off(a->lengths, 4)) return CFC_ERR_MISALIGNED;
  q->B = a->B; q->K = a->K; q->D = a->D;
  q->bf16 = a->dtype == CFC_BF16;
  q->has_z = a->z != nullptr;
  q->lengths = a->lengths;
  q->bias = a->bias; q->h0 = a->h0;
  return CFC_OK;
}

// What is kept in 8 bits; `read`: by the backward pass, which has no other word of z then.
int kept_call(const cfc_gated_kept* kept, bool read, cfc::GatedCall* q) {
  q->keep = kept != nullptr;
  if (!kept) return CFC_OK;
  if (read) q->has_z = kept->z.codes != nullptr;
  int rc = held_ok(&kept->x);
  if (rc == CFC_OK) rc = held_ok(&kept->f);
  if (rc == CFC_OK && q->has_z) rc = held_ok(&kept->z);
  if (rc != CFC_OK) return rc;
  q->x8 = held(&kept->x);
  q->f8 = held(&kept->f);
  if (q->has_z) q->z8 = held(&kept->z);
  return CFC_OK;
}

size_t gated_bytes(int B, int K, int D, bool backward) {
  return sizeof(float) * (cfc::gated_segments_floats(B, K, D, backward) +
                          (backward ? cfc::gated_partials_floats(B, K, D) : 0));
}

int weights4_check(int N, int K, int group) {
  if (N <= 0 || K <= 0 || N > kMaxWidth || K > kMaxWidth ||
      static_cast<long long>(N) * K > 1ll << 36)
    return CFC_ERR_INVALID_DIM;
  return group == 32 || group == 64 || group == 128 ? CFC_OK : CFC_ERR_INVALID_ARG;
}

}  // namespace

extern "C" {

int cfc_pack8(const void* x, long long ldx, int rows, int n, int dtype, const cfc_held8* h,
              cfc_stream_t stream) {
  cfc::Held8Call q{};
  const int rc = pack_call(x, ldx, kIn, rows, n, dtype, h, &q);
  if (rc != CFC_OK) return rc;
  q.x = x; q.ldx = ldx;
  return launched(cfc::pack8_launch(q, on(stream)));
}

int cfc_unpack8(const cfc_held8* h, int rows, int n, int dtype, void* y, long long ldy,
                cfc_stream_t stream) {
  cfc::Held8Call q{};
  const int rc = pack_call(y, ldy, kOut, rows, n, dtype, h, &q);
  if (rc != CFC_OK) return rc;
  q.y = y; q.ldy = ldy;
  return launched(cfc::unpack8_launch(q, on(stream)));
}

int cfc_rmsnorm_forward(const cfc_rmsnorm_args* a, void* s, long long lds, void* y, long long ldy,
                        const cfc_held8* s8, const cfc_held8* y8, float* rstd,
                        cfc_stream_t stream) {
  if (!a) return CFC_ERR_NULL_PTR;
  int rc = rows_check(a->rows, a->n, a->dtype);
  if (rc != CFC_OK) return rc;
  const Rows r[] = {{a->x, a->ldx, kIn}, {a->residual, a->ldr, kInOpt}, {s, lds, kOutOpt},
                    {y, ldy, kOutOpt}};
  rc = rows_ok(r, 4, a->n, a->dtype);
  if (rc != CFC_OK) return rc;
  if (!a->w) return CFC_ERR_NULL_PTR;
  if (s8) rc = held_ok(s8);
  if (rc == CFC_OK && y8) rc = held_ok(y8);
  if (rc != CFC_OK) return rc;
  if (off(a->w, 4) || off(rstd, 4)) return CFC_ERR_MISALIGNED;
  if (bad_eps(a->eps)) return CFC_ERR_INVALID_ARG;
  rc = cfc::device_ready();
  if (rc != CFC_OK) return rc;
  cfc::RmsCall q{};
  q.x = a->x; q.ldx = a->ldx; q.residual = a->residual; q.ldr = a->ldr; q.w = a->w;
  q.eps = a->eps; q.rows = a->rows; q.n = a->n; q.bf16 = a->dtype == CFC_BF16;
  q.s = s; q.lds = lds; q.y = y; q.ldy = ldy; q.s8 = held(s8); q.y8 = held(y8); q.rstd = rstd;
  return launched(cfc::rms_fwd_launch(q, on(stream)));
}

int cfc_rmsnorm_workspace_bytes(int rows, int n, size_t* bytes) {
  const int rc = rows_check(rows, n, CFC_F32);
  if (rc != CFC_OK) return rc;
  if (!bytes) return CFC_ERR_NULL_PTR;
  *bytes = cfc::rms_ws_floats(rows, n) * sizeof(float);
  return CFC_OK;
}

int cfc_rmsnorm_backward(const cfc_rmsnorm_args* a, const cfc_held8* s8, const float* rstd,
                         const void* dy, long long lddy, const void* ds, long long ldds, void* dx,
                         long long lddx, void* y, long long ldy, float* dw, void* ws,
                         size_t ws_bytes, cfc_stream_t stream) {
  if (!a) return CFC_ERR_NULL_PTR;
  int rc = rows_check(a->rows, a->n, a->dtype);
  if (rc != CFC_OK) return rc;
  const Rows r[] = {{s8 ? nullptr : a->x, a->ldx, s8 ? kInOpt : kIn}, {dy, lddy, kIn},
                    {ds, ldds, kInOpt}, {dx, lddx, kOut}, {y, ldy, kOutOpt}};
  rc = rows_ok(r, 5, a->n, a->dtype);
  if (rc != CFC_OK) return rc;
  if (!a->w || !rstd || !dw) return CFC_ERR_NULL_PTR;
  if (s8) rc = held_ok(s8);
  if (rc != CFC_OK) return rc;
  if (off(a->w, 4) || off(rstd, 4) || off(dw, 4)) return CFC_ERR_MISALIGNED;
  rc = ws_check(ws, ws_bytes, cfc::rms_ws_floats(a->rows, a->n) * sizeof(float));
  if (rc == CFC_OK) rc = cfc::device_ready();
  if (rc != CFC_OK) return rc;
  cfc::RmsCall q{};
  if (!s8) q.x = a->x, q.ldx = a->ldx;
  q.s8 = held(s8);
  q.w = a->w; q.rows = a->rows; q.n = a->n; q.bf16 = a->dtype == CFC_BF16;
  q.dy = dy; q.lddy = lddy; q.ds = ds; q.ldds = ldds; q.dx = dx; q.lddx = lddx;
  q.y = y; q.ldy = ldy; q.rstd = const_cast<float*>(rstd);
  return launched(cfc::rms_bwd_launch(q, dw, static_cast<float*>(ws), on(stream)));
}

int cfc_gated_forward(const cfc_gated_args* a, void* y, long long y_t, long long y_b,
                      float* h_last, float* states, const cfc_gated_kept* kept, void* ws,
                      size_t ws_bytes, cfc_stream_t stream) {
  cfc::GatedCall q{};
  int rc = gated_call(a, true, true, &q);
  if (rc != CFC_OK) return rc;
  const Seq out[] = {{y, y_t, y_b, kOut}};
  rc = seqs_ok(out, 1, a->dtype);
  if (rc == CFC_OK) rc = kept_call(kept, false, &q);
  if (rc != CFC_OK) return rc;
  if (off(h_last, 4) || off(states, 4)) return CFC_ERR_MISALIGNED;
  rc = ws_check(ws, ws_bytes, gated_bytes(q.B, q.K, q.D, false));
  if (rc == CFC_OK) rc = cfc::device_ready();
  if (rc != CFC_OK) return rc;
  q.y = y; q.y_t = y_t; q.y_b = y_b; q.h_last = h_last; q.states = states;
  q.ws = static_cast<float*>(ws);
  return launched(cfc::gated_fwd_launch(q, on(stream)));
}

int cfc_gated_workspace_bytes(int B, int K, int D, int backward, size_t* bytes) {
  const int rc = gated_check(B, K, D, CFC_F32, true);
  if (rc != CFC_OK) return rc;
  if (!bytes) return CFC_ERR_NULL_PTR;
  *bytes = gated_bytes(B, K, D, backward != 0);
  return CFC_OK;
}

int cfc_gated_backward(const cfc_gated_args* a, const cfc_gated_kept* kept, const float* states,
                       const void* dy, long long dy_t, long long dy_b, const float* dh_last,
                       const cfc_gated_grads* g, void* ws, size_t ws_bytes, cfc_stream_t stream) {
  cfc::GatedCall q{};
  int rc = gated_call(a, true, kept == nullptr, &q);
  if (rc != CFC_OK) return rc;
  if (!g || !states) return CFC_ERR_NULL_PTR;
  rc = kept_call(kept, true, &q);
  if (rc != CFC_OK) return rc;
  const Seq io[] = {{dy, dy_t, dy_b, kIn}, {g->dx, g->dx_t, g->dx_b, kOut},
                    {g->df, g->df_t, g->df_b, kOut},
                    {q.has_z ? g->dz : nullptr, g->dz_t, g->dz_b, q.has_z ? kOut : kOutOpt},
                    {g->y, g->y_t, g->y_b, kOutOpt}};
  rc = seqs_ok(io, 5, a->dtype);
  if (rc != CFC_OK) return rc;
  if (off(states, 4) || off(dh_last, 4) || off(g->dbias, 4) || off(g->dh0, 4))
    return CFC_ERR_MISALIGNED;
  rc = ws_check(ws, ws_bytes, gated_bytes(q.B, q.K, q.D, true));
  if (rc == CFC_OK) rc = cfc::device_ready();
  if (rc != CFC_OK) return rc;
  q.states = const_cast<float*>(states);
  q.dy = dy; q.dy_t = dy_t; q.dy_b = dy_b; q.dh_last = dh_last;
  q.dx = g->dx; q.dx_t = g->dx_t; q.dx_b = g->dx_b;
  q.df = g->df; q.df_t = g->df_t; q.df_b = g->df_b;
  q.dz = q.has_z ? g->dz : nullptr; q.dz_t = g->dz_t; q.dz_b = g->dz_b;
  q.y = g->y; q.y_t = g->y_t; q.y_b = g->y_b;
  q.dbias = g->dbias; q.dh0 = g->dh0;
  q.ws = static_cast<float*>(ws);
  return launched(cfc::gated_bwd_launch(q, on(stream)));
}

int cfc_gated_step(const cfc_gated_args* a, void* y, long long y_b, float* new_state,
                   cfc_stream_t stream) {
  cfc::GatedCall q{};
  int rc = gated_call(a, false, true, &q);
  if (rc != CFC_OK) return rc;
  const Seq out[] = {{y, 1, y_b, kOut}};
  rc = seqs_ok(out, 1, a->dtype, false);
  if (rc != CFC_OK) return rc;
  if (!a->h0 || !new_state) return CFC_ERR_NULL_PTR;
  if (off(new_state, 4)) return CFC_ERR_MISALIGNED;
  rc = cfc::device_ready();
  if (rc != CFC_OK) return rc;
  q.x_t = q.f_t = q.z_t = 0;
  q.y = y; q.y_b = y_b; q.h_last = new_state;
  return launched(cfc::gated_step_launch(q, on(stream)));
}

int cfc_weights4_quantize(const void* W, long long ldw, int N, int K, int group, int dtype,
                          void* codes, void* scales, cfc_stream_t stream) {
  int rc = weights4_check(N, K, group);
  if (rc != CFC_OK) return rc;
  if (!valid_dtype(dtype)) return CFC_ERR_INVALID_ARG;
  const Rows r[] = {{W, ldw, kIn}};
  rc = rows_ok(r, 1, K, dtype);
  if (rc != CFC_OK) return rc;
  if (!codes || !scales) return CFC_ERR_NULL_PTR;
  if (off(scales, 2)) return CFC_ERR_MISALIGNED;
  rc = cfc::device_ready();
  if (rc != CFC_OK) return rc;
  cfc::Weights4Call q{};
  q.N = N; q.K = K; q.group = group; q.bf16 = dtype == CFC_BF16; q.x = W; q.ldx = ldw;
  q.codes_out = static_cast<uint8_t*>(codes);
  q.scales_out = static_cast<uint16_t*>(scales);
  return launched(cfc::weights4_quantize_launch(q, on(stream)));
}

int cfc_weights4_bytes(int N, int K, int group, size_t* bytes) {
  const int rc = weights4_check(N, K, group);
  if (rc != CFC_OK) return rc;
  if (!bytes) return CFC_ERR_NULL_PTR;
  *bytes = cfc::weights4_bytes(N, K, group);
  return CFC_OK;
}

int cfc_weights4_lay_out(const void* codes, const void* scales, int N, int K, int group,
                         void* weights, size_t weights_bytes, cfc_stream_t stream) {
  int rc = weights4_check(N, K, group);
  if (rc != CFC_OK) return rc;
  if (!codes || !scales || !weights) return CFC_ERR_NULL_PTR;
  if (off(scales, 2) || off(weights, 16)) return CFC_ERR_MISALIGNED;
  if (weights_bytes < cfc::weights4_bytes(N, K, group)) return CFC_ERR_WS_TOO_SMALL;
  rc = cfc::device_ready();
  if (rc != CFC_OK) return rc;
  cfc::Weights4Call q{};
  q.N = N; q.K = K; q.group = group;
  q.codes = static_cast<const uint8_t*>(codes);
  q.scales = static_cast<const uint16_t*>(scales);
  q.laid_out = static_cast<uint8_t*>(weights);
  return launched(cfc::weights4_lay_out_launch(q, on(stream)));
}

int cfc_matvec4(const void* x, long long ldx, const void* weights, int M, int N, int K, int group,
                int dtype, void* y, long long ldy, cfc_stream_t stream) {
  int rc = weights4_check(N, K, group);
  if (rc != CFC_OK) return rc;
  if (M <= 0 || M > 1 << 19) return CFC_ERR_INVALID_DIM;
  if (!valid_dtype(dtype)) return CFC_ERR_INVALID_ARG;
  const Rows in[] = {{x, ldx, kIn}}, out[] = {{y, ldy, kOut}};
  rc = rows_ok(in, 1, K, dtype);
  if (rc == CFC_OK) rc = rows_ok(out, 1, N, dtype);
  if (rc != CFC_OK) return rc;
  if (!weights) return CFC_ERR_NULL_PTR;
  if (off(weights, 16)) return CFC_ERR_MISALIGNED;
  rc = cfc::device_ready();
  if (rc != CFC_OK) return rc;
  cfc::Weights4Call q{};
  q.M = M; q.N = N; q.K = K; q.group = group; q.bf16 = dtype == CFC_BF16;
  q.x = x; q.ldx = ldx; q.y = y; q.ldy = ldy; q.weights = static_cast<const uint8_t*>(weights);
  return launched(cfc::weights4_matvec_launch(q, on(stream)));
}

}  // extern "C"
