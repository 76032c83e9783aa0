// cfc_trunk_abi.cu -- extern "C" entry points of the trunk operators (layer norm, dropout, causal
// convolution, selective scan): argument checks on the host, then the launches.  Nothing is
// allocated, nothing synchronises, and a refused call has enqueued nothing.
#include <cmath>
#include <cstdint>

#include "cfc.h"
#include "cfc_trunk_checks.h"
#include "cfc_trunk_kernels.h"

using namespace cfc::checks;

namespace {

// ---- layer norm and dropout ----

// The held drop probability and its scale.
bool set_drop(float p, const void* rng, cfc::NormCall* q) {
  if (!(p >= 0.f && p <= 1.f)) return false;
  q->cut = static_cast<unsigned>(std::floor(static_cast<double>(p) * 65536.0 + 0.5));
  q->scale = q->cut < 65536u ? static_cast<float>(65536.0 / (65536.0 - q->cut)) : 0.f;
  q->rng = static_cast<const unsigned long long*>(rng);
  return true;
}

int norm_forward(cfc::NormCall q, int dtype, cfc_stream_t stream) {
  if (!q.w || !q.b || !q.stats) return CFC_ERR_NULL_PTR;
  if (off(q.w, 4) || off(q.b, 4) || off(q.stats, 8) || off(q.rng, 8)) return CFC_ERR_MISALIGNED;
  if (bad_eps(q.eps)) return CFC_ERR_INVALID_ARG;
  const int rc = cfc::device_ready();
  if (rc != CFC_OK) return rc;
  q.bf16 = dtype == CFC_BF16;
  return launched(cfc::norm_fwd_launch(q, static_cast<cudaStream_t>(stream)));
}

int norm_backward(cfc::NormCall q, int dtype, float* dw, float* db, void* ws, size_t ws_bytes,
                  cfc_stream_t stream) {
  if (!q.w || !q.stats || !dw || !db) return CFC_ERR_NULL_PTR;
  if (off(q.w, 4) || off(dw, 4) || off(db, 4) || off(q.stats, 8) || off(q.rng, 8))
    return CFC_ERR_MISALIGNED;
  int rc = ws_check(ws, ws_bytes, cfc::norm_ws_floats(q.rows, q.n) * sizeof(float));
  if (rc == CFC_OK) rc = cfc::device_ready();
  if (rc != CFC_OK) return rc;
  q.bf16 = dtype == CFC_BF16;
  return launched(cfc::norm_bwd_launch(q, dw, db, static_cast<float*>(ws),
                                       static_cast<cudaStream_t>(stream)));
}

// ---- convolution and scan ----

int conv_check(int B, int K, int D, int W, int dtype) {
  if (B <= 0 || B > kMaxSequences || K <= 0 || K > kMaxSteps || D <= 0 || D > kMaxWidth || W < 2 ||
      W > 4)
    return CFC_ERR_INVALID_DIM;
  return valid_dtype(dtype) ? CFC_OK : CFC_ERR_INVALID_ARG;
}

// Fills the common part of a call; the argument errors of the struct itself.
int conv_call(const cfc_conv_args* a, cfc::ConvCall* q) {
  if (!a) return CFC_ERR_NULL_PTR;
  int rc = conv_check(a->B, a->K, a->D, a->W, a->dtype);
  if (rc != CFC_OK) return rc;
  const Seq in[] = {{a->x, a->x_t, a->x_b, kIn}, {a->x0, 1, 1, kInOpt}};
  rc = seqs_ok(in, 2, a->dtype);
  if (rc != CFC_OK) return rc;
  if (!a->w) return CFC_ERR_NULL_PTR;
  if (off(a->w, 4) || off(a->bias, 4) || off(a->lengths, 4)) return CFC_ERR_MISALIGNED;
  q->B = a->B; q->K = a->K; q->D = a->D; q->W = a->W;
  q->bf16 = a->dtype == CFC_BF16;
  q->silu = a->silu != 0;
  q->lengths = a->lengths;
  q->x = a->x; q->x_t = a->x_t; q->x_b = a->x_b;
  q->x0 = a->x0; q->w = a->w; q->bias = a->bias;
  return CFC_OK;
}

int scan_sizes(const cfc_scan_args* a, bool steps) {
  if (!a) return CFC_ERR_NULL_PTR;
  if (a->B <= 0 || a->B > kMaxSequences || a->D <= 0 || a->D > kMaxWidth || a->N <= 0 ||
      a->N > cfc::kScanMaxStates || a->G <= 0 || a->D % a->G != 0)
    return CFC_ERR_INVALID_DIM;
  if (steps && (a->K <= 0 || a->K > kMaxSteps)) return CFC_ERR_INVALID_DIM;
  // Partial sums of the parameters are indexed by ints.
  if (static_cast<long long>(a->D) * (a->N + 2) >= (1LL << 31)) return CFC_ERR_INVALID_DIM;
  return valid_dtype(a->dtype) ? CFC_OK : CFC_ERR_INVALID_ARG;
}

cfc::ScanCall scan_shape(const cfc_scan_args* a) {
  cfc::ScanCall q{};
  q.B = a->B; q.K = a->K; q.D = a->D; q.N = a->N; q.G = a->G;
  q.bf16 = a->dtype == CFC_BF16;
  q.softplus = a->softplus != 0;
  return q;
}

int scan_call(const cfc_scan_args* a, bool steps, cfc::ScanCall* q) {
  int rc = scan_sizes(a, steps);
  if (rc != CFC_OK) return rc;
  const Seq in[] = {{a->x, a->x_t, a->x_b, kIn}, {a->dt, a->dt_t, a->dt_b, kIn},
                    {a->z, a->z_t, a->z_b, kInOpt}, {a->Bm, a->Bm_t, a->Bm_b, kIn},
                    {a->Cm, a->Cm_t, a->Cm_b, kIn}};
  rc = seqs_ok(in, 5, a->dtype, steps);
  if (rc != CFC_OK) return rc;
  if (!a->A) return CFC_ERR_NULL_PTR;
  if (off(a->A, 4) || off(a->skip, 4) || off(a->dt_bias, 4) || off(a->lengths, 4) || off(a->h0, 16))
    return CFC_ERR_MISALIGNED;
  *q = scan_shape(a);
  q->lengths = a->lengths;
  q->x = a->x; q->x_t = a->x_t; q->x_b = a->x_b;
  q->dt = a->dt; q->dt_t = a->dt_t; q->dt_b = a->dt_b;
  q->z = a->z; q->z_t = a->z_t; q->z_b = a->z_b;
  q->Bm = a->Bm; q->Bm_t = a->Bm_t; q->Bm_b = a->Bm_b;
  q->Cm = a->Cm; q->Cm_t = a->Cm_t; q->Cm_b = a->Cm_b;
  q->A = a->A; q->skip = a->skip; q->dt_bias = a->dt_bias; q->h0 = a->h0;
  return CFC_OK;
}

}  // namespace

extern "C" {

int cfc_layernorm_forward(const void* x, long long ldx, const float* w, const float* b, int rows,
                          int n, float eps, int dtype, void* y, long long ldy, float* stats,
                          cfc_stream_t stream) {
  int rc = rows_check(rows, n, dtype);
  if (rc != CFC_OK) return rc;
  const Rows r[] = {{x, ldx, kIn}, {y, ldy, kOut}};
  rc = rows_ok(r, 2, n, dtype);
  if (rc != CFC_OK) return rc;
  cfc::NormCall q{};
  q.x = x; q.ldx = ldx; q.w = w; q.b = b; q.rows = rows; q.n = n; q.eps = eps;
  q.y = y; q.ldy = ldy; q.stats = stats;
  return norm_forward(q, dtype, stream);
}

int cfc_layernorm_workspace_bytes(int rows, int n, size_t* bytes) {
  const int rc = rows_check(rows, n, CFC_F32);
  if (rc != CFC_OK) return rc;
  if (!bytes) return CFC_ERR_NULL_PTR;
  *bytes = cfc::norm_ws_floats(rows, n) * sizeof(float);
  return CFC_OK;
}

int cfc_layernorm_backward(const void* dy, long long lddy, const void* x, long long ldx,
                           const float* w, const float* stats, int rows, int n, int dtype, void* dx,
                           long long lddx, float* dw, float* db, void* ws, size_t ws_bytes,
                           cfc_stream_t stream) {
  int rc = rows_check(rows, n, dtype);
  if (rc != CFC_OK) return rc;
  const Rows r[] = {{dy, lddy, kIn}, {x, ldx, kIn}, {dx, lddx, kOut}};
  rc = rows_ok(r, 3, n, dtype);
  if (rc != CFC_OK) return rc;
  cfc::NormCall q{};
  q.x = x; q.ldx = ldx; q.dy = dy; q.lddy = lddy; q.w = w; q.rows = rows; q.n = n;
  q.dx = dx; q.lddx = lddx; q.stats = const_cast<float*>(stats);
  return norm_backward(q, dtype, dw, db, ws, ws_bytes, stream);
}

int cfc_dropout_forward(const void* x, long long ldx, const void* residual, long long ldr,
                        const void* rng, float p, int rows, int n, int dtype, void* y,
                        long long ldy, cfc_stream_t stream) {
  int rc = rows_check(rows, n, dtype);
  if (rc != CFC_OK) return rc;
  const Rows r[] = {{x, ldx, kIn}, {residual, ldr, kInOpt}, {y, ldy, kOut}};
  rc = rows_ok(r, 3, n, dtype);
  if (rc != CFC_OK) return rc;
  if (!rng) return CFC_ERR_NULL_PTR;
  if (off(rng, 8)) return CFC_ERR_MISALIGNED;
  cfc::NormCall q{};
  if (!set_drop(p, rng, &q)) return CFC_ERR_INVALID_ARG;
  rc = cfc::device_ready();
  if (rc != CFC_OK) return rc;
  q.x = x; q.ldx = ldx; q.residual = residual; q.ldr = ldr; q.rows = rows; q.n = n;
  q.s = y; q.lds = ldy; q.bf16 = dtype == CFC_BF16;
  return launched(cfc::dropout_launch(q, static_cast<cudaStream_t>(stream)));
}

int cfc_dropout_backward(const void* dy, long long lddy, const void* rng, float p, int rows, int n,
                         int dtype, void* dx, long long lddx, cfc_stream_t stream) {
  return cfc_dropout_forward(dy, lddy, nullptr, 0, rng, p, rows, n, dtype, dx, lddx, stream);
}

int cfc_dropout_layernorm_forward(const void* x, long long ldx, const void* residual,
                                  long long ldr, const void* rng, float p, const float* w,
                                  const float* b, int rows, int n, float eps, int dtype, void* s,
                                  long long lds, void* y, long long ldy, float* stats,
                                  cfc_stream_t stream) {
  int rc = rows_check(rows, n, dtype);
  if (rc != CFC_OK) return rc;
  const Rows r[] = {{x, ldx, kIn}, {residual, ldr, kInOpt}, {s, lds, kOut}, {y, ldy, kOut}};
  rc = rows_ok(r, 4, n, dtype);
  if (rc != CFC_OK) return rc;
  if (!rng) return CFC_ERR_NULL_PTR;
  cfc::NormCall q{};
  if (!set_drop(p, rng, &q)) return CFC_ERR_INVALID_ARG;
  q.x = x; q.ldx = ldx; q.residual = residual; q.ldr = ldr; q.w = w; q.b = b;
  q.rows = rows; q.n = n; q.eps = eps; q.s = s; q.lds = lds; q.y = y; q.ldy = ldy; q.stats = stats;
  return norm_forward(q, dtype, stream);
}

int cfc_dropout_layernorm_backward(const void* dy, long long lddy, const void* ds, long long ldds,
                                   const void* s, long long lds, const void* rng, float p,
                                   const float* w, const float* stats, int rows, int n, int dtype,
                                   void* dx, long long lddx, void* dres, long long lddr, float* dw,
                                   float* db, void* ws, size_t ws_bytes, cfc_stream_t stream) {
  int rc = rows_check(rows, n, dtype);
  if (rc != CFC_OK) return rc;
  const Rows r[] = {{dy, lddy, kIn}, {ds, ldds, kInOpt}, {s, lds, kIn}, {dx, lddx, kOut},
                    {dres, lddr, kOutOpt}};
  rc = rows_ok(r, 5, n, dtype);
  if (rc != CFC_OK) return rc;
  if (!rng) return CFC_ERR_NULL_PTR;
  cfc::NormCall q{};
  if (!set_drop(p, rng, &q)) return CFC_ERR_INVALID_ARG;
  q.x = s; q.ldx = lds; q.dy = dy; q.lddy = lddy; q.ds = ds; q.ldds = ldds; q.w = w;
  q.rows = rows; q.n = n; q.dx = dx; q.lddx = lddx; q.dres = dres; q.lddr = lddr;
  q.stats = const_cast<float*>(stats);
  return norm_backward(q, dtype, dw, db, ws, ws_bytes, stream);
}

int cfc_conv_forward(const cfc_conv_args* a, void* u, long long u_t, long long u_b, void* last,
                     cfc_stream_t stream) {
  cfc::ConvCall q{};
  int rc = conv_call(a, &q);
  if (rc != CFC_OK) return rc;
  const Seq out[] = {{u, u_t, u_b, kOut}, {last, 1, 1, kOutOpt}};
  rc = seqs_ok(out, 2, a->dtype);
  if (rc == CFC_OK) rc = cfc::device_ready();
  if (rc != CFC_OK) return rc;
  q.u = u; q.u_t = u_t; q.u_b = u_b; q.last = last;
  return launched(cfc::conv_fwd_launch(q, static_cast<cudaStream_t>(stream)));
}

int cfc_conv_workspace_bytes(int B, int K, int D, int W, int dtype, size_t* bytes) {
  const int rc = conv_check(B, K, D, W, dtype);
  if (rc != CFC_OK) return rc;
  if (!bytes) return CFC_ERR_NULL_PTR;
  const size_t P = static_cast<size_t>(cfc::conv_partials(B, K, D, dtype == CFC_BF16));
  *bytes = P == 1 ? 0 : P * static_cast<size_t>(D) * (W + 1) * sizeof(float);
  return CFC_OK;
}

int cfc_conv_backward(const cfc_conv_args* a, const void* du, long long du_t, long long du_b,
                      void* dx, long long dx_t, long long dx_b, float* dw, float* dbias, void* dx0,
                      void* ws, size_t ws_bytes, cfc_stream_t stream) {
  cfc::ConvCall q{};
  int rc = conv_call(a, &q);
  if (rc != CFC_OK) return rc;
  const Seq io[] = {{du, du_t, du_b, kIn}, {dx, dx_t, dx_b, kOut}, {dx0, 1, 1, kOutOpt}};
  rc = seqs_ok(io, 3, a->dtype);
  if (rc != CFC_OK) return rc;
  if (!dw || !dbias) return CFC_ERR_NULL_PTR;
  if (off(dw, 4) || off(dbias, 4)) return CFC_ERR_MISALIGNED;
  size_t need = 0;
  (void)cfc_conv_workspace_bytes(a->B, a->K, a->D, a->W, a->dtype, &need);
  rc = ws_check(ws, ws_bytes, need);
  if (rc == CFC_OK) rc = cfc::device_ready();
  if (rc != CFC_OK) return rc;
  q.du = du; q.du_t = du_t; q.du_b = du_b;
  q.dx = dx; q.dx_t = dx_t; q.dx_b = dx_b; q.dx0 = dx0;
  return launched(cfc::conv_bwd_launch(q, dw, dbias, static_cast<float*>(ws),
                                       static_cast<cudaStream_t>(stream)));
}

int cfc_conv_step(const void* x, long long x_b, const float* w, const float* bias,
                  const void* state, int B, int D, int W, int dtype, int silu, void* u,
                  long long u_b, void* new_state, cfc_stream_t stream) {
  int rc = conv_check(B, 1, D, W, dtype);
  if (rc != CFC_OK) return rc;
  const Seq io[] = {{x, 1, x_b, kIn}, {u, 1, u_b, kOut}, {state, 1, 1, kIn}, {new_state, 1, 1, kOut}};
  rc = seqs_ok(io, 4, dtype);
  if (rc != CFC_OK) return rc;
  if (!w) return CFC_ERR_NULL_PTR;
  if (off(w, 4) || off(bias, 4)) return CFC_ERR_MISALIGNED;
  rc = cfc::device_ready();
  if (rc != CFC_OK) return rc;
  cfc::ConvCall q{};
  q.B = B; q.K = 1; q.D = D; q.W = W;
  q.bf16 = dtype == CFC_BF16;
  q.silu = silu != 0;
  q.x = x; q.x_b = x_b; q.w = w; q.bias = bias; q.x0 = state;
  q.u = u; q.u_b = u_b; q.last = new_state;
  return launched(cfc::conv_step_launch(q, static_cast<cudaStream_t>(stream)));
}

int cfc_scan_workspace_bytes(const cfc_scan_args* a, int backward, size_t* bytes) {
  const int rc = scan_sizes(a, true);
  if (rc != CFC_OK) return rc;
  if (!bytes) return CFC_ERR_NULL_PTR;
  const cfc::ScanCall q = scan_shape(a);
  *bytes = (backward ? cfc::scan_bwd_ws_floats(q) : cfc::scan_fwd_ws_floats(q)) * sizeof(float);
  return CFC_OK;
}

int cfc_scan_states_bytes(const cfc_scan_args* a, size_t* bytes) {
  const int rc = scan_sizes(a, true);
  if (rc != CFC_OK) return rc;
  if (!bytes) return CFC_ERR_NULL_PTR;
  const size_t kept = (static_cast<size_t>(a->K) + cfc::kScanPeriod - 1) / cfc::kScanPeriod;
  *bytes = kept * a->B * a->D * a->N * sizeof(float);
  return CFC_OK;
}

int cfc_scan_forward(const cfc_scan_args* a, void* y, long long y_t, long long y_b, float* h_last,
                     float* states, void* ws, size_t ws_bytes, cfc_stream_t stream) {
  cfc::ScanCall q{};
  int rc = scan_call(a, true, &q);
  if (rc != CFC_OK) return rc;
  const Seq out[] = {{y, y_t, y_b, kOut}};
  rc = seqs_ok(out, 1, a->dtype);
  if (rc != CFC_OK) return rc;
  if (off(h_last, 16) || off(states, 16)) return CFC_ERR_MISALIGNED;
  rc = ws_check(ws, ws_bytes, cfc::scan_fwd_ws_floats(q) * sizeof(float));
  if (rc == CFC_OK) rc = cfc::device_ready();
  if (rc != CFC_OK) return rc;
  q.y = y; q.y_t = y_t; q.y_b = y_b; q.h_last = h_last; q.states = states;
  q.ws = static_cast<float*>(ws);
  return launched(cfc::scan_fwd_launch(q, static_cast<cudaStream_t>(stream)));
}

int cfc_scan_backward(const cfc_scan_args* a, const float* states, const void* dy, long long dy_t,
                      long long dy_b, const float* dh_last, const cfc_scan_grads* g, void* ws,
                      size_t ws_bytes, cfc_stream_t stream) {
  cfc::ScanCall q{};
  int rc = scan_call(a, true, &q);
  if (rc != CFC_OK) return rc;
  if (!g || !states || !g->dB || !g->dC || !g->dA) return CFC_ERR_NULL_PTR;
  const Seq io[] = {{dy, dy_t, dy_b, kIn}, {g->dx, g->dx_t, g->dx_b, kOut},
                    {g->ddt, g->ddt_t, g->ddt_b, kOut},
                    {a->z ? g->dz : nullptr, g->dz_t, g->dz_b, a->z ? kOut : kOutOpt},
                    {g->dB, 1, 1, kOut}, {g->dC, 1, 1, kOut}};
  rc = seqs_ok(io, 6, a->dtype);
  if (rc != CFC_OK) return rc;
  if (off(states, 16) || off(dh_last, 16) || off(g->dA, 4) || off(g->dskip, 4) ||
      off(g->ddt_bias, 4) || off(g->dh0, 16))
    return CFC_ERR_MISALIGNED;
  rc = ws_check(ws, ws_bytes, cfc::scan_bwd_ws_floats(q) * sizeof(float));
  if (rc == CFC_OK) rc = cfc::device_ready();
  if (rc != CFC_OK) return rc;
  q.states = const_cast<float*>(states);
  q.dy = dy; q.dy_t = dy_t; q.dy_b = dy_b; q.dh_last = dh_last;
  q.dx = g->dx; q.dx_t = g->dx_t; q.dx_b = g->dx_b;
  q.ddt = g->ddt; q.ddt_t = g->ddt_t; q.ddt_b = g->ddt_b;
  q.dz = a->z ? g->dz : nullptr; q.dz_t = g->dz_t; q.dz_b = g->dz_b;
  q.dB = g->dB; q.dC = g->dC; q.dA = g->dA; q.dskip = g->dskip; q.ddt_bias = g->ddt_bias;
  q.dh0 = g->dh0;
  q.ws = static_cast<float*>(ws);
  return launched(cfc::scan_bwd_launch(q, static_cast<cudaStream_t>(stream)));
}

int cfc_scan_step(const cfc_scan_args* a, void* y, long long y_b, float* new_state,
                  cfc_stream_t stream) {
  cfc::ScanCall q{};
  int rc = scan_call(a, false, &q);
  if (rc != CFC_OK) return rc;
  const Seq out[] = {{y, 1, y_b, kOut}};
  rc = seqs_ok(out, 1, a->dtype);
  if (rc != CFC_OK) return rc;
  if (!a->h0 || !new_state) return CFC_ERR_NULL_PTR;
  if (off(new_state, 16)) return CFC_ERR_MISALIGNED;
  rc = cfc::device_ready();
  if (rc != CFC_OK) return rc;
  q.y = y; q.y_b = y_b; q.h_last = new_state;
  return launched(cfc::scan_step_launch(q, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
