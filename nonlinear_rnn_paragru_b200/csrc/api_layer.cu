// api_layer.cu -- the C ABI of the gated linear recurrence and the block norm
// (include/pararnn.h): argument checks and launches.  Host code only.
#include <cmath>
#include <stdint.h>

#include "block_norm.cuh"
#include "linrec_cell.cuh"

namespace pararnn {
long long linrec_most_ctas(int B, int D);
size_t linrec_part_floats(int cell, int B, int T, int D);
int launch_linrec_fwd(int cell, bool bf16, const LinParams& p, cudaStream_t stream);
int launch_linrec_bwd(int cell, bool bf16, bool bf16_out, LinParams p, float* dlam, float* dbias,
                      cudaStream_t stream);
int launch_linrec_step(int cell, bool bf16, const LinParams& p, const float* h_prev, float* h_next,
                       cudaStream_t stream);
}  // namespace pararnn

using namespace pararnn;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool is_dtype(int t) { return t == PARARNN_F32 || t == PARARNN_BF16; }

constexpr unsigned long long kWaitNs = 2000000000ull;  // bound on a wait without opts

// what the opts of an _ex call say of its waits
void wait_opts(const pararnn_opts* opts, unsigned long long& wait_ns, int& withhold) {
  wait_ns = opts && opts->timeout_us ? 1000ull * opts->timeout_us : kWaitNs;
  withhold = opts && (opts->flags & PARARNN_FLAG_INJECT_WITHHOLD) ? opts->inject_chunk : -1;
}

// the status word starts at 0; kernels write it where a wait runs out
bool clear_status(int* status, cudaStream_t stream) {
  return !status || cudaMemsetAsync(status, 0, sizeof(int), stream) == cudaSuccess;
}

bool stride_ok(long long s) { return s >= 0 && s % 8 == 0; }

// Sizes whose indexes and grids fit the kernels' types: B * T * D <= 2^40 (as a
// division, since the product can pass 64 bits), T and D <= 2^30
bool lin_fits(int B, int T, int D) {
  return T <= (1 << 30) && D <= (1 << 30) && (long long)B * T <= (1LL << 40) / D;
}
// and of the scans
bool scan_fits(int B, int T, int D) { return lin_fits(B, T, D) && linrec_most_ctas(B, D) < (1LL << 31); }

// what the three recurrence calls check alike; T = 1 for the step
int lin_args(int cell, const void* u, int u_dtype, long long sb, long long st, long long sg, const float* lam,
             const float* bias, int B, int T, int D, float kappa) {
  if (cell != PARARNN_LIN_GRU && cell != PARARNN_LIN_DECAY) return PARARNN_ERR_INVALID_ARG;
  if (B < 1 || T < 1 || D < 1 || D % 8 != 0) return PARARNN_ERR_INVALID_ARG;
  if (!is_dtype(u_dtype)) return PARARNN_ERR_UNSUPPORTED_DTYPE;
  if (!u || (cell == PARARNN_LIN_DECAY) != (lam != nullptr)) return PARARNN_ERR_INVALID_ARG;
  if (cell == PARARNN_LIN_DECAY && !(kappa > 0.f && std::isfinite(kappa))) return PARARNN_ERR_INVALID_ARG;
  if (!stride_ok(sb) || !stride_ok(st) || !stride_ok(sg)) return PARARNN_ERR_INVALID_ARG;
  if (!lin_fits(B, T, D)) return PARARNN_ERR_TOO_LARGE;
  if (!aligned(u, 16) || (lam && !aligned(lam, 4)) || (bias && !aligned(bias, 4))) return PARARNN_ERR_MISALIGNED;
  return PARARNN_OK;
}

LinParams lin_params(const void* u, long long sb, long long st, long long sg, const float* lam, const float* bias,
                     const float* h0, const unsigned char* reset, int B, int T, int D, float kappa) {
  LinParams p = {};
  p.wait_ns = kWaitNs;
  p.withhold = -1;
  p.u = u;
  p.sb = sb;
  p.st = st;
  p.sg = sg;
  p.lam = lam;
  p.bias = bias;
  p.h0 = h0;
  p.reset = reset;
  p.kappa = kappa;
  p.B = B;
  p.T = T;
  p.D = D;
  return p;
}

int done(int e) { return e == 0 ? PARARNN_OK : PARARNN_ERR_CUDA; }

// what the two block-norm calls check alike
int norm_args(const void* h, int h_dtype, long long ld_h, const void* g, int g_dtype, long long ld_g, int act,
              const float* w_post, const void* res, int r_dtype, long long ld_r, const float* scale,
              const float* w_pre, float eps, long long N, int D) {
  if (N < 1 || D < 1 || D % 8 != 0 || !h || !(eps > 0.f && std::isfinite(eps))) return PARARNN_ERR_INVALID_ARG;
  if (D > norm_max_d() || N >= (1LL << 31)) return PARARNN_ERR_TOO_LARGE;
  if (g && act != PARARNN_ACT_SILU && act != PARARNN_ACT_SIGMOID) return PARARNN_ERR_INVALID_ARG;
  if (!is_dtype(h_dtype) || (g && !is_dtype(g_dtype)) || (res && !is_dtype(r_dtype)))
    return PARARNN_ERR_UNSUPPORTED_DTYPE;
  if (!stride_ok(ld_h) || (g && !stride_ok(ld_g)) || (res && !stride_ok(ld_r))) return PARARNN_ERR_INVALID_ARG;
  for (const void* p : {h, g, res, (const void*)w_post, (const void*)scale, (const void*)w_pre})
    if (!aligned(p, 16)) return PARARNN_ERR_MISALIGNED;
  return PARARNN_OK;
}

NormParams norm_params(const void* h, int h_dtype, long long ld_h, const void* g, int g_dtype, long long ld_g,
                       int act, const float* w_post, const void* res, int r_dtype, long long ld_r,
                       const float* scale, const float* w_pre, float eps, long long N, int D) {
  NormParams p = {};
  p.h = h;
  p.g = g;
  p.res = res;
  p.ld_h = ld_h;
  p.ld_g = ld_g;
  p.ld_r = ld_r;
  p.types = (h_dtype == PARARNN_F32 ? 1 : 0) | (g_dtype == PARARNN_F32 ? 2 : 0) | (r_dtype == PARARNN_F32 ? 4 : 0);
  p.w_post = w_post;
  p.scale = scale;
  p.w_pre = w_pre;
  p.act = act;
  p.eps = eps;
  p.N = N;
  p.D = D;
  return p;
}

}  // namespace

extern "C" {

int pararnn_linrec_solve(int cell, const void* u, int u_dtype, long long u_stride_b, long long u_stride_t,
                         long long u_stride_g, const float* lam, const float* bias, const float* h0,
                         const unsigned char* reset, float* h, int B, int T, int D, float kappa,
                         pararnn_stream_t stream) {
  return pararnn_linrec_solve_ex(cell, u, u_dtype, u_stride_b, u_stride_t, u_stride_g, lam, bias, h0, reset, h, B, T,
                                 D, kappa, nullptr, nullptr, stream);
}

int pararnn_linrec_solve_ex(int cell, const void* u, int u_dtype, long long u_stride_b, long long u_stride_t,
                            long long u_stride_g, const float* lam, const float* bias, const float* h0,
                            const unsigned char* reset, float* h, int B, int T, int D, float kappa, int* status,
                            const pararnn_opts* opts, pararnn_stream_t stream) {
  const int rc = lin_args(cell, u, u_dtype, u_stride_b, u_stride_t, u_stride_g, lam, bias, B, T, D, kappa);
  if (rc) return rc;
  if (!h) return PARARNN_ERR_INVALID_ARG;
  if (!scan_fits(B, T, D)) return PARARNN_ERR_TOO_LARGE;
  if (!aligned(h, 16) || (h0 && !aligned(h0, 4)) || (status && !aligned(status, 4))) return PARARNN_ERR_MISALIGNED;
  LinParams p = lin_params(u, u_stride_b, u_stride_t, u_stride_g, lam, bias, h0, reset, B, T, D, kappa);
  p.h = h;
  p.status = status;
  wait_opts(opts, p.wait_ns, p.withhold);
  if (!clear_status(status, (cudaStream_t)stream)) return PARARNN_ERR_CUDA;
  return done(launch_linrec_fwd(cell, u_dtype == PARARNN_BF16, p, (cudaStream_t)stream));
}

size_t pararnn_linrec_workspace_size(int cell, int B, int T, int D) {
  if (cell != PARARNN_LIN_GRU && cell != PARARNN_LIN_DECAY) return 0;
  if (B < 1 || T < 1 || D < 1 || D % 8 != 0 || !scan_fits(B, T, D)) return 0;
  return (linrec_part_floats(cell, B, T, D) * sizeof(float) + 255) / 256 * 256;
}

int pararnn_linrec_adjoint(int cell, const void* u, int u_dtype, long long u_stride_b, long long u_stride_t,
                           long long u_stride_g, const float* lam, const float* bias, const float* h0,
                           const unsigned char* reset, const float* h, const float* dLdh, void* du,
                           int du_dtype, float* dlam, float* dbias, float* dh0, int B, int T, int D,
                           float kappa, void* workspace, size_t ws_bytes, pararnn_stream_t stream) {
  return pararnn_linrec_adjoint_ex(cell, u, u_dtype, u_stride_b, u_stride_t, u_stride_g, lam, bias, h0, reset, h,
                                   dLdh, du, du_dtype, dlam, dbias, dh0, B, T, D, kappa, nullptr, workspace, ws_bytes,
                                   nullptr, stream);
}

int pararnn_linrec_adjoint_ex(int cell, const void* u, int u_dtype, long long u_stride_b, long long u_stride_t,
                              long long u_stride_g, const float* lam, const float* bias, const float* h0,
                              const unsigned char* reset, const float* h, const float* dLdh, void* du,
                              int du_dtype, float* dlam, float* dbias, float* dh0, int B, int T, int D,
                              float kappa, int* status, void* workspace, size_t ws_bytes,
                              const pararnn_opts* opts, pararnn_stream_t stream) {
  const int rc = lin_args(cell, u, u_dtype, u_stride_b, u_stride_t, u_stride_g, lam, bias, B, T, D, kappa);
  if (rc) return rc;
  if (!h || !dLdh || !du || !workspace || (cell == PARARNN_LIN_GRU && dlam)) return PARARNN_ERR_INVALID_ARG;
  if (!is_dtype(du_dtype) || (du_dtype == PARARNN_BF16 && u_dtype != PARARNN_BF16))
    return PARARNN_ERR_UNSUPPORTED_DTYPE;
  if (!scan_fits(B, T, D)) return PARARNN_ERR_TOO_LARGE;
  if (!aligned(h, 16) || !aligned(dLdh, 16) || !aligned(du, 16) || (h0 && !aligned(h0, 4)) ||
      (dlam && !aligned(dlam, 4)) || (dbias && !aligned(dbias, 4)) || (dh0 && !aligned(dh0, 4)) ||
      (status && !aligned(status, 4)) || !aligned(workspace, 256))
    return PARARNN_ERR_MISALIGNED;
  if (ws_bytes < pararnn_linrec_workspace_size(cell, B, T, D)) return PARARNN_ERR_WORKSPACE_TOO_SMALL;
  LinParams p = lin_params(u, u_stride_b, u_stride_t, u_stride_g, lam, bias, h0, reset, B, T, D, kappa);
  p.h = const_cast<float*>(h);
  p.g = dLdh;
  p.du = du;
  p.dh0 = dh0;
  p.part = static_cast<float*>(workspace);
  p.status = status;
  wait_opts(opts, p.wait_ns, p.withhold);
  if (!clear_status(status, (cudaStream_t)stream)) return PARARNN_ERR_CUDA;
  return done(launch_linrec_bwd(cell, u_dtype == PARARNN_BF16, du_dtype == PARARNN_BF16, p, dlam, dbias,
                                (cudaStream_t)stream));
}

int pararnn_linrec_step(int cell, const void* u_t, int u_dtype, long long u_stride_b, long long u_stride_g,
                        const float* lam, const float* bias, const float* h_prev, float* h_next, int B, int D,
                        float kappa, pararnn_stream_t stream) {
  const int rc = lin_args(cell, u_t, u_dtype, u_stride_b, 0, u_stride_g, lam, bias, B, 1, D, kappa);
  if (rc) return rc;
  if (!h_next) return PARARNN_ERR_INVALID_ARG;
  if ((long long)B * D >= (1LL << 38)) return PARARNN_ERR_TOO_LARGE;
  if ((h_prev && !aligned(h_prev, 4)) || !aligned(h_next, 4)) return PARARNN_ERR_MISALIGNED;
  const LinParams p = lin_params(u_t, u_stride_b, 0, u_stride_g, lam, bias, nullptr, nullptr, B, 1, D, kappa);
  return done(launch_linrec_step(cell, u_dtype == PARARNN_BF16, p, h_prev, h_next, (cudaStream_t)stream));
}

int pararnn_block_norm(const void* h, int h_dtype, long long h_stride, const void* gate, int gate_dtype,
                       long long gate_stride, int act, const float* w_post, const void* res, int res_dtype,
                       long long res_stride, const float* scale, const float* w_pre, void* s, int s_dtype,
                       void* x, int x_dtype, float eps, long long N, int D, pararnn_stream_t stream) {
  const int rc = norm_args(h, h_dtype, h_stride, gate, gate_dtype, gate_stride, act, w_post, res, res_dtype,
                           res_stride, scale, w_pre, eps, N, D);
  if (rc) return rc;
  if ((w_pre != nullptr) != (x != nullptr) || (!s && !x)) return PARARNN_ERR_INVALID_ARG;
  if ((s && !is_dtype(s_dtype)) || (x && !is_dtype(x_dtype))) return PARARNN_ERR_UNSUPPORTED_DTYPE;
  if (s && s == res && (s_dtype != res_dtype || res_stride != D)) return PARARNN_ERR_INVALID_ARG;
  if (!aligned(s, 16) || !aligned(x, 16)) return PARARNN_ERR_MISALIGNED;
  NormParams p = norm_params(h, h_dtype, h_stride, gate, gate_dtype, gate_stride, act, w_post, res, res_dtype,
                             res_stride, scale, w_pre, eps, N, D);
  p.s = s;
  p.x = x;
  p.types |= (s_dtype == PARARNN_F32 ? 8 : 0) | (x_dtype == PARARNN_F32 ? 16 : 0);
  return done(launch_norm_fwd(p, (cudaStream_t)stream));
}

size_t pararnn_block_norm_workspace_size(long long N, int D) {
  if (N < 1 || N >= (1LL << 31) || D < 1 || D % 8 != 0 || D > norm_max_d()) return 0;
  return (norm_part_floats(N, D) * sizeof(float) + 255) / 256 * 256;
}

int pararnn_block_norm_adjoint(const void* h, int h_dtype, long long h_stride, const void* gate, int gate_dtype,
                               long long gate_stride, int act, const float* w_post, const void* res,
                               int res_dtype, long long res_stride, const float* scale, const float* w_pre,
                               const void* ds, int ds_dtype, long long ds_stride, const void* dx, int dx_dtype,
                               long long dx_stride, void* dh, void* dgate, void* dres, float* dw_post,
                               float* dscale, float* dw_pre, float eps, long long N, int D, void* workspace,
                               size_t ws_bytes, pararnn_stream_t stream) {
  return pararnn_block_norm_adjoint_ex(h, h_dtype, h_stride, gate, gate_dtype, gate_stride, act, w_post, res, res_dtype,
                                       res_stride, scale, w_pre, ds, ds_dtype, ds_stride, dx, dx_dtype, dx_stride, dh,
                                       dgate, dres, dw_post, dscale, dw_pre, eps, N, D, nullptr, workspace, ws_bytes,
                                       nullptr, stream);
}

int pararnn_block_norm_adjoint_ex(const void* h, int h_dtype, long long h_stride, const void* gate, int gate_dtype,
                                  long long gate_stride, int act, const float* w_post, const void* res,
                                  int res_dtype, long long res_stride, const float* scale, const float* w_pre,
                                  const void* ds, int ds_dtype, long long ds_stride, const void* dx, int dx_dtype,
                                  long long dx_stride, void* dh, void* dgate, void* dres, float* dw_post,
                                  float* dscale, float* dw_pre, float eps, long long N, int D, int* status,
                                  void* workspace, size_t ws_bytes, const pararnn_opts* opts,
                                  pararnn_stream_t stream) {
  const int rc = norm_args(h, h_dtype, h_stride, gate, gate_dtype, gate_stride, act, w_post, res, res_dtype,
                           res_stride, scale, w_pre, eps, N, D);
  if (rc) return rc;
  if (!dh || !workspace || (!ds && !dx) || (w_pre != nullptr) != (dx != nullptr) ||
      (gate != nullptr) != (dgate != nullptr) || (dres && !res) || (dw_post && !w_post) ||
      (dscale && !scale) || (dw_pre && !w_pre))
    return PARARNN_ERR_INVALID_ARG;
  if ((ds && !is_dtype(ds_dtype)) || (dx && !is_dtype(dx_dtype))) return PARARNN_ERR_UNSUPPORTED_DTYPE;
  if ((ds && !stride_ok(ds_stride)) || (dx && !stride_ok(dx_stride))) return PARARNN_ERR_INVALID_ARG;
  for (const void* q : {ds, dx, (const void*)dh, (const void*)dgate, (const void*)dres, (const void*)dw_post,
                        (const void*)dscale, (const void*)dw_pre})
    if (!aligned(q, 16)) return PARARNN_ERR_MISALIGNED;
  if (!aligned(workspace, 256) || (status && !aligned(status, 4))) return PARARNN_ERR_MISALIGNED;
  if (ws_bytes < pararnn_block_norm_workspace_size(N, D)) return PARARNN_ERR_WORKSPACE_TOO_SMALL;
  NormParams p = norm_params(h, h_dtype, h_stride, gate, gate_dtype, gate_stride, act, w_post, res, res_dtype,
                             res_stride, scale, w_pre, eps, N, D);
  p.ds = ds;
  p.dx = dx;
  p.ld_ds = ds_stride;
  p.ld_dx = dx_stride;
  p.types |= (ds_dtype == PARARNN_F32 ? 8 : 0) | (dx_dtype == PARARNN_F32 ? 16 : 0);
  p.dh = dh;
  p.dg = dgate;
  p.dres = dres;
  p.part = static_cast<float*>(workspace);
  p.status = status;
  wait_opts(opts, p.wait_ns, p.withhold);
  if (!clear_status(status, (cudaStream_t)stream)) return PARARNN_ERR_CUDA;
  return done(launch_norm_bwd(p, dw_post, dscale, dw_pre, (cudaStream_t)stream));
}

}  // extern "C"
