// linrec_cell.cuh -- the cells of the gated linear recurrence
//   h_t = (1 - m_t) h_{t-1} + b_t
// whose gates read the projections u_t only (never the state), forward and
// adjoint, in fp32.
//
//   LIN_GRU    u = (z, c):     m = z = sig(u_z + b_z),  b = z tanh(u_c + b_c)
//   LIN_DECAY  u = (r, i, x):  w = kappa softplus(lam) sig(u_r + b_r) = -log a,
//              m = 1 - a = -expm1(-w),  b = sqrt(1 - a^2) sig(u_i + b_i) (u_x + b_x)
//
// Everything is written in m = 1 - a, not in a: a decay of 0.999 rounded to
// fp32 is off by 3e-8, which over the 1000 steps it remembers is 3e-5 of the
// state, while m = 1e-3 is held to 2^-24 of itself and h - m h + b rounds each
// state once.  sqrt(1 - a^2) = sqrt(m (2 - m)) has no cancellation either.
#pragma once
#include <cuda_bf16.h>

#include "common.cuh"

namespace pararnn {

// e^-|x|: the one exponential of a sigmoid that can neither overflow nor turn
// an infinite argument into NaN
__device__ __forceinline__ float exp_neg_abs(float x) { return ex2(-kLog2e * fabsf(x)); }

// sqrt on the special-function unit (about 1 ulp); 0 for denormals
__device__ __forceinline__ float sqrt_apx(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rsqrt_apx(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 1 - e^-w for w >= 0, to a few 2^-24 of itself for every w.  Below 1/2 the
// Taylor series w - w^2/2! + ... - w^8/8! (the next term is below 2^-26 of the
// sum there); above, 1 - ex2 (no cancellation: e^-w < 0.61).
__device__ __forceinline__ float one_minus_exp(float w) {
  float p = fmaf(w, -1.f / 40320.f, 1.f / 5040.f);
  p = fmaf(w, p, -1.f / 720.f);
  p = fmaf(w, p, 1.f / 120.f);
  p = fmaf(w, p, -1.f / 24.f);
  p = fmaf(w, p, 1.f / 6.f);
  p = fmaf(w, p, -0.5f);
  p = fmaf(w, p, 1.f);
  return w < 0.5f ? w * p : 1.f - ex2(-kLog2e * w);
}

// log(1 + e^x), once per channel
__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))); }

template <int CELL>
struct LinCell;

template <>
struct LinCell<PARARNN_LIN_GRU> {
  static constexpr int G = 2;
  float bz, bc;
  __device__ __forceinline__ void init(const float* /*lam*/, const float* bias, float /*kappa*/, int D,
                                       int d) {
    bz = bias ? bias[d] : 0.f;
    bc = bias ? bias[D + d] : 0.f;
  }
  // sig(x), 1 - sig(x) and tanh(y) with one reciprocal: 1 / (1 + e^-|x|) and
  // tanh|y| = q / (2 - q), q = 1 - e^-2|y|, over the product of denominators
  // (at most 4)
  __device__ __forceinline__ void gates(const float (&u)[G], float& z, float& zc, float& c) const {
    const float x = u[0] + bz, y = u[1] + bc;
    const float t = exp_neg_abs(x), q = one_minus_exp(2.f * fabsf(y));
    const float d1 = 1.f + t, d2 = 2.f - q, inv = rcp(d1 * d2);
    const float pos = d2 * inv, neg = t * pos;
    z = x >= 0.f ? pos : neg;
    zc = x >= 0.f ? neg : pos;
    c = copysignf(q * d1 * inv, y);
  }
  __device__ __forceinline__ void coef(const float (&u)[G], float& m, float& b) const {
    float zc, c;
    gates(u, m, zc, c);
    b = m * c;
  }
  __device__ __forceinline__ float forget(const float (&u)[G]) const {
    const float x = u[0] + bz, t = exp_neg_abs(x), pos = rcp(1.f + t);
    return x >= 0.f ? pos : t * pos;
  }
  // du and the share of d lam for one step: hp = h_{t-1} (0 at a reset)
  __device__ __forceinline__ void grad(const float (&u)[G], float hp, float lt, float (&du)[G],
                                       float& e) const {
    float z, zc, c;
    gates(u, z, zc, c);
    du[0] = lt * (c - hp) * (z * zc);
    du[1] = lt * z * fmaf(-c, c, 1.f);
    e = 0.f;
  }
  __device__ __forceinline__ float lam_scale(const float*, int) const { return 0.f; }
};

template <>
struct LinCell<PARARNN_LIN_DECAY> {
  static constexpr int G = 3;
  float br, bi, bx, k;  // k = kappa softplus(lam)
  __device__ __forceinline__ void init(const float* lam, const float* bias, float kappa, int D, int d) {
    br = bias ? bias[d] : 0.f;
    bi = bias ? bias[D + d] : 0.f;
    bx = bias ? bias[2 * D + d] : 0.f;
    k = kappa * softplus(lam[d]);
  }
  // the two sigmoids and their complements over one reciprocal
  __device__ __forceinline__ void gates(const float (&u)[G], float& r, float& rc, float& i, float& ic) const {
    const float x = u[0] + br, y = u[1] + bi;
    const float tx = exp_neg_abs(x), ty = exp_neg_abs(y);
    const float dx = 1.f + tx, dy = 1.f + ty, inv = rcp(dx * dy);
    const float px = dy * inv, py = dx * inv, nx = tx * px, ny = ty * py;
    r = x >= 0.f ? px : nx;
    rc = x >= 0.f ? nx : px;
    i = y >= 0.f ? py : ny;
    ic = y >= 0.f ? ny : py;
  }
  __device__ __forceinline__ void coef(const float (&u)[G], float& m, float& b) const {
    float r, rc, i, ic;
    gates(u, r, rc, i, ic);
    m = one_minus_exp(k * r);
    b = sqrt_apx(m * (2.f - m)) * i * (u[2] + bx);
  }
  __device__ __forceinline__ float forget(const float (&u)[G]) const {
    const float x = u[0] + br, t = exp_neg_abs(x), pos = rcp(1.f + t);
    return one_minus_exp(k * (x >= 0.f ? pos : t * pos));
  }
  __device__ __forceinline__ void grad(const float (&u)[G], float hp, float lt, float (&du)[G],
                                       float& e) const {
    float r, rc, i, ic;
    gates(u, r, rc, i, ic);
    const float x = u[2] + bx, w = k * r, m = one_minus_exp(w), a = 1.f - m, s = m * (2.f - m);
    const float rb = s >= 1.1754944e-38f ? rsqrt_apx(s) : 0.f;  // 1 / beta; w / beta -> 0 with w
    const float beta = s * rb;
    // dL/dr * r: beta' = -(a^2 / beta) (d log a), log a = -w
    e = lt * (a * i * x * (a * (w * rb)) - a * hp * w);
    du[0] = e * rc;
    du[1] = lt * beta * x * (i * ic);
    du[2] = lt * beta * i;
  }
  // dlam = (sum of e) sig(lam) / softplus(lam); the ratio is 1 where e^lam underflows
  __device__ __forceinline__ float lam_scale(const float* lam, int d) const {
    const float sp = softplus(lam[d]);
    return sp > 0.f ? 1.f / (1.f + expf(-lam[d])) / sp : 1.f;
  }
};

// Affine maps h -> P h + Q of consecutive steps.  P < 0 marks a run of steps
// with a reset in it: what came before is forgotten even where it is infinite
// or NaN (0 * inf would carry it on).
__device__ __forceinline__ float lin_apply(float P, float Q, float h) { return P < 0.f ? Q : fmaf(P, h, Q); }
// (P, Q) <- the run (P, Q) followed by the run (P2, Q2)
__device__ __forceinline__ void lin_then(float& P, float& Q, float P2, float Q2) {
  Q = lin_apply(P2, Q2, Q);
  P = (P < 0.f || P2 < 0.f) ? -1.f : P * P2;
}

// Two neighbouring channels of u.
template <bool kBF16>
struct LinRaw {
  using type = float2;
  static __device__ __forceinline__ float2 get(type v) { return v; }
};
template <>
struct LinRaw<true> {
  using type = unsigned;
  static __device__ __forceinline__ float2 get(type v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  }
};
template <bool kBF16>
__device__ __forceinline__ typename LinRaw<kBF16>::type lin_load(const void* u, long long i) {
  const char* p = static_cast<const char*>(u) + i * (kBF16 ? 2 : 4);
  return __ldg(reinterpret_cast<const typename LinRaw<kBF16>::type*>(p));
}

struct LinParams {
  const void* u;
  long long sb, st, sg;  // strides of u in elements: batch row, step, gate
  const float* lam;
  const float* bias;
  const float* h0;
  const unsigned char* reset;
  float kappa;
  float* h;              // states (out of the solve, in of the adjoint)
  const float* g;        // dL/dh
  void* du;
  float* dh0;
  float* part;           // adjoint: [B * CL][(G + 1) D] sums over a CTA's steps
  int B, T, D;
  int ntd;               // 64-channel tiles in D
  int steps;             // steps of a warp in one round
};

}  // namespace pararnn
