// linrec_cell.cuh -- the cells of the gated linear recurrence
//   h_t = (1 - m_t) h_{t-1} + b_t
// whose gates read the projections u_t only (never the state), forward and
// adjoint, in fp32.  A thread evaluates two neighbouring channels; sums and
// products are packed (one instruction for both, each half rounded alone).
//
//   LIN_GRU    u = (z, c):     m = z = sig(u_z + b_z),  b = z tanh(u_c + b_c)
//   LIN_DECAY  u = (r, i, x):  w = kappa softplus(lam) sig(u_r + b_r) = -log a,
//              m = 1 - a = -expm1(-w),  b = sqrt(1 - a^2) sig(u_i + b_i) (u_x + b_x)
//
// Everything is written in m = 1 - a, not in a: a decay of 0.999 rounded to
// fp32 is off by 3e-8, which over the 1000 steps it remembers is 3e-5 of the
// state, while m = 1e-3 is held to 2^-24 of itself and (h - m h) + b rounds each
// state twice.  sqrt(1 - a^2) = sqrt(m (2 - m)) has no cancellation either.
// The code holds nm = -m, the factor of the fma.
#pragma once
#include <cuda_bf16.h>

#include "common.cuh"

namespace pararnn {

// ------------------------------------------------------- packed arithmetic --
__device__ __forceinline__ float2 lfma(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 lmul(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 ladd(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 ex2_2(float2 v) { return make_float2(ex2(v.x), ex2(v.y)); }
// 2^-|v|: the exponential of a sigmoid that neither overflows nor turns an
// infinite argument into NaN
__device__ __forceinline__ float2 ex2_neg_abs(float2 v) { return make_float2(ex2(-fabsf(v.x)), ex2(-fabsf(v.y))); }
__device__ __forceinline__ float2 rcp_2(float2 v) { return make_float2(rcp(v.x), rcp(v.y)); }
__device__ __forceinline__ float2 neg2(float2 v) { return make_float2(-v.x, -v.y); }
// 2^v that overflowed made finite again, so that it times its 1 / (1 + 2^v) = 0
// is not NaN
__device__ __forceinline__ float2 finite(float2 t) { return make_float2(fminf(t.x, 8.5e37f), fminf(t.y, 8.5e37f)); }
// v > 0 ? a : b
__device__ __forceinline__ float2 sel_pos(float2 v, float2 a, float2 b) {
  return make_float2(v.x > 0.f ? a.x : b.x, v.y > 0.f ? a.y : b.y);
}
// square root and its reciprocal on the special-function unit (about 1 ulp;
// 0 and infinity for denormals)
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

constexpr float kLn2 = 0.69314718055994531f;

// 2^-v - 1 = -(1 - a) for v >= 0 (v = w log2 e), to a few 2^-24 of itself.
// Below v = 0.36 (w < 1/4) the Taylor series of -expm1 to w^6 (the next term
// is below 2^-24 of the sum there); above, no cancellation: 2^-v < 0.78.
__device__ __forceinline__ float2 decay_nm(float2 v) {
  constexpr float L1 = kLn2, L2 = L1 * kLn2, L3 = L2 * kLn2, L4 = L3 * kLn2, L5 = L4 * kLn2, L6 = L5 * kLn2;
  float2 p = lfma(v, both(L6 / 720.f), both(-L5 / 120.f));
  p = lfma(v, p, both(L4 / 24.f));
  p = lfma(v, p, both(-L3 / 6.f));
  p = lfma(v, p, both(L2 / 2.f));
  p = lfma(v, p, both(-L1));
  p = lmul(v, p);
  const float2 e = ladd(ex2_2(neg2(v)), both(-1.f));
  return make_float2(v.x < 0.36f ? p.x : e.x, v.y < 0.36f ? p.y : e.y);
}

// -tanh y and its slope 1 - tanh^2 = 4 t R^2 with t = e^2y, R = 1 / (1 + t): of
// its own size on both sides (4 (R - R^2) would be 0 from y = -8.5 down, where R
// rounds to 1).  -tanh below |y| = 0.2 is the Taylor series to y^7 (the next term
// is below 2^-24 of the sum there); above, 2 R - 1, whose rounding is 2^-23 at
// most (10 units of the last place of the smallest |tanh| it serves).
__device__ __forceinline__ float2 minus_tanh(float2 y, float2& slope) {
  const float2 t = ex2_2(lmul(y, both(2.f * kLog2e))), R = rcp_2(ladd(t, both(1.f)));
  slope = lmul(lmul(lmul(finite(t), R), R), both(4.f));
  const float2 big = lfma(R, both(2.f), both(-1.f));
  const float2 s = lmul(y, y);
  float2 p = lfma(s, both(17.f / 315.f), both(-2.f / 15.f));
  p = lfma(s, p, both(1.f / 3.f));
  p = lfma(s, p, both(-1.f));
  p = lmul(y, p);
  return make_float2(fabsf(y.x) < 0.2f ? p.x : big.x, fabsf(y.y) < 0.2f ? p.y : big.y);
}

// log(1 + e^x), once per channel
__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))); }
// its logarithm's derivative sig(x) / softplus(x), by e^-|x|, which does not
// overflow; 1 where e^x underflows
__device__ __forceinline__ float dlog_softplus(float x) {
  const float sp = softplus(x), e = expf(-fabsf(x));
  return sp > 0.f ? (x < 0.f ? e : 1.f) / ((1.f + e) * sp) : 1.f;
}

__device__ __forceinline__ float2 vec2(const float* p, int d) { return p ? make_float2(p[d], p[d + 1]) : both(0.f); }

template <int CELL>
struct LinCell;

template <>
struct LinCell<PARARNN_LIN_GRU> {
  static constexpr int G = 2;
  float2 bz, bc;  // -log2 e b_z, b_c
  __device__ __forceinline__ void init(const float* /*lam*/, const float* bias, float /*kappa*/, int D, int d) {
    bz = lmul(vec2(bias, d), both(-kLog2e));
    bc = vec2(bias ? bias + D : nullptr, d);
  }
  __device__ __forceinline__ float2 zarg(float2 u) const { return lfma(u, both(-kLog2e), bz); }
  __device__ __forceinline__ void coef(const float2 (&u)[G], float2& nm, float2& b) const {
    float2 slope;
    nm = rcp_2(neg2(ladd(ex2_2(zarg(u[0])), both(1.f))));  // -z; 0 where 2^v overflows
    b = lmul(nm, minus_tanh(ladd(u[1], bc), slope));
  }
  // The adjoint's first pass: nm from the first gate, and what the second
  // keeps of it: z (1 - z), of its own size where z is near 1 too.
  static constexpr int kKeep = 1;
  __device__ __forceinline__ void head(float2 u0, float2& nm, float2 (&keep)[kKeep]) const {
    const float2 t = ex2_2(zarg(u0));
    nm = rcp_2(neg2(ladd(t, both(1.f))));
    keep[0] = lmul(lmul(finite(t), nm), nm);
  }
  // The second: du of one step from lambda and h_{t-1}.
  __device__ __forceinline__ void grad(const float2 (&u)[G], float2 nm, const float2 (&keep)[kKeep], float2 hp,
                                       float2 lt, float2 (&du)[G], float2& /*e*/) const {
    float2 slope;
    const float2 nc = minus_tanh(ladd(u[1], bc), slope), nl = neg2(lt);
    du[0] = lmul(lmul(nl, keep[0]), ladd(hp, nc));
    du[1] = lmul(lmul(nl, nm), slope);
  }
  static __device__ __forceinline__ float2 lam_scale(const float*, int) { return both(0.f); }
};

template <>
struct LinCell<PARARNN_LIN_DECAY> {
  static constexpr int G = 3;
  float2 br, bi, bx, k;  // -log2 e b_r, -log2 e b_i, b_x, kappa softplus(lam) log2 e
  __device__ __forceinline__ void init(const float* lam, const float* bias, float kappa, int D, int d) {
    br = lmul(vec2(bias, d), both(-kLog2e));
    bi = lmul(vec2(bias ? bias + D : nullptr, d), both(-kLog2e));
    bx = vec2(bias ? bias + 2 * (size_t)D : nullptr, d);
    k = lmul(make_float2(softplus(lam[d]), softplus(lam[d + 1])), both(kappa * kLog2e));
  }
  __device__ __forceinline__ void coef(const float2 (&u)[G], float2& nm, float2& b) const {
    // r and i over one reciprocal (this cell's solve is bound by the
    // special-function unit): sig(x) is q = 1 / (1 + 2^-|v|) for x >= 0
    // (v <= 0), 2^-|v| q below
    const float2 vr = lfma(u[0], both(-kLog2e), br), vi = lfma(u[1], both(-kLog2e), bi);
    const float2 tr = ex2_neg_abs(vr), ti = ex2_neg_abs(vi);
    const float2 dr = ladd(tr, both(1.f)), di = ladd(ti, both(1.f)), inv = rcp_2(lmul(dr, di));
    const float2 r = lmul(sel_pos(vr, tr, both(1.f)), lmul(di, inv));
    const float2 i = lmul(sel_pos(vi, ti, both(1.f)), lmul(dr, inv));
    nm = decay_nm(lmul(k, r));
    const float2 s = lmul(nm, ladd(nm, both(2.f)));  // -(1 - a^2)
    b = lmul(lmul(make_float2(sqrt_apx(-s.x), sqrt_apx(-s.y)), i), ladd(u[2], bx));
  }
  // kept for the second pass: w = -log a and 1 - r
  static constexpr int kKeep = 2;
  __device__ __forceinline__ void head(float2 u0, float2& nm, float2 (&keep)[kKeep]) const {
    const float2 t = ex2_2(lfma(u0, both(-kLog2e), br)), r = rcp_2(ladd(t, both(1.f))), w = lmul(k, r);
    nm = decay_nm(w);
    keep[0] = lmul(w, both(kLn2));
    keep[1] = lmul(finite(t), r);  // where r is 0, so is all that it multiplies
  }
  __device__ __forceinline__ void grad(const float2 (&u)[G], float2 nm, const float2 (&keep)[kKeep], float2 hp,
                                       float2 lt, float2 (&du)[G], float2& e) const {
    const float2 t = ex2_2(lfma(u[1], both(-kLog2e), bi)), i = rcp_2(ladd(t, both(1.f)));
    // a from w, since 1 + nm is off by 2^-24 of 1, not of a
    const float2 x = ladd(u[2], bx), w = keep[0], a = ex2_2(lmul(w, both(-kLog2e)));
    const float2 s = lmul(neg2(nm), ladd(nm, both(2.f)));  // beta^2
    // 1 / beta; w / beta -> 0 with w
    const float2 rb = make_float2(s.x >= 1.1754944e-38f ? rsqrt_apx(s.x) : 0.f,
                                  s.y >= 1.1754944e-38f ? rsqrt_apx(s.y) : 0.f);
    // r dL/dr = lambda (a^2 i x w / beta - a h_{t-1} w):  d beta = (a^2 / beta) dw
    const float2 lw = lmul(lmul(lt, a), w);
    e = lmul(lw, lfma(lmul(a, rb), lmul(i, x), neg2(hp)));
    du[0] = lmul(e, keep[1]);
    const float2 lb = lmul(lt, lmul(s, rb));
    du[1] = lmul(lmul(lb, x), lmul(lmul(finite(t), i), i));
    du[2] = lmul(lb, i);
  }
  static __device__ __forceinline__ float2 lam_scale(const float* lam, int d) {
    return make_float2(dlog_softplus(lam[d]), dlog_softplus(lam[d + 1]));
  }
};

// h <- (h - m h) + b: the fma rounds (1 - m) h once, m near 1 included
__device__ __forceinline__ float2 lin_step(float2 nm, float2 b, float2 h) { return ladd(lfma(nm, h, h), b); }

// Affine maps h -> P h + Q of consecutive steps, two channels: (Px, Py, Qx, Qy).
// With resets, P < 0 marks a run of steps with one in it: what came before is
// forgotten even where it is infinite or NaN (0 * inf would carry it on).
template <bool kReset>
__device__ __forceinline__ float2 lin_apply(float4 v, float2 h) {
  const float2 n = lfma(make_float2(v.x, v.y), h, make_float2(v.z, v.w));
  if (!kReset) return n;
  return v.x < 0.f ? make_float2(v.z, v.w) : n;  // a reset holds for both channels
}
// the run `a` followed by the run `b`
template <bool kReset>
__device__ __forceinline__ float4 lin_then(float4 a, float4 b) {
  const float2 q = lin_apply<kReset>(b, make_float2(a.z, a.w));
  float2 p = lmul(make_float2(a.x, a.y), make_float2(b.x, b.y));
  if (kReset && (a.x < 0.f || b.x < 0.f)) p = both(-1.f);
  return make_float4(p.x, p.y, q.x, q.y);
}

__device__ __forceinline__ float2 bf16_pair(unsigned v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
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
  float* part;           // adjoint: [B * CL][G or, with dlam, G + 1][D] sums over a CTA's steps
  int B, T, D;
  int ntd;               // tiles of a batch row (set at the launch)
  int* status;           // device word for a wait that ran out, or NULL
  unsigned long long wait_ns;  // bound on a wait for the cluster's maps
  int withhold;          // testing: 8 round + rank that sends no map from that round on; -1: none
};

}  // namespace pararnn
