// block_norm.cu -- the norms around a block fused with its gate and residual
// scale, forward and adjoint.  Per row of D channels, every part optional:
//   n = h rsqrt(mean h^2 + eps) w_post     y = n act(g)
//   s = res + scale y                      x = s rsqrt(mean s^2 + eps) w_pre
// A row stays in the registers of the threads that own it from its first read
// to its last write, so each input is read once and each output written once;
// sums over the row and all arithmetic are fp32, each output is rounded once.
#include <algorithm>

#include "block_norm.cuh"
#include "linrec_cell.cuh"

namespace pararnn {

namespace {

// 8 channels of a row as they lie in memory: 16 bytes of bf16 or 32 of fp32.
struct Raw8 {
  uint4 a, b;
};
__device__ __forceinline__ Raw8 raw_zero() { return {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)}; }
__device__ __forceinline__ Raw8 raw_load(const void* p, long long i, bool f32) {
  Raw8 r = raw_zero();
  const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + i * (f32 ? 4 : 2));
  r.a = q[0];
  if (f32) r.b = q[1];
  return r;
}
__device__ __forceinline__ void raw_get(const Raw8& r, bool f32, float (&v)[8]) {
  const unsigned w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = bf16_pair(w[i]);
    v[2 * i] = f32 ? __uint_as_float(w[2 * i]) : t.x;
    v[2 * i + 1] = f32 ? __uint_as_float(w[2 * i + 1]) : t.y;
  }
}
__device__ __forceinline__ unsigned pack2(float a, float b) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const unsigned*>(&t);
}
__device__ __forceinline__ void store8(void* p, long long i, bool f32, const float (&v)[8]) {
  if (f32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + i) =
        make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
  }
}
__device__ __forceinline__ void vec8(const float* w, int c, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(w + c));
  const float4 b = __ldg(reinterpret_cast<const float4*>(w + c) + 1);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// sig(g) and its complement
__device__ __forceinline__ void sig2(float g, float& q, float& qc) {
  const float t = ex2(-kLog2e * fabsf(g)), pos = rcp(1.f + t), neg = t * pos;
  q = g >= 0.f ? pos : neg;
  qc = g >= 0.f ? neg : pos;
}
__device__ __forceinline__ float act(int kind, float g) {
  float q, qc;
  sig2(g, q, qc);
  return kind == PARARNN_ACT_SILU ? g * q : q;
}
__device__ __forceinline__ void act_grad(int kind, float g, float& v, float& dv) {
  float q, qc;
  sig2(g, q, qc);
  v = kind == PARARNN_ACT_SILU ? g * q : q;
  dv = kind == PARARNN_ACT_SILU ? q * fmaf(g, qc, 1.f) : q * qc;
}

constexpr int kNormMaxWarps = 32;

// Sums over the threads of a row, the same in every thread of it: shuffles in
// a warp, then the warps' sums in warp order.  `buf` alternates between two
// buffers from call to call, so one barrier a call is enough.
template <int NVAL>
__device__ __forceinline__ void row_sum(float (&v)[NVAL], int warps, float (*red)[kNormMaxWarps][2], int& buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < NVAL; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (warps == 1) return;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < NVAL; ++i) red[buf][threadIdx.x >> 5][i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NVAL; ++i) {
    v[i] = 0.f;
    for (int w = 0; w < warps; ++w) v[i] += red[buf][w][i];
  }
  buf ^= 1;
}

// tpr threads a row (a warp, or the whole block), NV x 8 channels a thread.
template <int NV>
__global__ void __launch_bounds__(512) norm_fwd(const NormParams p, const int tpr) {
  __shared__ float red[2][kNormMaxWarps][2];
  const int slot = threadIdx.x / tpr, t = threadIdx.x - slot * tpr, warps = tpr / 32;
  const long long row = (long long)blockIdx.x * (blockDim.x / tpr) + slot;
  if (row >= p.N) return;  // whole warps; blocks of one row never leave here
  int buf = 0;
  const float invD = 1.f / (float)p.D;
  Raw8 rh[NV], rg[NV], rr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = 8 * (i * tpr + t);
    rh[i] = rg[i] = rr[i] = raw_zero();
    if (c < p.D) {
      rh[i] = raw_load(p.h, row * p.ld_h + c, p.h32);
      if (p.g) rg[i] = raw_load(p.g, row * p.ld_g + c, p.g32);
      if (p.res) rr[i] = raw_load(p.res, row * p.ld_r + c, p.r32);
    }
  }
  float y[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) raw_get(rh[i], p.h32, y[i]);
  if (p.w_post) {
    float q[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) q[0] = fmaf(y[i][j], y[i][j], q[0]);
    row_sum(q, warps, red, buf);
    const float k = rsqrtf(fmaf(q[0], invD, p.eps));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * (i * tpr + t);
      if (c < p.D) {
        float w[8];
        vec8(p.w_post, c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[i][j] = y[i][j] * k * w[j];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = 8 * (i * tpr + t);
    if (c >= p.D) continue;
    float v[8];
    if (p.g) {
      raw_get(rg[i], p.g32, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[i][j] *= act(p.act, v[j]);
    }
    if (p.scale) {
      vec8(p.scale, c, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[i][j] *= v[j];
    }
    if (p.res) {
      raw_get(rr[i], p.r32, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[i][j] += v[j];
    }
    if (p.s) store8(p.s, row * p.D + c, p.s32, y[i]);
  }
  if (!p.w_pre) return;
  float q[1] = {0.f};
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) q[0] = fmaf(y[i][j], y[i][j], q[0]);  // 0 past D
  row_sum(q, warps, red, buf);
  const float k = rsqrtf(fmaf(q[0], invD, p.eps));
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = 8 * (i * tpr + t);
    if (c >= p.D) continue;
    float w[8];
    vec8(p.w_pre, c, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[i][j] = y[i][j] * k * w[j];
    store8(p.x, row * p.D + c, p.x32, y[i]);
  }
}

// Adjoint.  Blocks walk over rows; the sums for the [D] weights stay in
// registers and leave once per block.  With sh = s / rms(s), hh = h / rms(h):
//   d = ds + (dx w_pre - sh mean(dx w_pre sh)) / rms(s)      (= dres)
//   dw_pre = sum dx sh,  dscale = sum d y,  d' = d scale,  dg = d' n act'(g)
//   d'' = d' act(g),  dw_post = sum d'' hh
//   dh = (d'' w_post - hh mean(d'' w_post hh)) / rms(h)
template <int NV>
__global__ void __launch_bounds__(512) norm_bwd(const NormParams p, const int tpr) {
  __shared__ float red[2][kNormMaxWarps][2];
  const int slots = blockDim.x / tpr;
  const int slot = threadIdx.x / tpr, t = threadIdx.x - slot * tpr, warps = tpr / 32;
  int buf = 0;
  const float invD = 1.f / (float)p.D;
  float aw[NV][8], as[NV][8], ap[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) aw[i][j] = as[i][j] = ap[i][j] = 0.f;
  for (long long row = (long long)blockIdx.x * slots + slot; row < p.N; row += (long long)gridDim.x * slots) {
    Raw8 rh[NV], rg[NV], rr[NV], rs[NV], rx[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * (i * tpr + t);
      rh[i] = rg[i] = rr[i] = rs[i] = rx[i] = raw_zero();
      if (c < p.D) {
        rh[i] = raw_load(p.h, row * p.ld_h + c, p.h32);
        if (p.g) rg[i] = raw_load(p.g, row * p.ld_g + c, p.g32);
        if (p.res && p.w_pre) rr[i] = raw_load(p.res, row * p.ld_r + c, p.r32);
        if (p.ds) rs[i] = raw_load(p.ds, row * p.ld_ds + c, p.ds32);
        if (p.w_pre) rx[i] = raw_load(p.dx, row * p.ld_dx + c, p.dx32);
      }
    }
    float kh = 1.f;
    if (p.w_post) {
      float q[1] = {0.f};
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float h[8];
        raw_get(rh[i], p.h32, h);
#pragma unroll
        for (int j = 0; j < 8; ++j) q[0] = fmaf(h[j], h[j], q[0]);
      }
      row_sum(q, warps, red, buf);
      kh = rsqrtf(fmaf(q[0], invD, p.eps));
    }
    float d[NV][8], wp[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      raw_get(rs[i], p.ds32, d[i]);
      const int c = 8 * (i * tpr + t);
#pragma unroll
      for (int j = 0; j < 8; ++j) wp[i][j] = 1.f;
      if (p.w_post && c < p.D) vec8(p.w_post, c, wp[i]);
    }
    // y_j of this thread (recomputed where it is needed: cheaper than keeping it)
    auto y_of = [&](int i, int j, const float (&h)[8], const float (&g)[8]) {
      float n = h[j] * kh * wp[i][j];
      return p.g ? n * act(p.act, g[j]) : n;
    };
    if (p.w_pre) {
      float q[2] = {0.f, 0.f};
      float s[NV][8], dx[NV][8];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = 8 * (i * tpr + t);
        float h[8], g[8], r[8], sc[8], w[8];
        raw_get(rh[i], p.h32, h);
        raw_get(rg[i], p.g32, g);
        raw_get(rr[i], p.r32, r);
        raw_get(rx[i], p.dx32, dx[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) sc[j] = w[j] = 1.f;
        if (c < p.D) {
          if (p.scale) vec8(p.scale, c, sc);
          vec8(p.w_pre, c, w);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          s[i][j] = fmaf(sc[j], y_of(i, j, h, g), r[j]);
          q[0] = fmaf(s[i][j], s[i][j], q[0]);
          const float e = dx[i][j] * s[i][j];
          q[1] = fmaf(e, w[j], q[1]);
        }
      }
      row_sum(q, warps, red, buf);
      const float k = rsqrtf(fmaf(q[0], invD, p.eps)), mean = q[1] * k * invD;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = 8 * (i * tpr + t);
        if (c >= p.D) continue;
        float w[8];
        vec8(p.w_pre, c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float sh = s[i][j] * k;
          ap[i][j] = fmaf(dx[i][j], sh, ap[i][j]);
          d[i][j] = fmaf(k, fmaf(dx[i][j], w[j], -sh * mean), d[i][j]);
        }
      }
    }
    float q[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * (i * tpr + t);
      if (c >= p.D) continue;
      if (p.dres) store8(p.dres, row * p.D + c, p.r32, d[i]);
      float h[8], g[8], sc[8], dg[8];
      raw_get(rh[i], p.h32, h);
      raw_get(rg[i], p.g32, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) sc[j] = 1.f;
      if (p.scale) vec8(p.scale, c, sc);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float hh = h[j] * kh, n = hh * wp[i][j];
        float a = 1.f, da = 0.f;
        if (p.g) act_grad(p.act, g[j], a, da);
        as[i][j] = fmaf(d[i][j], n * a, as[i][j]);
        const float e = d[i][j] * sc[j];
        dg[j] = e * n * da;
        d[i][j] = e * a;
        if (p.w_post) {
          aw[i][j] = fmaf(d[i][j], hh, aw[i][j]);
          d[i][j] *= wp[i][j];
          q[0] = fmaf(d[i][j], hh, q[0]);
        }
      }
      if (p.g) store8(p.dg, row * p.D + c, p.g32, dg);
    }
    if (p.w_post) row_sum(q, warps, red, buf);
    const float mean = q[0] * invD;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * (i * tpr + t);
      if (c >= p.D) continue;
      if (p.w_post) {
        float h[8];
        raw_get(rh[i], p.h32, h);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[i][j] = kh * fmaf(-h[j] * kh, mean, d[i][j]);
      }
      store8(p.dh, row * p.D + c, p.h32, d[i]);
    }
  }
  if (!p.part) return;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = 8 * (i * tpr + t);
    if (c >= p.D) continue;
    float* q = p.part + ((size_t)blockIdx.x * slots + slot) * 3 * p.D + c;
    store8(q, 0, true, aw[i]);
    store8(q + p.D, 0, true, as[i]);
    store8(q + 2 * (size_t)p.D, 0, true, ap[i]);
  }
}

// Column sums of part [P][3][D] into up to three [D] vectors, in a fixed order.
__global__ void __launch_bounds__(256) norm_colsum(const float* __restrict__ part, int P, int D, float* o0,
                                                   float* o1, float* o2) {
  __shared__ float s[8][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
  float* const out = blockIdx.y == 0 ? o0 : blockIdx.y == 1 ? o1 : o2;
  if (!out) return;  // the whole block
  float v = 0.f;
  if (c < D)
    for (int i = y; i < P; i += 8) v += part[((size_t)i * 3 + blockIdx.y) * D + c];
  s[y][x] = v;
  __syncthreads();
  if (y == 0 && c < D) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += s[i][x];
    out[c] = v;
  }
}

constexpr int kNormMaxD = 8192;

// threads of a row, of a block and vectors of a thread for D channels
void norm_shape(int D, int& nv, int& tpr, int& threads) {
  nv = D <= 4096 ? 1 : 2;
  tpr = 32 * ((D + 256 * nv - 1) / (256 * nv));
  threads = tpr == 32 ? 256 : tpr;
}

int norm_bwd_blocks(long long N, int D) {
  int nv, tpr, threads;
  norm_shape(D, nv, tpr, threads);
  const int slots = threads / tpr;
  const long long most = 148 * std::max(1, 1024 / threads);
  return (int)std::min<long long>((N + slots - 1) / slots, most);
}

}  // namespace

int norm_max_d() { return kNormMaxD; }

size_t norm_part_floats(long long N, int D) {
  int nv, tpr, threads;
  norm_shape(D, nv, tpr, threads);
  return (size_t)norm_bwd_blocks(N, D) * (threads / tpr) * 3 * D;
}

int launch_norm_fwd(const NormParams& p, cudaStream_t stream) {
  int nv, tpr, threads;
  norm_shape(p.D, nv, tpr, threads);
  const int slots = threads / tpr;
  const unsigned grid = (unsigned)((p.N + slots - 1) / slots);
  if (nv == 1)
    norm_fwd<1><<<grid, threads, 0, stream>>>(p, tpr);
  else
    norm_fwd<2><<<grid, threads, 0, stream>>>(p, tpr);
  return (int)cudaGetLastError();
}

int launch_norm_bwd(NormParams p, float* dw_post, float* dscale, float* dw_pre, cudaStream_t stream) {
  int nv, tpr, threads;
  norm_shape(p.D, nv, tpr, threads);
  if (!dw_post && !dscale && !dw_pre) p.part = nullptr;
  const int blocks = norm_bwd_blocks(p.N, p.D);
  if (nv == 1)
    norm_bwd<1><<<blocks, threads, 0, stream>>>(p, tpr);
  else
    norm_bwd<2><<<blocks, threads, 0, stream>>>(p, tpr);
  int e = (int)cudaGetLastError();
  if (e || !p.part) return e;
  norm_colsum<<<dim3((p.D + 31) / 32, 3), 256, 0, stream>>>(p.part, blocks * (threads / tpr), p.D, dw_post,
                                                            dscale, dw_pre);
  return (int)cudaGetLastError();
}

}  // namespace pararnn
