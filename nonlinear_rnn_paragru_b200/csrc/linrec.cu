// linrec.cu -- the gated linear recurrence: solve (one scan over the
// sequence), adjoint (one reverse scan) and the single decode step.
//
// Layout of the scans.  A cluster of CL CTAs owns a 64-channel tile of one
// batch row and walks its sequence in rounds of CL x 8 x k steps: CTA r, warp
// w, takes k <= kLinSteps consecutive steps, lane l the channels 2l and 2l + 1.
// In a round a thread forms its steps' coefficients and their composed map
// (P, Q) in registers; the 8 warps' maps meet in shared memory, the CTAs' maps
// in each other's shared memory (one cluster barrier a round, two buffers in
// turn), and every thread composes what precedes its own steps and runs them
// again from the true state.  The state that enters a round is kept in a
// register of every warp.  So u is read once, h written once, and nothing
// waits on global memory: no workspace, no flags, no order of blocks.
#include <cooperative_groups.h>

#include <algorithm>

#include "linrec_cell.cuh"

namespace cg = cooperative_groups;

namespace pararnn {
namespace {

constexpr int kLinThreads = 256;
constexpr int kLinWarps = kLinThreads / 32;
constexpr int kLinSteps = 8;      // steps of a thread in one round
constexpr int kLinTile = 64;      // channels of a tile
constexpr int kLinMaxCluster = 8;

// The maps of a round: per warp, and per CTA of the cluster.
struct LinShared {
  float4 warp[2][kLinWarps][32];
  float4 cta[2][kLinMaxCluster][32];
};

__device__ __forceinline__ void lin_then4(float4& a, const float4& b) {
  lin_then(a.x, a.y, b.x, b.y);
  lin_then(a.z, a.w, b.z, b.w);
}

// Publish the warp's map and return the state that enters this thread's steps;
// `carry` is the state that enters the round, and becomes the one that leaves
// it.  Positions (wpos of the warp, rpos of the CTA) run in the order of the
// scan.
__device__ __forceinline__ float2 lin_exchange(LinShared& sh, int par, float4 mine, int wpos, int rpos,
                                               int CL, int lane, float2& carry) {
  sh.warp[par][wpos][lane] = mine;
  __syncthreads();
  if (CL > 1) {
    cg::cluster_group cl = cg::this_cluster();
    if (wpos < CL) {  // warp position w tells CTA position w
      float4 all = sh.warp[par][0][lane];
#pragma unroll
      for (int i = 1; i < kLinWarps; ++i) lin_then4(all, sh.warp[par][i][lane]);
      *cl.map_shared_rank(&sh.cta[par][rpos][lane], (unsigned)wpos) = all;
    }
    cl.sync();
    float2 in = carry;
    for (int i = 0; i < CL; ++i) {
      if (i == rpos) in = carry;
      const float4 v = sh.cta[par][i][lane];
      carry.x = lin_apply(v.x, v.y, carry.x);
      carry.y = lin_apply(v.z, v.w, carry.y);
    }
#pragma unroll
    for (int i = 0; i < kLinWarps; ++i)
      if (i < wpos) {
        const float4 v = sh.warp[par][i][lane];
        in.x = lin_apply(v.x, v.y, in.x);
        in.y = lin_apply(v.z, v.w, in.y);
      }
    return in;
  }
  float2 in = carry;
#pragma unroll
  for (int i = 0; i < kLinWarps; ++i) {
    if (i == wpos) in = carry;
    const float4 v = sh.warp[par][i][lane];
    carry.x = lin_apply(v.x, v.y, carry.x);
    carry.y = lin_apply(v.z, v.w, carry.y);
  }
  return in;
}

// bit j: the state entering step t0 + j is zero
__device__ __forceinline__ unsigned lin_resets(const unsigned char* reset, size_t row, int t0, int n,
                                               int lane) {
  if (!reset) return 0u;
  const bool r = lane < n && reset[row + t0 + lane] != 0;
  return __ballot_sync(0xffffffffu, r);
}

template <int CELL, bool kBF16>
__global__ void __launch_bounds__(kLinThreads) linrec_fwd(const LinParams p, const int CL) {
  using Cell = LinCell<CELL>;
  constexpr int G = Cell::G, K = kLinSteps;
  __shared__ LinShared sh;
  const int rank = CL > 1 ? (int)cg::this_cluster().block_rank() : 0;
  const int tile = blockIdx.x / CL;
  const int b = tile / p.ntd, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int d0 = (tile - b * p.ntd) * kLinTile + 2 * lane;
  const bool live = d0 < p.D;
  const int d = live ? d0 : p.D - 2;  // idle lanes read a channel pair that exists
  Cell cx, cy;
  cx.init(p.lam, p.bias, p.kappa, p.D, d);
  cy.init(p.lam, p.bias, p.kappa, p.D, d + 1);
  float2 carry = make_float2(0.f, 0.f);
  if (p.h0) {
    const float* q = p.h0 + (size_t)b * p.D + d;
    carry = make_float2(q[0], q[1]);
  }
  const size_t row = (size_t)b * p.T;
  const long long ub = (long long)b * p.sb + d;
  const int k = p.steps, round = CL * kLinWarps * k;
  if (CL > 1) cg::this_cluster().sync();  // every CTA runs before one writes into another
  int par = 0;
  for (int base = 0; base < p.T; base += round, par ^= 1) {
    const int t0 = base + (rank * kLinWarps + warp) * k;
    const int n = max(0, min(k, p.T - t0));
    typename LinRaw<kBF16>::type raw[K][G];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const long long at = ub + (long long)min(t0 + min(j, k - 1), p.T - 1) * p.st;
#pragma unroll
      for (int q = 0; q < G; ++q) raw[j][q] = lin_load<kBF16>(p.u, at + q * p.sg);
    }
    const unsigned resets = lin_resets(p.reset, row, t0, n, lane);
    float4 m[K];  // (m, b) of both channels
    float4 map = make_float4(1.f, 0.f, 1.f, 0.f);
#pragma unroll
    for (int j = 0; j < K; ++j) {
      float ux[G], uy[G];
#pragma unroll
      for (int q = 0; q < G; ++q) {
        const float2 v = LinRaw<kBF16>::get(raw[j][q]);
        ux[q] = v.x;
        uy[q] = v.y;
      }
      float4 c;
      cx.coef(ux, c.x, c.y);
      cy.coef(uy, c.z, c.w);
      if (j >= n) c = make_float4(0.f, 0.f, 0.f, 0.f);  // no step: the identity
      const bool rs = (resets >> j) & 1u;
      map.y = rs ? c.y : fmaf(-c.x, map.y, map.y + c.y);
      map.w = rs ? c.w : fmaf(-c.z, map.w, map.w + c.w);
      map.x = fmaf(-c.x, map.x, map.x);
      map.z = fmaf(-c.z, map.z, map.z);
      m[j] = c;
    }
    if (resets) map.x = map.z = -1.f;
    float2 s = lin_exchange(sh, par, map, warp, rank, CL, lane, carry);
    float* out = p.h + (row + t0) * p.D + d;
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const bool rs = (resets >> j) & 1u;
      s.x = rs ? m[j].y : fmaf(-m[j].x, s.x, s.x + m[j].y);
      s.y = rs ? m[j].w : fmaf(-m[j].z, s.y, s.y + m[j].w);
      if (j < n && live) *reinterpret_cast<float2*>(out + (size_t)j * p.D) = s;
    }
  }
}

// Reverse scan: lambda_t = g_t + mu_{t+1}, mu_t = (1 - m_t) lambda_t (0 at a
// reset, and mu_1 = dL/dh0).  Positions run from the last step to the first.
template <int CELL, bool kBF16, bool kBF16Out>
__global__ void __launch_bounds__(kLinThreads) linrec_bwd(const LinParams p, const int CL) {
  using Cell = LinCell<CELL>;
  constexpr int G = Cell::G, K = kLinSteps;
  __shared__ LinShared sh;
  const int rank = CL > 1 ? (int)cg::this_cluster().block_rank() : 0;
  const int tile = blockIdx.x / CL;
  const int b = tile / p.ntd, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int d0 = (tile - b * p.ntd) * kLinTile + 2 * lane;
  const bool live = d0 < p.D;
  const int d = live ? d0 : p.D - 2;
  Cell cx, cy;
  cx.init(p.lam, p.bias, p.kappa, p.D, d);
  cy.init(p.lam, p.bias, p.kappa, p.D, d + 1);
  const size_t row = (size_t)b * p.T;
  const long long ub = (long long)b * p.sb + d;
  const int k = p.steps, round = CL * kLinWarps * k;
  float2 carry = make_float2(0.f, 0.f);
  float2 sum[G + 1];
#pragma unroll
  for (int q = 0; q <= G; ++q) sum[q] = make_float2(0.f, 0.f);
  if (CL > 1) cg::this_cluster().sync();
  int par = 0;
  for (int end = p.T; end > 0; end -= round, par ^= 1) {
    // this thread's steps, last first: t1 - 1, t1 - 2, ..., t1 - n
    const int t1 = end - (rank * kLinWarps + warp) * k;
    const int n = max(0, min(k, t1));
    typename LinRaw<kBF16>::type raw[K][G];
    float2 hp[K], g[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const int t = max(t1 - 1 - min(j, k - 1), 0);
      const long long at = ub + (long long)t * p.st;
#pragma unroll
      for (int q = 0; q < G; ++q) raw[j][q] = lin_load<kBF16>(p.u, at + q * p.sg);
      g[j] = __ldg(reinterpret_cast<const float2*>(p.g + (row + t) * p.D + d));
      if (t > 0)
        hp[j] = __ldg(reinterpret_cast<const float2*>(p.h + (row + t - 1) * p.D + d));
      else if (p.h0)
        hp[j] = make_float2(p.h0[(size_t)b * p.D + d], p.h0[(size_t)b * p.D + d + 1]);
      else
        hp[j] = make_float2(0.f, 0.f);
    }
    unsigned resets = 0u;  // bit j: step t1 - 1 - j
    if (p.reset)
      resets = __ballot_sync(0xffffffffu, lane < n && p.reset[row + t1 - 1 - min(lane, n - 1)] != 0);
    float2 m[K];
    float4 map = make_float4(1.f, 0.f, 1.f, 0.f);
#pragma unroll
    for (int j = 0; j < K; ++j) {
      float ux[G], uy[G];
#pragma unroll
      for (int q = 0; q < G; ++q) {
        const float2 v = LinRaw<kBF16>::get(raw[j][q]);
        ux[q] = v.x;
        uy[q] = v.y;
      }
      m[j] = make_float2(cx.forget(ux), cy.forget(uy));
      if (j >= n) m[j] = g[j] = make_float2(0.f, 0.f);
      const bool rs = (resets >> j) & 1u;
      const float lx = g[j].x + map.y, ly = g[j].y + map.w;
      map.y = rs ? 0.f : fmaf(-m[j].x, lx, lx);
      map.w = rs ? 0.f : fmaf(-m[j].y, ly, ly);
      map.x = fmaf(-m[j].x, map.x, map.x);
      map.z = fmaf(-m[j].y, map.z, map.z);
    }
    if (resets) map.x = map.z = -1.f;
    float2 mu = lin_exchange(sh, par, map, warp, rank, CL, lane, carry);
    float2 add[G + 1];
#pragma unroll
    for (int q = 0; q <= G; ++q) add[q] = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const bool rs = (resets >> j) & 1u;
      const float lx = g[j].x + mu.x, ly = g[j].y + mu.y;
      mu.x = rs ? 0.f : fmaf(-m[j].x, lx, lx);
      mu.y = rs ? 0.f : fmaf(-m[j].y, ly, ly);
      float ux[G], uy[G], dx[G], dy[G], ex, ey;
#pragma unroll
      for (int q = 0; q < G; ++q) {
        const float2 v = LinRaw<kBF16>::get(raw[j][q]);
        ux[q] = v.x;
        uy[q] = v.y;
      }
      cx.grad(ux, rs ? 0.f : hp[j].x, lx, dx, ex);
      cy.grad(uy, rs ? 0.f : hp[j].y, ly, dy, ey);
      if (j < n && live) {
        const size_t at = ((row + t1 - 1 - j) * G) * p.D + d;
#pragma unroll
        for (int q = 0; q < G; ++q) {
          if constexpr (kBF16Out)
            *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(p.du) + at + (size_t)q * p.D) =
                __floats2bfloat162_rn(dx[q], dy[q]);
          else
            *reinterpret_cast<float2*>(static_cast<float*>(p.du) + at + (size_t)q * p.D) =
                make_float2(dx[q], dy[q]);
          add[q].x += dx[q];
          add[q].y += dy[q];
        }
        add[G].x += ex;
        add[G].y += ey;
      }
    }
    // a round's sums first, then the running sums: over long sequences the
    // error grows with the number of rounds only
#pragma unroll
    for (int q = 0; q <= G; ++q) {
      sum[q].x += add[q].x;
      sum[q].y += add[q].y;
    }
  }
  if (p.dh0 && rank == 0 && warp == 0 && live) {
    p.dh0[(size_t)b * p.D + d] = carry.x;
    p.dh0[(size_t)b * p.D + d + 1] = carry.y;
  }
  if (!p.part) return;
  sum[G].x *= cx.lam_scale(p.lam, d);
  sum[G].y *= cy.lam_scale(p.lam, d + 1);
  // the 8 warps' sums, in warp order
  __syncthreads();
  float2* const acc = reinterpret_cast<float2*>(&sh);  // [warp][G + 1][32]
  static_assert(sizeof(LinShared) >= kLinWarps * 4 * 32 * sizeof(float2), "sums fit");
#pragma unroll
  for (int q = 0; q <= G; ++q) acc[(warp * (G + 1) + q) * 32 + lane] = sum[q];
  __syncthreads();
  if (warp <= G && live) {
    float2 s = make_float2(0.f, 0.f);
    for (int i = 0; i < kLinWarps; ++i) {
      const float2 v = acc[(i * (G + 1) + warp) * 32 + lane];
      s.x += v.x;
      s.y += v.y;
    }
    float* q = p.part + ((size_t)(b * CL + rank) * (G + 1) + warp) * p.D + d;
    q[0] = s.x;
    q[1] = s.y;
  }
}

// Sums of the rows of part [P][C], in a fixed order: 32 columns a block, 8
// threads a column.  Columns [0, c1) go to out1, the rest to out2 (either may
// be NULL).
__global__ void __launch_bounds__(256) linrec_colsum(const float* __restrict__ part, int P, int C, int c1,
                                                     float* out1, float* out2) {
  __shared__ float s[8][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
  float v = 0.f;
  if (c < C)
    for (int i = y; i < P; i += 8) v += part[(size_t)i * C + c];
  s[y][x] = v;
  __syncthreads();
  if (y == 0 && c < C) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += s[i][x];
    if (c < c1) {
      if (out1) out1[c] = v;
    } else if (out2) {
      out2[c - c1] = v;
    }
  }
}

// One decode step: a thread owns two channels of one row; h_prev may be h_next.
template <int CELL, bool kBF16>
__global__ void __launch_bounds__(256) linrec_step(const LinParams p, const float* h_prev, float* h_next) {
  using Cell = LinCell<CELL>;
  constexpr int G = Cell::G;
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= (long long)p.B * (p.D / 2)) return;
  const int b = (int)(i / (p.D / 2)), d = 2 * (int)(i - (long long)b * (p.D / 2));
  float ux[G], uy[G];
#pragma unroll
  for (int q = 0; q < G; ++q) {
    const float2 v = LinRaw<kBF16>::get(lin_load<kBF16>(p.u, b * p.sb + q * p.sg + d));
    ux[q] = v.x;
    uy[q] = v.y;
  }
  Cell cx, cy;
  cx.init(p.lam, p.bias, p.kappa, p.D, d);
  cy.init(p.lam, p.bias, p.kappa, p.D, d + 1);
  float mx, bx, my, by;
  cx.coef(ux, mx, bx);
  cy.coef(uy, my, by);
  const size_t at = (size_t)b * p.D + d;
  const float hx = h_prev ? h_prev[at] : 0.f, hy = h_prev ? h_prev[at + 1] : 0.f;
  h_next[at] = fmaf(-mx, hx, hx + bx);
  h_next[at + 1] = fmaf(-my, hy, hy + by);
}

template <typename Kern>
int launch_scan(Kern kern, const LinParams& p, int CL, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kLinThreads);
  cfg.gridDim = dim3((unsigned)((long long)p.B * p.ntd * CL));
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CL;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CL > 1 ? 1 : 0;
  return (int)cudaLaunchKernelEx(&cfg, kern, p, CL);
}

}  // namespace

// CTAs of a cluster: enough for two CTAs on each of 148 SMs, no more than the
// sequence has 8-step pieces for.
int linrec_cluster(int B, int T, int D) {
  const long long tiles = (long long)B * ((D + kLinTile - 1) / kLinTile);
  int CL = 1;
  while (CL < kLinMaxCluster && tiles * CL < 2 * 148 && T > CL * kLinWarps * kLinSteps) CL *= 2;
  return CL;
}

long long linrec_ctas(int B, int T, int D) {
  return (long long)B * ((D + kLinTile - 1) / kLinTile) * linrec_cluster(B, T, D);
}

size_t linrec_part_floats(int cell, int B, int T, int D) {
  return (size_t)B * linrec_cluster(B, T, D) * (cell == PARARNN_LIN_GRU ? 3 : 4) * D;
}

static void lin_shape(LinParams& p, int CL) {
  p.ntd = (p.D + kLinTile - 1) / kLinTile;
  const long long lanes = (long long)CL * kLinWarps;
  p.steps = (int)std::min<long long>(kLinSteps, (p.T + lanes - 1) / lanes);
}

int launch_linrec_fwd(int cell, bool bf16, LinParams p, cudaStream_t stream) {
  const int CL = linrec_cluster(p.B, p.T, p.D);
  lin_shape(p, CL);
  if (cell == PARARNN_LIN_GRU)
    return bf16 ? launch_scan(linrec_fwd<PARARNN_LIN_GRU, true>, p, CL, stream)
                : launch_scan(linrec_fwd<PARARNN_LIN_GRU, false>, p, CL, stream);
  return bf16 ? launch_scan(linrec_fwd<PARARNN_LIN_DECAY, true>, p, CL, stream)
              : launch_scan(linrec_fwd<PARARNN_LIN_DECAY, false>, p, CL, stream);
}

template <int CELL>
static int launch_bwd_t(bool bf16, bool bf16_out, const LinParams& p, int CL, cudaStream_t stream) {
  if (!bf16) return launch_scan(linrec_bwd<CELL, false, false>, p, CL, stream);
  return bf16_out ? launch_scan(linrec_bwd<CELL, true, true>, p, CL, stream)
                  : launch_scan(linrec_bwd<CELL, true, false>, p, CL, stream);
}

int launch_linrec_bwd(int cell, bool bf16, bool bf16_out, LinParams p, float* dlam, float* dbias,
                      cudaStream_t stream) {
  const int CL = linrec_cluster(p.B, p.T, p.D);
  lin_shape(p, CL);
  if (!dlam && !dbias) p.part = nullptr;
  int e = cell == PARARNN_LIN_GRU ? launch_bwd_t<PARARNN_LIN_GRU>(bf16, bf16_out, p, CL, stream)
                                  : launch_bwd_t<PARARNN_LIN_DECAY>(bf16, bf16_out, p, CL, stream);
  if (e || !p.part) return e;
  const int G = cell == PARARNN_LIN_GRU ? 2 : 3;
  const int C = (G + 1) * p.D;
  linrec_colsum<<<(C + 31) / 32, 256, 0, stream>>>(p.part, p.B * CL, C, G * p.D, dbias, dlam);
  return (int)cudaGetLastError();
}

int launch_linrec_step(int cell, bool bf16, const LinParams& p, const float* h_prev, float* h_next,
                       cudaStream_t stream) {
  const int threads = 128;
  const long long n = (long long)p.B * (p.D / 2);
  const unsigned grid = (unsigned)((n + threads - 1) / threads);
  if (cell == PARARNN_LIN_GRU) {
    if (bf16)
      linrec_step<PARARNN_LIN_GRU, true><<<grid, threads, 0, stream>>>(p, h_prev, h_next);
    else
      linrec_step<PARARNN_LIN_GRU, false><<<grid, threads, 0, stream>>>(p, h_prev, h_next);
  } else {
    if (bf16)
      linrec_step<PARARNN_LIN_DECAY, true><<<grid, threads, 0, stream>>>(p, h_prev, h_next);
    else
      linrec_step<PARARNN_LIN_DECAY, false><<<grid, threads, 0, stream>>>(p, h_prev, h_next);
  }
  return (int)cudaGetLastError();
}

}  // namespace pararnn
