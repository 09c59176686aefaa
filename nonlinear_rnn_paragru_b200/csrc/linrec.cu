// linrec.cu -- the gated linear recurrence: solve (one scan over the
// sequence), adjoint (one reverse scan) and the single decode step.
//
// Layout of the scans.  A cluster of CL CTAs owns a 64-channel tile of one
// batch row and walks its sequence in rounds of CL x W x K steps (the adjoint
// from the last step to the first): CTA r, warp w, takes K consecutive steps,
// lane l the channels 2l and 2l + 1.  In a round a thread composes its steps'
// maps (P, Q); the W warps' maps meet in shared memory, the CTAs' maps in each
// other's shared memory (asynchronous stores, two buffers in turn), and every
// thread composes what precedes its own steps and applies its maps to that.  The state that enters a round stays in a register of
// every warp.  So each input is read once, each output written once, and
// nothing waits on global memory: no workspace, no flags, no order of blocks.
//
// Every warp copies its own rows into a ring of S rounds in shared memory
// (16-byte cp.async, S - 1 rounds ahead), which keeps HBM busy through the
// rounds' barriers without holding registers.
#include <cooperative_groups.h>

#include <algorithm>

#include "linrec_cell.cuh"

namespace cg = cooperative_groups;

namespace pararnn {
namespace {

constexpr int kLinTile = 64;  // channels of a tile
constexpr int kLinMaxCluster = 8;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// One kind of row in a warp's ring: 64 channels of kBytes each, 16 bytes a
// lane, so an instruction moves kRows rows.
template <int kBytes>
struct Rows {
  static constexpr int kRow = 64 * kBytes;       // bytes of a row
  static constexpr int kLanes = kRow / 16;       // lanes of a row
  static constexpr int kRows = 32 / kLanes;
  static constexpr int kPiece = 16 / kBytes;     // channels of a lane
};

// The warps' maps of a round, and the mbarriers that count the arrival of the
// CTAs' maps; those lie in dynamic shared memory, kLinBufs x CL x 512 bytes.
constexpr int kLinBufs = 2;
template <int W>
struct LinShared {
  float4 warp[2][W][32];
  uint64_t bar[kLinBufs];
};

__device__ __forceinline__ uint32_t map_rank(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// 16 bytes into another CTA of the cluster, counted by the mbarrier there: no
// fence, so the stores of states in flight are not waited for
__device__ __forceinline__ void st_async16(uint32_t addr, uint32_t bar, float4 v) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
      "r"(__float_as_uint(v.x)), "r"(__float_as_uint(v.y)), "r"(__float_as_uint(v.z)), "r"(__float_as_uint(v.w)),
      "r"(bar)
      : "memory");
}

constexpr uint64_t kLinWaitNs = 2000000000ull;

template <int CL, bool kReset>
__device__ __forceinline__ float2 lin_join(const float4* cta, int rpos, int lane, float2& carry) {
  float4 v[CL];
#pragma unroll
  for (int i = 0; i < CL; ++i) v[i] = cta[i * 32 + lane];
  float2 in = carry;
#pragma unroll
  for (int i = 0; i < CL; ++i) {
    if (i == rpos) in = carry;
    carry = lin_apply<kReset>(v[i], carry);
  }
  return in;
}

// Publish the warp's map of round r and return the state that enters this
// thread's steps; `carry`, the state that enters the round, becomes the one
// that leaves it.  Positions (wpos of the warp, rpos of the CTA) run in the
// order of the scan.  Buffers and mbarriers alternate: a CTA can only send the
// maps of round r + 2 after every CTA's of round r + 1 came, which each sends
// after all its warps have read those of round r.  The wait for the cluster is
// bounded; where it runs out the states become NaN.
template <int W, bool kReset>
__device__ __forceinline__ float2 lin_exchange(LinShared<W>& sh, float4* cta, unsigned r, float4 mine, int wpos,
                                               int rpos, int CL, int lane, float2& carry, bool& lost) {
  const int par = r & 1;
  sh.warp[par][wpos][lane] = mine;
  __syncthreads();
  float4 v[W];
#pragma unroll
  for (int i = 0; i < W; ++i) v[i] = sh.warp[par][i][lane];
  float2 in = carry;
  if (CL == 1) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if (i == wpos) in = carry;
      carry = lin_apply<kReset>(v[i], carry);
    }
    return in;
  }
  float4 before = make_float4(1.f, 1.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < W - 1; ++i)
    if (i < wpos) before = i ? lin_then<kReset>(before, v[i]) : v[0];
  if (wpos == W - 1) {
    const float4 all = lin_then<kReset>(before, mine);
    if (lane == 0) mbar_arrive_expect_tx(&sh.bar[par], CL * 512);
    const uint32_t at = smem_u32(&cta[(par * CL + rpos) * 32 + lane]), bar = smem_u32(&sh.bar[par]);
    for (int i = 0; i < CL; ++i) st_async16(map_rank(at, i), map_rank(bar, i), all);
  }
  if (!lost) lost = !mbar_wait_bounded(&sh.bar[par], (r >> 1) & 1, kLinWaitNs);
  const float4* maps = cta + par * CL * 32;
  if (CL == 2)
    in = lin_join<2, kReset>(maps, rpos, lane, carry);
  else if (CL == 4)
    in = lin_join<4, kReset>(maps, rpos, lane, carry);
  else
    in = lin_join<8, kReset>(maps, rpos, lane, carry);
  if (lost) carry = in = both(__int_as_float(0x7fffffff));
  return wpos ? lin_apply<kReset>(before, in) : in;
}

// Before the rounds: the mbarriers, and every CTA of the cluster runs before
// one writes into another.
template <int W>
__device__ __forceinline__ void lin_cluster_start(LinShared<W>& sh, int CL) {
  if (CL == 1) return;
  if (threadIdx.x == 0)
    for (int i = 0; i < kLinBufs; ++i) mbar_init(&sh.bar[i], 1);
  cg::this_cluster().sync();
}

// Shape of a scan kernel: W warps, K steps of a thread in a round, a ring of S
// rounds, at least R CTAs on an SM.
template <int CELL, bool kBF16>
struct FwdShape {
  static constexpr bool kGru = CELL == PARARNN_LIN_GRU;
#ifdef FW
  static constexpr int W = FW, K = FK, S = FS, R = FR;
#else
  static constexpr int W = 8, K = 8, S = kBF16 ? (kGru ? 3 : 4) : (kGru ? 3 : 2), R = kBF16 && kGru ? 3 : 2;
#endif
};

template <int CELL, bool kBF16>
struct FwdRing {
  using U = Rows<kBF16 ? 2 : 4>;
  static constexpr int K = FwdShape<CELL, kBF16>::K, G = LinCell<CELL>::G;
  static constexpr int kRound = K * G * U::kRow;  // bytes of a warp's round
  static constexpr int kWarp = FwdShape<CELL, kBF16>::S * kRound;
  static constexpr int kBytes = FwdShape<CELL, kBF16>::W * kWarp;
};

template <bool kBF16>
__device__ __forceinline__ float2 row_pair(const char* row, int lane) {
  if (kBF16) return bf16_pair(*reinterpret_cast<const unsigned*>(row + 4 * lane));
  return *reinterpret_cast<const float2*>(row + 8 * lane);
}

template <int CELL, bool kBF16, bool kReset>
__global__ void __launch_bounds__(32 * FwdShape<CELL, kBF16>::W, FwdShape<CELL, kBF16>::R)
    linrec_fwd(const LinParams p, const int CL) {
  using Cell = LinCell<CELL>;
  using Shape = FwdShape<CELL, kBF16>;
  using Ring = FwdRing<CELL, kBF16>;
  using U = typename Ring::U;
  constexpr int G = Cell::G, K = Shape::K, W = Shape::W, S = Shape::S, ES = kBF16 ? 2 : 4;
  extern __shared__ __align__(16) char ring[];
  __shared__ LinShared<W> sh;
  const int rank = CL > 1 ? (int)cg::this_cluster().block_rank() : 0;
  const int tile = blockIdx.x / CL;
  const int b = tile / p.ntd, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int dbase = (tile - b * p.ntd) * kLinTile, d0 = dbase + 2 * lane;
  const bool live = d0 < p.D;
  const int d = live ? d0 : p.D - 2;  // idle lanes read parameters that exist
  // copies: this lane's row of an instruction and its piece of the row
  const int crow = lane / U::kLanes, cpiece = lane % U::kLanes;
  const bool cok = dbase + cpiece * U::kPiece < p.D;
  const char* src = static_cast<const char*>(p.u) + (b * p.sb + dbase + cpiece * U::kPiece) * ES;
  const uint32_t dst = smem_u32(ring) + warp * Ring::kWarp + crow * G * U::kRow + cpiece * 16;
  static_assert(K % U::kRows == 0, "whole copies");
  const char* const mine = ring + warp * Ring::kWarp;
  float4* const cta = reinterpret_cast<float4*>(ring + Ring::kBytes);
  const int round = CL * W * K, first = (rank * W + warp) * K;
  auto copy = [&](int t0, int slot) {  // steps t0 .. t0 + K - 1 of this warp
#pragma unroll
    for (int i = 0; i < K; i += U::kRows) {
      const int t = t0 + i + crow;
      if (cok && t < p.T) {
        const char* s = src + t * (p.st * ES);
        const uint32_t o = dst + slot * Ring::kRound + i * G * U::kRow;
#pragma unroll
        for (int q = 0; q < G; ++q) cp_async16(o + q * U::kRow, s + q * (p.sg * ES));
      }
    }
  };
#pragma unroll
  for (int s = 0; s < S - 1; ++s) {
    copy(first + s * round, s);
    cp_async_commit();
  }
  Cell cell;
  cell.init(p.lam, p.bias, p.kappa, p.D, d);
  float2 carry = vec2(p.h0 ? p.h0 + (size_t)b * p.D : nullptr, d);
  const size_t row = (size_t)b * p.T;
  lin_cluster_start(sh, CL);
  bool lost = false;
  int slot = 0;
  unsigned nround = 0;
  for (int base = 0; base < p.T; base += round, ++nround) {
    const int t0 = base + first;
    bool mark = false;  // lane j: a reset at step t0 + j
    if (kReset) mark = lane < K && t0 + lane < p.T && p.reset[row + t0 + lane] != 0;
    cp_async_wait<S - 2>();
    __syncwarp();
    copy(t0 + (S - 1) * round, slot == 0 ? S - 1 : slot - 1);
    cp_async_commit();
    const unsigned resets = kReset ? __ballot_sync(0xffffffffu, mark) : 0u;
    const char* rows = mine + slot * Ring::kRound;
    slot = slot + 1 == S ? 0 : slot + 1;
    // steps past T compute on what the ring holds there: nothing after them is
    // stored
    float2 P[K], Q[K];  // h after step j is P[j] h_in + Q[j]
#pragma unroll
    for (int j = 0; j < K; ++j) {
      float2 u[G], nm, bb;
#pragma unroll
      for (int q = 0; q < G; ++q) u[q] = row_pair<kBF16>(rows + (j * G + q) * U::kRow, lane);
      cell.coef(u, nm, bb);
      P[j] = j ? lfma(nm, P[j - 1], P[j - 1]) : ladd(nm, both(1.f));
      Q[j] = j ? lin_step(nm, bb, Q[j - 1]) : bb;
      if (kReset && ((resets >> j) & 1u)) Q[j] = bb;
    }
    float4 map = make_float4(P[K - 1].x, P[K - 1].y, Q[K - 1].x, Q[K - 1].y);
    if (kReset && resets) map.x = map.y = -1.f;
    const float2 in = lin_exchange<W, kReset>(sh, cta, nround, map, warp, rank, CL, lane, carry, lost);
#pragma unroll
    for (int j = 0; j < K; ++j) {
      if (kReset && (resets & ((2u << j) - 1u))) continue;  // nothing is left of h_in
      Q[j] = lfma(P[j], in, Q[j]);
    }
    float* out = p.h + (row + t0) * p.D + d;
    if (t0 + K <= p.T) {
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (live) *reinterpret_cast<float2*>(out + (size_t)j * p.D) = Q[j];
    } else {
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (live && t0 + j < p.T) *reinterpret_cast<float2*>(out + (size_t)j * p.D) = Q[j];
    }
  }
  cp_async_wait<0>();
}

// Reverse scan: lambda_t = g_t + mu_{t+1}, mu_t = (1 - m_t) lambda_t (0 at a
// reset, and mu_1 = dL/dh0).  Positions run from the last step to the first.
template <int CELL, bool kBF16>
struct BwdShape {
  static constexpr bool kGru = CELL == PARARNN_LIN_GRU;
#ifdef BW
  static constexpr int W = BW, K = BK, S = BS, R = BR;
#else
  static constexpr int W = 8, K = 4, S = kBF16 ? (kGru ? 4 : 3) : (kGru ? 3 : 2), R = 2;
#endif
};

template <int CELL, bool kBF16>
struct BwdRing {
  using U = Rows<kBF16 ? 2 : 4>;
  using F = Rows<4>;
  static constexpr int K = BwdShape<CELL, kBF16>::K, G = LinCell<CELL>::G;
  static constexpr int kH = K * G * U::kRow, kG = kH + K * F::kRow;  // offsets of h_{t-1}, dL/dh
  static constexpr int kRound = kG + K * F::kRow;
  static constexpr int kWarp = BwdShape<CELL, kBF16>::S * kRound;
  static constexpr int kBytes = BwdShape<CELL, kBF16>::W * kWarp;
};

template <int CELL, bool kBF16, bool kBF16Out, bool kReset>
__global__ void __launch_bounds__(32 * BwdShape<CELL, kBF16>::W, BwdShape<CELL, kBF16>::R)
    linrec_bwd(const LinParams p, const int CL) {
  using Cell = LinCell<CELL>;
  using Shape = BwdShape<CELL, kBF16>;
  using Ring = BwdRing<CELL, kBF16>;
  using U = typename Ring::U;
  using F = typename Ring::F;
  constexpr int G = Cell::G, K = Shape::K, W = Shape::W, S = Shape::S, ES = kBF16 ? 2 : 4;
  extern __shared__ __align__(16) char ring[];
  __shared__ LinShared<W> sh;
  const int rank = CL > 1 ? (int)cg::this_cluster().block_rank() : 0;
  const int tile = blockIdx.x / CL;
  const int b = tile / p.ntd, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int dbase = (tile - b * p.ntd) * kLinTile, d0 = dbase + 2 * lane;
  const bool live = d0 < p.D;
  const int d = live ? d0 : p.D - 2;
  const size_t row = (size_t)b * p.T;
  const int crow = lane / U::kLanes, cpiece = lane % U::kLanes;
  const bool cok = dbase + cpiece * U::kPiece < p.D;
  const char* src = static_cast<const char*>(p.u) + (b * p.sb + dbase + cpiece * U::kPiece) * ES;
  static_assert(K % F::kRows == 0, "whole copies");
  const int frow = lane / F::kLanes, fpiece = lane % F::kLanes;
  const bool fok = dbase + fpiece * F::kPiece < p.D;
  const size_t fcol = row * p.D + dbase + fpiece * F::kPiece;
  const uint32_t dst = smem_u32(ring) + warp * Ring::kWarp;
  static_assert(K % U::kRows == 0, "whole copies");
  const char* const mine = ring + warp * Ring::kWarp;
  float4* const cta = reinterpret_cast<float4*>(ring + Ring::kBytes);
  const int round = CL * W * K, first = (rank * W + warp) * K;
  auto copy = [&](int t1, int slot) {  // steps t1 - 1, t1 - 2, ..., t1 - K of this warp
    const uint32_t to = dst + slot * Ring::kRound;
#pragma unroll
    for (int i = 0; i < K; i += U::kRows) {
      const int t = t1 - 1 - i - crow;
      if (cok && t >= 0) {
        const char* s = src + t * (p.st * ES);
        const uint32_t o = to + (i + crow) * G * U::kRow + cpiece * 16;
#pragma unroll
        for (int q = 0; q < G; ++q) cp_async16(o + q * U::kRow, s + q * (p.sg * ES));
      }
    }
#pragma unroll
    for (int i = 0; i < K; i += F::kRows) {
      const int t = t1 - 1 - i - frow;
      const uint32_t o = to + (i + frow) * F::kRow + fpiece * 16;
      if (fok && t >= 0) cp_async16(o + Ring::kG, p.g + fcol + (size_t)t * p.D);
      if (fok && t >= 1) cp_async16(o + Ring::kH, p.h + fcol + (size_t)(t - 1) * p.D);
    }
  };
#pragma unroll
  for (int s = 0; s < S - 1; ++s) {
    copy(p.T - first - s * round, s);
    cp_async_commit();
  }
  Cell cell;
  cell.init(p.lam, p.bias, p.kappa, p.D, d);
  const float2 h0 = vec2(p.h0 ? p.h0 + (size_t)b * p.D : nullptr, d);
  float2 carry = both(0.f);
  float2 sum[G + 1];
#pragma unroll
  for (int q = 0; q <= G; ++q) sum[q] = both(0.f);
  lin_cluster_start(sh, CL);
  bool lost = false;
  int slot = 0;
  unsigned nround = 0;
  for (int end = p.T; end > 0; end -= round, ++nround) {
    const int t1 = end - first;
    bool mark = false;  // lane j: a reset at step t1 - 1 - j
    if (kReset) mark = lane < K && t1 - 1 - lane >= 0 && p.reset[row + t1 - 1 - lane] != 0;
    cp_async_wait<S - 2>();
    __syncwarp();
    copy(t1 - (S - 1) * round, slot == 0 ? S - 1 : slot - 1);
    cp_async_commit();
    const unsigned resets = kReset ? __ballot_sync(0xffffffffu, mark) : 0u;
    const char* rows = mine + slot * Ring::kRound;
    float2 nm[K], P = both(1.f), Q = both(0.f);
#pragma unroll
    for (int j = 0; j < K; ++j) {
      float2 u[G];
#pragma unroll
      for (int q = 0; q < G; ++q) u[q] = row_pair<kBF16>(rows + (j * G + q) * U::kRow, lane);
      nm[j] = cell.nm(u);
      const float2 lt = ladd(row_pair<false>(rows + Ring::kG + j * F::kRow, lane), Q);
      Q = lfma(nm[j], lt, lt);
      P = lfma(nm[j], P, P);
      if (kReset && ((resets >> j) & 1u)) Q = both(0.f);
    }
    if (kReset && resets) P = both(-1.f);
    float2 mu = lin_exchange<W, kReset>(sh, cta, nround, make_float4(P.x, P.y, Q.x, Q.y), warp, rank, CL, lane, carry,
                                        lost);
    float2 add[G + 1];
#pragma unroll
    for (int q = 0; q <= G; ++q) add[q] = both(0.f);
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const int t = t1 - 1 - j;
      if (t < 0) break;  // a warp's steps before the sequence: all that follow too
      const bool rs = kReset && ((resets >> j) & 1u);
      const float2 lt = ladd(row_pair<false>(rows + Ring::kG + j * F::kRow, lane), mu);
      mu = rs ? both(0.f) : lfma(nm[j], lt, lt);
      float2 hp = t == 0 ? h0 : row_pair<false>(rows + Ring::kH + j * F::kRow, lane);
      if (rs) hp = both(0.f);
      float2 u[G], du[G], e;
#pragma unroll
      for (int q = 0; q < G; ++q) u[q] = row_pair<kBF16>(rows + (j * G + q) * U::kRow, lane);
      cell.grad(u, nm[j], hp, lt, du, e);
      const size_t at = ((row + t) * G) * p.D + d;
#pragma unroll
      for (int q = 0; q < G; ++q) {
        add[q] = ladd(add[q], du[q]);
        if (!live) continue;
        if constexpr (kBF16Out)
          *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(p.du) + at + (size_t)q * p.D) =
              __float22bfloat162_rn(du[q]);
        else
          *reinterpret_cast<float2*>(static_cast<float*>(p.du) + at + (size_t)q * p.D) = du[q];
      }
      if (CELL == PARARNN_LIN_DECAY) add[G] = ladd(add[G], e);
      if (t == 0 && p.dh0 && live) {
        p.dh0[(size_t)b * p.D + d] = mu.x;
        p.dh0[(size_t)b * p.D + d + 1] = mu.y;
      }
    }
    // a round's sums first, then the running sums: over long sequences the
    // error grows with the number of rounds only
#pragma unroll
    for (int q = 0; q <= G; ++q) sum[q] = ladd(sum[q], add[q]);
    slot = slot + 1 == S ? 0 : slot + 1;
  }
  cp_async_wait<0>();
  if (!p.part) return;
  if (CELL == PARARNN_LIN_DECAY) sum[G] = lmul(sum[G], Cell::lam_scale(p.lam, d));
  // the warps' sums, in warp order
  __syncthreads();
  float2* const acc = reinterpret_cast<float2*>(ring);  // [warp][G + 1][32]
  static_assert(Ring::kBytes >= W * (G + 1) * 32 * (int)sizeof(float2), "sums fit");
  static_assert(W > G, "a warp for each sum");
#pragma unroll
  for (int q = 0; q <= G; ++q) acc[(warp * (G + 1) + q) * 32 + lane] = sum[q];
  __syncthreads();
  if (warp <= G && live) {
    float2 s = both(0.f);
    for (int i = 0; i < W; ++i) s = ladd(s, acc[(i * (G + 1) + warp) * 32 + lane]);
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
  float2 u[G];
#pragma unroll
  for (int q = 0; q < G; ++q) {
    const char* at = static_cast<const char*>(p.u) + (b * p.sb + q * p.sg + d) * (kBF16 ? 2 : 4);
    u[q] = row_pair<kBF16>(at, 0);
  }
  Cell cell;
  cell.init(p.lam, p.bias, p.kappa, p.D, d);
  float2 nm, bb;
  cell.coef(u, nm, bb);
  const size_t at = (size_t)b * p.D + d;
  const float2 h = lin_step(nm, bb, vec2(h_prev ? h_prev + (size_t)b * p.D : nullptr, d));
  h_next[at] = h.x;
  h_next[at + 1] = h.y;
}

template <typename Kern>
int launch_scan(Kern kern, int threads, int smem, const LinParams& p, int CL, cudaStream_t stream) {
  if (CL > 1) smem += kLinBufs * CL * 512;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return (int)e;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(threads);
  cfg.gridDim = dim3((unsigned)((long long)p.B * p.ntd * CL));
  cfg.dynamicSmemBytes = smem;
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

template <int CELL, bool kBF16>
int launch_fwd_t(const LinParams& p, int CL, cudaStream_t stream) {
  constexpr int threads = 32 * FwdShape<CELL, kBF16>::W, smem = FwdRing<CELL, kBF16>::kBytes;
  return p.reset ? launch_scan(linrec_fwd<CELL, kBF16, true>, threads, smem, p, CL, stream)
                 : launch_scan(linrec_fwd<CELL, kBF16, false>, threads, smem, p, CL, stream);
}

template <int CELL, bool kBF16, bool kBF16Out>
int launch_bwd_t(const LinParams& p, int CL, cudaStream_t stream) {
  constexpr int threads = 32 * BwdShape<CELL, kBF16>::W, smem = BwdRing<CELL, kBF16>::kBytes;
  return p.reset ? launch_scan(linrec_bwd<CELL, kBF16, kBF16Out, true>, threads, smem, p, CL, stream)
                 : launch_scan(linrec_bwd<CELL, kBF16, kBF16Out, false>, threads, smem, p, CL, stream);
}

template <int CELL>
int launch_bwd_c(bool bf16, bool bf16_out, const LinParams& p, int CL, cudaStream_t stream) {
  if (!bf16) return launch_bwd_t<CELL, false, false>(p, CL, stream);
  return bf16_out ? launch_bwd_t<CELL, true, true>(p, CL, stream) : launch_bwd_t<CELL, true, false>(p, CL, stream);
}

// CTAs of a cluster: as many as fill one wave of `per_sm` CTAs on 148 SMs, no
// more than the sequence has rounds of one CTA (`steps`) for.
int cluster_for(int B, int T, int D, int per_sm, int steps) {
  const long long tiles = (long long)B * ((D + kLinTile - 1) / kLinTile);
  int CL = 1;
  while (CL < kLinMaxCluster && 2 * tiles * CL <= 148 * per_sm && T > CL * steps) CL *= 2;
  return CL;
}

template <int CELL>
int fwd_cluster(bool bf16, int B, int T, int D) {
  using H = FwdShape<CELL, true>;
  using F = FwdShape<CELL, false>;
  return bf16 ? cluster_for(B, T, D, H::R, H::W * H::K) : cluster_for(B, T, D, F::R, F::W * F::K);
}

// the same for both types of u, so that the workspace does not depend on it
template <int CELL>
int bwd_cluster(int B, int T, int D) {
  using H = BwdShape<CELL, true>;
  return cluster_for(B, T, D, H::R, H::W * H::K);
}

}  // namespace

int linrec_bwd_cluster(int cell, int B, int T, int D) {
  return cell == PARARNN_LIN_GRU ? bwd_cluster<PARARNN_LIN_GRU>(B, T, D) : bwd_cluster<PARARNN_LIN_DECAY>(B, T, D);
}

long long linrec_most_ctas(int B, int D) {
  return (long long)B * ((D + kLinTile - 1) / kLinTile) * kLinMaxCluster;
}

size_t linrec_part_floats(int cell, int B, int T, int D) {
  return (size_t)B * linrec_bwd_cluster(cell, B, T, D) * (cell == PARARNN_LIN_GRU ? 3 : 4) * D;
}

int launch_linrec_fwd(int cell, bool bf16, LinParams p, cudaStream_t stream) {
  p.ntd = (p.D + kLinTile - 1) / kLinTile;
  if (cell == PARARNN_LIN_GRU) {
    const int CL = fwd_cluster<PARARNN_LIN_GRU>(bf16, p.B, p.T, p.D);
    return bf16 ? launch_fwd_t<PARARNN_LIN_GRU, true>(p, CL, stream)
                : launch_fwd_t<PARARNN_LIN_GRU, false>(p, CL, stream);
  }
  const int CL = fwd_cluster<PARARNN_LIN_DECAY>(bf16, p.B, p.T, p.D);
  return bf16 ? launch_fwd_t<PARARNN_LIN_DECAY, true>(p, CL, stream)
              : launch_fwd_t<PARARNN_LIN_DECAY, false>(p, CL, stream);
}

int launch_linrec_bwd(int cell, bool bf16, bool bf16_out, LinParams p, float* dlam, float* dbias,
                      cudaStream_t stream) {
  const int CL = linrec_bwd_cluster(cell, p.B, p.T, p.D);
  p.ntd = (p.D + kLinTile - 1) / kLinTile;
  if (!dlam && !dbias) p.part = nullptr;
  int e = cell == PARARNN_LIN_GRU ? launch_bwd_c<PARARNN_LIN_GRU>(bf16, bf16_out, p, CL, stream)
                                  : launch_bwd_c<PARARNN_LIN_DECAY>(bf16, bf16_out, p, CL, stream);
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
