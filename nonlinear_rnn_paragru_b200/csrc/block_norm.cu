// block_norm.cu -- the norms around a block fused with its gate and residual
// scale, forward and adjoint.  Per row of D channels, every part optional:
//   n = h rsqrt(mean h^2 + eps) w_post     y = n act(g)
//   s = res + scale y                      x = s rsqrt(mean s^2 + eps) w_pre
// A row stays in the registers of the threads that own it from its first read
// to its last write, so each input is read once and each output written once;
// sums over the row and all arithmetic are fp32 (two channels an instruction),
// each output is rounded once.
//
// Blocks walk over rows: `tpr` threads a row of 8 NV channels each (a power of
// two up to a warp for D <= 256, several rows a block; else the whole block),
// and a thread loads its share of the next row before it works on this one, so
// that HBM stays busy through the row's two sums.
//
// Measured (B200, device time, warm): all parts, fp32 states, the rest bf16: N32768
// D1024 forward 65.5 us (403 MB: 6.1 TB/s, held by HBM), adjoint 139 us; N8192
// D4096 adjoint 141 us (671 MB: 4.8 TB/s).  The adjoint is held by its instructions
// (some 88 a channel of a thread, issued in 60% of the cycles) and the latency of a
// row's phases in the 16 warps that the registers (weights and their sums: 48)
// leave an SM.  Rows past 4096 channels spill: N4096 D8192 213 us.
#include <algorithm>
#include <utility>

#include "block_norm.cuh"
#include "colsum.cuh"
#include "linrec_cell.cuh"
#include "smem_once.cuh"

namespace pararnn {
namespace {

// Types of the tensors: a kernel for every combination in common use, with
// the types known to the compiler, and one (kAnyType) that looks at the
// parameters.  Bits: h, gate, res, s (or ds), x (or dx) are fp32.
constexpr int kH32 = 1, kG32 = 2, kR32 = 4, kS32 = 8, kX32 = 16, kAnyType = -1;
template <int TP>
__device__ __forceinline__ bool f32(const NormParams& p, int bit) {
  return ((TP == kAnyType ? p.types : TP) & bit) != 0;
}

// Parts that a call has, alike: known to the compiler for those in common use.
constexpr int kPost = 1, kGate = 2, kRes = 4, kScale = 8, kPre = 16, kDs = 32, kAnyPart = -1;
template <int PT>
__device__ __forceinline__ bool has(const NormParams& p, int bit) {
  return ((PT == kAnyPart ? p.parts : PT) & bit) != 0;
}

// 8 channels of a row as they lie in memory: 16 bytes of bf16 or 32 of fp32.
struct Raw8 {
  uint4 a, b;
};
__device__ __forceinline__ Raw8 raw_load(const void* p, long long i, bool f32, bool ok) {
  Raw8 r = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + i * (f32 ? 4 : 2));
  if (ok) r.a = q[0];
  if (ok && f32) r.b = q[1];
  return r;
}
struct F8 {
  float2 v[4];
};
__device__ __forceinline__ float2 bits2(unsigned x, unsigned y) {
  return make_float2(__uint_as_float(x), __uint_as_float(y));
}
__device__ __forceinline__ F8 raw_get(const Raw8& r, bool f32) {
  if (f32) return {bits2(r.a.x, r.a.y), bits2(r.a.z, r.a.w), bits2(r.b.x, r.b.y), bits2(r.b.z, r.b.w)};
  return {bf16_pair(r.a.x), bf16_pair(r.a.y), bf16_pair(r.a.z), bf16_pair(r.a.w)};
}
__device__ __forceinline__ unsigned pack2(float2 v) {
  const __nv_bfloat162 t = __float22bfloat162_rn(v);
  return *reinterpret_cast<const unsigned*>(&t);
}
__device__ __forceinline__ void store8(void* p, long long i, bool f32, const F8& x) {
  if (f32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(x.v[0].x, x.v[0].y, x.v[1].x, x.v[1].y);
    q[1] = make_float4(x.v[2].x, x.v[2].y, x.v[3].x, x.v[3].y);
  } else {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + i) =
        make_uint4(pack2(x.v[0]), pack2(x.v[1]), pack2(x.v[2]), pack2(x.v[3]));
  }
}
// 8 weights from channel c on; ones where there are none
__device__ __forceinline__ F8 weights(const float* w, int c, bool ok) {
  F8 r = {both(1.f), both(1.f), both(1.f), both(1.f)};
  if (w && ok) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(w + c));
    const float4 b = __ldg(reinterpret_cast<const float4*>(w + c) + 1);
    r = {make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y), make_float2(b.z, b.w)};
  }
  return r;
}

// The gate: act(g) = f s with s = sig(g) and f = g (silu) or 1.
struct Act {
  bool silu;
  __device__ __forceinline__ float2 factor(float2 g) const { return silu ? g : both(1.f); }
  __device__ __forceinline__ float2 operator()(float2 g) const {
    return lmul(factor(g), rcp_2(ladd(ex2_2(lmul(g, both(-kLog2e))), both(1.f))));
  }
  // and act'(g) = f s (1 - s) (+ s for silu), 1 - s = t s of its own size where
  // s is near 1 too (t = e^-g, kept finite: s is 0 where it overflows)
  __device__ __forceinline__ void grad(float2 g, float2& a, float2& da) const {
    const float2 t = ex2_2(lmul(g, both(-kLog2e))), s = rcp_2(ladd(t, both(1.f))), f = factor(g);
    const float2 ts = lmul(finite(t), s);
    a = lmul(f, s);
    da = lfma(a, ts, silu ? s : both(0.f));
  }
};

constexpr int kNormWarps = 16;  // of a block, at most
struct NormShared {
  float red[2][kNormWarps];
};
// entries of warps that a block does not have stay zero
__device__ __forceinline__ void norm_start(NormShared& sh) {
  if (threadIdx.x < 2 * kNormWarps) (&sh.red[0][0])[threadIdx.x] = 0.f;
  __syncthreads();
}

// The sum over the threads of a row, the same in every thread of it: shuffles in
// a warp, then over the warps' sums.  `buf` alternates from call to call, so
// one barrier a call is enough.
__device__ __forceinline__ float row_sum(float v, int tpr, NormShared& sh, int& buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < tpr) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (tpr <= 32) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) sh.red[buf][threadIdx.x >> 5] = v;
  __syncthreads();
  v = sh.red[buf][lane & (kNormWarps - 1)];
#pragma unroll
  for (int o = kNormWarps / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  buf ^= 1;
  return v;
}
// Six sums at once.  A warp's two halves take three of them each
// after the first exchange, so 30 shuffles do what 54 would.
struct NormShared6 {
  float red[2][6][kNormWarps];
};
template <bool kNarrow>
__device__ __forceinline__ void row_sum6(float (&v)[6], int tpr, NormShared6& sh, int& buf) {
  if (kNarrow) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (o < tpr)
#pragma unroll
        for (int i = 0; i < 6; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    return;
  }
  const int lane = threadIdx.x & 31, w = lane & (kNormWarps - 1);
  const bool high = lane >= 16;
  float h[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const float give = high ? v[i] : v[i + 3];
    h[i] = (high ? v[i + 3] : v[i]) + __shfl_xor_sync(0xffffffffu, give, 16);
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < 3; ++i) h[i] += __shfl_xor_sync(0xffffffffu, h[i], o);
  float(*red)[kNormWarps] = sh.red[buf] + (high ? 3 : 0);
  if (w == 0)
#pragma unroll
    for (int i = 0; i < 3; ++i) red[i][threadIdx.x >> 5] = h[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 3; ++i) h[i] = red[i][w];
#pragma unroll
  for (int o = 8; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < 3; ++i) h[i] += __shfl_xor_sync(0xffffffffu, h[i], o);
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const float other = __shfl_xor_sync(0xffffffffu, h[i], 16);
    v[i] = high ? other : h[i];
    v[i + 3] = high ? h[i] : other;
  }
  buf ^= 1;
}
__device__ __forceinline__ float dot8(const F8& a, const F8& b, float acc) {
  float2 q = make_float2(acc, 0.f);
#pragma unroll
  for (int j = 0; j < 4; ++j) q = lfma(a.v[j], b.v[j], q);
  return q.x + q.y;
}

template <int NV>
struct FwdRow {
  Raw8 h[NV], g[NV], r[NV];
};

template <int NV, int TP>
__global__ void __launch_bounds__(512) norm_fwd(const NormParams p, const int tpr) {
  __shared__ __align__(16) NormShared sh;
  const int slots = blockDim.x / tpr, slot = threadIdx.x / tpr, t = threadIdx.x % tpr;
  const long long step = (long long)gridDim.x * slots;
  const float invD = 1.f / (float)p.D;
  const Act act = {p.act == PARARNN_ACT_SILU};
  int buf = 0;
  norm_start(sh);
  auto load = [&](long long row, FwdRow<NV>& x) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * (i * tpr + t);
      const bool ok = c < p.D && row < p.N;
      x.h[i] = raw_load(p.h, row * p.ld_h + c, f32<TP>(p, kH32), ok);
      x.g[i] = raw_load(p.g, row * p.ld_g + c, f32<TP>(p, kG32), ok && p.g);
      x.r[i] = raw_load(p.res, row * p.ld_r + c, f32<TP>(p, kR32), ok && p.res);
    }
  };
  FwdRow<NV> cur, nxt;
  long long row = (long long)blockIdx.x * slots + slot;
  load(row, cur);
  // every thread of a block makes the same rounds; rows past N hold zeros
  for (long long r0 = (long long)blockIdx.x * slots; r0 < p.N; r0 += step, row += step) {
    load(row + step, nxt);
    F8 y[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) y[i] = raw_get(cur.h[i], f32<TP>(p, kH32));
    float2 k = both(1.f);
    if (p.w_post) {
      float q = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) q = dot8(y[i], y[i], q);
      k = both(rsqrtf(fmaf(row_sum(q, tpr, sh, buf), invD, p.eps)));
    }
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * (i * tpr + t);
      const bool ok = c < p.D && row < p.N;
      if (p.w_post) {
        const F8 w = weights(p.w_post, c, ok);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[i].v[j] = lmul(lmul(y[i].v[j], k), w.v[j]);
      }
      if (p.g) {
        const F8 g = raw_get(cur.g[i], f32<TP>(p, kG32));
#pragma unroll
        for (int j = 0; j < 4; ++j) y[i].v[j] = lmul(y[i].v[j], act(g.v[j]));
      }
      const F8 r = raw_get(cur.r[i], f32<TP>(p, kR32)), sc = weights(p.scale, c, ok);
#pragma unroll
      for (int j = 0; j < 4; ++j) y[i].v[j] = lfma(y[i].v[j], sc.v[j], r.v[j]);
      if (p.s && ok) store8(p.s, row * p.D + c, f32<TP>(p, kS32), y[i]);
      q = dot8(y[i], y[i], q);
    }
    if (p.w_pre) {
      const float2 ks = both(rsqrtf(fmaf(row_sum(q, tpr, sh, buf), invD, p.eps)));
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = 8 * (i * tpr + t);
        const bool ok = c < p.D && row < p.N;
        const F8 w = weights(p.w_pre, c, ok);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[i].v[j] = lmul(lmul(y[i].v[j], ks), w.v[j]);
        if (ok) store8(p.x, row * p.D + c, f32<TP>(p, kX32), y[i]);
      }
    }
    cur = nxt;
  }
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// `bytes` (a multiple of 16) into shared memory, counted by `bar`
__device__ __forceinline__ void copy_bulk(uint32_t dst, const void* src, unsigned bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// One tensor of the adjoint's ring: the next row to copy (of a narrow row, this
// thread's channels of it), the bytes to the one after, and where it lies in a
// slot.
struct RingTensor {
  const char* at;
  long long step;
  int offset;
};

// Adjoint.  With sh = s / rms(s), hh = h / rms(h):
//   d = ds + (dx w_pre - sh mean(dx w_pre sh)) / rms(s)      (= dres)
//   dw_pre = sum dx sh,  dscale = sum d y,  d' = d scale,  dg = d' n act'(g)
//   d'' = d' act(g),  dw_post = sum d'' hh
//   dh = (d'' w_post - hh mean(d'' w_post hh)) / rms(h)
// d'' w_post hh is d z with z = scale y, and d is linear in what the second
// norm's sums give, so one exchange serves a row: sums of s^2, s e, ds z, e z
// and s z (e = dx w_pre), and of the next row's h^2.
//
// Rows to come wait in a ring of `S` rows in shared memory, from where threads
// read what they need: five tensors of a row and a row ahead do not fit beside
// the weights and their sums in the registers.  A row that is the block's comes
// by one bulk copy a tensor, which thread 0 issues after the exchange that ends
// the last use of its slot; of narrow rows (kNarrow: of a warp at most, several
// a block) every thread copies its own channels.  The sums leave once per block.
template <int NV, bool kNarrow, int TP, int PT>
__global__ void __launch_bounds__(512) norm_bwd(const NormParams p, const int tpr, const int S) {
  extern __shared__ __align__(16) char smem[];
  __shared__ __align__(16) NormShared6 sh;
  __shared__ uint64_t full[4];
  const int threads = blockDim.x, slots = kNarrow ? threads / tpr : 1, slot = kNarrow ? threadIdx.x / tpr : 0;
  const int t = kNarrow ? threadIdx.x % tpr : threadIdx.x;
  const long long step = (long long)gridDim.x * slots;
  const float invD = 1.f / (float)p.D;
  const Act act = {p.act == PARARNN_ACT_SILU};
  int buf = 0;
  long long row = (long long)blockIdx.x * slots + slot;
  const bool post = has<PT>(p, kPost), gate = has<PT>(p, kGate), pre = has<PT>(p, kPre), res = has<PT>(p, kRes),
             sum = res && pre, scale = has<PT>(p, kScale), dsum = has<PT>(p, kDs);
  int bytes = 0;  // of a slot of the ring
  auto tensor = [&](const void* q, long long ld, int bit, bool on) {
    const int es = f32<TP>(p, bit) ? 4 : 2;
    RingTensor r = {static_cast<const char*>(q) + (row * ld + (kNarrow ? 8 * t : 0)) * es, step * ld * es, bytes};
    if (on) bytes += (kNarrow ? 8 * threads : p.D) * es;
    return r;
  };
  RingTensor th = tensor(p.h, p.ld_h, kH32, true), tg = tensor(p.g, p.ld_g, kG32, gate),
             tr = tensor(p.res, p.ld_r, kR32, sum), ts = tensor(p.ds, p.ld_ds, kS32, dsum),
             tx = tensor(p.dx, p.ld_dx, kX32, pre);
  if (!kNarrow && threadIdx.x < 4) mbar_init(&full[threadIdx.x], 1);
  if (threadIdx.x < kNormWarps)
    for (int i = 0; i < 12; ++i) (&sh.red[0][0][0])[i * kNormWarps + threadIdx.x] = 0.f;
  __syncthreads();
  F8 wreg[3];  // of one vector; two vectors a thread read them again for each row
  if (NV == 1) {
    wreg[0] = weights(p.w_post, 8 * t, 8 * t < p.D);
    wreg[1] = weights(p.scale, 8 * t, 8 * t < p.D);
    wreg[2] = weights(p.w_pre, 8 * t, 8 * t < p.D);
  }
  auto weight = [&](int k, int i) {
    if (NV == 1) return wreg[k];
    const int c = 8 * (i * tpr + t);
    return weights(k == 0 ? p.w_post : k == 1 ? p.scale : p.w_pre, c, c < p.D);
  };
  const uint32_t base = smem_u32(smem);
  auto copy1 = [&](RingTensor& r, int bit, bool on, bool in, int k) {
    if (!on) return;
    const int es = f32<TP>(p, bit) ? 4 : 2;
    if (!kNarrow) {
      if (in) copy_bulk(base + k * bytes + r.offset, r.at, p.D * es, &full[k]);
    } else {
      const int to = k * bytes + r.offset + 8 * threadIdx.x * es;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (i == 0 || es == 4) {
          // past D and N there are zeros
          if (in && 8 * t < p.D)
            copy16(base + to + 16 * i, r.at + 16 * i);
          else
            *reinterpret_cast<uint4*>(smem + to + 16 * i) = make_uint4(0, 0, 0, 0);
        }
    }
    r.at += r.step;
  };
  constexpr unsigned kNever = 0xffffffffu;
  unsigned lost_at = kNever;  // the row whose wait ran out
  auto copy = [&](long long row, int k) {  // the next row, into slot k
    const bool in = row < p.N && (kNarrow || (row != p.withhold && lost_at == kNever));
    if (!kNarrow && in) mbar_arrive_expect_tx(&full[k], bytes);
    copy1(th, kH32, true, in, k);
    copy1(tg, kG32, gate, in, k);
    copy1(tr, kR32, sum, in, k);
    copy1(ts, kS32, dsum, in, k);
    copy1(tx, kX32, pre, in, k);
    if (kNarrow) asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto get = [&](const RingTensor& r, int bit, int i, int k, bool on = true) {
    const int c = 8 * (i * tpr + t), es = f32<TP>(p, bit) ? 4 : 2;
    Raw8 v = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (on && (kNarrow || c < p.D)) {
      const uint4* q = reinterpret_cast<const uint4*>(smem + k * bytes + r.offset + (kNarrow ? 8 * threadIdx.x : c) * es);
      v.a = q[0];
      if (es == 4) v.b = q[1];
    }
    return raw_get(v, es == 4);
  };
  // Until row r is in slot k; of narrow rows, all but the S - 2 latest copies.
  // A thread whose wait runs out is lost: it waits no more, its part of the rows'
  // sums is NaN from there on (so all that depends on them is, in every thread),
  // it fills its own channels with NaN at the end, and thread 0 copies no more.
  auto wait = [&](unsigned r, int k) {
    if (!kNarrow) {
      if (lost_at == kNever && !mbar_wait_bounded(&full[k], (r / S) & 1, p.wait_ns)) lost_at = r;
    } else if (S == 4) {
      asm volatile("cp.async.wait_group 2;" ::: "memory");
    } else if (S == 3) {
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
  };
  auto squares = [&](int k) {
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const F8 h = get(th, kH32, i, k);
      q = dot8(h, h, q);
    }
    return q;
  };
  F8 aw[NV], as[NV], ap[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) aw[i].v[j] = as[i].v[j] = ap[i].v[j] = both(0.f);
  // the rows of the ring, but one slot for which the first exchange must pass
  if (kNarrow || threadIdx.x == 0)
    for (int k = 0; k < S - 1; ++k) copy(row + k * step, k);
  float kh1 = 1.f;  // 1 / rms(h) of the row at hand
  auto first_norm = [&](unsigned r, int k) {
    wait(r, k);
    float q[6] = {lost_at != kNever ? __int_as_float(0x7fffffff) : squares(k), 0.f, 0.f, 0.f, 0.f, 0.f};
    row_sum6<kNarrow>(q, tpr, sh, buf);
    kh1 = rsqrtf(fmaf(q[0], invD, p.eps));
  };
  // The next row's h^2 can only join this row's exchange where the next row is
  // on its way before it: with three slots, as the one freed by an exchange takes
  // the row S - 1 ahead (narrow rows are copied before it).  Else a row has an
  // exchange of its own for it.
  const bool join = kNarrow || S >= 3;
  if (post && join) first_norm(0, 0);
  int at = 0;  // slot of the row at hand
  unsigned nr = 0;
  for (long long r0 = (long long)blockIdx.x * slots; r0 < p.N; r0 += step, row += step, ++nr) {
    const int next = at + 1 == S ? 0 : at + 1;
    if (kNarrow) {
      copy(row + (S - 1) * step, at == 0 ? S - 1 : at - 1);
    } else if (S == 1) {  // a ring of one row: nothing is ahead
      __syncthreads();
      if (threadIdx.x == 0) copy(row, 0);
    }
    if (post && !join) first_norm(nr, at);
    wait(nr, at);
    const bool ahead = post && join && row + step < p.N;
    if (!kNarrow && ahead) wait(nr + 1, next);
    const float2 kh = both(kh1);
    float q[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    F8 hh[NV], s[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      hh[i] = get(th, kH32, i, at);
      const F8 wp = weight(0, i), sc = weight(1, i), w = weight(2, i);
      F8 z, e = get(tx, kX32, i, at, pre);
      const F8 g = get(tg, kG32, i, at, gate), ds = get(ts, kS32, i, at, dsum),
               r = get(tr, kR32, i, at, sum);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        z.v[j] = hh[i].v[j];
        if (post) z.v[j] = hh[i].v[j] = lmul(z.v[j], kh), z.v[j] = lmul(z.v[j], wp.v[j]);
        if (scale) z.v[j] = lmul(z.v[j], sc.v[j]);
        if (gate) z.v[j] = lmul(z.v[j], act(g.v[j]));
        s[i].v[j] = sum ? ladd(r.v[j], z.v[j]) : z.v[j];
        e.v[j] = lmul(e.v[j], w.v[j]);
      }
      if (pre) {
        q[0] = dot8(s[i], s[i], q[0]);
        q[1] = dot8(s[i], e, q[1]);
      }
      if (post && dsum) q[2] = dot8(ds, z, q[2]);
      if (post && pre) {
        q[3] = dot8(e, z, q[3]);
        q[4] = dot8(s[i], z, q[4]);
      }
    }
    if (ahead || (kNarrow && post)) q[5] = squares(next);
    const bool lost = !kNarrow && lost_at != kNever;
    if (lost) (pre ? q[0] : q[2]) = q[5] = __int_as_float(0x7fffffff);
    row_sum6<kNarrow>(q, tpr, sh, buf);
    // every thread is done with the row before: its slot takes a row again
    if (!kNarrow && S > 1 && threadIdx.x == 0) copy(row + (S - 1) * step, at == 0 ? S - 1 : at - 1);
    const float k1 = pre ? rsqrtf(fmaf(q[0], invD, p.eps)) : 0.f, nm1 = -(q[1] * k1 * invD);
    const float2 k = both(k1), nmean = both(nm1);
    const float2 nmean3 = both(-(fmaf(k1, fmaf(k1 * nm1, q[4], q[3]), q[2]) * invD));
    if (post && join) kh1 = rsqrtf(fmaf(q[5], invD, p.eps));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * (i * tpr + t);
      const bool ok = c < p.D && row < p.N;
      const F8 wp = weight(0, i), sc = weight(1, i), w = weight(2, i);
      F8 d = get(ts, kS32, i, at, dsum);
      const F8 dx = get(tx, kX32, i, at, pre);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (!pre) continue;
        const float2 sn = lmul(s[i].v[j], k);
        ap[i].v[j] = lfma(dx.v[j], sn, ap[i].v[j]);
        d.v[j] = lfma(k, lfma(sn, nmean, lmul(dx.v[j], w.v[j])), d.v[j]);
      }
      if (p.dres && ok) store8(p.dres, row * p.D + c, f32<TP>(p, kR32), d);
      if (gate) {
        const F8 g = get(tg, kG32, i, at);
        F8 dg;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float2 a, da;
          act.grad(g.v[j], a, da);
          const float2 n = post ? lmul(hh[i].v[j], wp.v[j]) : hh[i].v[j], e = scale ? lmul(d.v[j], sc.v[j]) : d.v[j];
          if (scale) as[i].v[j] = lfma(d.v[j], lmul(n, a), as[i].v[j]);
          dg.v[j] = lmul(lmul(e, n), da);
          d.v[j] = lmul(e, a);
        }
        if (ok) store8(p.dg, row * p.D + c, f32<TP>(p, kG32), dg);
      } else if (scale) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          as[i].v[j] = lfma(d.v[j], post ? lmul(hh[i].v[j], wp.v[j]) : hh[i].v[j], as[i].v[j]);
          d.v[j] = lmul(d.v[j], sc.v[j]);
        }
      }
      if (post)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          aw[i].v[j] = lfma(d.v[j], hh[i].v[j], aw[i].v[j]);
          d.v[j] = lmul(kh, lfma(hh[i].v[j], nmean3, lmul(d.v[j], wp.v[j])));
        }
      if (ok) store8(p.dh, row * p.D + c, f32<TP>(p, kH32), d);
    }
    at = next;
  }
  if (kNarrow) asm volatile("cp.async.wait_group 0;" ::: "memory");
  // [blocks][parts with a weight][D]: w_post, scale, w_pre
  const int n = (post ? 1 : 0) + (scale ? 1 : 0) + (pre ? 1 : 0);
  float* const out = p.part + (size_t)blockIdx.x * n * p.D;
  if (!kNarrow) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * (i * tpr + t);
      if (c >= p.D || !p.part) continue;
      float* q = out + c;
      if (post) store8(q, 0, true, aw[i]), q += p.D;
      if (scale) store8(q, 0, true, as[i]), q += p.D;
      if (pre) store8(q, 0, true, ap[i]);
    }
    if (lost_at == kNever) return;
    // what a lost thread wrote since, again
    if (p.status) *p.status = PARARNN_STATUS_TIMEOUT;
    const float2 nan = both(__int_as_float(0x7fffffff));
    const F8 nans = {nan, nan, nan, nan};
    for (int c = 8 * t; c < p.D; c += 8 * tpr) {
      for (row = blockIdx.x + lost_at * step; row < p.N; row += step) {
        if (p.dres) store8(p.dres, row * p.D + c, f32<TP>(p, kR32), nans);
        if (gate) store8(p.dg, row * p.D + c, f32<TP>(p, kG32), nans);
        store8(p.dh, row * p.D + c, f32<TP>(p, kH32), nans);
      }
      for (int i = 0; i < n && p.part; ++i) store8(out + i * p.D, c, true, nans);
    }
    // The block's shared memory must outlive its copies: of the rows from the
    // one lost on, S at most were copied (the waits for others run out).
    if (threadIdx.x == 0)
      for (unsigned r = lost_at; r < lost_at + S; ++r) mbar_wait_bounded(&full[r % S], (r / S) & 1, p.wait_ns);
    return;
  }
  if (!p.part) return;
  // several rows a block: its slots' sums, in their order
  float* const acc = reinterpret_cast<float*>(smem);  // [n][slots x 8 tpr]: 2048 channels each (256 threads of 8)
  const int width = 8 * tpr;
  __syncthreads();
  float* q = acc + slot * width + 8 * t;
  if (post) store8(q, 0, true, aw[0]), q += 2048;
  if (scale) store8(q, 0, true, as[0]), q += 2048;
  if (pre) store8(q, 0, true, ap[0]);
  __syncthreads();
  for (int i = threadIdx.x; i < n * p.D; i += blockDim.x) {
    const int k = i / p.D, c = i - k * p.D;
    float v = 0.f;
    for (int s = 0; s < slots; ++s) v += acc[k * 2048 + s * width + c];
    out[i] = v;
  }
}

constexpr int kNormMaxD = 8192;

// Vectors of a thread, threads of a row and of a block for D channels.
struct NormShape {
  int nv, tpr, threads;
  int slots() const { return threads / tpr; }
};
NormShape norm_shape(int D) {
  NormShape s;
  s.nv = D <= 4096 ? 1 : 2;
  if (D <= 256) {
    s.tpr = 1;
    while (8 * s.tpr < D) s.tpr *= 2;
    s.threads = 256;
  } else {
    s.tpr = s.threads = 32 * ((D + 256 * s.nv - 1) / (256 * s.nv));
  }
  return s;
}

// Blocks: all that the SMs hold at once (`sm_threads` threads each by their
// registers), or one for each of fewer groups of rows.
int norm_blocks(long long N, const NormShape& s, int sm_threads) {
  const long long most = kSMs * std::max(1, sm_threads / s.threads);
  return (int)std::min<long long>((N + s.slots() - 1) / s.slots(), most);
}
constexpr int kFwdThreads = 1024, kBwdThreads = 512, kBwdMost = 1024;

// The canonical type bits: those of absent tensors follow the others, so that
// they do not take a call off its kernel.
int canonical_types(const NormParams& p, bool s, bool x) {
  int present = kH32 | (p.g ? kG32 : 0) | (p.res ? kR32 : 0) | (s ? kS32 : 0) | (x ? kX32 : 0);
  int t = p.types & present;
  if (t == present) return kH32 | kG32 | kR32 | kS32 | kX32;
  if ((present & (kR32 | kS32)) == kR32 && (t & kR32)) t |= kS32;
  if ((present & (kR32 | kS32)) == kS32 && (t & kS32)) t |= kR32;
  return t;
}

template <int NV>
void launch_fwd_t(const NormParams& p, int types, int blocks, const NormShape& s, cudaStream_t stream) {
  switch (types) {
    case 0: norm_fwd<NV, 0><<<blocks, s.threads, 0, stream>>>(p, s.tpr); break;
    case kH32: norm_fwd<NV, kH32><<<blocks, s.threads, 0, stream>>>(p, s.tpr); break;
    case kR32 | kS32: norm_fwd<NV, kR32 | kS32><<<blocks, s.threads, 0, stream>>>(p, s.tpr); break;
    case kH32 | kR32 | kS32: norm_fwd<NV, kH32 | kR32 | kS32><<<blocks, s.threads, 0, stream>>>(p, s.tpr); break;
    case 31: norm_fwd<NV, 31><<<blocks, s.threads, 0, stream>>>(p, s.tpr); break;
    default: norm_fwd<NV, kAnyType><<<blocks, s.threads, 0, stream>>>(p, s.tpr); break;
  }
}
// Rows of the adjoint's ring and its shared memory: up to four, as many as
// leave room for the blocks that the registers allow on an SM (one for five
// fp32 tensors of nearly 8192 channels).  The slots' sums of several rows a
// block lie where the ring was.
int bwd_ring(const NormParams& p, const NormShape& s, int sm_threads, int& S) {
  int es = 0;
  for (auto [on, bit] : {std::pair<bool, int>{true, kH32}, {p.parts & kGate, kG32},
                         {(p.parts & kRes) && (p.parts & kPre), kR32}, {p.parts & kDs, kS32}, {p.parts & kPre, kX32}})
    if (on) es += p.types & bit ? 4 : 2;
  const int row = (s.slots() > 1 ? 8 * s.threads : p.D) * es, room = 220 * 1024 / std::max(1, sm_threads / s.threads);
  S = 4;
  while (S > 1 && S * row > room) --S;
  return std::max(S * row, s.slots() > 1 ? 3 * 2048 * 4 : 0);
}

template <int NV, bool kNarrow, int TP, int PT>
int launch_bwd_k(const NormParams& p, int sm_threads, const NormShape& s, cudaStream_t stream) {
  int S;
  const int smem = bwd_ring(p, s, sm_threads, S), blocks = norm_blocks(p.N, s, sm_threads);
  static SmemOnce once;
  const int e = once.allow(reinterpret_cast<const void*>(norm_bwd<NV, kNarrow, TP, PT>), smem);
  if (e) return e;
  norm_bwd<NV, kNarrow, TP, PT><<<blocks, s.threads, smem, stream>>>(p, s.tpr, S);
  return (int)cudaGetLastError();
}

// The kernels that know types and parts: a norm before a block over a residual
// stream; the gated norm after one; both in one, with and without a scale.
constexpr int kPartsPre = kPre | kRes | kDs, kPartsPost = kPost | kGate | kDs,
              kPartsBoth = kPost | kGate | kRes | kPre | kDs, kPartsAll = kPartsBoth | kScale;
template <bool kNarrow, int TP>
int launch_bwd_t(const NormParams& p, int sm_threads, const NormShape& s, cudaStream_t stream) {
  // (of narrow rows the kernels that know all parts spill: 48 us against 40 for
  // 65536 rows of 72 channels)
  switch (p.parts) {
    case kPartsPre: return launch_bwd_k<1, kNarrow, TP, kPartsPre>(p, sm_threads, s, stream);
    case kPartsPost: return launch_bwd_k<1, kNarrow, TP, kPartsPost>(p, sm_threads, s, stream);
    case kPartsBoth:
      return launch_bwd_k<1, kNarrow, TP, kNarrow ? kAnyPart : kPartsBoth>(p, sm_threads, s, stream);
    case kPartsAll: return launch_bwd_k<1, kNarrow, TP, kNarrow ? kAnyPart : kPartsAll>(p, sm_threads, s, stream);
    default: return launch_bwd_k<1, kNarrow, TP, kAnyPart>(p, sm_threads, s, stream);
  }
}
template <bool kNarrow>
int launch_bwd_w(const NormParams& p, int sm_threads, const NormShape& s, cudaStream_t stream) {
  switch (p.types) {
    case 0: return launch_bwd_t<kNarrow, 0>(p, sm_threads, s, stream);
    case kH32: return launch_bwd_t<kNarrow, kH32>(p, sm_threads, s, stream);
    case kR32 | kS32: return launch_bwd_t<kNarrow, kR32 | kS32>(p, sm_threads, s, stream);
    case kH32 | kR32 | kS32: return launch_bwd_t<kNarrow, kH32 | kR32 | kS32>(p, sm_threads, s, stream);
    case 31: return launch_bwd_t<kNarrow, 31>(p, sm_threads, s, stream);
    default: return launch_bwd_k<1, kNarrow, kAnyType, kAnyPart>(p, sm_threads, s, stream);
  }
}
int launch_bwd(const NormParams& p, int sm_threads, const NormShape& s, cudaStream_t stream) {
  if (s.nv == 2)
    return p.types == kH32 && p.parts == kPartsAll ? launch_bwd_k<2, false, kH32, kPartsAll>(p, sm_threads, s, stream)
                                                   : launch_bwd_k<2, false, kAnyType, kAnyPart>(p, sm_threads, s, stream);
  return s.slots() > 1 ? launch_bwd_w<true>(p, sm_threads, s, stream) : launch_bwd_w<false>(p, sm_threads, s, stream);
}

}  // namespace

int norm_max_d() { return kNormMaxD; }

size_t norm_part_floats(long long N, int D) {
  return (size_t)norm_blocks(N, norm_shape(D), kBwdMost) * 3 * D;
}

int launch_norm_fwd(const NormParams& p, cudaStream_t stream) {
  const NormShape s = norm_shape(p.D);
  const int blocks = norm_blocks(p.N, s, kFwdThreads), types = canonical_types(p, p.s, p.x);
  if (s.nv == 1)
    launch_fwd_t<1>(p, types, blocks, s, stream);
  else
    launch_fwd_t<2>(p, types, blocks, s, stream);
  return (int)cudaGetLastError();
}

int launch_norm_bwd(NormParams p, float* dw_post, float* dscale, float* dw_pre, cudaStream_t stream) {
  const NormShape s = norm_shape(p.D);
  p.types = canonical_types(p, p.ds, p.dx);
  p.parts = (p.w_post ? kPost : 0) | (p.g ? kGate : 0) | (p.res ? kRes : 0) | (p.scale ? kScale : 0) |
            (p.w_pre ? kPre : 0) | (p.ds ? kDs : 0);
  // Threads that an SM's registers hold: more where fewer parts leave more, and
  // its shared memory still holds a row ahead (a third with a first norm).  The
  // residual pre-norm's kernels have up to 64 registers a thread (1024 threads;
  // N32768 D1024 fp32 residual 104 us against 114 with 512), the gated norm's up
  // to 76 (768 threads: N32768 D1024 101 us against 113 with 512, 105 with 640).
  int sm_threads = kBwdThreads, S;
  if (p.D > 256 && p.D <= 4096 && (p.parts == kPartsPre || p.parts == kPartsPost)) {
    const int more = p.parts == kPartsPre ? kBwdMost : 768;
    bwd_ring(p, s, more, S);
    if (S >= (p.parts == kPartsPost ? 3 : 2)) sm_threads = more;
  }
  if (!dw_post && !dscale && !dw_pre) p.part = nullptr;
  const int e = launch_bwd(p, sm_threads, s, stream);
  if (e || !p.part) return e;
  ColSums sums = {p.part, norm_blocks(p.N, s, sm_threads), 0, p.D, {}};
  if (p.w_post) sums.out[sums.n++] = dw_post;
  if (p.scale) sums.out[sums.n++] = dscale;
  if (p.w_pre) sums.out[sums.n++] = dw_pre;
  return launch_colsum(sums, stream);
}

}  // namespace pararnn
