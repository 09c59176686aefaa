// linrec.cu -- the gated linear recurrence: solve (one scan over the
// sequence), adjoint (one reverse scan) and the single decode step.
//
// Layout of the scans.  A cluster of CL CTAs owns a tile of 2 GL channels of
// one batch row and walks its sequence in rounds (the adjoint from the last
// step to the first).  A thread owns two neighbouring channels; GL lanes are a
// group, and the groups of a round take K consecutive steps each, in the order
// of the scan: CTA, warp, group of the warp.  In a round a thread composes its
// steps' maps (P, Q); the groups' maps meet in shared memory, the CTAs' maps in
// each other's shared memory (asynchronous stores), in two buffers in turn, and
// every thread composes what precedes its own steps and applies its maps to
// that.  The state that enters a round stays in a register of every thread.  So
// each input is read once, each output written once, and nothing waits on
// global memory: no workspace, no flags, no order of blocks.
//
// Every warp copies its own rows into a ring of S rounds in shared memory
// (16-byte cp.async, S - 1 rounds ahead), which keeps HBM busy through the
// rounds' barriers without holding registers.
//
// Measured (B200, device time, warm): LIN_GRU B8 T4096 D1024 bf16 solve 58 us (268
// MB: 4.6 TB/s).  Nothing is full there (special functions 61% of their rate,
// issue 48%, HBM 56%): an SM's 12 warps wait for loads and for one another's
// rounds.  Its adjoint 94 us (537 MB: 5.7 TB/s) and the LIN_DECAY solve of 65536
// steps of 2048 channels in fp32, 344-370 us (2.15 GB: 5.8-6.2 TB/s), are held by
// HBM.  A call from Python among others, the GPU under load: 60, 104, 396 us.
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "colsum.cuh"
#include "linrec_cell.cuh"
#include "smem_once.cuh"

namespace cg = cooperative_groups;

namespace pararnn {
namespace {

constexpr int kLinMaxCluster = 8;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// One kind of row in a warp's ring: C rows (gates) a step, of a tile's 2 GL
// channels of kBytes each.  A round of a warp holds, per group, K steps and a
// row of padding (the groups' rows then lie in different banks).  An
// instruction moves kRows steps' rows, 16 bytes a lane.
template <int GL, int K, int C, int kBytes>
struct Rows {
  static constexpr int kNG = 32 / GL;
  static constexpr int kRow = 2 * GL * kBytes;   // bytes of a row
  static constexpr int kLanes = kRow / 16;       // lanes of a row
  static constexpr int kRows = 32 / kLanes;
  static constexpr int kPiece = 16 / kBytes;     // channels of a lane
  static constexpr int kGroup = K * C * kRow + (kNG > 1 ? kRow : 0);
  static constexpr int kRound = kNG * kGroup;
  static constexpr int kCopies = kNG * K / kRows;
  static_assert(kCopies * kRows == kNG * K && (K % kRows == 0 || kRows % K == 0), "whole copies");
  // where step i (of a warp's kNG K, in the order of the scan) lies
  static __host__ __device__ constexpr int at(int i) { return i / K * kGroup + i % K * C * kRow; }
};

// The groups' maps of a round, and the mbarriers that count the arrival of the
// CTAs' maps; those lie in dynamic shared memory, kLinBufs x CL x GL x 16 bytes.
constexpr int kLinBufs = 4;
template <int W>
struct LinShared {
  float4 map[2][W * 32];
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

template <int CL, int GL, bool kReset>
__device__ __forceinline__ float2 lin_join(const float4* cta, int rpos, int gl, float2& carry) {
  float4 v[CL];
#pragma unroll
  for (int i = 0; i < CL; ++i) v[i] = cta[i * GL + gl];
  float2 in = carry;
#pragma unroll
  for (int i = 0; i < CL; ++i) {
    if (i == rpos) in = carry;
    carry = lin_apply<kReset>(v[i], carry);
  }
  return in;
}

// What a thread keeps of a round between its exchange and its end: the maps of
// the CTA's steps before its own and, where the CTA is alone, of all its steps.
struct LinTurn {
  float4 before, all;
};

// Publish the thread's map of round r, and (with `send`) the CTA's to the
// cluster.  Positions (gpos of the group in the CTA, rpos of the CTA) run in the
// order of the scan.  The groups' buffers alternate: round r + 2's are written
// after the barrier of round r + 1, which each warp reaches after it read round
// r's.
template <int W, int GL, bool kReset>
__device__ __forceinline__ LinTurn lin_publish(LinShared<W>& sh, float4* cta, unsigned r, float4 mine, int rpos,
                                               int CL, bool send) {
  constexpr int NP = W * 32 / GL;
  const int gl = threadIdx.x % GL, gpos = threadIdx.x / GL;
  sh.map[r & 1][threadIdx.x] = mine;
  __syncthreads();
  const float4* maps = sh.map[r & 1] + gl;
  LinTurn t;
  t.before = make_float4(1.f, 1.f, 0.f, 0.f);
  t.all = maps[0];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const float4 v = maps[i * GL];
    if (i < gpos) t.before = i ? lin_then<kReset>(t.before, v) : v;
    if (i && CL == 1) t.all = lin_then<kReset>(t.all, v);
  }
  if (CL > 1 && gpos == NP - 1 && send) {
    const float4 all = lin_then<kReset>(t.before, mine);
    const int buf = r % kLinBufs;
    if (gl == 0) mbar_arrive_expect_tx(&sh.bar[buf], CL * GL * 16);
    const uint32_t at = smem_u32(&cta[(buf * CL + rpos) * GL + gl]), bar = smem_u32(&sh.bar[buf]);
    for (int i = 0; i < CL; ++i) st_async16(map_rank(at, i), map_rank(bar, i), all);
  }
  __syncwarp();
  return t;
}

// The state that enters this thread's steps of round r; `carry`, which enters
// the round, becomes what leaves it.  The CTAs' buffers are used in turn: a CTA
// sends round r + 4's map after it ended round r + 2, for which it had every
// CTA's map of that round, each sent after all its warps had ended round r
// (rounds are published at most one ahead of their end).  The wait is bounded;
// a thread whose wait runs out is lost (stop = 0): it carries NaN from there on,
// waits no more and sends no more, so that no buffer or mbarrier is used out of
// turn (the CTAs that miss its maps run out of time in turn, once each).
template <int W, int GL, bool kReset>
__device__ __forceinline__ float2 lin_enter(LinShared<W>& sh, const float4* cta, unsigned r, const LinTurn& t,
                                            int rpos, int CL, float2& carry, unsigned& stop, uint64_t wait_ns) {
  const int gl = threadIdx.x % GL, gpos = threadIdx.x / GL;
  float2 in = carry;
  if (CL == 1) {
    carry = lin_apply<kReset>(t.all, carry);
  } else {
    const int buf = r % kLinBufs;
    if (stop && !mbar_wait_bounded(&sh.bar[buf], (r / kLinBufs) & 1, wait_ns)) stop = 0;
    const float4* v = cta + buf * CL * GL;
    if (CL == 2)
      in = lin_join<2, GL, kReset>(v, rpos, gl, carry);
    else if (CL == 4)
      in = lin_join<4, GL, kReset>(v, rpos, gl, carry);
    else
      in = lin_join<8, GL, kReset>(v, rpos, gl, carry);
    if (!stop) carry = in = both(__int_as_float(0x7fffffff));
  }
  return gpos ? lin_apply<kReset>(t.before, in) : in;
}

// The round from which on this thread sends no map (see LinParams): none, and 0
// once it is lost.
__device__ __forceinline__ unsigned lin_stop(const LinParams& p, int rank, int CL) {
  return CL > 1 && p.withhold >= 0 && (p.withhold & 7) == rank ? p.withhold / 8 : 0xffffffffu;
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

// The last thing a thread does.  A CTA's shared memory must outlive the stores
// of its peers: one whose waits ended has them all; a lost thread waits until
// every thread of the cluster is lost too or has left (all waits are bounded),
// and then for the stores on their way, which take microseconds.
__device__ __forceinline__ void lin_leave(unsigned stop, int* status) {
  if (stop) return;
  if (status) *status = PARARNN_STATUS_TIMEOUT;
  asm volatile("barrier.cluster.arrive;\n barrier.cluster.wait;" ::: "memory");
  const uint64_t t0 = globaltimer_ns();
  while (globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
}

// A group's marks: its j-th step in the order of the scan has its mark at
// at[dir * j], `n` of the steps are within the sequence.  A lane loads those of
// steps gl, gl + GL, ... (a round before they are asked for, so that no round
// waits for them), and the vote makes them bits of the group's steps.
template <int GL, int K>
struct Marks {
  static constexpr int M = (K + GL - 1) / GL;
  unsigned char raw[M];
  __device__ __forceinline__ void load(const unsigned char* at, int dir, int n) {
    const int gl = threadIdx.x % GL;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      raw[m] = 0;
      if (gl + m * GL < min(K, n)) raw[m] = at[(long long)dir * (gl + m * GL)];
    }
  }
  __device__ __forceinline__ unsigned vote() const {
    const int shift = threadIdx.x % 32 / GL * GL;
    unsigned bits = 0;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const unsigned all = __ballot_sync(0xffffffffu, raw[m] != 0) >> shift;
      bits |= (GL == 32 ? all : all & ((1u << (GL % 32)) - 1u)) << (m * GL);
    }
    return bits;
  }
};

// Whether a warp's steps have no reset; and f(whether they may), so that the
// rounds without one, which are most, pay nothing for it.
__device__ __forceinline__ bool no_marks(unsigned resets) { return __all_sync(0xffffffffu, resets == 0u); }
template <bool kReset, typename F>
__device__ __forceinline__ void by_marks(unsigned resets, F f) {
  if (kReset && !no_marks(resets))
    f(std::true_type());
  else
    f(std::false_type());
}

// Shape of a scan kernel: GL lanes of a group, W warps, K steps of a thread in
// a round, a ring of S rounds, at least R CTAs on an SM.  More steps a round
// mean fewer exchanges, but more registers and shared memory, so fewer CTAs on
// an SM for the sequence to be split over.
//   kTall    the longest rounds that leave two to four CTAs on an SM.  With fp32
//            u a round is published before the round before it ends (kAhead), so
//            its exchange runs behind the next round's arithmetic, at twice the
//            registers for maps: LIN_DECAY T65536 D2048 344-370 us against
//            416-424, LIN_GRU B8 T4096 D1024 66 against 69.  With bf16 the
//            registers cost as many CTAs as that gains.
//   kShort   LIN_GRU with bf16 u: 8 steps, five CTAs, taken where that lets the
//            cluster grow (300 tiles of 2048 steps: 69 us against 80; 128 tiles
//            of 4096 steps: 62 against 58)
//   kNarrow  tiles of 16 channels, for problems of so few 64-channel tiles that
//            clusters of 8 CTAs leave SMs idle (one tile of 16384 steps: 16 us
//            against 51; 16 tiles of 65536 steps: 164 against 225)
enum Variant { kTall, kShort, kNarrow };
template <int CELL, bool kBF16, int V>
struct FwdShape {
  static constexpr bool kGru = CELL == PARARNN_LIN_GRU;
  static constexpr int GL = V == kNarrow ? 8 : 32, W = V == kNarrow ? 8 : 4;
  static constexpr bool kAhead = V == kTall && !kBF16;
  static constexpr int K = V == kNarrow ? 16 : V == kShort || (!kBF16 && kGru) ? 8 : kGru ? 16 : 12;
  static constexpr int S = V == kShort ? 3 : 2;
  static constexpr int R = V == kNarrow ? (kBF16 ? 2 : 1) : V == kShort ? 5 : kBF16 || kGru ? 4 : 2;
  using U = Rows<GL, K, LinCell<CELL>::G, kBF16 ? 2 : 4>;
  static constexpr int kWarp = S * U::kRound;   // bytes of a warp's ring
  static constexpr int kBytes = W * kWarp;
};

template <bool kBF16>
__device__ __forceinline__ float2 row_pair(const char* row, int lane) {
  if (kBF16) return bf16_pair(*reinterpret_cast<const unsigned*>(row + 4 * lane));
  return *reinterpret_cast<const float2*>(row + 8 * lane);
}

template <int CELL, bool kBF16, int V, bool kReset>
__global__ void __launch_bounds__(32 * FwdShape<CELL, kBF16, V>::W, FwdShape<CELL, kBF16, V>::R)
    linrec_fwd(const LinParams p, const int CL) {
  using Cell = LinCell<CELL>;
  using Shape = FwdShape<CELL, kBF16, V>;
  using U = typename Shape::U;
  constexpr int G = Cell::G, K = Shape::K, W = Shape::W, S = Shape::S, GL = Shape::GL, ES = kBF16 ? 2 : 4;
  constexpr int KW = U::kNG * K;  // steps of a warp in a round
  extern __shared__ __align__(16) char ring[];
  __shared__ LinShared<W> sh;
  const int rank = CL > 1 ? (int)cg::this_cluster().block_rank() : 0;
  const int tile = blockIdx.x / CL;
  const int b = tile / p.ntd, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gl = lane % GL, grp = lane / GL;
  const int dbase = (tile - b * p.ntd) * 2 * GL, d0 = dbase + 2 * gl;
  const bool live = d0 < p.D;
  const int d = live ? d0 : p.D - 2;  // idle lanes read parameters that exist
  // copies: this lane's row of an instruction and its piece of the row
  const int crow = lane / U::kLanes, cpiece = lane % U::kLanes;
  const bool cok = dbase + cpiece * U::kPiece < p.D;
  const uint32_t dst = smem_u32(ring) + warp * Shape::kWarp + U::at(crow) + cpiece * 16;
  const char* const mine = ring + warp * Shape::kWarp + U::at(grp * K);
  float4* const cta = reinterpret_cast<float4*>(ring + Shape::kBytes);
  const int round = CL * W * KW, first = (rank * W + warp) * KW;
  const long long pitch = p.st * ES, gate = p.sg * ES;
  // this lane's first row of the next round to copy, and the steps from it to
  // the end of the sequence (none for a lane past D)
  const char* src =
      static_cast<const char*>(p.u) + (b * p.sb + dbase + cpiece * U::kPiece) * ES + (first + crow) * pitch;
  int left = cok ? p.T - first - crow : 0;
  auto copy = [&](int slot) {
    const uint32_t to = dst + slot * U::kRound;
#pragma unroll
    for (int i = 0; i < U::kCopies; ++i)
      if (i * U::kRows < left) {
#pragma unroll
        for (int q = 0; q < G; ++q)
          cp_async16(to + U::at(i * U::kRows) + q * U::kRow, src + i * (U::kRows * pitch) + q * gate);
      }
    src += round * pitch;
    left -= round;
  };
#pragma unroll
  for (int s = 0; s < S - 1; ++s) {
    copy(s);
    cp_async_commit();
  }
  Cell cell;
  cell.init(p.lam, p.bias, p.kappa, p.D, d);
  float2 carry = vec2(p.h0 ? p.h0 + (size_t)b * p.D : nullptr, d);
  const size_t row = (size_t)b * p.T;
  lin_cluster_start(sh, CL);
  const int rounds = (p.T + round - 1) / round;
  unsigned stop = lin_stop(p, rank, CL);
  int slot = 0;
  struct Round {
    float2 P[K], Q[K];  // h after step j is P[j] h_in + Q[j]
    unsigned resets;
    LinTurn turn;
  };
  Marks<GL, K> marks;
  if (kReset) marks.load(p.reset + row + first + grp * K, 1, p.T - first - grp * K);
  auto begin = [&](int r, Round& x) {  // round r's maps, published
    const int t0 = r * round + first + grp * K;
    cp_async_wait<S - 2>();
    __syncwarp();
    copy(slot == 0 ? S - 1 : slot - 1);
    cp_async_commit();
    x.resets = 0u;
    if (kReset) {
      x.resets = marks.vote();
      marks.load(p.reset + row + t0 + round, 1, p.T - t0 - round);
    }
    const char* rows = mine + slot * U::kRound;
    slot = slot + 1 == S ? 0 : slot + 1;
    // steps past T compute on what the ring holds there: nothing after them is
    // stored
    auto compose = [&](auto marked) {
#pragma unroll
      for (int j = 0; j < K; ++j) {
        float2 u[G], nm, bb;
#pragma unroll
        for (int q = 0; q < G; ++q) u[q] = row_pair<kBF16>(rows + (j * G + q) * U::kRow, gl);
        cell.coef(u, nm, bb);
        x.P[j] = j ? lfma(nm, x.P[j - 1], x.P[j - 1]) : ladd(nm, both(1.f));
        x.Q[j] = j ? lin_step(nm, bb, x.Q[j - 1]) : bb;
        if (decltype(marked)::value && ((x.resets >> j) & 1u)) x.Q[j] = bb;
      }
    };
    by_marks<kReset>(x.resets, compose);
    float4 map = make_float4(x.P[K - 1].x, x.P[K - 1].y, x.Q[K - 1].x, x.Q[K - 1].y);
    if (kReset && x.resets) map.x = map.y = -1.f;
    x.turn = lin_publish<W, GL, kReset>(sh, cta, r, map, rank, CL, (unsigned)r < stop);
  };
  auto end = [&](int r, Round& x) {  // its states, stored
    const int t0 = r * round + first + grp * K;
    const float2 in = lin_enter<W, GL, kReset>(sh, cta, r, x.turn, rank, CL, carry, stop, p.wait_ns);
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const float2 h = lfma(x.P[j], in, x.Q[j]);
      if (!kReset || !(x.resets & ((2u << j) - 1u))) x.Q[j] = h;  // after a reset nothing is left of h_in
    }
    float* out = p.h + (row + t0) * p.D + d;
    if (t0 + K <= p.T) {
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (live) *reinterpret_cast<float2*>(out + (size_t)j * p.D) = x.Q[j];
    } else {
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (live && t0 + j < p.T) *reinterpret_cast<float2*>(out + (size_t)j * p.D) = x.Q[j];
    }
  };
  Round x;
  if constexpr (Shape::kAhead) {
    Round y;
    begin(0, x);
    for (int r = 0; r < rounds; r += 2) {
      if (r + 1 < rounds) begin(r + 1, y);
      end(r, x);
      if (r + 1 >= rounds) break;
      if (r + 2 < rounds) begin(r + 2, x);
      end(r + 1, y);
    }
  } else {
    for (int r = 0; r < rounds; ++r) {
      begin(r, x);
      end(r, x);
    }
  }
  cp_async_wait<0>();
  lin_leave(stop, p.status);
}

// Reverse scan: lambda_t = g_t + mu_{t+1}, mu_t = (1 - m_t) lambda_t (0 at a
// reset, and mu_1 = dL/dh0).  Positions run from the last step to the first.
// (kTall with fp32 u: 8 steps, 12 do not leave two CTAs on an SM)
template <int CELL, bool kBF16, int V>
struct BwdShape {
  static constexpr int GL = V == kNarrow ? 8 : 32, W = V == kNarrow ? 8 : 4;
  static constexpr int K = V == kTall && kBF16 ? 12 : 8, S = 2, R = V == kNarrow ? 1 : 2;
  using U = Rows<GL, K, LinCell<CELL>::G, kBF16 ? 2 : 4>;
  using F = Rows<GL, K, 1, 4>;
  static constexpr int kH = U::kRound, kG = kH + F::kRound;  // offsets of h_{t-1} and dL/dh in a round
  static constexpr int kRound = kG + F::kRound;
  static constexpr int kWarp = S * kRound;
  static constexpr int kBytes = W * kWarp;
};

template <int CELL, bool kBF16, bool kBF16Out, int V, bool kReset>
__global__ void __launch_bounds__(32 * BwdShape<CELL, kBF16, V>::W, BwdShape<CELL, kBF16, V>::R)
    linrec_bwd(const LinParams p, const int CL) {
  using Cell = LinCell<CELL>;
  using Shape = BwdShape<CELL, kBF16, V>;
  using U = typename Shape::U;
  using F = typename Shape::F;
  constexpr int G = Cell::G, K = Shape::K, W = Shape::W, S = Shape::S, GL = Shape::GL, ES = kBF16 ? 2 : 4;
  constexpr int KW = U::kNG * K;
  extern __shared__ __align__(16) char ring[];
  __shared__ LinShared<W> sh;
  const int rank = CL > 1 ? (int)cg::this_cluster().block_rank() : 0;
  const int tile = blockIdx.x / CL;
  const int b = tile / p.ntd, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gl = lane % GL, grp = lane / GL;
  const int dbase = (tile - b * p.ntd) * 2 * GL, d0 = dbase + 2 * gl;
  const bool live = d0 < p.D;
  const int d = live ? d0 : p.D - 2;
  const size_t row = (size_t)b * p.T;
  const int crow = lane / U::kLanes, cpiece = lane % U::kLanes;
  const bool cok = dbase + cpiece * U::kPiece < p.D;
  const int frow = lane / F::kLanes, fpiece = lane % F::kLanes;
  const bool fok = dbase + fpiece * F::kPiece < p.D;
  const uint32_t udst = smem_u32(ring) + warp * Shape::kWarp + U::at(crow) + cpiece * 16;
  const uint32_t fdst = smem_u32(ring) + warp * Shape::kWarp + F::at(frow) + fpiece * 16;
  const char* const umine = ring + warp * Shape::kWarp + U::at(grp * K);
  const char* const fmine = ring + warp * Shape::kWarp + F::at(grp * K);
  float4* const cta = reinterpret_cast<float4*>(ring + Shape::kBytes);
  const int round = CL * W * KW, first = (rank * W + warp) * KW;
  const long long pitch = p.st * ES, gate = p.sg * ES;
  // this lane's first rows of the next round to copy, and the steps from them
  // to the first of the sequence; h_{t-1} is a row before dL/dh_t's
  const char* src = static_cast<const char*>(p.u) + (b * p.sb + dbase + cpiece * U::kPiece) * ES +
                    (p.T - 1 - first - crow) * pitch;
  long long fat = ((long long)row + p.T - 1 - first - frow) * p.D + dbase + fpiece * F::kPiece;
  int uleft = cok ? p.T - first - crow : 0, fleft = fok ? p.T - first - frow : 0;
  auto copy = [&](int slot) {
    const uint32_t to = udst + slot * Shape::kRound, fto = fdst + slot * Shape::kRound;
#pragma unroll
    for (int i = 0; i < U::kCopies; ++i)
      if (i * U::kRows < uleft) {
#pragma unroll
        for (int q = 0; q < G; ++q)
          cp_async16(to + U::at(i * U::kRows) + q * U::kRow, src - i * (U::kRows * pitch) + q * gate);
      }
    const float* g = p.g + fat;
    const float* h = p.h + fat - p.D;
#pragma unroll
    for (int i = 0; i < F::kCopies; ++i) {
      const long long o = (long long)i * F::kRows * p.D;
      if (i * F::kRows < fleft) cp_async16(fto + F::at(i * F::kRows) + Shape::kG, g - o);
      if (i * F::kRows + 1 < fleft) cp_async16(fto + F::at(i * F::kRows) + Shape::kH, h - o);
    }
    src -= round * pitch;
    fat -= (long long)round * p.D;
    uleft -= round;
    fleft -= round;
  };
#pragma unroll
  for (int s = 0; s < S - 1; ++s) {
    copy(s);
    cp_async_commit();
  }
  Cell cell;
  cell.init(p.lam, p.bias, p.kappa, p.D, d);
  float2 carry = both(0.f);
  float2 sum[G + 1];
#pragma unroll
  for (int q = 0; q <= G; ++q) sum[q] = both(0.f);
  lin_cluster_start(sh, CL);
  unsigned stop = lin_stop(p, rank, CL);
  int slot = 0;
  unsigned nround = 0;
  using Out = typename std::conditional<kBF16Out, __nv_bfloat162, float2>::type;
  const size_t pairs = p.D / 2;  // channel pairs of a row of du
  Out* du_at = static_cast<Out*>(p.du) + ((long long)row + p.T - 1 - first - grp * K) * (long long)(G * pairs) + d / 2;
  Marks<GL, K> marks;
  if (kReset) marks.load(p.reset + row + p.T - 1 - first - grp * K, -1, p.T - first - grp * K);
  for (int end = p.T; end > 0; end -= round, ++nround) {
    const int t1 = end - first - grp * K;  // this thread's steps: t1 - 1, ..., t1 - K
    cp_async_wait<S - 2>();
    __syncwarp();
    copy(slot == 0 ? S - 1 : slot - 1);
    cp_async_commit();
    unsigned resets = 0u;
    if (kReset) {
      resets = marks.vote();
      marks.load(p.reset + row + t1 - 1 - round, -1, t1 - round);
    }
    const char* urows = umine + slot * Shape::kRound;
    const char* grows = fmine + slot * Shape::kRound + Shape::kG;
    const char* hrows = fmine + slot * Shape::kRound + Shape::kH;
    slot = slot + 1 == S ? 0 : slot + 1;
    // lambda of step j is L[j] + P[j] mu, mu what comes from the steps after
    float2 nm[K], L[K], P[K], keep[K][Cell::kKeep], mu = both(0.f), pr = both(1.f);
    auto compose = [&](auto marked) {
#pragma unroll
      for (int j = 0; j < K; ++j) {
        cell.head(row_pair<kBF16>(urows + j * G * U::kRow, gl), nm[j], keep[j]);
        L[j] = ladd(row_pair<false>(grows + j * F::kRow, gl), mu);
        P[j] = pr;
        mu = lfma(nm[j], L[j], L[j]);
        pr = lfma(nm[j], pr, pr);
        if (decltype(marked)::value && ((resets >> j) & 1u)) mu = pr = both(0.f);
      }
    };
    by_marks<kReset>(resets, compose);
    if (kReset && resets) pr = both(-1.f);
    const LinTurn turn =
        lin_publish<W, GL, kReset>(sh, cta, nround, make_float4(pr.x, pr.y, mu.x, mu.y), rank, CL,
                                   nround < stop);
    mu = lin_enter<W, GL, kReset>(sh, cta, nround, turn, rank, CL, carry, stop, p.wait_ns);
    float2 add[G + 1];
#pragma unroll
    for (int q = 0; q <= G; ++q) add[q] = both(0.f);
    auto step = [&](int j, bool first_step, bool marked) {
      float2 lt = lfma(P[j], mu, L[j]);
      if (marked && (resets & ((1u << j) - 1u))) lt = L[j];  // nothing of mu comes before a reset
      const bool rs = marked && ((resets >> j) & 1u);
      float2 hp = row_pair<false>(hrows + j * F::kRow, gl);
      if (first_step) {
        hp = vec2(p.h0 ? p.h0 + (size_t)b * p.D : nullptr, d);
        if (p.dh0 && live) {
          const float2 v = rs ? both(0.f) : lfma(nm[j], lt, lt);
          p.dh0[(size_t)b * p.D + d] = v.x;
          p.dh0[(size_t)b * p.D + d + 1] = v.y;
        }
      }
      if (rs) hp = both(0.f);
      float2 u[G], du[G], e;
#pragma unroll
      for (int q = 1; q < G; ++q) u[q] = row_pair<kBF16>(urows + (j * G + q) * U::kRow, gl);
      cell.grad(u, nm[j], keep[j], hp, lt, du, e);
      Out* out = du_at - j * (G * pairs);
#pragma unroll
      for (int q = 0; q < G; ++q) {
        add[q] = ladd(add[q], du[q]);
        if (!live) continue;
        if constexpr (kBF16Out)
          out[q * pairs] = __float22bfloat162_rn(du[q]);
        else
          out[q * pairs] = du[q];
      }
      if (CELL == PARARNN_LIN_DECAY) add[G] = ladd(add[G], e);
    };
    const bool clean = !kReset || no_marks(resets);  // asked by the whole warp: t1 differs between its groups
    if (t1 > K && clean) {
#pragma unroll
      for (int j = 0; j < K; ++j) step(j, false, false);
    } else {  // a round with resets, or the sequence's first steps
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (t1 - 1 - j >= 0) step(j, t1 - 1 - j == 0, kReset);
    }
    du_at -= (long long)round * (long long)(G * pairs);
    // a round's sums first, then the running sums: over long sequences the
    // error grows with the number of rounds only
#pragma unroll
    for (int q = 0; q <= G; ++q) sum[q] = ladd(sum[q], add[q]);
  }
  cp_async_wait<0>();
  if (p.part) {
    if (CELL == PARARNN_LIN_DECAY) sum[G] = lmul(sum[G], Cell::lam_scale(p.lam, d));
    // the groups' sums, in their order
    constexpr int NS = CELL == PARARNN_LIN_DECAY ? G + 1 : G;
    __syncthreads();
    float2* const acc = reinterpret_cast<float2*>(ring);  // [NS][W * 32]
    static_assert(Shape::kBytes >= W * NS * 32 * (int)sizeof(float2), "sums fit");
    static_assert(W >= NS, "a warp for each sum");
#pragma unroll
    for (int q = 0; q < NS; ++q) acc[q * W * 32 + threadIdx.x] = sum[q];
    __syncthreads();
    if (warp < NS && lane < GL && live) {
      float2 s = both(0.f);
      for (int i = 0; i < W * 32 / GL; ++i) s = ladd(s, acc[warp * W * 32 + i * GL + lane]);
      float* q = p.part + ((size_t)(b * CL + rank) * NS + warp) * p.D + d;
      q[0] = s.x;
      q[1] = s.y;
    }
  }
  lin_leave(stop, p.status);
}

// One decode step: a thread owns two channels of one row; h_prev may be h_next.
// A launch: 2 us for one row of 1024 channels; 6.5 us for 256 of 4096, 1.7 waves of
// blocks.
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
int launch_scan(Kern kern, int GL, int threads, int smem, LinParams p, int CL, SmemOnce& once, cudaStream_t stream) {
  p.ntd = (p.D + 2 * GL - 1) / (2 * GL);
  const int e = once.allow(reinterpret_cast<const void*>(kern), smem + kLinBufs * kLinMaxCluster * GL * 16);
  if (e) return e;
  if (CL > 1) smem += kLinBufs * CL * GL * 16;
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

long long tiles_of(int B, int D, int GL) { return (long long)B * ((D + 2 * GL - 1) / (2 * GL)); }

// clusters of 8 on 64-channel tiles would not fill the SMs
bool few_tiles(int B, int D) { return tiles_of(B, D, 32) * kLinMaxCluster <= kSMs; }

// CTAs of a cluster: as many as fill one wave of H::R CTAs on each SM,
// no more than the sequence has rounds of one CTA for.
template <typename H>
int cluster_of(int B, int T, int D) {
  const long long tiles = tiles_of(B, D, H::GL);
  int CL = 1;
  while (CL < kLinMaxCluster && 2 * tiles * CL <= kSMs * H::R && T > CL * H::W * H::U::kNG * H::K) CL *= 2;
  return CL;
}

template <int CELL, bool kBF16, int V>
int launch_fwd_v(const LinParams& p, cudaStream_t stream) {
  using H = FwdShape<CELL, kBF16, V>;
  static SmemOnce once[2];
  const int CL = cluster_of<H>(p.B, p.T, p.D);
  return p.reset
             ? launch_scan(linrec_fwd<CELL, kBF16, V, true>, H::GL, 32 * H::W, H::kBytes, p, CL, once[1], stream)
             : launch_scan(linrec_fwd<CELL, kBF16, V, false>, H::GL, 32 * H::W, H::kBytes, p, CL, once[0], stream);
}

template <int CELL, bool kBF16>
int launch_fwd_t(const LinParams& p, cudaStream_t stream) {
  if (few_tiles(p.B, p.D)) return launch_fwd_v<CELL, kBF16, kNarrow>(p, stream);
  if constexpr (CELL == PARARNN_LIN_GRU && kBF16)
    if (cluster_of<FwdShape<CELL, true, kShort>>(p.B, p.T, p.D) > cluster_of<FwdShape<CELL, true, kTall>>(p.B, p.T, p.D))
      return launch_fwd_v<CELL, true, kShort>(p, stream);
  return launch_fwd_v<CELL, kBF16, kTall>(p, stream);
}

// the same for both types of u, so that the workspace does not depend on it
template <int CELL>
int bwd_cluster(int B, int T, int D) {
  return few_tiles(B, D) ? cluster_of<BwdShape<CELL, true, kNarrow>>(B, T, D)
                         : cluster_of<BwdShape<CELL, true, kTall>>(B, T, D);
}

template <int CELL, bool kBF16, bool kBF16Out, int V>
int launch_bwd_v(const LinParams& p, cudaStream_t stream) {
  using H = BwdShape<CELL, kBF16, V>;
  static SmemOnce once[2];
  const int CL = bwd_cluster<CELL>(p.B, p.T, p.D);
  return p.reset ? launch_scan(linrec_bwd<CELL, kBF16, kBF16Out, V, true>, H::GL, 32 * H::W, H::kBytes, p, CL,
                               once[1], stream)
                 : launch_scan(linrec_bwd<CELL, kBF16, kBF16Out, V, false>, H::GL, 32 * H::W, H::kBytes, p, CL,
                               once[0], stream);
}

template <int CELL, bool kBF16, bool kBF16Out>
int launch_bwd_t(const LinParams& p, cudaStream_t stream) {
  return few_tiles(p.B, p.D) ? launch_bwd_v<CELL, kBF16, kBF16Out, kNarrow>(p, stream)
                             : launch_bwd_v<CELL, kBF16, kBF16Out, kTall>(p, stream);
}

template <int CELL>
int launch_bwd_c(bool bf16, bool bf16_out, const LinParams& p, cudaStream_t stream) {
  if (!bf16) return launch_bwd_t<CELL, false, false>(p, stream);
  return bf16_out ? launch_bwd_t<CELL, true, true>(p, stream) : launch_bwd_t<CELL, true, false>(p, stream);
}

}  // namespace

int linrec_bwd_cluster(int cell, int B, int T, int D) {
  return cell == PARARNN_LIN_GRU ? bwd_cluster<PARARNN_LIN_GRU>(B, T, D) : bwd_cluster<PARARNN_LIN_DECAY>(B, T, D);
}

// more CTAs than any launch for this problem has (tiles of at least 8 channels)
long long linrec_most_ctas(int B, int D) { return (long long)B * (D / 8) * kLinMaxCluster; }

size_t linrec_part_floats(int cell, int B, int T, int D) {
  return (size_t)B * linrec_bwd_cluster(cell, B, T, D) * (cell == PARARNN_LIN_GRU ? 2 : 4) * D;
}

int launch_linrec_fwd(int cell, bool bf16, const LinParams& p, cudaStream_t stream) {
  if (cell == PARARNN_LIN_GRU)
    return bf16 ? launch_fwd_t<PARARNN_LIN_GRU, true>(p, stream) : launch_fwd_t<PARARNN_LIN_GRU, false>(p, stream);
  return bf16 ? launch_fwd_t<PARARNN_LIN_DECAY, true>(p, stream) : launch_fwd_t<PARARNN_LIN_DECAY, false>(p, stream);
}

int launch_linrec_bwd(int cell, bool bf16, bool bf16_out, LinParams p, float* dlam, float* dbias,
                      cudaStream_t stream) {
  if (!dlam && !dbias) p.part = nullptr;
  int e = cell == PARARNN_LIN_GRU ? launch_bwd_c<PARARNN_LIN_GRU>(bf16, bf16_out, p, stream)
                                  : launch_bwd_c<PARARNN_LIN_DECAY>(bf16, bf16_out, p, stream);
  if (e || !p.part) return e;
  const int G = cell == PARARNN_LIN_GRU ? 2 : 3;
  ColSums sums = {p.part, p.B * linrec_bwd_cluster(cell, p.B, p.T, p.D), cell == PARARNN_LIN_GRU ? G : G + 1, p.D, {}};
  for (int q = 0; q < G; ++q) sums.out[q] = dbias ? dbias + (size_t)q * p.D : nullptr;
  if (cell == PARARNN_LIN_DECAY) sums.out[G] = dlam;
  return launch_colsum(sums, stream);
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
