// colsum.cuh -- the second step of sums over rows: the blocks' partial sums
// part [P][n][D] into n vectors of D, in a fixed order.
#pragma once
#include <cuda_runtime.h>

namespace pararnn {
namespace {

struct ColSums {
  const float* part;
  int P, n, D;    // D a multiple of 8
  float* out[4];  // NULL: not wanted
};

// 32 columns of one vector a block: 8 threads of 4 columns side by side, kDeep
// deep; then a warp folds a column (of 4 kDeep / 32 at a time).  32 deep, or 128
// for so many partial sums that 32 threads wait for their loads (1184 of 1000
// columns: 6 us against 13; of 16 of 4096 columns and three vectors the adjoint
// takes 15 us with 128, 10 with 32).
template <int kDeep>
__global__ void __launch_bounds__(8 * kDeep) colsum_kernel(const ColSums s) {
  __shared__ float4 part[kDeep][9];
  __shared__ float fold[32][33];
  const int x = threadIdx.x & 7, y = threadIdx.x >> 3, c = blockIdx.x * 32 + 4 * x;
  float* const out = s.out[blockIdx.y];
  if (!out) return;  // the whole block
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < s.D) {
    const float* p = s.part + (size_t)blockIdx.y * s.D + c;
    const size_t row = (size_t)s.n * s.D;
#pragma unroll 8
    for (int i = y; i < s.P; i += kDeep) {
      const float4 a = *reinterpret_cast<const float4*>(p + i * row);
      v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
    }
  }
  part[y][x] = v;
  __syncthreads();
  constexpr int W = kDeep / 4;  // warps
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float t = 0.f;  // column `lane`, four of the kDeep
#pragma unroll
  for (int i = 0; i < 4; ++i) t += reinterpret_cast<const float*>(&part[4 * warp + i][0])[lane];
  fold[warp][lane] = t;
  __syncthreads();
  for (int col = warp; col < 32; col += W) {
    t = lane < W ? fold[lane][col] : 0.f;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (lane == 0 && blockIdx.x * 32 + col < s.D) out[blockIdx.x * 32 + col] = t;
  }
}

int launch_colsum(const ColSums& s, cudaStream_t stream) {
  const dim3 grid((s.D + 31) / 32, s.n);
  if (s.P > 320)
    colsum_kernel<128><<<grid, 1024, 0, stream>>>(s);
  else
    colsum_kernel<32><<<grid, 256, 0, stream>>>(s);
  return (int)cudaGetLastError();
}

}  // namespace
}  // namespace pararnn
