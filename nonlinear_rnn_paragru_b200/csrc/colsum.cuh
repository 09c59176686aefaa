// colsum.cuh -- the second step of sums over rows: the blocks' partial sums
// part [P][n][D] into n vectors of D, in a fixed order.
#pragma once
#include <cuda_runtime.h>

namespace pararnn {

struct ColSums {
  const float* part;
  int P, n, D;    // D a multiple of 8
  float* out[4];  // NULL: not wanted
};

// 32 columns of one vector a block, 8 threads of 4 columns side by side, 32
// deep; launched while the kernel before it still runs (its blocks wait for
// that one's end here).
static __global__ void __launch_bounds__(256) colsum_kernel(const ColSums s) {
  __shared__ float4 sum[32][9];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int x = threadIdx.x & 7, y = threadIdx.x >> 3, c = blockIdx.x * 32 + 4 * x;
  float* const out = s.out[blockIdx.y];
  if (!out) return;  // the whole block
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < s.D) {
    const float* p = s.part + (size_t)blockIdx.y * s.D + c;
    const size_t row = (size_t)s.n * s.D;
#pragma unroll 8
    for (int i = y; i < s.P; i += 32) {
      const float4 a = *reinterpret_cast<const float4*>(p + i * row);
      v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
    }
  }
  sum[y][x] = v;
  __syncthreads();
  // a column each for 32 threads
  if (threadIdx.x < 32 && blockIdx.x * 32 + threadIdx.x < s.D) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += reinterpret_cast<const float*>(&sum[i][0])[threadIdx.x];
    out[blockIdx.x * 32 + threadIdx.x] = t;
  }
}

static inline int launch_colsum(const ColSums& s, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((s.D + 31) / 32, s.n);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return (int)cudaLaunchKernelEx(&cfg, colsum_kernel, s);
}

}  // namespace pararnn
