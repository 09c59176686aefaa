// block_norm.cuh -- what the host and the kernels of the block norm share.
#pragma once
#include <cuda_runtime.h>

#include "pararnn.h"

namespace pararnn {

struct NormParams {
  const void *h, *g, *res, *ds, *dx;
  long long ld_h, ld_g, ld_r, ld_ds, ld_dx;  // row strides in elements
  int types;                                 // bits 0-4: h, g, res, s (ds), x (dx) are fp32, else bf16
  int parts;                                 // adjoint: bits of the parts present (set at the launch)
  const float *w_post, *scale, *w_pre;
  int act;
  void *s, *x;                               // forward outputs [N][D]
  void *dh, *dg, *dres;                      // adjoint outputs [N][D], types of h, g, res
  float* part;                               // adjoint: [blocks][3][D] sums
  float eps;
  long long N;
  int D;
  int* status;                 // adjoint: device word for a wait that ran out, or NULL
  unsigned long long wait_ns;  // adjoint: bound on a wait for a row's copies
  int withhold;                // testing: the row that is not copied; -1: none
};

int norm_max_d();
size_t norm_part_floats(long long N, int D);
int launch_norm_fwd(const NormParams& p, cudaStream_t stream);
int launch_norm_bwd(NormParams p, float* dw_post, float* dscale, float* dw_pre, cudaStream_t stream);

}  // namespace pararnn
