// The norm of a residual stream to which a block's output is added through
// dropout (dropout.cuh): arguments and host launchers.
//
// Forward, per row of `cols` channels (x the stream, f the block's output, m the
// mask, k = 65536 / (65536 - cut)):
//   y = x + m k f     r = 1 / sqrt(mean(y^2) + eps)     h = y r w
// h to the activations' type and / or to MXFP8 by rows.  Backward, from dy
// (gradient of y from later uses) and dh, with yn = y r:
//   t = dy + r (dh w - yn mean(dh w yn)),  dx = t,  df = m k t,  dw = sum_rows dh yn
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "dropout.cuh"
#include "mx8.cuh"

namespace dmuon {

struct AddNormFwdArgs {
  const void *x, *f;            // x: nullptr for 0
  const float* w;
  void *y, *h;                  // h, q: nullptr where not wanted
  uint8_t *q, *q_scales;
  float* rstd;
  int64_t rows, cols, ldx, ldf, ldy, ldh;
  float eps;
  Drop drop;
  uint32_t up;                  // added to the bits of magnitudes (mx8.cuh)
  int vec;                      // rows and w 16-byte aligned
};

struct AddNormBwdArgs {
  const void *dy, *dh, *y;      // dy: nullptr for 0
  const float *w, *rstd;
  void *dx, *df;                // dx: nullptr where not wanted
  float* parts;                 // [CTAs][part_ld]: column sums of a CTA's rows
  int64_t rows, cols, lddy, lddh, ldy, lddx, lddf, part_ld;
  Drop drop;
  int vec;
};

// Before the launches.
cudaError_t add_norm_configure();
cudaError_t launch_add_norm_fwd(const AddNormFwdArgs& a, int dtype, int sms, cudaStream_t s);
// CTAs of the backward: each writes one row of parts.
int64_t add_norm_bwd_ctas(int64_t rows, int64_t cols, int sms);
cudaError_t launch_add_norm_bwd(const AddNormBwdArgs& a, int dtype, int64_t ctas, cudaStream_t s);

}  // namespace dmuon
