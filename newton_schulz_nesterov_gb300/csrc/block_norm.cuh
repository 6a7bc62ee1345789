// Norms after and before a block, fused with the block's gate and residual
// scale: arguments and host launchers.
//
// Forward, per row of `cols` channels (x the residual stream, f the block's
// output, g the gate row of the row's group):
//   r1 = 1 / sqrt(mean(f^2) + eps)     y = s x + g (f r1 w_post)
//   r2 = 1 / sqrt(mean(y^2) + eps)     h = y r2 w_pre
// Backward, from dy (gradient of y from later uses) and dh:
//   t  = dy + r2 (dh w_pre - yn mean(dh w_pre yn)),  yn = y r2
//   dx = s t,  ds = sum_rows t x,  dw_pre = sum_rows dh yn
//   dn = g t,  fn = f r1,  dw_post = sum_rows dn fn,  dg = sum_group t fn w_post
//   df = r1 (dn w_post - fn mean(dn w_post fn))
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace dmuon {

struct NormFwdArgs {
  const void *x, *f;
  const float *post_w, *pre_w, *gate, *res;   // gate, res may be nullptr
  void *y, *h;
  float* rstd;                                // [2][rows]
  int64_t rows, cols, ldx, ldf, ldy, ldh, per_gate;
  float eps;
  int* err;                                   // a wait inside a cluster ran out
  unsigned long long timeout_ns;              // its limit, 0: kWaitNs
  int vec;                                    // rows and parameters 16-byte aligned, columns a multiple of 8
};

// Rows are cut into chunks that lie inside one gate group, so that a chunk's
// column sum of t fn belongs to one gate row.
struct NormBwdArgs {
  const void *dy, *dh, *x, *f, *y;            // dy may be nullptr (0), x nullptr without d_res
  const float *post_w, *pre_w, *gate, *res, *rstd;
  void *dx, *df;
  float *d_post_w, *d_pre_w, *d_gate, *d_res;  // d_gate, d_res may be nullptr
  int64_t rows, cols, lddy, lddh, ldx, ldf, ldy, lddx, lddf, per_gate;
  int64_t groups, chunk_rows, chunks_per_group;
  int64_t units;                              // rows of each partial array
  int64_t part_ld;                            // pitch of the partial arrays: columns to a multiple of 4
  int cta_units;                              // units whose sums one CTA has added up in its first's row
  int* err;
  unsigned long long timeout_ns;
  int vec;
  float *part_pre, *part_post, *part_res;     // [units][cols]
  float* part_gate;                           // [groups * chunks_per_group][cols] (several chunks a group)
};

// Before the launches.
cudaError_t block_norm_configure();
// kept: what is asked of the device once, eight integers of the handle, 0 at first.
cudaError_t launch_norm_fwd(const NormFwdArgs& a, int dtype, int sms, int* kept, cudaStream_t s);
cudaError_t launch_norm_bwd(const NormBwdArgs& a, int dtype, cudaStream_t s);
// Row units of the backward pass: each writes one row of the partial arrays.
int64_t norm_bwd_units(int64_t rows, int64_t cols, int sms, int* kept);
int norm_bwd_cta_units(int64_t cols, int64_t units);

}  // namespace dmuon
