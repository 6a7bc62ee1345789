// Host side of the operators around a 4-bit projection (include/dmuon.h):
// MXFP4 quantisation, reading back and product, and the norms around a block.
// Argument checks and launches (tile choice and workspace in ops_api.cuh).
#include <algorithm>
#include <cmath>

#include "../../include/dmuon.h"
#include "block_norm.cuh"
#include "mx.cuh"
#include "ops_api.cuh"

using namespace dmuon;

extern "C" {

int dmuon_mxfp4_bytes(int64_t rows, int64_t k, size_t* data_bytes, size_t* scale_bytes) {
  if (rows < 0 || k < 0 || rows > kMaxSide || k > kMaxSide) return DMUON_ERR_ARG;
  if (data_bytes) *data_bytes = (size_t)(rows * mx_pitch(k));
  if (scale_bytes) *scale_bytes = (size_t)mx_scale_bytes(rows, k);
  return DMUON_OK;
}

int dmuon_mxfp4_quantize(dmuon_handle_t h, const void* src, int dtype, int64_t rows, int64_t cols, int64_t ld,
                         int scale_mode, const uint8_t* noise, int64_t noise_ld, void* row_data, void* row_scales,
                         void* col_data, void* col_scales, void* stream_) {
  if (!h) return DMUON_ERR_ARG;
  if (!elem_size(dtype) || rows < 0 || cols < 0 || rows > kMaxSide || cols > kMaxSide ||
      (scale_mode != DMUON_MXFP4_SCALE_FLOOR && scale_mode != DMUON_MXFP4_SCALE_CEIL))
    return fail(h, DMUON_ERR_ARG, "mxfp4_quantize: size, type or scale mode");
  const bool by_rows = row_data || row_scales, by_cols = col_data || col_scales;
  if (!by_rows && !by_cols) return fail(h, DMUON_ERR_ARG, "mxfp4_quantize: no output");
  if (rows == 0 || cols == 0) return DMUON_OK;
  int rc;
  if ((rc = check_matrix(h, src, dtype, cols, ld, "mxfp4_quantize: src"))) return rc;
  if (noise && noise_ld < cols) return fail(h, DMUON_ERR_ARG, "mxfp4_quantize: noise");
  if (by_rows && (rc = check_packed(h, row_data, row_scales, "mxfp4_quantize: output by rows"))) return rc;
  if (by_cols && (rc = check_packed(h, col_data, col_scales, "mxfp4_quantize: output by columns"))) return rc;
  const void* outs[4] = {row_data, row_scales, col_data, col_scales};
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < i; ++j)
      if (outs[i] && outs[i] == outs[j]) return fail(h, DMUON_ERR_ARG, "mxfp4_quantize: outputs overlap");
  for (const void* o : outs)
    if (o && (o == src || o == (const void*)noise)) return fail(h, DMUON_ERR_ARG, "mxfp4_quantize: an output is an input");
  if (((rows + 127) / 128) * ((cols + 127) / 128) > INT32_MAX)
    return fail(h, DMUON_ERR_ARG, "mxfp4_quantize: too many tiles");
  if (cudaSetDevice(h->device) != cudaSuccess) return fail(h, DMUON_ERR_CUDA, "cudaSetDevice");
  if ((rc = ready(h, h->quant_ready, mx_quant_configure, "mxfp4_quantize: configure"))) return rc;
  cudaStream_t stream = (cudaStream_t)stream_;
  MxQuantArgs a{};
  a.src = src;
  a.rows = rows;
  a.cols = cols;
  a.ld = ld;
  a.noise = noise;
  a.noise_ld = noise_ld;
  a.row_data = (uint8_t*)row_data;
  a.row_scales = (uint8_t*)row_scales;
  a.col_data = (uint8_t*)col_data;
  a.col_scales = (uint8_t*)col_scales;
  a.ceil_scale = scale_mode == DMUON_MXFP4_SCALE_CEIL;
  a.vec = aligned(src, 16) && (ld * elem_size(dtype)) % 16 == 0;
  a.noise_vec = noise && aligned(noise, 16) && noise_ld % 16 == 0;
  LaunchGuard g(h, stream, DMUON_KIND_MX_QUANTIZE);
  const cudaError_t e = launch_mx_quant(a, dtype, stream);
  if (e != cudaSuccess) return fail(h, cuda_err(e), "mxfp4_quantize launch", e);
  h->last_stream = stream;
  return DMUON_OK;
}

int dmuon_mxfp4_dequantize(dmuon_handle_t h, const void* data, const void* scales, int64_t rows, int64_t k, void* dst,
                           int dtype, int64_t ld, void* stream_) {
  if (!h) return DMUON_ERR_ARG;
  if (!elem_size(dtype) || rows < 0 || k < 0 || rows > kMaxSide || k > kMaxSide)
    return fail(h, DMUON_ERR_ARG, "mxfp4_dequantize: size or type");
  if (rows == 0 || k == 0) return DMUON_OK;
  int rc;
  if ((rc = check_packed(h, data, scales, "mxfp4_dequantize: matrix"))) return rc;
  if ((rc = check_matrix(h, dst, dtype, k, ld, "mxfp4_dequantize: dst"))) return rc;
  if (dst == data || dst == scales) return fail(h, DMUON_ERR_ARG, "mxfp4_dequantize: dst is an input");
  if (((rows + 31) / 32) * ((k + 255) / 256) > INT32_MAX) return fail(h, DMUON_ERR_ARG, "mxfp4_dequantize: too many tiles");
  if (cudaSetDevice(h->device) != cudaSuccess) return fail(h, DMUON_ERR_CUDA, "cudaSetDevice");
  cudaStream_t stream = (cudaStream_t)stream_;
  MxDequantArgs a{};
  a.data = (const uint8_t*)data;
  a.scales = (const uint8_t*)scales;
  a.rows = rows;
  a.k = k;
  a.dst = dst;
  a.ld = ld;
  a.vec = aligned(dst, 32) && (ld * elem_size(dtype)) % 32 == 0;
  LaunchGuard g(h, stream, DMUON_KIND_MX_DEQUANTIZE);
  const cudaError_t e = launch_mx_dequant(a, dtype, stream);
  if (e != cudaSuccess) return fail(h, cuda_err(e), "mxfp4_dequantize launch", e);
  h->last_stream = stream;
  return DMUON_OK;
}

int dmuon_mxfp4_gemm(dmuon_handle_t h, const void* a_data, const void* a_scales, const void* b_data,
                     const void* b_scales, int64_t m, int64_t n, int64_t k, void* d, int dtype, int64_t ldd,
                     float alpha, float beta, void* stream_) {
  if (!h) return DMUON_ERR_ARG;
  if (!elem_size(dtype) || m < 0 || n < 0 || k < 1 || m > kMaxSide || n > kMaxSide || k > kMaxSide ||
      !std::isfinite(alpha) || !std::isfinite(beta))
    return fail(h, DMUON_ERR_ARG, "mxfp4_gemm: size, type or factor");
  if (m == 0 || n == 0) return DMUON_OK;
  int rc;
  if ((rc = check_packed(h, a_data, a_scales, "mxfp4_gemm: A"))) return rc;
  if ((rc = check_packed(h, b_data, b_scales, "mxfp4_gemm: B"))) return rc;
  if ((rc = check_matrix(h, d, dtype, n, ldd, "mxfp4_gemm: D"))) return rc;
  if (d == a_data || d == a_scales || d == b_data || d == b_scales)
    return fail(h, DMUON_ERR_ARG, "mxfp4_gemm: D is an operand");
  if (!tensor_map_encoder()) return fail(h, DMUON_ERR_CUDA, "mxfp4_gemm: tensor-map encoder");
  if (cudaSetDevice(h->device) != cudaSuccess) return fail(h, DMUON_ERR_CUDA, "cudaSetDevice");
  cudaStream_t stream = (cudaStream_t)stream_;
  MxGemmArgs a{};
  a.d = d;
  a.ldd = ldd;
  a.alpha = alpha;
  a.beta = beta;
  a.dtype = dtype;
  a.vec = rows_aligned(d, ldd, dtype);
  const Product<MxGemmArgs> product{4, launch_mx_gemm, launch_mx_gemm_pair};
  return launch_product(h, a, product, a_data, a_scales, b_data, b_scales, m, n, k, stream, "mxfp4_gemm: tiles, tensor map or launch");
}

int dmuon_block_norm_forward(dmuon_handle_t h, const dmuon_block_norm_t* p, void* stream_) {
  if (!h || !p) return DMUON_ERR_ARG;
  const int64_t cols = p->cols;
  if (!elem_size(p->dtype) || p->rows < 0 || cols < 1 || p->rows > kMaxSide || cols > kMaxSide || p->rows_per_gate < 1 ||
      !std::isfinite(p->eps) || p->eps < 0.f)
    return fail(h, DMUON_ERR_ARG, "block_norm_forward: size, type or eps");
  if (p->rows == 0) return DMUON_OK;
  int rc;
  if ((rc = check_matrix(h, p->x, p->dtype, cols, p->ldx, "block_norm_forward: x")) ||
      (rc = check_matrix(h, p->f, p->dtype, cols, p->ldf, "block_norm_forward: f")) ||
      (rc = check_matrix(h, p->y, p->dtype, cols, p->ldy, "block_norm_forward: y")) ||
      (rc = check_matrix(h, p->h, p->dtype, cols, p->ldh, "block_norm_forward: h")) ||
      (rc = check_matrix(h, p->post_w, DMUON_F32, 0, 0, "block_norm_forward: post_w")) ||
      (rc = check_matrix(h, p->pre_w, DMUON_F32, 0, 0, "block_norm_forward: pre_w")) ||
      (rc = check_matrix(h, p->rstd, DMUON_F32, 0, 0, "block_norm_forward: rstd")))
    return rc;
  if (!aligned(p->gate, 4) || !aligned(p->res_scale, 4)) return fail(h, DMUON_ERR_ALIGN, "block_norm_forward: gate or res_scale");
  if (p->y == p->h || p->y == p->x || p->y == p->f || p->h == p->x || p->h == p->f)
    return fail(h, DMUON_ERR_ARG, "block_norm_forward: outputs overlap");
  if (cudaSetDevice(h->device) != cudaSuccess) return fail(h, DMUON_ERR_CUDA, "cudaSetDevice");
  if ((rc = ready(h, h->norm_ready, block_norm_configure, "block_norm_forward: configure"))) return rc;
  cudaStream_t stream = (cudaStream_t)stream_;
  NormFwdArgs a{};
  a.x = p->x;
  a.f = p->f;
  a.post_w = p->post_w;
  a.pre_w = p->pre_w;
  a.gate = p->gate;
  a.res = p->res_scale;
  a.y = p->y;
  a.h = p->h;
  a.rstd = p->rstd;
  a.rows = p->rows;
  a.cols = cols;
  a.ldx = p->ldx;
  a.ldf = p->ldf;
  a.ldy = p->ldy;
  a.ldh = p->ldh;
  a.per_gate = p->rows_per_gate;
  a.eps = p->eps;
  a.err = h->d_op_err;
  a.timeout_ns = h->wait_timeout_ns;
  a.vec = cols % 8 == 0 && rows_aligned(p->x, p->ldx, p->dtype) && rows_aligned(p->f, p->ldf, p->dtype) &&
          rows_aligned(p->y, p->ldy, p->dtype) && rows_aligned(p->h, p->ldh, p->dtype) && aligned(p->post_w, 16) &&
          aligned(p->pre_w, 16) && aligned(p->gate, 16) && aligned(p->res_scale, 16);
  LaunchGuard g(h, stream, DMUON_KIND_NORM_FWD);
  const cudaError_t e = launch_norm_fwd(a, p->dtype, h->num_sms, h->norm_places, stream);
  if (e != cudaSuccess) return fail(h, cuda_err(e), "block_norm_forward launch", e);
  h->last_stream = stream;
  return DMUON_OK;
}

int dmuon_block_norm_backward(dmuon_handle_t h, const dmuon_block_norm_t* p, const dmuon_block_norm_grad_t* q,
                              void* stream_) {
  if (!h || !p || !q) return DMUON_ERR_ARG;
  const int64_t cols = p->cols, rows = p->rows;
  if (!elem_size(p->dtype) || rows < 0 || cols < 1 || rows > kMaxSide || cols > kMaxSide || p->rows_per_gate < 1)
    return fail(h, DMUON_ERR_ARG, "block_norm_backward: size or type");
  if ((q->d_gate && !p->gate) || (q->d_res_scale && !p->res_scale))
    return fail(h, DMUON_ERR_ARG, "block_norm_backward: gradient of an absent gate or scale");
  int rc = DMUON_OK;
  if (rows > 0 && ((q->dy && (rc = check_matrix(h, q->dy, p->dtype, cols, q->lddy, "block_norm_backward: dy"))) ||
                   (rc = check_matrix(h, q->dh, p->dtype, cols, q->lddh, "block_norm_backward: dh")) ||
                   (rc = check_matrix(h, p->f, p->dtype, cols, p->ldf, "block_norm_backward: f")) ||
                   (rc = check_matrix(h, p->y, p->dtype, cols, p->ldy, "block_norm_backward: y")) ||
                   (q->d_res_scale && (rc = check_matrix(h, p->x, p->dtype, cols, p->ldx, "block_norm_backward: x"))) ||
                   (rc = check_matrix(h, q->dx, p->dtype, cols, q->lddx, "block_norm_backward: dx")) ||
                   (rc = check_matrix(h, q->df, p->dtype, cols, q->lddf, "block_norm_backward: df")) ||
                   (rc = check_matrix(h, p->rstd, DMUON_F32, 0, 0, "block_norm_backward: rstd"))))
    return rc;
  if ((rc = check_matrix(h, p->post_w, DMUON_F32, 0, 0, "block_norm_backward: post_w")) ||
      (rc = check_matrix(h, p->pre_w, DMUON_F32, 0, 0, "block_norm_backward: pre_w")) ||
      (rc = check_matrix(h, q->d_post_w, DMUON_F32, 0, 0, "block_norm_backward: d_post_w")) ||
      (rc = check_matrix(h, q->d_pre_w, DMUON_F32, 0, 0, "block_norm_backward: d_pre_w")))
    return rc;
  if (!aligned(p->gate, 4) || !aligned(p->res_scale, 4) || !aligned(q->d_gate, 4) || !aligned(q->d_res_scale, 4))
    return fail(h, DMUON_ERR_ALIGN, "block_norm_backward: gate or res_scale");
  const void* ins[] = {q->dy, q->dh, p->x, p->f, p->y};
  if (rows > 0) {
    if (q->dx == q->df) return fail(h, DMUON_ERR_ARG, "block_norm_backward: outputs overlap");
    for (const void* i : ins)
      if (i && (i == q->dx || i == q->df)) return fail(h, DMUON_ERR_ARG, "block_norm_backward: an output is an input");
  }
  if (q->d_post_w == q->d_pre_w) return fail(h, DMUON_ERR_ARG, "block_norm_backward: outputs overlap");
  if (cudaSetDevice(h->device) != cudaSuccess) return fail(h, DMUON_ERR_CUDA, "cudaSetDevice");
  if ((rc = ready(h, h->norm_ready, block_norm_configure, "block_norm_backward: configure"))) return rc;
  cudaStream_t stream = (cudaStream_t)stream_;
  NormBwdArgs a{};
  a.dy = q->dy;
  a.dh = q->dh;
  a.x = p->x;
  a.f = p->f;
  a.y = p->y;
  a.post_w = p->post_w;
  a.pre_w = p->pre_w;
  a.gate = p->gate;
  a.res = p->res_scale;
  a.rstd = p->rstd;
  a.dx = q->dx;
  a.df = q->df;
  a.d_post_w = q->d_post_w;
  a.d_pre_w = q->d_pre_w;
  a.d_gate = q->d_gate;
  a.d_res = q->d_res_scale;
  a.rows = rows;
  a.cols = cols;
  a.lddy = q->lddy;
  a.lddh = q->lddh;
  a.ldx = p->ldx;
  a.ldf = p->ldf;
  a.ldy = p->ldy;
  a.lddx = q->lddx;
  a.lddf = q->lddf;
  a.per_gate = p->gate ? std::min(p->rows_per_gate, std::max<int64_t>(rows, 1)) : std::max<int64_t>(rows, 1);
  a.groups = (rows + a.per_gate - 1) / a.per_gate;
  a.units = norm_bwd_units(rows, cols, h->num_sms, h->norm_places);
  a.cta_units = norm_bwd_cta_units(cols, a.units);
  a.err = h->d_op_err;
  a.timeout_ns = h->wait_timeout_ns;
  // Chunks lie inside a group; no more of them than units where that can be,
  // so that no unit has two while another has one.
  a.chunks_per_group = std::max<int64_t>(1, std::min(a.per_gate, a.units / std::max<int64_t>(1, a.groups)));
  a.chunk_rows = (a.per_gate + a.chunks_per_group - 1) / a.chunks_per_group;
  a.chunks_per_group = (a.per_gate + a.chunk_rows - 1) / a.chunk_rows;
  a.vec = cols % 8 == 0;
  const struct { const void* p; int64_t ld; } mats[] = {{q->dy, q->lddy}, {q->dh, q->lddh}, {q->d_res_scale ? p->x : nullptr, p->ldx},
                                                        {p->f, p->ldf}, {p->y, p->ldy}, {q->dx, q->lddx}, {q->df, q->lddf}};
  for (const auto& m : mats)
    if (m.p && !rows_aligned(m.p, m.ld, p->dtype)) a.vec = 0;
  for (const void* v : {(const void*)p->post_w, (const void*)p->pre_w, (const void*)p->gate, (const void*)p->res_scale,
                        (const void*)q->d_gate})
    if (!aligned(v, 16)) a.vec = 0;
  a.part_ld = (cols + 3) / 4 * 4;
  const size_t line = (size_t)a.part_ld * 4;
  const bool gate_parts = q->d_gate && a.chunks_per_group > 1;
  const size_t need = line * ((size_t)a.units * (q->d_res_scale ? 3 : 2) +
                              (gate_parts ? (size_t)(a.groups * a.chunks_per_group) : 0));
  if ((rc = op_workspace(h, need, stream, "block_norm_backward: workspace (the first call of a larger size is not captured)"))) return rc;
  float* w = (float*)h->op_ws;
  a.part_pre = w;
  a.part_post = w + (size_t)a.units * a.part_ld;
  a.part_res = a.part_post + (size_t)a.units * a.part_ld;
  a.part_gate = a.part_post + (size_t)a.units * a.part_ld * (q->d_res_scale ? 2 : 1);
  LaunchGuard g(h, stream, DMUON_KIND_NORM_BWD);
  ++h->launches;  // rows, then column sums
  const cudaError_t e = launch_norm_bwd(a, p->dtype, stream);
  if (e != cudaSuccess) return fail(h, cuda_err(e), "block_norm_backward launch", e);
  h->last_stream = stream;
  return DMUON_OK;
}

}  // extern "C"
