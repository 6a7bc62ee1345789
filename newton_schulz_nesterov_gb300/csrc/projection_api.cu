// Host side of the operators around an 8-bit projection (include/dmuon.h):
// MXFP8 quantisation and reading back, the projection with its epilogue, that
// epilogue's backward, the residual norm with dropout and dropout by itself.
// Argument checks and launches.
#include "../../include/dmuon.h"
#include "add_norm.cuh"
#include "dropout.cuh"
#include "mx.cuh"
#include "mx8.cuh"
#include "ops_api.cuh"

using namespace dmuon;

namespace {

bool sizes_ok(int64_t rows, int64_t cols) { return rows >= 0 && cols >= 0 && rows <= kMaxSide && cols <= kMaxSide; }
bool mode_ok(int mode) { return mode == DMUON_MXFP4_SCALE_FLOOR || mode == DMUON_MXFP4_SCALE_CEIL; }
uint32_t up_of(int mode) { return mode == DMUON_MXFP4_SCALE_CEIL ? mx8::kCeil : mx8::kFloor; }
int64_t part_pitch(int64_t cols) { return (cols + 31) / 32 * 32; }

// No pointer of `outs` is another's or one of `ins` (NULL: none).
template <int O, int I>
bool apart(const void* const (&outs)[O], const void* const (&ins)[I]) {
  for (int i = 0; i < O; ++i) {
    if (!outs[i]) continue;
    for (int j = 0; j < i; ++j)
      if (outs[i] == outs[j]) return false;
    for (const void* p : ins)
      if (p == outs[i]) return false;
  }
  return true;
}

// The 128 x 128 tiles of a matrix are numbered by 31 bits.
bool tiles_ok(int64_t rows, int64_t cols) { return ((rows + 127) / 128) * ((cols + 127) / 128) <= INT32_MAX; }

// Tiles that a CTA goes down, one after the other: as many as fill its ring and
// still leave six CTAs for each of two on an SM, so that their ends are spread.
int64_t tiles_down(const dmuon_ctx* h, int64_t rows, int64_t cols) {
  const int64_t rt = (rows + 127) / 128, ct = (cols + 127) / 128;
  return std::max<int64_t>(1, std::min<int64_t>(16, rt * ct / (12 * h->num_sms)));
}

}  // namespace

extern "C" {

int dmuon_mxfp8_bytes(int64_t rows, int64_t k, size_t* data_bytes, size_t* scale_bytes) {
  if (!sizes_ok(rows, k)) return DMUON_ERR_ARG;
  if (data_bytes) *data_bytes = (size_t)(rows * mx_pitch(k, 8));
  if (scale_bytes) *scale_bytes = (size_t)mx_scale_bytes(rows, k);
  return DMUON_OK;
}

int dmuon_mxfp8_quantize(dmuon_handle_t h, const void* src, int dtype, int64_t rows, int64_t cols, int64_t ld, int scale_mode,
                         void* row_data, void* row_scales, void* col_data, void* col_scales, void* stream_) {
  if (!h) return DMUON_ERR_ARG;
  if (!elem_size(dtype) || !sizes_ok(rows, cols) || !mode_ok(scale_mode))
    return fail(h, DMUON_ERR_ARG, "mxfp8_quantize: size, type or scale mode");
  const bool by_rows = row_data || row_scales, by_cols = col_data || col_scales;
  if (!by_rows && !by_cols) return fail(h, DMUON_ERR_ARG, "mxfp8_quantize: no output");
  if (rows == 0 || cols == 0) return DMUON_OK;
  int rc;
  if ((rc = check_matrix(h, src, dtype, cols, ld, "mxfp8_quantize: src"))) return rc;
  if (by_rows && (rc = check_packed(h, row_data, row_scales, "mxfp8_quantize: output by rows"))) return rc;
  if (by_cols && (rc = check_packed(h, col_data, col_scales, "mxfp8_quantize: output by columns"))) return rc;
  if (!apart({row_data, row_scales, col_data, col_scales}, {src}))
    return fail(h, DMUON_ERR_ARG, "mxfp8_quantize: an output is another or an input");
  if (!tiles_ok(rows, cols)) return fail(h, DMUON_ERR_ARG, "mxfp8_quantize: too many tiles");
  if (cudaSetDevice(h->device) != cudaSuccess) return fail(h, DMUON_ERR_CUDA, "cudaSetDevice");
  if ((rc = ready(h, h->quant8_ready, mx8_configure, "mxfp8_quantize: configure"))) return rc;
  cudaStream_t stream = (cudaStream_t)stream_;
  Mx8Args a{};
  a.src = src;
  a.rows = rows;
  a.cols = cols;
  a.ld = ld;
  a.row_data = (uint8_t*)row_data;
  a.row_scales = (uint8_t*)row_scales;
  a.col_data = (uint8_t*)col_data;
  a.col_scales = (uint8_t*)col_scales;
  a.tiles = tiles_down(h, rows, cols);
  a.up = up_of(scale_mode);
  a.vec = rows_aligned(src, ld, dtype);
  LaunchGuard g(h, stream, DMUON_KIND_MX_QUANTIZE);
  const cudaError_t e = launch_mx8_tiles(a, dtype, stream);
  if (e != cudaSuccess) return fail(h, cuda_err(e), "mxfp8_quantize launch", e);
  h->last_stream = stream;
  return DMUON_OK;
}

int dmuon_mxfp8_dequantize(dmuon_handle_t h, const void* data, const void* scales, int64_t rows, int64_t k, void* dst, int dtype,
                           int64_t ld, void* stream_) {
  if (!h) return DMUON_ERR_ARG;
  if (!elem_size(dtype) || !sizes_ok(rows, k)) return fail(h, DMUON_ERR_ARG, "mxfp8_dequantize: size or type");
  if (rows == 0 || k == 0) return DMUON_OK;
  int rc;
  if ((rc = check_packed(h, data, scales, "mxfp8_dequantize: matrix"))) return rc;
  if ((rc = check_matrix(h, dst, dtype, k, ld, "mxfp8_dequantize: dst"))) return rc;
  if (dst == data || dst == scales) return fail(h, DMUON_ERR_ARG, "mxfp8_dequantize: dst is an input");
  if (((rows + 31) / 32) * ((k + 255) / 256) > INT32_MAX) return fail(h, DMUON_ERR_ARG, "mxfp8_dequantize: too many tiles");
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
  const cudaError_t e = launch_mx8_dequant(a, dtype, stream);
  if (e != cudaSuccess) return fail(h, cuda_err(e), "mxfp8_dequantize launch", e);
  h->last_stream = stream;
  return DMUON_OK;
}

int dmuon_mx_linear(dmuon_handle_t h, const dmuon_mx_linear_t* p, void* stream_) {
  if (!h || !p) return DMUON_ERR_ARG;
  const int64_t m = p->m, n = p->n, k = p->k;
  if ((p->bits != 4 && p->bits != 8) || !elem_size(p->dtype) || !sizes_ok(m, n) || k < 1 || k > kMaxSide || !std::isfinite(p->alpha) ||
      !std::isfinite(p->beta) || p->act < DMUON_ACT_NONE || p->act > DMUON_ACT_GELU_TANH)
    return fail(h, DMUON_ERR_ARG, "mx_linear: format, size, type, factor or activation");
  if (m == 0 || n == 0) return DMUON_OK;
  int rc;
  if ((rc = check_packed(h, p->a_data, p->a_scales, "mx_linear: A")) || (rc = check_packed(h, p->b_data, p->b_scales, "mx_linear: B")) ||
      (rc = check_matrix(h, p->d, p->dtype, n, p->ldd, "mx_linear: D")) ||
      (p->pre && (rc = check_matrix(h, p->pre, p->dtype, n, p->ldpre, "mx_linear: pre"))) ||
      (p->c && (rc = check_matrix(h, p->c, p->dtype, n, p->ldc, "mx_linear: C"))))
    return rc;
  if (!aligned(p->bias, 4)) return fail(h, DMUON_ERR_ALIGN, "mx_linear: bias");
  if (!apart({p->d, p->pre}, {p->a_data, p->a_scales, p->b_data, p->b_scales, p->bias}) || (p->pre && p->pre == p->c))
    return fail(h, DMUON_ERR_ARG, "mx_linear: an output is another or an input");
  if (m > 1 && p->c == p->d && p->ldc != p->ldd) return fail(h, DMUON_ERR_ARG, "mx_linear: C is D with another leading dimension");
  if (!tensor_map_encoder()) return fail(h, DMUON_ERR_CUDA, "mx_linear: tensor-map encoder");
  if (cudaSetDevice(h->device) != cudaSuccess) return fail(h, DMUON_ERR_CUDA, "cudaSetDevice");
  const bool eight = p->bits == 8;
  if ((rc = ready(h, h->linear_ready[eight], eight ? mx_linear8_configure : mx_linear4_configure, "mx_linear: configure"))) return rc;
  MxLinearArgs a{};
  a.d = p->d;
  a.ldd = p->ldd;
  a.alpha = p->alpha;
  a.beta = p->beta;
  a.dtype = p->dtype;
  a.c = p->beta != 0.f ? p->c : nullptr;
  a.ldc = p->ldc;
  a.bias = p->bias;
  a.pre = p->pre;
  a.ldpre = p->ldpre;
  a.act = act_of(p->act);
  a.vec = rows_aligned(p->d, p->ldd, p->dtype) && (!a.c || rows_aligned(a.c, a.ldc, p->dtype)) &&
          (!p->pre || rows_aligned(p->pre, p->ldpre, p->dtype)) && aligned(p->bias, 16);
  const Product<MxLinearArgs> product = eight ? Product<MxLinearArgs>{8, launch_mx_linear8, launch_mx_linear8_pair}
                                              : Product<MxLinearArgs>{4, launch_mx_linear4, launch_mx_linear4_pair};
  return launch_product(h, a, product, p->a_data, p->a_scales, p->b_data, p->b_scales, m, n, k, (cudaStream_t)stream_,
                        "mx_linear: tiles, tensor map or launch");
}

int dmuon_act_backward(dmuon_handle_t h, const dmuon_act_backward_t* p, void* stream_) {
  if (!h || !p) return DMUON_ERR_ARG;
  const int64_t rows = p->rows, cols = p->cols;
  if (!elem_size(p->dtype) || !sizes_ok(rows, cols) || !mode_ok(p->scale_mode) || p->act < DMUON_ACT_NONE || p->act > DMUON_ACT_GELU_TANH)
    return fail(h, DMUON_ERR_ARG, "act_backward: size, type, activation or scale mode");
  const bool by_rows = p->row_data || p->row_scales, by_cols = p->col_data || p->col_scales;
  if (cols == 0 || (rows == 0 && !p->d_bias)) return DMUON_OK;
  if (!by_rows && !by_cols && !p->dz && !p->d_bias) return fail(h, DMUON_ERR_ARG, "act_backward: no output");
  const void* pre = p->act == DMUON_ACT_NONE ? nullptr : p->pre;
  int rc = DMUON_OK;
  if (rows > 0) {
    if ((rc = check_matrix(h, p->dout, p->dtype, cols, p->lddout, "act_backward: dout")) ||
        (p->act != DMUON_ACT_NONE && (rc = check_matrix(h, pre, p->dtype, cols, p->ldpre, "act_backward: pre"))) ||
        (p->dz && (rc = check_matrix(h, p->dz, p->dtype, cols, p->lddz, "act_backward: dz"))) ||
        (by_rows && (rc = check_packed(h, p->row_data, p->row_scales, "act_backward: output by rows"))) ||
        (by_cols && (rc = check_packed(h, p->col_data, p->col_scales, "act_backward: output by columns"))))
      return rc;
    if (!apart({p->row_data, p->row_scales, p->col_data, p->col_scales, p->dz, p->d_bias}, {p->dout, pre}))
      return fail(h, DMUON_ERR_ARG, "act_backward: an output is another or an input");
  }
  if (!aligned(p->d_bias, 4)) return fail(h, DMUON_ERR_ALIGN, "act_backward: d_bias");
  if (!tiles_ok(rows, cols)) return fail(h, DMUON_ERR_ARG, "act_backward: too many tiles");
  if (cudaSetDevice(h->device) != cudaSuccess) return fail(h, DMUON_ERR_CUDA, "cudaSetDevice");
  if ((rc = pre ? ready(h, h->act_ready, mx8_act_configure, "act_backward: configure") : ready(h, h->quant8_ready, mx8_configure, "act_backward: configure"))) return rc;
  cudaStream_t stream = (cudaStream_t)stream_;
  Mx8Args a{};
  a.src = p->dout;
  a.pre = pre;
  a.act = act_of(p->act);
  a.rows = rows;
  a.cols = cols;
  a.ld = p->lddout;
  a.ldpre = p->ldpre;
  a.row_data = (uint8_t*)p->row_data;
  a.row_scales = (uint8_t*)p->row_scales;
  a.col_data = (uint8_t*)p->col_data;
  a.col_scales = (uint8_t*)p->col_scales;
  a.dz = p->dz;
  a.lddz = p->lddz;
  a.up = up_of(p->scale_mode);
  a.vec = rows_aligned(p->dout, p->lddout, p->dtype) && (!pre || rows_aligned(pre, p->ldpre, p->dtype)) &&
          (!p->dz || rows_aligned(p->dz, p->lddz, p->dtype));
  const int64_t rt = (rows + 127) / 128;
  a.tiles = tiles_down(h, rows, cols);
  const int64_t chunks = (rt + a.tiles - 1) / a.tiles;
  if (p->d_bias) {
    a.part_ld = part_pitch(cols);
    a.parts = p->d_bias;
    if (chunks > 1) {
      if ((rc = op_workspace(h, (size_t)chunks * a.part_ld * 4, stream, "act_backward: workspace (the first call of a larger size is not captured)")))
        return rc;
      a.parts = (float*)h->op_ws;
    }
  }
  LaunchGuard g(h, stream, DMUON_KIND_ACT_BWD);
  cudaError_t e = cudaSuccess;
  if (rows > 0) e = pre ? launch_mx8_act(a, p->dtype, stream) : launch_mx8_tiles(a, p->dtype, stream);
  if (e == cudaSuccess && p->d_bias && chunks != 1) {
    if (rows > 0) ++h->launches;
    e = launch_column_sums(a.parts, chunks, a.part_ld, cols, p->d_bias, stream);
  }
  if (e != cudaSuccess) return fail(h, cuda_err(e), "act_backward launch", e);
  h->last_stream = stream;
  return DMUON_OK;
}

int dmuon_add_norm_forward(dmuon_handle_t h, const dmuon_add_norm_t* p, void* stream_) {
  if (!h || !p) return DMUON_ERR_ARG;
  const int64_t rows = p->rows, cols = p->cols;
  AddNormFwdArgs a{};
  if (!elem_size(p->dtype) || !sizes_ok(rows, cols) || cols < 1 || !std::isfinite(p->eps) || p->eps < 0.f || !mode_ok(p->scale_mode) ||
      !drop_of(p->p, p->seed, p->offset, &a.drop))
    return fail(h, DMUON_ERR_ARG, "add_norm_forward: size, type, eps, scale mode or p");
  const bool q = p->q_data || p->q_scales;
  if (rows == 0) return DMUON_OK;
  if (!p->h && !q) return fail(h, DMUON_ERR_ARG, "add_norm_forward: neither h nor q");
  int rc;
  if ((p->x && (rc = check_matrix(h, p->x, p->dtype, cols, p->ldx, "add_norm_forward: x"))) ||
      (rc = check_matrix(h, p->f, p->dtype, cols, p->ldf, "add_norm_forward: f")) ||
      (rc = check_matrix(h, p->y, p->dtype, cols, p->ldy, "add_norm_forward: y")) ||
      (p->h && (rc = check_matrix(h, p->h, p->dtype, cols, p->ldh, "add_norm_forward: h"))) ||
      (q && (rc = check_packed(h, p->q_data, p->q_scales, "add_norm_forward: q"))) ||
      (rc = check_matrix(h, p->w, DMUON_F32, 0, 0, "add_norm_forward: w")) ||
      (rc = check_matrix(h, p->rstd, DMUON_F32, 0, 0, "add_norm_forward: rstd")))
    return rc;
  if (!apart({p->y, p->h, p->q_data, p->q_scales, p->rstd}, {p->x, p->f, p->w}))
    return fail(h, DMUON_ERR_ARG, "add_norm_forward: an output is another or an input");
  if (cudaSetDevice(h->device) != cudaSuccess) return fail(h, DMUON_ERR_CUDA, "cudaSetDevice");
  if ((rc = ready(h, h->add_norm_ready, add_norm_configure, "add_norm_forward: configure"))) return rc;
  cudaStream_t stream = (cudaStream_t)stream_;
  a.x = p->x;
  a.f = p->f;
  a.w = p->w;
  a.y = p->y;
  a.h = p->h;
  a.q = (uint8_t*)p->q_data;
  a.q_scales = (uint8_t*)p->q_scales;
  a.rstd = p->rstd;
  a.rows = rows;
  a.cols = cols;
  a.ldx = p->ldx;
  a.ldf = p->ldf;
  a.ldy = p->ldy;
  a.ldh = p->ldh;
  a.eps = p->eps;
  a.up = up_of(p->scale_mode);
  a.vec = aligned(p->w, 16) && rows_aligned(p->f, p->ldf, p->dtype) && rows_aligned(p->y, p->ldy, p->dtype) &&
          (!p->x || rows_aligned(p->x, p->ldx, p->dtype)) && (!p->h || rows_aligned(p->h, p->ldh, p->dtype));
  LaunchGuard g(h, stream, DMUON_KIND_ADD_NORM_FWD);
  const cudaError_t e = launch_add_norm_fwd(a, p->dtype, h->num_sms, stream);
  if (e != cudaSuccess) return fail(h, cuda_err(e), "add_norm_forward launch", e);
  h->last_stream = stream;
  return DMUON_OK;
}

int dmuon_add_norm_backward(dmuon_handle_t h, const dmuon_add_norm_t* p, const dmuon_add_norm_grad_t* g_, void* stream_) {
  if (!h || !p || !g_) return DMUON_ERR_ARG;
  const int64_t rows = p->rows, cols = p->cols;
  AddNormBwdArgs a{};
  if (!elem_size(p->dtype) || !sizes_ok(rows, cols) || cols < 1 || !drop_of(p->p, p->seed, p->offset, &a.drop))
    return fail(h, DMUON_ERR_ARG, "add_norm_backward: size, type or p");
  int rc = DMUON_OK;
  if (rows > 0) {
    if ((g_->dy && (rc = check_matrix(h, g_->dy, p->dtype, cols, g_->lddy, "add_norm_backward: dy"))) ||
        (rc = check_matrix(h, g_->dh, p->dtype, cols, g_->lddh, "add_norm_backward: dh")) ||
        (rc = check_matrix(h, p->y, p->dtype, cols, p->ldy, "add_norm_backward: y")) ||
        (g_->dx && (rc = check_matrix(h, g_->dx, p->dtype, cols, g_->lddx, "add_norm_backward: dx"))) ||
        (rc = check_matrix(h, g_->df, p->dtype, cols, g_->lddf, "add_norm_backward: df")) ||
        (rc = check_matrix(h, p->w, DMUON_F32, 0, 0, "add_norm_backward: w")) ||
        (rc = check_matrix(h, p->rstd, DMUON_F32, 0, 0, "add_norm_backward: rstd")))
      return rc;
    if (!apart({g_->dx, g_->df, g_->d_w}, {g_->dy, g_->dh, p->y, p->w, p->rstd}))
      return fail(h, DMUON_ERR_ARG, "add_norm_backward: an output is another or an input");
  }
  if ((rc = check_matrix(h, g_->d_w, DMUON_F32, 0, 0, "add_norm_backward: d_w"))) return rc;
  if (cudaSetDevice(h->device) != cudaSuccess) return fail(h, DMUON_ERR_CUDA, "cudaSetDevice");
  if ((rc = ready(h, h->add_norm_ready, add_norm_configure, "add_norm_backward: configure"))) return rc;
  cudaStream_t stream = (cudaStream_t)stream_;
  a.dy = g_->dy;
  a.dh = g_->dh;
  a.y = p->y;
  a.w = p->w;
  a.rstd = p->rstd;
  a.dx = g_->dx;
  a.df = g_->df;
  a.rows = rows;
  a.cols = cols;
  a.lddy = g_->lddy;
  a.lddh = g_->lddh;
  a.ldy = p->ldy;
  a.lddx = g_->lddx;
  a.lddf = g_->lddf;
  a.vec = aligned(p->w, 16) && rows_aligned(g_->dh, g_->lddh, p->dtype) && rows_aligned(p->y, p->ldy, p->dtype) &&
          rows_aligned(g_->df, g_->lddf, p->dtype) && (!g_->dy || rows_aligned(g_->dy, g_->lddy, p->dtype)) &&
          (!g_->dx || rows_aligned(g_->dx, g_->lddx, p->dtype));
  const int64_t ctas = add_norm_bwd_ctas(rows, cols, h->num_sms);
  a.part_ld = part_pitch(cols);
  a.parts = g_->d_w;
  if (ctas > 1) {
    if ((rc = op_workspace(h, (size_t)ctas * a.part_ld * 4, stream, "add_norm_backward: workspace (the first call of a larger size is not captured)")))
      return rc;
    a.parts = (float*)h->op_ws;
  }
  LaunchGuard g(h, stream, DMUON_KIND_ADD_NORM_BWD);
  cudaError_t e = cudaSuccess;
  if (rows > 0) e = launch_add_norm_bwd(a, p->dtype, ctas, stream);
  if (e == cudaSuccess && ctas != 1) {  // no rows: zeros
    if (rows > 0) ++h->launches;
    e = launch_column_sums(a.parts, ctas, a.part_ld, cols, g_->d_w, stream);
  }
  if (e != cudaSuccess) return fail(h, cuda_err(e), "add_norm_backward launch", e);
  h->last_stream = stream;
  return DMUON_OK;
}

int dmuon_dropout(dmuon_handle_t h, const void* x, int dtype, int64_t rows, int64_t cols, int64_t ldx, const void* residual,
                  int64_t ldres, void* out, int64_t ldout, float p, uint64_t seed, uint64_t offset, void* stream_) {
  if (!h) return DMUON_ERR_ARG;
  DropoutArgs a{};
  if (!elem_size(dtype) || !sizes_ok(rows, cols) || !drop_of(p, seed, offset, &a.drop))
    return fail(h, DMUON_ERR_ARG, "dropout: size, type or p");
  if (rows == 0 || cols == 0) return DMUON_OK;
  int rc;
  if ((rc = check_matrix(h, x, dtype, cols, ldx, "dropout: x")) ||
      (residual && (rc = check_matrix(h, residual, dtype, cols, ldres, "dropout: residual"))) ||
      (rc = check_matrix(h, out, dtype, cols, ldout, "dropout: out")))
    return rc;
  if (rows > 1 && ((out == x && ldout != ldx) || (out == residual && ldout != ldres)))
    return fail(h, DMUON_ERR_ARG, "dropout: out is an input with another leading dimension");
  if (((rows + 7) / 8) * ((cols + 255) / 256) > INT32_MAX) return fail(h, DMUON_ERR_ARG, "dropout: too many tiles");
  if (cudaSetDevice(h->device) != cudaSuccess) return fail(h, DMUON_ERR_CUDA, "cudaSetDevice");
  cudaStream_t stream = (cudaStream_t)stream_;
  a.x = x;
  a.res = residual;
  a.out = out;
  a.rows = rows;
  a.cols = cols;
  a.ldx = ldx;
  a.ldres = ldres;
  a.ldout = ldout;
  a.vec = rows_aligned(x, ldx, dtype) && rows_aligned(out, ldout, dtype) && (!residual || rows_aligned(residual, ldres, dtype));
  LaunchGuard g(h, stream, DMUON_KIND_DROPOUT);
  const cudaError_t e = launch_dropout(a, dtype, h->num_sms, stream);
  if (e != cudaSuccess) return fail(h, cuda_err(e), "dropout launch", e);
  h->last_stream = stream;
  return DMUON_OK;
}

}  // extern "C"
