// Host side of the operators around a 4-bit projection (include/dmuon.h):
// MXFP4 quantisation, reading back and product, and the norms around a block.
// Argument checks, tensor maps, tile choice, workspace and launches.
#include <algorithm>
#include <cmath>

#include "../../include/dmuon.h"
#include "block_norm.cuh"
#include "ctx.cuh"
#include "mxfp4.cuh"

using namespace dmuon;

namespace {

constexpr int64_t kMaxSide = int64_t(1) << 30;

int elem_size(int dtype) {
  switch (dtype) {
    case DMUON_F32: return 4;
    case DMUON_BF16: case DMUON_F16: return 2;
    default: return 0;
  }
}

bool aligned(const void* p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }

// Every row starts on 16 bytes.
bool rows_aligned(const void* p, int64_t ld, int dtype) { return aligned(p, 16) && (ld * elem_size(dtype)) % 16 == 0; }

// A rows x cols matrix of `dtype` at p with leading dimension ld: DMUON_OK or
// the error code (also recorded).
int check_matrix(dmuon_ctx* h, const void* p, int dtype, int64_t cols, int64_t ld, const char* what) {
  if (!p || ld < cols) return fail(h, DMUON_ERR_ARG, what);
  if (!aligned(p, elem_size(dtype))) return fail(h, DMUON_ERR_ALIGN, what);
  return DMUON_OK;
}

int check_packed(dmuon_ctx* h, const void* data, const void* scales, const char* what) {
  if (!data || !scales || data == scales) return fail(h, DMUON_ERR_ARG, what);
  if (!aligned(data, 16) || !aligned(scales, 16)) return fail(h, DMUON_ERR_ALIGN, what);
  return DMUON_OK;
}

// The kernels' limits of shared memory, set by a handle's first call (loading
// the norms' kernels takes 15 ms, which a handle without norms does not pay).
int ready(dmuon_ctx* h, bool& done, cudaError_t (*configure)(), const char* what) {
  if (done) return DMUON_OK;
  const cudaError_t e = configure();
  if (e != cudaSuccess) return fail(h, cuda_err(e), what, e);
  done = true;
  return DMUON_OK;
}

bool encode(CUtensorMap* map, CUtensorMapDataType type, int dims, void* base, const cuuint64_t* size,
            const cuuint64_t* stride, const cuuint32_t* box, CUtensorMapSwizzle swizzle) {
  const cuuint32_t one[3] = {1, 1, 1};
  return tensor_map_encoder()(map, type, dims, base, size, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Maps of one operand: boxes of box_rows x 128 bytes of codes (256 elements
// of K) and of two scale tiles for each of `scale_tiles` x 128 rows.
bool operand_maps(CUtensorMap* data_map, CUtensorMap* scale_map, const void* data, const void* scales, int64_t rows,
                  int64_t k, int box_rows, int scale_tiles) {
  const cuuint64_t pitch = (cuuint64_t)mx_pitch(k);
  const cuuint64_t dsize[2] = {pitch, (cuuint64_t)rows}, dstride[1] = {pitch};
  const cuuint32_t dbox[2] = {128, (cuuint32_t)box_rows};
  const cuuint64_t kt = (cuuint64_t)mx_scale_cols(k), rt = (cuuint64_t)((rows + 127) / 128);
  const cuuint64_t ssize[3] = {128, kt, rt}, sstride[2] = {kMxScaleTile, kt * kMxScaleTile};
  const cuuint32_t sbox[3] = {128, 2, (cuuint32_t)scale_tiles};
  return encode(data_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(data), dsize, dstride, dbox,
                CU_TENSOR_MAP_SWIZZLE_128B) &&
         encode(scale_map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void*>(scales), ssize, sstride, sbox,
                CU_TENSOR_MAP_SWIZZLE_NONE);
}

}  // namespace

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
  a.k = k;
  a.d = d;
  a.ldd = ldd;
  a.alpha = alpha;
  a.beta = beta;
  a.dtype = dtype;
  a.vec = rows_aligned(d, ldd, dtype);
  a.err = h->d_op_err;
  a.timeout_ns = h->wait_timeout_ns;
  // CTA pairs once the 128 x 128 tiles of the one-CTA kernel would need a
  // second wave (an SM takes about 70 bytes a clock from L2 either way, and a
  // pair's tile asks half as many of it for a product): 1024 x 4096 x 4096
  // (256 tiles) 10.5 us against 15.0, 512 x 4096 x 4096 (128) 10.2 against 8.2.
  const int64_t small_tiles = ((m + 127) / 128) * ((n + 127) / 128);
  const int64_t pair_tiles = ((m + 255) / 256) * ((n + 255) / 256);
  const bool pairs = h->max_clusters > 0 && m > 128 && n > 128 && small_tiles > h->num_sms;
  a.swapped = !pairs && m <= 256;
  a.p_rows = a.swapped ? n : m;
  a.q_rows = a.swapped ? m : n;
  const void *pd = a.swapped ? b_data : a_data, *ps = a.swapped ? b_scales : a_scales;
  const void *qd = a.swapped ? a_data : b_data, *qs = a.swapped ? a_scales : b_scales;
  // A Q of at most 128 rows is one tile (a tile of fewer than 128 rows has
  // to start on a scale tile).
  const int nt = pairs ? 256 : a.q_rows <= 32 ? 32 : a.q_rows <= 64 ? 64 : 128;
  a.q_tiles = (int)((a.q_rows + nt - 1) / nt);
  const int64_t tiles = (a.p_rows + 127) / 128 * a.q_tiles;
  if (tiles > INT32_MAX / 8) return fail(h, DMUON_ERR_ARG, "mxfp4_gemm: too many tiles");
  if (!operand_maps(&a.p_data, &a.p_scales, pd, ps, a.p_rows, k, 128, 1) ||
      !operand_maps(&a.q_data, &a.q_scales, qd, qs, a.q_rows, k, pairs ? 128 : nt, (nt + 127) / 128))
    return fail(h, DMUON_ERR_CUDA, "mxfp4_gemm: tensor map");
  cudaError_t e;
  LaunchGuard g(h, stream, DMUON_KIND_MX_GEMM);
  if (pairs) {
    e = launch_mx_gemm_pair(a, (int)std::min<int64_t>(pair_tiles, h->max_clusters), stream);
  } else {
    // K split over a cluster while that fills idle SMs.  Joining costs 0.3 us at
    // NT = 32 and about 2 us at 128, a stage 0.25 us: 1 x 4096 x 4096 6.7 us
    // whole, 4.6 in four; 512 x 512 x 512 4.4 whole, 6.2 in two.  Eight ranks of
    // 210 KB each do not all find an SM at once (128 x 4096 x 4096: 22 us).
    const int64_t stages = (k + 255) / 256;
    const int most = nt == 128 ? 4 : 8;
    int split = 1;
    while (split < most && tiles * split * 2 <= h->num_sms && stages >= split * 2 && (nt == 32 || stages >= 8)) split *= 2;
    e = launch_mx_gemm(a, nt, split, stream);
  }
  if (e != cudaSuccess) return fail(h, cuda_err(e), "mxfp4_gemm launch", e);
  h->last_stream = stream;
  return DMUON_OK;
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
  if (h->op_ws_cap < need) {
    if (capturing(stream)) return fail(h, DMUON_ERR_ARG, "block_norm_backward: first call of this size under capture");
    if (h->op_ws && h->op_ws_captured) {
      h->op_ws_kept.push_back(h->op_ws);
    } else if (h->op_ws) {
      cudaDeviceSynchronize();  // earlier work may still use it
      cudaFree(h->op_ws);
    }
    h->op_ws = nullptr;
    h->op_ws_cap = 0;
    h->op_ws_captured = false;
    const cudaError_t e = cudaMalloc(&h->op_ws, need);
    if (e != cudaSuccess) {
      h->op_ws = nullptr;
      cudaGetLastError();
      return fail(h, DMUON_ERR_OOM, "block_norm_backward workspace", e);
    }
    h->op_ws_cap = need;
  }
  if (!h->op_ws_captured) h->op_ws_captured = capturing(stream);
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
