// What the operators' entry points share (include/dmuon.h): argument checks,
// tensor maps of block-scaled operands, tile choice of their products, workspace.
#pragma once

#include <algorithm>
#include <cmath>

#include "ctx.cuh"
#include "mx.cuh"

namespace dmuon {

constexpr int64_t kMaxSide = int64_t(1) << 30;

inline int elem_size(int dtype) {
  switch (dtype) {
    case DMUON_F32: return 4;
    case DMUON_BF16: case DMUON_F16: return 2;
    default: return 0;
  }
}

inline bool aligned(const void* p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }

// Every row starts on 16 bytes.
inline bool rows_aligned(const void* p, int64_t ld, int dtype) { return aligned(p, 16) && (ld * elem_size(dtype)) % 16 == 0; }

// A rows x cols matrix of `dtype` at p with leading dimension ld: DMUON_OK or
// the error code (also recorded).
inline int check_matrix(dmuon_ctx* h, const void* p, int dtype, int64_t cols, int64_t ld, const char* what) {
  if (!p || ld < cols) return fail(h, DMUON_ERR_ARG, what);
  if (!aligned(p, elem_size(dtype))) return fail(h, DMUON_ERR_ALIGN, what);
  return DMUON_OK;
}

inline int check_packed(dmuon_ctx* h, const void* data, const void* scales, const char* what) {
  if (!data || !scales || data == scales) return fail(h, DMUON_ERR_ARG, what);
  if (!aligned(data, 16) || !aligned(scales, 16)) return fail(h, DMUON_ERR_ALIGN, what);
  return DMUON_OK;
}

// The kernels' limits of shared memory, set by a handle's first call (loading
// the norms' kernels takes 15 ms, which a handle without norms does not pay).
inline int ready(dmuon_ctx* h, bool& done, cudaError_t (*configure)(), const char* what) {
  if (done) return DMUON_OK;
  const cudaError_t e = configure();
  if (e != cudaSuccess) return fail(h, cuda_err(e), what, e);
  done = true;
  return DMUON_OK;
}

inline bool encode(CUtensorMap* map, CUtensorMapDataType type, int dims, void* base, const cuuint64_t* size,
            const cuuint64_t* stride, const cuuint32_t* box, CUtensorMapSwizzle swizzle) {
  const cuuint32_t one[3] = {1, 1, 1};
  return tensor_map_encoder()(map, type, dims, base, size, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Maps of one operand of `bits` an element: boxes of box_rows x 128 bytes of
// codes (256 or 128 elements of K) and of their scale tiles (two or one) for
// each of `scale_tiles` x 128 rows.
inline bool operand_maps(CUtensorMap* data_map, CUtensorMap* scale_map, const void* data, const void* scales, int64_t rows,
                  int64_t k, int bits, int box_rows, int scale_tiles) {
  const cuuint64_t pitch = (cuuint64_t)mx_pitch(k, bits);
  const cuuint64_t dsize[2] = {pitch, (cuuint64_t)rows}, dstride[1] = {pitch};
  const cuuint32_t dbox[2] = {128, (cuuint32_t)box_rows};
  const cuuint64_t kt = (cuuint64_t)mx_scale_cols(k), rt = (cuuint64_t)((rows + 127) / 128);
  const cuuint64_t ssize[3] = {128, kt, rt}, sstride[2] = {kMxScaleTile, kt * kMxScaleTile};
  const cuuint32_t sbox[3] = {128, (cuuint32_t)(8 / bits), (cuuint32_t)scale_tiles};
  return encode(data_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(data), dsize, dstride, dbox,
                CU_TENSOR_MAP_SWIZZLE_128B) &&
         encode(scale_map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void*>(scales), ssize, sstride, sbox,
                CU_TENSOR_MAP_SWIZZLE_NONE);
}


// One product's launchers.
template <typename Args>
struct Product {
  int bits;
  cudaError_t (*tiles)(const Args&, int nt, int split, cudaStream_t);
  cudaError_t (*pairs)(const Args&, int pairs, cudaStream_t);
};

// Tile choice, tensor maps and launch of D (m x n) = A B^T and so on: `a` holds
// all but P and Q.  Device and arguments are checked.
template <typename Args>
int launch_product(dmuon_ctx* h, Args& a, const Product<Args>& product, const void* a_data, const void* a_scales, const void* b_data,
                   const void* b_scales, int64_t m, int64_t n, int64_t k, cudaStream_t stream, const char* what) {
  a.k = k;
  a.err = h->d_op_err;
  a.timeout_ns = h->wait_timeout_ns;
  // CTA pairs once the 128 x 128 tiles of the one-CTA kernel would need a
  // second wave (an SM takes about 70 bytes a clock from L2 either way, and a
  // pair's tile asks half as many of it for a product): 1024 x 4096 x 4096
  // (256 tiles) 10.5 us against 15.0, 512 x 4096 x 4096 (128) 10.2 against 8.2.
  // The border is the same at 8 bits and with bias, GELU and two bf16 outputs (us,
  // operands from HBM, one-CTA tiles against pairs): 512 x 4096 x 4096 16.3 against 18.5,
  // K = 320 7.5 against 9.7; 608 x 4096 x 4096 (160 tiles) 26.8 against 18.9, K = 320
  // 12.3 against 9.7; at 4 bits 11.9 against 14.1 and 19.7 against 14.2.
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
  if (tiles > INT32_MAX / 8) return fail(h, DMUON_ERR_ARG, what);
  if (!operand_maps(&a.p_data, &a.p_scales, pd, ps, a.p_rows, k, product.bits, 128, 1) ||
      !operand_maps(&a.q_data, &a.q_scales, qd, qs, a.q_rows, k, product.bits, pairs ? 128 : nt, (nt + 127) / 128))
    return fail(h, DMUON_ERR_CUDA, what);
  cudaError_t e;
  LaunchGuard g(h, stream, DMUON_KIND_MX_GEMM);
  if (pairs) {
    e = product.pairs(a, (int)std::min<int64_t>(pair_tiles, h->max_clusters), stream);
  } else {
    // K split over a cluster while that fills idle SMs.  Joining costs 0.3 us at
    // NT = 32 and about 2 us at 128, a stage 0.25 us: 1 x 4096 x 4096 6.7 us
    // whole, 4.6 in four; 512 x 512 x 512 4.4 whole, 6.2 in two.  Eight ranks of
    // 210 KB each do not all find an SM at once (128 x 4096 x 4096: 22 us).
    // At 8 bits, with bias and a residual, operands from HBM: 1 x 4096 x 14336 25.3
    // whole, 16.0 in two, 13.8 in four; 64 x 4096 x 4096 14.1, 15.2 and 11.4;
    // 512 x 2048 x 14336 39.2, 31.7 and 37.9.  A residual at 129 to 256 rows, read a
    // column a lane where shares meet, is what the rule does not see: 256 x 4096 x 4096
    // 23.5 in two (as chosen), 20.5 whole, 18.1 on pairs; without one 14.3, 16.9, 16.4.
    const int64_t stages = (k * product.bits + 1023) / 1024;
    const int most = nt == 128 ? 4 : 8;
    int split = 1;
    while (split < most && tiles * split * 2 <= h->num_sms && stages >= split * 2 && (nt == 32 || stages >= 8)) split *= 2;
    e = product.tiles(a, nt, split, stream);
  }
  if (e != cudaSuccess) return fail(h, cuda_err(e), what, e);
  h->last_stream = stream;
  return DMUON_OK;
}

// The handle's workspace for `need` bytes of this call.  Growing it waits for
// earlier work; what a captured graph holds is kept until the handle goes.
inline int op_workspace(dmuon_ctx* h, size_t need, cudaStream_t stream, const char* what) {
  if (h->op_ws_cap < need) {
    if (capturing(stream)) return fail(h, DMUON_ERR_ARG, what);
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
      return fail(h, DMUON_ERR_OOM, what, e);
    }
    h->op_ws_cap = need;
  }
  if (!h->op_ws_captured) h->op_ws_captured = capturing(stream);
  return DMUON_OK;
}

}  // namespace dmuon
