// out = dropout(x) + residual over a matrix (generator in dropout.cuh).
//
// A lane has one group of eight columns, whose bits one call of the generator
// gives, in four rows, all loaded before one is used; in one row where four would
// leave SMs without work (777 x 2061 fp32).  Short rows share a warp.
#include "../../include/dmuon.h"
#include "chunk8.cuh"
#include "dropout.cuh"

namespace dmuon {

namespace {

constexpr int kThreads = 256;

template <typename T, bool VEC, int kRows>  // rows a lane has
__global__ void __launch_bounds__(kThreads) dropout_kernel(const DropoutArgs a, int lanes) {  // lanes of a row: a power of two
  const int64_t ct = (a.cols + 255) / 256;
  const int at_once = kThreads / lanes, lane = threadIdx.x & (lanes - 1);
  const int64_t row0 = (int64_t)(blockIdx.x / ct) * kRows * at_once + threadIdx.x / lanes;
  const int64_t col = (int64_t)(blockIdx.x % ct) * 256 + lane * 8;
  const int64_t left = a.cols - col;  // below 1: a lane past the row
  const int n = (int)max((int64_t)0, min((int64_t)8, left));
  Raw8<T, VEC> x[kRows], res[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t r = row0 + at_once * i;
    const int here = r < a.rows ? n : 0;
    load_raw8<T, VEC>(x[i], (const T*)a.x + r * a.ldx + col, here);
    if (a.res) load_raw8<T, VEC>(res[i], (const T*)a.res + r * a.ldres + col, here);
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t r = row0 + at_once * i;
    float f[8];
    values8<T, VEC>(f, x[i], (const T*)a.x + r * a.ldx + col, n);
    if (a.drop.cut) {
      uint32_t w[4];
      philox(w, a.drop, (uint32_t)(col >> 3), (uint32_t)r);
      drop8(f, a.drop, w);
    }
    if (a.res) {
      float g[8];
      values8<T, VEC>(g, res[i], (const T*)a.res + r * a.ldres + col, n);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] += g[e];
    }
    T* out = (T*)a.out + r * a.ldout + col;
    if (lanes == 32) store8_warp<T, VEC, true>(out, f, left, lane == 0, lane == lanes - 1, r < a.rows);
    else store8_warp<T, VEC>(out, f, left, lane == 0, lane == lanes - 1, r < a.rows);
  }
}

template <typename T, int kRows>
cudaError_t launch_rows(const DropoutArgs& a, int lanes, cudaStream_t s) {
  const int64_t per = kRows * (kThreads / lanes);
  const int64_t ctas = (a.rows + per - 1) / per * ((a.cols + 255) / 256);
  if (a.vec) dropout_kernel<T, true, kRows><<<(unsigned)ctas, kThreads, 0, s>>>(a, lanes);
  else dropout_kernel<T, false, kRows><<<(unsigned)ctas, kThreads, 0, s>>>(a, lanes);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch(const DropoutArgs& a, int sms, cudaStream_t s) {
  int lanes = 1;
  while (lanes < 32 && lanes * 8 < a.cols) lanes *= 2;
  const int64_t per = 4 * (kThreads / lanes);
  const bool few = (a.rows + per - 1) / per * ((a.cols + 255) / 256) < 4 * sms;
  return few ? launch_rows<T, 1>(a, lanes, s) : launch_rows<T, 4>(a, lanes, s);
}

}  // namespace

cudaError_t launch_dropout(const DropoutArgs& a, int dtype, int sms, cudaStream_t s) {
  if (dtype == DMUON_BF16) return launch<__nv_bfloat16>(a, sms, s);
  if (dtype == DMUON_F16) return launch<__half>(a, sms, s);
  return launch<float>(a, sms, s);
}

}  // namespace dmuon
