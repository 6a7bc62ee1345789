// out = dropout(x) + residual over a matrix (generator in dropout.cuh).
//
// A lane has 32 bytes of a row, one or two groups of eight columns, and two rows, all
// loaded before one is used; one row where two would leave SMs without work
// (777 x 2061 fp32).  Short rows share a warp.  Bound by HBM: 16384 x 14336 bf16
// with a residual 213 us (6.6 TB/s).
#include "../../include/dmuon.h"
#include "chunk8.cuh"
#include "dropout.cuh"

namespace dmuon {

namespace {

constexpr int kThreads = 256;

template <typename T>
constexpr int lane_cols() { return 32 / (int)sizeof(T); }

template <typename T, bool VEC, int ROWS>  // rows a lane has
__global__ void __launch_bounds__(kThreads) dropout_kernel(const DropoutArgs a, int lanes) {  // lanes of a row: a power of two
  constexpr int E = lane_cols<T>(), S = (int)sizeof(T);
  const int64_t ct = (a.cols + 32 * E - 1) / (32 * E);
  const int at_once = kThreads / lanes, lane = threadIdx.x & (lanes - 1);
  const int64_t row0 = (int64_t)(blockIdx.x / ct) * ROWS * at_once + threadIdx.x / lanes;
  const int64_t col = (int64_t)(blockIdx.x % ct) * (32 * E) + lane * E;
  const int left = (int)min((int64_t)64, (a.cols - col) * S);  // bytes, below 1: a lane past the row
  const uint8_t* x = (const uint8_t*)a.x + (row0 * a.ldx + col) * S;
  const uint8_t* res = (const uint8_t*)a.res + (row0 * a.ldres + col) * S;
  Raw32<VEC> xr[ROWS], rr[ROWS];
  auto load = [&](auto end) {
    constexpr bool kEnd = decltype(end)::value;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int here = row0 + at_once * i < a.rows ? left : 0;
      load_raw32<S, VEC, kEnd>(xr[i], x + i * at_once * a.ldx * S, here);
      if (a.res) load_raw32<S, VEC, kEnd>(rr[i], res + i * at_once * a.ldres * S, here);
    }
  };
  // Sixteen rows of the matrix, 16 bytes at least, follow all of a CTA's but in the last CTAs.
  if ((int64_t)(blockIdx.x / ct + 1) * ROWS * at_once + 16 <= a.rows) load(std::false_type());
  else load(std::true_type());
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int64_t r = row0 + at_once * i;
    f2 f[E / 2];
    values32<T, VEC>(f, xr[i], x + i * at_once * a.ldx * S);
    if (a.drop.cut) {
#pragma unroll
      for (int g = 0; g < E / 8; ++g) {
        uint32_t w[4];
        philox(w, a.drop, (uint32_t)(col >> 3) + g, (uint32_t)r);
        drop8(*reinterpret_cast<f2(*)[4]>(f + 4 * g), a.drop, w);
      }
    }
    if (a.res) {
      f2 more[E / 2];
      values32<T, VEC>(more, rr[i], res + i * at_once * a.ldres * S);
#pragma unroll
      for (int e = 0; e < E / 2; ++e) f[e] = add2(f[e], more[e]);
    }
    uint32_t w[16];
#pragma unroll
    for (int g = 0; g < E / 8; ++g) {
      float o[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 p = unpack2(f[4 * g + e]);
        o[2 * e] = p.x;
        o[2 * e + 1] = p.y;
      }
      pack8<T>(w + 4 + g * words8<T>(), o);
    }
    store32<S, VEC>((uint8_t*)a.out + (r * a.ldout + col) * S, w, left, lane, lanes, r < a.rows);
  }
}

template <typename T, int ROWS>
cudaError_t launch_rows(const DropoutArgs& a, int lanes, int64_t ct, cudaStream_t s) {
  const int64_t per = ROWS * (kThreads / lanes), ctas = (a.rows + per - 1) / per * ct;
  if (a.vec) dropout_kernel<T, true, ROWS><<<(unsigned)ctas, kThreads, 0, s>>>(a, lanes);
  else dropout_kernel<T, false, ROWS><<<(unsigned)ctas, kThreads, 0, s>>>(a, lanes);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch(const DropoutArgs& a, int sms, cudaStream_t s) {
  constexpr int E = lane_cols<T>();
  int lanes = 1;
  while (lanes < 32 && lanes * E < a.cols) lanes *= 2;
  const int64_t per = 2 * (kThreads / lanes), ct = (a.cols + 32 * E - 1) / (32 * E);
  const bool few = (a.rows + per - 1) / per * ct < 4 * sms;
  return few ? launch_rows<T, 1>(a, lanes, ct, s) : launch_rows<T, 2>(a, lanes, ct, s);
}

}  // namespace

cudaError_t launch_dropout(const DropoutArgs& a, int dtype, int sms, cudaStream_t s) {
  if (dtype == DMUON_BF16) return launch<__nv_bfloat16>(a, sms, s);
  if (dtype == DMUON_F16) return launch<__half>(a, sms, s);
  return launch<float>(a, sms, s);
}

}  // namespace dmuon
