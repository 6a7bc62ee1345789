// Norms after and before a block with the block's gate and residual scale,
// forward and backward (formulas in block_norm.cuh).  Everything is computed
// in fp32; y, h, dx and df are rounded once to the activations' type, and the
// second norm takes y before it is rounded.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/dmuon.h"
#include "block_norm.cuh"

namespace dmuon {

namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ float widen(T v);
template <>
__device__ __forceinline__ float widen<float>(float v) { return v; }
template <>
__device__ __forceinline__ float widen<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float widen<__half>(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ float narrow<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half narrow<__half>(float v) { return __float2half_rn(v); }

// Sums of N values over the block, in a fixed order, to every thread.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* red) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll
  for (int k = 0; k < N; ++k)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < N; ++k) red[warp * N + k] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    float s = 0.f;
    for (int w = 0; w < warps; ++w) s += red[w * N + k];
    v[k] = s;
  }
  __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kThreads) norm_fwd_kernel(const NormFwdArgs a) {
  __shared__ float red[kThreads / 32];
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = (const T*)a.x + row * a.ldx;
    const T* f = (const T*)a.f + row * a.ldf;
    T* y = (T*)a.y + row * a.ldy;
    T* h = (T*)a.h + row * a.ldh;
    const float* gate = a.gate ? a.gate + row / a.per_gate * a.cols : nullptr;
    float s[1] = {0.f};
    for (int64_t c = threadIdx.x; c < a.cols; c += kThreads) {
      const float v = widen(f[c]);
      s[0] = fmaf(v, v, s[0]);
    }
    block_sum<1>(s, red);
    const float r1 = 1.f / sqrtf(s[0] / (float)a.cols + a.eps);
    auto value = [&](int64_t c) {
      float n = widen(f[c]) * r1 * a.post_w[c];
      if (gate) n *= gate[c];
      const float v = widen(x[c]);
      return a.res ? fmaf(v, a.res[c], n) : v + n;
    };
    s[0] = 0.f;
    for (int64_t c = threadIdx.x; c < a.cols; c += kThreads) {
      const float v = value(c);
      s[0] = fmaf(v, v, s[0]);
    }
    block_sum<1>(s, red);
    const float r2 = 1.f / sqrtf(s[0] / (float)a.cols + a.eps);
    for (int64_t c = threadIdx.x; c < a.cols; c += kThreads) {
      const float v = value(c);
      y[c] = narrow<T>(v);
      h[c] = narrow<T>(v * r2 * a.pre_w[c]);
    }
    if (threadIdx.x == 0) {
      a.rstd[row] = r1;
      a.rstd[a.rows + row] = r2;
    }
  }
}

// Column sums: each thread owns the columns c = threadIdx.x mod kThreads of
// its CTA's rows of the partial arrays.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_bwd_kernel(const NormBwdArgs a) {
  __shared__ float red[3 * kThreads / 32];
  const int64_t n_chunks = a.groups * a.chunks_per_group;
  float* pre = a.part_pre + (int64_t)blockIdx.x * a.cols;
  float* post = a.part_post + (int64_t)blockIdx.x * a.cols;
  float* res = a.d_res ? a.part_res + (int64_t)blockIdx.x * a.cols : nullptr;
  for (int64_t c = threadIdx.x; c < a.cols; c += kThreads) {
    pre[c] = post[c] = 0.f;
    if (res) res[c] = 0.f;
  }
  const float inv = 1.f / (float)a.cols;
  for (int64_t chunk = blockIdx.x; chunk < n_chunks; chunk += gridDim.x) {
    const int64_t group = chunk / a.chunks_per_group, part = chunk % a.chunks_per_group;
    const int64_t r0 = group * a.per_gate + part * a.chunk_rows;
    const int64_t r1_ = min(min(r0 + a.chunk_rows, (group + 1) * a.per_gate), a.rows);
    const float* gate = a.gate ? a.gate + group * a.cols : nullptr;
    // Column sums of t fn over the chunk: where they are wanted for the gate
    // they go to the chunk's own row, else straight to the CTA's sum.
    float* own = a.d_gate ? (a.chunks_per_group > 1 ? a.part_gate + chunk * a.cols : a.d_gate + group * a.cols) : nullptr;
    if (own)
      for (int64_t c = threadIdx.x; c < a.cols; c += kThreads) own[c] = 0.f;
    for (int64_t row = r0; row < r1_; ++row) {
      const T* dy = a.dy ? (const T*)a.dy + row * a.lddy : nullptr;
      const T* dh = (const T*)a.dh + row * a.lddh;
      const T* f = (const T*)a.f + row * a.ldf;
      const T* y = (const T*)a.y + row * a.ldy;
      const float r1 = a.rstd[row], r2 = a.rstd[a.rows + row];
      auto t_of = [&](int64_t c, float mean) {
        const float u = (dy ? widen(dy[c]) : 0.f);
        return u + r2 * (widen(dh[c]) * a.pre_w[c] - widen(y[c]) * r2 * mean);
      };
      float s[1] = {0.f};
      for (int64_t c = threadIdx.x; c < a.cols; c += kThreads) s[0] += widen(dh[c]) * a.pre_w[c] * (widen(y[c]) * r2);
      block_sum<1>(s, red);
      const float m2 = s[0] * inv;
      s[0] = 0.f;
      for (int64_t c = threadIdx.x; c < a.cols; c += kThreads) {
        const float t = t_of(c, m2);
        s[0] += (gate ? gate[c] * t : t) * a.post_w[c] * (widen(f[c]) * r1);
      }
      block_sum<1>(s, red);
      const float m1 = s[0] * inv;
      for (int64_t c = threadIdx.x; c < a.cols; c += kThreads) {
        const float t = t_of(c, m2), fn = widen(f[c]) * r1;
        const float dn = gate ? gate[c] * t : t;
        pre[c] += widen(dh[c]) * (widen(y[c]) * r2);
        if (own) own[c] += t * fn;
        else post[c] += dn * fn;
        if (res) res[c] += t * widen(((const T*)a.x + row * a.ldx)[c]);
        ((T*)a.dx + row * a.lddx)[c] = narrow<T>(a.res ? a.res[c] * t : t);
        ((T*)a.df + row * a.lddf)[c] = narrow<T>(r1 * (dn * a.post_w[c] - fn * m1));
      }
    }
    if (own)
      for (int64_t c = threadIdx.x; c < a.cols; c += kThreads) {
        post[c] += (gate ? gate[c] : 1.f) * own[c];
        if (a.chunks_per_group == 1) own[c] *= a.post_w[c];
      }
  }
}

// Column sums over the CTAs' partial rows (blockIdx.y: 0 pre, 1 post, 2 res)
// and, from 3 on, over the chunks of gate group blockIdx.y - 3; 32 columns a
// block, eight warps over the rows in turn, then the warps in order.
__global__ void __launch_bounds__(256) norm_bwd_sums_kernel(const NormBwdArgs a) {
  __shared__ float red[8][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  const float* src;
  float* dst;
  int64_t n = a.ctas;
  if (blockIdx.y == 0) { src = a.part_pre; dst = a.d_pre_w; }
  else if (blockIdx.y == 1) { src = a.part_post; dst = a.d_post_w; }
  else if (blockIdx.y == 2) { src = a.part_res; dst = a.d_res; }
  else {
    const int64_t g = blockIdx.y - 3;
    n = a.chunks_per_group;
    src = a.part_gate + g * n * a.cols;
    dst = a.d_gate + g * a.cols;
  }
  if (!dst) return;
  float s = 0.f;
  if (c < a.cols)
    for (int64_t i = warp; i < n; i += 8) s += src[i * a.cols + c];
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < a.cols) {
    for (int w = 1; w < 8; ++w) s += red[w][lane];
    dst[c] = blockIdx.y >= 3 ? s * a.post_w[c] : s;
  }
}

template <typename T>
cudaError_t fwd(const NormFwdArgs& a, int sms, cudaStream_t s) {
  const int64_t grid = a.rows < (int64_t)sms * 8 ? a.rows : (int64_t)sms * 8;
  norm_fwd_kernel<T><<<(unsigned)grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t bwd(const NormBwdArgs& a, cudaStream_t s) {
  norm_bwd_kernel<T><<<a.ctas, kThreads, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const unsigned ys = 3 + (a.d_gate && a.chunks_per_group > 1 ? (unsigned)a.groups : 0u);
  norm_bwd_sums_kernel<<<dim3((unsigned)((a.cols + 31) / 32), ys), 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

int norm_bwd_ctas(int64_t cols, int sms) { return sms * 4; }

cudaError_t launch_norm_fwd(const NormFwdArgs& a, int dtype, int sms, cudaStream_t s) {
  if (dtype == DMUON_BF16) return fwd<__nv_bfloat16>(a, sms, s);
  if (dtype == DMUON_F16) return fwd<__half>(a, sms, s);
  return fwd<float>(a, sms, s);
}

cudaError_t launch_norm_bwd(const NormBwdArgs& a, int dtype, cudaStream_t s) {
  if (dtype == DMUON_BF16) return bwd<__nv_bfloat16>(a, s);
  if (dtype == DMUON_F16) return bwd<__half>(a, s);
  return bwd<float>(a, s);
}

}  // namespace dmuon
