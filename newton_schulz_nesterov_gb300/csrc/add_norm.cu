// Residual norm with dropout on the branch (formulas in add_norm.cuh).
// Everything is computed in fp32; y, h, dx and df are rounded once to the
// activations' type, and h and its MXFP8 codes come from y before it is rounded.
//
// A row is held by a unit of threads, V chunks of eight columns a thread, so that
// it is read once: part of a warp up to 256 columns, a warp up to 512, a CTA up
// to 16384.  A unit goes from row to row with its columns' weights (and, backward,
// their sums) in registers, and loads the next row ahead of the present one's
// sums.  Longer rows are read in two passes by one CTA (add_norm_long_*).
// A block of 32 columns is four lanes, so its scale byte takes two exchanges.
#include <algorithm>

#include "../../include/dmuon.h"
#include "add_norm.cuh"
#include "chunk8.cuh"
#include "mx.cuh"
#include "mx8.cuh"

namespace dmuon {

namespace {

constexpr int kLongThreads = 512;
constexpr int kMostFwd = 16384, kMostBwd = 8192;  // columns that a unit holds

// Where a unit's threads stand.  MULTI: the CTA is one unit; else units of tpr <=
// 32 lanes share warps.
struct Unit {
  int tpr, unit, units, t, lane, warp;
  bool first, last;  // of the runs of a warp's stores
  __device__ __forceinline__ Unit(int tpr_, bool multi) {
    tpr = tpr_;
    lane = threadIdx.x & 31;
    warp = threadIdx.x >> 5;
    unit = multi ? 0 : threadIdx.x / tpr;
    units = multi ? 1 : blockDim.x / tpr;
    t = multi ? threadIdx.x : threadIdx.x & (tpr - 1);
    first = lane == 0 || t == 0;
    last = lane == 31 || t == tpr - 1;
  }
};

// Sum over a unit, in a fixed order, to all of it.  Consecutive calls of a CTA
// alternate between the halves of `red`: one is written again only after the
// next call's barrier, when every thread has read it.
template <bool MULTI>
__device__ __forceinline__ float unit_sum(float v, const Unit& u, float (*red)[16], uint32_t& calls) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (MULTI || o < u.tpr) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (!MULTI) return v;
  float* mine = red[calls++ & 1];
  if (u.lane == 0) mine[u.warp] = v;
  __syncthreads();
  const int n = blockDim.x >> 5;
  v = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < n) v += mine[i];
  return v;
}

// Scale bytes past the matrix are zero: rows from `rows` to the tile's end, by
// all threads of the grid; blocks past a row's last, with the row.
__device__ __forceinline__ void zero_rows_behind(uint8_t* scales, int64_t rows, int64_t cols) {
  const int64_t kt = mx_scale_cols(cols), all = (128 - (rows & 127)) % 128 * kt;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < all; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t r = rows + i / kt;
    *reinterpret_cast<uint32_t*>(scales + ((r >> 7) * kt + i % kt) * kMxScaleTile + (r & 31) * 16 + ((r >> 5) & 3) * 4) = 0u;
  }
}
__device__ __forceinline__ uint8_t* scale_at(uint8_t* scales, int64_t row, int64_t blk, int64_t cols) {
  return scales + ((row >> 7) * mx_scale_cols(cols) + (blk >> 2)) * kMxScaleTile + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (blk & 3);
}

// Eight values of columns col .. of a row to codes; a warp's lanes together, four
// consecutive ones a block.
__device__ __forceinline__ void quantise8(const AddNormFwdArgs& a, const float (&h)[8], int64_t row, int64_t col, bool live) {
  const float m = mx8::max_abs(h);
  uint32_t key = mx8::keys2(m, m, a.up);
  key = mx8::max_halves(key, __shfl_xor_sync(0xffffffffu, key, 1));
  key = mx8::max_halves(key, __shfl_xor_sync(0xffffffffu, key, 2));
  uint32_t bad = 0;  // the block holds Inf or NaN
  if (__any_sync(0xffffffffu, mx8::may_not_be_finite(key))) {
    bad = mx8::not_finite(m);
    bad |= __shfl_xor_sync(0xffffffffu, bad, 1);
    bad |= __shfl_xor_sync(0xffffffffu, bad, 2);
  }
  if (!live || col >= mx_blocks(a.cols) * kMxBlock) return;
  const uint32_t ex = mx8::exponents2(key);
  const float inv = mx8::factors2(ex).y;
  uint2 w = make_uint2(mx8::codes4(h[0] * inv, h[1] * inv, h[2] * inv, h[3] * inv), mx8::codes4(h[4] * inv, h[5] * inv, h[6] * inv, h[7] * inv));
  if (bad) w = make_uint2(0, 0);
  *reinterpret_cast<uint2*>(a.q + row * mx_pitch(a.cols, 8) + col) = w;
  if ((col & 31) == 0) *scale_at(a.q_scales, row, col >> 5, a.cols) = bad ? 255 : (uint8_t)mx8::byte_of(ex, 1);
}
__device__ __forceinline__ void zero_blocks_behind(const AddNormFwdArgs& a, int64_t row, int t, bool live) {
  const int64_t nb = mx_blocks(a.cols);
  if (live && t < mx_scale_cols(a.cols) * 4 - nb) *scale_at(a.q_scales, row, nb + t, a.cols) = 0;
}

template <typename T, bool VEC, int V, bool MULTI>
__global__ void __launch_bounds__(MULTI ? 512 : 256) add_norm_fwd_kernel(const AddNormFwdArgs a, int tpr) {
  __shared__ float red[2][16];
  const Unit u(tpr, MULTI);
  uint32_t calls = 0;
  const int64_t step = (int64_t)gridDim.x * u.units;
  int64_t row = (int64_t)blockIdx.x * u.units + u.unit;
  int n[V];
  float w[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * tpr + u.t) * 8;
    n[v] = (int)a.cols - c;
    load8<float, VEC>(w[v], a.w + c, n[v]);
  }
  if (a.q) zero_rows_behind(a.q_scales, a.rows, a.cols);
  Raw8<T, VEC> xr[V], fr[V];
  auto at = [&](const void* base, int64_t r, int64_t ld, int v) { return (const T*)base + r * ld + (v * tpr + u.t) * 8; };
  auto fetch = [&](int64_t r) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int k = r < a.rows ? n[v] : 0;
      load_raw8<T, VEC>(fr[v], at(a.f, r, a.ldf, v), k);
      if (a.x) load_raw8<T, VEC>(xr[v], at(a.x, r, a.ldx, v), k);
    }
  };
  fetch(row);
  const float inv = 1.f / (float)a.cols;
  for (int64_t base = (int64_t)blockIdx.x * u.units; base < a.rows; base += step, row += step) {  // as often for every unit
    const bool live = MULTI || row < a.rows;
    float y[V][8];
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      values8<T, VEC>(y[v], fr[v], at(a.f, row, a.ldf, v), n[v]);
      if (a.drop.cut) {
        uint32_t bits[4];
        philox(bits, a.drop, (uint32_t)(v * tpr + u.t), (uint32_t)row);
        drop8(y[v], a.drop, bits);
      }
      if (a.x) {
        float x[8];
        values8<T, VEC>(x, xr[v], at(a.x, row, a.ldx, v), n[v]);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[v][e] += x[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) s = fmaf(y[v][e], y[v][e], s);
    }
    fetch(row + step);
#pragma unroll
    for (int v = 0; v < V; ++v) store8_warp<T, VEC>((T*)a.y + row * a.ldy + (v * tpr + u.t) * 8, y[v], n[v], u.first, u.last, live);
    s = unit_sum<MULTI>(s, u, red, calls);
    const float r = rsqrtf(fmaf(s, inv, a.eps));
    if (live && u.t == 0) a.rstd[row] = r;
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[v][e] = y[v][e] * r * w[v][e];
      if (a.h) store8_warp<T, VEC>((T*)a.h + row * a.ldh + (v * tpr + u.t) * 8, y[v], n[v], u.first, u.last, live);
      if (a.q) quantise8(a, y[v], row, (v * tpr + u.t) * 8, live);
    }
    if (a.q) zero_blocks_behind(a, row, u.t, live);
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kLongThreads) add_norm_long_fwd_kernel(const AddNormFwdArgs a) {
  __shared__ float red[2][16];
  const Unit u(kLongThreads, true);
  uint32_t calls = 0;
  if (a.q) zero_rows_behind(a.q_scales, a.rows, a.cols);
  const int64_t panels = (a.cols + kLongThreads * 8 - 1) / (kLongThreads * 8);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    auto sum_at = [&](float (&y)[8], int64_t c) {
      const int n = (int)max((int64_t)0, min((int64_t)8, a.cols - c));
      load8<T, VEC>(y, (const T*)a.f + row * a.ldf + c, n);
      if (a.drop.cut) {
        uint32_t bits[4];
        philox(bits, a.drop, (uint32_t)(c >> 3), (uint32_t)row);
        drop8(y, a.drop, bits);
      }
      if (a.x) {
        float x[8];
        load8<T, VEC>(x, (const T*)a.x + row * a.ldx + c, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] += x[e];
      }
    };
    float s = 0.f, y[8];
#pragma unroll 2
    for (int64_t p = 0; p < panels; ++p) {
      const int64_t c = (p * kLongThreads + threadIdx.x) * 8;
      sum_at(y, c);
#pragma unroll
      for (int e = 0; e < 8; ++e) s = fmaf(y[e], y[e], s);
      store8_warp<T, VEC>((T*)a.y + row * a.ldy + c, y, a.cols - c, u.first, u.last, true);
    }
    s = unit_sum<true>(s, u, red, calls);
    const float r = rsqrtf(fmaf(s, 1.f / (float)a.cols, a.eps));
    if (threadIdx.x == 0) a.rstd[row] = r;
#pragma unroll 2
    for (int64_t p = 0; p < panels; ++p) {
      const int64_t c = (p * kLongThreads + threadIdx.x) * 8;
      float w[8];
      sum_at(y, c);
      load8<float, VEC>(w, a.w + c, (int)max((int64_t)0, min((int64_t)8, a.cols - c)));
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = y[e] * r * w[e];
      if (a.h) store8_warp<T, VEC>((T*)a.h + row * a.ldh + c, y, a.cols - c, u.first, u.last, true);
      if (a.q) quantise8(a, y, row, c, true);
    }
    if (a.q) zero_blocks_behind(a, row, u.t, true);
  }
}

// t and a row's share of the column sums, from the row's sum of dh w y.
__device__ __forceinline__ void into_t(float (&t)[8], float (&sums)[8], const float (&dy)[8], const float (&dh)[8], const float (&y)[8],
                                       const float (&w)[8], float r, float back) {  // back: r^3 mean(dh w y)
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float dhr = dh[e] * r;
    sums[e] = fmaf(dhr, y[e], sums[e]);
    t[e] = fmaf(dhr, w[e], dy[e]) - back * y[e];
  }
}

template <typename T, bool VEC, int V, bool MULTI>
__global__ void __launch_bounds__(MULTI ? 512 : 256) add_norm_bwd_kernel(const AddNormBwdArgs a, int tpr) {
  __shared__ float red[2][16];
  __shared__ float lines[MULTI ? 1 : 32 * V * 8];
  const Unit u(tpr, MULTI);
  uint32_t calls = 0;
  const int64_t step = (int64_t)gridDim.x * u.units;
  int64_t row = (int64_t)blockIdx.x * u.units + u.unit;
  int n[V];
  float w[V][8], sums[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * tpr + u.t) * 8;
    n[v] = (int)a.cols - c;
    load8<float, VEC>(w[v], a.w + c, n[v]);
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[v][e] = 0.f;
  }
  Raw8<T, VEC> dyr[V], dhr[V], yr[V];
  auto at = [&](const void* base, int64_t r, int64_t ld, int v) { return (const T*)base + r * ld + (v * tpr + u.t) * 8; };
  float next_r = 0.f;
  auto fetch = [&](int64_t r) {
    const bool live = r < a.rows;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int k = live ? n[v] : 0;
      load_raw8<T, VEC>(dhr[v], at(a.dh, r, a.lddh, v), k);
      load_raw8<T, VEC>(yr[v], at(a.y, r, a.ldy, v), k);
      if (a.dy) load_raw8<T, VEC>(dyr[v], at(a.dy, r, a.lddy, v), k);
    }
    next_r = live ? a.rstd[r] : 0.f;
  };
  fetch(row);
  const float inv = 1.f / (float)a.cols;
  for (int64_t base = (int64_t)blockIdx.x * u.units; base < a.rows; base += step, row += step) {
    const bool live = MULTI || row < a.rows;
    const float r = next_r;
    float dy[V][8], dh[V][8], y[V][8];
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      values8<T, VEC>(dh[v], dhr[v], at(a.dh, row, a.lddh, v), n[v]);
      values8<T, VEC>(y[v], yr[v], at(a.y, row, a.ldy, v), n[v]);
      if (a.dy) values8<T, VEC>(dy[v], dyr[v], at(a.dy, row, a.lddy, v), n[v]);
      else
#pragma unroll
        for (int e = 0; e < 8; ++e) dy[v][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) s = fmaf(dh[v][e] * w[v][e], y[v][e], s);
    }
    fetch(row + step);
    s = unit_sum<MULTI>(s, u, red, calls);
    const float back = r * r * r * (s * inv);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float t[8];
      into_t(t, sums[v], dy[v], dh[v], y[v], w[v], r, back);
      const int64_t c = (v * tpr + u.t) * 8;
      if (a.dx) store8_warp<T, VEC>((T*)a.dx + row * a.lddx + c, t, n[v], u.first, u.last, live);
      if (a.drop.cut) {
        uint32_t bits[4];
        philox(bits, a.drop, (uint32_t)(v * tpr + u.t), (uint32_t)row);
        drop8(t, a.drop, bits);
      }
      store8_warp<T, VEC>((T*)a.df + row * a.lddf + c, t, n[v], u.first, u.last, live);
    }
  }
  float* out = a.parts + (int64_t)blockIdx.x * a.part_ld;
  if constexpr (MULTI) {
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n[v]) out[(v * tpr + u.t) * 8 + e] = sums[v][e];
  } else {  // the units of a warp, then the warps, one after the other
    for (int o = tpr; o < 32; o *= 2)
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[v][e] += __shfl_xor_sync(0xffffffffu, sums[v][e], o);
    for (int k = 0; k < (int)blockDim.x >> 5; ++k) {
      if (u.warp == k && u.lane < tpr)
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int c = (v * tpr + u.t) * 8 + e;
            lines[c] = k ? lines[c] + sums[v][e] : sums[v][e];
          }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < (int)a.cols; c += blockDim.x) out[c] = lines[c];
  }
}

// The column sums of long rows are kept in the CTA's row of parts.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kLongThreads) add_norm_long_bwd_kernel(const AddNormBwdArgs a) {
  __shared__ float red[2][16];
  const Unit u(kLongThreads, true);
  uint32_t calls = 0;
  const int64_t panels = (a.cols + kLongThreads * 8 - 1) / (kLongThreads * 8);
  float* out = a.parts + (int64_t)blockIdx.x * a.part_ld;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    float s = 0.f, dh[8], y[8], w[8];
    auto load = [&](int64_t c, int n) {
      load8<T, VEC>(dh, (const T*)a.dh + row * a.lddh + c, n);
      load8<T, VEC>(y, (const T*)a.y + row * a.ldy + c, n);
      load8<float, VEC>(w, a.w + c, n);
    };
    for (int64_t p = 0; p < panels; ++p) {
      const int64_t c = (p * kLongThreads + threadIdx.x) * 8;
      load(c, (int)max((int64_t)0, min((int64_t)8, a.cols - c)));
#pragma unroll
      for (int e = 0; e < 8; ++e) s = fmaf(dh[e] * w[e], y[e], s);
    }
    s = unit_sum<true>(s, u, red, calls);
    const float r = a.rstd[row], back = r * r * r * (s * (1.f / (float)a.cols));
    for (int64_t p = 0; p < panels; ++p) {
      const int64_t c = (p * kLongThreads + threadIdx.x) * 8, left = a.cols - c;
      const int n = (int)max((int64_t)0, min((int64_t)8, left));
      load(c, n);
      float dy[8] = {}, sums[8], t[8];
      if (a.dy) load8<T, VEC>(dy, (const T*)a.dy + row * a.lddy + c, n);
#pragma unroll
      for (int e = 0; e < 8; ++e) sums[e] = row != blockIdx.x && e < n ? out[c + e] : 0.f;
      into_t(t, sums, dy, dh, y, w, r, back);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) out[c + e] = sums[e];
      if (a.dx) store8_warp<T, VEC>((T*)a.dx + row * a.lddx + c, t, left, u.first, u.last, true);
      if (a.drop.cut) {
        uint32_t bits[4];
        philox(bits, a.drop, (uint32_t)(c >> 3), (uint32_t)row);
        drop8(t, a.drop, bits);
      }
      store8_warp<T, VEC>((T*)a.df + row * a.lddf + c, t, left, u.first, u.last, true);
    }
  }
}

// Threads of a unit, and of a CTA, and chunks a thread.
struct Shape {
  int tpr, threads, v;
  int units() const { return threads / tpr; }
};
Shape shape_of(int64_t cols) {
  if (cols > 8192) return {512, 512, 4};
  int tpr = 4;
  while (tpr * 16 < cols) tpr *= 2;
  return {tpr, std::max(tpr, tpr <= 32 ? 256 : 64), 2};
}
// CTAs that are resident together, of `threads` threads of at most 128 registers.
int64_t resident(int threads, int sms) { return (int64_t)sms * std::max(1, 512 / threads) * 2; }

template <typename T, bool VEC>
cudaError_t launch_fwd(const AddNormFwdArgs& a, int sms, cudaStream_t s) {
  if (a.cols > kMostFwd) {
    add_norm_long_fwd_kernel<T, VEC><<<(unsigned)std::min<int64_t>(a.rows, resident(kLongThreads, sms)), kLongThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
  const Shape sh = shape_of(a.cols);
  const unsigned ctas = (unsigned)std::min<int64_t>((a.rows + sh.units() - 1) / sh.units(), resident(sh.threads, sms));
  if (sh.v == 4) add_norm_fwd_kernel<T, VEC, 4, true><<<ctas, sh.threads, 0, s>>>(a, sh.tpr);
  else if (sh.tpr > 32) add_norm_fwd_kernel<T, VEC, 2, true><<<ctas, sh.threads, 0, s>>>(a, sh.tpr);
  else add_norm_fwd_kernel<T, VEC, 2, false><<<ctas, sh.threads, 0, s>>>(a, sh.tpr);
  return cudaGetLastError();
}

template <typename T, bool VEC>
cudaError_t launch_bwd(const AddNormBwdArgs& a, unsigned ctas, cudaStream_t s) {
  if (a.cols > kMostBwd) {
    add_norm_long_bwd_kernel<T, VEC><<<ctas, kLongThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
  const Shape sh = shape_of(a.cols);
  if (sh.tpr > 32) add_norm_bwd_kernel<T, VEC, 2, true><<<ctas, sh.threads, 0, s>>>(a, sh.tpr);
  else add_norm_bwd_kernel<T, VEC, 2, false><<<ctas, sh.threads, 0, s>>>(a, sh.tpr);
  return cudaGetLastError();
}

}  // namespace

int64_t add_norm_bwd_ctas(int64_t rows, int64_t cols, int sms) {
  if (cols > kMostBwd) return std::min<int64_t>(rows, resident(kLongThreads, sms));
  const Shape sh = shape_of(cols);
  return std::min<int64_t>((rows + sh.units() - 1) / sh.units(), resident(sh.threads, sms));
}

cudaError_t launch_add_norm_fwd(const AddNormFwdArgs& a, int dtype, int sms, cudaStream_t s) {
  if (dtype == DMUON_BF16) return a.vec ? launch_fwd<__nv_bfloat16, true>(a, sms, s) : launch_fwd<__nv_bfloat16, false>(a, sms, s);
  if (dtype == DMUON_F16) return a.vec ? launch_fwd<__half, true>(a, sms, s) : launch_fwd<__half, false>(a, sms, s);
  return a.vec ? launch_fwd<float, true>(a, sms, s) : launch_fwd<float, false>(a, sms, s);
}

cudaError_t launch_add_norm_bwd(const AddNormBwdArgs& a, int dtype, int64_t ctas_, cudaStream_t s) {
  const unsigned ctas = (unsigned)ctas_;
  if (dtype == DMUON_BF16) return a.vec ? launch_bwd<__nv_bfloat16, true>(a, ctas, s) : launch_bwd<__nv_bfloat16, false>(a, ctas, s);
  if (dtype == DMUON_F16) return a.vec ? launch_bwd<__half, true>(a, ctas, s) : launch_bwd<__half, false>(a, ctas, s);
  return a.vec ? launch_bwd<float, true>(a, ctas, s) : launch_bwd<float, false>(a, ctas, s);
}

}  // namespace dmuon
