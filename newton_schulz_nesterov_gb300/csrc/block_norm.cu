// Norms after and before a block with the block's gate and residual scale,
// forward and backward (formulas in block_norm.cuh).  Everything is computed
// in fp32; y, h, dx and df are rounded once to the activations' type, and the
// second norm takes y before it is rounded.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "../../include/dmuon.h"
#include "block_norm.cuh"
#include "ptx.cuh"

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

// ------------------------------------------------------------ rows up to 32768 columns
//
// A row is held by a unit of threads, eight columns a thread, so that it is
// read once: up to 4096 columns by one unit of a CTA (several units when rows
// are short), longer rows by a cluster of CTAs with 4096 columns each, whose
// row sums meet in distributed shared memory.  Both kernels are bound by HBM;
// a thread copies its own columns of the coming rows into a private ring in
// shared memory (cp.async: no registers, no barrier, kRing rows ahead) and
// keeps its columns' weights, gate row and column sums in registers over a
// run of consecutive rows.
//
// VEC: eight consecutive columns a thread, 16-byte accesses (every row 16-byte
// aligned, columns a multiple of 8).  Otherwise columns a unit apart, so that
// the scalar accesses of a warp are consecutive, loaded without the ring.
constexpr int kMaxThreads = 512;
constexpr int kPerThread = 8;
constexpr int64_t kCtaCols = (int64_t)kMaxThreads * kPerThread;
constexpr int kMaxCluster = 8;

struct RowUnit {
  int tpr;        // threads of a unit
  int unit, t;    // this thread's unit in the CTA and place in it
  int warps;      // of a unit
  int64_t col0, cols;  // columns of this CTA: [col0, col0 + cols)
};

__device__ __forceinline__ RowUnit row_unit(int64_t cols, int tpr) {
  RowUnit u;
  const uint32_t rank = ptx::cluster_ctarank();
  u.tpr = tpr;
  u.unit = threadIdx.x / tpr;
  u.t = threadIdx.x % tpr;
  u.warps = tpr / 32;
  u.col0 = rank * kCtaCols;
  u.cols = min(kCtaCols, cols - u.col0);
  return u;
}

template <bool VEC>
__device__ __forceinline__ int64_t col_of(const RowUnit& u, int e) {
  return VEC ? u.t * kPerThread + e : (int64_t)e * u.tpr + u.t;
}

// Sums of N <= 4 values over a row's threads, in a fixed order, to all of them.
// One barrier: consecutive calls alternate between two halves of `red`
// ([2][units][kMaxCluster * 16] float4), and a half is written again only
// after the next call's barrier, when every thread has read it.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], const RowUnit& u, float4* red, int& half, uint32_t clusters) {
#pragma unroll
  for (int k = 0; k < N; ++k)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if (clusters == 1 && u.warps == 1) return;
  const int units = blockDim.x / u.tpr;
  float4* mine = red + (half * units + u.unit) * (clusters == 1 ? 16 : kMaxCluster * 16);
  half ^= 1;
  const int warp = u.t >> 5;
  const float4 w = make_float4(v[0], N > 1 ? v[N > 1 ? 1 : 0] : 0.f, N > 2 ? v[N > 2 ? 2 : 0] : 0.f, N > 3 ? v[N > 3 ? 3 : 0] : 0.f);
  int n = u.warps;
  if (clusters == 1) {
    if ((u.t & 31) == 0) mine[warp] = w;
    asm volatile("bar.sync %0, %1;" ::"r"(u.unit + 1), "r"(u.tpr) : "memory");
  } else {
    n = u.warps * (int)clusters;
    const uint32_t rank = ptx::cluster_ctarank();
    if ((u.t & 31) < (int)clusters) {  // lane r tells rank r
      const uint32_t at = ptx::mapa_shared(ptx::smem_addr(mine + rank * u.warps + warp), u.t & 31);
      asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(w.x), "f"(w.y), "f"(w.z), "f"(w.w) : "memory");
    }
    ptx::cluster_sync();
  }
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = 0.f;
  for (int i = 0; i < n; ++i) {
    const float4 p = mine[i];
    const float q[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += q[k];
  }
}

// This thread's eight values of one row.
template <typename T>
struct Row8 {
  uint32_t w[sizeof(T) * 2];
  __device__ __forceinline__ float at(int e) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
    const uint32_t p = w[e >> 1];
    if constexpr (std::is_same<T, __half>::value) {
      const __half2 h = *reinterpret_cast<const __half2*>(&p);
      return (e & 1) ? __high2float(h) : __low2float(h);
    } else {
      return __uint_as_float((e & 1) ? (p & 0xFFFF0000u) : (p << 16));
    }
  }
};

constexpr int chunks_of(int size) { return size * kPerThread / 16; }  // 16-byte chunks a thread and row

template <typename T, bool VEC>
__device__ __forceinline__ Row8<T> load_direct(const T* row, const RowUnit& u) {
  Row8<T> r;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(T) * 2); ++i) r.w[i] = 0;
#pragma unroll
  for (int e = 0; e < kPerThread; ++e) {
    const int64_t c = col_of<VEC>(u, e);
    if (c >= u.cols) continue;
    if constexpr (sizeof(T) == 4) r.w[e] = reinterpret_cast<const uint32_t*>(row)[u.col0 + c];
    else r.w[e >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(row)[u.col0 + c] << (16 * (e & 1));
  }
  return r;
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_row(T* row, const RowUnit& u, const float (&v)[kPerThread]) {
  if constexpr (VEC) {
    if (u.t * kPerThread >= u.cols) return;
    __align__(16) T o[kPerThread];
#pragma unroll
    for (int e = 0; e < kPerThread; ++e) o[e] = narrow<T>(v[e]);
    uint4* dst = reinterpret_cast<uint4*>(row + u.col0 + u.t * kPerThread);
#pragma unroll
    for (int i = 0; i < chunks_of(sizeof(T)); ++i) dst[i] = reinterpret_cast<const uint4*>(o)[i];
  } else {
#pragma unroll
    for (int e = 0; e < kPerThread; ++e) {
      const int64_t c = col_of<VEC>(u, e);
      if (c < u.cols) row[u.col0 + c] = narrow<T>(v[e]);
    }
  }
}

// A parameter's (fp32, per column) eight values; absent: `other`.
template <bool VEC>
__device__ __forceinline__ void load_param(float (&v)[kPerThread], const float* p, const RowUnit& u, float other) {
#pragma unroll
  for (int e = 0; e < kPerThread; ++e) {
    const int64_t c = col_of<VEC>(u, e);
    v[e] = c < u.cols ? (p ? p[u.col0 + c] : other) : 0.f;
  }
}

template <bool VEC>
__device__ __forceinline__ void store_param(float* p, const RowUnit& u, const float (&v)[kPerThread]) {
#pragma unroll
  for (int e = 0; e < kPerThread; ++e) {
    const int64_t c = col_of<VEC>(u, e);
    if (c < u.cols) p[u.col0 + c] = v[e];
  }
}

// The private ring: slot s, array k, chunk i of this thread.
template <typename T, int ARRAYS>
struct Ring {
  uint8_t* base;
  __device__ __forceinline__ uint8_t* at(int s, int k, int i) const {
    return base + ((size_t)((s * ARRAYS + k) * chunks_of(sizeof(T)) + i) * blockDim.x + threadIdx.x) * 16;
  }
  __device__ __forceinline__ void fetch(int s, int k, const T* row, const RowUnit& u) const {
    if (u.t * kPerThread >= u.cols) return;
    const uint8_t* src = reinterpret_cast<const uint8_t*>(row + u.col0 + u.t * kPerThread);
#pragma unroll
    for (int i = 0; i < chunks_of(sizeof(T)); ++i)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_addr(at(s, k, i))), "l"(src + 16 * i) : "memory");
  }
  __device__ __forceinline__ Row8<T> take(int s, int k, const RowUnit& u) const {
    Row8<T> r;
#pragma unroll
    for (int i = 0; i < chunks_of(sizeof(T)); ++i) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (u.t * kPerThread < u.cols) v = *reinterpret_cast<const uint4*>(at(s, k, i));
      r.w[4 * i] = v.x; r.w[4 * i + 1] = v.y; r.w[4 * i + 2] = v.z; r.w[4 * i + 3] = v.w;
    }
    return r;
  }
};

__device__ __forceinline__ void commit_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_group() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <typename T>
constexpr int fwd_ring() { return sizeof(T) == 4 ? 3 : 4; }
template <typename T>
constexpr int bwd_ring() { return sizeof(T) == 4 ? 2 : 4; }
constexpr int red_bytes(int units, int clusters) { return 2 * units * (clusters == 1 ? 16 : kMaxCluster * 16) * 16; }

// Unit u of all takes rows [u n, (u + 1) n): consecutive, so that the gate row
// stays in registers.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kMaxThreads, 2) norm_fwd_rows_kernel(const NormFwdArgs a, int tpr, int clusters) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int kRing = fwd_ring<T>();
  const RowUnit u = row_unit(a.cols, tpr);
  const int units = blockDim.x / tpr;
  float4* red = reinterpret_cast<float4*>(smem);
  const Ring<T, 2> ring{smem + red_bytes(units, clusters)};
  const int64_t all = (int64_t)gridDim.x / clusters * units, id = (int64_t)(blockIdx.x / clusters) * units + u.unit;
  const int64_t per = (a.rows + all - 1) / all, row0 = id * per, row1 = min(row0 + per, a.rows);
  auto fetch = [&](int64_t row, int s) {
    if (row < row1) {
      ring.fetch(s, 0, (const T*)a.x + row * a.ldx, u);
      ring.fetch(s, 1, (const T*)a.f + row * a.ldf, u);
    }
    commit_group();
  };
  if constexpr (VEC)
    for (int s = 0; s < kRing; ++s) fetch(row0 + s, s);
  float post[kPerThread], pre[kPerThread], res[kPerThread], gw[kPerThread];
  load_param<VEC>(post, a.post_w, u, 1.f);
  load_param<VEC>(pre, a.pre_w, u, 1.f);
  load_param<VEC>(res, a.res, u, 1.f);
#pragma unroll
  for (int e = 0; e < kPerThread; ++e) gw[e] = post[e];
  const float inv = 1.f / (float)a.cols;
  int64_t group = -1, group_end = a.gate ? 0 : INT64_MAX;  // first row past the gate row in gw
  int slot = 0, half = 0;
  for (int64_t row = row0; row < row1; ++row) {
    if (row >= group_end) {
      group = row / a.per_gate;
      group_end = (group + 1) * a.per_gate;
      load_param<VEC>(gw, a.gate + group * a.cols, u, 1.f);
#pragma unroll
      for (int e = 0; e < kPerThread; ++e) gw[e] *= post[e];
    }
    Row8<T> x, f;
    if constexpr (VEC) {
      wait_group<kRing - 1>();
      x = ring.take(slot, 0, u);
      f = ring.take(slot, 1, u);
    } else {
      x = load_direct<T, VEC>((const T*)a.x + row * a.ldx, u);
      f = load_direct<T, VEC>((const T*)a.f + row * a.ldf, u);
    }
    float s[1] = {0.f};
#pragma unroll
    for (int e = 0; e < kPerThread; ++e) s[0] = fmaf(f.at(e), f.at(e), s[0]);
    row_sum<1>(s, u, red, half, clusters);
    const float r1 = 1.f / sqrtf(s[0] * inv + a.eps);
    float y[kPerThread];
    s[0] = 0.f;
#pragma unroll
    for (int e = 0; e < kPerThread; ++e) {
      y[e] = fmaf(x.at(e), res[e], f.at(e) * r1 * gw[e]);
      s[0] = fmaf(y[e], y[e], s[0]);
    }
    if constexpr (VEC) {
      fetch(row + kRing, slot);  // this thread has taken its slot
      if (++slot == kRing) slot = 0;
    }
    store_row<T, VEC>((T*)a.y + row * a.ldy, u, y);
    row_sum<1>(s, u, red, half, clusters);
    const float r2 = 1.f / sqrtf(s[0] * inv + a.eps);
#pragma unroll
    for (int e = 0; e < kPerThread; ++e) y[e] *= r2 * pre[e];
    store_row<T, VEC>((T*)a.h + row * a.ldh, u, y);
    if (u.t == 0 && u.col0 == 0) {
      a.rstd[row] = r1;
      a.rstd[a.rows + row] = r2;
    }
  }
  if (clusters > 1) ptx::cluster_sync();  // a peer may still read this CTA's shared memory
}

// The rows of a unit, chunk after chunk.
struct ChunkRows {
  const NormBwdArgs& a;
  int64_t all, chunk, row, end;
  __device__ __forceinline__ ChunkRows(const NormBwdArgs& a_, int64_t id, int64_t all_) : a(a_), all(all_), chunk(id), row(0), end(0) { open(); }
  __device__ __forceinline__ void open() {  // the first non-empty chunk from `chunk` on
    const int64_t n = a.groups * a.chunks_per_group;
    for (; chunk < n; chunk += all) {
      const int64_t group = chunk / a.chunks_per_group, part = chunk % a.chunks_per_group;
      row = group * a.per_gate + part * a.chunk_rows;
      end = min(min(row + a.chunk_rows, (group + 1) * a.per_gate), a.rows);
      if (row < end) return;
    }
    chunk = INT64_MAX;
  }
  __device__ __forceinline__ bool done() const { return chunk == INT64_MAX; }
  __device__ __forceinline__ void next() {
    if (++row == end) {
      chunk += all;
      open();
    }
  }
};

// One row needs mean(dh w_pre yn) for t and then mean(g t w_post fn) for df;
// with t = dy + r2 (i - yn m2), i = dh w_pre, the second is
//   mean(g w fn (dy + r2 i)) - r2 m2 mean(g w fn yn)
// so that one round of three sums serves both (the rounding is that of t's own
// terms).  Units' column sums go to their own rows of the partial arrays, in
// a fixed order, and are added up by norm_bwd_sums_kernel.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kMaxThreads, 1) norm_bwd_rows_kernel(const NormBwdArgs a, int tpr, int clusters) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int kRing = bwd_ring<T>();
  const RowUnit u = row_unit(a.cols, tpr);
  const int units = blockDim.x / tpr;
  float4* red = reinterpret_cast<float4*>(smem);
  const Ring<T, 5> ring{smem + red_bytes(units, clusters)};
  const int64_t all = (int64_t)gridDim.x / clusters * units, id = (int64_t)(blockIdx.x / clusters) * units + u.unit;
  const bool with_x = a.d_res != nullptr;
  ChunkRows ahead(a, id, all), at(a, id, all);
  auto fetch = [&](int s) {
    if (!ahead.done()) {
      const int64_t row = ahead.row;
      if (a.dy) ring.fetch(s, 0, (const T*)a.dy + row * a.lddy, u);
      ring.fetch(s, 1, (const T*)a.dh + row * a.lddh, u);
      ring.fetch(s, 2, (const T*)a.y + row * a.ldy, u);
      ring.fetch(s, 3, (const T*)a.f + row * a.ldf, u);
      if (with_x) ring.fetch(s, 4, (const T*)a.x + row * a.ldx, u);
      ahead.next();
    }
    commit_group();
  };
  if constexpr (VEC)
    for (int s = 0; s < kRing; ++s) fetch(s);
  float pre[kPerThread], res[kPerThread], gw[kPerThread];
  load_param<VEC>(pre, a.pre_w, u, 1.f);
  load_param<VEC>(res, a.res, u, 1.f);
  float sum_pre[kPerThread], sum_post[kPerThread], sum_res[kPerThread], sum_t[kPerThread];
#pragma unroll
  for (int e = 0; e < kPerThread; ++e) sum_pre[e] = sum_post[e] = sum_res[e] = sum_t[e] = 0.f;
  const float inv = 1.f / (float)a.cols;
  int64_t chunk = -1;
  int slot = 0, half = 0;
  // t fn summed over a chunk belongs to one gate row.
  auto flush = [&]() {
    float g[kPerThread], w[kPerThread];
    const int64_t group = chunk / a.chunks_per_group;
    load_param<VEC>(g, a.gate ? a.gate + group * a.cols : nullptr, u, 1.f);
#pragma unroll
    for (int e = 0; e < kPerThread; ++e) sum_post[e] = fmaf(g[e], sum_t[e], sum_post[e]);
    if (a.d_gate) {
      if (a.chunks_per_group > 1) {
        store_param<VEC>(a.part_gate + chunk * a.cols, u, sum_t);
      } else {
        load_param<VEC>(w, a.post_w, u, 1.f);
#pragma unroll
        for (int e = 0; e < kPerThread; ++e) w[e] *= sum_t[e];
        store_param<VEC>(a.d_gate + group * a.cols, u, w);
      }
    }
#pragma unroll
    for (int e = 0; e < kPerThread; ++e) sum_t[e] = 0.f;
  };
  float n1 = 0.f, n2 = 0.f;
  if (!at.done()) {
    n1 = a.rstd[at.row];
    n2 = a.rstd[a.rows + at.row];
  }
  while (!at.done()) {
    const int64_t row = at.row;
    const float r1 = n1, r2 = n2;
    if (at.chunk != chunk) {
      if (chunk >= 0) flush();
      chunk = at.chunk;
      load_param<VEC>(gw, a.post_w, u, 1.f);
      if (a.gate) {
        float g[kPerThread];
        load_param<VEC>(g, a.gate + chunk / a.chunks_per_group * a.cols, u, 1.f);
#pragma unroll
        for (int e = 0; e < kPerThread; ++e) gw[e] *= g[e];
      }
    }
    at.next();
    if (!at.done()) {  // the next row's, before it is needed
      n1 = a.rstd[at.row];
      n2 = a.rstd[a.rows + at.row];
    }
    Row8<T> dy, dh, y, f, x;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) * 2); ++i) dy.w[i] = x.w[i] = 0;
    if constexpr (VEC) {
      wait_group<kRing - 1>();
      if (a.dy) dy = ring.take(slot, 0, u);
      dh = ring.take(slot, 1, u);
      y = ring.take(slot, 2, u);
      f = ring.take(slot, 3, u);
      if (with_x) x = ring.take(slot, 4, u);
    } else {
      if (a.dy) dy = load_direct<T, VEC>((const T*)a.dy + row * a.lddy, u);
      dh = load_direct<T, VEC>((const T*)a.dh + row * a.lddh, u);
      y = load_direct<T, VEC>((const T*)a.y + row * a.ldy, u);
      f = load_direct<T, VEC>((const T*)a.f + row * a.ldf, u);
      if (with_x) x = load_direct<T, VEC>((const T*)a.x + row * a.ldx, u);
    }
    float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < kPerThread; ++e) {
      const float i = dh.at(e) * pre[e], yn = y.at(e) * r2, b = gw[e] * (f.at(e) * r1);
      s[0] = fmaf(i, yn, s[0]);
      s[1] = fmaf(b, fmaf(r2, i, dy.at(e)), s[1]);
      s[2] = fmaf(b, yn, s[2]);
    }
    row_sum<3>(s, u, red, half, clusters);
    const float m2 = s[0] * inv, m1 = (s[1] - r2 * m2 * s[2]) * inv;
    float dx[kPerThread], df[kPerThread];
#pragma unroll
    for (int e = 0; e < kPerThread; ++e) {
      const float yn = y.at(e) * r2, fn = f.at(e) * r1;
      const float t = fmaf(r2, fmaf(-yn, m2, dh.at(e) * pre[e]), dy.at(e));
      sum_pre[e] = fmaf(dh.at(e), yn, sum_pre[e]);
      sum_t[e] = fmaf(t, fn, sum_t[e]);
      sum_res[e] = fmaf(t, x.at(e), sum_res[e]);
      dx[e] = res[e] * t;
      df[e] = r1 * fmaf(-fn, m1, gw[e] * t);
    }
    if constexpr (VEC) {
      fetch(slot);
      if (++slot == kRing) slot = 0;
    }
    store_row<T, VEC>((T*)a.dx + row * a.lddx, u, dx);
    store_row<T, VEC>((T*)a.df + row * a.lddf, u, df);
  }
  if (chunk >= 0) flush();
  store_param<VEC>(a.part_pre + id * a.cols, u, sum_pre);
  store_param<VEC>(a.part_post + id * a.cols, u, sum_post);
  if (with_x) store_param<VEC>(a.part_res + id * a.cols, u, sum_res);
  if (clusters > 1) ptx::cluster_sync();  // a peer may still read this CTA's shared memory
}

// ------------------------------------------------------------ longer rows
//
// One CTA a row (forward) or chunk (backward), passes over the row from L2.

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

// Column sums over the units' partial rows (blockIdx.y: 0 pre, 1 post, 2 res)
// and, from 3 on, over the chunks of gate group blockIdx.y - 3: 32 columns a
// block, its 32 warps over the rows in turn, then the warps in order.
__global__ void __launch_bounds__(1024) norm_bwd_sums_kernel(const NormBwdArgs a) {
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  const float* src;
  float* dst;
  int64_t n = a.units;
  if (blockIdx.y == 0) { src = a.part_pre; dst = a.d_pre_w; }
  else if (blockIdx.y == 1) { src = a.part_post; dst = a.d_post_w; }
  else if (blockIdx.y == 2) { src = a.part_res; dst = a.d_res; }
  else {
    const int64_t g = blockIdx.y - 3;
    // The last group may be short: its chunks past the rows are not written.
    n = (min(a.per_gate, a.rows - g * a.per_gate) + a.chunk_rows - 1) / a.chunk_rows;
    src = a.part_gate + g * a.chunks_per_group * a.cols;
    dst = a.d_gate + g * a.cols;
  }
  if (!dst) return;
  float s = 0.f;
  if (c < a.cols) {
#pragma unroll 8
    for (int64_t i = warp; i < n; i += 32) s += src[i * a.cols + c];
  }
  red[warp][lane] = s;
  __syncthreads();
  // Transposed: warp w adds up column w, lane by lane in a fixed tree.
  float v = red[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int64_t out = (int64_t)blockIdx.x * 32 + warp;
  if (lane == 0 && out < a.cols) dst[out] = blockIdx.y >= 3 ? v * a.post_w[out] : v;
}

// ------------------------------------------------------------ launches

// Threads of a unit, CTAs of a cluster and units of a CTA for rows of `cols`.
struct RowShape {
  int tpr, clusters, units;
};
RowShape row_shape(int64_t cols) {
  RowShape r;
  r.clusters = cols <= kCtaCols ? 1 : cols <= 2 * kCtaCols ? 2 : cols <= 4 * kCtaCols ? 4 : kMaxCluster;
  r.tpr = cols <= kCtaCols ? (int)((cols + 32 * kPerThread - 1) / (32 * kPerThread)) * 32 : kMaxThreads;
  r.units = r.clusters > 1 ? 1 : std::max(1, std::min(kMaxThreads / r.tpr, 15));
  return r;
}
bool held(int64_t cols) { return cols <= kMaxCluster * kCtaCols; }

template <typename K, typename A>
cudaError_t launch_rows(K kernel, const A& a, const RowShape& r, int64_t ctas, int smem, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = r.clusters;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(ctas * r.clusters), 1, 1);
  cfg.blockDim = dim3(r.tpr * r.units, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, r.tpr, r.clusters);
}

template <typename T>
int ring_bytes(const RowShape& r, int arrays, int depth) {
  return red_bytes(r.units, r.clusters) + depth * arrays * chunks_of(sizeof(T)) * r.tpr * r.units * 16;
}

template <typename T>
cudaError_t fwd(const NormFwdArgs& a, int sms, cudaStream_t s) {
  if (!held(a.cols)) {
    const int64_t grid = std::min(a.rows, (int64_t)sms * 8);
    norm_fwd_kernel<T><<<(unsigned)grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
  const RowShape r = row_shape(a.cols);
  const int64_t ctas = std::min((a.rows + r.units - 1) / r.units, (int64_t)std::max(1, sms * 2 / r.clusters));
  if (a.vec) return launch_rows(norm_fwd_rows_kernel<T, true>, a, r, ctas, ring_bytes<T>(r, 2, fwd_ring<T>()), s);
  return launch_rows(norm_fwd_rows_kernel<T, false>, a, r, ctas, red_bytes(r.units, r.clusters), s);
}

template <typename T>
cudaError_t bwd(const NormBwdArgs& a, cudaStream_t s) {
  cudaError_t e;
  if (!held(a.cols)) {
    norm_bwd_kernel<T><<<(unsigned)a.units, kThreads, 0, s>>>(a);
    e = cudaGetLastError();
  } else {
    const RowShape r = row_shape(a.cols);
    const int64_t ctas = a.units / r.units;
    if (a.vec) e = launch_rows(norm_bwd_rows_kernel<T, true>, a, r, ctas, ring_bytes<T>(r, 5, bwd_ring<T>()), s);
    else e = launch_rows(norm_bwd_rows_kernel<T, false>, a, r, ctas, red_bytes(r.units, r.clusters), s);
  }
  if (e != cudaSuccess) return e;
  const unsigned ys = 3 + (a.d_gate && a.chunks_per_group > 1 ? (unsigned)a.groups : 0u);
  norm_bwd_sums_kernel<<<dim3((unsigned)((a.cols + 31) / 32), ys), 1024, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

// One CTA or cluster a SM share; no more units than rows.
int64_t norm_bwd_units(int64_t rows, int64_t cols, int sms) {
  if (!held(cols)) return std::min<int64_t>(std::max<int64_t>(rows, 1), (int64_t)sms * 4);
  const RowShape r = row_shape(cols);
  const int64_t ctas = std::min<int64_t>(std::max(1, sms / r.clusters), (std::max<int64_t>(rows, 1) + r.units - 1) / r.units);
  return ctas * r.units;
}

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
