// Norms after and before a block with the block's gate and residual scale,
// forward and backward (formulas in block_norm.cuh).  Everything is computed
// in fp32; y, h, dx and df are rounded once to the activations' type, and the
// second norm takes y before it is rounded.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <climits>
#include <type_traits>

#include "../../include/dmuon.h"
#include "block_norm.cuh"
#include "bounded_wait.cuh"
#include "f32x2.cuh"
#include "pieces.cuh"
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
// A row is held by a unit of threads, two chunks of eight columns a thread, so
// that it is read once.  Rows too long for a CTA go to a cluster of CTAs whose
// row sums meet in distributed shared memory.  Both kernels are bound by HBM;
// a thread copies its own columns of the coming rows into a private ring in
// shared memory (cp.async: no registers, no barrier) and keeps its columns'
// weights, gate row and column sums in registers over consecutive rows.
// Beside its traffic a row costs issue slots and the latency of its sums.  At
// 16384 x 4096 bf16 the forward takes 87 us (6.2 TB/s) and the backward 146
// and 7 for the column sums (6.1 TB/s); the forward took 172 with one chunk a
// thread (every second instruction belongs to sums and loops) and 137 with
// four and the weights from L1.
//
// VEC: chunks of eight consecutive columns, 16-byte accesses (every row and
// parameter 16-byte aligned, columns a multiple of 8).  Otherwise columns a
// unit apart, so that the scalar accesses of a warp are consecutive, loaded
// without the ring; but the backward of 2-byte types, whose loads and stores
// these would bind, gives a thread sixteen consecutive columns: the ring takes
// the three aligned 16-byte pieces around them, they are shifted together from
// there, and shifted back for aligned stores with the neighbour's last words
// (16384 x 4095 bf16 backward 290 us one by one, 232 so; 65535 x 255 182 and
// 84).  The forward is no faster that way (16384 x 4095 bf16 134 us
// against 128, and 4.4 against 3.3 at 300 x 501).
// Rows on any element cost registers: 12 of their 27 instances spill, the worst
// (fp32 backward of rows that share a warp) 208 bytes of stores and 304 of loads.
constexpr int V = 2;                             // chunks of eight columns a thread
constexpr int kFwdThreads = 512, kBwdThreads = 256;  // of an SM: 128 and 255 registers a thread
constexpr int kMaxCluster = 8;

struct RowUnit {
  int tpr;        // threads of a unit: a power of two below 32, or whole warps
  int unit, t;    // this thread's unit in the CTA and place in it
  int warps;      // of a unit
  int col0, cols; // columns of this CTA: [col0, col0 + cols)
};

__device__ __forceinline__ RowUnit row_unit(int64_t cols, int tpr) {
  RowUnit u;
  u.tpr = tpr;
  u.unit = threadIdx.x / tpr;
  u.t = threadIdx.x % tpr;
  u.warps = max(1, tpr / 32);
  u.col0 = (int)ptx::cluster_ctarank() * tpr * V * 8;
  u.cols = max(0, min(tpr * V * 8, (int)cols - u.col0));
  return u;
}

// Column of value e of chunk v, in the CTA: runs of E columns a thread (the 16
// bytes of an access, 1, or all of them), runs of the unit's threads side by side.
template <int E>
__device__ __forceinline__ int col_of(const RowUnit& u, int v, int e) {
  if constexpr (E == 8 * V) return u.t * E + v * 8 + e;
  else return ((v * (8 / E) + e / E) * u.tpr + u.t) * E + e % E;
}
// How a thread's values come: whole chunks, one by one, or by shifted pieces.
enum Access { kChunks, kSingles, kPieces };
template <typename T>
constexpr int run_of(Access how) { return how == kChunks ? 16 / (int)sizeof(T) : how == kSingles ? 1 : 8 * V; }

// Sums of N values over a row's threads, in a fixed order, to all of them.
// Consecutive calls alternate between two halves of `red` ([2][units][3]
// [kRedRow] floats, zero at first) and, in clusters, two barriers.  A half is
// written again only after the next call's barrier, when every thread has read
// it.  In a cluster every warp sends its sums to every CTA (st.async, counted
// on that CTA's barrier): a cluster barrier a row would wait for the row's
// global stores too (4096 x 8192 bf16 backward: 135 us against 112).
constexpr int kRedRow = kMaxCluster * 16;  // warps of a row at most
// Kinds of units: narrower than a warp, of one CTA, of a cluster of CTAs.
enum Kind { kSub, kCta, kCluster };
struct RowSums {
  float* red;
  uint32_t bars;          // two mbarriers, in clusters
  int clusters, units;
  uint32_t calls;
  int* err;
  uint64_t limit_ns;
  __device__ __forceinline__ void init(float* r, uint64_t* b, int cl, int un, int* e, uint64_t limit) {
    red = r;
    bars = ptx::smem_addr(b);
    clusters = cl;
    units = un;
    calls = 0;
    err = e;
    limit_ns = limit;
    if (cl > 1 || blockDim.x / un > 32)
      for (int i = threadIdx.x; i < 2 * un * 3 * kRedRow; i += blockDim.x) r[i] = 0.f;
    if (cl > 1 && threadIdx.x == 0) {
      ptx::mbar_init(bars, 1);
      ptx::mbar_init(bars + 8, 1);
      ptx::fence_mbar_init();
    }
  }
};

// A wait of row_sum in a cluster, with the same answer for a whole warp.  One
// that passes the handle's limit sets *err; its sums then have kWaitNs more to
// come, and if they do the kernel goes on with them, its barriers in step.
// False: they do not come.  Nothing but this wait decides: *err may hold what
// an earlier call of the handle left there.
__device__ __forceinline__ bool wait_sums(uint32_t bar, uint32_t parity, int* err, uint64_t limit_ns) {
  if (__all_sync(0xffffffffu, ptx::mbar_try(bar, parity))) return true;
  const uint64_t limit = limit_ns ? limit_ns : kWaitNs;
  uint64_t t0 = ptx::globaltimer();
  bool late = false;
  while (!__all_sync(0xffffffffu, ptx::mbar_try(bar, parity))) {
    if (!__any_sync(0xffffffffu, ptx::globaltimer() - t0 > (late ? kWaitNs : limit))) continue;
    if (late) return false;
    late = true;
    if ((threadIdx.x & 31) == 0) atomicOr(err, 1);
    t0 = ptx::globaltimer();
  }
  return true;
}

// After a wait that returned false and the cluster barrier behind which no CTA
// sends any more: what was sent to this CTA lands before it exits.  Peers are at
// most one call ahead, since they wait for this CTA's sums too.
__device__ __forceinline__ void land_sums(const RowSums& s) {
  for (uint32_t c = s.calls; c < s.calls + 2; ++c) {
    const uint64_t t0 = ptx::globaltimer();
    while (!ptx::mbar_try(s.bars + 8 * (c & 1), (c >> 1) & 1) && ptx::globaltimer() - t0 < kWaitNs) {
    }
  }
}

// False only in a cluster, one of whose CTAs does not come: the kernel leaves its rows.
template <int N, int KIND>
__device__ __forceinline__ bool row_sum(float (&v)[N], const RowUnit& u, RowSums& s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (KIND != kSub || o < u.tpr)
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if (KIND == kSub || (KIND == kCta && u.warps == 1)) return true;
  const int lane = threadIdx.x & 31, warp = u.t >> 5, half = s.calls & 1;
  float* mine = s.red + (half * s.units + u.unit) * 3 * kRedRow;
  int n = u.warps;
  if constexpr (KIND == kCta) {
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < N; ++k) mine[k * kRedRow + warp] = v[k];
    asm volatile("bar.sync %0, %1;" ::"r"(u.unit + 1), "r"(u.tpr) : "memory");
  } else {
    n = u.warps * s.clusters;
    const uint32_t bar = s.bars + 8 * half;
    if (threadIdx.x == 0) ptx::mbar_expect_tx(bar, n * N * 4);
    if (lane < s.clusters) {  // lane r tells rank r
      const uint32_t rank = ptx::cluster_ctarank(), there = ptx::mapa_shared(bar, lane);
#pragma unroll
      for (int k = 0; k < N; ++k)
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(
                         ptx::mapa_shared(ptx::smem_addr(mine + k * kRedRow + rank * u.warps + warp), lane)),
                     "r"(__float_as_uint(v[k])), "r"(there)
                     : "memory");
    }
    if (!wait_sums(bar, (s.calls >> 1) & 1, s.err, s.limit_ns)) return false;
  }
  ++s.calls;
  if (KIND == kCta && n <= 8) {  // what no warp writes is zero
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float4 p = *reinterpret_cast<const float4*>(mine + k * kRedRow), q = *reinterpret_cast<const float4*>(mine + k * kRedRow + 4);
      v[k] = ((p.x + p.y) + (p.z + p.w)) + ((q.x + q.y) + (q.z + q.w));
    }
    return true;
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    v[k] = 0.f;
    for (int i = lane; i < n; i += 32) v[k] += mine[k * kRedRow + i];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  return true;
}

// A chunk: eight values of one row in their type.
template <typename T>
struct Chunk8 {
  uint32_t w[sizeof(T) * 2];
  __device__ __forceinline__ f2 pair(int i) const {  // values 2i, 2i + 1
    if constexpr (sizeof(T) == 4) return pack2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    if constexpr (std::is_same<T, __half>::value) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      return pack2(f.x, f.y);
    }
    return pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) * 2); ++i) w[i] = 0;
  }
};

constexpr int parts_of(int size) { return size / 2; }  // 16-byte parts of a chunk

// Eight values in their type.
template <typename T>
__device__ __forceinline__ void pack4(const f2 (&val)[4], uint32_t* w) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack2(val[i]);
    if constexpr (std::is_same<T, __half>::value) {
      const __half2 h = __floats2half2_rn(p.x, p.y);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(p.x, p.y);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
}

// `row` is the first of this CTA's columns, here and below.
template <typename T>
__device__ __forceinline__ Chunk8<T> load_direct(const T* row, const RowUnit& u, int v) {
  Chunk8<T> r;
  r.zero();
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int c = col_of<1>(u, v, e);
    if (c >= u.cols) continue;
    if constexpr (sizeof(T) == 4) r.w[e] = reinterpret_cast<const uint32_t*>(row)[c];
    else r.w[e >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(row)[c] << (16 * (e & 1));
  }
  return r;
}

template <typename T, int E>
__device__ __forceinline__ void store_chunk(T* row, const RowUnit& u, int v, const f2 (&val)[4]) {
  float o[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack2(val[i]);
    o[2 * i] = p.x;
    o[2 * i + 1] = p.y;
  }
  if constexpr (E == 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = col_of<1>(u, v, e);
      if (c < u.cols) row[c] = narrow<T>(o[e]);
    }
  } else if constexpr (sizeof(T) == 4) {
    const bool wide = E < 8 * V || ((uintptr_t)row & 15) == 0;
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
      const int c = col_of<E>(u, v, e);
      if (wide && c + 3 < u.cols) {
        *reinterpret_cast<uint4*>(row + c) = make_uint4(__float_as_uint(o[e]), __float_as_uint(o[e + 1]), __float_as_uint(o[e + 2]),
                                                        __float_as_uint(o[e + 3]));
      } else if (E == 8 * V) {
#pragma unroll
        for (int j = e; j < e + 4; ++j) {
          const int cj = col_of<E>(u, v, j);
          if (cj < u.cols) row[cj] = o[j];
        }
      }
    }
  } else {
    const int c = col_of<E>(u, v, 0);
    if (c >= u.cols) return;
    uint32_t w[4];
    pack4<T>(val, w);
    *reinterpret_cast<uint4*>(row + c) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Sixteen values of 2 bytes a thread.  All lanes of a warp call it.
template <typename T>
__device__ __forceinline__ void store_shifted(T* row, const RowUnit& u, const f2 (&val)[V][4], bool live) {
  uint32_t w[16];
#pragma unroll
  for (int v = 0; v < V; ++v) pack4<T>(val[v], w + 4 + 4 * v);
  const int lane = threadIdx.x & 31, c = u.t * 8 * V;
  store_pieces<2>(reinterpret_cast<uint8_t*>(row + c), w, (u.cols - c) * 2, lane == 0 || u.t == 0,
                  lane == 31 || u.t + 1 == u.tpr || c + 32 > u.cols, live);
}

// Eight fp32 values of a parameter (its first column is column 0 of the row);
// 0 past the columns.
template <int E>
__device__ __forceinline__ void load_param(f2 (&val)[4], const float* p, const RowUnit& u, int v) {
  p += u.col0;
  if constexpr (E == 8 * V) {
    const bool wide = ((uintptr_t)p & 15) == 0;
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
      const int c = col_of<E>(u, v, e);
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      if (wide && c + 3 < u.cols) {
        a = *reinterpret_cast<const float4*>(p + c);
      } else {
        if (c < u.cols) a.x = p[c];
        if (c + 1 < u.cols) a.y = p[c + 1];
        if (c + 2 < u.cols) a.z = p[c + 2];
        if (c + 3 < u.cols) a.w = p[c + 3];
      }
      val[e / 2] = pack2(a.x, a.y);
      val[e / 2 + 1] = pack2(a.z, a.w);
    }
  } else if constexpr (E > 1) {
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
      const int c = col_of<E>(u, v, e);
      const float4 a = c < u.cols ? *reinterpret_cast<const float4*>(p + c) : make_float4(0.f, 0.f, 0.f, 0.f);
      val[e / 2] = pack2(a.x, a.y);
      val[e / 2 + 1] = pack2(a.z, a.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c0 = col_of<1>(u, v, 2 * i), c1 = col_of<1>(u, v, 2 * i + 1);
      val[i] = pack2(c0 < u.cols ? p[c0] : 0.f, c1 < u.cols ? p[c1] : 0.f);
    }
  }
}

template <int E>
__device__ __forceinline__ void store_param(float* p, const RowUnit& u, int v, const f2 (&val)[4]) {
  store_chunk<float, E>(p + u.col0, u, v, val);
}

// The private ring: slot s, array k, part i of chunk v of this thread, or
// (rows on any element) piece i of the three around both chunks.
template <typename T>
constexpr int row_parts(Access how) { return how == kPieces ? 3 : V * parts_of(sizeof(T)); }
template <typename T, int ARRAYS, Access HOW>
struct Ring {
  static constexpr int E = 16 / (int)sizeof(T);
  uint32_t base, step;  // this thread's part 0; bytes from one part to the next
  __device__ __forceinline__ uint32_t slot(int s) const { return base + s * ARRAYS * row_parts<T>(HOW) * step; }
  __device__ __forceinline__ void fetch(uint32_t slot, int k, const T* row, const RowUnit& u) const {
    if constexpr (HOW == kPieces) {
      // Aligned pieces, cut off at the row's end (zeros from there on); before
      // the row they begin at most 14 bytes early, in the piece of its first byte.
      if (u.t * 8 * V >= u.cols) return;
      const uint32_t m = past16(row);
      const uint8_t* from = reinterpret_cast<const uint8_t*>(row + u.t * 8 * V) - m;
      const int left = (u.cols - u.t * 8 * V) * 2 + (int)m;  // bytes to the row's end
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const int n = i == 2 && m == 0 ? 0 : max(0, min(16, left - 16 * i));
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(slot + (k * 3 + i) * step), "l"(n ? from + 16 * i : from), "r"(n)
                     : "memory");
      }
      return;
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < parts_of(sizeof(T)); ++i) {
        const int c = col_of<E>(u, v, i * E);
        if (c < u.cols)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot + ((k * V + v) * parts_of(sizeof(T)) + i) * step), "l"(row + c)
                       : "memory");
      }
  }
  // Both chunks of a row that is m bytes past a 16-byte boundary.
  __device__ __forceinline__ void take_shifted(Chunk8<T> (&r)[V], uint32_t slot, int k, uint32_t m, const RowUnit& u) const {
    uint32_t w[12], o[8];
#pragma unroll
    for (int i = 0; i < 12; ++i) w[i] = 0;
    if (u.t * 8 * V < u.cols)
#pragma unroll
      for (int i = 0; i < 3; ++i)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3])
                     : "r"(slot + (k * 3 + i) * step)
                     : "memory");
    shift_out<8>(o, w, m);
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i / 4].w[i % 4] = o[i];
  }
  __device__ __forceinline__ Chunk8<T> take(uint32_t slot, int k, int v, const RowUnit& u) const {
    Chunk8<T> r;
    r.zero();
#pragma unroll
    for (int i = 0; i < parts_of(sizeof(T)); ++i)
      if (col_of<E>(u, v, i * E) < u.cols)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r.w[4 * i]), "=r"(r.w[4 * i + 1]), "=r"(r.w[4 * i + 2]), "=r"(r.w[4 * i + 3])
                     : "r"(slot + ((k * V + v) * parts_of(sizeof(T)) + i) * step)
                     : "memory");
    return r;
  }
};

// Rows that are loaded directly: the whole 16-byte pieces of a coming one to L2.
template <typename T>
__device__ __forceinline__ void prefetch_row(const T* row, int cols) {
  const uintptr_t from = ((uintptr_t)row + 15) & ~(uintptr_t)15, to = (uintptr_t)(row + cols) & ~(uintptr_t)15;
  if (from < to)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"((uint32_t)(to - from)) : "memory");
}

__device__ __forceinline__ void commit_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_group() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <typename T>
constexpr int ring_depth(Access how) { return sizeof(T) == 4 ? 2 : how == kPieces ? 3 : 4; }
// Row sums (only of units of several warps), then two barriers; the ring after
// them starts on 128 bytes (16 further on, every access of it took two lines:
// norm_bwd 147 -> 158 us).
__host__ __device__ constexpr int red_bytes(int units, int tpr) { return (tpr > 32 ? 2 * units * 3 * kRedRow * 4 : 0) + 128; }

// Unit u of all takes rows [u n, (u + 1) n).  Units narrower than a warp stay
// together while any of them has rows.
template <typename T, bool VEC, int KIND>
__global__ void __launch_bounds__(kFwdThreads, 1) norm_fwd_rows_kernel(const NormFwdArgs a, int tpr, int clusters) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr Access kHow = VEC ? kChunks : kSingles;
  constexpr int kRing = ring_depth<T>(kHow), E = run_of<T>(kHow);
  const RowUnit u = row_unit(a.cols, tpr);
  const int units = blockDim.x / tpr;
  uint8_t* after = smem + red_bytes(units, tpr);
  RowSums sums;
  sums.init(reinterpret_cast<float*>(smem), reinterpret_cast<uint64_t*>(after - 128), clusters, units, a.err, a.timeout_ns);
  const Ring<T, 2, kHow> ring{ptx::smem_addr(after) + threadIdx.x * 16, blockDim.x * 16};
  const int64_t all = (int64_t)gridDim.x / clusters * units, id = (int64_t)(blockIdx.x / clusters) * units + u.unit;
  const int64_t per = (a.rows + all - 1) / all;
  const int row0 = (int)min(id * per, a.rows), row1 = (int)min(row0 + per, a.rows);
  const T* x = (const T*)a.x + row0 * a.ldx + u.col0;  // the row that is fetched next (VEC), or this one
  const T* f = (const T*)a.f + row0 * a.ldf + u.col0;
  T* y_out = (T*)a.y + row0 * a.ldy + u.col0;
  T* h_out = (T*)a.h + row0 * a.ldh + u.col0;
  int ahead = row0;
  auto fetch = [&](int s) {
    if (ahead < row1) {
      const uint32_t slot = ring.slot(s);
      ring.fetch(slot, 0, x, u);
      ring.fetch(slot, 1, f, u);
      x += a.ldx;
      f += a.ldf;
      ++ahead;
    }
    commit_group();
  };
  if constexpr (VEC)
    for (int s = 0; s < kRing; ++s) fetch(s);
  if constexpr (KIND == kCluster) ptx::cluster_sync();
  else __syncthreads();
  const float inv = 1.f / (float)a.cols;
  f2 pre[V][4], gw[V][4], res[V][4];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    load_param<E>(pre[v], a.pre_w, u, v);
    load_param<E>(gw[v], a.post_w, u, v);
    if (a.res) load_param<E>(res[v], a.res, u, v);
    else
#pragma unroll
      for (int i = 0; i < 4; ++i) res[v][i] = both(1.f);
  }
  int group_end = a.gate ? row0 : INT_MAX;  // first row past the gate row in gw
  int slot = 0;
  bool lost = false;
  const int last = KIND == kSub ? row0 + (int)per : row1;  // as often for every unit of a warp
  for (int row = row0; row < last; ++row) {
    const bool live = KIND != kSub || row < row1;
    if (live && row == group_end) {
      const int64_t group = row / a.per_gate;
      group_end = (int)min((group + 1) * a.per_gate, a.rows);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        f2 g[4];
        load_param<E>(g, a.gate + group * a.cols, u, v);
        load_param<E>(gw[v], a.post_w, u, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) gw[v][i] = mul2(gw[v][i], g[i]);
      }
    }
    Chunk8<T> xr[V], fr[V];
    if constexpr (VEC) {
      wait_group<kRing - 1>();
#pragma unroll
      for (int v = 0; v < V; ++v) {
        xr[v] = ring.take(ring.slot(slot), 0, v, u);  // a unit past its rows sums what its slots hold and stores nothing
        fr[v] = ring.take(ring.slot(slot), 1, v, u);
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        xr[v].zero();
        fr[v].zero();
        if (live) {
          xr[v] = load_direct<T>(x, u, v);
          fr[v] = load_direct<T>(f, u, v);
        }
      }
      x += a.ldx;
      f += a.ldf;
      if (row + 2 < row1 && u.t < 2) prefetch_row(u.t ? f + a.ldf : x + a.ldx, u.cols);
    }
    f2 q = 0;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) q = fma2(fr[v].pair(i), fr[v].pair(i), q);
    float s[1] = {add_up(q)};
    if (!row_sum<1, KIND>(s, u, sums)) { lost = true; break; }
    const float r1 = rsqrtf(fmaf(s[0], inv, a.eps));
    const f2 rr1 = both(r1);
    f2 y[V][4];
    q = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[v][i] = fma2(mul2(fr[v].pair(i), rr1), gw[v][i], mul2(xr[v].pair(i), res[v][i]));
        q = fma2(y[v][i], y[v][i], q);
      }
      if (live) store_chunk<T, E>(y_out, u, v, y[v]);
    }
    if constexpr (VEC) {
      fetch(slot);  // this thread has taken its slot
      if (++slot == kRing) slot = 0;
    }
    s[0] = add_up(q);
    if (!row_sum<1, KIND>(s, u, sums)) { lost = true; break; }
    const float r2 = rsqrtf(fmaf(s[0], inv, a.eps));
    const f2 rr2 = both(r2);
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int i = 0; i < 4; ++i) y[v][i] = mul2(mul2(y[v][i], rr2), pre[v][i]);
      if (live) store_chunk<T, E>(h_out, u, v, y[v]);
    }
    y_out += a.ldy;
    h_out += a.ldh;
    if (live && u.t == 0 && u.col0 == 0) {
      a.rstd[row] = r1;
      a.rstd[a.rows + row] = r2;
    }
  }
  if constexpr (KIND == kCluster) {
    if (lost) wait_group<0>();
    __syncwarp();
    ptx::cluster_sync();  // a peer may still send to this CTA's shared memory
    if (lost) land_sums(sums);
  }
}

// The rows of a unit, chunk after chunk (rows and chunks fit 31 bits).
struct ChunkRows {
  int all, chunk, row, end;
  __device__ __forceinline__ void open(const NormBwdArgs& a) {  // the first non-empty chunk from `chunk` on
    const int n = (int)(a.groups * a.chunks_per_group), cpg = (int)a.chunks_per_group;
    for (; chunk < n; chunk += all) {
      const int group = chunk / cpg, part = chunk - group * cpg;
      const int64_t r = group * a.per_gate + part * a.chunk_rows;
      const int64_t e = min(min(r + a.chunk_rows, (group + 1) * a.per_gate), a.rows);
      if (r < e) {
        row = (int)r;
        end = (int)e;
        return;
      }
    }
    chunk = INT_MAX;
  }
  __device__ __forceinline__ bool done() const { return chunk == INT_MAX; }
  __device__ __forceinline__ void next(const NormBwdArgs& a) {
    if (++row == end) {
      chunk += all;
      open(a);
    }
  }
};

template <typename T, bool VEC>
__host__ __device__ constexpr Access bwd_access() { return VEC ? kChunks : sizeof(T) == 2 ? kPieces : kSingles; }

// One row needs mean(dh w_pre yn) for t and then mean(g t w_post fn) for df;
// with t = dy + r2 (i - yn m2), i = dh w_pre, the second is
//   mean(g w fn (dy + r2 i)) - r2 m2 mean(g w fn yn)
// so that one round of three sums serves both (the rounding is that of t's own
// terms).  Units' column sums stay in registers over their rows, go to their
// own rows of the partial arrays and are added up, in a fixed order, by
// norm_bwd_sums_kernel.
// WHICH: 1 dy is given, 2 d_res is wanted; 4: asked at run time (the kinds of
// units for which a variant of its own gains less).
template <typename T, bool VEC, int KIND, int WHICH>
__global__ void __launch_bounds__(kBwdThreads, 1) norm_bwd_rows_kernel(const NormBwdArgs a, int tpr, int clusters) {
  const bool DY = WHICH == 4 ? a.dy != nullptr : (WHICH & 1) != 0;
  const bool X = WHICH == 4 ? a.d_res != nullptr : (WHICH & 2) != 0;
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr Access kHow = bwd_access<T, VEC>();
  constexpr int kRing = ring_depth<T>(kHow), E = run_of<T>(kHow);
  constexpr bool kHasRing = kHow != kSingles, kShifted = kHow == kPieces;
  const RowUnit u = row_unit(a.cols, tpr);
  const int units = blockDim.x / tpr;
  uint8_t* after = smem + red_bytes(units, tpr);
  RowSums sums;
  sums.init(reinterpret_cast<float*>(smem), reinterpret_cast<uint64_t*>(after - 128), clusters, units, a.err, a.timeout_ns);
  const Ring<T, 5, kHow> ring{ptx::smem_addr(after) + threadIdx.x * 16, blockDim.x * 16};
  const int64_t all = (int64_t)gridDim.x / clusters * units, id = (int64_t)(blockIdx.x / clusters) * units + u.unit;
  ChunkRows at{(int)all, (int)id, 0, 0};
  at.open(a);
  ChunkRows ahead = at;
  const T *f_dy = nullptr, *f_dh = nullptr, *f_y = nullptr, *f_f = nullptr, *f_x = nullptr;  // the row fetched next
  auto seek = [&]() {
    const int64_t row = ahead.row;
    if (DY) f_dy = (const T*)a.dy + row * a.lddy + u.col0;
    f_dh = (const T*)a.dh + row * a.lddh + u.col0;
    f_y = (const T*)a.y + row * a.ldy + u.col0;
    f_f = (const T*)a.f + row * a.ldf + u.col0;
    if (X) f_x = (const T*)a.x + row * a.ldx + u.col0;
  };
  if (!ahead.done()) seek();
  auto fetch = [&](int s) {
    if (!ahead.done()) {
      const uint32_t slot = ring.slot(s);
      if (DY) ring.fetch(slot, 0, f_dy, u);
      ring.fetch(slot, 1, f_dh, u);
      ring.fetch(slot, 2, f_y, u);
      ring.fetch(slot, 3, f_f, u);
      if (X) ring.fetch(slot, 4, f_x, u);
      const int was = ahead.chunk;
      ahead.next(a);
      if (ahead.chunk == was) {
        if (DY) f_dy += a.lddy;
        f_dh += a.lddh;
        f_y += a.ldy;
        f_f += a.ldf;
        if (X) f_x += a.ldx;
      } else if (!ahead.done()) {
        seek();
      }
    }
    commit_group();
  };
  if constexpr (kHasRing)
    for (int s = 0; s < kRing; ++s) fetch(s);
  if constexpr (KIND == kCluster) ptx::cluster_sync();
  else __syncthreads();
  f2 sum_pre[V][4], sum_res[V][4], sum_t[V][4];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 4; ++i) sum_pre[v][i] = sum_res[v][i] = sum_t[v][i] = 0;
  f2 pre[V][4], gw[V][4], res[V][4];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    load_param<E>(pre[v], a.pre_w, u, v);
    if (a.res) load_param<E>(res[v], a.res, u, v);
    else
#pragma unroll
      for (int i = 0; i < 4; ++i) res[v][i] = both(1.f);
  }
  const float inv = 1.f / (float)a.cols;
  float* part_post = a.part_post + id * a.part_ld;
  bool post_written = false;
  T *dx_row = nullptr, *df_row = nullptr;
  int chunk = -1;
  const float* gate = nullptr;
  int slot = 0;
  // t fn summed over a chunk belongs to one gate row.  The sum over a unit's
  // chunks is kept in its row of part_post.
  auto flush = [&]() {
    const int64_t group = chunk / (int)a.chunks_per_group;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      f2 w[4], o[4];
      if (a.gate) load_param<E>(w, gate, u, v);
      if (post_written) load_param<E>(o, part_post, u, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f2 g = a.gate ? w[i] : both(1.f);
        o[i] = post_written ? fma2(g, sum_t[v][i], o[i]) : mul2(g, sum_t[v][i]);
      }
      store_param<E>(part_post, u, v, o);
      if (a.d_gate) {
        if (a.chunks_per_group > 1) {
          store_param<E>(a.part_gate + (int64_t)chunk * a.part_ld, u, v, sum_t[v]);
        } else {
          load_param<E>(w, a.post_w, u, v);
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = mul2(w[i], sum_t[v][i]);
          store_param<E>(a.d_gate + group * a.cols, u, v, w);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) sum_t[v][i] = 0;
    }
    post_written = true;
  };
  bool lost = false;
  float n1 = 0.f, n2 = 0.f;
  if (!at.done()) {
    n1 = a.rstd[at.row];
    n2 = a.rstd[a.rows + at.row];
  }
  while (KIND == kSub ? __any_sync(0xffffffffu, !at.done()) : !at.done()) {  // as long as any unit of the warp has rows
    const bool live = KIND != kSub || !at.done();
    const int64_t row = at.row;
    const float r1 = n1, r2 = n2;
    if (live && at.chunk != chunk) {
      if (chunk >= 0) flush();
      chunk = at.chunk;
      dx_row = (T*)a.dx + row * a.lddx + u.col0;
      df_row = (T*)a.df + row * a.lddf + u.col0;
      if (a.gate) gate = a.gate + (int64_t)(chunk / (int)a.chunks_per_group) * a.cols;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        load_param<E>(gw[v], a.post_w, u, v);
        if (a.gate) {
          f2 g[4];
          load_param<E>(g, gate, u, v);
#pragma unroll
          for (int i = 0; i < 4; ++i) gw[v][i] = mul2(gw[v][i], g[i]);
        }
      }
    }
    if (live) at.next(a);
    if (!at.done()) {  // the next row's, before it is needed
      n1 = a.rstd[at.row];
      n2 = a.rstd[a.rows + at.row];
    }
    // Kept over the sums: yn, fn and q = dy + r2 dh w_pre, from which t is one operation.
    const f2 rr1 = both(r1), rr2 = both(r2);
    f2 yn[V][4], fn[V][4], q[V][4], s0 = 0, s1 = 0, s2 = 0;
    Chunk8<T> x[V];
    if constexpr (kHasRing) wait_group<kRing - 1>();
    const uint32_t from = ring.slot(slot);
    Chunk8<T> s_dy[V], s_dh[V], s_y[V], s_f[V];
    if constexpr (kShifted) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        s_dy[v].zero();
        s_dh[v].zero();
        s_y[v].zero();
        s_f[v].zero();
        x[v].zero();
      }
      if (live) {
        if (DY) ring.take_shifted(s_dy, from, 0, past16((const T*)a.dy + row * a.lddy + u.col0), u);
        ring.take_shifted(s_dh, from, 1, past16((const T*)a.dh + row * a.lddh + u.col0), u);
        ring.take_shifted(s_y, from, 2, past16((const T*)a.y + row * a.ldy + u.col0), u);
        ring.take_shifted(s_f, from, 3, past16((const T*)a.f + row * a.ldf + u.col0), u);
        if (X) ring.take_shifted(x, from, 4, past16((const T*)a.x + row * a.ldx + u.col0), u);
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      Chunk8<T> dy, dh, y, f;
      if constexpr (kShifted) {
        dy = s_dy[v];
        dh = s_dh[v];
        y = s_y[v];
        f = s_f[v];
      } else {
        dy.zero();
        dh.zero();
        y.zero();
        f.zero();
        x[v].zero();
        if (live) {
          if constexpr (VEC) {
            if (DY) dy = ring.take(from, 0, v, u);
            dh = ring.take(from, 1, v, u);
            y = ring.take(from, 2, v, u);
            f = ring.take(from, 3, v, u);
            if (X) x[v] = ring.take(from, 4, v, u);
          } else {
            if (DY) dy = load_direct<T>((const T*)a.dy + row * a.lddy + u.col0, u, v);
            dh = load_direct<T>((const T*)a.dh + row * a.lddh + u.col0, u, v);
            y = load_direct<T>((const T*)a.y + row * a.ldy + u.col0, u, v);
            f = load_direct<T>((const T*)a.f + row * a.ldf + u.col0, u, v);
            if (X) x[v] = load_direct<T>((const T*)a.x + row * a.ldx + u.col0, u, v);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f2 g = dh.pair(i), in = mul2(g, pre[v][i]);
        yn[v][i] = mul2(y.pair(i), rr2);
        fn[v][i] = mul2(f.pair(i), rr1);
        q[v][i] = fma2(rr2, in, dy.pair(i));
        const f2 b = mul2(gw[v][i], fn[v][i]);
        sum_pre[v][i] = fma2(g, yn[v][i], sum_pre[v][i]);
        s0 = fma2(in, yn[v][i], s0);
        s1 = fma2(b, q[v][i], s1);
        s2 = fma2(b, yn[v][i], s2);
      }
    }
    if constexpr (!kHasRing) {
      if (live && row + 2 < at.end) {  // the row after next, to L2
        if (DY && u.t == 0) prefetch_row((const T*)a.dy + (row + 2) * a.lddy + u.col0, u.cols);
        if (u.t == 1) prefetch_row((const T*)a.dh + (row + 2) * a.lddh + u.col0, u.cols);
        if (u.t == 2) prefetch_row((const T*)a.y + (row + 2) * a.ldy + u.col0, u.cols);
        if (u.t == 3) prefetch_row((const T*)a.f + (row + 2) * a.ldf + u.col0, u.cols);
        if (X && u.t == 4) prefetch_row((const T*)a.x + (row + 2) * a.ldx + u.col0, u.cols);
      }
    }
    float s[3] = {add_up(s0), add_up(s1), add_up(s2)};
    if (!row_sum<3, KIND>(s, u, sums)) { lost = true; break; }
    if constexpr (kHasRing) {
      fetch(slot);  // this thread has taken its slot
      if (++slot == kRing) slot = 0;
    }
    const float m2 = r2 * s[0] * inv, m1 = (s[1] - m2 * s[2]) * inv;
    const f2 nm2 = both(-m2), nm1 = both(-m1);
    f2 dx[V][4], df[V][4];
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f2 t = fma2(yn[v][i], nm2, q[v][i]);
        sum_t[v][i] = fma2(t, fn[v][i], sum_t[v][i]);
        if (X) sum_res[v][i] = fma2(t, x[v].pair(i), sum_res[v][i]);
        dx[v][i] = mul2(res[v][i], t);
        df[v][i] = mul2(rr1, fma2(fn[v][i], nm1, mul2(gw[v][i], t)));
      }
      if (!kShifted && live) {
        store_chunk<T, E>(dx_row, u, v, dx[v]);
        store_chunk<T, E>(df_row, u, v, df[v]);
      }
    }
    if constexpr (kShifted) {
      store_shifted(dx_row, u, dx, live);
      store_shifted(df_row, u, df, live);
    }
    dx_row += a.lddx;
    df_row += a.lddf;
  }
  if (chunk >= 0) flush();
  if (a.cta_units == 1) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!post_written) store_param<E>(part_post, u, v, sum_t[v]);  // no rows: zeros
      store_param<E>(a.part_pre + id * a.part_ld, u, v, sum_pre[v]);
      if (X) store_param<E>(a.part_res + id * a.part_ld, u, v, sum_res[v]);
    }
  } else {  // one row of sums a CTA, in its first unit's place: added up where the ring was
    float* fold = reinterpret_cast<float*>(after);  // [3][units][cols]
    const int n = (int)a.cols;
    if constexpr (kHasRing) wait_group<0>();
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) {
      f2 post[4];
      if (post_written) load_param<E>(post, part_post, u, v);
      store_param<E>(fold + u.unit * n, u, v, sum_pre[v]);
      store_param<E>(fold + (units + u.unit) * n, u, v, post_written ? post : sum_t[v]);
      if (X) store_param<E>(fold + (2 * units + u.unit) * n, u, v, sum_res[v]);
    }
    __syncthreads();
    const int64_t first = (id - u.unit) * a.part_ld;
    for (int c = threadIdx.x; c < (X ? 3 : 2) * n; c += blockDim.x) {
      const int k = c / n, col = c - k * n;
      float sum = 0.f;
      for (int i = 0; i < units; ++i) sum += fold[(k * units + i) * n + col];
      (k == 0 ? a.part_pre : k == 1 ? a.part_post : a.part_res)[first + col] = sum;
    }
  }
  if constexpr (KIND == kCluster) {
    if (lost) wait_group<0>();
    __syncwarp();
    ptx::cluster_sync();  // a peer may still send to this CTA's shared memory
    if (lost) land_sums(sums);
  }
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
  float* pre = a.part_pre + (int64_t)blockIdx.x * a.part_ld;
  float* post = a.part_post + (int64_t)blockIdx.x * a.part_ld;
  float* res = a.d_res ? a.part_res + (int64_t)blockIdx.x * a.part_ld : nullptr;
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
    float* own = a.d_gate ? (a.chunks_per_group > 1 ? a.part_gate + chunk * a.part_ld : a.d_gate + group * a.cols) : nullptr;
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

__device__ __forceinline__ void add4(float4& s, const float4& v) {
  s.x += v.x;
  s.y += v.y;
  s.z += v.z;
  s.w += v.w;
}

// Column sums over the units' partial rows (blockIdx.y: 0 pre, 1 post, 2 res)
// and, from 3 on, over the chunks of gate group blockIdx.y - 3: 32 columns a
// block, four a thread (the rows' pitch is whole 16 bytes), 32 rows at a time,
// eight loads in flight, then the 32 in a fixed order.  Groups of few chunks
// have a warp each and 128 columns: 30000 x 100 fp32, 1875 groups of two, 53 us
// in all where a block each took 67; 60000 x 64, 60 of 81 chunks, 43 with warps
// and 26 with blocks.  Launched as a programmatic dependent of the rows kernel,
// whose end is what starts it (nothing triggers it earlier): the gap between two
// launches is saved, and what it reads is there after the wait (an ordinary
// launch, eight rows at a time, 1.1 us more at 1000 x 1111).
__host__ __device__ __forceinline__ bool warp_a_group(const NormBwdArgs& a) { return a.chunks_per_group <= 16; }
__global__ void __launch_bounds__(256) norm_bwd_sums_kernel(const NormBwdArgs a) {
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, turn = threadIdx.x >> 3;
  // The last group may be short: its chunks past the rows are not written.
  auto chunks = [&](int64_t g) { return (int)((min(a.per_gate, a.rows - g * a.per_gate) + a.chunk_rows - 1) / a.chunk_rows); };
  if (blockIdx.y >= 3 && warp_a_group(a)) {
    const int64_t g = (int64_t)(blockIdx.y - 3) * 8 + warp, c = (int64_t)blockIdx.x * 128 + lane * 4;
    if (g >= a.groups || c >= a.cols) return;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int n = chunks(g);
    const float* src = a.part_gate + g * a.chunks_per_group * a.part_ld + c;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < n; i += 8) {
      float4 v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        v[k] = i + k < n ? *reinterpret_cast<const float4*>(src + (i + k) * a.part_ld) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 8; ++k) add4(s, v[k]);
    }
    const float t[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (c + k < a.cols) a.d_gate[g * a.cols + c + k] = t[k] * a.post_w[c + k];
    return;
  }
  const int64_t c0 = (int64_t)blockIdx.x * 32;
  const float* src;
  float* dst;
  int n = (int)(a.units / a.cta_units);
  int64_t step = a.cta_units * a.part_ld;  // a CTA's sums are in its first unit's row
  if (blockIdx.y == 0) { src = a.part_pre; dst = a.d_pre_w; }
  else if (blockIdx.y == 1) { src = a.part_post; dst = a.d_post_w; }
  else if (blockIdx.y == 2) { src = a.part_res; dst = a.d_res; }
  else {
    const int64_t g = blockIdx.y - 3;
    n = chunks(g);
    step = a.part_ld;
    src = a.part_gate + g * a.chunks_per_group * a.part_ld;
    dst = a.d_gate + g * a.cols;
  }
  if (!dst) return;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  const int64_t c4 = c0 + (threadIdx.x & 7) * 4;
  if (c4 < a.cols) {
    src += c4;
    for (int i = turn; i < n; i += 256) {
      float4 v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        v[k] = i + 32 * k < n ? *reinterpret_cast<const float4*>(src + (i + 32 * k) * step) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 8; ++k) add4(s, v[k]);
    }
  }
  float* mine = red[turn] + (threadIdx.x & 7) * 4;
  mine[0] = s.x;
  mine[1] = s.y;
  mine[2] = s.z;
  mine[3] = s.w;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t c = c0 + warp * 4 + k;
    float t = red[lane][warp * 4 + k];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (lane == 0 && c < a.cols) dst[c] = blockIdx.y >= 3 ? t * a.post_w[c] : t;
  }
}

// ------------------------------------------------------------ launches

// Threads of a unit, CTAs of a cluster, units of a CTA and CTAs of an SM for
// rows of `cols`, with `threads` on an SM.
struct RowShape {
  int tpr, clusters, units, resident;
};
RowShape row_shape(int64_t cols, int threads, int cta_threads) {
  RowShape r;
  const int64_t cta = (int64_t)threads * V * 8;
  r.clusters = cols <= cta ? 1 : cols <= 2 * cta ? 2 : cols <= 4 * cta ? 4 : kMaxCluster;
  const int lanes = (int)((cols + 8 * V * r.clusters - 1) / (8 * V * r.clusters));  // even shares of a cluster
  r.tpr = 8;  // rows of up to 128 columns
  while (r.tpr < lanes && r.tpr < 32) r.tpr *= 2;
  if (lanes > 32) r.tpr = (lanes + 31) / 32 * 32;
  r.units = r.clusters > 1 ? 1 : std::max(1, cta_threads / r.tpr);
  r.resident = std::max(1, threads / (r.tpr * r.units));
  return r;
}
RowShape fwd_shape(int64_t cols) { return row_shape(cols, kFwdThreads, 128); }
RowShape bwd_shape(int64_t cols) { return row_shape(cols, kBwdThreads, kBwdThreads); }
constexpr int64_t kHeld = 32768;  // longest rows held
static_assert(kMaxCluster * kBwdThreads * V * 8 >= kHeld && kMaxCluster * kFwdThreads * V * 8 >= kHeld, "held rows");

template <typename K, typename A>
cudaError_t launch_rows(K kernel, const A& a, const RowShape& r, int64_t ctas, int smem, cudaStream_t s) {
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
int ring_bytes(const RowShape& r, int arrays, Access how) {
  return red_bytes(r.units, r.tpr) + (how == kSingles ? 0 : ring_depth<T>(how) * arrays * row_parts<T>(how) * r.tpr * r.units * 16);
}

// Shared memory of a CTA: the ring, and in the backward where the ring was the
// sums of the CTA's units.
template <typename T, bool VEC>
int fwd_bytes(const RowShape& r) { return ring_bytes<T>(r, 2, VEC ? kChunks : kSingles); }
template <typename T, bool VEC>
int bwd_bytes(const RowShape& r, int64_t cols, bool fold) {
  return std::max(ring_bytes<T>(r, 5, bwd_access<T, VEC>()), red_bytes(r.units, r.tpr) + (fold ? 3 * r.units * (int)cols * 4 : 0));
}

// CTAs (clusters) of rows that are resident together.  How many clusters of
// four or more fit depends on how the device's SMs are grouped: it is asked
// once and kept (2048 x 16384 bf16 backward, clusters of four, a grid of SMs / 4
// of them took 204 us, the last ones alone; 126 with as many as fit).
int places(const RowShape& r, int sms, int* kept, bool backward) {
  if (r.clusters == 1) return std::max(1, sms * r.resident);
  int& n = kept[(backward ? 0 : 4) + (r.clusters == 2 ? 0 : r.clusters == 4 ? 1 : 2)];
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = r.clusters;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(sms / r.clusters * r.clusters, 1, 1);
    cfg.blockDim = dim3(backward ? kBwdThreads : kFwdThreads, 1, 1);  // the most: one CTA an SM
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const RowShape full{(int)cfg.blockDim.x, r.clusters, 1, 1};
    auto ask = [&](auto kernel, int arrays) {
      cfg.dynamicSmemBytes = ring_bytes<__nv_bfloat16>(full, arrays, kChunks);
      return cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
    };
    const cudaError_t e = backward ? ask(norm_bwd_rows_kernel<__nv_bfloat16, true, kCluster, 4>, 5)
                                   : ask(norm_fwd_rows_kernel<__nv_bfloat16, true, kCluster>, 2);
    if (e != cudaSuccess || n < 1) {
      cudaGetLastError();
      n = std::max(1, sms / r.clusters);
    }
  }
  return n;
}

template <typename T>
cudaError_t fwd(const NormFwdArgs& a, int sms, int* kept, cudaStream_t s) {
  if (a.cols > kHeld) {
    const int64_t grid = std::min(a.rows, (int64_t)sms * 8);
    norm_fwd_kernel<T><<<(unsigned)grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
  const RowShape r = fwd_shape(a.cols);
  const int64_t ctas = std::min((a.rows + r.units - 1) / r.units, (int64_t)places(r, sms, kept, false));
  const int smem = a.vec ? fwd_bytes<T, true>(r) : fwd_bytes<T, false>(r);
  auto go = [&](auto kernel) { return launch_rows(kernel, a, r, ctas, smem, s); };
  if (r.tpr < 32) return a.vec ? go(norm_fwd_rows_kernel<T, true, kSub>) : go(norm_fwd_rows_kernel<T, false, kSub>);
  if (r.clusters > 1) return a.vec ? go(norm_fwd_rows_kernel<T, true, kCluster>) : go(norm_fwd_rows_kernel<T, false, kCluster>);
  return a.vec ? go(norm_fwd_rows_kernel<T, true, kCta>) : go(norm_fwd_rows_kernel<T, false, kCta>);
}

template <typename T>
cudaError_t bwd(const NormBwdArgs& a, cudaStream_t s) {
  cudaError_t e;
  if (a.cols > kHeld) {
    norm_bwd_kernel<T><<<(unsigned)a.units, kThreads, 0, s>>>(a);
    e = cudaGetLastError();
  } else {
    const RowShape r = bwd_shape(a.cols);
    const int64_t ctas = a.units / r.units;
    const bool fold = a.cta_units > 1;
    const int smem = a.vec ? bwd_bytes<T, true>(r, a.cols, fold) : bwd_bytes<T, false>(r, a.cols, fold);
    auto go = [&](auto kernel) { return launch_rows(kernel, a, r, ctas, smem, s); };
    const bool dy = a.dy != nullptr, x = a.d_res != nullptr;
    auto pick = [&](auto vec) {
      constexpr bool kVec = decltype(vec)::value;
      if (r.tpr < 32) return go(norm_bwd_rows_kernel<T, kVec, kSub, 4>);
      if (r.clusters > 1) return go(norm_bwd_rows_kernel<T, kVec, kCluster, 4>);
      return dy ? (x ? go(norm_bwd_rows_kernel<T, kVec, kCta, 3>) : go(norm_bwd_rows_kernel<T, kVec, kCta, 1>))
                : (x ? go(norm_bwd_rows_kernel<T, kVec, kCta, 2>) : go(norm_bwd_rows_kernel<T, kVec, kCta, 0>));
    };
    e = a.vec ? pick(std::true_type()) : pick(std::false_type());
  }
  if (e != cudaSuccess) return e;
  const unsigned ys = 3 + (a.d_gate && a.chunks_per_group > 1 ? (unsigned)(warp_a_group(a) ? (a.groups + 7) / 8 : a.groups) : 0u);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)((a.cols + 31) / 32), ys, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_bwd_sums_kernel, a);
}

// The limit of dynamic shared memory belongs to the kernel on its device and not
// to a call or a handle: it is set once, to the most that any width of rows
// takes (widths of one shape end on a multiple of 16).
template <typename T, bool VEC>
cudaError_t configure() {
  int fwd_most = 0, bwd_most = 0;
  for (int64_t cols = 16; cols <= kHeld; cols += 16) {
    fwd_most = std::max(fwd_most, fwd_bytes<T, VEC>(fwd_shape(cols)));
    const RowShape r = bwd_shape(cols);
    bwd_most = std::max(bwd_most, bwd_bytes<T, VEC>(r, cols, r.units > 1));
  }
  cudaError_t e = cudaSuccess;
  auto set = [&](auto kernel, int bytes) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  };
  set(norm_fwd_rows_kernel<T, VEC, kSub>, fwd_most);
  set(norm_fwd_rows_kernel<T, VEC, kCta>, fwd_most);
  set(norm_fwd_rows_kernel<T, VEC, kCluster>, fwd_most);
  set(norm_bwd_rows_kernel<T, VEC, kSub, 4>, bwd_most);
  set(norm_bwd_rows_kernel<T, VEC, kCta, 0>, bwd_most);
  set(norm_bwd_rows_kernel<T, VEC, kCta, 1>, bwd_most);
  set(norm_bwd_rows_kernel<T, VEC, kCta, 2>, bwd_most);
  set(norm_bwd_rows_kernel<T, VEC, kCta, 3>, bwd_most);
  set(norm_bwd_rows_kernel<T, VEC, kCluster, 4>, bwd_most);
  return e;
}

}  // namespace

cudaError_t block_norm_configure() {
  for (auto one : {configure<float, true>, configure<float, false>, configure<__nv_bfloat16, true>, configure<__nv_bfloat16, false>,
                   configure<__half, true>, configure<__half, false>}) {
    const cudaError_t e = one();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// Units whose sums a CTA adds up itself: its own where there are many units in
// all (fewer are added up sooner by norm_bwd_sums_kernel alone: 3 us at two a CTA).
int norm_bwd_cta_units(int64_t cols, int64_t units) { return cols > kHeld || units <= 512 ? 1 : bwd_shape(cols).units; }

// As many units as are resident, no more than rows.
int64_t norm_bwd_units(int64_t rows, int64_t cols, int sms, int* kept) {
  if (cols > kHeld) return std::min<int64_t>(std::max<int64_t>(rows, 1), (int64_t)sms * 4);
  const RowShape r = bwd_shape(cols);
  const int64_t ctas = std::min<int64_t>(places(r, sms, kept, true), (std::max<int64_t>(rows, 1) + r.units - 1) / r.units);
  return ctas * r.units;
}

cudaError_t launch_norm_fwd(const NormFwdArgs& a, int dtype, int sms, int* kept, cudaStream_t s) {
  if (dtype == DMUON_BF16) return fwd<__nv_bfloat16>(a, sms, kept, s);
  if (dtype == DMUON_F16) return fwd<__half>(a, sms, kept, s);
  return fwd<float>(a, sms, kept, s);
}

cudaError_t launch_norm_bwd(const NormBwdArgs& a, int dtype, cudaStream_t s) {
  if (dtype == DMUON_BF16) return bwd<__nv_bfloat16>(a, s);
  if (dtype == DMUON_F16) return bwd<__half>(a, s);
  return bwd<float>(a, s);
}

}  // namespace dmuon
