// Residual norm with dropout on the branch (formulas in add_norm.cuh).
// Everything is computed in fp32; y, h, dx and df are rounded once to the
// activations' type, and h and its MXFP8 codes come from y before it is rounded.
//
// A row is held by a unit of threads, V chunks of eight columns a thread, so that
// it is read once: part of a warp up to 256 columns, a warp up to 512, a CTA of as
// many warps as it takes up to 16384.  A unit goes from row to row
// with its columns' weights (and, backward, their sums) in registers; the coming
// rows are on their way to a ring in shared memory (cp.async: no registers), each
// warp's part its own, so that only the row's sums meet at a barrier.  Longer rows
// are read in two passes by one CTA (add_norm_long_*).
// A block of 32 columns is four lanes (two of 16 columns), so its scale byte takes
// two exchanges or one.
#include <algorithm>

#include "../../include/dmuon.h"
#include "add_norm.cuh"
#include "chunk8.cuh"
#include "mx.cuh"
#include "mx8.cuh"
#include "ptx.cuh"

namespace dmuon {

namespace {

constexpr int kLongThreads = 512;
constexpr int kMost = 16384;  // columns that a unit holds

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

// Sums over a unit, to all of it.  A chunk's eight products are added up by its lane,
// then chunks pairwise by the bits of their number, from the lowest: the order
// does not depend on which lane has which chunk, nor on the type.  N sums a lane
// are those of chunks that lie a unit's threads apart, so each is a sum of 32
// chunks when it leaves its warp.
// Consecutive calls of a CTA alternate between the halves of `red`: one is written
// again only after the next call's barrier, when every thread has read it.  What no
// warp writes is zero (clear_sums, ahead of the first call's barrier).
constexpr int kSums = 64;  // of a half: 16 warps, up to four each
__device__ __forceinline__ void clear_sums(float* red, int sums) {
  for (int i = threadIdx.x; i < 2 * kSums; i += blockDim.x)
    if (i % kSums >= sums * ((int)blockDim.x / 32)) red[i] = 0.f;
}
template <int N>
__device__ __forceinline__ float pairwise(const float (&v)[N]) {
  if constexpr (N == 1) return v[0];
  else if constexpr (N == 2) return v[0] + v[1];
  else return (v[0] + v[1]) + (v[2] + v[3]);
}
__device__ __forceinline__ float sum16(const float* p) {
  float s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 q = reinterpret_cast<const float4*>(p)[i];
    s[i] = (q.x + q.y) + (q.z + q.w);
  }
  return pairwise(s);
}
template <bool MULTI, int N>
__device__ __forceinline__ float unit_sum(float (&v)[N], const Unit& u, float* red, uint32_t& calls) {
#pragma unroll
  for (int o = 1; o < 32; o *= 2)
    if (MULTI || o < u.tpr)
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if constexpr (!MULTI) return pairwise(v);
  float* mine = red + (calls++ & 1) * kSums;
  const int warps = blockDim.x >> 5;
  if (u.lane == 0)
#pragma unroll
    for (int k = 0; k < N; ++k) mine[k * warps + u.warp] = v[k];
  __syncthreads();
  float s = sum16(mine);
  if (N * warps > 16) {
    s += sum16(mine + 16);
    if (N * warps > 32) s += sum16(mine + 32) + sum16(mine + 48);
  }
  return s;
}

// Scale bytes past the matrix are zero: rows from `rows` to the last tile's end, a
// warp of the grid a tile (a lane has the 16 bytes of rows lane, lane + 32, ..);
// blocks past a row's last, with the row.
__device__ __forceinline__ void zero_rows_behind(uint8_t* scales, int64_t rows, int64_t cols) {
  const int left = (int)(rows & 127), lane = threadIdx.x & 31;  // rows of the last tile
  if (left == 0) return;
  const int64_t kt = mx_scale_cols(cols), warps = (int64_t)gridDim.x * (blockDim.x >> 5);
  uint8_t* last = scales + (rows >> 7) * kt * kMxScaleTile + lane * 16;
  for (int64_t i = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); i < kt; i += warps) {
    uint8_t* p = last + i * kMxScaleTile;
    if (lane >= left) {
      *reinterpret_cast<uint4*>(p) = make_uint4(0, 0, 0, 0);
      continue;
    }
#pragma unroll
    for (int q = 1; q < 4; ++q)
      if (lane + 32 * q >= left) *reinterpret_cast<uint32_t*>(p + 4 * q) = 0u;
  }
}
__device__ __forceinline__ uint8_t* scale_at(uint8_t* scales, int64_t row, int64_t blk, int64_t cols) {
  return scales + ((row >> 7) * mx_scale_cols(cols) + (blk >> 2)) * kMxScaleTile + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (blk & 3);
}

// 8 C consecutive values of a row, from column col on, to codes; a warp's lanes
// together, 4 / C consecutive ones a block.
template <int C>
__device__ __forceinline__ void quantise(const AddNormFwdArgs& a, const float (&h)[C][8], int64_t row, int col, bool live) {
  float m = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) m = mx8::max_abs(m, mx8::max_abs(h[c]), 0.f);
  uint32_t key = mx8::keys2(m, m, a.up);
#pragma unroll
  for (int o = 1; o < 4 / C; o *= 2) key = mx8::max_halves(key, __shfl_xor_sync(0xffffffffu, key, o));
  uint32_t bad = 0;  // the block holds Inf or NaN
  if (__any_sync(0xffffffffu, mx8::may_not_be_finite(key))) {
    bad = mx8::not_finite(m);
#pragma unroll
    for (int o = 1; o < 4 / C; o *= 2) bad |= __shfl_xor_sync(0xffffffffu, bad, o);
  }
  if (!live || col >= (int)mx_blocks(a.cols) * kMxBlock) return;
  const uint32_t ex = mx8::exponents2(key);
  const float inv = mx8::factors2(ex).y;
  uint32_t w[2 * C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    w[2 * c] = mx8::codes4(h[c][0] * inv, h[c][1] * inv, h[c][2] * inv, h[c][3] * inv);
    w[2 * c + 1] = mx8::codes4(h[c][4] * inv, h[c][5] * inv, h[c][6] * inv, h[c][7] * inv);
  }
  if (bad)
#pragma unroll
    for (int i = 0; i < 2 * C; ++i) w[i] = 0;
  uint8_t* q = a.q + row * mx_pitch(a.cols, 8) + col;
  if constexpr (C == 1) *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
  else
#pragma unroll
    for (int i = 0; i < 2 * C; i += 4) reinterpret_cast<uint4*>(q)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
  if ((col & 31) == 0) *scale_at(a.q_scales, row, col >> 5, a.cols) = bad ? 255 : (uint8_t)mx8::byte_of(ex, 1);
}
__device__ __forceinline__ void quantise8(const AddNormFwdArgs& a, const float (&h)[8], int64_t row, int col, bool live) {
  quantise<1>(a, reinterpret_cast<const float (&)[1][8]>(h), row, col, live);
}
__device__ __forceinline__ void zero_blocks_behind(const AddNormFwdArgs& a, int64_t row, int t, bool live) {
  const int64_t nb = mx_blocks(a.cols);
  if (live && t < mx_scale_cols(a.cols) * 4 - nb) *scale_at(a.q_scales, row, nb + t, a.cols) = 0;
}

// Rows on their way, as shared memory has room for them.
template <typename T, int V>
constexpr int depth() { return (sizeof(T) == 4 ? 2 : 3) - (V == 4 ? 1 : 0); }

// The ring of a warp: DEPTH slots of ARRAYS x RUNS runs.  A run is the 16-byte pieces
// that C chunks of each of a unit's lanes of this warp lie in, one after the other
// (rows on any element: one piece more), copied by those lanes piece by piece.
template <typename T, bool VEC, int UNITS, int RUNS, int C, int ARRAYS, int DEPTH>  // UNITS of a warp at most
struct Ring {
  static constexpr int W = C * words8<T>() / 4;                  // pieces of a lane
  static constexpr int kRun = (32 * W + (VEC ? 0 : UNITS)) * 16; // bytes
  static constexpr int kSlot = ARRAYS * RUNS * kRun;
  static constexpr int kWarp = DEPTH * kSlot;
  const uint8_t* mine;     // this lane's first piece in slot 0
  uint32_t copies;         // where it copies its first piece to
  int lanes, l;            // of its unit in this warp; its place among them
  __device__ __forceinline__ Ring(uint8_t* smem, const Unit& u) {
    lanes = u.tpr < 32 ? u.tpr : 32;
    l = u.lane & (lanes - 1);
    const int run = u.lane / lanes * (lanes * W + (VEC ? 0 : 1)) * 16;
    uint8_t* warp = smem + u.warp * kWarp;
    mine = warp + run + l * W * 16;
    copies = ptx::smem_addr(warp + run + l * 16);
  }
  // Run (array, r) of the slot at `slot` bytes: p its first element (of the unit's
  // first lane in this warp), left the elements of the row from there on (none:
  // below 1), inside an address of the matrix.
  __device__ __forceinline__ void fetch(int slot, int array, int r, const uint8_t* p, int left, const void* inside) const {
    const uint32_t dst = copies + slot + (array * RUNS + r) * kRun;
    const uint32_t m = VEC ? 0u : past16(p);
    const uint8_t* from = p - m + l * 16;
    if (left >= lanes * 8 * C) {
#pragma unroll
      for (int k = 0; k < W; ++k) copy16(dst + k * lanes * 16, from + k * lanes * 16);
      if (!VEC && l == 0) copy16(dst + W * lanes * 16, m ? from + W * lanes * 16 : from, (int)m);
      return;
    }
    const int bytes = left > 0 ? min(left, lanes * 8 * C) * (int)sizeof(T) + (int)m : 0;
    const uint8_t* other = reinterpret_cast<const uint8_t*>(inside) - past16(reinterpret_cast<const uint8_t*>(inside));
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const int at = (k * lanes + l) * 16, n = max(0, min(16, bytes - at));
      copy16(dst + k * lanes * 16, n ? from + k * lanes * 16 : other, n);
    }
    if (!VEC && l == 0) {
      const int n = max(0, min(16, bytes - W * lanes * 16));
      copy16(dst + W * lanes * 16, n ? from + W * lanes * 16 : other, n);
    }
  }
  // Chunk v of the lane: of run v, or the vth of the one run.
  __device__ __forceinline__ void take(f2 (&f)[4], int slot, int array, int v, uint32_t m) const {
    take8<T, VEC, true>(f, mine + slot + (array * RUNS + v / C) * kRun + v % C * (W / C * 16), m);
  }
};
// How a thread's V chunks lie: one after the other where a row has warps of its own
// and 16-bit elements (one run; 32 bytes a lane, and on any element half the shifting
// and half the ends: 16384 x 4095 bf16 forward 164 -> 140 us, backward 212 -> 176), a
// unit's threads apart otherwise (V runs; fp32 on any element 1371 x 6082 backward
// 48 us so, 57 one after the other; four chunks one after the other meet in the
// banks of shared memory, 2048 x 16384 bf16 forward 57 us against 47).
template <typename T, bool MULTI, int V>
constexpr bool wide() { return MULTI && sizeof(T) == 2 && V == 2; }
template <typename T, bool VEC, bool MULTI, int V, int ARRAYS, int DEPTH>
using RingOf = Ring<T, VEC, MULTI ? 1 : 8, wide<T, MULTI, V>() ? 1 : V, wide<T, MULTI, V>() ? V : 1, ARRAYS, DEPTH>;

// The rows of one matrix that a unit goes through: the run that its warp fetches
// next, and how far a row's first byte is past a 16-byte boundary.
template <typename T, bool VEC>
struct Rows {
  const uint8_t* next;
  int64_t step;         // bytes from one row of the unit to its next
  const void* inside;
  uint32_t first, ld;   // modulo 16
  __device__ __forceinline__ Rows(const void* base, int64_t ld_, int64_t row, int64_t rows_on, int64_t col) {
    next = (const uint8_t*)base + (row * ld_ + col) * (int)sizeof(T);
    step = rows_on * ld_ * (int)sizeof(T);
    inside = base;
    first = (uint32_t)(uintptr_t)base;
    ld = (uint32_t)ld_ * (uint32_t)sizeof(T);
  }
  // Of any chunk of the row: chunks are 16 or 32 bytes.
  __device__ __forceinline__ uint32_t past(int64_t row) const { return VEC ? 0u : (first + (uint32_t)row * ld) & 15u; }
};

__device__ __forceinline__ void unpack8(float (&o)[8], const f2 (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack2(f[i]);
    o[2 * i] = p.x;
    o[2 * i + 1] = p.y;
  }
}
// A row's chunks of a thread; next_run as in the kernels, n: columns from each chunk on.
template <typename T, bool VEC, bool MULTI, int V>
__device__ __forceinline__ void store_chunks(T* p, int next_run, const f2 (&f)[V][4], const int (&n)[V], const Unit& u, bool live) {
  if constexpr (wide<T, MULTI, V>()) {
    store_wide<T, VEC, V>(p, f, n[0]);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float o[8];
      unpack8(o, f[v]);
      store8_warp<T, VEC, MULTI>(p + v * next_run, o, n[v], u.first, u.last, live);
    }
  }
}
__device__ __forceinline__ void load_weights(f2 (&w)[4], const float* p, int n, bool vec) {
  float f[8];
  if (vec) load8<float, true>(f, p, n);
  else load8<float, false>(f, p, n);
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack2(f[2 * i], f[2 * i + 1]);
}

// kThreads: of a CTA at most; kCtas: of them on an SM.
template <typename T, bool VEC, int V, int kThreads, int kCtas, bool MULTI>
__global__ void __launch_bounds__(kThreads, kCtas) add_norm_fwd_kernel(const AddNormFwdArgs a, int tpr) {
  constexpr int D = depth<T, V>();
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) float red[2 * kSums];
  const Unit u(tpr, MULTI);
  constexpr bool kWide = wide<T, MULTI, V>();
  constexpr int kRuns = kWide ? 1 : V, kApart = kWide || !MULTI ? 1 : V;
  const RingOf<T, VEC, MULTI, V, 2, D> ring(smem, u);
  auto col = [&](int v) { return kWide ? (u.t * V + v) * 8 : (v * tpr + u.t) * 8; };
  uint32_t calls = 0;
  const int64_t step = (int64_t)gridDim.x * u.units;
  int64_t row = (int64_t)blockIdx.x * u.units + u.unit, ahead = row;
  int n[V];
  f2 w[V][4];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = col(v);
    n[v] = (int)a.cols - c;
    load_weights(w[v], a.w + c, n[v], VEC);
  }
  const int run0 = col(0) - ring.l * (kWide ? 8 * V : 8), next_run = tpr * 8;  // columns of the warp's first run, and from there to the next
  Rows<T, VEC> x(a.x, a.ldx, row, step, run0), f(a.f, a.ldf, row, step, run0);
  int fetch_slot = 0;
  auto fetch = [&]() {
    const int cols = ahead < a.rows ? (int)a.cols - run0 : 0;
#pragma unroll
    for (int v = 0; v < kRuns; ++v) {
      const int64_t off = (int64_t)(v * next_run) * (int)sizeof(T);
      ring.fetch(fetch_slot, 0, v, f.next + off, cols - v * next_run, f.inside);
      if (a.x) ring.fetch(fetch_slot, 1, v, x.next + off, cols - v * next_run, x.inside);
    }
    f.next += f.step;
    x.next += x.step;
    ahead += step;
    if ((fetch_slot += ring.kSlot) == ring.kWarp) fetch_slot = 0;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int s = 0; s < D; ++s) fetch();
  if (a.q) zero_rows_behind(a.q_scales, a.rows, a.cols);
  clear_sums(red, kApart);
  const float inv = 1.f / (float)a.cols;
  T* y_out = (T*)a.y + row * a.ldy + col(0);
  T* h_out = (T*)a.h + row * a.ldh + col(0);
  const int64_t y_step = step * a.ldy, h_step = step * a.ldh;
  int slot = 0;
  for (int64_t base = (int64_t)blockIdx.x * u.units; base < a.rows; base += step, row += step) {  // as often for every unit
    const bool live = MULTI || row < a.rows;
    f2 y[V][4];
    float s[V];
    uint32_t bits[V][4];
    if (a.drop.cut) {
#pragma unroll
      for (int v = 0; v < V; ++v) philox(bits[v], a.drop, (uint32_t)(col(v) >> 3), (uint32_t)row);
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory");
    __syncwarp();
#pragma unroll
    for (int v = 0; v < V; ++v) {
      ring.take(y[v], slot, 0, v, f.past(row));
      if (a.drop.cut) drop8(y[v], a.drop, bits[v]);
      if (a.x) {
        f2 more[4];
        ring.take(more, slot, 1, v, x.past(row));
#pragma unroll
        for (int i = 0; i < 4; ++i) y[v][i] = add2(y[v][i], more[i]);
      }
      f2 square = mul2(y[v][0], y[v][0]);
#pragma unroll
      for (int i = 1; i < 4; ++i) square = fma2(y[v][i], y[v][i], square);
      s[v] = add_up(square);
    }
    __syncwarp();
    fetch();
    if ((slot += ring.kSlot) == ring.kWarp) slot = 0;
    store_chunks<T, VEC, MULTI>(y_out, next_run, y, n, u, live);
    y_out += y_step;
    float total[kApart];
    if constexpr (kApart == 1) total[0] = pairwise(s);
    else
#pragma unroll
      for (int v = 0; v < V; ++v) total[v] = s[v];
    const float r = rsqrtf(fmaf(unit_sum<MULTI>(total, u, red, calls), inv, a.eps));
    if (live && u.t == 0) a.rstd[row] = r;
    const f2 rr = both(r);
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) y[v][i] = mul2(mul2(y[v][i], rr), w[v][i]);
    if (a.h) store_chunks<T, VEC, MULTI>(h_out, next_run, y, n, u, live);
    if (a.q) {
      float o[V][8];
#pragma unroll
      for (int v = 0; v < V; ++v) unpack8(o[v], y[v]);
      if constexpr (kWide) {
        quantise<V>(a, o, row, col(0), live);
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) quantise8(a, o[v], row, col(v), live);
      }
    }
    h_out += h_step;
    if (a.q) zero_blocks_behind(a, row, u.t, live);
  }
}

// A thread's sum over the panels of a long row, with what its additions lose beside it
// (Knuth, The Art of Computer Programming 2, 4.2.2: exact): thousands of like terms
// fall the same way, and 1 / rms of 4M values of 0.3 was off by 3.3e-5 without.
struct PanelSum {
  float s = 0.f, lost = 0.f;
  __device__ __forceinline__ void add(float v) {
    const float t = s + v, b = t - s;
    lost += (s - (t - b)) + (v - b);
    s = t;
  }
  __device__ __forceinline__ float total() const {  // Inf and NaN stay
    const float t = s + lost;
    return t == t ? t : s;
  }
};

template <typename T, bool VEC>
__global__ void __launch_bounds__(kLongThreads) add_norm_long_fwd_kernel(const AddNormFwdArgs a) {
  __shared__ __align__(16) float red[2 * kSums];
  const Unit u(kLongThreads, true);
  clear_sums(red, 1);
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
    PanelSum sum;
    float y[8];
#pragma unroll 4
    for (int64_t p = 0; p < panels; ++p) {
      const int64_t c = (p * kLongThreads + threadIdx.x) * 8;
      sum_at(y, c);
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) s = fmaf(y[e], y[e], s);
      sum.add(s);
      store8_warp<T, VEC, true>((T*)a.y + row * a.ldy + c, y, a.cols - c, u.first, u.last, true);
    }
    float one[1] = {sum.total()};
    const float s = unit_sum<true>(one, u, red, calls);
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
      if (a.h) store8_warp<T, VEC, true>((T*)a.h + row * a.ldh + c, y, a.cols - c, u.first, u.last, true);
      if (a.q) quantise8(a, y, row, (int)c, true);
    }
    if (a.q) zero_blocks_behind(a, row, u.t, true);
  }
}

// The backward knows a row by yn = y r alone, which is of size one whatever y's size:
// r^2 or r^3 by itself leaves fp32's range for rows that y, r and the gradients are
// well inside of (r^3 below 2^-126 from a row of size 5e12 on, above 2^127 below 1e-13).

template <typename T, bool VEC, int V, int kThreads, int kCtas, bool MULTI>
__global__ void __launch_bounds__(kThreads, kCtas) add_norm_bwd_kernel(const AddNormBwdArgs a, int tpr) {
  constexpr int D = depth<T, V>();
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) float red[2 * kSums];
  __shared__ float lines[MULTI ? 1 : 32 * V * 8];
  const Unit u(tpr, MULTI);
  constexpr bool kWide = wide<T, MULTI, V>();
  constexpr int kRuns = kWide ? 1 : V, kApart = kWide || !MULTI ? 1 : V;
  const RingOf<T, VEC, MULTI, V, 3, D> ring(smem, u);
  auto col = [&](int v) { return kWide ? (u.t * V + v) * 8 : (v * tpr + u.t) * 8; };
  uint32_t calls = 0;
  const int64_t step = (int64_t)gridDim.x * u.units;
  int64_t row = (int64_t)blockIdx.x * u.units + u.unit, ahead = row;
  int n[V];
  // 32 columns a thread leave no registers for the weights and for the row's values
  // beside their sums: they are read where they are used, the values twice.
  constexpr bool kReread = V == 4;
  f2 w[kReread ? 1 : V][4], sums[V][4];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = col(v);
    n[v] = (int)a.cols - c;
    if constexpr (!kReread) load_weights(w[v], a.w + c, n[v], VEC);
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[v][i] = 0;
  }
  const int run0 = col(0) - ring.l * (kWide ? 8 * V : 8), next_run = tpr * 8;  // columns of the warp's first run, and from there to the next
  Rows<T, VEC> dy(a.dy, a.lddy, row, step, run0), dh(a.dh, a.lddh, row, step, run0), y(a.y, a.ldy, row, step, run0);
  int fetch_slot = 0;
  auto fetch = [&]() {
    const int cols = ahead < a.rows ? (int)a.cols - run0 : 0;
#pragma unroll
    for (int v = 0; v < kRuns; ++v) {
      const int64_t off = (int64_t)(v * next_run) * (int)sizeof(T);
      ring.fetch(fetch_slot, 0, v, dh.next + off, cols - v * next_run, dh.inside);
      ring.fetch(fetch_slot, 1, v, y.next + off, cols - v * next_run, y.inside);
      if (a.dy) ring.fetch(fetch_slot, 2, v, dy.next + off, cols - v * next_run, dy.inside);
    }
    dh.next += dh.step;
    y.next += y.step;
    dy.next += dy.step;
    ahead += step;
    if ((fetch_slot += ring.kSlot) == ring.kWarp) fetch_slot = 0;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int s = 0; s < D; ++s) fetch();
  clear_sums(red, kApart);
  const float inv = 1.f / (float)a.cols;
  float next_r = row < a.rows ? a.rstd[row] : 0.f;
  T* dx_out = (T*)a.dx + row * a.lddx + col(0);
  T* df_out = (T*)a.df + row * a.lddf + col(0);
  const int64_t dx_step = step * a.lddx, df_step = step * a.lddf;
  int slot = 0;
  for (int64_t base = (int64_t)blockIdx.x * u.units; base < a.rows; base += step, row += step) {
    const bool live = MULTI || row < a.rows;
    const float r = next_r;
    next_r = row + step < a.rows ? a.rstd[row + step] : 0.f;
    float s[V], total[kApart];
    asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory");
    __syncwarp();
    f2 dv[V][4];
    f2 (&t)[V][4] = dv;
    auto sum = [&]() {  // minus the mean of dh w yn over the row
      if constexpr (kApart == 1) total[0] = pairwise(s);
      else
#pragma unroll
        for (int v = 0; v < V; ++v) total[v] = s[v];
      return both(-(unit_sum<MULTI>(total, u, red, calls) * inv));
    };
    const f2 rr = both(r);
    // y to yn and dh to dh w.
    auto normalise = [&](f2 (&g)[4], f2 (&yn)[4], const f2 (&weight)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        yn[i] = mul2(yn[i], rr);
        g[i] = mul2(g[i], weight[i]);
      }
    };
    // The same, with the row's share of the column sums; the sum of dh w yn.
    auto product = [&](int v, f2 (&g)[4], f2 (&yn)[4], const f2 (&weight)[4]) {
      f2 d[4], p;
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = g[i];
      normalise(g, yn, weight);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sums[v][i] = fma2(d[i], yn[i], sums[v][i]);
        p = i ? fma2(g[i], yn[i], p) : mul2(g[i], yn[i]);
      }
      return add_up(p);
    };
    auto take_dy = [&](int v) {
      if (a.dy) ring.take(dv[v], slot, 2, v, dy.past(row));
      else
#pragma unroll
        for (int i = 0; i < 4; ++i) dv[v][i] = 0;
    };
    auto into_t = [&](int v, const f2 (&g)[4], const f2 (&yn)[4], f2 back) {
#pragma unroll
      for (int i = 0; i < 4; ++i) t[v][i] = fma2(rr, fma2(back, yn[i], g[i]), dv[v][i]);
    };
    if constexpr (!kReread) {
      f2 gv[V][4], yv[V][4];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        ring.take(gv[v], slot, 0, v, dh.past(row));
        ring.take(yv[v], slot, 1, v, y.past(row));
        s[v] = product(v, gv[v], yv[v], w[v]);
      }
#pragma unroll
      for (int v = 0; v < V; ++v) take_dy(v);  // last: before the products 16384 x 4096 bf16 takes 106 us, so 103
      __syncwarp();
      fetch();
      const f2 back = sum();
#pragma unroll
      for (int v = 0; v < V; ++v) into_t(v, gv[v], yv[v], back);
    } else {
      f2 g[4], yv[4], weight[4];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        ring.take(g, slot, 0, v, dh.past(row));
        ring.take(yv, slot, 1, v, y.past(row));
        load_weights(weight, a.w + col(v), n[v], VEC);
        s[v] = product(v, g, yv, weight);
      }
      const f2 back = sum();
#pragma unroll
      for (int v = 0; v < V; ++v) {
        ring.take(g, slot, 0, v, dh.past(row));
        ring.take(yv, slot, 1, v, y.past(row));
        take_dy(v);
        load_weights(weight, a.w + col(v), n[v], VEC);
        normalise(g, yv, weight);
        into_t(v, g, yv, back);
      }
      __syncwarp();
      fetch();
    }
    if ((slot += ring.kSlot) == ring.kWarp) slot = 0;
    if (a.dx) store_chunks<T, VEC, MULTI>(dx_out, next_run, t, n, u, live);
    if (a.drop.cut) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        uint32_t bits[4];
        philox(bits, a.drop, (uint32_t)(col(v) >> 3), (uint32_t)row);
        drop8(t[v], a.drop, bits);
      }
    }
    store_chunks<T, VEC, MULTI>(df_out, next_run, t, n, u, live);
    dx_out += dx_step;
    df_out += df_step;
  }
  float* out = a.parts + (int64_t)blockIdx.x * a.part_ld;
  if constexpr (MULTI) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float o[8];
      unpack8(o, sums[v]);
      if (((uintptr_t)out & 15) == 0) store8<float>(out + col(v), o, n[v]);
      else
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e < n[v]) out[col(v) + e] = o[e];
    }
  } else {  // the units of a warp, then the warps, one after the other
    float o[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) unpack8(o[v], sums[v]);
    for (int k = tpr; k < 32; k *= 2)
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) o[v][e] += __shfl_xor_sync(0xffffffffu, o[v][e], k);
    for (int k = 0; k < (int)blockDim.x >> 5; ++k) {
      if (u.warp == k && u.lane < tpr)
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int c = col(v) + e;
            lines[c] = k ? lines[c] + o[v][e] : o[v][e];
          }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < (int)a.cols; c += blockDim.x) out[c] = lines[c];
  }
}

// The column sums of long rows are kept in the CTA's row of parts.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kLongThreads) add_norm_long_bwd_kernel(const AddNormBwdArgs a) {
  __shared__ __align__(16) float red[2 * kSums];
  const Unit u(kLongThreads, true);
  clear_sums(red, 1);
  uint32_t calls = 0;
  const int64_t panels = (a.cols + kLongThreads * 8 - 1) / (kLongThreads * 8);
  float* out = a.parts + (int64_t)blockIdx.x * a.part_ld;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float r = a.rstd[row];
    PanelSum sum;
    float dh[8], yn[8], w[8];
    auto load = [&](int64_t c, int n) {
      load8<T, VEC>(dh, (const T*)a.dh + row * a.lddh + c, n);
      load8<T, VEC>(yn, (const T*)a.y + row * a.ldy + c, n);
      load8<float, VEC>(w, a.w + c, n);
#pragma unroll
      for (int e = 0; e < 8; ++e) yn[e] *= r;
    };
#pragma unroll 4
    for (int64_t p = 0; p < panels; ++p) {
      const int64_t c = (p * kLongThreads + threadIdx.x) * 8;
      load(c, (int)max((int64_t)0, min((int64_t)8, a.cols - c)));
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) s = fmaf(dh[e] * w[e], yn[e], s);
      sum.add(s);
    }
    float one[1] = {sum.total()};
    const float back = unit_sum<true>(one, u, red, calls) * (1.f / (float)a.cols);  // the mean of dh w yn
#pragma unroll 2
    for (int64_t p = 0; p < panels; ++p) {
      const int64_t c = (p * kLongThreads + threadIdx.x) * 8, left = a.cols - c;
      const int n = (int)max((int64_t)0, min((int64_t)8, left));
      load(c, n);
      float dy[8] = {}, sums[8], t[8];
      if (a.dy) load8<T, VEC>(dy, (const T*)a.dy + row * a.lddy + c, n);
#pragma unroll
      for (int e = 0; e < 8; ++e) sums[e] = row != blockIdx.x && e < n ? out[c + e] : 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sums[e] = fmaf(dh[e], yn[e], sums[e]);
        t[e] = fmaf(r, fmaf(-back, yn[e], dh[e] * w[e]), dy[e]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) out[c + e] = sums[e];
      if (a.dx) store8_warp<T, VEC, true>((T*)a.dx + row * a.lddx + c, t, left, u.first, u.last, true);
      if (a.drop.cut) {
        uint32_t bits[4];
        philox(bits, a.drop, (uint32_t)(c >> 3), (uint32_t)row);
        drop8(t, a.drop, bits);
      }
      store8_warp<T, VEC, true>((T*)a.df + row * a.lddf + c, t, left, u.first, u.last, true);
    }
  }
}

// Threads of a unit and of a CTA, chunks a thread.
struct Shape {
  int tpr, threads, v;
  int units() const { return threads / tpr; }
};
// Two chunks a thread while 512 threads hold a row so, four past that.  Four throughout
// take as many warps as they save instructions, and rows on any element more (dropout,
// forward and backward, us, two against four): 16384 x 4096 bf16 95 and 103 against 95
// and 129, 4095 columns 159 and 165 against 251 and 352, 16384 x 1024 26 and 33 against
// 28 and 43, one row of 4096 3.3 and 3.6 against 3.7 and 5.3; fp32 of 8192 x 8192 180
// and 226 against 173 and 224.
Shape shape_of(int64_t cols) {
  if (cols > 512) {
    const int v = cols > 8192 ? 4 : 2, threads = (int)((cols + v * 256 - 1) / (v * 256)) * 32;
    return {threads, threads, v};
  }
  int tpr = 4;
  while (tpr * 16 < cols) tpr *= 2;
  return {tpr, 256, 2};
}
constexpr int kFwdCtas = 3, kBwdCtas = 2;  // of 256 threads on an SM
// CTAs for `rows`: what an SM holds together, and two rows a unit where that many
// units have them (each CTA of the backward writes a row of partial sums).
int64_t ctas_of(const Shape& sh, int64_t rows, int sms, int ctas256) {
  const int64_t most = (int64_t)sms * std::max(1, ctas256 * 256 / sh.threads);
  const int64_t few = (rows + 2 * sh.units() - 1) / (2 * sh.units());
  return std::min(most, std::max<int64_t>(few, std::min<int64_t>((rows + sh.units() - 1) / sh.units(), sms)));
}

template <typename K, typename A>
cudaError_t start(K kernel, const A& a, int64_t ctas, int threads, int smem, int tpr, cudaStream_t s) {
  kernel<<<(unsigned)ctas, threads, smem, s>>>(a, tpr);
  return cudaGetLastError();
}

// f(kernel, shared memory of a warp) for a shape.
template <typename T, bool VEC, typename F>
cudaError_t with_fwd(const Shape& sh, F f) {
  constexpr int two = RingOf<T, VEC, true, 2, 2, depth<T, 2>()>::kWarp;
  if (sh.v == 4) return f(add_norm_fwd_kernel<T, VEC, 4, 512, 1, true>, RingOf<T, VEC, true, 4, 2, depth<T, 4>()>::kWarp);
  if (sh.tpr > 256) return f(add_norm_fwd_kernel<T, VEC, 2, 512, 1, true>, two);
  if (sh.tpr > 32) return f(add_norm_fwd_kernel<T, VEC, 2, 256, kFwdCtas, true>, two);
  return f(add_norm_fwd_kernel<T, VEC, 2, 256, kFwdCtas, false>, RingOf<T, VEC, false, 2, 2, depth<T, 2>()>::kWarp);
}
template <typename T, bool VEC, typename F>
cudaError_t with_bwd(const Shape& sh, F f) {
  constexpr int two = RingOf<T, VEC, true, 2, 3, depth<T, 2>()>::kWarp;
  if (sh.v == 4) return f(add_norm_bwd_kernel<T, VEC, 4, 512, 1, true>, RingOf<T, VEC, true, 4, 3, depth<T, 4>()>::kWarp);
  if (sh.tpr > 256) return f(add_norm_bwd_kernel<T, VEC, 2, 512, 1, true>, two);
  if (sh.tpr > 32) return f(add_norm_bwd_kernel<T, VEC, 2, 256, kBwdCtas, true>, two);
  return f(add_norm_bwd_kernel<T, VEC, 2, 256, kBwdCtas, false>, RingOf<T, VEC, false, 2, 3, depth<T, 2>()>::kWarp);
}

template <typename T, bool VEC>
cudaError_t launch_fwd(const AddNormFwdArgs& a, int sms, cudaStream_t s) {
  if (a.cols > kMost) {
    add_norm_long_fwd_kernel<T, VEC><<<(unsigned)std::min<int64_t>(a.rows, 2 * sms), kLongThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
  const Shape sh = shape_of(a.cols);
  const int64_t ctas = ctas_of(sh, a.rows, sms, kFwdCtas);
  return with_fwd<T, VEC>(sh, [&](auto kernel, int warp) { return start(kernel, a, ctas, sh.threads, sh.threads / 32 * warp, sh.tpr, s); });
}

template <typename T, bool VEC>
cudaError_t launch_bwd(const AddNormBwdArgs& a, int64_t ctas, cudaStream_t s) {
  if (a.cols > kMost) {
    add_norm_long_bwd_kernel<T, VEC><<<(unsigned)ctas, kLongThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
  const Shape sh = shape_of(a.cols);
  return with_bwd<T, VEC>(sh, [&](auto kernel, int warp) { return start(kernel, a, ctas, sh.threads, sh.threads / 32 * warp, sh.tpr, s); });
}

template <typename T, bool VEC>
cudaError_t configure() {
  for (const int64_t cols : {512, 4096, 8192, 16384}) {  // every kernel, with its most threads
    for (const bool fwd : {true, false}) {
      const Shape sh = shape_of(cols);
      auto set = [&](auto kernel, int warp) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sh.threads / 32 * warp);
      };
      const cudaError_t e = fwd ? with_fwd<T, VEC>(sh, set) : with_bwd<T, VEC>(sh, set);
      if (e != cudaSuccess) return e;
    }
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t add_norm_configure() {
  for (auto one : {configure<float, true>, configure<float, false>, configure<__nv_bfloat16, true>, configure<__nv_bfloat16, false>,
                   configure<__half, true>, configure<__half, false>}) {
    const cudaError_t e = one();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

int64_t add_norm_bwd_ctas(int64_t rows, int64_t cols, int sms) {
  // Long rows: at most a gigabyte of partial sums.
  if (cols > kMost) return std::min<int64_t>(rows, std::min<int64_t>(2 * sms, std::max<int64_t>(1, (1 << 28) / cols)));
  return ctas_of(shape_of(cols), rows, sms, kBwdCtas);
}

cudaError_t launch_add_norm_fwd(const AddNormFwdArgs& a, int dtype, int sms, cudaStream_t s) {
  if (dtype == DMUON_BF16) return a.vec ? launch_fwd<__nv_bfloat16, true>(a, sms, s) : launch_fwd<__nv_bfloat16, false>(a, sms, s);
  if (dtype == DMUON_F16) return a.vec ? launch_fwd<__half, true>(a, sms, s) : launch_fwd<__half, false>(a, sms, s);
  return a.vec ? launch_fwd<float, true>(a, sms, s) : launch_fwd<float, false>(a, sms, s);
}

cudaError_t launch_add_norm_bwd(const AddNormBwdArgs& a, int dtype, int64_t ctas, cudaStream_t s) {
  if (dtype == DMUON_BF16) return a.vec ? launch_bwd<__nv_bfloat16, true>(a, ctas, s) : launch_bwd<__nv_bfloat16, false>(a, ctas, s);
  if (dtype == DMUON_F16) return a.vec ? launch_bwd<__half, true>(a, ctas, s) : launch_bwd<__half, false>(a, ctas, s);
  return a.vec ? launch_bwd<float, true>(a, ctas, s) : launch_bwd<float, false>(a, ctas, s);
}

}  // namespace dmuon
