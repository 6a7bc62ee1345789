// A pass over a matrix in tiles of 128 x 128: MXFP8 quantisation by rows, by
// columns or both (codes in mx8.cuh), of a matrix or of dout * act'(pre), whose
// values go to a matrix of their own and whose column sums to d_bias besides.
//
// A warp takes 32 x 32 elements into registers at a time, four rows by eight
// columns a lane, so that a block of either direction is eight or four values
// of a lane and two or three exchanges between lanes, two exponents in a word.
// Codes by rows leave from the registers (32 bytes a row); by columns they pass
// through 1.1 KB of shared memory a warp as words of four rows.  A tile's scale
// bytes of a direction are exactly one 512-byte scale tile.  The values stay fp32
// from the load to the codes: a gradient is not rounded to 16 bits on the way.
// A CTA goes down a column of tiles; each warp's coming 32 x 32 elements are on
// their way to a ring of its own (cp.async: no registers, no barrier).
// Column sums are kept in registers meanwhile, added up in a fixed order and
// written once a CTA.
#pragma once

#include "../../include/dmuon.h"
#include "act.cuh"
#include "chunk8.cuh"
#include "mx.cuh"
#include "mx8.cuh"
#include "ptx.cuh"

namespace dmuon {

namespace {

constexpr int kNoSlope = -1;  // else a kind of act.cuh
constexpr int kTile = 128;
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kColWords = 32 * 8 + 3 * 8;  // a warp's codes by columns: 8 words a column, 8 more between groups of 8 columns

// Dynamic shared memory: the ring, then Rest.
template <typename T, int KIND, bool VEC>
struct Geometry {
  static constexpr int kPieces = 4 * words8<T>() / 4 + (VEC ? 0 : 1);  // 16-byte pieces that a row's 32 elements lie in
  static constexpr int kRowBytes = kPieces * 16;
  static constexpr int kWarpBytes = 32 * kRowBytes;                      // 32 rows of one matrix
  static constexpr int kStage = (KIND == kNoSlope ? 1 : 2) * kWarps * kWarpBytes;
  static constexpr int kStages = sizeof(T) == 4 ? 2 : VEC ? 3 : 2;
  struct Rest {
    uint8_t scales[2][2][kMxScaleTile];  // of this tile and the one before; by rows, by columns
    uint32_t cols[kWarps][kColWords];
    float sums[kWarps][64];
  };
  static constexpr int kSmem = kStages * kStage + (int)sizeof(Rest);
  static_assert(VEC || kWarpBytes >= 32 * 33 * (int)sizeof(T), "dz passes through a slot");
};

// 32 x 32 elements (rows, cols of them in the matrix) to a warp's slot, zeros
// outside the matrix; `row` is this lane's first row (a quad a row, whole lines an
// access), `down` the bytes from it to its next one, eight rows on, `inside` an
// aligned piece of the matrix.  Rows on any element come by the aligned pieces
// around them, the last cut off at the row's end; a row's first piece begins at
// most 15 bytes before it.
template <typename T, int KIND, bool VEC>
__device__ __forceinline__ void fetch_tile(uint32_t slot, const uint8_t* row, int64_t down, const uint8_t* inside, int rows, int cols, int lane) {
  using G = Geometry<T, KIND, VEC>;
  constexpr int W = words8<T>() / 4;  // pieces of a lane
  const int q = lane & 3, rq = lane >> 2;
  slot += rq * G::kRowBytes + q * 16;
  if (VEC && rows >= 32 && cols >= 32) {
    row += q * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i, row += down)
#pragma unroll
      for (int k = 0; k < W; ++k) copy16(slot + i * 8 * G::kRowBytes + k * 64, row + k * 64);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i, row += down) {
    const uint32_t m = VEC ? 0u : past16(row);
    const uint8_t* from = row - m;
    const int bytes = i * 8 + rq < rows && cols > 0 ? (int)m + min(cols, 32) * (int)sizeof(T) : 0;
#pragma unroll
    for (int k = 0; k < W + (VEC ? 0 : 1); ++k) {
      const int at = k * 64 + q * 16, n = max(0, min(16, bytes - at));
      if (k < W || q == 0) copy16(slot + i * 8 * G::kRowBytes + k * 64, n ? from + at : inside, n);
    }
  }
}

template <typename T, int KIND, bool VEC>
__global__ void __launch_bounds__(kThreads, Geometry<T, KIND, VEC>::kSmem <= 113 * 1024 ? 2 : 1) mx8_tiles_kernel(const Mx8Args a) {
  using G = Geometry<T, KIND, VEC>;
  extern __shared__ __align__(128) uint8_t smem[];
  typename G::Rest& sh = *reinterpret_cast<typename G::Rest*>(smem + G::kStages * G::kStage);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = lane & 3, rq = lane >> 2;                  // columns 8 q + e, rows 4 rq + i of a warp's 32 x 32
  const int rb = warp & 3, half = warp >> 2;               // the warp's block of rows; its two blocks of columns
  const int64_t ct = (a.cols + kTile - 1) / kTile, rt = (a.rows + kTile - 1) / kTile;
  const int64_t tc = blockIdx.x % ct, chunk = blockIdx.x / ct;
  const int64_t tr0 = chunk * a.tiles;
  const int tiles = (int)min(a.tiles, rt - tr0);
  const int64_t row_pitch = mx_pitch(a.cols, 8), col_pitch = mx_pitch(a.rows, 8);
  const int64_t row00 = tr0 * kTile + rb * 32, col00 = tc * kTile + half * 64;  // the warp's first element
  const int rows_left = (int)min(a.rows - row00, (int64_t)1 << 20), cols_left = (int)min(a.cols - col00, (int64_t)1 << 20);
  constexpr bool slope = KIND != kNoSlope;
  uint8_t* ring = smem + warp * G::kWarpBytes;
  // Step 2 t + j: the jth 32 columns in the tth tile.  A matrix's rows as bytes:
  // the lane's first row of the step that is fetched next.
  const int64_t ld = a.ld * (int)sizeof(T), ldpre = a.ldpre * (int)sizeof(T);
  const uint8_t* f_src = (const uint8_t*)a.src + (row00 + rq) * ld + col00 * (int)sizeof(T);
  const uint8_t* f_pre = slope ? (const uint8_t*)a.pre + (row00 + rq) * ldpre + col00 * (int)sizeof(T) : nullptr;
  const uint8_t *in_src = (const uint8_t*)a.src - past16((const uint8_t*)a.src), *in_pre = (const uint8_t*)a.pre - past16((const uint8_t*)a.pre);
  const uint32_t ring0 = ptx::smem_addr(ring);
  int ahead = 0, ahead_slot = 0;
  auto fetch = [&]() {
    const int rows = rows_left - (ahead >> 1) * kTile, cols = cols_left - (ahead & 1) * 32;
    if (ahead < 2 * tiles) {
      const uint32_t slot = ring0 + ahead_slot;
      fetch_tile<T, KIND, VEC>(slot, f_src, 8 * ld, in_src, rows, cols, lane);
      if (slope) fetch_tile<T, KIND, VEC>(slot + kWarps * G::kWarpBytes, f_pre, 8 * ldpre, in_pre, rows, cols, lane);
    }
    const int64_t right = 32 * (int)sizeof(T);
    f_src += ahead & 1 ? kTile * ld - right : right;
    if (slope) f_pre += ahead & 1 ? kTile * ldpre - right : right;
    ++ahead;
    if ((ahead_slot += G::kStage) == G::kStages * G::kStage) ahead_slot = 0;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int s = 0; s < G::kStages; ++s) fetch();
  f2 sums[2][4];
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) sums[j][k] = 0;

  uint8_t* row_out = a.row_data + (row00 + 4 * rq) * row_pitch + col00 + 8 * q;
  uint8_t* col_out = a.col_data + (col00 + (lane >> 1)) * col_pitch + row00 + (lane & 1) * 16;
  const uint32_t* col_words = sh.cols[warp] + (lane >> 1) * 8 + (lane >> 4) * 8 + (lane & 1) * 4;  // column lane / 2
  uint8_t* row_bytes = sh.scales[0][0] + (4 * rq + q) * 16 + rb * 4 + half * 2;
  uint8_t* col_bytes = sh.scales[0][1] + (8 * q + rq) * 16 + half * 8 + rb;
  uint8_t* row_scales = a.row_scales + (tr0 * mx_scale_cols(a.cols) + tc) * kMxScaleTile + threadIdx.x * 16;
  uint8_t* col_scales = a.col_scales + (tc * mx_scale_cols(a.rows) + tr0) * kMxScaleTile + (threadIdx.x - 32) * 16;
  const int64_t scale_row = mx_scale_cols(a.cols) * kMxScaleTile;
  int slot_at = 0;
  const uint8_t* my_slot = ring + 4 * rq * G::kRowBytes + q * words8<T>() * 4;
#pragma unroll 1
  for (int step = 0; step < 2 * tiles; ++step) {
    const int j = step & 1, buf = (step >> 1) & 1;
    const int rows = rows_left - (step >> 1) * kTile, cols = cols_left - j * 32;  // below 1: none; 32 or more: all
    asm volatile("cp.async.wait_group %0;" ::"n"(G::kStages - 1) : "memory");
    __syncwarp();
    f2 v[4][4];
    {
      const uint8_t* slot = my_slot + slot_at;
      auto past = [&](const void* base, int64_t pitch, int i) {  // of the lane's ith row
        const int64_t row = row00 + (step >> 1) * kTile + 4 * rq + i;
        return VEC ? 0u : (uint32_t)((uintptr_t)base + (uint64_t)(row * pitch) + (uint64_t)((col00 + j * 32) * (int)sizeof(T))) & 15u;
      };
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        take8<T, VEC>(v[i], slot + i * G::kRowBytes, past(a.src, ld, i));
        if constexpr (slope) {
          f2 z[4];
          take8<T, VEC>(z, slot + kWarps * G::kWarpBytes + i * G::kRowBytes, past(a.pre, ldpre, i));
          act_slopes<KIND>(v[i], z, a.act);
        }
      }
    }
    __syncwarp();
    if constexpr (VEC) fetch();
    {
      if (a.parts) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const f2 s = add2(add2(v[0][k], v[1][k]), add2(v[2][k], v[3][k]));
          if (j == 0) sums[0][k] = add2(sums[0][k], s);
          else sums[1][k] = add2(sums[1][k], s);
        }
      }
      if (a.dz && rows > 0 && cols > 0) {
        T* dz = (T*)a.dz + (row00 + (step >> 1) * kTile) * a.lddz + col00 + j * 32;
        T* mine = reinterpret_cast<T*>(ring + slot_at);  // rows on any element: the slot, whose elements are taken
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float f[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 p = unpack2(v[i][k]);
            f[2 * k] = p.x;
            f[2 * k + 1] = p.y;
          }
          if constexpr (VEC) {
            if (4 * rq + i < rows) store8<T>(dz + (4 * rq + i) * a.lddz + 8 * q, f, cols - 8 * q);
          } else {  // through shared memory, so that the lanes of a store hold consecutive elements
            uint32_t w[words8<T>()];
            pack8<T>(w, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              if constexpr (sizeof(T) == 4) reinterpret_cast<uint32_t*>(mine)[(4 * rq + i) * 33 + 8 * q + e] = w[e];
              else reinterpret_cast<uint16_t*>(mine)[(4 * rq + i) * 33 + 8 * q + e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
            }
          }
        }
        if constexpr (!VEC) {
          __syncwarp();
          if (lane < cols)
            for (int r = 0; r < min(rows, 32); ++r) dz[r * a.lddz + lane] = mine[r * 33 + lane];
          __syncwarp();
        }
      }
    }
    if constexpr (!VEC) fetch();
    if ((slot_at += G::kStage) == G::kStages * G::kStage) slot_at = 0;
    if (a.row_data) {
      float m[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        m[i] = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 p = unpack2(v[i][k]);
          m[i] = mx8::max_abs(m[i], p.x, p.y);
        }
      }
      uint32_t two[2] = {mx8::keys2(m[0], m[1], a.up), mx8::keys2(m[2], m[3], a.up)};
#pragma unroll
      for (int o = 1; o < 4; o *= 2)
#pragma unroll
        for (int k = 0; k < 2; ++k) two[k] = mx8::max_halves(two[k], __shfl_xor_sync(0xffffffffu, two[k], o));
      uint32_t bad = 0;  // bit i: row i's block holds Inf or NaN
      const bool look = __any_sync(0xffffffffu, mx8::may_not_be_finite(mx8::max_halves(two[0], two[1])));
      if (look) {
#pragma unroll
        for (int i = 0; i < 4; ++i) bad |= (uint32_t)mx8::not_finite(m[i]) << i;
#pragma unroll
        for (int o = 1; o < 4; o *= 2) bad |= __shfl_xor_sync(0xffffffffu, bad, o);
      }
      two[0] = mx8::exponents2(two[0]);
      two[1] = mx8::exponents2(two[1]);
      {  // lane q has row q's byte
        const uint32_t mine = q & 2 ? two[1] : two[0];
        uint32_t byte = q & 1 ? mx8::byte_of(mine, 1) : mx8::byte_of(mine, 0);
        if (look && (bad >> q & 1)) byte = 255u;
        row_bytes[buf * 2 * kMxScaleTile + j] = (uint8_t)byte;
      }
      uint8_t* out = row_out;
      const int live = cols > 0 ? rows - 4 * rq : 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 both_rows = mx8::factors2(two[i / 2]);
        const f2 inv = both(i & 1 ? both_rows.y : both_rows.x);
        float2 f[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = unpack2(mul2(v[i][k], inv));
        uint2 w = make_uint2(mx8::codes4(f[0].x, f[0].y, f[1].x, f[1].y), mx8::codes4(f[2].x, f[2].y, f[3].x, f[3].y));
        if (look && (bad >> i & 1)) w = make_uint2(0, 0);
        if (i < live) *reinterpret_cast<uint2*>(out) = w;
        out += row_pitch;
      }
      row_out += j ? kTile * row_pitch - 32 : 32;
    }
    if (a.col_data) {
      float m[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float2 p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = unpack2(v[i][k]);
        m[2 * k] = mx8::max_abs(mx8::max_abs(p[0].x, p[1].x, p[2].x), p[3].x, 0.f);
        m[2 * k + 1] = mx8::max_abs(mx8::max_abs(p[0].y, p[1].y, p[2].y), p[3].y, 0.f);
      }
      uint32_t two[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) two[k] = mx8::keys2(m[2 * k], m[2 * k + 1], a.up);
#pragma unroll
      for (int o = 4; o < 32; o *= 2)
#pragma unroll
        for (int k = 0; k < 4; ++k) two[k] = mx8::max_halves(two[k], __shfl_xor_sync(0xffffffffu, two[k], o));
      uint32_t bad = 0;  // bit e: column 8 q + e's block holds Inf or NaN
      const bool look = __any_sync(
          0xffffffffu, mx8::may_not_be_finite(mx8::max_halves(mx8::max_halves(two[0], two[1]), mx8::max_halves(two[2], two[3]))));
      if (look) {
#pragma unroll
        for (int e = 0; e < 8; ++e) bad |= (uint32_t)mx8::not_finite(m[e]) << e;
#pragma unroll
        for (int o = 4; o < 32; o *= 2) bad |= __shfl_xor_sync(0xffffffffu, bad, o);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) two[k] = mx8::exponents2(two[k]);
      {  // lane rq has column 8 q + rq's byte
        const uint32_t lo = rq & 2 ? two[1] : two[0], hi = rq & 2 ? two[3] : two[2], mine = rq & 4 ? hi : lo;
        uint32_t byte = rq & 1 ? mx8::byte_of(mine, 1) : mx8::byte_of(mine, 0);
        if (look && (bad >> rq & 1)) byte = 255u;
        col_bytes[buf * 2 * kMxScaleTile + j * 4] = (uint8_t)byte;
      }
      uint32_t* mine = sh.cols[warp] + 72 * q + rq;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = mx8::factors2(two[k]);
        const f2 inv = pack2(f.x, f.y);
        float2 p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = unpack2(mul2(v[i][k], inv));
        uint32_t w[2] = {mx8::codes4(p[0].x, p[1].x, p[2].x, p[3].x), mx8::codes4(p[0].y, p[1].y, p[2].y, p[3].y)};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (look && (bad >> (2 * k + h) & 1)) w[h] = 0;
          mine[(2 * k + h) * 8] = w[h];
        }
      }
      __syncwarp();
      uint8_t* out = col_out;
      const int live = rows > 0 ? cols - (lane >> 1) : 0;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint4 w = *reinterpret_cast<const uint4*>(col_words + k * (16 * 8 + 2 * 8));
        if (16 * k < live) *reinterpret_cast<uint4*>(out) = w;
        out += 16 * col_pitch;
      }
      col_out += j ? kTile - 32 * col_pitch : 32 * col_pitch;
      __syncwarp();
    }
    // The bytes of a tile are complete behind its one barrier; they are read
    // before the next one, and written again after it.
    if (j == 1 && (a.row_data || a.col_data)) {
      __syncthreads();
      const int t = threadIdx.x;
      if (t < 32 && a.row_data) *reinterpret_cast<uint4*>(row_scales) = reinterpret_cast<const uint4*>(sh.scales[buf][0])[t];
      if (t >= 32 && t < 64 && a.col_data) *reinterpret_cast<uint4*>(col_scales) = reinterpret_cast<const uint4*>(sh.scales[buf][1])[t - 32];
      row_scales += scale_row;
      col_scales += kMxScaleTile;
    }
  }
  {
    if (a.parts) {  // over the warp's lanes of a column, then over the four warps down the tile
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 p = unpack2(sums[j][e / 2]);
          float s = e & 1 ? p.y : p.x;
#pragma unroll
          for (int o = 4; o < 32; o *= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
          if (rq == e) sh.sums[warp][j * 32 + 8 * q + e] = s;
        }
      __syncthreads();
      const int c = threadIdx.x;
      if (c < kTile && tc * kTile + c < a.cols) {
        const int w = c / 64 * 4, at = c % 64;
        a.parts[chunk * a.part_ld + tc * kTile + c] = (sh.sums[w][at] + sh.sums[w + 1][at]) + (sh.sums[w + 2][at] + sh.sums[w + 3][at]);
      }
    }
  }
}

template <typename T, int KIND>
struct Tiles {
  static cudaError_t configure() {
    const cudaError_t e = cudaFuncSetAttribute(mx8_tiles_kernel<T, KIND, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, Geometry<T, KIND, true>::kSmem);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(mx8_tiles_kernel<T, KIND, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, Geometry<T, KIND, false>::kSmem);
  }
  static cudaError_t launch(const Mx8Args& a, cudaStream_t s) {
    const int64_t ct = (a.cols + kTile - 1) / kTile, rt = (a.rows + kTile - 1) / kTile;
    const unsigned ctas = (unsigned)(ct * ((rt + a.tiles - 1) / a.tiles));
    if (a.vec) mx8_tiles_kernel<T, KIND, true><<<ctas, kThreads, Geometry<T, KIND, true>::kSmem, s>>>(a);
    else mx8_tiles_kernel<T, KIND, false><<<ctas, kThreads, Geometry<T, KIND, false>::kSmem, s>>>(a);
    return cudaGetLastError();
  }
};

template <int KIND>
cudaError_t configure_kind() {
  cudaError_t e;
  if ((e = Tiles<float, KIND>::configure()) != cudaSuccess) return e;
  if ((e = Tiles<__nv_bfloat16, KIND>::configure()) != cudaSuccess) return e;
  return Tiles<__half, KIND>::configure();
}
template <int KIND>
cudaError_t launch_kind(const Mx8Args& a, int dtype, cudaStream_t s) {
  if (dtype == DMUON_BF16) return Tiles<__nv_bfloat16, KIND>::launch(a, s);
  if (dtype == DMUON_F16) return Tiles<__half, KIND>::launch(a, s);
  return Tiles<float, KIND>::launch(a, s);
}

}  // namespace

}  // namespace dmuon
