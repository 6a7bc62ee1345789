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
#include "../../include/dmuon.h"
#include "act.cuh"
#include "chunk8.cuh"
#include "mx.cuh"
#include "mx8.cuh"
#include "ptx.cuh"

namespace dmuon {

namespace {

constexpr int kTile = 128;
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kColWords = 32 * 8 + 3 * 8;  // a warp's codes by columns: 8 words a column, 8 more between groups of 8 columns

// Dynamic shared memory: the ring, then Rest.
template <typename T, bool GRAD, bool VEC>
struct Geometry {
  static constexpr int kPieces = 4 * words8<T>() / 4 + (VEC ? 0 : 1);  // 16-byte pieces that a row's 32 elements lie in
  static constexpr int kRowBytes = kPieces * 16;
  static constexpr int kWarpBytes = 32 * kRowBytes;                      // 32 rows of one matrix
  static constexpr int kStage = (GRAD ? 2 : 1) * kWarps * kWarpBytes;
  static constexpr int kStages = sizeof(T) == 4 ? 2 : VEC ? 3 : 2;
  struct Rest {
    uint8_t scales[2][2][kMxScaleTile];  // of this tile and the one before; by rows, by columns
    uint32_t cols[kWarps][kColWords];
    float sums[GRAD ? kWarps : 1][GRAD ? 64 : 1];
    T dz[GRAD && !VEC ? kWarps : 1][GRAD && !VEC ? 32 * 33 : 1];
  };
  static constexpr int kSmem = kStages * kStage + (int)sizeof(Rest);
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// 32 x 32 elements (rows, cols of them in the matrix, from p on) to a warp's slot,
// zeros outside the matrix.  Rows on any element come by the aligned pieces
// around them, the last cut off at the row's end; a row's first piece begins at
// most 15 bytes before it.
template <typename T, bool GRAD, bool VEC>
__device__ __forceinline__ void fetch_tile(uint32_t slot, const T* p, int64_t ld, int rows, int cols, int lane) {
  using G = Geometry<T, GRAD, VEC>;
  constexpr int W = words8<T>() / 4;  // pieces of a lane
  const int q = lane & 3, rq = lane >> 2;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 8 + rq;  // a quad a row: whole lines
    const T* row = p + r * ld;
    const uint32_t m = VEC ? 0u : past16(row);
    const uint8_t* from = reinterpret_cast<const uint8_t*>(row) - m;
    const int bytes = r < rows ? (int)m + max(0, min(cols, 32)) * (int)sizeof(T) : 0;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const int piece = k * 4 + q, n = max(0, min(16, bytes - piece * 16));
      copy16(slot + r * G::kRowBytes + piece * 16, n ? from + piece * 16 : reinterpret_cast<const uint8_t*>(p) - (VEC ? 0u : past16(p)), n);
    }
    if (!VEC && q == 0) {
      const int piece = W * 4, n = max(0, min(16, bytes - piece * 16));
      copy16(slot + r * G::kRowBytes + piece * 16, n ? from + piece * 16 : reinterpret_cast<const uint8_t*>(p) - past16(p), n);
    }
  }
}

// Eight values from a slot's row; m: bytes of the matrix's row past a 16-byte boundary.
template <typename T, bool VEC>
__device__ __forceinline__ void take8(f2 (&f)[4], const uint8_t* at, uint32_t m) {
  constexpr int W = words8<T>(), N = W + (VEC ? 0 : 4);
  uint32_t w[N];
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(at + i * 4);
    w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
  }
  if constexpr (!VEC) {
#pragma unroll
    for (int i = 0; i < W + 2; ++i) w[i] = m & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < W + 1; ++i) w[i] = m & 4 ? w[i + 1] : w[i];
    if constexpr (sizeof(T) == 2)
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], (m & 2) * 8);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (sizeof(T) == 4) {
      f[k] = pack2(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
    } else if constexpr (std::is_same<T, __half>::value) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
      f[k] = pack2(v.x, v.y);
    } else {
      f[k] = pack2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u));
    }
  }
}

template <typename T, bool GRAD, bool VEC>
__global__ void __launch_bounds__(kThreads, Geometry<T, GRAD, VEC>::kSmem <= 113 * 1024 ? 2 : 1) mx8_tiles_kernel(const Mx8Args a) {
  using G = Geometry<T, GRAD, VEC>;
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
  const bool slope = GRAD && a.pre;
  uint8_t* ring = smem + warp * G::kWarpBytes;
  auto fetch = [&](int step) {  // step 2 t + j: the jth 32 columns in the tth tile
    if (step < 2 * tiles) {
      const int64_t row = row00 + (step >> 1) * kTile, col = col00 + (step & 1) * 32;
      const int rows = (int)max((int64_t)0, min((int64_t)32, a.rows - row)), cols = (int)max((int64_t)0, min((int64_t)32, a.cols - col));
      if (rows > 0 && cols > 0) {
        const uint32_t slot = ptx::smem_addr(ring + step % G::kStages * G::kStage);
        fetch_tile<T, GRAD, VEC>(slot, (const T*)a.src + row * a.ld + col, a.ld, rows, cols, lane);
        if (slope) fetch_tile<T, GRAD, VEC>(slot + kWarps * G::kWarpBytes, (const T*)a.pre + row * a.ldpre + col, a.ldpre, rows, cols, lane);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int s = 0; s < G::kStages; ++s) fetch(s);
  f2 sums[2][4];
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) sums[j][k] = 0;

#pragma unroll 1
  for (int step = 0; step < 2 * tiles; ++step) {
    const int j = step & 1, buf = (step >> 1) & 1;
    const int64_t row0 = row00 + (step >> 1) * kTile, col0 = col00 + j * 32;
    const int rows = (int)min((int64_t)32, a.rows - row0), cols = (int)min((int64_t)32, a.cols - col0);  // below 1: none
    asm volatile("cp.async.wait_group %0;" ::"n"(G::kStages - 1) : "memory");
    __syncwarp();
    f2 v[4][4];
    if (rows > 0 && cols > 0) {
      const uint8_t* slot = ring + step % G::kStages * G::kStage + 4 * rq * G::kRowBytes + q * words8<T>() * 4;
      const T* src = (const T*)a.src + (row0 + 4 * rq) * a.ld + col0;
#pragma unroll
      for (int i = 0; i < 4; ++i) take8<T, VEC>(v[i], slot + i * G::kRowBytes, VEC ? 0u : past16(src + i * a.ld));
      if (slope) {
        const T* pre = (const T*)a.pre + (row0 + 4 * rq) * a.ldpre + col0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f2 z[4];
          take8<T, VEC>(z, slot + kWarps * G::kWarpBytes + i * G::kRowBytes, VEC ? 0u : past16(pre + i * a.ldpre));
          act_slopes(v[i], z, a.act);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) v[i][k] = 0;
    }
    __syncwarp();
    fetch(step + G::kStages);
    if constexpr (GRAD) {
      if (a.parts) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const f2 s = add2(add2(v[0][k], v[1][k]), add2(v[2][k], v[3][k]));
          if (j == 0) sums[0][k] = add2(sums[0][k], s);
          else sums[1][k] = add2(sums[1][k], s);
        }
      }
      if (a.dz && rows > 0 && cols > 0) {
        T* dz = (T*)a.dz + row0 * a.lddz + col0;
        T* mine = sh.dz[VEC ? 0 : warp];
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
            for (int r = 0; r < rows; ++r) dz[r * a.lddz + lane] = mine[r * 33 + lane];
          __syncwarp();
        }
      }
    }
    if (a.row_data) {
      uint32_t two[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float m[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          m[h] = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 p = unpack2(v[2 * k + h][e]);
            m[h] = mx8::max_abs(m[h], p.x, p.y);
          }
        }
        two[k] = mx8::keys2(m[0], m[1], a.rounding);
      }
#pragma unroll
      for (int o = 1; o < 4; o *= 2)
#pragma unroll
        for (int k = 0; k < 2; ++k) two[k] = mx8::max_halves(two[k], __shfl_xor_sync(0xffffffffu, two[k], o));
      const bool bad = __any_sync(0xffffffffu, mx8::any_not_finite(two[0], a.rounding) || mx8::any_not_finite(two[1], a.rounding));
      {  // lane q has row q's byte
        const uint32_t mine = q & 2 ? two[1] : two[0];
        sh.scales[buf][0][(4 * rq + q) * 16 + rb * 4 + half * 2 + j] =
            (uint8_t)(q & 1 ? mx8::byte_of(mine, 1, a.rounding) : mx8::byte_of(mine, 0, a.rounding));
      }
      uint8_t* out = a.row_data + (row0 + 4 * rq) * row_pitch + col0 + 8 * q;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f2 inv = both(mx8::factor_of(mx8::exponent_of(two[i / 2], i & 1)));
        float f[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 p = unpack2(mul2(v[i][k], inv));
          f[2 * k] = p.x;
          f[2 * k + 1] = p.y;
        }
        uint2 w = make_uint2(mx8::codes4(f[0], f[1], f[2], f[3]), mx8::codes4(f[4], f[5], f[6], f[7]));
        if (bad && mx8::byte_of(two[i / 2], i & 1, a.rounding) == 255u) w = make_uint2(0, 0);
        if (4 * rq + i < rows && cols > 0) *reinterpret_cast<uint2*>(out + i * row_pitch) = w;
      }
    }
    if (a.col_data) {
      uint32_t two[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float2 p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = unpack2(v[i][k]);
        two[k] = mx8::keys2(mx8::max_abs(mx8::max_abs(p[0].x, p[1].x, p[2].x), p[3].x, 0.f),
                            mx8::max_abs(mx8::max_abs(p[0].y, p[1].y, p[2].y), p[3].y, 0.f), a.rounding);
      }
#pragma unroll
      for (int o = 4; o < 32; o *= 2)
#pragma unroll
        for (int k = 0; k < 4; ++k) two[k] = mx8::max_halves(two[k], __shfl_xor_sync(0xffffffffu, two[k], o));
      const bool bad = __any_sync(0xffffffffu, mx8::any_not_finite(two[0], a.rounding) || mx8::any_not_finite(two[1], a.rounding) ||
                                                   mx8::any_not_finite(two[2], a.rounding) || mx8::any_not_finite(two[3], a.rounding));
      {  // lane rq has column 8 q + rq's byte
        const uint32_t lo = rq & 2 ? two[1] : two[0], hi = rq & 2 ? two[3] : two[2], mine = rq & 4 ? hi : lo;
        const int c = half * 64 + j * 32 + 8 * q + rq;  // row of the transposed matrix within the tile
        sh.scales[buf][1][(c & 31) * 16 + (c >> 5) * 4 + rb] =
            (uint8_t)(rq & 1 ? mx8::byte_of(mine, 1, a.rounding) : mx8::byte_of(mine, 0, a.rounding));
      }
      uint32_t* mine = sh.cols[warp];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const f2 inv = pack2(mx8::factor_of(mx8::exponent_of(two[k], 0)), mx8::factor_of(mx8::exponent_of(two[k], 1)));
        float2 p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = unpack2(mul2(v[i][k], inv));
        uint32_t w[2] = {mx8::codes4(p[0].x, p[1].x, p[2].x, p[3].x), mx8::codes4(p[0].y, p[1].y, p[2].y, p[3].y)};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (bad && mx8::byte_of(two[k], h, a.rounding) == 255u) w[h] = 0;
          mine[(8 * q + 2 * k + h) * 8 + rq + q * 8] = w[h];
        }
      }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int c = 16 * k + (lane >> 1);
        const uint4 w = *reinterpret_cast<const uint4*>(mine + c * 8 + (c >> 3) * 8 + (lane & 1) * 4);
        if (c < cols && rows > 0) *reinterpret_cast<uint4*>(a.col_data + (col0 + c) * col_pitch + row0 + (lane & 1) * 16) = w;
      }
      __syncwarp();
    }
    // The bytes of a tile are complete behind its one barrier; they are read
    // before the next one, and written again after it.
    if (j == 1 && (a.row_data || a.col_data)) {
      __syncthreads();
      const int64_t tr = tr0 + (step >> 1);
      const int t = threadIdx.x;
      if (t < 32 && a.row_data)
        reinterpret_cast<uint4*>(a.row_scales + (tr * mx_scale_cols(a.cols) + tc) * kMxScaleTile)[t] = reinterpret_cast<const uint4*>(sh.scales[buf][0])[t];
      if (t >= 32 && t < 64 && a.col_data)
        reinterpret_cast<uint4*>(a.col_scales + (tc * mx_scale_cols(a.rows) + tr) * kMxScaleTile)[t - 32] =
            reinterpret_cast<const uint4*>(sh.scales[buf][1])[t - 32];
    }
  }
  if constexpr (GRAD) {
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

template <typename T, bool GRAD>
cudaError_t configure_tiles() {
  const cudaError_t e = cudaFuncSetAttribute(mx8_tiles_kernel<T, GRAD, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, Geometry<T, GRAD, true>::kSmem);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(mx8_tiles_kernel<T, GRAD, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, Geometry<T, GRAD, false>::kSmem);
}

template <typename T, bool GRAD>
cudaError_t launch_tiles(const Mx8Args& a, cudaStream_t s) {
  const int64_t ct = (a.cols + kTile - 1) / kTile, rt = (a.rows + kTile - 1) / kTile;
  const unsigned ctas = (unsigned)(ct * ((rt + a.tiles - 1) / a.tiles));
  if (a.vec) mx8_tiles_kernel<T, GRAD, true><<<ctas, kThreads, Geometry<T, GRAD, true>::kSmem, s>>>(a);
  else mx8_tiles_kernel<T, GRAD, false><<<ctas, kThreads, Geometry<T, GRAD, false>::kSmem, s>>>(a);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_tiles(const Mx8Args& a, bool grad, cudaStream_t s) {
  return grad ? launch_tiles<T, true>(a, s) : launch_tiles<T, false>(a, s);
}

// ------------------------------------------------------------ reading back

template <typename T>
__device__ __forceinline__ uint32_t value_word(float lo, float hi) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// A lane reads the codes of 32 bytes of output (16 or 8 elements, all of one
// block) and stores them whole, four rows in flight; rows of dst on any element
// by aligned pieces.  Short rows share a warp.
constexpr int kDqRows = 32;  // per CTA: 8 warps x 4 rows, 32 / lanes times as many short ones
template <typename T>
constexpr int dq_cols() { return 32 * 32 / (int)sizeof(T); }

template <typename T, bool ANY>
__global__ void __launch_bounds__(256) mx8_dequant_kernel(const MxDequantArgs a, int lanes) {  // lanes of a row: a power of two
  constexpr int kPer = 32 / (int)sizeof(T), kWords = kPer / 4;
  const int64_t ct = (a.k + dq_cols<T>() - 1) / dq_cols<T>();
  const int at_once = 256 / lanes, lane = threadIdx.x & (lanes - 1);
  const int64_t row0 = (int64_t)(blockIdx.x / ct) * 4 * at_once + threadIdx.x / lanes;
  const int64_t col = (int64_t)(blockIdx.x % ct) * dq_cols<T>() + lane * kPer;
  if (!ANY && col >= a.k) return;
  const int64_t pitch = mx_pitch(a.k, 8), blk = col / kMxBlock, sc = mx_scale_cols(a.k);
  uint32_t q[4][kWords] = {};
  uint32_t byte[4] = {};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = row0 + at_once * i;
    if (r >= a.rows || (ANY && col >= a.k)) continue;
    const uint8_t* src = a.data + r * pitch + col;
    if constexpr (kWords == 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(src);
      q[i][0] = v.x; q[i][1] = v.y; q[i][kWords - 2] = v.z; q[i][kWords - 1] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(src);
      q[i][0] = v.x; q[i][1] = v.y;
    }
    byte[i] = a.scales[((r >> 7) * sc + (blk >> 2)) * kMxScaleTile + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (blk & 3)];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = row0 + at_once * i;
    if (!ANY && r >= a.rows) continue;
    const float s = mx8::scale_value(byte[i]);
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < kPer / 2; ++j) {
      const float2 v = mx8::values2(q[i][j / 2] >> (16 * (j & 1)));
      if constexpr (sizeof(T) == 4) {
        w[4 + 2 * j] = __float_as_uint(v.x * s);
        w[5 + 2 * j] = __float_as_uint(v.y * s);
      } else {
        w[4 + j] = value_word<T>(v.x * s, v.y * s);
      }
    }
    T* dst = (T*)a.dst + r * a.ld + col;
    const int64_t left = (a.k - col) * (int64_t)sizeof(T);
    if constexpr (ANY) {
      store_pieces<sizeof(T)>(reinterpret_cast<uint8_t*>(dst), w, left, lane == 0, lane == lanes - 1 || left < 64, r < a.rows);
    } else if (left >= 32) {
      ptx::st_global_v8(dst, w + 4);
    } else {
#pragma unroll
      for (int j = 0; j < kPer - 1; ++j)
        if (col + j < a.k) {
          if constexpr (sizeof(T) == 4) reinterpret_cast<uint32_t*>(dst)[j] = w[4 + j];
          else reinterpret_cast<uint16_t*>(dst)[j] = (uint16_t)(w[4 + j / 2] >> (16 * (j & 1)));
        }
    }
  }
}

template <typename T>
cudaError_t launch_dequant(const MxDequantArgs& a, cudaStream_t s) {
  int lanes = 1;
  while (lanes < 32 && lanes * 32 / (int)sizeof(T) < a.k) lanes *= 2;
  const int64_t rows = kDqRows * (32 / lanes);
  const int64_t tiles = (a.rows + rows - 1) / rows * ((a.k + dq_cols<T>() - 1) / dq_cols<T>());
  if (a.vec) mx8_dequant_kernel<T, false><<<(unsigned)tiles, 256, 0, s>>>(a, lanes);
  else mx8_dequant_kernel<T, true><<<(unsigned)tiles, 256, 0, s>>>(a, lanes);
  return cudaGetLastError();
}

// ------------------------------------------------------------ column sums

// 32 columns a CTA, a row of 32 lanes every 32nd of the partial rows; then the
// 32 sums of a column, in order.
__global__ void __launch_bounds__(1024) column_sums_kernel(const float* parts, int64_t n, int64_t ld, int64_t cols, float* out) {
  __shared__ float part[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int64_t r = warp; r < n; r += 32) s += parts[r * ld + c];
  }
  part[warp][lane] = s;
  __syncthreads();
  s = part[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int64_t mine = (int64_t)blockIdx.x * 32 + warp;
  if (lane == 0 && mine < cols) out[mine] = s;
}

}  // namespace

cudaError_t mx8_configure() {
  for (auto one : {configure_tiles<float, false>, configure_tiles<float, true>, configure_tiles<__nv_bfloat16, false>,
                   configure_tiles<__nv_bfloat16, true>, configure_tiles<__half, false>, configure_tiles<__half, true>}) {
    const cudaError_t e = one();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_mx8_tiles(const Mx8Args& a, int dtype, bool grad, cudaStream_t s) {
  if (dtype == DMUON_BF16) return launch_tiles<__nv_bfloat16>(a, grad, s);
  if (dtype == DMUON_F16) return launch_tiles<__half>(a, grad, s);
  return launch_tiles<float>(a, grad, s);
}

cudaError_t launch_mx8_dequant(const MxDequantArgs& a, int dtype, cudaStream_t s) {
  if (dtype == DMUON_BF16) return launch_dequant<__nv_bfloat16>(a, s);
  if (dtype == DMUON_F16) return launch_dequant<__half>(a, s);
  return launch_dequant<float>(a, s);
}

cudaError_t launch_column_sums(const float* parts, int64_t n, int64_t ld, int64_t cols, float* out, cudaStream_t s) {
  column_sums_kernel<<<(unsigned)((cols + 31) / 32), 1024, 0, s>>>(parts, n, ld, cols, out);
  return cudaGetLastError();
}

}  // namespace dmuon
