// A pass over a matrix in tiles of 128 x 128: MXFP8 quantisation by rows, by
// columns or both (codes in mx8.cuh), of a matrix or of dout * act'(pre), whose
// values go to a matrix of their own and whose column sums to d_bias besides.
//
// A warp takes 32 x 32 elements into registers at a time, four rows by eight
// columns a lane, so that a block of either direction is eight or four values
// of a lane and two or three exchanges between lanes.  What is exchanged is the
// scale byte, two in a word: it does not fall as the magnitude grows.  Codes by
// rows leave from the registers (32 bytes a row); by columns they pass through
// 1.2 KB of shared memory a warp as words of four rows.  A tile's scale bytes of
// a direction are exactly one 512-byte scale tile.  The values stay fp32
// from the load to the codes: a gradient is not rounded to 16 bits on the way.
// Column sums are kept in registers while the CTA goes down its tiles, added up
// in a fixed order and written once a CTA.
#include "../../include/dmuon.h"
#include "act.cuh"
#include "chunk8.cuh"
#include "mx.cuh"
#include "mx8.cuh"
#include "ptx.cuh"

namespace dmuon {

namespace {

constexpr int kTile = 128;
constexpr int kThreads = 256;
constexpr int kColWords = 32 * 8 + 3 * 8;  // a warp's codes by columns: 8 words a column, 8 more between groups of 8 columns


template <typename T, bool GRAD, bool VEC>
struct Shared {
  uint8_t scales[2][kMxScaleTile];
  uint32_t cols[kThreads / 32][kColWords];
  float sums[GRAD ? kThreads / 32 : 1][GRAD ? 64 : 1];
  T dz[GRAD && !VEC ? kThreads / 32 : 1][GRAD && !VEC ? 32 * 33 : 1];
};

template <typename T, bool GRAD, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) mx8_tiles_kernel(const Mx8Args a) {
  __shared__ __align__(16) Shared<T, GRAD, VEC> sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = lane & 3, rq = lane >> 2;                  // columns 8 q + e, rows 4 rq + i of a warp's 32 x 32
  const int rb = warp & 3, half = warp >> 2;               // the warp's block of rows; its two blocks of columns
  const int64_t ct = (a.cols + kTile - 1) / kTile, rt = (a.rows + kTile - 1) / kTile;
  const int64_t tc = blockIdx.x % ct, chunk = blockIdx.x / ct;
  const int64_t tr1 = min((chunk + 1) * a.tiles, rt);
  const int64_t row_pitch = mx_pitch(a.cols, 8), col_pitch = mx_pitch(a.rows, 8);
  float sums[2][8];
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[j][e] = 0.f;

  for (int64_t tr = chunk * a.tiles; tr < tr1; ++tr) {
    const int64_t row0 = tr * kTile + rb * 32;
    const int rows = (int)min((int64_t)32, a.rows - row0);  // of this warp's, below 1: none
#pragma unroll 1
    for (int j = 0; j < 2; ++j) {
      const int64_t col0 = tc * kTile + half * 64 + j * 32;
      const int cols = (int)min((int64_t)32, a.cols - col0);
      float v[4][8];
      {
        const T* src = (const T*)a.src + (row0 + 4 * rq) * a.ld + col0 + 8 * q;
        const T* pre = GRAD ? (const T*)a.pre + (row0 + 4 * rq) * a.ldpre + col0 + 8 * q : nullptr;
        Raw8<T, VEC> rs[4], rp[4];
        const bool slope = GRAD && a.pre;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int n = 4 * rq + i < rows ? cols - 8 * q : 0;
          load_raw8<T, VEC>(rs[i], src + i * a.ld, n);
          if (slope) load_raw8<T, VEC>(rp[i], pre + i * a.ldpre, n);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int n = 4 * rq + i < rows ? cols - 8 * q : 0;
          values8<T, VEC>(v[i], rs[i], src + i * a.ld, n);
          if (slope) {
            float z[8];
            values8<T, VEC>(z, rp[i], pre + i * a.ldpre, n);
            act_slopes(v[i], z, a.act);
          }
        }
      }
      if constexpr (GRAD) {
        if (a.parts) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float s = (v[0][e] + v[1][e]) + (v[2][e] + v[3][e]);
            if (j == 0) sums[0][e] += s;
            else sums[1][e] += s;
          }
        }
        if (a.dz) {
          T* dz = (T*)a.dz + row0 * a.lddz + col0;
          if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (4 * rq + i < rows) store8<T>(dz + (4 * rq + i) * a.lddz + 8 * q, v[i], cols - 8 * q);
          } else {
            T* mine = sh.dz[warp];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t w[words8<T>()];
              pack8<T>(w, v[i]);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                if constexpr (sizeof(T) == 4) reinterpret_cast<uint32_t*>(mine)[(4 * rq + i) * 33 + 8 * q + e] = w[e];
                else reinterpret_cast<uint16_t*>(mine)[(4 * rq + i) * 33 + 8 * q + e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
              }
            }
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
        for (int k = 0; k < 2; ++k)
          two[k] = mx8::scale_byte(mx8::max_abs(v[2 * k]), a.round_up) | mx8::scale_byte(mx8::max_abs(v[2 * k + 1]), a.round_up) << 16;
#pragma unroll
        for (int o = 1; o < 4; o *= 2)
#pragma unroll
          for (int k = 0; k < 2; ++k) two[k] = mx8::max_halves(two[k], __shfl_xor_sync(0xffffffffu, two[k], o));
        uint8_t* out = a.row_data + (row0 + 4 * rq) * row_pitch + col0 + 8 * q;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t byte = i & 1 ? two[i / 2] >> 16 : two[i / 2] & 0xFFFFu;
          const int r = 4 * rq + i;
          if (q == i) sh.scales[0][r * 16 + rb * 4 + half * 2 + j] = (uint8_t)byte;
          const float inv = mx8::inv_scale(byte);
          uint32_t w[2];
#pragma unroll
          for (int k = 0; k < 2; ++k)
            w[k] = mx8::codes4(v[i][4 * k] * inv, v[i][4 * k + 1] * inv, v[i][4 * k + 2] * inv, v[i][4 * k + 3] * inv);
          if (byte == 255u) w[0] = w[1] = 0;
          if (r < rows && cols > 0) *reinterpret_cast<uint2*>(out + i * row_pitch) = make_uint2(w[0], w[1]);
        }
      }
      if (a.col_data) {
        uint32_t two[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t b[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int e = 2 * k + h;
            b[h] = mx8::scale_byte(mx8::max_abs(mx8::max_abs(v[0][e], v[1][e], v[2][e]), v[3][e], 0.f), a.round_up);
          }
          two[k] = b[0] | b[1] << 16;
        }
#pragma unroll
        for (int o = 4; o < 32; o *= 2)
#pragma unroll
          for (int k = 0; k < 4; ++k) two[k] = mx8::max_halves(two[k], __shfl_xor_sync(0xffffffffu, two[k], o));
        uint32_t* mine = sh.cols[warp];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t byte = e & 1 ? two[e / 2] >> 16 : two[e / 2] & 0xFFFFu;
          const int c = half * 64 + j * 32 + 8 * q + e;  // row of the transposed matrix within the tile
          if (rq == e) sh.scales[1][(c & 31) * 16 + (c >> 5) * 4 + rb] = (uint8_t)byte;
          const float inv = mx8::inv_scale(byte);
          uint32_t w = mx8::codes4(v[0][e] * inv, v[1][e] * inv, v[2][e] * inv, v[3][e] * inv);
          if (byte == 255u) w = 0;
          mine[(8 * q + e) * 8 + rq + q * 8] = w;
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
    }
    if (a.row_data || a.col_data) {
      __syncthreads();
      const int t = threadIdx.x;
      if (t < 32 && a.row_data)
        reinterpret_cast<uint4*>(a.row_scales + (tr * mx_scale_cols(a.cols) + tc) * kMxScaleTile)[t] = reinterpret_cast<const uint4*>(sh.scales[0])[t];
      if (t >= 32 && t < 64 && a.col_data)
        reinterpret_cast<uint4*>(a.col_scales + (tc * mx_scale_cols(a.rows) + tr) * kMxScaleTile)[t - 32] =
            reinterpret_cast<const uint4*>(sh.scales[1])[t - 32];
      __syncthreads();
    }
  }
  if constexpr (GRAD) {
    if (a.parts) {  // over the warp's lanes of a column, then over the four warps down the tile
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
#pragma unroll
          for (int o = 4; o < 32; o *= 2) sums[j][e] += __shfl_xor_sync(0xffffffffu, sums[j][e], o);
          if (rq == e) sh.sums[warp][j * 32 + 8 * q + e] = sums[j][e];
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
cudaError_t launch_tiles(const Mx8Args& a, cudaStream_t s) {
  const int64_t ct = (a.cols + kTile - 1) / kTile, rt = (a.rows + kTile - 1) / kTile;
  const unsigned ctas = (unsigned)(ct * ((rt + a.tiles - 1) / a.tiles));
  if (a.vec) mx8_tiles_kernel<T, GRAD, true><<<ctas, kThreads, 0, s>>>(a);
  else mx8_tiles_kernel<T, GRAD, false><<<ctas, kThreads, 0, s>>>(a);
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
