// MXFP4 quantisation along rows, along columns or both in one read of the
// matrix, and reading back.
//
// Block of 32 elements x_i, amax = max |x_i|:
//   floor  e = floor(log2 amax) - 2     ceil  e = least with amax <= 6 2^e
//   (clamped to [-127, 127]; amax = 0: -127), scale byte e + 127
//   code of |x_i| 2^-e on {0, 1/2, 1, 3/2, 2, 3, 4, 6}: nearest, ties to the
//   even code, or stochastic (below); above 6 saturates
//   amax Inf or NaN: scale byte 255 (NaN), codes 0
// 2^-e is a power of two, so the scaled value is exact in fp32 and the codes
// do not depend on how it is computed.
//
// One CTA takes a 128 x 128 tile: it is read once into shared memory
// (16-byte chunks, cp.async, zero fill outside the matrix), quantised along
// its rows (thread = one block of one row) and along its columns (thread =
// one block of two adjacent columns), and each direction's scale bytes of the
// tile are exactly one 512-byte scale tile.  Both directions write 64
// contiguous bytes per row.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/dmuon.h"
#include "mxfp4.cuh"
#include "ptx.cuh"

namespace dmuon {

namespace {

constexpr int kTile = 128;
constexpr int kQThreads = 256;

// ------------------------------------------------------------ scalar pieces

// Scale byte from the bits of amax as fp32 (sign clear).
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax, int ceil_scale) {
  const uint32_t ex = amax >> 23;
  if (ex == 255) return 255;
  // amax = 1.m x 2^(ex-127): floor(log2 amax) - 2 + 127 = ex - 2; amax / 6 =
  // 2^(ex-129) x 1.m / 1.5 exceeds 2^(ex-129) when 1.m > 1.5.
  int b = (int)ex - 2;
  if (ceil_scale && (amax & 0x7FFFFFu) > 0x400000u) ++b;
  return (uint32_t)max(b, 0);
}

// 2^(127 - byte): the factor that takes a block to the E2M1 range.
__device__ __forceinline__ float inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Eight scaled values to eight codes, nearest, ties to even, saturating.
__device__ __forceinline__ uint32_t codes_nearest(const float (&f)[8]) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return w;
}

// Stochastic: w is the scaled value in steps of its grid interval (step 1/2
// below 2, 1 below 4, 2 from there), whose code is `base` + w at a grid value
// (base 0, 2, 4); the code is base + floor(w) + (256 (w - floor(w)) > r + 1/2)
// = base + ceil(w - (r + 1/2) / 256).  w is exact (a power of two times v), so
// is the difference wherever it can be near an integer (a multiple of w's own
// last place, below w), and its sign always is; adding 2^23 + base rounding
// up is the ceiling.  Step and base come from the exponent bits of v.
__device__ __forceinline__ uint32_t code_stochastic(float f, uint32_t noise, uint32_t sel) {
  const float v = fminf(fabsf(f), 6.f);
  const uint32_t ex = max(__float_as_uint(v) & 0x7F800000u, 0x3F800000u);  // 2^0, 2^1 or 2^2
  const float w = v * __uint_as_float(0x7F800000u - ex);                   // 2, 1 or 1/2
  const float top = __uint_as_float(0x4B000000u + ((ex - 0x3F800000u) >> 22));
  const float r = __uint_as_float(__byte_perm(noise, 0x4B000000u, 0x7440u | sel)) - 8388607.5f;  // byte + 1/2
  const float u = fmaxf(fmaf(r, -1.f / 256.f, w), 0.f);
  const uint32_t code = __float_as_uint(__fadd_ru(u, top)) & 7u;
  return code | ((__float_as_uint(f) >> 28) & 8u);
}

__device__ __forceinline__ uint32_t codes_stochastic(const float (&f)[8], uint32_t n0, uint32_t n1) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) w |= code_stochastic(f[i], n0, i) << (4 * i);
#pragma unroll
  for (int i = 0; i < 4; ++i) w |= code_stochastic(f[4 + i], n1, i) << (16 + 4 * i);
  return w;
}

// ------------------------------------------------------------ input types

template <typename T>
struct In;
template <>
struct In<float> {
  static constexpr int kSize = 4;
};
template <>
struct In<__nv_bfloat16> {
  static constexpr int kSize = 2;
  static __device__ __forceinline__ uint32_t absmax(uint32_t m, uint32_t w) {
    const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<__nv_bfloat162*>(&m),
                                         __habs2(*reinterpret_cast<__nv_bfloat162*>(&w)));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  static __device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
  static __device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
};
template <>
struct In<__half> {
  static constexpr int kSize = 2;
  static __device__ __forceinline__ uint32_t absmax(uint32_t m, uint32_t w) {
    const __half2 r = __hmax2_nan(*reinterpret_cast<__half2*>(&m), __habs2(*reinterpret_cast<__half2*>(&w)));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  static __device__ __forceinline__ float lo(uint32_t w) { return __low2float(*reinterpret_cast<__half2*>(&w)); }
  static __device__ __forceinline__ float hi(uint32_t w) { return __high2float(*reinterpret_cast<__half2*>(&w)); }
};

// |x| maxima as integers of the fp32 bits: NaN > Inf > every finite value.
__device__ __forceinline__ uint32_t absbits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// ------------------------------------------------------------ shared tile

// Chunk (16 bytes) c of row r of the tile is kept at position swz(c, r) of
// the row: the row phase reads the same chunk of four blocks of two rows at
// once, the column phase chunk pairs of rows r, r + 32, r + 64, r + 96, and
// either set falls on distinct banks.
template <int SIZE>
__device__ __forceinline__ uint32_t swz(uint32_t c, uint32_t r) {
  if (SIZE == 2) return c ^ (c >> 3) ^ ((r & 1u) << 1) ^ (((r >> 5) & 3u) << 1);
  return c ^ ((c >> 3) & 3u) ^ ((r & 1u) << 2) ^ (((r >> 5) & 3u) << 1);
}
__device__ __forceinline__ uint32_t swz_noise(uint32_t c, uint32_t r) { return c ^ (r & 1u); }

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// Tile rows of SIZE-byte elements into shared memory, zero outside the matrix.
template <int SIZE, bool NOISE>
__device__ __forceinline__ void load_tile(uint8_t* tile, const uint8_t* src, int64_t ld, int64_t row0, int64_t col0,
                                          int64_t rows, int64_t cols, int vec) {
  constexpr int kChunks = kTile * SIZE / 16;  // per row
  constexpr int kPer = 16 / SIZE;
  for (int i = threadIdx.x; i < kTile * kChunks; i += kQThreads) {
    const uint32_t r = i / kChunks, c = i % kChunks;
    const int64_t row = row0 + r, col = col0 + c * kPer;
    uint8_t* dst = tile + r * (kTile * SIZE) + (NOISE ? swz_noise(c, r) : swz<SIZE>(c, r)) * 16;
    const int64_t left = row < rows ? min((int64_t)kPer, cols - col) : 0;
    const uint8_t* p = src + (row * ld + col) * SIZE;
    if (vec) {
      copy16(ptx::smem_addr(dst), left > 0 ? p : src, left > 0 ? (uint32_t)left * SIZE : 0u);
    } else {
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        if (SIZE == 4) reinterpret_cast<uint32_t*>(dst)[k] = k < left ? reinterpret_cast<const uint32_t*>(p)[k] : 0u;
        else if (SIZE == 2) reinterpret_cast<uint16_t*>(dst)[k] = k < left ? reinterpret_cast<const uint16_t*>(p)[k] : (uint16_t)0;
        else dst[k] = k < left ? p[k] : (uint8_t)0;
      }
    }
  }
}

template <typename T>
__device__ __forceinline__ void row_phase(const MxQuantArgs& a, const uint8_t* tile, const uint8_t* noise,
                                          uint8_t* scales, int64_t row0, int64_t col0) {
  constexpr int S = In<T>::kSize;
  const int64_t pitch = mx_pitch(a.cols), nb = mx_blocks(a.cols);
#pragma unroll 1
  for (int q = threadIdx.x; q < kTile * 4; q += kQThreads) {
    const uint32_t r = q >> 2, b = q & 3;
    const uint8_t* line = tile + r * (kTile * S);
    uint32_t w[8 * S];
#pragma unroll
    for (int i = 0; i < 2 * S; ++i) {
      const uint4 v = *reinterpret_cast<const uint4*>(line + swz<S>(b * 2 * S + i, r) * 16);
      w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
    }
    uint32_t amax;
    if constexpr (S == 4) {
      amax = 0;
#pragma unroll
      for (int i = 0; i < 32; ++i) amax = max(amax, w[i] & 0x7FFFFFFFu);
    } else {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) m = In<T>::absmax(m, w[i]);
      amax = max(absbits(In<T>::lo(m)), absbits(In<T>::hi(m)));
    }
    const uint32_t byte = scale_byte(amax, a.ceil_scale);
    scales[(r & 31) * 16 + (r >> 5) * 4 + b] = (uint8_t)byte;
    const float inv = inv_scale(min(byte, 254u));
    uint32_t out[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (S == 4) f[i] = __uint_as_float(w[8 * g + i]) * inv;
        else f[i] = ((i & 1) ? In<T>::hi(w[4 * g + i / 2]) : In<T>::lo(w[4 * g + i / 2])) * inv;
      }
      if (noise) {
        const uint2 n = *reinterpret_cast<const uint2*>(noise + r * kTile + swz_noise(b * 2 + g / 2, r) * 16 + (g & 1) * 8);
        out[g] = codes_stochastic(f, n.x, n.y);
      } else {
        out[g] = codes_nearest(f);
      }
      if (byte == 255) out[g] = 0;
    }
    const int64_t row = row0 + r, blk = col0 / kMxBlock + b;
    if (row < a.rows && blk < nb)
      *reinterpret_cast<uint4*>(a.row_data + row * pitch + blk * 16) = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

template <typename T>
__device__ __forceinline__ void col_phase(const MxQuantArgs& a, const uint8_t* tile, const uint8_t* noise,
                                          uint8_t* scales, int64_t row0, int64_t col0) {
  constexpr int S = In<T>::kSize;
  const int64_t pitch = mx_pitch(a.rows), nb = mx_blocks(a.rows);
  const uint32_t pair = threadIdx.x >> 2, rb = threadIdx.x & 3;  // columns 2 pair, 2 pair + 1; rows 32 rb ..
  const uint32_t chunk = pair * 2 * S / 16, at = pair * 2 * S % 16;
  auto line = [&](uint32_t j) { const uint32_t r = rb * 32 + j; return tile + r * (kTile * S) + swz<S>(chunk, r) * 16 + at; };
  uint32_t amax[2];
  uint32_t w[32];  // 16-bit types: rows' pairs
  if constexpr (S == 4) {
    amax[0] = amax[1] = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const uint2 v = *reinterpret_cast<const uint2*>(line(j));
      amax[0] = max(amax[0], v.x & 0x7FFFFFFFu);
      amax[1] = max(amax[1], v.y & 0x7FFFFFFFu);
    }
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      w[j] = *reinterpret_cast<const uint32_t*>(line(j));
      m = In<T>::absmax(m, w[j]);
    }
    amax[0] = absbits(In<T>::lo(m));
    amax[1] = absbits(In<T>::hi(m));
  }
  uint32_t byte[2];
  float inv[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    byte[h] = scale_byte(amax[h], a.ceil_scale);
    inv[h] = inv_scale(min(byte[h], 254u));
    const uint32_t r = 2 * pair + h;  // row of the transposed matrix within the tile
    scales[(r & 31) * 16 + (r >> 5) * 4 + rb] = (uint8_t)byte[h];
  }
  uint32_t out[2][4];
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    float f[2][8];
    uint32_t n[2][2] = {{0, 0}, {0, 0}};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (S == 4) {
        const float2 v = *reinterpret_cast<const float2*>(line(8 * g + i));
        f[0][i] = v.x * inv[0];
        f[1][i] = v.y * inv[1];
      } else {
        f[0][i] = In<T>::lo(w[8 * g + i]) * inv[0];
        f[1][i] = In<T>::hi(w[8 * g + i]) * inv[1];
      }
      if (noise) {
        const uint32_t r = rb * 32 + 8 * g + i;
        const uint32_t b2 = *reinterpret_cast<const uint16_t*>(noise + r * kTile + swz_noise(pair / 8, r) * 16 + (pair % 8) * 2);
        n[0][i / 4] |= (b2 & 0xFFu) << (8 * (i & 3));
        n[1][i / 4] |= (b2 >> 8) << (8 * (i & 3));
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      out[h][g] = noise ? codes_stochastic(f[h], n[h][0], n[h][1]) : codes_nearest(f[h]);
      if (byte[h] == 255) out[h][g] = 0;
    }
  }
  const int64_t blk = row0 / kMxBlock + rb;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t col = col0 + 2 * pair + h;
    if (col < a.cols && blk < nb)
      *reinterpret_cast<uint4*>(a.col_data + col * pitch + blk * 16) = make_uint4(out[h][0], out[h][1], out[h][2], out[h][3]);
  }
}

template <typename T>
__global__ void __launch_bounds__(kQThreads) mx_quant_kernel(const MxQuantArgs a) {
  constexpr int S = In<T>::kSize;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* scales = smem;                        // rows' and columns' scale tile
  uint8_t* tile = smem + 2 * kMxScaleTile;
  uint8_t* noise = a.noise ? tile + kTile * kTile * S : nullptr;
  const int64_t ct = (a.cols + kTile - 1) / kTile;
  const int64_t tr = blockIdx.x / ct, tc = blockIdx.x % ct;
  const int64_t row0 = tr * kTile, col0 = tc * kTile;
  load_tile<S, false>(tile, (const uint8_t*)a.src, a.ld, row0, col0, a.rows, a.cols, a.vec);
  if (noise) load_tile<1, true>(noise, a.noise, a.noise_ld, row0, col0, a.rows, a.cols, a.noise_vec);
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  if (a.row_data) row_phase<T>(a, tile, noise, scales, row0, col0);
  if (a.col_data) col_phase<T>(a, tile, noise, scales + kMxScaleTile, row0, col0);
  __syncthreads();
  const int t = threadIdx.x;
  if (t < 32 && a.row_data)
    reinterpret_cast<uint4*>(a.row_scales + (tr * mx_scale_cols(a.cols) + tc) * kMxScaleTile)[t] =
        reinterpret_cast<const uint4*>(scales)[t];
  if (t >= 32 && t < 64 && a.col_data)
    reinterpret_cast<uint4*>(a.col_scales + (tc * mx_scale_cols(a.rows) + tr) * kMxScaleTile)[t - 32] =
        reinterpret_cast<const uint4*>(scales + kMxScaleTile)[t - 32];
}

// ------------------------------------------------------------ reading back

// A code as fp32 is sign, two exponent bits and one mantissa bit moved to
// fp32's places and scaled by 2^126 (code 1, 0.5, is then a subnormal times
// 2^126); the product with the block's 2^e is exact.
__device__ __forceinline__ float code_value(uint32_t code, float scale) {
  const float v = __uint_as_float(((code & 8u) << 28) | ((code & 7u) << 22)) * 8.507059173023462e37f;
  return v * scale;
}

__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7FFFFFFFu : (byte == 0u ? 0x00400000u : byte << 23));
}

template <typename T>
__device__ __forceinline__ T narrow(float f);
template <>
__device__ __forceinline__ float narrow<float>(float f) { return f; }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float f) { return __float2bfloat16_rn(f); }
template <>
__device__ __forceinline__ __half narrow<__half>(float f) { return __float2half_rn(f); }

constexpr int kDqRows = 32, kDqCols = 512;  // per CTA: 8 warps x 4 rows, 32 lanes x 16 elements

template <typename T>
__global__ void __launch_bounds__(256) mx_dequant_kernel(const MxDequantArgs a) {
  const int64_t ct = (a.k + kDqCols - 1) / kDqCols;
  const int64_t row0 = (int64_t)(blockIdx.x / ct) * kDqRows + (threadIdx.x >> 5);
  const int64_t col = (int64_t)(blockIdx.x % ct) * kDqCols + (threadIdx.x & 31) * 16;
  if (col >= a.k) return;
  const int64_t pitch = mx_pitch(a.k), blk = col / kMxBlock, sc = mx_scale_cols(a.k);
  uint2 q[4];
  uint32_t byte[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = row0 + 8 * i;
    if (r >= a.rows) continue;
    q[i] = *reinterpret_cast<const uint2*>(a.data + r * pitch + col / 2);
    byte[i] = a.scales[((r >> 7) * sc + (blk >> 2)) * kMxScaleTile + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (blk & 3)];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = row0 + 8 * i;
    if (r >= a.rows) continue;
    const float s = scale_value(byte[i]);
    __align__(16) T v[16];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = narrow<T>(code_value(q[i].x >> (4 * j), s));
      v[8 + j] = narrow<T>(code_value(q[i].y >> (4 * j), s));
    }
    T* dst = (T*)a.dst + r * a.ld + col;
    if (a.vec && col + 16 <= a.k) {
#pragma unroll
      for (int j = 0; j < (int)sizeof(T); ++j) reinterpret_cast<uint4*>(dst)[j] = reinterpret_cast<const uint4*>(v)[j];
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (col + j < a.k) dst[j] = v[j];
    }
  }
}

template <typename T>
cudaError_t launch_quant(const MxQuantArgs& a, cudaStream_t s) {
  const int64_t tiles = (a.rows + kTile - 1) / kTile * ((a.cols + kTile - 1) / kTile);
  const int smem = 2 * kMxScaleTile + kTile * kTile * ((int)sizeof(T) + (a.noise ? 1 : 0));
  const cudaError_t e = cudaFuncSetAttribute(mx_quant_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             2 * kMxScaleTile + kTile * kTile * ((int)sizeof(T) + 1));
  if (e != cudaSuccess) return e;
  mx_quant_kernel<T><<<(unsigned)tiles, kQThreads, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_dequant(const MxDequantArgs& a, cudaStream_t s) {
  const int64_t tiles = (a.rows + kDqRows - 1) / kDqRows * ((a.k + kDqCols - 1) / kDqCols);
  mx_dequant_kernel<T><<<(unsigned)tiles, 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mx_quant(const MxQuantArgs& a, int dtype, cudaStream_t s) {
  if (dtype == DMUON_BF16) return launch_quant<__nv_bfloat16>(a, s);
  if (dtype == DMUON_F16) return launch_quant<__half>(a, s);
  return launch_quant<float>(a, s);
}

cudaError_t launch_mx_dequant(const MxDequantArgs& a, int dtype, cudaStream_t s) {
  if (dtype == DMUON_BF16) return launch_dequant<__nv_bfloat16>(a, s);
  if (dtype == DMUON_F16) return launch_dequant<__half>(a, s);
  return launch_dequant<float>(a, s);
}

}  // namespace dmuon
