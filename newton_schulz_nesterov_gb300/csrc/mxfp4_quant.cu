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
// contiguous bytes per row.  Bound by HBM without noise (14336 x 4096 fp32 in
// both directions 54 us, 5.5 TB/s; 16384 x 14336 bf16 134 us, 5.4 TB/s), by
// the ALU pipe with it (214 us, 4.5 TB/s).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/dmuon.h"
#include "mx.cuh"
#include "pieces.cuh"
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

// Stochastic rounding on integers.  2^-126 |v| as fp32 has E2M1's own layout
// scaled up (v < 1 is a subnormal on either side): its bits are the code with
// 22 bits of fraction, code(v) 2^22, linear inside every interval of the grid.
// The code rounds up when fraction / 2^22 > (r + 1/2) / 256, so it is
//   (bits + 2^22 - 1 - (2r + 1) 2^13) >> 22 = (4 bits - (r << 16 | 0xFF008001)) >> 24
// Scaling rounds up: a value that is not representable stays on its side of
// every threshold.  In float arithmetic (nineteen instructions an element)
// quantising 16384 x 14336 bf16 in both directions with noise took 403 us,
// this 214; byte permutes and logic then fill 77 % of the ALU pipe's slots.
// cvt.rs.satfinite.e2m1x4.f32 takes four elements and a word of random bits; its
// rule for these bits would take the place of the header's byte an element, and
// it has not been measured.
constexpr float kTiny = 1.1754943508222875e-38f;  // 2^-126

// 4 bits - threshold of an element: its code is the top byte (8 only for a
// value past 6 that rounds up).  `sel` picks the element's byte of the noise.
__device__ __forceinline__ uint32_t stochastic(float v, float inv, uint32_t noise, uint32_t sel) {
  const uint32_t bits = __float_as_uint(__fmul_ru(__fmul_ru(fabsf(v), inv), kTiny));
  return (bits << 2) - __byte_perm(noise, 0xFF008001u, 0x7054u | (sel << 8));
}

__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}

// Top bytes of eight results to eight 4-bit codes.  s0, s1 hold the elements'
// sign bits in bit 7 of their bytes (even, odd elements).
__device__ __forceinline__ uint32_t gather_codes(const uint32_t (&a)[8], uint32_t s0, uint32_t s1, int ceil_scale) {
  uint32_t even = top_bytes(a[0], a[2], a[4], a[6]), odd = top_bytes(a[1], a[3], a[5], a[7]);
  if (!ceil_scale) {  // 8 saturates
    even -= (even >> 3) & 0x01010101u;
    odd -= (odd >> 3) & 0x01010101u;
  }
  return (even | ((s0 >> 4) & 0x08080808u)) | ((odd << 4) | (s1 & 0x80808080u));
}

// Sign bytes of two pairs of 16-bit values: bytes 1 (low halves) of a, b, then
// bytes 3 (high halves) of a, b.
__device__ __forceinline__ uint32_t sign_bytes(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7351); }

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
  // Larger magnitude of each half (its sign means nothing), NaN if either is.
  static __device__ __forceinline__ uint32_t absmax(uint32_t m, uint32_t w) {
    uint32_t r;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(w));
    return r;
  }
  static __device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
  static __device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
};
template <>
struct In<__half> {
  static constexpr int kSize = 2;
  static __device__ __forceinline__ uint32_t absmax(uint32_t m, uint32_t w) {
    uint32_t r;
    asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(w));
    return r;
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

// Tile rows of SIZE-byte elements into shared memory, zero outside the matrix
// (rows and cols: those that are left of it in this tile, at most kTile).
// Rows on any element: 4-byte elements one by one; the others by the aligned
// 16-byte pieces around a row, the last of which goes to `extra` (16 bytes a
// row), and realign() shifts them into place.  A piece is cut off at the row's
// end and begins at most 15 bytes before the row, in the piece of its first byte.
// 8191 x 8191 in both directions, bf16: 54 us, with noise 87, loaded one by one
// 71 and 164; fp32 83 either way, and 777 x 2061 4.8 one by one, 6.2 by pieces.
template <int SIZE, bool NOISE>
__device__ __forceinline__ uint8_t* place(uint8_t* tile, uint32_t r, uint32_t c) {
  return tile + r * (kTile * SIZE) + (NOISE ? swz_noise(c, r) : swz<SIZE>(c, r)) * 16;
}
template <int SIZE, bool NOISE>
__device__ __forceinline__ void load_tile(uint8_t* tile, uint8_t* extra, const uint8_t* src, int64_t pitch, int rows, int cols, int vec) {
  constexpr int kChunks = kTile * SIZE / 16;  // per row
  constexpr int kPer = 16 / SIZE;
  if (vec) {
    for (int i = threadIdx.x; i < kTile * kChunks; i += kQThreads) {
      const int r = i / kChunks, c = i % kChunks;
      const int left = r < rows ? max(0, min(kPer, cols - c * kPer)) : 0;
      copy16(ptx::smem_addr(place<SIZE, NOISE>(tile, r, c)), left ? src + r * pitch + c * 16 : src, left * SIZE);
    }
  } else if constexpr (SIZE == 4) {
#pragma unroll 4
    for (int i = threadIdx.x; i < kTile * kChunks; i += kQThreads) {
      const int r = i / kChunks, c = i % kChunks;
      const int left = r < rows ? max(0, min(16, cols * SIZE - c * 16)) : 0;  // bytes
      const uint8_t* p = src + r * pitch + c * 16;
      const uint32_t dst = ptx::smem_addr(place<SIZE, NOISE>(tile, r, c));
#pragma unroll
      for (int k = 0; k < 16; k += 4)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst + k), "l"(k < left ? p + k : src), "r"(k < left ? 4u : 0u)
                     : "memory");
    }
  } else {
    auto piece = [&](uint8_t* dst, int r, int c) {
      const uint8_t* row = src + r * pitch;
      const int m = (int)((uintptr_t)row & 15);
      const int n = r < rows ? max(0, min(16, m + cols * SIZE - c * 16)) : 0;
      copy16(ptx::smem_addr(dst), n ? row - m + c * 16 : src - ((uintptr_t)src & 15), n);
    };
    for (int i = threadIdx.x; i < kTile * kChunks; i += kQThreads) {
      const int r = i / kChunks, c = i % kChunks;
      piece(place<SIZE, NOISE>(tile, r, c), r, c);
    }
    if (threadIdx.x < kTile) piece(extra + threadIdx.x * 16, threadIdx.x, kChunks);
  }
}

// A warp has whole rows: every chunk is read before one is written.
template <int SIZE, bool NOISE>
__device__ __forceinline__ void realign(uint8_t* tile, const uint8_t* extra, const uint8_t* src, int64_t pitch, int rows) {
  constexpr int kChunks = kTile * SIZE / 16, kRows = 32 / kChunks;  // rows a warp has at a time
  const int lane = threadIdx.x & 31, c = lane % kChunks;
#pragma unroll 2
  for (int r = (threadIdx.x >> 5) * kRows + lane / kChunks; r < kTile; r += kQThreads / 32 * kRows) {
    const uint32_t m = r < rows ? (uint32_t)(uintptr_t)(src + r * pitch) & 15u : 0u;
    uint8_t* dst = place<SIZE, NOISE>(tile, r, c);
    const uint4 a = *reinterpret_cast<const uint4*>(dst);
    const uint4 b = *reinterpret_cast<const uint4*>(c + 1 < kChunks ? place<SIZE, NOISE>(tile, r, c + 1) : extra + r * 16);
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = m & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = m & 4 ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], (m & 3) * 8);
    __syncwarp();
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <typename T, bool NOISE>
__device__ __forceinline__ void row_phase(const MxQuantArgs& a, const uint8_t* tile, const uint8_t* noise,
                                          uint8_t* scales, int64_t row0, int64_t col0, int rows, int cols) {
  constexpr int S = In<T>::kSize;
  const int64_t pitch = mx_pitch(a.cols);
  uint8_t* out_tile = a.row_data + row0 * pitch + col0 / kMxBlock * 16;
#pragma unroll 1
  for (int q = threadIdx.x; q < kTile * 4; q += kQThreads) {
    const uint32_t r = q >> 2, b = q & 3;
    if ((int)r >= rows || (int)b * kMxBlock >= cols) {  // padding
      scales[(r & 31) * 16 + (r >> 5) * 4 + b] = 0;
      continue;
    }
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
        if constexpr (S == 4) f[i] = __uint_as_float(w[8 * g + i]);
        else f[i] = (i & 1) ? In<T>::hi(w[4 * g + i / 2]) : In<T>::lo(w[4 * g + i / 2]);
      }
      if constexpr (NOISE) {
        const uint2 n = *reinterpret_cast<const uint2*>(noise + r * kTile + swz_noise(b * 2 + g / 2, r) * 16 + (g & 1) * 8);
        uint32_t a8[8], s0, s1;
#pragma unroll
        for (int i = 0; i < 8; ++i) a8[i] = stochastic(f[i], inv, i < 4 ? n.x : n.y, i & 3);
        if constexpr (S == 4) {
          s0 = top_bytes(w[8 * g], w[8 * g + 2], w[8 * g + 4], w[8 * g + 6]);
          s1 = top_bytes(w[8 * g + 1], w[8 * g + 3], w[8 * g + 5], w[8 * g + 7]);
        } else {
          const uint32_t p = sign_bytes(w[4 * g], w[4 * g + 1]), q = sign_bytes(w[4 * g + 2], w[4 * g + 3]);
          s0 = __byte_perm(p, q, 0x5410);
          s1 = __byte_perm(p, q, 0x7632);
        }
        out[g] = gather_codes(a8, s0, s1, a.ceil_scale);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= inv;
        out[g] = codes_nearest(f);
      }
      if (byte == 255) out[g] = 0;
    }
    *reinterpret_cast<uint4*>(out_tile + r * pitch + b * 16) = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

template <typename T, bool NOISE>
__device__ __forceinline__ void col_phase(const MxQuantArgs& a, const uint8_t* tile, const uint8_t* noise,
                                          uint8_t* scales, int64_t row0, int64_t col0, int rows, int cols) {
  constexpr int S = In<T>::kSize;
  const int64_t pitch = mx_pitch(a.rows);
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
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (S == 4) {
        const float2 v = *reinterpret_cast<const float2*>(line(8 * g + i));
        f[0][i] = v.x;
        f[1][i] = v.y;
      } else {
        f[0][i] = In<T>::lo(w[8 * g + i]);
        f[1][i] = In<T>::hi(w[8 * g + i]);
      }
    }
    if constexpr (NOISE) {
      uint32_t a8[2][8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t r = rb * 32 + 8 * g + i;
        const uint32_t n = *reinterpret_cast<const uint16_t*>(noise + r * kTile + swz_noise(pair / 8, r) * 16 + (pair % 8) * 2);
        a8[0][i] = stochastic(f[0][i], inv[0], n, 0);
        a8[1][i] = stochastic(f[1][i], inv[1], n, 1);
      }
      uint32_t s0[2], s1[2];  // signs of the even and odd rows, by column
      if constexpr (S == 4) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const auto bits = [&](int i) { return __float_as_uint(f[h][i]); };
          s0[h] = top_bytes(bits(0), bits(2), bits(4), bits(6));
          s1[h] = top_bytes(bits(1), bits(3), bits(5), bits(7));
        }
      } else {
        const uint32_t* p = w + 8 * g;
        const uint32_t e0 = sign_bytes(p[0], p[2]), e1 = sign_bytes(p[4], p[6]), o0 = sign_bytes(p[1], p[3]), o1 = sign_bytes(p[5], p[7]);
        s0[0] = __byte_perm(e0, e1, 0x5410);
        s0[1] = __byte_perm(e0, e1, 0x7632);
        s1[0] = __byte_perm(o0, o1, 0x5410);
        s1[1] = __byte_perm(o0, o1, 0x7632);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) out[h][g] = gather_codes(a8[h], s0[h], s1[h], a.ceil_scale);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[h][i] *= inv[h];
        out[h][g] = codes_nearest(f[h]);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (byte[h] == 255) out[h][g] = 0;
  }
  uint8_t* dst = a.col_data + (col0 + 2 * pair) * pitch + (row0 / kMxBlock + rb) * 16;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if ((int)pair * 2 + h < cols && (int)rb * 32 < rows)
      *reinterpret_cast<uint4*>(dst + h * pitch) = make_uint4(out[h][0], out[h][1], out[h][2], out[h][3]);
}

template <typename T, bool NOISE>
__global__ void __launch_bounds__(kQThreads, sizeof(T) == 4 ? 2 : 4) mx_quant_kernel(const MxQuantArgs a) {
  constexpr int S = In<T>::kSize;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* scales = smem;                        // rows' and columns' scale tile
  uint8_t* tile = smem + 2 * kMxScaleTile;
  uint8_t* noise = tile + kTile * kTile * S;
  const int64_t ct = (a.cols + kTile - 1) / kTile;
  const int64_t tr = blockIdx.x / ct, tc = blockIdx.x % ct;
  const int64_t row0 = tr * kTile, col0 = tc * kTile;
  const int rows = (int)min((int64_t)kTile, a.rows - row0), cols = (int)min((int64_t)kTile, a.cols - col0);
  const uint8_t* src = (const uint8_t*)a.src + (row0 * a.ld + col0) * S;
  const uint8_t* src_noise = NOISE ? a.noise + row0 * a.noise_ld + col0 : nullptr;
  uint8_t *extra = noise + (NOISE ? kTile * kTile : 0), *extra_noise = extra + kTile * 16;
  load_tile<S, false>(tile, extra, src, a.ld * S, rows, cols, a.vec);
  if constexpr (NOISE) load_tile<1, true>(noise, extra_noise, src_noise, a.noise_ld, rows, cols, a.noise_vec);
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  if ((S < 4 && !a.vec) || (NOISE && !a.noise_vec)) {
    if constexpr (S < 4)
      if (!a.vec) realign<S, false>(tile, extra, src, a.ld * S, rows);
    if constexpr (NOISE)
      if (!a.noise_vec) realign<1, true>(noise, extra_noise, src_noise, a.noise_ld, rows);
    __syncthreads();
  }
  if (a.row_data) row_phase<T, NOISE>(a, tile, noise, scales, row0, col0, rows, cols);
  if (a.col_data) col_phase<T, NOISE>(a, tile, noise, scales + kMxScaleTile, row0, col0, rows, cols);
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
// 2^126); the product with the block's 2^e is exact, or Inf past fp32's range
// (4 or 6 times 2^126, 2 or more times 2^127).
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

// A lane reads the codes of 32 bytes of output (16 or 8 elements, all of one
// block) and stores them whole, four rows 8 apart in flight.  ANY: rows of dst on
// any element, by aligned pieces (8191 x 8191 bf16 40 us, fp32 56; two elements
// a lane, stored side by side, took 71 and 68).  Short rows share a warp.
constexpr int kDqRows = 32;  // per CTA: 8 warps x 4 rows, 32 / lanes times as many short ones
template <typename T>
constexpr int dq_cols() { return 32 * 32 / (int)sizeof(T); }

template <typename T>
__device__ __forceinline__ uint32_t value_word(uint32_t codes, float s) {  // the first one or two codes
  if constexpr (sizeof(T) == 4) return __float_as_uint(code_value(codes, s));
  const T lo = narrow<T>(code_value(codes, s)), hi = narrow<T>(code_value(codes >> 4, s));
  return (uint32_t)*reinterpret_cast<const uint16_t*>(&lo) | ((uint32_t)*reinterpret_cast<const uint16_t*>(&hi) << 16);
}

template <typename T, bool ANY>
__global__ void __launch_bounds__(256) mx_dequant_kernel(const MxDequantArgs a, int lanes) {  // lanes of a row: a power of two
  constexpr int kPer = 32 / (int)sizeof(T);  // elements a lane
  const int64_t ct = (a.k + dq_cols<T>() - 1) / dq_cols<T>();
  const int at_once = 256 / lanes, lane = threadIdx.x & (lanes - 1);
  const int64_t row0 = (int64_t)(blockIdx.x / ct) * 4 * at_once + threadIdx.x / lanes;
  const int64_t col = (int64_t)(blockIdx.x % ct) * dq_cols<T>() + lane * kPer;
  if (!ANY && col >= a.k) return;
  const int64_t pitch = mx_pitch(a.k), blk = col / kMxBlock, sc = mx_scale_cols(a.k);
  uint32_t q[4][kPer / 8] = {};
  uint32_t byte[4] = {};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = row0 + at_once * i;
    if (r >= a.rows || (ANY && col >= a.k)) continue;
    const uint32_t* src = reinterpret_cast<const uint32_t*>(a.data + r * pitch + col / 2);
    if constexpr (kPer == 16) {
      const uint2 v = *reinterpret_cast<const uint2*>(src);
      q[i][0] = v.x;
      q[i][kPer / 8 - 1] = v.y;
    } else {
      q[i][0] = *src;
    }
    byte[i] = a.scales[((r >> 7) * sc + (blk >> 2)) * kMxScaleTile + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (blk & 3)];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = row0 + at_once * i;
    if (!ANY && r >= a.rows) continue;
    const float s = scale_value(byte[i]);
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[4 + j] = value_word<T>(q[i][kPer == 16 ? j / 4 : 0] >> (kPer == 16 ? 8 * (j & 3) : 4 * j), s);
    T* dst = (T*)a.dst + r * a.ld + col;
    const int64_t left = (a.k - col) * (int64_t)sizeof(T);
    if constexpr (ANY) {
      store_pieces<sizeof(T)>(reinterpret_cast<uint8_t*>(dst), w, left, lane == 0, lane == lanes - 1 || left < 64, r < a.rows);
    } else if (left >= 32) {
      ptx::st_global_v8(dst, *reinterpret_cast<uint32_t(*)[8]>(w + 4));
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

// whole: rows are loaded by whole chunks, without the last pieces around them.
template <typename T, bool NOISE>
constexpr int quant_bytes(bool whole) {
  return 2 * kMxScaleTile + kTile * kTile * ((int)sizeof(T) + (NOISE ? 1 : 0)) + (whole ? 0 : 2 * kTile * 16);
}
// The limit belongs to the kernel on its device, not to a call: set once, to the larger.
template <typename T, bool NOISE>
cudaError_t configure_quant() {
  return cudaFuncSetAttribute(mx_quant_kernel<T, NOISE>, cudaFuncAttributeMaxDynamicSharedMemorySize, quant_bytes<T, NOISE>(false));
}

template <typename T, bool NOISE>
cudaError_t launch_quant_one(const MxQuantArgs& a, cudaStream_t s) {
  const int64_t tiles = (a.rows + kTile - 1) / kTile * ((a.cols + kTile - 1) / kTile);
  const int smem = quant_bytes<T, NOISE>((sizeof(T) == 4 || a.vec) && (!NOISE || a.noise_vec));
  mx_quant_kernel<T, NOISE><<<(unsigned)tiles, kQThreads, smem, s>>>(a);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_quant(const MxQuantArgs& a, cudaStream_t s) {
  return a.noise ? launch_quant_one<T, true>(a, s) : launch_quant_one<T, false>(a, s);
}

template <typename T>
cudaError_t launch_dequant(const MxDequantArgs& a, cudaStream_t s) {
  int lanes = 1;
  while (lanes < 32 && lanes * 32 / (int)sizeof(T) < a.k) lanes *= 2;
  const int64_t rows = kDqRows * (32 / lanes);
  const int64_t tiles = (a.rows + rows - 1) / rows * ((a.k + dq_cols<T>() - 1) / dq_cols<T>());
  if (a.vec) mx_dequant_kernel<T, false><<<(unsigned)tiles, 256, 0, s>>>(a, lanes);
  else mx_dequant_kernel<T, true><<<(unsigned)tiles, 256, 0, s>>>(a, lanes);
  return cudaGetLastError();
}

}  // namespace

cudaError_t mx_quant_configure() {
  for (auto one : {configure_quant<float, true>, configure_quant<float, false>, configure_quant<__nv_bfloat16, true>,
                   configure_quant<__nv_bfloat16, false>, configure_quant<__half, true>, configure_quant<__half, false>}) {
    const cudaError_t e = one();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

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
