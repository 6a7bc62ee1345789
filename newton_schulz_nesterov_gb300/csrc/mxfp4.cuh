// MXFP4 matrices (OCP microscaling: blocks of 32 E2M1 elements along a row,
// one E8M0 scale each): layout, kernel arguments and host launchers.
//
// A matrix of `rows` x `k`:
//   data    row-major, pitch 16 * ceil(k / 32) bytes; element 2i in the low,
//           2i + 1 in the high half of byte i; elements past k are zero
//   scales  one byte per block, in tiles of 128 rows x 4 blocks (512 bytes),
//           tiles row-major: row r, block j of a tile at
//           (r % 32) * 16 + (r / 32) * 4 + j; bytes past the matrix are zero
// The scale tile is the order in which the tensor core takes 128 rows' scales
// of 128 elements: one 32 x 16-byte copy into tensor memory per tile.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace dmuon {

constexpr int kMxBlock = 32;          // elements per scale
constexpr int kMxScaleTile = 512;     // bytes: 128 rows x 4 blocks

__host__ __device__ inline int64_t mx_blocks(int64_t k) { return (k + kMxBlock - 1) / kMxBlock; }
__host__ __device__ inline int64_t mx_pitch(int64_t k) { return mx_blocks(k) * 16; }
__host__ __device__ inline int64_t mx_scale_cols(int64_t k) { return (mx_blocks(k) + 3) / 4; }   // tiles per row of tiles
__host__ __device__ inline int64_t mx_scale_bytes(int64_t rows, int64_t k) {
  return (rows + 127) / 128 * mx_scale_cols(k) * kMxScaleTile;
}

struct MxQuantArgs {
  const void* src;
  int64_t rows, cols, ld;      // ld in elements
  const uint8_t* noise;        // rows x cols random bytes, or nullptr
  int64_t noise_ld;
  uint8_t *row_data, *row_scales;   // rows x cols quantised along cols, or nullptr
  uint8_t *col_data, *col_scales;   // cols x rows quantised along rows, or nullptr
  int ceil_scale;
  int vec, noise_vec;          // 16-byte aligned base and pitch
};

struct MxDequantArgs {
  const uint8_t *data, *scales;
  int64_t rows, k;
  void* dst;
  int64_t ld;
  int vec;
};

// D = alpha A B^T + beta D on P (rows in the MMA's M) and Q (rows in its N):
// P = A, Q = B and D[p][q], or swapped P = B, Q = A and D[q][p].
struct MxGemmArgs {
  CUtensorMap p_data, p_scales, q_data, q_scales;
  int64_t p_rows, q_rows, k;
  void* d;
  int64_t ldd;
  float alpha, beta;
  int swapped;
  int dtype;                   // DMUON_F32 / _BF16 / _F16
  int q_tiles;
  int vec;                     // D's rows are 16-byte aligned
  int* err;
  unsigned long long timeout_ns;
};

cudaError_t launch_mx_quant(const MxQuantArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_mx_dequant(const MxDequantArgs& a, int dtype, cudaStream_t s);
// Before the launches.
cudaError_t mx_quant_configure();
cudaError_t mx_gemm_configure();
cudaError_t launch_mx_gemm(const MxGemmArgs& a, int nt, int split, cudaStream_t s);
cudaError_t launch_mx_gemm_pair(const MxGemmArgs& a, int pairs, cudaStream_t s);

}  // namespace dmuon
