// MXFP4 and MXFP8 matrices (OCP microscaling: blocks of 32 E2M1 or E4M3
// elements along a row, one E8M0 scale each): layout, kernel arguments and host
// launchers.
//
// A matrix of `rows` x `k`:
//   data    row-major, elements past k are zero; MXFP4: pitch 16 * ceil(k / 32)
//           bytes, element 2i in the low, 2i + 1 in the high half of byte i;
//           MXFP8: pitch 32 * ceil(k / 32) bytes
//   scales  one byte per block, in tiles of 128 rows x 4 blocks (512 bytes),
//           tiles row-major: row r, block j of a tile at
//           (r % 32) * 16 + (r / 32) * 4 + j; bytes past the matrix are zero
// The scale tile is the order in which the tensor core takes 128 rows' scales
// of 128 elements: one 32 x 16-byte copy into tensor memory per tile.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "act.cuh"
#include "mx8.cuh"

namespace dmuon {

constexpr int kMxBlock = 32;          // elements per scale
constexpr int kMxScaleTile = 512;     // bytes: 128 rows x 4 blocks

__host__ __device__ inline int64_t mx_blocks(int64_t k) { return (k + kMxBlock - 1) / kMxBlock; }
__host__ __device__ inline int64_t mx_pitch(int64_t k, int bits = 4) { return mx_blocks(k) * 4 * bits; }
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

// An MXFP8 pass over a matrix: values (src, or dout * act'(pre)) to codes by rows
// and / or by columns, to dz and to column sums.
struct Mx8Args {
  const void *src, *pre;            // pre: nullptr for a quantisation
  int64_t rows, cols, ld, ldpre;
  Act act;
  uint8_t *row_data, *row_scales;   // or nullptr
  uint8_t *col_data, *col_scales;   // or nullptr
  void* dz;                         // rows x cols of src's type, or nullptr
  int64_t lddz;
  float* parts;                     // [chunks][part_ld] column sums, or nullptr
  int64_t part_ld;
  int64_t tiles;                    // tiles of 128 rows a CTA goes down
  uint32_t up;                      // added to the bits of magnitudes (mx8.cuh)
  int vec;                          // every matrix's rows are 16-byte aligned
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

// z = alpha A B^T + bias, D = act(z) + beta C, z to pre.
struct MxLinearArgs : MxGemmArgs {
  const void* c;               // as D, or nullptr
  int64_t ldc;
  const float* bias;           // columns of D, or nullptr
  void* pre;                   // as D, or nullptr
  int64_t ldpre;
  Act act;
};

cudaError_t launch_mx_quant(const MxQuantArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_mx_dequant(const MxDequantArgs& a, int dtype, cudaStream_t s);
// Before the launches.
cudaError_t mx_quant_configure();
cudaError_t mx_gemm_configure();
cudaError_t launch_mx_gemm(const MxGemmArgs& a, int nt, int split, cudaStream_t s);
cudaError_t launch_mx_gemm_pair(const MxGemmArgs& a, int pairs, cudaStream_t s);
cudaError_t mx_linear4_configure();
cudaError_t launch_mx_linear4(const MxLinearArgs& a, int nt, int split, cudaStream_t s);
cudaError_t launch_mx_linear4_pair(const MxLinearArgs& a, int pairs, cudaStream_t s);
cudaError_t mx_linear8_configure();
cudaError_t launch_mx_linear8(const MxLinearArgs& a, int nt, int split, cudaStream_t s);
cudaError_t launch_mx_linear8_pair(const MxLinearArgs& a, int pairs, cudaStream_t s);
cudaError_t mx8_configure();
cudaError_t launch_mx8_tiles(const Mx8Args& a, int dtype, cudaStream_t s);
// dout * act'(pre) in place of src.
cudaError_t mx8_act_configure();
cudaError_t launch_mx8_act(const Mx8Args& a, int dtype, cudaStream_t s);
cudaError_t launch_mx8_dequant(const MxDequantArgs& a, int dtype, cudaStream_t s);
// out[c] = the sum over `n` rows of parts, in a fixed order.
cudaError_t launch_column_sums(const float* parts, int64_t n, int64_t ld, int64_t cols, float* out, cudaStream_t s);

}  // namespace dmuon
