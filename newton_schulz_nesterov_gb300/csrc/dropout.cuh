// Dropout from a counter-based generator: whether an element stays depends on
// seed, offset, its row and its column alone, so the mask is made again wherever
// it is wanted and stored nowhere.
//
// Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as
// 1, 2, 3", SC 2011) with the seed as key and (column / 8, row, offset) as
// counter gives eight columns 16 bits each, column 8 g + 2 j in the low and
// 8 g + 2 j + 1 in the high half of word j.  An element stays where its bits are
// at least `cut`, and is then multiplied by 65536 / (65536 - cut).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "f32x2.cuh"

namespace dmuon {

struct Drop {
  uint32_t cut;         // in the high half of a word; 0: everything stays
  float factor;
  uint32_t key[20], offset[2];  // key: of the ten rounds
};

// cut = round(65536 p); false for p that leaves nothing, or is no probability.
inline bool drop_of(float p, uint64_t seed, uint64_t offset, Drop* d) {
  if (!(p >= 0.f && p < 1.f)) return false;
  const uint32_t cut = (uint32_t)((double)p * 65536.0 + 0.5);
  if (cut >= 65536u) return false;
  d->cut = cut << 16;
  d->factor = 65536.f / (float)(65536u - cut);
  for (uint32_t i = 0; i < 10; ++i) {
    d->key[2 * i] = (uint32_t)seed + i * 0x9E3779B9u;
    d->key[2 * i + 1] = (uint32_t)(seed >> 32) + i * 0xBB67AE85u;
  }
  d->offset[0] = (uint32_t)offset;
  d->offset[1] = (uint32_t)(offset >> 32);
  return true;
}

// The four words of columns 8 group .. 8 group + 7 of a row.
__device__ __forceinline__ void philox(uint32_t (&w)[4], const Drop& d, uint32_t group, uint32_t row) {
  uint32_t c0 = group, c1 = row, c2 = d.offset[0], c3 = d.offset[1];
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ d.key[2 * i];
    c2 = (uint32_t)(a >> 32) ^ c3 ^ d.key[2 * i + 1];
    c1 = (uint32_t)b;
    c3 = (uint32_t)a;
  }
  w[0] = c0; w[1] = c1; w[2] = c2; w[3] = c3;
}

// f[i] through the mask of the group; what goes is 0, also where it was Inf or NaN.
__device__ __forceinline__ void drop8(f2 (&f)[4], const Drop& d, const uint32_t (&w)[4]) {
  const f2 factor = both(d.factor);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 p = unpack2(mul2(f[j], factor));
    f[j] = pack2((w[j] << 16) >= d.cut ? p.x : 0.f, w[j] >= d.cut ? p.y : 0.f);
  }
}
__device__ __forceinline__ void drop8(float (&f)[8], const Drop& d, const uint32_t (&w)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = (w[j] << 16) >= d.cut ? f[2 * j] * d.factor : 0.f;
    f[2 * j + 1] = w[j] >= d.cut ? f[2 * j + 1] * d.factor : 0.f;
  }
}

// out = dropout(x) (+ residual) over rows x cols.
struct DropoutArgs {
  const void *x, *res;
  void* out;
  int64_t rows, cols, ldx, ldres, ldout;
  Drop drop;
  int vec;
};
cudaError_t launch_dropout(const DropoutArgs& a, int dtype, int sms, cudaStream_t s);

}  // namespace dmuon
