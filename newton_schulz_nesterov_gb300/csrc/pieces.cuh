// Rows on any element, by the aligned 16-byte pieces that they lie in.
#pragma once

#include <cstdint>
#include <type_traits>

namespace dmuon {

// Bytes of `p` past a 16-byte boundary.
template <typename T>
__device__ __forceinline__ uint32_t past16(const T* p) { return (uint32_t)(uintptr_t)p & 15u; }

// out[i] = the word at byte 4 i + m of w (m even, below 16).
template <int N>
__device__ __forceinline__ void shift_out(uint32_t (&out)[N], const uint32_t (&w)[N + 4], uint32_t m) {
  const uint32_t sh = (m & 2) * 8;
  auto from = [&](auto k) {
    constexpr int K = decltype(k)::value;
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = __funnelshift_r(w[K + i], w[K + i + 1], sh);
  };
  switch (m >> 2) {
    case 0: from(std::integral_constant<int, 0>()); break;
    case 1: from(std::integral_constant<int, 1>()); break;
    case 2: from(std::integral_constant<int, 2>()); break;
    default: from(std::integral_constant<int, 3>()); break;
  }
}

// 32 bytes a lane (w[4] .. w[11]; the rest is scratch) to `own`, on any element
// of SIZE (2 or 4) bytes: stored by the aligned pieces that they begin in, the
// first of which takes the last words of the lane before.  `first`: the lane
// before does not hold the 32 bytes before these; `last`: the lane after does
// not hold 32 whole bytes after these; either side then stores its own bytes.
// left: bytes of the row from `own` on (32 or more: all are stored).  All lanes
// of a warp call it; one that is not live stores nothing.
template <int SIZE>
__device__ __forceinline__ void store_pieces(uint8_t* own, uint32_t (&w)[16], int64_t left, bool first, bool last, bool live) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = __shfl_up_sync(0xffffffffu, w[8 + i], 1);
    w[12 + i] = 0;
  }
  if (!live || left <= 0) return;
  if (left < 32) {  // the row's last elements
#pragma unroll
    for (int e = 0; e < 32 / SIZE - 1; ++e)
      if (e * SIZE < left) {
        if constexpr (SIZE == 4) reinterpret_cast<uint32_t*>(own)[e] = w[4 + e];
        else reinterpret_cast<uint16_t*>(own)[e] = (uint16_t)(w[4 + e / 2] >> (16 * (e & 1)));
      }
    return;
  }
  const uint32_t m = past16(own);
  uint32_t o[12];  // words from this lane's first piece on
  if (m == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = w[4 + i];
  } else {
    shift_out<12>(o, w, 16 - m);
  }
  uint32_t* piece = reinterpret_cast<uint32_t*>(own - m);
  if (m == 0 || !first) {
    *reinterpret_cast<uint4*>(piece) = make_uint4(o[0], o[1], o[2], o[3]);
  } else {  // from byte m on
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (4 * i >= (int)m) piece[i] = o[i];
      else if (SIZE == 2 && 4 * i + 2 == (int)m) reinterpret_cast<uint16_t*>(piece)[2 * i + 1] = (uint16_t)(o[i] >> 16);
    }
  }
  *reinterpret_cast<uint4*>(piece + 4) = make_uint4(o[4], o[5], o[6], o[7]);
  if (m && last) {  // the last m bytes
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (4 * i + 4 <= (int)m) piece[8 + i] = o[8 + i];
      else if (SIZE == 2 && 4 * i + 2 == (int)m) reinterpret_cast<uint16_t*>(piece + 8)[2 * i] = (uint16_t)o[8 + i];
    }
  }
}

}  // namespace dmuon
