// Eight consecutive elements of a row, loaded and stored by one thread, in rows
// that are 16-byte aligned (VEC) or on any element.
//
// Loads take the aligned 16-byte pieces that hold one of the wanted elements and
// shift them together: 8191 columns of bf16 cost two loads and fifteen selects for
// eight elements, where single elements would cost eight loads that touch a line a
// lane.  A row's first piece begins at most 15 bytes before it (where it does, the
// matrix does not begin an allocation); its last is cut off at the row's end, or at
// the matrix's.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <type_traits>

#include "f32x2.cuh"
#include "pieces.cuh"
#include "ptx.cuh"

namespace dmuon {

template <typename T>
constexpr int words8() { return (int)sizeof(T) * 2; }  // 32-bit words of eight elements

// Pieces of a run of eight as they are loaded; values8 puts them together.
template <typename T, bool VEC>
struct Raw8 {
  static constexpr int kWords = words8<T>() + (VEC ? 0 : 4);
  uint32_t w[kWords];
};

// The first `bytes` (a multiple of SIZE) of a 16-byte piece, zeros behind them.
template <int SIZE>
__device__ __forceinline__ uint4 load_piece(const uint4* piece, int bytes) {
  if (bytes >= 16) return *piece;
  uint32_t w[4] = {0, 0, 0, 0};
  const uint32_t* p = reinterpret_cast<const uint32_t*>(piece);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (4 * k + 4 <= bytes) w[k] = p[k];
    else if (SIZE == 2 && 4 * k + 2 <= bytes) w[k] = reinterpret_cast<const uint16_t*>(piece)[2 * k];
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// n: elements of the row from p on; those past the eighth are not wanted.
template <typename T, bool VEC>
__device__ __forceinline__ void load_raw8(Raw8<T, VEC>& r, const T* p, int n) {
  const uint32_t m = VEC ? 0u : past16(p);
  const uint4* piece = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(p) - m);
  const int bytes = (int)m + min(n, 8) * (int)sizeof(T);
#pragma unroll
  for (int i = 0; i < Raw8<T, VEC>::kWords / 4; ++i) {
    const uint4 v = load_piece<(int)sizeof(T)>(piece + i, n > 0 ? (n >= 8 + 16 / (int)sizeof(T) ? 16 : bytes - 16 * i) : 0);
    r.w[4 * i] = v.x; r.w[4 * i + 1] = v.y; r.w[4 * i + 2] = v.z; r.w[4 * i + 3] = v.w;
  }
}

// The elements as fp32, zero from the nth on.  p as in load_raw8.
template <typename T, bool VEC>
__device__ __forceinline__ void values8(float (&f)[8], Raw8<T, VEC> r, const T* p, int n) {
  constexpr int W = words8<T>();
  if constexpr (!VEC) {
    const uint32_t m = past16(p);
#pragma unroll
    for (int i = 0; i < W + 2; ++i) r.w[i] = m & 8 ? r.w[i + 2] : r.w[i];
#pragma unroll
    for (int i = 0; i < W + 1; ++i) r.w[i] = m & 4 ? r.w[i + 1] : r.w[i];
    if constexpr (sizeof(T) == 2)
#pragma unroll
      for (int i = 0; i < W; ++i) r.w[i] = __funnelshift_r(r.w[i], r.w[i + 1], (m & 2) * 8);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (sizeof(T) == 4) {
      f[e] = __uint_as_float(r.w[e]);
    } else if constexpr (std::is_same<T, __half>::value) {
      const __half2 h = *reinterpret_cast<const __half2*>(&r.w[e / 2]);
      f[e] = e & 1 ? __high2float(h) : __low2float(h);
    } else {
      f[e] = __uint_as_float(e & 1 ? r.w[e / 2] & 0xFFFF0000u : r.w[e / 2] << 16);
    }
  }
  if (n < 8)
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e >= n) f[e] = 0.f;
}

template <typename T, bool VEC>
__device__ __forceinline__ void load8(float (&f)[8], const T* p, int n) {
  Raw8<T, VEC> r;
  load_raw8<T, VEC>(r, p, n);
  values8<T, VEC>(f, r, p, n);
}

// A 16-byte piece to shared memory, the first `bytes` of it (zeros behind them).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Eight values from shared memory, where the aligned pieces around them are; m: bytes
// that the first of them is past a 16-byte boundary.  UNIFORM: it is mostly the same
// for a whole warp, so a branch is cheaper than selects.
template <typename T, bool VEC, bool UNIFORM = false>
__device__ __forceinline__ void take8(f2 (&f)[4], const uint8_t* at, uint32_t m) {
  constexpr int W = words8<T>(), N = W + (VEC ? 0 : 4);
  uint32_t w[N];
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(at + i * 4);
    w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
  }
  if constexpr (!VEC && UNIFORM) {
    uint32_t o[W];
    shift_out<W>(o, w, m);
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = o[i];
  } else if constexpr (!VEC) {
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

// 32 bytes of a row a lane, as loaded: the aligned pieces that hold one of them.
template <bool VEC>
struct Raw32 {
  uint32_t w[VEC ? 8 : 12];
};
// bytes: of the row from p on (none wanted: below 1).  END: the matrix may end with
// it, so its last piece is cut off; else 16 bytes of the matrix follow the row.
template <int SIZE, bool VEC, bool END>
__device__ __forceinline__ void load_raw32(Raw32<VEC>& r, const uint8_t* p, int bytes) {
  const uint32_t m = VEC ? 0u : past16(p);
  const uint4* piece = reinterpret_cast<const uint4*>(p - m);
  const int end = bytes > 0 ? (int)m + min(bytes, 32) : 0;
#pragma unroll
  for (int i = 0; i < (VEC ? 2 : 3); ++i) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (16 * i < end) v = END ? load_piece<SIZE>(piece + i, end - 16 * i) : piece[i];
    r.w[4 * i] = v.x; r.w[4 * i + 1] = v.y; r.w[4 * i + 2] = v.z; r.w[4 * i + 3] = v.w;
  }
}
// The values, those of the first `bytes` the row's.
template <typename T, bool VEC>
__device__ __forceinline__ void values32(f2 (&f)[16 / sizeof(T)], const Raw32<VEC>& r, const uint8_t* p) {
  uint32_t w[8];
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = r.w[i];
  } else {
    shift_out<8>(w, r.w, past16(p));
  }
#pragma unroll
  for (int k = 0; k < 16 / (int)sizeof(T); ++k) {
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

// Eight values rounded to T, as words.
template <typename T>
__device__ __forceinline__ void pack8(uint32_t* w, const float (&f)[8]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(f[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(f[2 * e], f[2 * e + 1]);
        w[e] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
        w[e] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
  }
}

// N words to p, 16-byte aligned; 32 bytes at a time where it is aligned to them.
template <int N>
__device__ __forceinline__ void store_words(uint8_t* p, const uint32_t (&w)[N]) {
  if (N % 8 == 0 && ((uintptr_t)p & 31) == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 8) ptx::st_global_v8(p + 4 * i, w + i);
    return;
  }
#pragma unroll
  for (int i = 0; i < N; i += 4) *reinterpret_cast<uint4*>(p + 4 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
}

// The first n of eight values to p, 16-byte aligned.
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8], int n) {
  uint32_t w[words8<T>()];
  pack8<T>(w, f);
  if (n >= 8) {
    store_words(reinterpret_cast<uint8_t*>(p), w);
    return;
  }
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (e < n) {
      if constexpr (sizeof(T) == 4) reinterpret_cast<uint32_t*>(p)[e] = w[e];
      else reinterpret_cast<uint16_t*>(p)[e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
    }
}

// A warp's words, N consecutive ones a lane, to a row on any element of SIZE bytes, p
// this lane's place in it.  Lane k > 0 stores the 16 bytes that its first element
// lies in, the first words of which lane k - 1 has, and those behind them; the
// elements before lane 1's and behind lane 31's pieces, fewer than eight either
// side, are stored one a lane.
template <int K, int N>
__device__ __forceinline__ void shift_up(uint32_t (&o)[N], const uint32_t (&w)[N], uint32_t sh) {  // o[i] = stream word K + i, shifted
  uint32_t s[N + 1];
#pragma unroll
  for (int i = 0; i <= N; ++i) {
    const int at = K + i;  // of the four last words of the lane before and then this lane's
    s[i] = at < 4 ? __shfl_up_sync(0xffffffffu, w[at < 4 ? N - 4 + at : 0], 1) : w[at < 4 ? 0 : at - 4];
  }
#pragma unroll
  for (int i = 0; i < N; ++i) o[i] = __funnelshift_r(s[i], s[i + 1], sh);
}
template <int SIZE, int N>
__device__ __forceinline__ void store_row(uint8_t* p, const uint32_t (&w)[N]) {
  const int lane = threadIdx.x & 31;
  const uint32_t m = __shfl_sync(0xffffffffu, past16(p), 0);
  if (m == 0) {
    store_words(p, w);
    return;
  }
  uint32_t o[N];
  const uint32_t sh = (m & 2) * 8;
  switch ((16 - m) >> 2) {
    case 0: shift_up<0>(o, w, sh); break;
    case 1: shift_up<1>(o, w, sh); break;
    case 2: shift_up<2>(o, w, sh); break;
    default: shift_up<3>(o, w, sh); break;
  }
  if (lane > 0) *reinterpret_cast<uint4*>(p - m) = make_uint4(o[0], o[1], o[2], o[3]);
#pragma unroll
  for (int i = 4; i < N; i += 4) *reinterpret_cast<uint4*>(p - m + 4 * i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
  // Element e of lane 0's first 16 bytes, or of lane 31's last.
  constexpr int kPer = 16 / SIZE;
  const int e = lane & (kPer - 1);
  const bool end = lane & kPer;
  uint32_t g[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) g[i] = __shfl_sync(0xffffffffu, lane == 31 ? w[N - 4 + i] : w[i], end ? 31 : 0);
  const int at = e * SIZE / 4;
  const uint32_t low = at & 1 ? g[1] : g[0], high = at & 1 ? g[3] : g[2], word = at & 2 ? high : low;
  if (lane < 2 * kPer && (end ? e * SIZE >= 16 - (int)m : e * SIZE < 16 - (int)m)) {
    uint8_t* to = p - lane * 4 * N + (end ? 32 * 4 * N - 16 : 0) + e * SIZE;
    if constexpr (SIZE == 4) *reinterpret_cast<uint32_t*>(to) = word;
    else *reinterpret_cast<uint16_t*>(to) = (uint16_t)(e & 1 ? word >> 16 : word);
  }
}

// 32 bytes a lane, consecutive lanes' after one another in rows of `lanes` lanes;
// bytes: of the row from p on.  w: words 4 to 11, the rest is scratch.
template <int SIZE, bool VEC>
__device__ __forceinline__ void store32(uint8_t* p, uint32_t (&w)[16], int64_t bytes, int lane, int lanes, bool live) {
  if constexpr (VEC) {
    if (!live || bytes <= 0) return;
    if (bytes >= 32) {
      store_words(p, *reinterpret_cast<const uint32_t(*)[8]>(w + 4));
      return;
    }
#pragma unroll
    for (int e = 0; e < 32 / SIZE - 1; ++e)
      if (e * SIZE < bytes) {
        if constexpr (SIZE == 4) reinterpret_cast<uint32_t*>(p)[e] = w[4 + e];
        else reinterpret_cast<uint16_t*>(p)[e] = (uint16_t)(w[4 + e / 2] >> (16 * (e & 1)));
      }
  } else {
    if (lanes == 32 && __all_sync(0xffffffffu, live && bytes >= 32)) store_row<SIZE>(p, *reinterpret_cast<const uint32_t(*)[8]>(w + 4));
    else store_pieces<SIZE>(p, w, bytes, lane == 0, lane == lanes - 1 || bytes < 64, live);
  }
}

// 8 V consecutive values a lane, a warp's after one another, to a row on any
// element (VEC: 16-byte aligned); n: of the row from p on.
template <typename T, bool VEC, int V>
__device__ __forceinline__ void store_wide(T* p, const f2 (&f)[V][4], int n) {
  constexpr int N = words8<T>();
  uint32_t w[V * N];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 q = unpack2(f[v][i]);
      o[2 * i] = q.x;
      o[2 * i + 1] = q.y;
    }
    pack8<T>(w + v * N, o);
  }
  if (VEC) {
    if (n >= 8 * V) {
      store_words(reinterpret_cast<uint8_t*>(p), w);
      return;
    }
  } else if (__all_sync(0xffffffffu, n >= 8 * V)) {
    store_row<(int)sizeof(T)>(reinterpret_cast<uint8_t*>(p), w);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8 * V; ++e)
    if (e < n) {
      if constexpr (sizeof(T) == 4) reinterpret_cast<uint32_t*>(p)[e] = w[e];
      else reinterpret_cast<uint16_t*>(p)[e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
    }
}

// The same for a warp whose lanes hold consecutive runs of eight of one row (ROW) or
// of several; n: elements of the row from p on.  `first`, `last`, `live` as in
// store_pieces.
template <typename T, bool VEC, bool ROW = false>
__device__ __forceinline__ void store8_warp(T* p, const float (&f)[8], int64_t n, bool first, bool last, bool live) {
  if constexpr (VEC) {
    if (live) store8<T>(p, f, (int)min((int64_t)8, n));
  } else {
    if (ROW && __all_sync(0xffffffffu, live && n >= 8)) {
      uint32_t w[words8<T>()];
      pack8<T>(w, f);
      store_row<(int)sizeof(T)>(reinterpret_cast<uint8_t*>(p), w);
      return;
    }
    constexpr int W = words8<T>();
    uint32_t w[W + 8];
    pack8<T>(w + 4, f);
    store_pieces<sizeof(T)>(reinterpret_cast<uint8_t*>(p), w, n * (int64_t)sizeof(T), first, last || n < 16, live);
  }
}

}  // namespace dmuon
