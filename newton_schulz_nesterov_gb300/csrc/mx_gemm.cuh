// Products of block-scaled matrices on the tensor cores, fp32 accumulators, one
// E8M0 scale per 32 elements of either operand:
//   BITS = 4  MXFP4 (tcgen05.mma kind::mxf4, K = 64 an instruction)
//   BITS = 8  MXFP8 (kind::mxf8f6f4 of E4M3, K = 32 an instruction)
//   EPI = 0   D = alpha A B^T + beta D (MXFP4 only)
//   EPI = 1   z = alpha A B^T + bias; D = act(z) + beta C, z itself to `pre`
// The kernels are the same for both formats: an instruction takes 32 bytes of K
// and a stage 128 bytes of every row, which is 256 or 128 elements.
//
// Products of two E2M1 values are multiples of 1/4 below 36, so a block's dot
// product is exact, and those of two E4M3 values have 8 bits; what is rounded is
// the fp32 accumulation and the store.
//
// Products that fill the device run on CTA pairs (below).  The others: one CTA
// computes a tile of 128 rows of P by NT rows of Q (P, Q = A, B, or B, A when A
// has few rows: the tokens are then the MMA's N and the weights fill its 128
// lanes).  Few tiles leave SMs idle while K is long, so a cluster of `split`
// CTAs may share a tile: each accumulates a run of K blocks, sends every rank
// its share of the rows of the fp32 partial tile, and each rank then adds up
// what it got, in rank order -- no workspace, no second launch, and the same
// order every time.  The shares go by bulk copies from shared memory to shared
// memory: with one remote store a value, halving K over two CTAs cost 8.4 us
// more at 512 x 512 x 512.
//
// Warps: 0 TMA producer, 1 TMEM allocator and MMA issuer, 2-5 epilogue.
// A stage is 128-byte rows of codes (128-byte swizzle) and a 512-byte scale
// tile (two at 4 bits) per 128 rows, which tcgen05.cp takes
// from shared memory to tensor memory (32 lanes x 16 bytes, repeated for the
// four warps) ahead of the MMAs that read them; tcgen05 operations of one
// thread run in order, and consecutive stages alternate between two sets of
// scale columns.  Bound by launch and latency: 512 x 512 x 512 4.3 us; one
// token, 1 x 14336 x 4096, 7.3 us for 31 MB of weights (4.3 TB/s).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "../../include/dmuon.h"
#include "act.cuh"
#include "bounded_wait.cuh"
#include "mx.cuh"
#include "ptx.cuh"

namespace dmuon {

namespace {

constexpr int kStageRow = 128;                   // bytes of a row per stage
constexpr int kPRows = 128;
constexpr int kThreads = 192;
constexpr int kPBytes = kPRows * kStageRow;      // 16 KB

template <int BITS>
struct Fmt {
  static constexpr int kStageK = kStageRow * 8 / BITS;          // elements of K per stage
  static constexpr int kInstK = kStageK / 4;                    // and per instruction
  static constexpr int kTiles = kStageK / 128;                  // scale tiles per 128 rows and stage
  static constexpr int kScaleBytes = kTiles * kMxScaleTile;
};
template <bool EPI>
using GemmArgs = typename std::conditional<EPI, MxLinearArgs, MxGemmArgs>::type;

// ------------------------------------------------------------ PTX

// Three-dimensional tile load (scale tiles).
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// One 512-byte scale tile (32 rows of 16 bytes, no swizzle) to four columns
// of all four 32-lane groups of tensor memory.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t saddr) {
  const uint64_t desc = (uint64_t)((saddr & 0x3FFFFu) >> 4) | (1ull << 16) | ((uint64_t)(128 >> 4) << 32) | (1ull << 46);
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

template <int BITS>
__device__ __forceinline__ void mma_mx(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                       uint32_t sfb, uint32_t accumulate) {
  if constexpr (BITS == 4)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// Instruction descriptor of product j of a stage: both operands E2M1 (format 1;
// E4M3: 0) and K-major, scales E8M0 (bit 23).  The data ids in bits 29-30 and 4-5
// say where in a scale word's four bytes the instruction's scales begin: it takes
// two of them at 4 bits (K = 64), one at 8 (K = 32).
template <int BITS>
__host__ __device__ constexpr uint32_t idesc_mx(int m, int n, int j) {
  const uint32_t id = BITS == 4 ? (j & 1) * 2 : j, type = BITS == 4 ? 1 : 0;
  return (id << 4) | (type << 7) | (type << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(m >> 4) << 24) | (id << 29);
}
// The scale tile of product j of a stage.
template <int BITS>
__host__ __device__ constexpr int tile_of_product(int j) { return BITS == 4 ? j / 2 : 0; }

// High word of a K-major, 128-byte-swizzled shared-memory descriptor
// (1024 bytes between groups of eight rows).
constexpr uint32_t desc_hi() { return (1024u >> 4) | (1u << 14) | (2u << 29); }
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | (1u << 16); }

// One lane of a converged warp: the warp's loops stay uniform, so addresses
// and descriptors are kept in uniform registers, which the tensor core and
// TMA instructions take.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Bulk copy of this CTA's shared memory to another's, counted on its barrier.
__device__ __forceinline__ void send(uint32_t dst_cluster, uint32_t src, uint32_t bytes, uint32_t bar_cluster) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst_cluster),
               "r"(src), "r"(bytes), "r"(bar_cluster)
               : "memory");
}

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

// 32 lanes x 96 columns of tensor memory, waited for.
__device__ __forceinline__ void tmem_ld96(uint32_t taddr, uint32_t (&v)[96]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
      "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%96];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, %75, %76, %77, %78, %79, "
      "%80, %81, %82, %83, %84, %85, %86, %87, %88, %89, %90, %91, %92, %93, %94, %95}, [%97];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
        "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
        "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31]),
        "=r"(v[32]), "=r"(v[33]), "=r"(v[34]), "=r"(v[35]), "=r"(v[36]), "=r"(v[37]), "=r"(v[38]), "=r"(v[39]),
        "=r"(v[40]), "=r"(v[41]), "=r"(v[42]), "=r"(v[43]), "=r"(v[44]), "=r"(v[45]), "=r"(v[46]), "=r"(v[47]),
        "=r"(v[48]), "=r"(v[49]), "=r"(v[50]), "=r"(v[51]), "=r"(v[52]), "=r"(v[53]), "=r"(v[54]), "=r"(v[55]),
        "=r"(v[56]), "=r"(v[57]), "=r"(v[58]), "=r"(v[59]), "=r"(v[60]), "=r"(v[61]), "=r"(v[62]), "=r"(v[63]),
        "=r"(v[64]), "=r"(v[65]), "=r"(v[66]), "=r"(v[67]), "=r"(v[68]), "=r"(v[69]), "=r"(v[70]), "=r"(v[71]),
        "=r"(v[72]), "=r"(v[73]), "=r"(v[74]), "=r"(v[75]), "=r"(v[76]), "=r"(v[77]), "=r"(v[78]), "=r"(v[79]),
        "=r"(v[80]), "=r"(v[81]), "=r"(v[82]), "=r"(v[83]), "=r"(v[84]), "=r"(v[85]), "=r"(v[86]), "=r"(v[87]),
        "=r"(v[88]), "=r"(v[89]), "=r"(v[90]), "=r"(v[91]), "=r"(v[92]), "=r"(v[93]), "=r"(v[94]), "=r"(v[95])
      : "r"(taddr), "r"(taddr + 64)
      : "memory");
}

// Arrive on a barrier of another CTA of the cluster.  What it releases are
// reads or writes of tensor memory, which are complete (tcgen05.wait) and
// ordered by tcgen05.fence; release at cluster scope would wait for a memory
// barrier besides (1200 clocks measured).
__device__ __forceinline__ void arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// ------------------------------------------------------------ geometry

constexpr int kScratch = 32 * 36;  // words of an epilogue warp's transposing scratch

template <int BITS, int NT>
struct Cfg {
  static constexpr int kQBytes = NT * kStageRow;
  static constexpr int kScaleBytes = Fmt<BITS>::kScaleBytes;
  static constexpr int kStage = kPBytes + kQBytes + 2 * kScaleBytes;  // a multiple of 1024
  static constexpr int kN = NT == 32 ? 8 : NT == 64 ? 6 : 4;  // stages
  static constexpr int kShare = kPRows * (NT + 4) * 4;      // partial rows, here and from the ranks: row pitch NT + 4 floats
  static constexpr int kEpi = kShare > 4 * kScratch * 4 ? kShare : 4 * kScratch * 4;
  static constexpr int kSmem = 1024 + kN * kStage + kEpi + 256;
  static constexpr int kTmem = NT <= 32 ? 64 : NT <= 64 ? 128 : 256;  // the accumulator, two sets of 16 scale columns
  static_assert(kStage % 1024 == 0, "128-byte swizzle atoms start on 1 KB");
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(NT + 32 <= kTmem, "tensor memory");
  static_assert(kShare <= kN * kStage, "this CTA's partial rows lie where its stages were");
};

template <typename T>
__device__ __forceinline__ float widen(T v);
template <>
__device__ __forceinline__ float widen<float>(float v) { return v; }
template <>
__device__ __forceinline__ float widen<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float widen<__half>(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ float narrow<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half narrow<__half>(float v) { return __float2half_rn(v); }

// The first n of N elements of D, `step` apart, from accumulated products;
// beta = 0 does not read D.  All are read before one is written: one by one,
// 16384 x 8191 x 512 with beta = 1 took 2663 us in bf16 and 3182 in fp32, this
// 460 and 392.
// Here they begin at (row, col) and go down a column (DOWN) or along a row.
template <int N, bool DOWN, typename T, typename F>
__device__ __forceinline__ void put(const MxGemmArgs& a, int64_t row, int64_t col, int64_t n, F acc) {
  T* d = (T*)a.d + row * a.ldd + col;
  const int64_t step = DOWN ? a.ldd : 1;
  if (a.beta == 0.f) {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (j < n) d[j * step] = narrow<T>(a.alpha * acc(j));
    return;
  }
  T old[N];
#pragma unroll
  for (int j = 0; j < N; ++j) old[j] = j < n ? d[j * step] : narrow<T>(0.f);
#pragma unroll
  for (int j = 0; j < N; ++j)
    if (j < n) d[j * step] = narrow<T>(fmaf(a.beta, widen<T>(old[j]), a.alpha * acc(j)));
}

// The same with the whole epilogue; C may be D, element by element.
template <int N, bool DOWN, typename T, typename F>
__device__ __forceinline__ void put(const MxLinearArgs& a, int64_t row, int64_t col, int64_t n, F acc) {
  T old[N];
  if (a.c) {
    const T* c = (const T*)a.c + row * a.ldc + col;
#pragma unroll
    for (int j = 0; j < N; ++j) old[j] = j < n ? c[DOWN ? j * a.ldc : j] : narrow<T>(0.f);
  }
  float f[N];
#pragma unroll
  for (int j = 0; j < N; ++j) f[j] = a.alpha * acc(j);
  if (a.bias) {
    if constexpr (DOWN) {
      const float b = n > 0 ? a.bias[col] : 0.f;
#pragma unroll
      for (int j = 0; j < N; ++j) f[j] += b;
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) f[j] += j < n ? a.bias[col + j] : 0.f;
    }
  }
  if (a.pre) {
    T* pre = (T*)a.pre + row * a.ldpre + col;
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (j < n) pre[DOWN ? j * a.ldpre : j] = narrow<T>(f[j]);
  }
  f2 g[N / 2];
#pragma unroll
  for (int j = 0; j < N / 2; ++j) g[j] = pack2(f[2 * j], f[2 * j + 1]);
  act_values(g, a.act);
#pragma unroll
  for (int j = 0; j < N / 2; ++j) {
    const float2 p = unpack2(g[j]);
    f[2 * j] = p.x;
    f[2 * j + 1] = p.y;
  }
  T* d = (T*)a.d + row * a.ldd + col;
#pragma unroll
  for (int j = 0; j < N; ++j)
    if (j < n) d[DOWN ? j * a.ldd : j] = narrow<T>(a.c ? fmaf(a.beta, widen<T>(old[j]), f[j]) : f[j]);
}

// Two values of a 32-bit word of D's type (16-bit types), or one (fp32).
template <typename T>
struct Pack;
template <>
struct Pack<float> {
  static constexpr int kPer = 1;
  static __device__ __forceinline__ uint32_t pack(const float* v) { return __float_as_uint(v[0]); }
  static __device__ __forceinline__ void unpack(uint32_t w, float* v) { v[0] = __uint_as_float(w); }
};
template <>
struct Pack<__nv_bfloat16> {
  static constexpr int kPer = 2;
  static __device__ __forceinline__ uint32_t pack(const float* v) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(v[0], v[1]);
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  static __device__ __forceinline__ void unpack(uint32_t w, float* v) {
    v[0] = __uint_as_float(w << 16);
    v[1] = __uint_as_float(w & 0xFFFF0000u);
  }
};
template <>
struct Pack<__half> {
  static constexpr int kPer = 2;
  static __device__ __forceinline__ uint32_t pack(const float* v) {
    const __half2 r = __floats2half2_rn(v[0], v[1]);
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  static __device__ __forceinline__ void unpack(uint32_t w, float* v) {
    const float2 f = __half22float2(*reinterpret_cast<__half2*>(&w));
    v[0] = f.x;
    v[1] = f.y;
  }
};

// 32 columns of D from one row a lane: rows row0 + lane, columns col0 ..
// The block passes through the warp's scratch so that the lanes of an access
// cover whole rows: with a row a lane an access touches 32 lines, and at
// 14336 x 4096 x 8192 in fp32 the stores took 33 us of 154, reading D another 20.
// Rows 16 (packed, beta = 0) or 32 words long are kept 4 words apart, so that
// 16-byte accesses by rows and by columns of lanes fall on distinct banks.
template <typename T, typename A>
__device__ __forceinline__ void store_block(const A& a, int64_t row0, int64_t col0, int64_t rows, int64_t cols,
                                            const uint32_t* v, uint32_t* scratch, int lane) {
  constexpr int kPer = Pack<T>::kPer, kWords = 32 / kPer;
  constexpr int kLanes = kWords / 4, kRows = 32 / kLanes;  // lanes a row, rows an access of 16 bytes a lane
  T* d = (T*)a.d;
  if (a.vec && col0 + 32 <= cols) {
    const int lr = lane / kLanes, lc = lane % kLanes;
    T* dst = d + (row0 + lr) * a.ldd + col0 + lc * 4 * kPer;
    const int64_t step = (int64_t)kRows * a.ldd;
    if constexpr (std::is_same<A, MxLinearArgs>::value) {
      // A copy an activation, so that the instructions that run lie together: with the
      // branch inside the unrolled loop the epilogue waited for its instructions
      // (10822 x 8548 x 318 of MXFP8 to fp32 without an activation 125 us, so 88), and
      // in two passes over the scratch, with a loop up to the activation, it took 109.
      const int64_t at_row = row0 + lr, at_col = col0 + lc * 4 * kPer;
#pragma unroll
      for (int q = 0; q < 8; ++q)
        *reinterpret_cast<uint4*>(scratch + lane * 36 + q * 4) = make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
      uint4 old[kLanes];
      if (a.c) {
        const T* c = (const T*)a.c + at_row * a.ldc + at_col;
#pragma unroll
        for (int q = 0; q < kLanes; ++q)
          old[q] = at_row + q * kRows < rows ? *reinterpret_cast<const uint4*>(c + (int64_t)(q * kRows) * a.ldc) : make_uint4(0, 0, 0, 0);
      }
      f2 bias[2 * kPer];
#pragma unroll
      for (int e = 0; e < 2 * kPer; e += 2) {
        const float4 b = a.bias ? *reinterpret_cast<const float4*>(a.bias + at_col + 2 * e) : make_float4(0.f, 0.f, 0.f, 0.f);
        bias[e] = pack2(b.x, b.y);
        bias[e + 1] = pack2(b.z, b.w);
      }
      __syncwarp();
      const uint32_t* mine = scratch + lr * 36 + lc * 4 * kPer;
      auto to_words = [&](const f2 (&g)[2 * kPer]) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float f[2];
          if constexpr (kPer == 2) {
            const float2 p = unpack2(g[k]);
            f[0] = p.x;
            f[1] = p.y;
          } else {
            const float2 p = unpack2(g[k / 2]);
            f[0] = k & 1 ? p.y : p.x;
          }
          w[k] = Pack<T>::pack(f);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
      };
      const f2 beta = both(a.beta), alpha = both(a.alpha);
      auto values = [&](auto kind) {
        constexpr int kKind = decltype(kind)::value;
        T* pre = (T*)a.pre + at_row * a.ldpre + at_col;
#pragma unroll
        for (int q = 0; q < kLanes; ++q) {
          const uint32_t* p = mine + q * kRows * 36;
          f2 g[2 * kPer];
#pragma unroll
          for (int e = 0; e < 2 * kPer; e += 2) {
            const float4 x = *reinterpret_cast<const float4*>(p + 2 * e);
            g[e] = fma2(alpha, pack2(x.x, x.y), bias[e]);
            g[e + 1] = fma2(alpha, pack2(x.z, x.w), bias[e + 1]);
          }
          const bool live = at_row + q * kRows < rows;
          if (a.pre && live) *reinterpret_cast<uint4*>(pre + (int64_t)(q * kRows) * a.ldpre) = to_words(g);
          act_values_of<kKind>(g, a.act);
          if (a.c) {
            const uint32_t o4[4] = {old[q].x, old[q].y, old[q].z, old[q].w};
            float o[4 * kPer];
#pragma unroll
            for (int k = 0; k < 4; ++k) Pack<T>::unpack(o4[k], o + k * kPer);
#pragma unroll
            for (int e = 0; e < 2 * kPer; ++e) g[e] = fma2(beta, pack2(o[2 * e], o[2 * e + 1]), g[e]);
          }
          if (live) *reinterpret_cast<uint4*>(dst + q * step) = to_words(g);
        }
      };
      if (a.act.kind == kActClamp) values(std::integral_constant<int, kActClamp>());
      else if (a.act.kind == kActGate) values(std::integral_constant<int, kActGate>());
      else values(std::integral_constant<int, kActErf>());
    } else if (a.beta == 0.f) {
#pragma unroll
      for (int q = 0; q < kLanes; ++q) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float f[2];
#pragma unroll
          for (int e = 0; e < kPer; ++e) f[e] = a.alpha * __uint_as_float(v[(q * 4 + k) * kPer + e]);
          w[k] = Pack<T>::pack(f);
        }
        *reinterpret_cast<uint4*>(scratch + lane * (kWords + 4) + q * 4) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      __syncwarp();
#pragma unroll
      for (int q = 0; q < kLanes; ++q) {
        const uint4 w = *reinterpret_cast<const uint4*>(scratch + (q * kRows + lr) * (kWords + 4) + lc * 4);
        if (row0 + q * kRows + lr < rows) *reinterpret_cast<uint4*>(dst + q * step) = w;
      }
    } else {
      uint4 old[kLanes];
#pragma unroll
      for (int q = 0; q < kLanes; ++q)
        old[q] = row0 + q * kRows + lr < rows ? *reinterpret_cast<const uint4*>(dst + q * step) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int q = 0; q < 8; ++q)
        *reinterpret_cast<uint4*>(scratch + lane * 36 + q * 4) = make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
      __syncwarp();
#pragma unroll
      for (int q = 0; q < kLanes; ++q) {
        const uint32_t* acc = scratch + (q * kRows + lr) * 36 + lc * 4 * kPer;
        uint32_t w[4] = {old[q].x, old[q].y, old[q].z, old[q].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float f[2], o[2];
          Pack<T>::unpack(w[k], o);
#pragma unroll
          for (int e = 0; e < kPer; ++e) f[e] = fmaf(a.beta, o[e], a.alpha * __uint_as_float(acc[k * kPer + e]));
          w[k] = Pack<T>::pack(f);
        }
        if (row0 + q * kRows + lr < rows) *reinterpret_cast<uint4*>(dst + q * step) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j) scratch[lane * 33 + j] = v[j];
    __syncwarp();
    if (col0 + lane < cols) {  // 16 rows in flight: with 32 the aligned path spills (70 us of 16384 x 8192 x 512 become 89)
#pragma unroll 1
      for (int r0 = 0; r0 < 32; r0 += 16)
        put<16, true, T>(a, row0 + r0, col0 + lane, rows - row0 - r0,
                         [&](int r) { return __uint_as_float(scratch[(r0 + r) * 33 + lane]); });
    }
  }
  __syncwarp();
}

// Rows [p0, p0 + r_here) x columns [q0, q0 + q_here) of the product: the sum
// of the SPLIT ranks' shares ([rank][128 / SPLIT][pitch], this rank's own at
// `mine`) in rank order, by 128 threads, four columns and several rows a
// thread in flight.
template <int SPLIT, typename T, typename A>
__device__ __forceinline__ void add_shares(const A& a, const float* mine, const float* theirs, int rank, int pitch,
                                           int r_here, int q_here, int p0, int q0, int t) {
  constexpr int kRows = kPRows / SPLIT;
  const float* from[SPLIT];
#pragma unroll
  for (int k = 0; k < SPLIT; ++k) from[k] = k == rank ? mine : theirs + k * kRows * pitch;
  auto sum_at = [&](int off) {
    float4 v[SPLIT];
#pragma unroll
    for (int k = 0; k < SPLIT; ++k) v[k] = *reinterpret_cast<const float4*>(from[k] + off);
#pragma unroll
    for (int k = 1; k < SPLIT; ++k) {
      v[0].x += v[k].x; v[0].y += v[k].y; v[0].z += v[k].z; v[0].w += v[k].w;
    }
    return v[0];
  };
  T* d = (T*)a.d;
  if (a.swapped) {  // lanes hold consecutive columns of D, four rows of it each
    const int r = t % kRows;
    if (r >= r_here) return;
#pragma unroll 2
    for (int q = t / kRows * 4; q < q_here; q += 128 / kRows * 4) {
      const float4 v = sum_at(r * pitch + q);
      const float o[4] = {v.x, v.y, v.z, v.w};
      put<4, true, T>(a, q0 + q, p0 + r, q_here - q, [&](int e) { return o[e]; });
    }
  } else {
    const int lane = t & 31;
    for (int q = lane * 4; q < q_here; q += 128) {
      T* dst = d + (int64_t)p0 * a.ldd + q0 + q;
#pragma unroll 4
      for (int r = t >> 5; r < r_here; r += 4) {
        const float4 v = sum_at(r * pitch + q);
        const float o[4] = {v.x, v.y, v.z, v.w};
        T* at = dst + (int64_t)r * a.ldd;
        if constexpr (std::is_same<A, MxLinearArgs>::value) {
          put<4, false, T>(a, p0 + r, q0 + q, q_here - q, [&](int e) { return o[e]; });
        } else if (a.vec && q + 4 <= q_here) {  // rows on 16 bytes: four columns whole
          constexpr int kPer = Pack<T>::kPer, kWords = 4 / kPer;
          uint32_t w[kWords];
          float f[4];
          if (a.beta != 0.f) {
            if constexpr (kWords == 4) {
              const uint4 x = *reinterpret_cast<const uint4*>(at);
              w[0] = x.x; w[1] = x.y; w[kWords - 2] = x.z; w[kWords - 1] = x.w;
            } else {
              const uint2 x = *reinterpret_cast<const uint2*>(at);
              w[0] = x.x; w[1] = x.y;
            }
#pragma unroll
            for (int k = 0; k < kWords; ++k) Pack<T>::unpack(w[k], f + k * kPer);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] = a.beta != 0.f ? fmaf(a.beta, f[e], a.alpha * o[e]) : a.alpha * o[e];
#pragma unroll
          for (int k = 0; k < kWords; ++k) w[k] = Pack<T>::pack(f + k * kPer);
          if constexpr (kWords == 4) *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[kWords - 2], w[kWords - 1]);
          else *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
        } else {
          put<4, false, T>(a, p0 + r, q0 + q, q_here - q, [&](int e) { return o[e]; });
        }
      }
    }
  }
}

template <int BITS, bool EPI, int NT, typename T>
__global__ void __launch_bounds__(kThreads, 1) mx_gemm_kernel(const __grid_constant__ GemmArgs<EPI> a) {
  using C = Cfg<BITS, NT>;
  using F = Fmt<BITS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stages = smem_raw + ((1024u - (ptx::smem_addr(smem_raw) & 1023u)) & 1023u);
  uint32_t* scratch = reinterpret_cast<uint32_t*>(stages + C::kN * C::kStage);  // or the ranks' partial rows
  uint64_t* full = reinterpret_cast<uint64_t*>(stages + C::kN * C::kStage + C::kEpi);
  uint64_t* empty = full + C::kN;
  uint64_t* done = empty + C::kN;       // the accumulator is complete
  uint64_t* drain = done + 1;
  uint64_t* shares = drain + 1;         // the other ranks' partial rows are here
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(shares + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint64_t tmo = a.timeout_ns ? a.timeout_ns : kWaitNs;
  const int split = (int)cluster_size(), rank = (int)ptx::cluster_ctarank();
  const int tile = blockIdx.x / split;
  const int p0 = (tile / a.q_tiles) * kPRows, q0 = (tile % a.q_tiles) * NT;
  const int q_here = min(NT, (int)a.q_rows - q0);  // columns of the accumulator that count
  // This CTA's run of K stages: the first `extra` ranks take one more (the
  // host never asks for more ranks than stages).
  const int total = (int)((a.k + F::kStageK - 1) / F::kStageK);
  const int base = total / split, extra = total % split;
  const int kb0 = rank * base + min(rank, extra), kbn = base + (rank < extra ? 1 : 0);
  // Split: rank r adds up rows [r rows, (r + 1) rows) of the tile, `pitch` floats apart.
  const int rows = kPRows / split, pitch = ((q_here + 3) & ~3) + 4;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kN; ++s) {
      ptx::mbar_init(ptx::smem_addr(full + s), 1);
      ptx::mbar_init(ptx::smem_addr(empty + s), 1);
    }
    ptx::mbar_init(ptx::smem_addr(done), 1);
    ptx::mbar_init(ptx::smem_addr(drain), 1);
    ptx::mbar_init(ptx::smem_addr(shares), 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
    if (split > 1) ptx::mbar_expect_tx(ptx::smem_addr(shares), (split - 1) * rows * pitch * 4);
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_addr(tmem_slot), C::kTmem);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (split > 1) cluster_arrive();  // this rank's barrier of shares is ready
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t full0 = ptx::smem_addr(full), empty0 = ptx::smem_addr(empty), stage0 = ptx::smem_addr(stages);

  bool have = true;     // epilogue warps: the accumulator may be read
  uint32_t issued = 0;  // warp 0: stages that are being loaded; warp 1: being multiplied
  const bool elected = elect_one();
  if (warp == 0) {
    uint32_t s = 0, ph = 0;
    for (int it = 0; it < kbn; ++it) {
      if (!bounded_wait_warp(empty0 + s * 8, ph ^ 1u, abort_flag, a.err, tmo)) break;
      if (elected) {
        const uint32_t fb = full0 + s * 8, st = stage0 + s * C::kStage;
        const int kb = kb0 + it;
        ptx::mbar_expect_tx(fb, C::kStage);
        ptx::tma_load_2d(st, &a.p_data, kb * kStageRow, p0, fb);
        ptx::tma_load_2d(st + kPBytes, &a.q_data, kb * kStageRow, q0, fb);
        tma_load_3d(st + kPBytes + C::kQBytes, &a.p_scales, 0, kb * F::kTiles, p0 / 128, fb);
        tma_load_3d(st + kPBytes + C::kQBytes + C::kScaleBytes, &a.q_scales, 0, kb * F::kTiles, q0 / 128, fb);
      }
      ++issued;
      if (++s == (uint32_t)C::kN) { s = 0; ph ^= 1u; }
    }
  } else if (warp == 1) {
    // A tile of NT < 128 is Q's only one, so every tile starts on a scale tile.
    const int last_parts = (int)((a.k - (int64_t)(total - 1) * F::kStageK + F::kInstK - 1) / F::kInstK);  // products of the last stage
    uint32_t s = 0, ph = 0;
    for (int it = 0; it < kbn; ++it) {
      if (!bounded_wait_warp(full0 + s * 8, ph, abort_flag, a.err, tmo)) break;
      ptx::tc_fence_after();
      if (elected) {
        const uint32_t st = stage0 + s * C::kStage, sc = st + kPBytes + C::kQBytes;
        const uint32_t tp = tmem + NT + (it & 1) * 16, tq = tp + 8;
#pragma unroll
        for (int t = 0; t < F::kTiles; ++t) {
          copy_scales(tp + t * 4, sc + t * kMxScaleTile);
          copy_scales(tq + t * 4, sc + C::kScaleBytes + t * kMxScaleTile);
        }
        const int parts = kb0 + it + 1 < total ? 4 : last_parts;  // products past K would only add zeros
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < parts)
            mma_mx<BITS>(tmem, ptx::desc_sw128(st + j * 32, 16, 1024), ptx::desc_sw128(st + kPBytes + j * 32, 16, 1024),
                         idesc_mx<BITS>(kPRows, NT, j), tp + tile_of_product<BITS>(j) * 4, tq + tile_of_product<BITS>(j) * 4,
                         (it | j) != 0);
        ptx::mma_commit(empty0 + s * 8);
        if (it + 1 == kbn) ptx::mma_commit(ptx::smem_addr(done));
      }
      ++issued;
      if (++s == (uint32_t)C::kN) { s = 0; ph ^= 1u; }
    }
  } else {
    have = bounded_wait_warp(ptx::smem_addr(done), 0, abort_flag, a.err, tmo);
    ptx::tc_fence_after();
  }

  // ------------------------------------------------------------ epilogue
  const int quad = warp & 3, p = quad * 32 + lane;
  if (split == 1) {
    if (warp >= 2 && have) {
#pragma unroll 1
      for (int c = 0; c < q_here; c += 32) {
        uint32_t v[32];
        ptx::tmem_ld32(tmem + ((uint32_t)(quad * 32) << 16) + c, v);
        if (!a.swapped) {
          store_block<T>(a, p0 + quad * 32, q0 + c, a.p_rows, a.q_rows, v, scratch + (warp - 2) * kScratch, lane);
        } else if (p0 + p < a.p_rows) {  // lanes hold consecutive columns of D
          put<32, true, T>(a, q0 + c, p0 + p, q_here - c, [&](int j) { return __uint_as_float(v[j]); });
        }
      }
    }
  } else {
    cluster_wait();  // every rank's barrier is
    if (warp >= 2) {
      // All MMAs of this CTA are complete, so its stages are free.
      float* mine = reinterpret_cast<float*>(stages);
      if (have) {
#pragma unroll 1
        for (int c = 0; c < q_here; c += 32) {
          uint32_t v[32];
          ptx::tmem_ld32(tmem + ((uint32_t)(quad * 32) << 16) + c, v);
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            if (c + j < q_here)
              *reinterpret_cast<uint4*>(mine + p * pitch + c + j) = make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");
      const uint32_t bytes = (uint32_t)(rows * pitch) * 4;
      const float* theirs = reinterpret_cast<const float*>(scratch);  // [rank][rows][pitch]
      const int t = threadIdx.x - 64;
      // A rank that gave up sends too (what its stages hold: the status says
      // that the product is not to be used), so that every rank's shares land.
      if (t < split && t != rank)
        send(ptx::mapa_shared(ptx::smem_addr(scratch) + rank * bytes, t), ptx::smem_addr(mine) + t * bytes, bytes,
             ptx::mapa_shared(ptx::smem_addr(shares), t));
      if (have) have = bounded_wait_warp(ptx::smem_addr(shares), 0, abort_flag, a.err, tmo);
      if (!have) bounded_wait_slow(ptx::smem_addr(shares), 0, abort_flag, a.err, false, kWaitNs);  // what is on its way lands
      if (have) {
        const int pr0 = p0 + rank * rows, r_here = min(rows, (int)a.p_rows - pr0);
        mine += rank * rows * pitch;
        if (split == 2) add_shares<2, T>(a, mine, theirs, rank, pitch, r_here, q_here, pr0, q0, t);
        else if (split == 4) add_shares<4, T>(a, mine, theirs, rank, pitch, r_here, q_here, pr0, q0, t);
        else add_shares<8, T>(a, mine, theirs, rank, pitch, r_here, q_here, pr0, q0, t);
      }
    }
    __syncwarp();
    ptx::cluster_sync();  // no rank leaves while its shares are being read or written
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (*abort_flag) {  // neither copies nor products may outlive the CTA
    if (warp == 0 && lane == 0) drain_stages(full0, C::kN, issued, abort_flag, a.err);
    if (warp == 1 && issued) {
      if (elected) ptx::mma_commit(ptx::smem_addr(drain));
      bounded_wait_slow(ptx::smem_addr(drain), 0, abort_flag, a.err, false, kWaitNs);
      __syncwarp();
    }
  }
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::kTmem);
  }
}

// ---------------------------------------------------------------------------
// CTA pairs (cta_group::2) for products that fill the device: persistent
// pairs, a 256 x 256 tile of D each, rank r holding rows [128 r, +128) of it
// in its tensor memory.  Per stage a rank loads its 128 rows of A, 128 rows of
// B, its A scales and the scales of all 256 rows of B (each rank's tensor core
// multiplies its rows by the whole of B).
//
// Scales go to tensor memory by four warps' own stores (tcgen05.st; lane l of
// each 32-lane group holds the words of rows l, l + 32, ..), not by
// tcgen05.cp: copies queue with the products.  Per stage of four products (512
// clocks) and six copies, issued by one thread they took 853 clocks, from two
// threads 690; the stores run beside the products.  From a set's last product
// to its next one goes by two barriers and the stores (several hundred
// clocks), so there are four sets of 24 scale columns.
//
// Tensor memory: two 256-column accumulators and 96 scale columns (64 at 8 bits)
// do not fit 512 columns side by side, so the accumulators share as many:
// accumulator 0 is columns [0, 256), 1 is [160, 416), the scales are from 416 on
// (8 bits: 192, 448).  The epilogue drains the shared columns of a tile first and signals that apart;
// the next tile's products begin then, while the rest is stored.
//
// Bound by the tensor cores, and by what an SM takes from L2 (about 70 bytes a
// clock: 70 KB a stage and pair in 560 clocks where the products alone are
// 512): 16384 x 14336 x 4096 to bf16 265 us, 7.26 PFLOP/s.
// ---------------------------------------------------------------------------
constexpr int kPairN = 5;
constexpr int kPairSets = 4;
// A tile's products take 18000 clocks at K = 4096; an epilogue by four warps takes
// about as many without, and 26000 with bias, GELU and two outputs (8192 x 14336 x
// 4096 of MXFP8 460 and 612 thousand clocks), so that one has eight warps (472).
template <int BITS, bool EPI>
struct Pair {
  static constexpr int kEpiWarps = EPI ? 8 : 4;
  static constexpr int kThreads = 32 * (2 + kEpiWarps + 4);
  static constexpr int kScales = Fmt<BITS>::kScaleBytes * 3;                       // A's 128 rows, B's 256
  static constexpr int kStage = (2 * kPBytes + kScales + 1023) / 1024 * 1024;      // 35 KB, 34 at 8 bits
  static constexpr int kSmem = 1024 + kPairN * kStage + kEpiWarps * kScratch * 4 + 256;
  static constexpr int kSetCols = BITS == 4 ? 24 : 16;                             // A's words from 0, B's from 8
  static constexpr int kScaleCol = 512 - kPairSets * kSetCols;                     // 416, 448
  static constexpr int kAccStride = kScaleCol - 256;                               // 160, 192
  static constexpr int kSharedCols = 256 - kAccStride;                             // 96, 64
  static_assert(kSmem <= 227 * 1024, "pair geometry");
};

// Words of this warp's 32 lanes into columns of its lane group.
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint4& a) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w)
               : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint4& a, const uint4& b) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(a.x),
               "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// The four products of a stage: shared-memory descriptors by their low
// words (the high words are the same for every operand), 32 bytes of K apart.
constexpr uint32_t kDescHi = desc_hi();
template <int BITS>
__device__ __forceinline__ void mma_mx_pair(uint32_t d, uint32_t alo, uint32_t blo, uint32_t idesc, uint32_t sfa,
                                            uint32_t sfb, uint32_t accumulate) {
  if constexpr (BITS == 4)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, %7};\n\t"
        "mov.b64 db, {%2, %7};\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], da, db, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "r"(alo), "r"(blo), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "n"(kDescHi)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, %7};\n\t"
        "mov.b64 db, {%2, %7};\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], da, db, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "r"(alo), "r"(blo), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "n"(kDescHi)
        : "memory");
}

// Tile t of a pair's walk: groups of kGroup tile rows, column by column inside
// a group, so that the pairs running together read a block of few tile rows
// by few tile columns.
constexpr int kGroup = 8;
__device__ __forceinline__ void tile_of(int t, int tm, int tn, int& m, int& n) {
  const int g = t / (kGroup * tn), rem = t - g * kGroup * tn, rows = min(kGroup, tm - g * kGroup);
  m = g * kGroup + rem % rows;
  n = rem / rows;
}

template <int BITS, bool EPI, typename T>
__global__ void __launch_bounds__(Pair<BITS, EPI>::kThreads, 1) mx_gemm_pair_kernel(const __grid_constant__ GemmArgs<EPI> a) {
  using F = Fmt<BITS>;
  using P = Pair<BITS, EPI>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stages = smem_raw + ((1024u - (ptx::smem_addr(smem_raw) & 1023u)) & 1023u);
  uint32_t* scratch = reinterpret_cast<uint32_t*>(stages + kPairN * P::kStage);
  uint64_t* full = reinterpret_cast<uint64_t*>(scratch + P::kEpiWarps * kScratch);
  uint64_t* empty = full + kPairN;
  uint64_t* tfull = empty + kPairN;     // [2] accumulator complete
  uint64_t* tempty = tfull + 2;         // [2] accumulator stored
  uint64_t* tshared = tempty + 2;       // a tile's shared columns drained
  uint64_t* sfull = tshared + 1;        // [kPairSets] both ranks' scales are in tensor memory
  uint64_t* sready = sfull + kPairSets; // [kPairN] this rank's scales are in shared memory
  uint64_t* drain = sready + kPairN;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile uint32_t* peer_gave_up = tmem_slot + 2;  // the peer stores both before the roles' last barrier
  volatile uint32_t* peer_issued = tmem_slot + 3;
  // Stages that warp 0 loads and warp 1 multiplies, for the drains only: kept
  // here, since two more registers live through the kernel cost its epilogue
  // 1 to 2 % (16384 x 8191 x 512 bf16 with beta = 1 466 -> 472 us).
  volatile uint32_t* loaded = tmem_slot + 4;
  volatile uint32_t* multiplied = tmem_slot + 5;

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint64_t tmo = a.timeout_ns ? a.timeout_ns : kWaitNs;
  const uint32_t rank = ptx::cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int tm = (int)((a.p_rows + 255) / 256), tn = a.q_tiles, tiles = tm * tn;
  const int kbn = (int)((a.k + F::kStageK - 1) / F::kStageK);
  const int last_parts = (int)((a.k - (int64_t)(kbn - 1) * F::kStageK + F::kInstK - 1) / F::kInstK);  // products of the last stage

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairN; ++s) {
      ptx::mbar_init(ptx::smem_addr(full + s), 1);
      ptx::mbar_init(ptx::smem_addr(empty + s), 1);
      ptx::mbar_init(ptx::smem_addr(sready + s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(ptx::smem_addr(tfull + i), 1);
      ptx::mbar_init(ptx::smem_addr(tempty + i), 2 * P::kEpiWarps);  // of both ranks
    }
    ptx::mbar_init(ptx::smem_addr(tshared), 2 * P::kEpiWarps);
    for (int i = 0; i < kPairSets; ++i) ptx::mbar_init(ptx::smem_addr(sfull + i), 8);  // 4 scale warps x 2 ranks
    ptx::mbar_init(ptx::smem_addr(drain), 1);
    *abort_flag = 0;
    *peer_gave_up = 0;
    *loaded = 0;
    *multiplied = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(ptx::smem_addr(tmem_slot), 512);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();  // both ranks' barriers exist before any remote signal
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const bool elected = elect_one();
    const uint32_t full0 = ptx::smem_addr(full), remote = ptx::mapa_shared(full0, 0), ready0 = ptx::smem_addr(sready);
    const uint32_t empty0 = ptx::smem_addr(empty), stage0 = ptx::smem_addr(stages);
    uint32_t s = 0, ph = 0, issued = 0;
    bool ok = true;
    for (int t = pair; ok && t < tiles; t += npairs) {
      int mt, nt;
      tile_of(t, tm, tn, mt, nt);
      const int rowA = mt * 256 + (int)rank * 128, rowB = nt * 256 + (int)rank * 128;
      for (int kb = 0; kb < kbn; ++kb) {
        if (!bounded_wait_warp(empty0 + s * 8, ph ^ 1u, abort_flag, a.err, tmo)) { ok = false; break; }
        if (elected) {
          const uint32_t st = stage0 + s * P::kStage, sc = st + 2 * kPBytes;
          ptx::mbar_expect_tx(ready0 + s * 8, P::kScales);
          if (leader) ptx::mbar_expect_tx(full0 + s * 8, 4 * kPBytes);
          tma_load_3d(sc, &a.p_scales, 0, kb * F::kTiles, rowA / 128, ready0 + s * 8);
          tma_load_3d(sc + F::kScaleBytes, &a.q_scales, 0, kb * F::kTiles, nt * 2, ready0 + s * 8);
          ptx::tma_load_2d_pair(st, &a.p_data, kb * kStageRow, rowA, remote + s * 8);
          ptx::tma_load_2d_pair(st + kPBytes, &a.q_data, kb * kStageRow, rowB, remote + s * 8);
        }
        ++issued;
        if (++s == kPairN) { s = 0; ph ^= 1u; }
      }
    }
    if (lane == 0) {
      *loaded = issued;
      if (!leader) ptx::st_cluster(ptx::mapa_shared(ptx::smem_addr(tmem_slot + 3), 0), issued);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (leader) {
      const bool elected = elect_one();
      const uint32_t full0 = ptx::smem_addr(full), empty0 = ptx::smem_addr(empty), sfull0 = ptx::smem_addr(sfull);
      const uint32_t desc0 = desc_lo(ptx::smem_addr(stages));
      uint32_t s = 0, ph = 0, set = 0, sph = 0, tc = 0, issued = 0;
      bool ok = true;
      for (int t = pair; ok && t < tiles; t += npairs, ++tc) {
        const uint32_t acc = tc & 1u;
        if (!bounded_wait_warp(ptx::smem_addr(tempty + acc), ((tc >> 1) & 1u) ^ 1u, abort_flag, a.err, tmo) ||
            (tc > 0 && !bounded_wait_warp(ptx::smem_addr(tshared), (tc - 1) & 1u, abort_flag, a.err, tmo))) { ok = false; break; }
        const uint32_t dt = tmem + acc * P::kAccStride;
        for (int kb = 0; kb < kbn; ++kb) {
          if (!bounded_wait_warp(full0 + s * 8, ph, abort_flag, a.err, tmo) ||
              !bounded_wait_warp(sfull0 + set * 8, sph, abort_flag, a.err, tmo)) { ok = false; break; }
          ptx::tc_fence_after();
          if (elected) {
            const uint32_t da = desc0 + s * (P::kStage >> 4), db = da + (kPBytes >> 4);
            const uint32_t ta = tmem + P::kScaleCol + set * P::kSetCols, tb = ta + 8;
            // A K tail: products past it would only add zeros.
            const int parts = kb + 1 < kbn ? 4 : last_parts;
            constexpr int kT = tile_of_product<BITS>(2);
            mma_mx_pair<BITS>(dt, da, db, idesc_mx<BITS>(256, 256, 0), ta, tb, kb != 0);
            if (parts > 1) mma_mx_pair<BITS>(dt, da + 2, db + 2, idesc_mx<BITS>(256, 256, 1), ta, tb, 1);
            if (parts > 2) mma_mx_pair<BITS>(dt, da + 4, db + 4, idesc_mx<BITS>(256, 256, 2), ta + kT * 4, tb + kT * 8, 1);
            if (parts > 3) mma_mx_pair<BITS>(dt, da + 6, db + 6, idesc_mx<BITS>(256, 256, 3), ta + kT * 4, tb + kT * 8, 1);
            ptx::mma_commit_multicast(empty0 + s * 8, 0x3);
            if (kb + 1 == kbn) ptx::mma_commit_multicast(ptx::smem_addr(tfull + acc), 0x3);
          }
          ++issued;
          if (++s == kPairN) { s = 0; ph ^= 1u; }
          if (++set == kPairSets) { set = 0; sph ^= 1u; }
        }
      }
      if (lane == 0) *multiplied = issued;
    }
  } else if (warp >= 2 + P::kEpiWarps) {
    // ------------------------------------------------------------ scales
    const uint32_t ready0 = ptx::smem_addr(sready), empty0 = ptx::smem_addr(empty);
    const uint32_t sfull0 = ptx::mapa_shared(ptx::smem_addr(sfull), 0);
    const uint32_t cols = tmem + ((uint32_t)((warp & 3) * 32) << 16) + P::kScaleCol;
    const int total = (tiles - pair + npairs - 1) / npairs * kbn;
    uint32_t s = 0, ph = 0, set = 0, back = 0, bph = 0;  // back: the stage whose products had the set last
    for (int it = 0; it < total; ++it) {
      if (it >= kPairSets) {
        if (!bounded_wait_warp(empty0 + back * 8, bph, abort_flag, a.err, tmo)) break;
        if (++back == kPairN) { back = 0; bph ^= 1u; }
      }
      if (!bounded_wait_warp(ready0 + s * 8, ph, abort_flag, a.err, tmo)) break;
      ptx::tc_fence_after();
      const uint4* sc = reinterpret_cast<const uint4*>(stages + s * P::kStage + 2 * kPBytes) + lane;  // 32 x 16 bytes a tile
      const uint32_t ta = cols + set * P::kSetCols;
      if constexpr (BITS == 4) {
        tmem_st8(ta, sc[0], sc[32]);             // A: first, second 128 elements of K
        tmem_st8(ta + 8, sc[64], sc[128]);       // B, first 128 elements: rows 0-127, 128-255
        tmem_st8(ta + 16, sc[96], sc[160]);      // B, second
      } else {
        tmem_st4(ta, sc[0]);                     // A
        tmem_st8(ta + 8, sc[32], sc[64]);        // B: rows 0-127, 128-255
      }
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_remote(sfull0 + set * 8);
      if (++s == kPairN) { s = 0; ph ^= 1u; }
      if (++set == kPairSets) set = 0;
    }
  } else {
    const int quad = warp & 3;
    uint32_t* mine = scratch + (warp - 2) * kScratch;
    const T* added = (const T*)a.d;  // the matrix whose tile is added
    int64_t ld_added = a.ldd;
    bool adds = a.beta != 0.f;
    if constexpr (EPI) {
      added = (const T*)a.c;
      ld_added = a.ldc;
      adds = a.c != nullptr && warp < 6;  // one of the two warps of a quarter
    }
    // A tile of it comes to L2 while its products run: whole 16-byte pieces, the
    // first of them the row's first element's.  (A tile ahead, while the one before
    // is stored, 10822 x 8548 x 318 plus C to fp32 took 206 us, so 176, without 216.)
    auto prefetch = [&](int t) {
      if (!adds || t >= tiles) return;
      int mt, nt;
      tile_of(t, tm, tn, mt, nt);
      const int64_t row = (int64_t)mt * 256 + rank * 128 + quad * 32 + lane, col0 = (int64_t)nt * 256;
      if (row >= a.p_rows) return;
      const T* old = added + row * ld_added + col0;
      const uintptr_t from = (uintptr_t)old & ~(uintptr_t)15, to = (uintptr_t)(old + min((int64_t)256, a.q_rows - col0)) & ~(uintptr_t)15;
      if (from < to)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"((uint32_t)(to - from)) : "memory");
    };
    uint32_t tc = 0;
    for (int t = pair; t < tiles; t += npairs, ++tc) {
      const uint32_t acc = tc & 1u;
      int mt, nt;
      tile_of(t, tm, tn, mt, nt);
      const int64_t row0 = (int64_t)mt * 256 + rank * 128 + quad * 32, col0 = (int64_t)nt * 256;
      prefetch(t);
      if (!bounded_wait_warp(ptx::smem_addr(tfull + acc), (tc >> 1) & 1u, abort_flag, a.err, tmo)) break;
      ptx::tc_fence_after();
      const uint32_t tq = tmem + acc * P::kAccStride + ((uint32_t)(quad * 32) << 16);
      constexpr int kShared = P::kSharedCols / 32, kRest = P::kAccStride / 32;
      const int shared0 = acc ? 0 : P::kAccStride, rest0 = acc ? P::kSharedCols : 0;
      // The shared columns first: the last 96 (8 bits: 64) of accumulator 0, the first of 1.
      if constexpr (EPI) {
        // Of the two warps of a quarter one has the shared blocks 0, 2 and the
        // others 1, 3, .., one the shared block 1 and the others 0, 2, ..: four each.
        const int h = (warp - 2) >> 2, first = (kShared + 1 - h) / 2;
        auto block = [&](int i) { return i < first ? shared0 + (h + 2 * i) * 32 : rest0 + (1 - h + 2 * (i - first)) * 32; };
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          const int c = block(i);
          uint32_t v[32];
          ptx::tmem_ld32(tq + c, v);
          if (i + 1 == first || i == 3) {
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_remote(ptx::mapa_shared(ptx::smem_addr(i == 3 ? tempty + acc : tshared), 0));
          }
          if (col0 + c < a.q_rows) store_block<T>(a, row0, col0 + c, a.p_rows, a.q_rows, v, mine, lane);
        }
      } else {
        static_assert(BITS == 4, "the product without an epilogue is MXFP4's");
        uint32_t v[P::kSharedCols];
        tmem_ld96(tq + shared0, v);
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_remote(ptx::mapa_shared(ptx::smem_addr(tshared), 0));
#pragma unroll
        for (int q = 0; q < kShared; ++q)
          if (col0 + shared0 + q * 32 < a.q_rows)
            store_block<T>(a, row0, col0 + shared0 + q * 32, a.p_rows, a.q_rows, v + q * 32, mine, lane);
#pragma unroll 1
        for (int i = 0; i < kRest; ++i) {
          const int c = rest0 + i * 32;
          uint32_t w[32];
          ptx::tmem_ld32(tq + c, w);
          if (i == kRest - 1) {
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_remote(ptx::mapa_shared(ptx::smem_addr(tempty + acc), 0));
          }
          if (col0 + c < a.q_rows) store_block<T>(a, row0, col0 + c, a.p_rows, a.q_rows, w, mine, lane);
        }
      }
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) ptx::st_cluster(ptx::mapa_shared(ptx::smem_addr(tmem_slot + 2), rank ^ 1u), 1);
  __syncwarp();
  ptx::cluster_sync();  // no rank frees tensor memory or exits while its pair is busy
  if (*abort_flag || *peer_gave_up) {  // nor while its copies or products are in flight
    if (warp == 0 && lane == 0) {
      drain_stages(ptx::smem_addr(sready), kPairN, *loaded, abort_flag, a.err);
      if (leader)
        drain_pair_stages(ptx::smem_addr(full), kPairN, *loaded, *peer_issued, 2 * kPBytes, abort_flag, a.err);
    }
    if (warp == 1 && *multiplied) {
      if (elect_one()) ptx::mma_commit_pair(ptx::smem_addr(drain));
      bounded_wait_slow(ptx::smem_addr(drain), 0, abort_flag, a.err, false, kWaitNs);
    }
    __syncthreads();
    ptx::cluster_sync();
  }
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, 512);
  }
}

// Limits of shared memory and launches of one format and epilogue.
template <int BITS, bool EPI>
struct MxKernels {
  using Args = GemmArgs<EPI>;

  template <typename T, typename F>
  static cudaError_t each_nt(F f) {
    cudaError_t e;
    if ((e = f(mx_gemm_kernel<BITS, EPI, 32, T>, Cfg<BITS, 32>::kSmem)) != cudaSuccess) return e;
    if ((e = f(mx_gemm_kernel<BITS, EPI, 64, T>, Cfg<BITS, 64>::kSmem)) != cudaSuccess) return e;
    if ((e = f(mx_gemm_kernel<BITS, EPI, 128, T>, Cfg<BITS, 128>::kSmem)) != cudaSuccess) return e;
    return f(mx_gemm_pair_kernel<BITS, EPI, T>, Pair<BITS, EPI>::kSmem);
  }

  static cudaError_t configure() {
    auto set = [](auto kernel, int bytes) { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes); };
    cudaError_t e;
    if ((e = each_nt<float>(set)) != cudaSuccess) return e;
    if ((e = each_nt<__nv_bfloat16>(set)) != cudaSuccess) return e;
    return each_nt<__half>(set);
  }

  template <typename K>
  static cudaError_t start(K kernel, const Args& a, int64_t ctas, int cluster, int threads, int smem, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)ctas, 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
  }

  template <int NT>
  static cudaError_t launch_nt(const Args& a, int split, cudaStream_t s) {
    const int64_t ctas = (a.p_rows + kPRows - 1) / kPRows * a.q_tiles * split;
    auto go = [&](auto kernel) { return start(kernel, a, ctas, split, kThreads, Cfg<BITS, NT>::kSmem, s); };
    if (a.dtype == DMUON_BF16) return go(mx_gemm_kernel<BITS, EPI, NT, __nv_bfloat16>);
    if (a.dtype == DMUON_F16) return go(mx_gemm_kernel<BITS, EPI, NT, __half>);
    return go(mx_gemm_kernel<BITS, EPI, NT, float>);
  }

  static cudaError_t launch(const Args& a, int nt, int split, cudaStream_t s) {
    if (nt == 32) return launch_nt<32>(a, split, s);
    if (nt == 64) return launch_nt<64>(a, split, s);
    return launch_nt<128>(a, split, s);
  }

  static cudaError_t launch_pair(const Args& a, int pairs, cudaStream_t s) {
    auto go = [&](auto kernel) { return start(kernel, a, 2 * (int64_t)pairs, 2, Pair<BITS, EPI>::kThreads, Pair<BITS, EPI>::kSmem, s); };
    if (a.dtype == DMUON_BF16) return go(mx_gemm_pair_kernel<BITS, EPI, __nv_bfloat16>);
    if (a.dtype == DMUON_F16) return go(mx_gemm_pair_kernel<BITS, EPI, __half>);
    return go(mx_gemm_pair_kernel<BITS, EPI, float>);
  }
};

}  // namespace

}  // namespace dmuon
