// MXFP4 product D = alpha A B^T + beta D on the block-scaled tensor cores
// (tcgen05.mma kind::mxf4, K = 64 an instruction, one E8M0 scale per 32
// elements of either operand, fp32 accumulators).
//
// Products of two E2M1 values are multiples of 1/4 below 36, so a block's dot
// product is exact; what is rounded is the fp32 accumulation over blocks and
// the store.
//
// One CTA computes a tile of 128 rows of P by NT rows of Q (P, Q = A, B, or
// B, A when A has few rows: the tokens are then the MMA's N and the weights
// fill its 128 lanes).  Few tiles leave SMs idle while K is long, so a cluster
// of `split` CTAs may share a tile: each accumulates a run of K blocks, puts
// its fp32 partial tile in its own shared memory, and each then adds up its
// share of the columns over the cluster in rank order -- no workspace, no
// second launch, and the same order every time.
//
// Warps: 0 TMA producer, 1 TMEM allocator and MMA issuer, 2-5 epilogue.
// A stage is 256 elements of K: 128-byte rows of packed codes (128-byte
// swizzle) and two 512-byte scale tiles per 128 rows, which tcgen05.cp takes
// from shared memory to tensor memory (32 lanes x 16 bytes, repeated for the
// four warps) ahead of the MMAs that read them; tcgen05 operations of one
// thread run in order, and consecutive stages alternate between two sets of
// scale columns.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/dmuon.h"
#include "bounded_wait.cuh"
#include "mxfp4.cuh"
#include "ptx.cuh"

namespace dmuon {

namespace {

constexpr int kStageK = 256;                     // elements of K per stage
constexpr int kPRows = 128;
constexpr int kThreads = 192;
constexpr int kPBytes = kPRows * kStageK / 2;    // 16 KB
constexpr int kScaleBytes = 2 * kMxScaleTile;    // per 128 rows and stage

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

__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                         uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// Instruction descriptor of kind::mxf4: both operands E2M1 (format 1) and
// K-major, scales E8M0 (bit 23); `half` selects which two of a scale word's
// four bytes the K = 64 instruction takes (data ids in bits 29-30 and 4-5).
__host__ __device__ constexpr uint32_t idesc_mxf4(int m, int n, int half) {
  return ((uint32_t)(half * 2) << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) |
         ((uint32_t)(m >> 4) << 24) | ((uint32_t)(half * 2) << 29);
}

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// ------------------------------------------------------------ geometry

template <int NT>
struct Cfg {
  static constexpr int kQBytes = NT * kStageK / 2;
  static constexpr int kQTiles = (NT + 127) / 128;          // 128-row scale tiles of Q
  static constexpr int kScales = kScaleBytes * (1 + kQTiles);
  static constexpr int kStage = kPBytes + kQBytes + kScales;  // a multiple of 1024
  static constexpr int kN = NT == 256 ? 4 : (NT == 128 ? 5 : 6);
  static constexpr int kSmem = 1024 + kN * kStage + 256;
  static constexpr int kScaleCols = 8 + 8 * kQTiles;        // of one stage
  static constexpr int kCols = NT + 2 * kScaleCols;
  static constexpr int kTmem = kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
  static constexpr int kPitch = kPRows + 1;                 // floats of a partial tile's column
  static_assert(kStage % 1024 == 0, "128-byte swizzle atoms start on 1 KB");
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(NT * kPitch * 4 <= kN * kStage, "the partial tile fits the stages");
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

// D element from an accumulated product; beta = 0 does not read D.
template <typename T>
__device__ __forceinline__ void put(const MxGemmArgs& a, T* d, float acc) {
  float v = a.alpha * acc;
  if (a.beta != 0.f) v = fmaf(a.beta, widen<T>(*d), v);
  *d = narrow<T>(v);
}

template <int NT, typename T>
__global__ void __launch_bounds__(kThreads, 1) mx_gemm_kernel(const __grid_constant__ MxGemmArgs a) {
  using C = Cfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stages = smem_raw + ((1024u - (ptx::smem_addr(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(stages + C::kN * C::kStage);
  uint64_t* empty = full + C::kN;
  uint64_t* done = empty + C::kN;       // the accumulator is complete
  uint64_t* drain = done + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t tmo = a.timeout_ns ? a.timeout_ns : kWaitNs;
  const uint32_t split = cluster_size(), rank = ptx::cluster_ctarank();
  const int tile = blockIdx.x / split;
  const int p0 = (tile / a.q_tiles) * kPRows, q0 = (tile % a.q_tiles) * NT;
  // This CTA's run of K stages: the first `extra` ranks take one more.
  const int total = (int)((a.k + kStageK - 1) / kStageK);
  const int base = total / (int)split, extra = total % (int)split;
  const int kb0 = (int)rank * base + min((int)rank, extra), kbn = base + ((int)rank < extra ? 1 : 0);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kN; ++s) {
      ptx::mbar_init(ptx::smem_addr(full + s), 1);
      ptx::mbar_init(ptx::smem_addr(empty + s), 1);
    }
    ptx::mbar_init(ptx::smem_addr(done), 1);
    ptx::mbar_init(ptx::smem_addr(drain), 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_addr(tmem_slot), C::kTmem);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  bool have = kbn > 0;  // epilogue warps: the accumulator may be read
  if (warp == 0) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (; it < kbn; ++it) {
        const uint32_t s = it % C::kN;
        if (!bounded_wait(ptx::smem_addr(empty + s), ((it / C::kN) & 1u) ^ 1u, abort_flag, a.err, tmo)) { ok = false; break; }
        const uint32_t fb = ptx::smem_addr(full + s), st = ptx::smem_addr(stages + s * C::kStage);
        const int kb = kb0 + it;
        ptx::mbar_expect_tx(fb, C::kStage);
        ptx::tma_load_2d(st, &a.p_data, kb * (kStageK / 2), p0, fb);
        ptx::tma_load_2d(st + kPBytes, &a.q_data, kb * (kStageK / 2), q0, fb);
        tma_load_3d(st + kPBytes + C::kQBytes, &a.p_scales, 0, kb * 2, p0 / 128, fb);
        tma_load_3d(st + kPBytes + C::kQBytes + kScaleBytes, &a.q_scales, 0, kb * 2, q0 / 128, fb);
      }
      if (!ok || *abort_flag) {  // no copy may land after the CTA has gone
        const int out = it < C::kN ? it : C::kN;
        for (int i = it - out; i < it; ++i)
          bounded_wait_slow(ptx::smem_addr(full + i % C::kN), (i / C::kN) & 1u, abort_flag, a.err, false, kWaitNs);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && kbn > 0) {
      // A tile of NT < 128 is Q's only one, so every tile starts on a scale tile.
      bool ok = true, issued = false;
      for (int it = 0; it < kbn; ++it) {
        const uint32_t s = it % C::kN;
        if (!bounded_wait(ptx::smem_addr(full + s), (it / C::kN) & 1u, abort_flag, a.err, tmo)) { ok = false; break; }
        ptx::tc_fence_after();
        const uint32_t st = ptx::smem_addr(stages + s * C::kStage);
        const uint32_t sc = st + kPBytes + C::kQBytes;
        const uint32_t tp = tmem + NT + (it & 1) * C::kScaleCols, tq = tp + 8;
        // Scale columns: P [k tile][4], Q [k tile][row tile][4].
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          copy_scales(tp + t * 4, sc + t * kMxScaleTile);
#pragma unroll
          for (int r = 0; r < C::kQTiles; ++r)
            copy_scales(tq + (t * C::kQTiles + r) * 4, sc + kScaleBytes + (r * 2 + t) * kMxScaleTile);
        }
        const int64_t left = a.k - (int64_t)(kb0 + it) * kStageK;  // elements of K from this stage on
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j * 64 < left)
            mma_mxf4(tmem, ptx::desc_sw128(st + j * 32, 16, 1024), ptx::desc_sw128(st + kPBytes + j * 32, 16, 1024),
                     idesc_mxf4(kPRows, NT, j & 1), tp + (j / 2) * 4, tq + (j / 2) * C::kQTiles * 4, (it | j) != 0);
        }
        issued = true;
        ptx::mma_commit(ptx::smem_addr(empty + s));
      }
      if (ok) ptx::mma_commit(ptx::smem_addr(done));
      if (issued && (!ok || *abort_flag)) {
        ptx::mma_commit(ptx::smem_addr(drain));
        bounded_wait_slow(ptx::smem_addr(drain), 0, abort_flag, a.err, false, kWaitNs);
      }
    }
  } else if (have) {
    have = bounded_wait(ptx::smem_addr(done), 0, abort_flag, a.err, tmo);
    ptx::tc_fence_after();
  }

  // ------------------------------------------------------------ epilogue
  float* part = reinterpret_cast<float*>(stages);  // [NT][kPitch], once the stages are free
  const int quad = warp & 3, p = quad * 32 + lane;
  if (split == 1) {
    if (warp >= 2 && have) {
      T* d = (T*)a.d;
#pragma unroll 1
      for (int c = 0; c < NT; c += 32) {
        if (q0 + c >= a.q_rows) break;
        if constexpr (NT >= 32) {
          uint32_t v[32];
          ptx::tmem_ld32(tmem + ((uint32_t)(quad * 32) << 16) + c, v);
          if (p0 + p < a.p_rows)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (q0 + c + j < a.q_rows)
                put<T>(a, a.swapped ? d + (q0 + c + j) * a.ldd + p0 + p : d + (p0 + p) * a.ldd + q0 + c + j,
                       __uint_as_float(v[j]));
        }
      }
    }
  } else {
    if (warp >= 2) {
      // All MMAs of this CTA are complete, so its stages are free.
#pragma unroll 1
      for (int c = 0; c < NT; c += 32) {
        uint32_t v[32];
        if (have) ptx::tmem_ld32(tmem + ((uint32_t)(quad * 32) << 16) + c, v);
#pragma unroll
        for (int j = 0; j < 32; ++j) part[(c + j) * C::kPitch + p] = have ? __uint_as_float(v[j]) : 0.f;
      }
    }
    ptx::cluster_sync();
    if (!*abort_flag) {
      // Rank r stores columns [r NT / split, (r + 1) NT / split), the sum over ranks in order.
      const int c0 = NT * (int)rank / (int)split, c1 = NT * ((int)rank + 1) / (int)split;
      const uint32_t mine = ptx::smem_addr(part);
      T* d = (T*)a.d;
      for (int i = threadIdx.x; i < (c1 - c0) * kPRows; i += kThreads) {
        const int pp = a.swapped ? i % kPRows : i / (c1 - c0), q = c0 + (a.swapped ? i / kPRows : i % (c1 - c0));
        if (p0 + pp >= a.p_rows || q0 + q >= a.q_rows) continue;
        float sum = 0.f;
        for (uint32_t r = 0; r < split; ++r)
          sum += ld_cluster(ptx::mapa_shared(mine + (q * C::kPitch + pp) * 4, r));
        put<T>(a, a.swapped ? d + (q0 + q) * a.ldd + p0 + pp : d + (p0 + pp) * a.ldd + q0 + q, sum);
      }
    }
    ptx::cluster_sync();  // a peer may still read this CTA's tile
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::kTmem);
  }
}

template <int NT, typename T>
cudaError_t configure_one() {
  return cudaFuncSetAttribute(mx_gemm_kernel<NT, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<NT>::kSmem);
}

template <int NT, typename T>
cudaError_t launch_one(const MxGemmArgs& a, int split, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)((a.p_rows + kPRows - 1) / kPRows * a.q_tiles * split), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = Cfg<NT>::kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, mx_gemm_kernel<NT, T>, a);
}

template <int NT>
cudaError_t launch_nt(const MxGemmArgs& a, int split, cudaStream_t s) {
  if (a.dtype == DMUON_BF16) return launch_one<NT, __nv_bfloat16>(a, split, s);
  if (a.dtype == DMUON_F16) return launch_one<NT, __half>(a, split, s);
  return launch_one<NT, float>(a, split, s);
}

template <int NT>
cudaError_t configure_nt() {
  cudaError_t e;
  if ((e = configure_one<NT, float>()) != cudaSuccess) return e;
  if ((e = configure_one<NT, __nv_bfloat16>()) != cudaSuccess) return e;
  return configure_one<NT, __half>();
}

}  // namespace

cudaError_t mx_gemm_configure() {
  cudaError_t e;
  if ((e = configure_nt<32>()) != cudaSuccess) return e;
  if ((e = configure_nt<64>()) != cudaSuccess) return e;
  if ((e = configure_nt<128>()) != cudaSuccess) return e;
  return configure_nt<256>();
}

cudaError_t launch_mx_gemm(const MxGemmArgs& a, int nt, int split, cudaStream_t s) {
  if (nt == 32) return launch_nt<32>(a, split, s);
  if (nt == 64) return launch_nt<64>(a, split, s);
  if (nt == 128) return launch_nt<128>(a, split, s);
  return launch_nt<256>(a, split, s);
}

}  // namespace dmuon
