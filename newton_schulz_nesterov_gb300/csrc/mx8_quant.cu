// MXFP8 quantisation (kernels in mx8_tiles.cuh), reading back, column sums.
#include "mx8_tiles.cuh"

namespace dmuon {

namespace {

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
// 32 sums of a column, in order.  Launched ahead of the end of the kernel before
// it, which it waits for (griddepcontrol.wait: its stores are then visible).
__global__ void __launch_bounds__(1024) column_sums_kernel(const float* parts, int64_t n, int64_t ld, int64_t cols, float* out) {
  __shared__ float part[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.f;
  asm volatile("griddepcontrol.wait;" ::: "memory");
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

cudaError_t mx8_configure() { return configure_kind<kNoSlope>(); }

cudaError_t launch_mx8_tiles(const Mx8Args& a, int dtype, cudaStream_t s) { return launch_kind<kNoSlope>(a, dtype, s); }

cudaError_t launch_mx8_dequant(const MxDequantArgs& a, int dtype, cudaStream_t s) {
  if (dtype == DMUON_BF16) return launch_dequant<__nv_bfloat16>(a, s);
  if (dtype == DMUON_F16) return launch_dequant<__half>(a, s);
  return launch_dequant<float>(a, s);
}

cudaError_t launch_column_sums(const float* parts, int64_t n, int64_t ld, int64_t cols, float* out, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)((cols + 31) / 32), 1, 1);
  cfg.blockDim = dim3(1024, 1, 1);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, column_sums_kernel, parts, n, ld, cols, out);
}

}  // namespace dmuon
