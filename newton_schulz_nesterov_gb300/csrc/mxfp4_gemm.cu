// D = alpha A B^T + beta D of MXFP4 matrices (kernels in mx_gemm.cuh).
#include "mx_gemm.cuh"

namespace dmuon {

using Kernels = MxKernels<4, false>;

cudaError_t mx_gemm_configure() { return Kernels::configure(); }
cudaError_t launch_mx_gemm(const MxGemmArgs& a, int nt, int split, cudaStream_t s) { return Kernels::launch(a, nt, split, s); }
cudaError_t launch_mx_gemm_pair(const MxGemmArgs& a, int pairs, cudaStream_t s) { return Kernels::launch_pair(a, pairs, s); }

}  // namespace dmuon
