// D = act(alpha A B^T + bias) + beta C of MXFP4 matrices (kernels in mx_gemm.cuh).
#include "mx_gemm.cuh"

namespace dmuon {

using Kernels = MxKernels<4, true>;

cudaError_t mx_linear4_configure() { return Kernels::configure(); }
cudaError_t launch_mx_linear4(const MxLinearArgs& a, int nt, int split, cudaStream_t s) { return Kernels::launch(a, nt, split, s); }
cudaError_t launch_mx_linear4_pair(const MxLinearArgs& a, int pairs, cudaStream_t s) { return Kernels::launch_pair(a, pairs, s); }

}  // namespace dmuon
