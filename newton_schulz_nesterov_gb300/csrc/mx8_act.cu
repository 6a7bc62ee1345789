// MXFP8 and 16- or 32-bit gradients through an activation (kernels in mx8_tiles.cuh).
#include "mx8_tiles.cuh"

namespace dmuon {

cudaError_t mx8_act_configure() {
  cudaError_t e;
  if ((e = configure_kind<kActClamp>()) != cudaSuccess) return e;
  if ((e = configure_kind<kActGate>()) != cudaSuccess) return e;
  return configure_kind<kActErf>();
}

cudaError_t launch_mx8_act(const Mx8Args& a, int dtype, cudaStream_t s) {
  if (a.act.kind == kActClamp) return launch_kind<kActClamp>(a, dtype, s);
  if (a.act.kind == kActGate) return launch_kind<kActGate>(a, dtype, s);
  return launch_kind<kActErf>(a, dtype, s);
}

}  // namespace dmuon
