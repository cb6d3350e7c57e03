// add_rmsnorm.cu -- the RMS norm with the residual's addition before it, and with
// its output in 8 bits (rmsnorm.cuh with kAdd and kEight).
#include "rmsnorm.cuh"

namespace rcc {
namespace lm {

cudaError_t launch_add_rmsnorm_forward(const NormArgs& a, cudaStream_t stream) {
  if (!a.y_scales) return forward_with<kAdd>(a, stream);
  return a.residual ? forward_with<kAdd | kEight>(a, stream) : forward_with<kEight>(a, stream);
}

cudaError_t launch_add_rmsnorm_backward(const NormGradArgs& a, cudaStream_t stream,
                                        uint64_t* launches) {
  return backward_with<kAdd>(a, stream, launches);
}

}  // namespace lm
}  // namespace rcc
