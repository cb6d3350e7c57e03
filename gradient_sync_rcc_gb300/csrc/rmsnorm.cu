// rmsnorm.cu -- the RMS norm of one input (rmsnorm.cuh).
#include "rmsnorm.cuh"

namespace rcc {
namespace lm {

cudaError_t launch_rmsnorm_forward(const NormArgs& a, cudaStream_t stream) {
  return forward_with<0>(a, stream);
}

size_t rmsnorm_backward_workspace(size_t tokens, size_t dim) {
  const NormShape s = norm_shape(dim);
  const size_t ld = (dim + kKeepGroup - 1) / kKeepGroup * kKeepGroup;
  const int most = std::max(1, std::max(kBackThreads, kBackDirect) / norm_threads(s));
  return norm_blocks(tokens, s, most) * norm_rows_per_block(s) * ld * sizeof(float);
}

cudaError_t launch_rmsnorm_backward(const NormGradArgs& a, cudaStream_t stream,
                                    uint64_t* launches) {
  return backward_with<0>(a, stream, launches);
}

}  // namespace lm
}  // namespace rcc
