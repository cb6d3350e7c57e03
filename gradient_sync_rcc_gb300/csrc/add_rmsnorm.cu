// add_rmsnorm.cu -- the RMS norm with the residual's addition before it, and with
// its output in 8 bits (rmsnorm.cuh with kAdd and kEight).
//
// Memory bound: one pass over both inputs, the sum written on the way and held in
// registers between the row's sum of squares and its outputs.  16,384 x 4,096 bf16:
// forward with the sum kept in 8 bits 91 us (606 MB, 6.6 TB/s), backward 69 and 5
// for dweight (472 MB), output in 8 bits 72 (472 MB) -- under the profiler; 170 us
// a forward and backward pass, 73 the 8-bit one, among others.
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
