// lm_internal.h -- launch interface between the host layer of the
// language-model operators (rcc_lm_host.cpp) and their kernels
// (embedding.cu, rmsnorm.cu, linear_ce.cu).  Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "rcc.h"

namespace rcc {
namespace lm {

// ---- embedding ---------------------------------------------------------------

struct EmbedArgs {
  const void* table;
  const void* ids;
  void* out;
  size_t ld_table;  // elements between rows of the table
  size_t tokens, vocab, dim;
  int table_type, out_type, ids64;
  bool vec;  // rows of whole 8-element vectors, each on a boundary of its size
  float scale;
};
cudaError_t launch_embedding_forward(const EmbedArgs& a, cudaStream_t stream);

struct EmbedGradArgs {
  const void* dout;
  const void* ids;
  void* dtable;
  void* workspace;
  size_t ld_dout;
  size_t tokens, vocab, dim;
  int dout_type, dtable_type, ids64;
  bool vec, accumulate;
  float scale;
};
size_t embedding_backward_workspace(size_t tokens, size_t vocab, size_t dim);
// *launches: kernels enqueued
cudaError_t launch_embedding_backward(const EmbedGradArgs& a, cudaStream_t stream,
                                      uint64_t* launches);

// ---- RMS norm ------------------------------------------------------------------

constexpr size_t kMaxNormDim = 32768;
constexpr size_t kKeepGroup = 128;  // columns that share one scale of the 8-bit form

struct NormArgs {
  const void* x;
  const float* weight;
  void* y;
  int8_t* kept;        // [tokens][groups * kKeepGroup], or NULL: nothing kept
  float* scales;       // [tokens][groups]
  size_t ld_x, ld_y;
  size_t tokens, dim;
  int type;
  bool vec;
  float eps;
};
cudaError_t launch_rmsnorm_forward(const NormArgs& a, cudaStream_t stream);

struct NormGradArgs {
  const void* dy;
  const int8_t* kept;
  const float* scales;
  const float* weight;
  void* dx;
  float* dweight;
  void* workspace;
  size_t ld_dy, ld_dx;
  size_t tokens, dim;
  int type;
  bool vec, accumulate;
  float eps;
};
size_t rmsnorm_backward_workspace(size_t tokens, size_t dim);
cudaError_t launch_rmsnorm_backward(const NormGradArgs& a, cudaStream_t stream,
                                    uint64_t* launches);

// ---- output layer + softmax cross entropy ----------------------------------------

struct CeArgs {
  const void* x;       // [tokens][dim] bf16
  const void* w;       // [vocab][dim] bf16
  const void* labels;  // [tokens]
  size_t ld_x, ld_w;
  size_t tokens, vocab, dim;
  int labels64;
  float* loss;         // forward: [tokens]
  float* lse;          // forward: [tokens], written; backward: read
  const float* dloss;  // backward: [tokens]
  void* dx;            // backward: [tokens][dim], or NULL
  void* dw;            // backward: [vocab][dim], or NULL
  int grad_type;
  bool accumulate;     // dw += instead of dw =
  void* workspace;
};
size_t linear_ce_workspace(size_t tokens, size_t vocab, size_t dim, bool backward, int grad_type);
cudaError_t launch_linear_ce_forward(const CeArgs& a, cudaStream_t stream, uint64_t* launches);
cudaError_t launch_linear_ce_backward(const CeArgs& a, cudaStream_t stream, uint64_t* launches);

}  // namespace lm
}  // namespace rcc
