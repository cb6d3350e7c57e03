// lm_internal.h -- launch interface between the host layer of the
// language-model operators (rcc_lm_host.cpp) and their kernels
// (embedding.cu, rmsnorm.cu, add_rmsnorm.cu, rotary.cu, adamw.cu, linear_ce.cu).
// Not part of the public ABI.
#pragma once

#include <cuda_bf16.h>
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
  // the residual's addition and the output in 8 bits (add_rmsnorm.cu)
  const void* residual;  // added to x, or NULL
  void* sum;             // [tokens][dim], with a residual
  float* y_scales;       // [tokens][groups]: y is e4m3; or NULL
  size_t ld_residual;
};
cudaError_t launch_rmsnorm_forward(const NormArgs& a, cudaStream_t stream);
cudaError_t launch_add_rmsnorm_forward(const NormArgs& a, cudaStream_t stream);

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
  const void* dsum;  // the sum's own gradient (add_rmsnorm.cu)
  size_t ld_dsum;
};
size_t rmsnorm_backward_workspace(size_t tokens, size_t dim);
cudaError_t launch_rmsnorm_backward(const NormGradArgs& a, cudaStream_t stream,
                                    uint64_t* launches);
cudaError_t launch_add_rmsnorm_backward(const NormGradArgs& a, cudaStream_t stream,
                                        uint64_t* launches);

// ---- rotary positions ------------------------------------------------------------

struct RotaryRows {
  const void* in;
  void* out;
  size_t heads;
  size_t in_token, in_head, out_token, out_head;  // elements apart
};
struct RotaryArgs {
  RotaryRows q, k;        // k.heads may be 0
  const uint64_t* turns;  // [pairs]
  const void* positions;  // [tokens], or NULL: 0, 1, ...
  int64_t offset;         // added to the positions
  size_t tokens, head_dim, pairs;
  int type, index64;
  bool half, inverse;
  bool copies;            // the columns past the pairs are written too
  int wide;               // elements of a vector: 8, 4, 2 or 1, as every row allows
  float scale;
  int units, block_tokens, block_heads;  // set by the launch
};
constexpr size_t kMaxHeads = 65536;
constexpr size_t kMaxHeadDim = 8192;
cudaError_t launch_rotary(RotaryArgs a, cudaStream_t stream);

// ---- AdamW over many tensors -------------------------------------------------------

constexpr int kAdamWItem = 2048;  // elements of a tensor that are one item

struct AdamWTensor {
  const void* grad;
  float* param;
  void *m, *v;                // fp32, or e4m3 with
  float *m_scales, *v_scales;
  __nv_bfloat16* copy;        // or NULL
  uint64_t numel;
  uint8_t bf16;               // the gradient's type
  uint8_t vec;                // every buffer on a boundary of 16 bytes (8-bit states of 8)
  uint8_t wide;               // and the fp32 ones of 32
  uint8_t bulk;               // vec, and the 8-bit states on one of 16 bytes
};
struct AdamWItem {
  uint32_t tensor, chunk;
};
struct AdamWRow {             // a block's part of the norm
  double sum;
  uint32_t bad, unused;
};
struct AdamWDecision {
  uint32_t skip, step;        // step: steps taken before, its low bits
  float coef, step_size, inv_root;
};
struct AdamWArgs {
  const AdamWTensor* tensors;
  const AdamWItem* items;
  AdamWRow* rows;
  rcc_adamw_status* status;
  AdamWDecision* decision;
  uint32_t* arrived;          // blocks whose row is written; 0 between steps
  uint64_t num_items;
  int sms;                    // that the rows have room for
  bool all_bf16;              // every gradient
  uint32_t seed;
  double inv_scale64, max_norm, lr, beta1, beta2;
  float inv_scale, b1, one_minus_b1, b2, one_minus_b2, eps, decay;
  float one;                  // 1, where the compiler must not see it
};
int adamw_sms();              // of the current device
int adamw_rows(int sms);
cudaError_t launch_adamw(const AdamWArgs& a, bool eight, cudaStream_t stream, uint64_t* launches);

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
