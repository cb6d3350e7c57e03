// rcc_lm_host.cpp -- entry points of the language-model operators: argument
// checks and launches.  No session, no allocation, no synchronisation.
//
// Every call checks on the host before it launches anything, in this order:
//   1. sizes and types the operator does not have (INVALID_ARGUMENT)
//   2. strides and workspace bytes too small (SHAPE_MISMATCH)
//   3. no tokens: RCC_OK here, except that a gradient written whole is still
//      written (as zeros)
//   4. NULL buffers, misaligned buffers, overlaps (INVALID_ARGUMENT)
#include "host_internal.h"
#include "lm_internal.h"

using namespace rcc::host;
using namespace rcc::lm;

namespace {

constexpr size_t kMaxCount = 0x7FFFFFFF - 256;  // tokens, vocabulary entries
constexpr size_t kMaxDim = 1u << 20;
constexpr size_t kMaxStride = 1u << 30;
constexpr size_t kMaxBlocks = 0x7FFFFFFF;       // of one launch

bool valid_type(int t) { return t == RCC_F32 || t == RCC_BF16; }
size_t bytes_of(int t) { return t == RCC_F32 ? 4 : 2; }

// Bytes of `rows` rows at a stride of `ld` elements, the last one `dim` long
size_t extent(size_t rows, size_t ld, size_t dim, size_t size) {
  return rows ? ((rows - 1) * ld + dim) * size : 0;
}

// Rows of whole vectors of eight elements, each on a boundary of `align` bytes
bool vectors(const void* p, size_t ld, size_t dim, size_t size, size_t align) {
  return reinterpret_cast<uintptr_t>(p) % align == 0 && dim % 8 == 0 && (ld * size) % align == 0;
}

struct Buffer {
  const char* name;
  const void* p;
  size_t bytes;
  size_t align;
  bool written;
};

// NULL and misaligned buffers, and written ones that overlap any other
rcc_status check_buffers(const Buffer* b, int n) {
  for (int i = 0; i < n; ++i) {
    if (!b[i].p) return fail(RCC_ERR_INVALID_ARGUMENT, "%s is NULL", b[i].name);
    if (reinterpret_cast<uintptr_t>(b[i].p) % b[i].align)
      return fail(RCC_ERR_INVALID_ARGUMENT, "%s must be %zu-byte aligned", b[i].name, b[i].align);
  }
  for (int i = 0; i < n; ++i)
    for (int j = i + 1; j < n; ++j)
      if ((b[i].written || b[j].written) && overlap(b[i].p, b[i].bytes, b[j].p, b[j].bytes))
        return fail(RCC_ERR_INVALID_ARGUMENT, "%s overlaps %s", b[i].name, b[j].name);
  return RCC_OK;
}

rcc_status check_sizes(size_t tokens, size_t dim, size_t vocab) {
  if (tokens > kMaxCount) return fail(RCC_ERR_INVALID_ARGUMENT, "%zu tokens: too many", tokens);
  if (dim < 1 || dim > kMaxDim)
    return fail(RCC_ERR_INVALID_ARGUMENT, "dim %zu outside [1, %zu]", dim, kMaxDim);
  if (vocab < 1 || vocab > kMaxCount)
    return fail(RCC_ERR_INVALID_ARGUMENT, "vocab %zu outside [1, %zu]", vocab, kMaxCount);
  return RCC_OK;
}
rcc_status check_type(const char* name, int t) {
  if (!valid_type(t)) return fail(RCC_ERR_INVALID_ARGUMENT, "%s %d is not an rcc_dtype", name, t);
  return RCC_OK;
}
rcc_status check_index(int t) {
  if (t != RCC_I32 && t != RCC_I64)
    return fail(RCC_ERR_INVALID_ARGUMENT, "index type %d is not an rcc_index", t);
  return RCC_OK;
}
rcc_status check_ld(const char* name, size_t ld, size_t dim) {
  if (ld < dim)
    return fail(RCC_ERR_SHAPE_MISMATCH, "rows of %s are %zu elements apart, dim is %zu", name, ld,
                dim);
  if (ld > kMaxStride)
    return fail(RCC_ERR_INVALID_ARGUMENT, "rows of %s are %zu elements apart: over %zu", name, ld,
                kMaxStride);
  return RCC_OK;
}
// The elements of [tokens][dim], as pieces of at least 2,048, fit one launch
rcc_status check_launch(size_t tokens, size_t dim) {
  if (tokens * ((dim + 2047) / 2048) > kMaxBlocks)
    return fail(RCC_ERR_INVALID_ARGUMENT, "%zu tokens of dim %zu: too many for one call", tokens,
                dim);
  return RCC_OK;
}
rcc_status check_workspace(size_t have, size_t need) {
  if (have < need)
    return fail(RCC_ERR_SHAPE_MISMATCH, "the workspace has %zu bytes, %zu are needed", have, need);
  return RCC_OK;
}
rcc_status done(cudaError_t e, const char* what, uint64_t launches) {
  rcc::add_launches(launches);
  return e == cudaSuccess ? RCC_OK : cuda_fail(e, what);
}

#define RCC_TRY(call)                     \
  do {                                    \
    const rcc_status st_ = (call);        \
    if (st_ != RCC_OK) return st_;        \
  } while (0)

// Widths the output layer takes: rows that TMA can address
rcc_status check_ce(size_t tokens, size_t dim, size_t vocab, size_t ld_x, size_t ld_w,
                    rcc_index index) {
  RCC_TRY(check_sizes(tokens, dim, vocab));
  RCC_TRY(check_index(index));
  RCC_TRY(check_launch(tokens, dim));
  if ((tokens + 127) / 128 * ((vocab + 255) / 256) > kMaxBlocks / 2)
    return fail(RCC_ERR_INVALID_ARGUMENT, "%zu tokens and %zu vocabulary entries: too many for "
                "one call", tokens, vocab);
  if (dim % 8)
    return fail(RCC_ERR_INVALID_ARGUMENT, "dim %zu must be a multiple of 8", dim);
  RCC_TRY(check_ld("x", ld_x, dim));
  RCC_TRY(check_ld("w", ld_w, dim));
  if (ld_x % 8 || ld_w % 8)
    return fail(RCC_ERR_INVALID_ARGUMENT, "row strides of x (%zu) and w (%zu) must be multiples of 8",
                ld_x, ld_w);
  return RCC_OK;
}

}  // namespace

extern "C" {

rcc_status rcc_embedding_forward(const void* table, rcc_dtype table_type, size_t ld_table,
                                 const void* ids, rcc_index index, size_t tokens, size_t vocab,
                                 size_t dim, float scale, void* out, rcc_dtype out_type,
                                 rcc_stream_t stream) {
  rcc::NvtxRange nvtx_range("rcc_embedding_forward");
  t_err.clear();
  RCC_TRY(check_sizes(tokens, dim, vocab));
  RCC_TRY(check_type("table_type", table_type));
  RCC_TRY(check_type("out_type", out_type));
  RCC_TRY(check_index(index));
  RCC_TRY(check_launch(tokens, dim));
  RCC_TRY(check_ld("table", ld_table, dim));
  if (tokens == 0) return RCC_OK;
  const size_t ts = bytes_of(table_type), os = bytes_of(out_type), is = index == RCC_I64 ? 8 : 4;
  const Buffer b[] = {{"table", table, extent(vocab, ld_table, dim, ts), ts, false},
                      {"ids", ids, tokens * is, is, false},
                      {"out", out, tokens * dim * os, os, true}};
  RCC_TRY(check_buffers(b, 3));
  EmbedArgs a = {};
  a.table = table;
  a.ids = ids;
  a.out = out;
  a.ld_table = ld_table;
  a.tokens = tokens;
  a.vocab = vocab;
  a.dim = dim;
  a.table_type = table_type;
  a.out_type = out_type;
  a.ids64 = index == RCC_I64;
  a.vec = vectors(table, ld_table, dim, ts, 8 * ts) && vectors(out, dim, dim, os, 8 * os);
  a.scale = scale;
  return done(launch_embedding_forward(a, reinterpret_cast<cudaStream_t>(stream)),
              "rcc_embedding_forward", 1);
}

size_t rcc_embedding_backward_workspace(size_t tokens, size_t vocab, size_t dim) {
  if (tokens > kMaxCount || vocab > kMaxCount || dim > kMaxDim) return 0;
  return embedding_backward_workspace(tokens, vocab, dim);
}

rcc_status rcc_embedding_backward(const void* dout, rcc_dtype dout_type, size_t ld_dout,
                                  const void* ids, rcc_index index, size_t tokens, size_t vocab,
                                  size_t dim, float scale, void* dtable, rcc_dtype dtable_type,
                                  int accumulate, void* workspace, size_t workspace_bytes,
                                  rcc_stream_t stream) {
  rcc::NvtxRange nvtx_range("rcc_embedding_backward");
  t_err.clear();
  RCC_TRY(check_sizes(tokens, dim, vocab));
  RCC_TRY(check_type("dout_type", dout_type));
  RCC_TRY(check_type("dtable_type", dtable_type));
  RCC_TRY(check_index(index));
  RCC_TRY(check_launch(tokens, dim));
  RCC_TRY(check_ld("dout", ld_dout, dim));
  const size_t need = embedding_backward_workspace(tokens, vocab, dim);
  RCC_TRY(check_workspace(workspace_bytes, need));
  const size_t ds = bytes_of(dout_type), gs = bytes_of(dtable_type), is = index == RCC_I64 ? 8 : 4;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (tokens == 0) {
    if (accumulate) return RCC_OK;
    const Buffer b[] = {{"dtable", dtable, vocab * dim * gs, gs, true}};
    RCC_TRY(check_buffers(b, 1));
    return done(cudaMemsetAsync(dtable, 0, vocab * dim * gs, st), "rcc_embedding_backward", 0);
  }
  const Buffer b[] = {{"dout", dout, extent(tokens, ld_dout, dim, ds), ds, false},
                      {"ids", ids, tokens * is, is, false},
                      {"dtable", dtable, vocab * dim * gs, gs, true},
                      {"workspace", workspace, need, 256, true}};
  RCC_TRY(check_buffers(b, 4));
  EmbedGradArgs a = {};
  a.dout = dout;
  a.ids = ids;
  a.dtable = dtable;
  a.workspace = workspace;
  a.ld_dout = ld_dout;
  a.tokens = tokens;
  a.vocab = vocab;
  a.dim = dim;
  a.dout_type = dout_type;
  a.dtable_type = dtable_type;
  a.ids64 = index == RCC_I64;
  a.vec = vectors(dout, ld_dout, dim, ds, 8 * ds) && vectors(dtable, dim, dim, gs, 8 * gs);
  a.accumulate = accumulate != 0;
  a.scale = scale;
  uint64_t launches = 0;
  const cudaError_t e = launch_embedding_backward(a, st, &launches);
  return done(e, "rcc_embedding_backward", launches);
}

rcc_status rcc_rmsnorm_forward(const void* x, rcc_dtype type, size_t ld_x, const float* weight,
                               float eps, size_t tokens, size_t dim, void* y, int8_t* kept,
                               float* scales, rcc_stream_t stream) {
  rcc::NvtxRange nvtx_range("rcc_rmsnorm_forward");
  t_err.clear();
  RCC_TRY(check_sizes(tokens, dim, 1));
  if (dim > kMaxNormDim)
    return fail(RCC_ERR_INVALID_ARGUMENT, "dim %zu is over %zu", dim, kMaxNormDim);
  RCC_TRY(check_type("type", type));
  if (!(eps >= 0.f) || std::isinf(eps))
    return fail(RCC_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
  RCC_TRY(check_ld("x", ld_x, dim));
  if ((kept == nullptr) != (scales == nullptr))
    return fail(RCC_ERR_INVALID_ARGUMENT, "kept and scales come together");
  if (tokens == 0) return RCC_OK;
  const size_t s = bytes_of(type), groups = (dim + kKeepGroup - 1) / kKeepGroup;
  const Buffer b[] = {{"x", x, extent(tokens, ld_x, dim, s), s, false},
                      {"weight", weight, dim * 4, 4, false},
                      {"y", y, tokens * dim * s, s, true},
                      {"kept", kept, tokens * groups * kKeepGroup, 16, true},
                      {"scales", scales, tokens * groups * 4, 4, true}};
  RCC_TRY(check_buffers(b, kept ? 5 : 3));
  NormArgs a = {};
  a.x = x;
  a.weight = weight;
  a.y = y;
  a.kept = kept;
  a.scales = scales;
  a.ld_x = ld_x;
  a.ld_y = dim;
  a.tokens = tokens;
  a.dim = dim;
  a.type = type;
  a.vec = vectors(x, ld_x, dim, s, 16) && vectors(y, dim, dim, s, 16) && aligned16(weight);
  a.eps = eps;
  return done(launch_rmsnorm_forward(a, reinterpret_cast<cudaStream_t>(stream)),
              "rcc_rmsnorm_forward", 1);
}

size_t rcc_rmsnorm_backward_workspace(size_t tokens, size_t dim) {
  if (tokens > kMaxCount || dim < 1 || dim > kMaxNormDim) return 0;
  return rmsnorm_backward_workspace(tokens, dim);
}

rcc_status rcc_rmsnorm_backward(const void* dy, rcc_dtype type, size_t ld_dy, const int8_t* kept,
                                const float* scales, const float* weight, float eps,
                                size_t tokens, size_t dim, void* dx, float* dweight,
                                int accumulate, void* workspace, size_t workspace_bytes,
                                rcc_stream_t stream) {
  rcc::NvtxRange nvtx_range("rcc_rmsnorm_backward");
  t_err.clear();
  RCC_TRY(check_sizes(tokens, dim, 1));
  if (dim > kMaxNormDim)
    return fail(RCC_ERR_INVALID_ARGUMENT, "dim %zu is over %zu", dim, kMaxNormDim);
  RCC_TRY(check_type("type", type));
  if (!(eps >= 0.f) || std::isinf(eps))
    return fail(RCC_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
  RCC_TRY(check_ld("dy", ld_dy, dim));
  const size_t need = rmsnorm_backward_workspace(tokens, dim);
  RCC_TRY(check_workspace(workspace_bytes, need));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (tokens == 0) {
    if (accumulate) return RCC_OK;
    const Buffer b[] = {{"dweight", dweight, dim * 4, 4, true}};
    RCC_TRY(check_buffers(b, 1));
    return done(cudaMemsetAsync(dweight, 0, dim * 4, st), "rcc_rmsnorm_backward", 0);
  }
  const size_t s = bytes_of(type), groups = (dim + kKeepGroup - 1) / kKeepGroup;
  const Buffer b[] = {{"dy", dy, extent(tokens, ld_dy, dim, s), s, false},
                      {"kept", kept, tokens * groups * kKeepGroup, 16, false},
                      {"scales", scales, tokens * groups * 4, 4, false},
                      {"weight", weight, dim * 4, 4, false},
                      {"dx", dx, tokens * dim * s, s, true},
                      {"dweight", dweight, dim * 4, 4, true},
                      {"workspace", workspace, need, 256, true}};
  RCC_TRY(check_buffers(b, 7));
  NormGradArgs a = {};
  a.dy = dy;
  a.kept = kept;
  a.scales = scales;
  a.weight = weight;
  a.dx = dx;
  a.dweight = dweight;
  a.workspace = workspace;
  a.ld_dy = ld_dy;
  a.ld_dx = dim;
  a.tokens = tokens;
  a.dim = dim;
  a.type = type;
  a.vec = vectors(dy, ld_dy, dim, s, 16) && vectors(dx, dim, dim, s, 16) && aligned16(weight);
  a.accumulate = accumulate != 0;
  a.eps = eps;
  uint64_t launches = 0;
  const cudaError_t e = launch_rmsnorm_backward(a, st, &launches);
  return done(e, "rcc_rmsnorm_backward", launches);
}

size_t rcc_linear_ce_workspace(size_t tokens, size_t vocab, size_t dim, int backward,
                               rcc_dtype grad_type) {
  if (tokens < 1 || tokens > kMaxCount || vocab < 1 || vocab > kMaxCount || dim < 1 ||
      dim > kMaxDim || !valid_type(grad_type))
    return 0;
  return linear_ce_workspace(tokens, vocab, dim, backward != 0, grad_type);
}

rcc_status rcc_linear_ce_forward(const void* x, size_t ld_x, const void* w, size_t ld_w,
                                 const void* labels, rcc_index index, size_t tokens, size_t vocab,
                                 size_t dim, float* loss, float* lse, void* workspace,
                                 size_t workspace_bytes, rcc_stream_t stream) {
  rcc::NvtxRange nvtx_range("rcc_linear_ce_forward");
  t_err.clear();
  RCC_TRY(check_ce(tokens, dim, vocab, ld_x, ld_w, index));
  if (tokens == 0) return RCC_OK;
  const size_t need = linear_ce_workspace(tokens, vocab, dim, false, RCC_F32);
  RCC_TRY(check_workspace(workspace_bytes, need));
  const size_t is = index == RCC_I64 ? 8 : 4;
  const Buffer b[] = {{"x", x, extent(tokens, ld_x, dim, 2), 16, false},
                      {"w", w, extent(vocab, ld_w, dim, 2), 16, false},
                      {"labels", labels, tokens * is, is, false},
                      {"loss", loss, tokens * 4, 4, true},
                      {"lse", lse, tokens * 4, 4, true},
                      {"workspace", workspace, need, 256, true}};
  RCC_TRY(check_buffers(b, 6));
  CeArgs a = {};
  a.x = x;
  a.w = w;
  a.labels = labels;
  a.ld_x = ld_x;
  a.ld_w = ld_w;
  a.tokens = tokens;
  a.vocab = vocab;
  a.dim = dim;
  a.labels64 = index == RCC_I64;
  a.loss = loss;
  a.lse = lse;
  a.workspace = workspace;
  uint64_t launches = 0;
  const cudaError_t e =
      launch_linear_ce_forward(a, reinterpret_cast<cudaStream_t>(stream), &launches);
  return done(e, "rcc_linear_ce_forward", launches);
}

rcc_status rcc_linear_ce_backward(const void* x, size_t ld_x, const void* w, size_t ld_w,
                                  const void* labels, rcc_index index, const float* lse,
                                  const float* dloss, size_t tokens, size_t vocab, size_t dim,
                                  void* dx, void* dw, rcc_dtype grad_type, int accumulate,
                                  void* workspace, size_t workspace_bytes, rcc_stream_t stream) {
  rcc::NvtxRange nvtx_range("rcc_linear_ce_backward");
  t_err.clear();
  RCC_TRY(check_ce(tokens, dim, vocab, ld_x, ld_w, index));
  RCC_TRY(check_type("grad_type", grad_type));
  const size_t gs = bytes_of(grad_type);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (tokens == 0) {
    if (accumulate || !dw) return RCC_OK;
    return done(cudaMemsetAsync(dw, 0, vocab * dim * gs, st), "rcc_linear_ce_backward", 0);
  }
  if (!dx && !dw) return fail(RCC_ERR_INVALID_ARGUMENT, "neither dx nor dw is wanted");
  const size_t need = linear_ce_workspace(tokens, vocab, dim, true, grad_type);
  RCC_TRY(check_workspace(workspace_bytes, need));
  const size_t is = index == RCC_I64 ? 8 : 4;
  Buffer b[8] = {{"x", x, extent(tokens, ld_x, dim, 2), 16, false},
                 {"w", w, extent(vocab, ld_w, dim, 2), 16, false},
                 {"labels", labels, tokens * is, is, false},
                 {"lse", lse, tokens * 4, 4, false},
                 {"dloss", dloss, tokens * 4, 4, false},
                 {"workspace", workspace, need, 256, true}};
  int n = 6;
  if (dx) b[n++] = {"dx", dx, tokens * dim * gs, 16, true};
  if (dw) b[n++] = {"dw", dw, vocab * dim * gs, 16, true};
  RCC_TRY(check_buffers(b, n));
  CeArgs a = {};
  a.x = x;
  a.w = w;
  a.labels = labels;
  a.ld_x = ld_x;
  a.ld_w = ld_w;
  a.tokens = tokens;
  a.vocab = vocab;
  a.dim = dim;
  a.labels64 = index == RCC_I64;
  a.lse = const_cast<float*>(lse);
  a.dloss = dloss;
  a.dx = dx;
  a.dw = dw;
  a.grad_type = grad_type;
  a.accumulate = accumulate != 0;
  a.workspace = workspace;
  uint64_t launches = 0;
  const cudaError_t e = launch_linear_ce_backward(a, st, &launches);
  return done(e, "rcc_linear_ce_backward", launches);
}

}  // extern "C"
