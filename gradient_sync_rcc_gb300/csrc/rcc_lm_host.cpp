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
constexpr size_t kMaxHeadStride = size_t{1} << 40;
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

rcc_status check_norm(size_t tokens, size_t dim, int type, float eps) {
  RCC_TRY(check_sizes(tokens, dim, 1));
  if (dim > kMaxNormDim)
    return fail(RCC_ERR_INVALID_ARGUMENT, "dim %zu is over %zu", dim, kMaxNormDim);
  RCC_TRY(check_type("type", type));
  if (!(eps >= 0.f) || std::isinf(eps))
    return fail(RCC_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
  return RCC_OK;
}

// ---- rotary positions: rows of heads, whose strides may interleave -----------------

// [tokens][heads][head_dim] at p, elements apart
struct Heads {
  const char* name;
  const void* p;
  size_t heads, token, head;
};

// No two heads share an element: one of the orders of tokens and heads nests
bool apart(const Heads& r, size_t tokens, size_t head_dim) {
  const size_t heads = (r.heads - 1) * r.head + head_dim, rows = (tokens - 1) * r.token + head_dim;
  return (r.heads < 2 || r.head >= head_dim) && (tokens < 2 || r.token >= head_dim) &&
         (r.heads < 2 || tokens < 2 || r.token >= heads || r.head >= rows);
}

// Whether two of them may share elements: overlapping extents, unless both have
// the same step from token to token and each token's heads lie apart within it
bool may_share(const Heads& a, const Heads& b, size_t tokens, size_t head_dim, size_t size) {
  auto heads = [&](const Heads& r) { return ((r.heads - 1) * r.head + head_dim) * size; };
  auto bytes = [&](const Heads& r) { return (tokens - 1) * r.token * size + heads(r); };
  if (!overlap(a.p, bytes(a), b.p, bytes(b))) return false;
  if (a.token != b.token) return true;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  const size_t step = a.token * size;
  const bool a_first = pa <= pb;
  const size_t off = (a_first ? pb - pa : pa - pb);
  const size_t before = heads(a_first ? a : b), behind = heads(a_first ? b : a);
  return !(off >= before && off + behind <= step);
}

rcc_status check_heads(const Heads& r, size_t tokens, size_t head_dim, size_t size) {
  if (r.heads > kMaxHeads)
    return fail(RCC_ERR_INVALID_ARGUMENT, "%s has %zu heads: over %zu", r.name, r.heads, kMaxHeads);
  if (r.token > kMaxStride || r.head > kMaxHeadStride)
    return fail(RCC_ERR_INVALID_ARGUMENT, "tokens of %s are over %zu elements apart, or heads over "
                "%zu", r.name, kMaxStride, kMaxHeadStride);
  if (!r.p) return fail(RCC_ERR_INVALID_ARGUMENT, "%s is NULL", r.name);
  if (reinterpret_cast<uintptr_t>(r.p) % size)
    return fail(RCC_ERR_INVALID_ARGUMENT, "%s must be %zu-byte aligned", r.name, size);
  if (!apart(r, tokens, head_dim))
    return fail(RCC_ERR_SHAPE_MISMATCH, "the heads of %s overlap", r.name);
  return RCC_OK;
}

// Every head in vectors of n elements, each on a boundary of its size
bool head_vectors(const Heads& r, size_t size, size_t n) {
  return reinterpret_cast<uintptr_t>(r.p) % (n * size) == 0 && r.token % n == 0 && r.head % n == 0;
}

rcc_status rotary(const char* what, const rcc_rotary_rows* q, const rcc_rotary_rows* k,
                  rcc_dtype type, size_t tokens, size_t head_dim, const uint64_t* turns,
                  size_t pairs, rcc_rotary_layout layout, const void* positions, rcc_index index,
                  int64_t offset, float scale, bool inverse, rcc_stream_t stream) {
  rcc::NvtxRange nvtx_range(what);
  t_err.clear();
  if (!q) return fail(RCC_ERR_INVALID_ARGUMENT, "q is NULL");
  RCC_TRY(check_type("type", type));
  if (tokens > kMaxCount) return fail(RCC_ERR_INVALID_ARGUMENT, "%zu tokens: too many", tokens);
  if (head_dim < 2 || head_dim > kMaxHeadDim)
    return fail(RCC_ERR_INVALID_ARGUMENT, "head_dim %zu outside [2, %zu]", head_dim, kMaxHeadDim);
  if (pairs < 1 || pairs > head_dim / 2)
    return fail(RCC_ERR_INVALID_ARGUMENT, "%zu pairs of head_dim %zu", pairs, head_dim);
  if (layout != RCC_ROTARY_HALF && layout != RCC_ROTARY_INTERLEAVED)
    return fail(RCC_ERR_INVALID_ARGUMENT, "layout %d is not an rcc_rotary_layout", (int)layout);
  if (positions) RCC_TRY(check_index(index));
  if (offset < 0 || offset > (int64_t)kMaxCount)
    return fail(RCC_ERR_INVALID_ARGUMENT, "offset %lld outside [0, %zu]", (long long)offset,
                kMaxCount);
  if (!std::isfinite(scale)) return fail(RCC_ERR_INVALID_ARGUMENT, "scale must be finite");
  const size_t heads = q->heads + (k ? k->heads : 0);
  if (tokens == 0 || heads == 0) return RCC_OK;
  const size_t s = bytes_of(type), is = index == RCC_I64 ? 8 : 4;
  Heads in[2], out[2];
  int n = 0;
  bool copies = false;
  for (const rcc_rotary_rows* r : {q, k}) {
    if (!r || r->heads == 0) continue;
    const bool first = r == q;
    in[n] = {first ? "q" : "k", r->in, r->heads, r->in_token, r->in_head};
    out[n] = {first ? "q's output" : "k's output", r->out, r->heads, r->out_token, r->out_head};
    RCC_TRY(check_heads(in[n], tokens, head_dim, s));
    RCC_TRY(check_heads(out[n], tokens, head_dim, s));
    copies = copies || r->in != r->out;
    ++n;
  }
  const Buffer b[] = {{"turns", turns, pairs * 8, 8, false},
                      {"positions", positions, positions ? tokens * is : 0, is, false}};
  RCC_TRY(check_buffers(b, positions ? 2 : 1));
  auto same = [](const Heads& x, const Heads& y) {
    return x.p == y.p && x.token == y.token && x.head == y.head && x.heads == y.heads;
  };
  for (int i = 0; i < n; ++i) {
    for (int j = 0; j < n; ++j) {
      if (!(i == j && same(in[i], out[j])) && may_share(in[i], out[j], tokens, head_dim, s))
        return fail(RCC_ERR_INVALID_ARGUMENT, "%s overlaps %s", in[i].name, out[j].name);
      if (j > i && may_share(out[i], out[j], tokens, head_dim, s))
        return fail(RCC_ERR_INVALID_ARGUMENT, "%s overlaps %s", out[i].name, out[j].name);
    }
    const size_t bytes =
        ((tokens - 1) * out[i].token + (out[i].heads - 1) * out[i].head + head_dim) * s;
    for (int j = 0; j < (positions ? 2 : 1); ++j)
      if (overlap(out[i].p, bytes, b[j].p, b[j].bytes))
        return fail(RCC_ERR_INVALID_ARGUMENT, "%s overlaps %s", out[i].name, b[j].name);
  }
  const size_t units = pairs + head_dim;  // of a token's head, at most
  if (tokens > kMaxBlocks * 64 / units / heads)
    return fail(RCC_ERR_INVALID_ARGUMENT, "%zu tokens of %zu heads of %zu: too many for one call",
                tokens, heads, head_dim);
  RotaryArgs a = {};
  // the widest vectors: of both halves of the pairs, or of neighbours
  auto fits = [&](size_t w) {
    bool ok = head_dim % w == 0 && (layout == RCC_ROTARY_INTERLEAVED || pairs % w == 0);
    for (int i = 0; i < n; ++i)
      ok = ok && head_vectors(in[i], s, w) && head_vectors(out[i], s, w);
    return ok;
  };
  a.wide = fits(8) ? 8 : fits(4) ? 4 : fits(2) ? 2 : 1;
  for (int i = 0; i < n; ++i) {
    RotaryRows& r = in[i].name[0] == 'q' ? a.q : a.k;
    r = {in[i].p, const_cast<void*>(out[i].p), in[i].heads, in[i].token, in[i].head, out[i].token,
         out[i].head};
  }
  a.turns = turns;
  a.positions = positions;
  a.offset = offset;
  a.tokens = tokens;
  a.head_dim = head_dim;
  a.pairs = pairs;
  a.type = type;
  a.index64 = index == RCC_I64;
  a.half = layout == RCC_ROTARY_HALF;
  a.inverse = inverse;
  a.copies = copies && 2 * pairs < head_dim;
  a.scale = scale;
  return done(launch_rotary(a, reinterpret_cast<cudaStream_t>(stream)), what, 1);
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

rcc_status rcc_add_rmsnorm_forward(const void* x, size_t ld_x, const void* residual,
                                   size_t ld_residual, rcc_dtype type, const float* weight,
                                   float eps, size_t tokens, size_t dim, void* sum, void* y,
                                   float* y_scales, int8_t* kept, float* scales,
                                   rcc_stream_t stream) {
  rcc::NvtxRange nvtx_range("rcc_add_rmsnorm_forward");
  t_err.clear();
  RCC_TRY(check_norm(tokens, dim, type, eps));
  RCC_TRY(check_ld("x", ld_x, dim));
  if ((kept == nullptr) != (scales == nullptr))
    return fail(RCC_ERR_INVALID_ARGUMENT, "kept and scales come together");
  if (residual) RCC_TRY(check_ld("residual", ld_residual, dim));
  if (tokens == 0) return RCC_OK;
  if ((residual == nullptr) != (sum == nullptr))
    return fail(RCC_ERR_INVALID_ARGUMENT, "residual and sum come together");
  if (!residual && !y_scales)
    return fail(RCC_ERR_INVALID_ARGUMENT, "without a residual y has to be 8-bit");
  const size_t s = bytes_of(type), groups = (dim + kKeepGroup - 1) / kKeepGroup;
  // sum in place of an input: that buffer counts once, as written
  const bool over_x = sum && sum == x && ld_x == dim;
  const bool over_residual = sum && sum == residual && ld_residual == dim;
  Buffer b[9] = {{"weight", weight, dim * 4, 4, false},
                 {"y", y, tokens * dim * (y_scales ? 1 : s), y_scales ? 1 : s, true}};
  int n = 2;
  if (!over_x) b[n++] = {"x", x, extent(tokens, ld_x, dim, s), s, false};
  if (residual && !over_residual)
    b[n++] = {"residual", residual, extent(tokens, ld_residual, dim, s), s, false};
  if (residual) b[n++] = {"sum", sum, tokens * dim * s, s, true};
  if (y_scales) b[n++] = {"y_scales", y_scales, tokens * groups * 4, 4, true};
  if (kept) {
    b[n++] = {"kept", kept, tokens * groups * kKeepGroup, 16, true};
    b[n++] = {"scales", scales, tokens * groups * 4, 4, true};
  }
  RCC_TRY(check_buffers(b, n));
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
  a.vec = vectors(x, ld_x, dim, s, 16) && aligned16(weight) &&
          (y_scales ? vectors(y, dim, dim, 1, 8) : vectors(y, dim, dim, s, 16)) &&
          (!residual || (vectors(residual, ld_residual, dim, s, 16) &&
                         vectors(sum, dim, dim, s, 16)));
  a.eps = eps;
  a.residual = residual;
  a.sum = sum;
  a.y_scales = y_scales;
  a.ld_residual = ld_residual;
  return done(launch_add_rmsnorm_forward(a, reinterpret_cast<cudaStream_t>(stream)),
              "rcc_add_rmsnorm_forward", 1);
}

rcc_status rcc_add_rmsnorm_backward(const void* dy, size_t ld_dy, const void* dsum,
                                    size_t ld_dsum, rcc_dtype type, const int8_t* kept,
                                    const float* scales, const float* weight, float eps,
                                    size_t tokens, size_t dim, void* dx, float* dweight,
                                    int accumulate, void* workspace, size_t workspace_bytes,
                                    rcc_stream_t stream) {
  if (!dsum)
    return rcc_rmsnorm_backward(dy, type, ld_dy, kept, scales, weight, eps, tokens, dim, dx,
                                dweight, accumulate, workspace, workspace_bytes, stream);
  rcc::NvtxRange nvtx_range("rcc_add_rmsnorm_backward");
  t_err.clear();
  RCC_TRY(check_norm(tokens, dim, type, eps));
  RCC_TRY(check_ld("dy", ld_dy, dim));
  RCC_TRY(check_ld("dsum", ld_dsum, dim));
  const size_t need = rmsnorm_backward_workspace(tokens, dim);
  RCC_TRY(check_workspace(workspace_bytes, need));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (tokens == 0) {
    if (accumulate) return RCC_OK;
    const Buffer b[] = {{"dweight", dweight, dim * 4, 4, true}};
    RCC_TRY(check_buffers(b, 1));
    return done(cudaMemsetAsync(dweight, 0, dim * 4, st), "rcc_add_rmsnorm_backward", 0);
  }
  const size_t s = bytes_of(type), groups = (dim + kKeepGroup - 1) / kKeepGroup;
  const bool over_dsum = dx == dsum && ld_dsum == dim;
  Buffer b[8] = {{"dy", dy, extent(tokens, ld_dy, dim, s), s, false},
                 {"kept", kept, tokens * groups * kKeepGroup, 16, false},
                 {"scales", scales, tokens * groups * 4, 4, false},
                 {"weight", weight, dim * 4, 4, false},
                 {"dx", dx, tokens * dim * s, s, true},
                 {"dweight", dweight, dim * 4, 4, true},
                 {"workspace", workspace, need, 256, true}};
  if (!over_dsum) b[7] = {"dsum", dsum, extent(tokens, ld_dsum, dim, s), s, false};
  RCC_TRY(check_buffers(b, over_dsum ? 7 : 8));
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
  a.vec = vectors(dy, ld_dy, dim, s, 16) && vectors(dx, dim, dim, s, 16) &&
          vectors(dsum, ld_dsum, dim, s, 16) && aligned16(weight);
  a.accumulate = accumulate != 0;
  a.eps = eps;
  a.dsum = dsum;
  a.ld_dsum = ld_dsum;
  uint64_t launches = 0;
  const cudaError_t e = launch_add_rmsnorm_backward(a, st, &launches);
  return done(e, "rcc_add_rmsnorm_backward", launches);
}

rcc_status rcc_rotary_turns(size_t pairs, double base, const rcc_rotary_scaling* scaling,
                            uint64_t* turns) {
  t_err.clear();
  if (pairs < 1 || pairs > kMaxHeadDim / 2)
    return fail(RCC_ERR_INVALID_ARGUMENT, "%zu pairs outside [1, %zu]", pairs, kMaxHeadDim / 2);
  if (!(base >= 1.0) || std::isinf(base))
    return fail(RCC_ERR_INVALID_ARGUMENT, "base must be finite and >= 1");
  if (!turns) return fail(RCC_ERR_INVALID_ARGUMENT, "turns is NULL");
  const rcc_rotary_scaling none = {RCC_ROTARY_NONE, 1.0, 0.0, 0.0, 0.0};
  const rcc_rotary_scaling& sc = scaling ? *scaling : none;
  if (sc.kind < RCC_ROTARY_NONE || sc.kind > RCC_ROTARY_PARTS)
    return fail(RCC_ERR_INVALID_ARGUMENT, "scaling %d is not an rcc_rotary_kind", (int)sc.kind);
  if (sc.kind != RCC_ROTARY_NONE && (!(sc.factor >= 1.0) || std::isinf(sc.factor)))
    return fail(RCC_ERR_INVALID_ARGUMENT, "the scaling's factor must be finite and >= 1");
  if (sc.kind == RCC_ROTARY_PARTS &&
      (!(sc.length > 0.0) || std::isinf(sc.length) || !(sc.low >= 0.0) || !(sc.high > sc.low) ||
       std::isinf(sc.high)))
    return fail(RCC_ERR_INVALID_ARGUMENT, "the scaling needs length > 0 and 0 <= low < high");
  const double n = (double)pairs, two_pi = 6.283185307179586;
  if (sc.kind == RCC_ROTARY_BASE && pairs > 1) base *= std::pow(sc.factor, n / (n - 1.0));
  for (size_t i = 0; i < pairs; ++i) {
    double f = std::pow(base, -(double)i / n) / two_pi;  // turns a position, at most 0.16
    if (sc.kind == RCC_ROTARY_LINEAR) f /= sc.factor;
    if (sc.kind == RCC_ROTARY_PARTS) {
      const double k = std::min(1.0, std::max(0.0, (sc.length * f - sc.low) / (sc.high - sc.low)));
      f *= k + (1.0 - k) / sc.factor;
    }
    turns[i] = (uint64_t)std::ldexp(f, 64);
  }
  return RCC_OK;
}

rcc_status rcc_rotary_forward(const rcc_rotary_rows* q, const rcc_rotary_rows* k, rcc_dtype type,
                              size_t tokens, size_t head_dim, const uint64_t* turns, size_t pairs,
                              rcc_rotary_layout layout, const void* positions, rcc_index index,
                              int64_t offset, float scale, rcc_stream_t stream) {
  return rotary("rcc_rotary_forward", q, k, type, tokens, head_dim, turns, pairs, layout,
                positions, index, offset, scale, false, stream);
}

rcc_status rcc_rotary_backward(const rcc_rotary_rows* dq, const rcc_rotary_rows* dk,
                               rcc_dtype type, size_t tokens, size_t head_dim,
                               const uint64_t* turns, size_t pairs, rcc_rotary_layout layout,
                               const void* positions, rcc_index index, int64_t offset,
                               float scale, rcc_stream_t stream) {
  return rotary("rcc_rotary_backward", dq, dk, type, tokens, head_dim, turns, pairs, layout,
                positions, index, offset, scale, true, stream);
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
