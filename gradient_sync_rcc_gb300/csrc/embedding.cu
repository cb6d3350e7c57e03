// embedding.cu -- token embedding with scaling, and its gradient by sorted tokens.
//
//   forward    out[t] = scale W[id_t]              (a padding id: zeros)
//   gradient   dW[v] (+)= scale sum_{t: id_t = v} dout[t]
//
// The gradient sorts the tokens by id (stable, so equal ids keep the order of
// the tokens) and adds each run of equal ids in that order in fp32: no atomic
// touches a sum, and the bits are the same from run to run.  The sorted list
// is cut into windows; a run inside one window is summed and written at once,
// a run that crosses windows leaves one fp32 row per window, which a last
// kernel joins.
#include <algorithm>

#include "lm_common.cuh"
#include "lm_internal.h"

namespace rcc {
namespace lm {
namespace {

constexpr int kRowThreads = 256;
constexpr int kSlab = kRowThreads * 8;  // columns of a row that one block covers

// ---- forward -------------------------------------------------------------------

constexpr int kTokensPerBlock = 4;

// A block copies one slab of columns of kTokensPerBlock tokens: all of its
// loads are issued before its first store.
template <typename T, typename O, bool VEC>
__global__ void __launch_bounds__(kRowThreads) embed_kernel(const EmbedArgs a) {
  pdl_wait_then_release();
  const size_t slabs = (a.dim + kSlab - 1) / kSlab;
  const size_t t0 = blockIdx.x / slabs * kTokensPerBlock;
  const size_t col = blockIdx.x % slabs * kSlab + threadIdx.x * 8;
  if (col >= a.dim) return;
  int64_t id[kTokensPerBlock];
#pragma unroll
  for (int i = 0; i < kTokensPerBlock; ++i)
    id[i] = t0 + i < a.tokens ? load_id(a.ids, a.ids64, t0 + i, a.vocab) : -1;
  float v[kTokensPerBlock][8];
#pragma unroll
  for (int i = 0; i < kTokensPerBlock; ++i) {
    if (id[i] >= 0) {
      load_row8<VEC>(static_cast<const T*>(a.table) + (size_t)id[i] * a.ld_table, col, a.dim, v[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < kTokensPerBlock; ++i) {
    if (t0 + i >= a.tokens) break;
    if (id[i] >= 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] *= a.scale;
    }
    store_row8<VEC>(static_cast<O*>(a.out) + (t0 + i) * a.dim, col, a.dim, v[i]);
  }
}

template <typename T, typename O>
cudaError_t embed_of(const EmbedArgs& a, cudaStream_t stream) {
  const size_t slabs = (a.dim + kSlab - 1) / kSlab;
  const dim3 grid((unsigned)((a.tokens + kTokensPerBlock - 1) / kTokensPerBlock * slabs));
  return a.vec ? launch_kernel(embed_kernel<T, O, true>, grid, dim3(kRowThreads), 0, stream, a)
               : launch_kernel(embed_kernel<T, O, false>, grid, dim3(kRowThreads), 0, stream, a);
}

// ---- the sort --------------------------------------------------------------------

// One cluster sorts all tokens by least-significant digits.  Each warp owns a
// contiguous piece of the list, so counting its digits, a prefix sum over
// (digit, block, warp) and handing out places in the piece's order keeps the
// sort stable.
constexpr int kSortBlocks = 8;       // one cluster
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kDigitBits = 9;
constexpr int kDigits = 1 << kDigitBits;
constexpr size_t kSortShared = (size_t)(kSortWarps * kDigits + 2 * kDigits) * sizeof(uint32_t);

// What the gradient keeps in its workspace.  Keys are ids, with `vocab` for
// padding, which therefore sorts to the end.
struct GradPlan {
  uint32_t* keys[2];      // [tokens] each: the list before and after a digit
  uint32_t* order[2];     // [tokens] each: token of each place of the list
  uint32_t* starts;       // [tokens]: first places of the items, in no order
  uint32_t* count;        // [1]: how many items there are
  uint32_t* present;      // [ceil(vocab/32)]: one bit for each row with a token
  float* part;            // [2 windows][dim]: sums of runs that cross windows
  int window;             // places of the sorted list in one window
  int passes, bits;       // digits, and bits of each
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// reads a word of another block's shared memory
__device__ __forceinline__ uint32_t peer_word(const uint32_t* p, int rank) {
  uint32_t at = (uint32_t)__cvta_generic_to_shared(p), peer, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(peer) : "r"(at), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(peer) : "memory");
  return v;
}

__global__ void __launch_bounds__(kSortThreads)
    sort_kernel(const void* ids, int ids64, uint32_t tokens, uint32_t vocab, const GradPlan p) {
  extern __shared__ uint32_t sm[];
  uint32_t* counts = sm;                          // [warps][digits]
  uint32_t* total = sm + kSortWarps * kDigits;    // [digits]: this block's
  uint32_t* base = total + kDigits;               // [digits]
  pdl_wait_then_release();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x;  // the grid is one cluster
  const int gtid = rank * kSortThreads + tid;

  for (uint32_t i = gtid; i < (vocab + 31) / 32; i += kSortBlocks * kSortThreads) p.present[i] = 0;
  if (gtid == 0) *p.count = 0;

  // this warp's piece of the list, a multiple of 32 places
  const uint32_t pieces = kSortBlocks * kSortWarps;
  const uint32_t piece = ((tokens + pieces - 1) / pieces + 31) / 32 * 32;
  const uint64_t from = (uint64_t)(rank * kSortWarps + warp) * piece;
  const uint32_t lo = from < tokens ? (uint32_t)from : tokens;
  const uint32_t hi = from + piece < tokens ? (uint32_t)(from + piece) : tokens;
  const int digits = 1 << p.bits;

  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * p.bits;
    const uint32_t* kin = p.keys[pass & 1];
    const uint32_t* oin = p.order[pass & 1];
    uint32_t* kout = p.keys[(pass & 1) ^ 1];
    uint32_t* oout = p.order[(pass & 1) ^ 1];
    uint32_t* mine = counts + warp * kDigits;
    for (int d = lane; d < digits; d += 32) mine[d] = 0;
    __syncwarp();
    for (uint32_t i = lo + lane; i < hi; i += 32) {
      uint32_t key;
      if (pass == 0) {
        const int64_t id = load_id(ids, ids64, i, vocab);
        key = id < 0 ? vocab : (uint32_t)id;
      } else {
        key = kin[i];
      }
      atomicAdd(&mine[(key >> shift) & (digits - 1)], 1u);
    }
    __syncthreads();
    // counts of the warps before this one, and the block's totals
    for (int d = tid; d < digits; d += kSortThreads) {
      uint32_t s = 0;
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = counts[w * kDigits + d];
        counts[w * kDigits + d] = s;
        s += c;
      }
      total[d] = s;
    }
    cluster_sync();
    // places before this block's first of each digit: smaller digits of all
    // blocks, and the same digit of earlier blocks
    if (tid < digits) {
      uint32_t before = 0, all = 0;
      for (int b = 0; b < kSortBlocks; ++b) {
        const uint32_t c = peer_word(&total[tid], b);
        before += b < rank ? c : 0;
        all += c;
      }
      base[tid] = all;
      counts[tid] += before;  // warp 0's row holds zeros: it carries the block's offset
    }
    __syncthreads();
    // exclusive prefix sum of base over the digits (at most 512), by warp 0
    if (warp == 0) {
      uint32_t run = 0;
      for (int d0 = 0; d0 < digits; d0 += 32) {
        const uint32_t c = d0 + lane < digits ? base[d0 + lane] : 0;
        uint32_t s = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, s, o);
          if (lane >= o) s += u;
        }
        if (d0 + lane < digits) base[d0 + lane] = run + s - c;
        run += __shfl_sync(0xFFFFFFFFu, s, 31);
      }
    }
    __syncthreads();
    for (int d = tid; d < digits; d += kSortThreads) {
      const uint32_t before = counts[d];  // earlier blocks
      base[d] += before;
      counts[d] = 0;
    }
    __syncthreads();
    for (uint32_t i0 = lo; i0 < hi; i0 += 32) {
      const uint32_t i = i0 + lane;
      const bool live = i < hi;
      uint32_t key = 0, tok = i;
      if (live) {
        if (pass == 0) {
          const int64_t id = load_id(ids, ids64, i, vocab);
          key = id < 0 ? vocab : (uint32_t)id;
        } else {
          key = kin[i];
          tok = oin[i];
        }
      }
      const uint32_t d = live ? (key >> shift) & (digits - 1) : 0xFFFFFFFFu;
      const uint32_t same = __match_any_sync(0xFFFFFFFFu, d);
      const uint32_t ahead = __popc(same & ((1u << lane) - 1u));
      uint32_t at = 0;
      if (live) at = base[d] + mine[d] + ahead;
      __syncwarp();
      if (live && ahead == 0) mine[d] += __popc(same);
      __syncwarp();
      if (live) {
        kout[at] = key;
        oout[at] = tok;
      }
    }
    cluster_sync();  // the list is whole, and no block still reads `total`
  }

  // items: runs of one key, cut where a window ends
  const uint32_t* keys = p.keys[p.passes & 1];
  for (uint32_t i0 = lo; i0 < hi; i0 += 32) {
    const uint32_t i = i0 + lane;
    bool starts = false;
    if (i < hi) {
      const uint32_t key = keys[i];
      const bool first = i == 0 || keys[i - 1] != key;
      starts = key < vocab && (first || i % p.window == 0);
      if (key < vocab && first) atomicOr(&p.present[key / 32], 1u << (key % 32));
    }
    const uint32_t who = __ballot_sync(0xFFFFFFFFu, starts);
    uint32_t at = 0;
    if (lane == 0 && who) at = atomicAdd(p.count, (uint32_t)__popc(who));
    at = __shfl_sync(0xFFFFFFFFu, at, 0);
    if (starts) p.starts[at + __popc(who & ((1u << lane) - 1u))] = i;
  }
}

// ---- the sums --------------------------------------------------------------------

// Every row of dW without a token is set to zero (when not accumulating), and
// every item is summed.  Work is (row or item, slab of columns), dealt to the
// blocks in turn; which block takes which changes no result.
template <typename T, typename G, bool VEC>
__global__ void __launch_bounds__(kRowThreads) sum_kernel(const EmbedGradArgs a, const GradPlan p) {
  pdl_wait_then_release();
  const size_t slabs = (a.dim + kSlab - 1) / kSlab;
  const uint32_t* keys = p.keys[p.passes & 1];
  const uint32_t* order = p.order[p.passes & 1];
  const uint32_t tokens = (uint32_t)a.tokens;
  const size_t items = (size_t)*p.count * slabs;
  for (size_t j = blockIdx.x; j < items; j += gridDim.x) {
    const size_t col = j % slabs * kSlab + threadIdx.x * 8;
    if (col >= a.dim) continue;
    const uint32_t start = p.starts[j / slabs];
    const uint32_t key = keys[start];
    const uint32_t stop = min(tokens, (start / p.window + 1) * p.window);
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    uint32_t i = start;
    for (; i < stop && keys[i] == key; ++i) {
      float v[8];
      load_row8<VEC>(static_cast<const T*>(a.dout) + (size_t)order[i] * a.ld_dout, col, a.dim, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] += v[e];
    }
    const bool before = start > 0 && keys[start - 1] == key;
    const bool after = i < tokens && keys[i] == key;
    if (before || after) {
      // a run that goes on: slot 2w when it comes from the window before, else 2w + 1
      store8(p.part + (size_t)(2 * (start / p.window) + (before ? 0 : 1)) *
                          ((a.dim + 7) / 8 * 8) + col, s);
    } else {
      G* out = static_cast<G*>(a.dtable) + (size_t)key * a.dim;
      float old[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (a.accumulate) load_row8<VEC>(out, col, a.dim, old);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] = old[e] + s[e] * a.scale;
      store_row8<VEC>(out, col, a.dim, s);
    }
  }
  if (a.accumulate) return;
  const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (size_t j = blockIdx.x; j < a.vocab * slabs; j += gridDim.x) {
    const size_t col = j % slabs * kSlab + threadIdx.x * 8, row = j / slabs;
    if (col < a.dim && !(p.present[row / 32] >> (row % 32) & 1u))
      store_row8<VEC>(static_cast<G*>(a.dtable) + row * a.dim, col, a.dim, zero);
  }
}

// Joins a run that crosses windows, at the window where it begins: that
// window's slot 2w + 1, then slot 2w of each window the run reaches.
template <typename G, bool VEC>
__global__ void __launch_bounds__(kRowThreads) join_kernel(const EmbedGradArgs a, const GradPlan p) {
  pdl_wait_then_release();
  const size_t slabs = (a.dim + kSlab - 1) / kSlab;
  const size_t w = blockIdx.x / slabs;
  const size_t col = blockIdx.x % slabs * kSlab + threadIdx.x * 8;
  if (col >= a.dim) return;
  const uint32_t* keys = p.keys[p.passes & 1];
  const size_t next = (w + 1) * p.window;  // < tokens: one block less than windows
  const uint32_t key = keys[next];
  if (key >= a.vocab || keys[next - 1] != key) return;  // no run crosses here
  if (keys[w * p.window] == key && w > 0 && keys[w * p.window - 1] == key) return;  // begun earlier
  const size_t ld = (a.dim + 7) / 8 * 8;
  float s[8];
  load8(p.part + (2 * w + 1) * ld + col, s);
  for (size_t at = next; at < a.tokens && keys[at] == key; at += p.window) {
    float v[8];
    load8(p.part + 2 * (at / p.window) * ld + col, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] += v[e];
  }
  G* out = static_cast<G*>(a.dtable) + (size_t)key * a.dim;
  float old[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (a.accumulate) load_row8<VEC>(out, col, a.dim, old);
#pragma unroll
  for (int e = 0; e < 8; ++e) s[e] = old[e] + s[e] * a.scale;
  store_row8<VEC>(out, col, a.dim, s);
}

// A run of c tokens costs its window's length in one block, then c / window
// rows in the join: windows grow with the list.
int grad_window(size_t tokens) { return tokens <= 4096 ? 32 : tokens <= 65536 ? 64 : 256; }

GradPlan grad_plan(void* ws, size_t tokens, size_t vocab, size_t dim, size_t* bytes) {
  GradPlan p = {};
  size_t at = 0;
  char* base = static_cast<char*>(ws);
  auto take = [&](size_t n) {
    char* q = base + at;
    at += (n + 255) / 256 * 256;
    return reinterpret_cast<void*>(q);
  };
  p.window = grad_window(tokens);
  const size_t windows = (tokens + p.window - 1) / p.window;
  for (int k = 0; k < 2; ++k) p.keys[k] = static_cast<uint32_t*>(take(tokens * 4));
  for (int k = 0; k < 2; ++k) p.order[k] = static_cast<uint32_t*>(take(tokens * 4));
  p.starts = static_cast<uint32_t*>(take(tokens * 4));
  p.count = static_cast<uint32_t*>(take(4));
  p.present = static_cast<uint32_t*>(take((vocab + 31) / 32 * 4));
  p.part = static_cast<float*>(take(windows > 1 ? 2 * windows * ((dim + 7) / 8 * 8) * 4 : 0));
  int need = 1;  // bits that hold ids and `vocab`, the padding's key
  while (need < 32 && (vocab >> need)) ++need;
  p.passes = (need + kDigitBits - 1) / kDigitBits;
  p.bits = (need + p.passes - 1) / p.passes;
  *bytes = at;
  return p;
}

template <typename T, typename G, bool VEC>
cudaError_t sums_of(const EmbedGradArgs& a, const GradPlan& p, cudaStream_t stream,
                    uint64_t* launches) {
  const size_t slabs = (a.dim + kSlab - 1) / kSlab;
  const size_t most = (a.tokens + (a.accumulate ? 0 : a.vocab)) * slabs;
  const size_t fill = (size_t)sm_count() * 8;
  cudaError_t e = launch_kernel(sum_kernel<T, G, VEC>, dim3((unsigned)std::min(most, fill)),
                                dim3(kRowThreads), 0, stream, a, p);
  if (e != cudaSuccess) return e;
  ++*launches;
  const size_t windows = (a.tokens + p.window - 1) / p.window;
  if (windows < 2) return cudaSuccess;
  e = launch_kernel(join_kernel<G, VEC>, dim3((unsigned)((windows - 1) * slabs)),
                    dim3(kRowThreads), 0, stream, a, p);
  if (e == cudaSuccess) ++*launches;
  return e;
}

template <typename T, typename G>
cudaError_t sums_of(const EmbedGradArgs& a, const GradPlan& p, cudaStream_t stream,
                    uint64_t* launches) {
  return a.vec ? sums_of<T, G, true>(a, p, stream, launches)
               : sums_of<T, G, false>(a, p, stream, launches);
}

}  // namespace

cudaError_t launch_embedding_forward(const EmbedArgs& a, cudaStream_t stream) {
  if (a.table_type == RCC_F32)
    return a.out_type == RCC_F32 ? embed_of<float, float>(a, stream)
                                 : embed_of<float, __nv_bfloat16>(a, stream);
  return a.out_type == RCC_F32 ? embed_of<__nv_bfloat16, float>(a, stream)
                               : embed_of<__nv_bfloat16, __nv_bfloat16>(a, stream);
}

size_t embedding_backward_workspace(size_t tokens, size_t vocab, size_t dim) {
  size_t bytes = 0;
  grad_plan(nullptr, tokens, vocab, dim, &bytes);
  return bytes;
}

cudaError_t launch_embedding_backward(const EmbedGradArgs& a, cudaStream_t stream,
                                      uint64_t* launches) {
  size_t bytes = 0;
  const GradPlan p = grad_plan(a.workspace, a.tokens, a.vocab, a.dim, &bytes);
  cudaError_t e = cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)kSortShared);
  if (e != cudaSuccess) return e;
  e = launch_cluster(sort_kernel, dim3(kSortBlocks), dim3(kSortThreads), kSortShared, kSortBlocks,
                     stream, a.ids, a.ids64, (uint32_t)a.tokens, (uint32_t)a.vocab, p);
  if (e != cudaSuccess) return e;
  *launches = 1;
  if (a.dout_type == RCC_F32)
    return a.dtable_type == RCC_F32 ? sums_of<float, float>(a, p, stream, launches)
                                    : sums_of<float, __nv_bfloat16>(a, p, stream, launches);
  return a.dtable_type == RCC_F32 ? sums_of<__nv_bfloat16, float>(a, p, stream, launches)
                                  : sums_of<__nv_bfloat16, __nv_bfloat16>(a, p, stream, launches);
}

}  // namespace lm
}  // namespace rcc
