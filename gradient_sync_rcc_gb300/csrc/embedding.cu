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

// G threads take one slab of 8 G columns of a row; a block has kRowThreads / G
// such groups.  A warp to a row up to 512 columns, else the whole block.
template <int G>
struct Groups {
  static constexpr int kCount = kRowThreads / G;
  static constexpr int kColumns = G * 8;
};
constexpr size_t kWarpRow = 512;

// ---- forward -------------------------------------------------------------------

// Bound by its reads and writes: all rows of a group's tokens are asked for
// before the first is used.  32,768 tokens of 4,096 fp32 columns out of 131,072
// rows as bf16: 4 tokens 78.6 us (5.9 TB/s), 1 95.9, 8 79.5; of bf16 rows 64.8,
// 87.2, 72.8.
constexpr int kTokens = 4;

template <typename T, typename O, bool VEC, int G>
__global__ void __launch_bounds__(kRowThreads) embed_kernel(const EmbedArgs a) {
  using Gr = Groups<G>;
  pdl_wait_then_release();
  const size_t slabs = (a.dim + Gr::kColumns - 1) / Gr::kColumns;
  const size_t j = (size_t)blockIdx.x * Gr::kCount + threadIdx.x / G;
  const size_t t0 = j / slabs * kTokens, base = j % slabs * Gr::kColumns;
  const int t = threadIdx.x % G;
  if (t0 >= a.tokens || !slab_live<VEC, G>(base, t, a.dim)) return;
  int64_t id[kTokens];
#pragma unroll
  for (int i = 0; i < kTokens; ++i)
    id[i] = t0 + i < a.tokens ? load_id(a.ids, a.ids64, t0 + i, a.vocab) : -1;
  float v[kTokens][8];
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    if (id[i] >= 0) {
      load_slab<VEC, G>(static_cast<const T*>(a.table) + (size_t)id[i] * a.ld_table, base, t, a.dim,
                        v[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    if (t0 + i >= a.tokens) break;
    if (id[i] >= 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] *= a.scale;
    }
    store_slab<VEC, G>(static_cast<O*>(a.out) + (t0 + i) * a.dim, base, t, a.dim, v[i]);
  }
}

template <typename T, typename O, bool VEC, int G>
cudaError_t embed_by(const EmbedArgs& a, cudaStream_t stream) {
  using Gr = Groups<G>;
  const size_t slabs = (a.dim + Gr::kColumns - 1) / Gr::kColumns;
  const size_t groups = (a.tokens + kTokens - 1) / kTokens * slabs;
  return launch_kernel(embed_kernel<T, O, VEC, G>,
                       dim3((unsigned)((groups + Gr::kCount - 1) / Gr::kCount)), dim3(kRowThreads),
                       0, stream, a);
}

template <typename T, typename O>
cudaError_t embed_of(const EmbedArgs& a, cudaStream_t stream) {
  if (a.dim <= kWarpRow)
    return a.vec ? embed_by<T, O, true, 32>(a, stream) : embed_by<T, O, false, 32>(a, stream);
  return a.vec ? embed_by<T, O, true, kRowThreads>(a, stream)
               : embed_by<T, O, false, kRowThreads>(a, stream);
}

// ---- the sort --------------------------------------------------------------------

// One block or one cluster of blocks sorts all tokens by least-significant
// digits.  Each warp owns a contiguous piece of the list, so counting its
// digits, a prefix sum over (digit, block, warp) and handing out places in the
// piece's order keeps the sort stable.
constexpr int kSortBlocks = 8;       // of the cluster
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
  uint2* items;           // [tokens]: (first place, key) of the items, in no order
  uint32_t* count;        // [1]: how many items there are
  uint32_t* present;      // [ceil(vocab/32)]: one bit for each row with a token
  float* part;            // [2 windows][dim]: sums of runs that cross windows
  int window;             // places of the sorted list in one window
  int passes, bits;       // digits, and bits of each
  bool mark;              // `present` is wanted
};

// the list after its last digit
__device__ __forceinline__ const uint32_t* sorted_keys(const GradPlan& p) {
  return p.passes & 1 ? p.keys[1] : p.keys[0];
}
__device__ __forceinline__ const uint32_t* sorted_order(const GradPlan& p) {
  return p.passes & 1 ? p.order[1] : p.order[0];
}

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

// every thread of the sort: its block's, or the cluster's
template <int BLOCKS>
__device__ __forceinline__ void sort_sync() {
  if constexpr (BLOCKS > 1)
    cluster_sync();
  else
    __syncthreads();
}

// HOLD: groups of 32 places of its piece that a warp holds in registers
template <int BLOCKS, int HOLD>
__global__ void __launch_bounds__(kSortThreads)
    sort_kernel(const void* ids, int ids64, uint32_t tokens, uint32_t vocab, const GradPlan p) {
  extern __shared__ uint32_t sm[];
  uint32_t* counts = sm;                          // [warps][digits]
  uint32_t* total = sm + kSortWarps * kDigits;    // [digits]: this block's
  uint32_t* base = total + kDigits;               // [digits]
  __shared__ uint32_t warp_total[kDigits / 32];
  pdl_wait_then_release();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x;  // the grid is one cluster
  const int gtid = rank * kSortThreads + tid;

  if (p.mark)
    for (uint32_t i = gtid; i < (vocab + 31) / 32; i += BLOCKS * kSortThreads) p.present[i] = 0;
  if (gtid == 0) *p.count = 0;

  // this warp's piece of the list, a multiple of 32 places
  const uint32_t pieces = BLOCKS * kSortWarps;
  const uint32_t piece = ((tokens + pieces - 1) / pieces + 31) / 32 * 32;
  const uint64_t from = (uint64_t)(rank * kSortWarps + warp) * piece;
  const uint32_t lo = from < tokens ? (uint32_t)from : tokens;
  const uint32_t hi = from + piece < tokens ? (uint32_t)(from + piece) : tokens;
  const int digits = 1 << p.bits;

  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * p.bits;
    const uint32_t* kin = pass & 1 ? p.keys[1] : p.keys[0];
    const uint32_t* oin = pass & 1 ? p.order[1] : p.order[0];
    uint32_t* kout = pass & 1 ? p.keys[0] : p.keys[1];
    uint32_t* oout = pass & 1 ? p.order[0] : p.order[1];
    uint32_t* mine = counts + warp * kDigits;
    for (int d = lane; d < digits; d += 32) mine[d] = 0;
    __syncwarp();
    // HOLD groups of 32 places are read at once
    uint32_t key[HOLD], tok[HOLD];
    auto read = [&](uint32_t i0) {
#pragma unroll
      for (int h = 0; h < HOLD; ++h) {
        const uint32_t i = i0 + h * 32 + lane;
        key[h] = vocab;
        tok[h] = i;
        if (i < hi) {
          if (pass == 0) {
            const int64_t id = load_id(ids, ids64, i, vocab);
            key[h] = id < 0 ? vocab : (uint32_t)id;
          } else {
            key[h] = kin[i];
            tok[h] = oin[i];
          }
        }
      }
    };
    for (uint32_t i0 = lo; i0 < hi; i0 += 32 * HOLD) {
      read(i0);
#pragma unroll
      for (int h = 0; h < HOLD; ++h)
        if (i0 + h * 32 + lane < hi) atomicAdd(&mine[(key[h] >> shift) & (digits - 1)], 1u);
    }
    __syncthreads();
    // counts of the warps before this one, and the block's totals: two threads
    // a digit, 16 warps each (every thread takes part in the exchange)
    {
      static_assert(kSortThreads == 2 * kDigits, "two threads a digit");
      const int d = tid >> 1;
      uint32_t* c = counts + (tid & 1) * (kSortWarps / 2) * kDigits + d;
      uint32_t v[kSortWarps / 2], s = 0;
#pragma unroll
      for (int w = 0; w < kSortWarps / 2; ++w) v[w] = d < digits ? c[w * kDigits] : 0;
#pragma unroll
      for (int w = 0; w < kSortWarps / 2; ++w) s += v[w];
      const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, s, 1);
      uint32_t run = tid & 1 ? other : 0;
      if (d < digits) {
#pragma unroll
        for (int w = 0; w < kSortWarps / 2; ++w) {
          c[w * kDigits] = run;
          run += v[w];
        }
        if (tid & 1) total[d] = run;
      }
    }
    sort_sync<BLOCKS>();
    // places before this block's first of each digit: smaller digits of all
    // blocks, and the same digit of earlier blocks
    uint32_t before = 0, all = 0, upto = 0;
    if (tid < kDigits) {  // whole warps
      if (tid < digits) {
        uint32_t c[BLOCKS];
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b)
          c[b] = BLOCKS > 1 ? peer_word(&total[tid], b) : total[tid];
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) {
          before += b < rank ? c[b] : 0;
          all += c[b];
        }
      }
      upto = all;  // with the digits before it in the warp
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += u;
      }
      if (lane == 31) warp_total[warp] = upto;
    }
    __syncthreads();
    if (tid < digits) {
      uint32_t s = upto - all + before;
#pragma unroll
      for (int w = 0; w < kDigits / 32; ++w) s += w < warp ? warp_total[w] : 0;
      base[tid] = s;
    }
    __syncthreads();
    for (uint32_t i0 = lo; i0 < hi; i0 += 32 * HOLD) {
      if (piece > 32 * HOLD) read(i0);  // a piece of up to HOLD groups is still held
#pragma unroll
      for (int h = 0; h < HOLD; ++h) {
        if (i0 + h * 32 >= hi) break;
        const bool live = i0 + h * 32 + lane < hi;
        const uint32_t d = live ? (key[h] >> shift) & (digits - 1) : 0xFFFFFFFFu;
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, d);
        const uint32_t ahead = __popc(same & ((1u << lane) - 1u));
        uint32_t at = 0;
        if (live) at = base[d] + mine[d] + ahead;
        __syncwarp();
        if (live && ahead == 0) mine[d] += __popc(same);
        __syncwarp();
        if (live) {
          kout[at] = key[h];
          oout[at] = tok[h];
        }
      }
    }
    sort_sync<BLOCKS>();  // the list is whole, and no block still reads `total`
  }

  // items: runs of one key, cut where a window ends
  const uint32_t* keys = sorted_keys(p);
  for (uint32_t i0 = lo; i0 < hi; i0 += 32) {
    const uint32_t i = i0 + lane;
    bool starts = false;
    uint32_t key = vocab;
    if (i < hi) {
      key = keys[i];
      const bool first = i == 0 || keys[i - 1] != key;
      starts = key < vocab && (first || i % p.window == 0);
      if (p.mark && key < vocab && first) atomicOr(&p.present[key / 32], 1u << (key % 32));
    }
    const uint32_t who = __ballot_sync(0xFFFFFFFFu, starts);
    uint32_t at = 0;
    if (lane == 0 && who) at = atomicAdd(p.count, (uint32_t)__popc(who));
    at = __shfl_sync(0xFFFFFFFFu, at, 0);
    if (starts) p.items[at + __popc(who & ((1u << lane) - 1u))] = make_uint2(i, key);
  }
}

// Few tokens: a thread a token, whose place is the number of smaller
// (id, token) pairs.
constexpr int kFewTokens = 256;
__global__ void __launch_bounds__(kFewTokens)
    sort_few_kernel(const void* ids, int ids64, uint32_t tokens, uint32_t vocab, const GradPlan p) {
  __shared__ __align__(16) uint32_t keys[kFewTokens];
  __shared__ uint32_t sorted[kFewTokens];
  __shared__ uint32_t count;
  pdl_wait_then_release();
  const uint32_t i = threadIdx.x;
  if (p.mark)
    for (uint32_t w = i; w < (vocab + 31) / 32; w += kFewTokens) p.present[w] = 0;
  uint32_t key = 0xFFFFFFFFu;
  if (i < tokens) {
    const int64_t id = load_id(ids, ids64, i, vocab);
    key = id < 0 ? vocab : (uint32_t)id;
  }
  keys[i] = key;
  if (i == 0) count = 0;
  __syncthreads();
  uint32_t at = 0;
  for (uint32_t j = 0; j < tokens; j += 4) {
    const uint4 k = *reinterpret_cast<const uint4*>(keys + j);  // past the tokens: the largest
    at += (k.x < key || (k.x == key && j < i)) + (k.y < key || (k.y == key && j + 1 < i)) +
          (k.z < key || (k.z == key && j + 2 < i)) + (k.w < key || (k.w == key && j + 3 < i));
  }
  uint32_t* list = p.passes & 1 ? p.keys[1] : p.keys[0];
  uint32_t* order = p.passes & 1 ? p.order[1] : p.order[0];
  if (i < tokens) {
    sorted[at] = key;
    list[at] = key;
    order[at] = i;
  }
  __syncthreads();
  if (i < tokens) {
    key = sorted[i];
    const bool first = i == 0 || sorted[i - 1] != key;
    if (key < vocab && (first || i % p.window == 0))
      p.items[atomicAdd(&count, 1u)] = make_uint2(i, key);
    if (p.mark && key < vocab && first) atomicOr(&p.present[key / 32], 1u << (key % 32));
  }
  __syncthreads();
  if (i == 0) *p.count = count;
}

// ---- the sums --------------------------------------------------------------------

// s += U rows of dout, whose tokens lanes j to j + U - 1 hold.  All rows are
// asked for before the first is used: a thread whose columns do not exist
// reads the slab's first ones (t = 0) rather than waiting behind a branch.
template <int U, typename T, bool VEC, int G>
__device__ __forceinline__ void add_rows(const EmbedGradArgs& a, uint32_t tok, int j, size_t base,
                                         int t, float (&s)[8]) {
  float v[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t of = __shfl_sync(0xFFFFFFFFu, tok, j + u);
    load_slab<VEC, G>(static_cast<const T*>(a.dout) + (size_t)of * a.ld_dout, base, t, a.dim, v[u]);
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] += v[u][e];
}

// The sum of an item's rows of dout, in the order of the list.  The places are
// read 32 at a time, the rows four at a time.
template <typename T, bool VEC, int G>
__device__ __forceinline__ void sum_item(const EmbedGradArgs& a, const uint32_t* keys,
                                         const uint32_t* order, uint32_t key, uint32_t start,
                                         uint32_t stop, size_t base, int t, float (&s)[8]) {
  const int lane = threadIdx.x & 31;
  for (uint32_t i0 = start; i0 < stop; i0 += 32) {
    const uint32_t i = i0 + lane;
    uint32_t k = ~0u, tok = 0;
    if (i < stop) {
      k = keys[i];
      tok = order[i];
    }
    const int n = __popc(__ballot_sync(0xFFFFFFFFu, k == key));  // a run: the first n lanes
    int j = 0;
    for (; j + 4 <= n; j += 4) add_rows<4, T, VEC, G>(a, tok, j, base, t, s);
    if (n - j >= 2) {
      add_rows<2, T, VEC, G>(a, tok, j, base, t, s);
      j += 2;
    }
    if (n - j >= 1) add_rows<1, T, VEC, G>(a, tok, j, base, t, s);
    if (n < 32) break;
  }
}

// Blocks of the sums for each SM, of which kSumResident are there at a time:
// the more, the evener the load, as items differ in length.  32,768 tokens,
// 131,072 x 4,096 in fp32 (8,191 tokens added to 50,021 x 2,048): 64 blocks 403
// (43.7) us, 32 411 (43.4), 16 420 (44.0), 8 450 (46.8).
constexpr int kSumBlocks = 64, kSumResident = 4;

// Every row of dW without a token is set to zero (when not accumulating), and
// every item is summed.  Work is dealt to the blocks in turn; which block
// takes which changes no result.  Half of the blocks begin with the zeros, so
// that writing and summing overlap.
template <typename T, typename O, bool VEC, int G>
__global__ void __launch_bounds__(kRowThreads, kSumResident) sum_kernel(const EmbedGradArgs a, const GradPlan p) {
  using Gr = Groups<G>;
  pdl_wait_then_release();
  const size_t slabs = (a.dim + Gr::kColumns - 1) / Gr::kColumns;
  const uint32_t* keys = sorted_keys(p);
  const uint32_t* order = sorted_order(p);
  const uint32_t tokens = (uint32_t)a.tokens;
  const size_t group = (size_t)blockIdx.x * Gr::kCount + threadIdx.x / G;
  const size_t all_groups = (size_t)gridDim.x * Gr::kCount;
  const int t = threadIdx.x % G;

  auto zeros = [&]() {
    // a byte of the bit map, eight rows, at a time
    const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const size_t units = (a.vocab + 7) / 8 * slabs;
    for (size_t j = group; j < units; j += all_groups) {
      const size_t base = j % slabs * Gr::kColumns, row0 = j / slabs * 8;
      const uint32_t bits = reinterpret_cast<const uint8_t*>(p.present)[row0 / 8];
      if (!slab_live<VEC, G>(base, t, a.dim)) continue;
      O* out = static_cast<O*>(a.dtable) + row0 * a.dim;
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (row0 + r < a.vocab && !(bits >> r & 1u))
          store_slab<VEC, G>(out + r * a.dim, base, t, a.dim, zero);
    }
  };
  const bool zeros_first = blockIdx.x & 1;
  if (!a.accumulate && zeros_first) zeros();

  const size_t items = (size_t)*p.count * slabs;
  uint2 next = make_uint2(0u, 0u);
  if (group < items) next = p.items[group / slabs];
  for (size_t j = group; j < items; j += all_groups) {
    const size_t base = j % slabs * Gr::kColumns;
    const bool live = slab_live<VEC, G>(base, t, a.dim);
    const uint32_t start = next.x, key = next.y;
    if (j + all_groups < items) next = p.items[(j + all_groups) / slabs];
    const uint32_t stop = min(tokens, (start / p.window + 1) * p.window);
    const bool before = start > 0 && keys[start - 1] == key;
    const bool after = stop < tokens && keys[stop] == key && keys[stop - 1] == key;
    O* out = static_cast<O*>(a.dtable) + (size_t)key * a.dim;
    float old[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (a.accumulate && live && !before && !after)
      load_slab<VEC, G>(out, base, t, a.dim, old);
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    sum_item<T, VEC, G>(a, keys, order, key, start, stop, base, live ? t : 0, s);
    if (!live) continue;
    if (before || after) {
      // a run that goes on: slot 2w when it comes from the window before, else 2w + 1
      store_slab<VEC, G>(p.part + (size_t)(2 * (start / p.window) + (before ? 0 : 1)) * a.dim, base,
                         t, a.dim, s);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] = old[e] + s[e] * a.scale;
      store_slab<VEC, G>(out, base, t, a.dim, s);
    }
  }
  if (!a.accumulate && !zeros_first) zeros();
}

// Joins a run that crosses windows, at the window where it begins: that
// window's slot 2w + 1, then slot 2w of each window the run reaches.
template <typename O, bool VEC, int G>
__global__ void __launch_bounds__(kRowThreads) join_kernel(const EmbedGradArgs a, const GradPlan p,
                                                           uint32_t windows) {
  using Gr = Groups<G>;
  pdl_wait_then_release();
  const size_t slabs = (a.dim + Gr::kColumns - 1) / Gr::kColumns;
  const size_t j = (size_t)blockIdx.x * Gr::kCount + threadIdx.x / G;
  const uint32_t w = (uint32_t)(j / slabs);
  if (w + 1 >= windows) return;  // whole warps
  const size_t base = j % slabs * Gr::kColumns;
  const int t = threadIdx.x % G;
  const uint32_t* keys = sorted_keys(p);
  const uint32_t next = (w + 1) * p.window;  // < tokens
  const uint32_t key = keys[next];
  if (key >= a.vocab || keys[next - 1] != key) return;  // no run crosses here
  if (w > 0 && keys[w * p.window] == key && keys[w * p.window - 1] == key) return;  // begun earlier
  const int lane = threadIdx.x & 31;
  const bool live = slab_live<VEC, G>(base, t, a.dim);
  O* out = static_cast<O*>(a.dtable) + (size_t)key * a.dim;
  float s[8], old[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (live) load_slab<VEC, G>(p.part + (2 * (size_t)w + 1) * a.dim, base, t, a.dim, s);
  if (live && a.accumulate) load_slab<VEC, G>(out, base, t, a.dim, old);
  for (uint32_t v0 = w + 1; v0 < windows; v0 += 32) {
    const uint32_t at = v0 + lane;
    const int n = __popc(__ballot_sync(0xFFFFFFFFu, at < windows && keys[at * p.window] == key));
    if (live) {
      for (int i = 0; i < n; i += 8) {
        float v[8][8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (i + u < n)
            load_slab<VEC, G>(p.part + 2 * (size_t)(v0 + i + u) * a.dim, base, t, a.dim, v[u]);
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (i + u < n) {
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] += v[u][e];
          }
      }
    }
    if (n < 32) break;
  }
  if (!live) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) s[e] = old[e] + s[e] * a.scale;
  store_slab<VEC, G>(out, base, t, a.dim, s);
}

// A run of c tokens costs its window's length in one block, then c / window
// rows in the join: windows grow with the list.
// Up to 128 tokens are one window, and nothing has to be joined.
int grad_window(size_t tokens) {
  return tokens <= 128 ? 128 : tokens <= 4096 ? 32 : tokens <= 65536 ? 64 : 256;
}

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
  p.items = static_cast<uint2*>(take(tokens * sizeof(uint2)));
  p.count = static_cast<uint32_t*>(take(4));
  p.present = static_cast<uint32_t*>(take((vocab + 31) / 32 * 4));
  p.part = static_cast<float*>(take(windows > 1 ? 2 * windows * dim * 4 : 0));
  int need = 1;  // bits that hold ids and `vocab`, the padding's key
  while (need < 32 && (vocab >> need)) ++need;
  p.passes = (need + kDigitBits - 1) / kDigitBits;
  p.bits = (need + p.passes - 1) / p.passes;
  *bytes = at;
  return p;
}

template <typename T, typename O, bool VEC, int G>
cudaError_t sums_by(const EmbedGradArgs& a, const GradPlan& p, cudaStream_t stream,
                    uint64_t* launches) {
  using Gr = Groups<G>;
  const size_t slabs = (a.dim + Gr::kColumns - 1) / Gr::kColumns;
  const size_t most = (a.tokens + (a.accumulate ? 0 : (a.vocab + 7) / 8)) * slabs;
  const size_t blocks = (most + Gr::kCount - 1) / Gr::kCount;
  const size_t fill = (size_t)sm_count() * kSumBlocks;
  cudaError_t e = launch_kernel(sum_kernel<T, O, VEC, G>, dim3((unsigned)std::min(blocks, fill)),
                                dim3(kRowThreads), 0, stream, a, p);
  if (e != cudaSuccess) return e;
  ++*launches;
  const size_t windows = (a.tokens + p.window - 1) / p.window;
  if (windows < 2) return cudaSuccess;
  e = launch_kernel(join_kernel<O, VEC, G>,
                    dim3((unsigned)(((windows - 1) * slabs + Gr::kCount - 1) / Gr::kCount)),
                    dim3(kRowThreads), 0, stream, a, p, (uint32_t)windows);
  if (e == cudaSuccess) ++*launches;
  return e;
}

template <typename T, typename O>
cudaError_t sums_of(const EmbedGradArgs& a, const GradPlan& p, cudaStream_t stream,
                    uint64_t* launches) {
  if (a.dim <= kWarpRow)
    return a.vec ? sums_by<T, O, true, 32>(a, p, stream, launches)
                 : sums_by<T, O, false, 32>(a, p, stream, launches);
  return a.vec ? sums_by<T, O, true, kRowThreads>(a, p, stream, launches)
               : sums_by<T, O, false, kRowThreads>(a, p, stream, launches);
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
  GradPlan p = grad_plan(a.workspace, a.tokens, a.vocab, a.dim, &bytes);
  p.mark = !a.accumulate;
  // Measured, the whole gradient (50,021 x 2,048, accumulating): 8 tokens 4.9 us
  // by counting, 8.8 in one block; 256 tokens 10.2 and 13.2; 1,000 tokens 17.7
  // in one block, 19.6 in a cluster; 4,000 tokens 29.6 and 25.2.
  cudaError_t e;
  const uint32_t tokens = (uint32_t)a.tokens, vocab = (uint32_t)a.vocab;
  if (a.tokens <= (size_t)kFewTokens) {
    e = launch_kernel(sort_few_kernel, dim3(1), dim3(kFewTokens), 0, stream, a.ids, a.ids64, tokens,
                      vocab, p);
  } else if (a.tokens <= (size_t)kSortThreads) {
    static std::atomic<uint64_t> allowed{0};
    e = allow_shared(sort_kernel<1, 1>, (int)kSortShared, allowed);
    if (e != cudaSuccess) return e;
    e = launch_kernel(sort_kernel<1, 1>, dim3(1), dim3(kSortThreads), kSortShared, stream, a.ids,
                      a.ids64, tokens, vocab, p);
  } else {
    static std::atomic<uint64_t> allowed{0};
    e = allow_shared(sort_kernel<kSortBlocks, 4>, (int)kSortShared, allowed);
    if (e != cudaSuccess) return e;
    e = launch_cluster(sort_kernel<kSortBlocks, 4>, dim3(kSortBlocks), dim3(kSortThreads),
                       kSortShared, kSortBlocks, stream, a.ids, a.ids64, tokens, vocab, p);
  }
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
