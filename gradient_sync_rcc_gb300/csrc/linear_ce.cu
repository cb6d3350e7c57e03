// linear_ce.cu -- output layer and softmax cross entropy without keeping the
// logits, and its gradients.
//
//   z = x W^T      lse_t = log sum_v exp z_tv      loss_t = lse_t - z_t,label
//   dz = dloss_t / F (exp(z - lse_t) - [v = label])
//   dx = F dz W    dW = F dz^T x     F = the largest finite |dloss_t|
//
// Four matrix products on the tensor cores, all of them the one kernel below:
//   scores   x W^T, whose epilogue leaves one (max, sum) pair per row and
//            256 vocabulary entries; a small kernel joins the pairs
//   dz       x W^T again for a piece of the vocabulary, whose epilogue writes
//            dz of the piece in bf16 (for fp32 gradients as the sum of three
//            bf16 numbers, which hold all of its 24 bits)
//   dx       dz W, added up over the pieces
//   dW       dz^T x, the piece's rows; of x with zeros for padding tokens
// Sums are fp32 in tensor memory, softmax statistics fp32.  The common factor F
// stays out of dz: with one dloss for all tokens, as a mean has, its rounding
// would put the same error on every label's term (bf16 gradients 0.0026 off 64
// bits instead of 0.0020, of which the output's own rounding is 0.0017).
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "lm_common.cuh"
#include "lm_internal.h"

namespace rcc {
namespace lm {
namespace {

// ---- PTX ---------------------------------------------------------------------------

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// the same shared-memory address in block `rank` of the cluster
__device__ __forceinline__ uint32_t peer_addr(uint32_t at, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
// `bar` is an address of any block of the cluster.  Relaxed: the arrival
// publishes nothing of this thread's, only the bytes the copies will bring.
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(
                   bar), "r"(bytes) : "memory");
}
// Relaxed: what the arrival announces are reads of tensor memory, which are
// complete; a release would wait for this thread's stores of the tile before.
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
// Waits for a phase, at most about two seconds; false when that ran out.
constexpr long long kWaitCycles = 4000000000ll;
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity) {
  if (bar_try(bar, parity)) return true;
  const long long t0 = clock64();
  do {
    if (bar_try(bar, parity)) return true;
  } while (clock64() - t0 < kWaitCycles);
  return false;
}

// One box of a two-dimensional tensor map into this block's shared memory;
// the bytes count on `bar`, which with CG = 2 is the pair's first block's.
template <int CG>
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y,
                                         uint32_t bar) {
  if constexpr (CG == 2) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".cta_group::2 [%0], [%1, {%3, %4}], [%2];" ::"r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y)
        : "memory");
  } else {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y)
        : "memory");
  }
}

template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t dst, uint32_t cols) {
  if constexpr (CG == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst),
                 "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst),
                 "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
}
template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t at, uint32_t cols) {
  if constexpr (CG == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(cols));
  else
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(cols));
}
template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                    bool accumulate) {
  if constexpr (CG == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b),
        "r"(idesc), "r"((uint32_t)accumulate) : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b),
        "r"(idesc), "r"((uint32_t)accumulate) : "memory");
}
// Arrives on `bar` (in every block of the pair) once all products issued so
// far are done.
template <int CG>
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  if constexpr (CG == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(bar), "h"((uint16_t)3) : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     bar) : "memory");
}
__device__ __forceinline__ void tmem_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// v = 128 columns of this thread's row; the whole warp calls it
#define RCC_8(v, i) "=f"(v[i]), "=f"(v[i + 1]), "=f"(v[i + 2]), "=f"(v[i + 3]), \
                    "=f"(v[i + 4]), "=f"(v[i + 5]), "=f"(v[i + 6]), "=f"(v[i + 7])
#define RCC_32(v, i) RCC_8(v, i), RCC_8(v, i + 8), RCC_8(v, i + 16), RCC_8(v, i + 24)
__device__ __forceinline__ void tmem_load128(uint32_t at, float (&v)[128]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, "
      "%8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, "
      "%24, %25, %26, %27, %28, %29, %30, %31}, [%128];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%32, %33, %34, %35, %36, %37, %38, %39, "
      "%40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, "
      "%56, %57, %58, %59, %60, %61, %62, %63}, [%129];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%64, %65, %66, %67, %68, %69, %70, %71, "
      "%72, %73, %74, %75, %76, %77, %78, %79, "
      "%80, %81, %82, %83, %84, %85, %86, %87, "
      "%88, %89, %90, %91, %92, %93, %94, %95}, [%130];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%96, %97, %98, %99, %100, %101, %102, %103, "
      "%104, %105, %106, %107, %108, %109, %110, %111, "
      "%112, %113, %114, %115, %116, %117, %118, %119, "
      "%120, %121, %122, %123, %124, %125, %126, %127}, [%131];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : RCC_32(v, 0), RCC_32(v, 32), RCC_32(v, 64), RCC_32(v, 96)
      : "r"(at), "r"(at + 32), "r"(at + 64), "r"(at + 96)
      : "memory");
}
// v += 32 columns of this thread's row; the whole warp calls it
__device__ __forceinline__ void tmem_add32(uint32_t at, float* v) {
  float r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, "
      "%8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, "
      "%24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : RCC_32(r, 0)
      : "r"(at) : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] += r[i];
}

#undef RCC_32
#undef RCC_8

// ---- the product -------------------------------------------------------------------

constexpr int kBM = 128;   // rows of C of one block
constexpr int kBN = 256;   // columns of C of one block (of a pair: the same)
constexpr int kBK = 64;    // of the sum per stage: 128 bytes, one swizzle row
constexpr int kEpiWarps = 8;  // two for each 32 rows, half of the columns each
constexpr int kHalf = kBN / 2;
constexpr int kGemmThreads = 128 + 32 * kEpiWarps;
constexpr int kTmemCols = 512;  // two accumulators of kBN columns
// Additions on the tensor cores drop what does not fit the accumulator instead
// of rounding it, a loss that grows with their number (3.7e-5 of dx after
// 4,000 of them).  So an accumulator takes a few instructions of 16 products
// each, and the epilogue adds the accumulators up in registers, rounding to
// nearest.  Scores of 2,000 x 50,021 x 2,048, the loss's distance from 64 bits
// (plain fp32 sums 6.6e-7): 64 instructions 8.2e-7 and 237 us, 48 5.3e-7 and
// 242, 32 3.7e-7 and 244, 16 1.8e-7 and 266; where a pass waits for W anyway,
// 16: 100 x 50,021 x 1,024 1.8e-7 (plain 4.1e-7) and 21.1 us, 8 1.1e-7 and
// 23.5.  For fp32 gradients (2,048 x 32,000 x 1,024): 96 1.3e-6, 48 7e-7, 24
// 4.9e-7 for 1.5% of the time.  A gradient that is rounded to bf16 is taken
// whole, its accumulator as long as the sum: what that drops (3.7e-5 after
// 4,000 additions) is far below the rounding of dz and of the result.
constexpr int kScoreMmas = 48, kScoreMmasFew = 16, kOutMmas = 48;

// bf16 numbers that make one fp32 value of dz: 24 bits, eight each.  2,048 x
// 32,000 x 1,024: three leave dx and dW 7e-7 off 64 bits (plain fp32: 3.3e-6
// and 8e-7) and take 603 us, two 2.0e-6 and 1.7e-6 and 445 us.
constexpr int kMaxParts = 3;

enum Epi { kEpiStats = 0, kEpiDz = 1, kEpiOut = 2 };

struct GemmArgs {
  CUtensorMap a[kMaxParts], b;  // a[i]: the i-th bf16 number of A's values
  CUtensorMap c[kMaxParts];     // C in boxes of 32 rows of 128 bytes, or dz's parts
  int copy_out;                 // C goes out by TMA, through c
  int m, n;              // of C
  int m_tiles, n_tiles;  // of kBM * CG rows, of bn columns
  int bn;                // columns of a tile, a multiple of 16 up to kBN
  int a_rows;            // rows of A's box (not MN), a multiple of 8 up to kBM
  int stages, stage_size, a_bytes;  // in shared memory: how many, of what size, of it A's
  int k_blocks, splits;  // of bk; pieces of the sum, each with a C of its own
  int bk;                // of the sum per stage, a multiple of 16 up to kBK
  int chunk;             // k_blocks that one accumulator takes
  int group;             // tiles of rows that share a run over the columns
  int b_row0;            // first row of B (vocabulary entry) of this piece
  // stats
  float2* part;          // [2 n_tiles][m]
  float* zlab;           // [m]
  const void* labels;
  int labels64;
  int vocab;
  // dz and out
  const float* dloss;    // [tokens]
  int tokens;
  // dz
  const float* lse;
  __nv_bfloat16* dz[kMaxParts];  // [m][ld_dz], NULL past the parts
  size_t ld_dz;
  const uint4* x;        // [tokens] rows of x_words, ld_x apart
  uint4* x_copy;         // [tokens][x_words]: x, zeros for padding; or NULL
  size_t ld_x, x_words;
  // out
  void* out;
  size_t ld_c, split_stride;  // elements
  int c_type;
  int add;               // C += instead of C =
  int wide;              // C is on a 32-byte boundary
};

// Shared-memory descriptor of a tile in rows of 128 bytes, swizzled by 128.
// Along the sum (K major): a row holds 64 of the sum, eight rows are 1,024
// bytes.  Across it (MN major): a row holds 64 rows of the matrix, eight of
// the sum are 1,024 bytes, and 64 rows of the matrix a block of 128 bk.
template <bool MN>
__device__ __forceinline__ uint64_t smem_desc(uint32_t at, int bk) {
  uint64_t d = (uint64_t)((at >> 4) & 0x3FFF);
  d |= (uint64_t)(MN ? (bk * 128) >> 4 : 1) << 16;  // between blocks of 64 rows
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// Stages in shared memory: as many as fit, each a box of A (PARTS of them) and
// one of B on boundaries of 1,024 bytes.
constexpr int kStageMemory = 192 * 1024, kMaxStages = 24;
// After them the barriers, and for each warp of the epilogue 32 rows of 128
// bytes on their way to global memory.
constexpr int kBarBytes = 1024, kOutBytes = 32 * 128;
constexpr int kGemmShared = 1024 + kStageMemory + kBarBytes + kEpiWarps * kOutBytes;

struct Tile {
  int m, n, k0, k1, split;
};
__device__ __forceinline__ Tile tile_of(const GemmArgs& g, int t) {
  Tile r;
  const int plane = g.m_tiles * g.n_tiles;
  r.split = t / plane;
  t -= r.split * plane;
  const int band = g.group * g.n_tiles;
  const int m0 = t / band * g.group;
  t -= m0 * g.n_tiles;
  const int rows = min(g.group, g.m_tiles - m0);
  r.m = m0 + t % rows;
  r.n = t / rows;
  r.k0 = (int)((long long)g.k_blocks * r.split / g.splits);
  r.k1 = (int)((long long)g.k_blocks * (r.split + 1) / g.splits);
  return r;
}

constexpr float kLog2e = 1.44269504f;

// exp2, denormal results as zero
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 32 bytes on a boundary of 32
__device__ __forceinline__ void store_words(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Half a row of scores: (max, sum of exp) of the columns that exist.
__device__ __forceinline__ void epilogue_stats(const GemmArgs& g, float (&v)[kHalf], int row,
                                               int col0, int left, int slot, bool failed) {
  if (row >= g.m) return;
  float2* part = g.part + (size_t)slot * g.m + row;
  if (left <= 0) {
    *part = make_float2(-INFINITY, 0.f);
    return;
  }
  const float nan = __uint_as_float(0x7FC00000u);
  const int64_t at = load_id(g.labels, g.labels64, row, g.vocab) - col0;
  if (at >= 0 && at < left && at < kHalf) {
    float z = v[0];
#pragma unroll
    for (int i = 1; i < kHalf; ++i) z = i == at ? v[i] : z;
    g.zlab[row] = failed ? nan : z;
  }
  if (left < kHalf) {
#pragma unroll
    for (int i = 0; i < kHalf; ++i)
      if (i >= left) v[i] = -INFINITY;
  }
  float top[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
  for (int i = 4; i < kHalf; ++i) top[i & 3] = fmaxf(top[i & 3], v[i]);
  const float m = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
  // The difference is taken before it is scaled: the largest score gives 1
  // exactly, and no rounding of m log2(e), which grows with m, enters the sum.
  // Two columns an instruction.  Where no score is above -inf every
  // exponential is 0, not exp(-inf + inf).
  const float2 less = both(m == -INFINITY ? 0.f : -m), to2 = both(kLog2e);
  float2 sum[2] = {both(0.f), both(0.f)};
#pragma unroll
  for (int i = 0; i < kHalf; i += 2) {
    const float2 d = mul2(add2(make_float2(v[i], v[i + 1]), less), to2);
    sum[i / 2 & 1] = add2(sum[i / 2 & 1], make_float2(exp2_fast(d.x), exp2_fast(d.y)));
  }
  const float2 all = add2(sum[0], sum[1]);
  *part = failed ? make_float2(nan, nan) : make_float2(m, all.x + all.y);
}

// One box of 32 rows of 128 bytes on its way out.  Lane r holds row r as eight
// words of 16 bytes, which lie swizzled as TMA expects them, so that no two of
// a quarter warp share a bank.
__device__ __forceinline__ void out_begin(int lane) {
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncwarp();  // the box before has been read
}
__device__ __forceinline__ void out_put(uint32_t at, int lane, int i, uint32_t a, uint32_t b,
                                        uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                   at + lane * 128 + ((i ^ (lane & 7)) << 4)), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ void out_send(uint32_t at, int lane, const CUtensorMap* map, int x,
                                         int y) {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if (lane == 0) {
    asm volatile(
        "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map),
        "r"(at), "r"(x), "r"(y) : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
}

// dz of half a row, WIDTH columns at a time; columns past the piece are not
// written.  COPY: through `box` and TMA, which needs 32 rows that exist and
// whole boxes of 64 columns; else 32-byte vectors.
template <bool COPY>
__device__ __forceinline__ void epilogue_dz(const GemmArgs& g, float (&v)[kHalf], int row,
                                            int col0, int left, float scale, bool failed,
                                            uint32_t box) {
  constexpr int kWidth = COPY ? 64 : 16;
  if (row >= g.m || left <= 0) return;  // COPY: of none or all of the warp
  const int lane = threadIdx.x & 31;
  const int64_t label = load_id(g.labels, g.labels64, row, g.vocab);
  const int64_t from = label - (g.b_row0 + col0);
  const int at = from >= 0 && from < kHalf ? (int)from : -1;
  const float f = __fdiv_rn(g.dloss[row], scale);
  // two results as they go out: zeros of a padding row, whatever it holds
  const uint32_t keep = label >= 0 ? 0xFFFFFFFFu : 0u, bad = failed ? 0x7FC07FC0u : 0u;
  const float2 less = both(-g.lse[row]), to2 = both(kLog2e);  // scaled after, as for the scores
  const size_t at_row = (size_t)row * g.ld_dz + col0;
#pragma unroll
  for (int c0 = 0; c0 < kHalf; c0 += kWidth) {
    // ld_dz is a multiple of 256 and a tile begins on a boundary of 16, so
    // whole 32-byte vectors stay inside the tile and the row
    if (c0 >= left) break;
#pragma unroll
    for (int i = c0; i < c0 + kWidth; i += 2) {
      const float2 d = mul2(add2(make_float2(v[i], v[i + 1]), less), to2);
      const float2 p = make_float2(exp2_fast(d.x), exp2_fast(d.y));
      v[i] = f * (i == at ? p.x - 1.f : p.x);
      v[i + 1] = f * (i + 1 == at ? p.y - 1.f : p.y);
    }
#pragma unroll
    for (int part = 0; part < kMaxParts; ++part) {
      if (!g.dz[part]) break;
      if constexpr (COPY) out_begin(lane);
#pragma unroll
      for (int c = c0; c < c0 + kWidth; c += 16) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          w[i] = pack2(v[c + 2 * i], v[c + 2 * i + 1]);
          float lo, hi;
          widen2(w[i], lo, hi);
          v[c + 2 * i] -= lo;  // exact
          v[c + 2 * i + 1] -= hi;
          w[i] = (w[i] & keep) | bad;
        }
        if constexpr (COPY) {
          out_put(box, lane, (c - c0) / 8, w[0], w[1], w[2], w[3]);
          out_put(box, lane, (c - c0) / 8 + 1, w[4], w[5], w[6], w[7]);
        } else {
          store_words(g.dz[part] + at_row + c, w);
        }
      }
      if constexpr (COPY) out_send(box, lane, &g.c[part], col0 + c0, row - lane);
    }
  }
}

// Half a row of C.  Whole 32-byte sectors where C's rows allow it (wide).
template <typename T>
__device__ __forceinline__ void epilogue_out(const GemmArgs& g, float (&v)[kHalf], int row,
                                             int col0, int left, int split, float scale,
                                             bool failed, uint32_t box) {
  constexpr int kE = 16 / (int)sizeof(T);  // elements of 16 bytes
  const int lane = threadIdx.x & 31, first = row - lane;
  if (g.copy_out && first + 32 <= g.m) {
    // a slice's rows follow those of the slice before
    const int y = split * g.m + first;
#pragma unroll
    for (int c0 = 0; c0 < kHalf; c0 += 8 * kE) {
      if (c0 >= left) break;
      out_begin(lane);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int at = c0 + i * kE + e * (kE / 4);
          if constexpr (kE == 4)
            w[e] = __float_as_uint(v[at] * scale);
          else
            w[e] = pack2(v[at] * scale, v[at + 1] * scale);
          if (failed) w[e] = kE == 4 ? 0x7FC00000u : 0x7FC07FC0u;
        }
        out_put(box, lane, i, w[0], w[1], w[2], w[3]);
      }
      out_send(box, lane, &g.c[0], col0 + c0, y);
    }
    return;
  }
  if (row >= g.m) return;
  T* out = static_cast<T*>(g.out) + (size_t)split * g.split_stride + (size_t)row * g.ld_c + col0;
#pragma unroll
  for (int c = 0; c < kHalf; c += 2 * kE) {
    if (c >= left) break;  // left is a multiple of 8, and of 16 where wide
#pragma unroll
    for (int i = 0; i < 2 * kE; ++i) v[c + i] *= scale;
    if (g.add) {
#pragma unroll
      for (int h = 0; h < 2 * kE; h += kE) {
        if (c + h >= left) break;
        const uint4 o = *reinterpret_cast<const uint4*>(out + c + h);
        if constexpr (kE == 4) {
          v[c + h] += __uint_as_float(o.x);
          v[c + h + 1] += __uint_as_float(o.y);
          v[c + h + 2] += __uint_as_float(o.z);
          v[c + h + 3] += __uint_as_float(o.w);
        } else {
          float f[8];
          widen2(o.x, f[0], f[1]);
          widen2(o.y, f[2], f[3]);
          widen2(o.z, f[4], f[5]);
          widen2(o.w, f[6], f[7]);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[c + h + e] += f[e];
        }
      }
    }
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (kE == 4)
        w[i] = __float_as_uint(v[c + i]);
      else
        w[i] = pack2(v[c + 2 * i], v[c + 2 * i + 1]);
      if (failed) w[i] = kE == 4 ? 0x7FC00000u : 0x7FC07FC0u;
    }
    if (g.wide) {
      store_words(out + c, w);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (c + h * kE < left)
          *reinterpret_cast<uint4*>(out + c + h * kE) =
              make_uint4(w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]);
    }
  }
}

// F: the largest finite |dloss| of the tokens that count, 1 if there is none.
// The epilogue's 256 threads read it while the first tile is summed.
__device__ __forceinline__ float common_factor(const GemmArgs& g, int thread, float* red) {
  float top = 0.f;
  for (int t = thread; t < g.tokens; t += 32 * kEpiWarps) {
    const float f = fabsf(g.dloss[t]);
    if (f < INFINITY && load_id(g.labels, g.labels64, t, g.vocab) >= 0) top = fmaxf(top, f);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  if (thread % 32 == 0) red[thread / 32] = top;
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpiWarps) : "memory");
#pragma unroll
  for (int w = 0; w < kEpiWarps; ++w) top = fmaxf(top, red[w]);
  return top > 0.f ? top : 1.f;
}

// x for the product dz^T x, with zeros in the rows of padding tokens: their dz
// is 0, and 0 times what such a row may hold (a NaN, an infinity) need not be.
// `warp` of the grid's `warps` that have nothing else to do takes rows in turn,
// beside the product and without a launch: 100 x 50,021 x 1,024 with both
// gradients takes 113.8 us, 112.7 without; longer steps do not tell.
__device__ __forceinline__ void copy_counted(const GemmArgs& g, size_t warp, size_t warps,
                                             int lane) {
  for (size_t row = warp; row < (size_t)g.tokens; row += warps) {
    const bool counted = load_id(g.labels, g.labels64, row, g.vocab) >= 0;
    const uint4* from = g.x + row * g.ld_x;
    uint4* to = g.x_copy + row * g.x_words;
#pragma unroll 8
    for (size_t i = lane; i < g.x_words; i += 32)
      to[i] = counted ? from[i] : make_uint4(0u, 0u, 0u, 0u);
  }
}

// C = A B^T tile by tile, one block (CG = 1) or a pair of blocks on two SMs
// (CG = 2) per tile, every block or pair taking tiles in turn.  Warp 0 fills
// the stages by TMA, warp 1 issues the products, the last warps take the
// finished accumulator out of tensor memory while the next one is summed.
template <int CG, int PARTS, bool A_MN, bool B_MN, int EPI, bool WHOLE>
__global__ void __launch_bounds__(kGemmThreads, 1) gemm_kernel(const __grid_constant__ GemmArgs g) {
  constexpr int kBRows = kBN / CG;  // columns of C whose B this block holds
  __shared__ float factor[kEpiWarps];
  extern __shared__ uint8_t raw[];
  const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
  const uint32_t bars = base + kStageMemory;
  const uint32_t full = bars, empty = bars + 8 * kMaxStages;
  const uint32_t acc_full = empty + 8 * kMaxStages, acc_empty = acc_full + 16;
  const uint32_t tmem_slot = acc_empty + 16;
  static_assert(16 * kMaxStages + 36 <= kBarBytes, "barriers");
  // Whole boxes have sizes known here, which is worth 5% of a long pass to the
  // threads that fill the stages and issue the products.
  constexpr uint32_t kWholeA = kBM * kBK * 2, kWholeStage = PARTS * kWholeA + kBRows * kBK * 2;
  const int stages = WHOLE ? (int)(kStageMemory / kWholeStage) : g.stages;
  const uint32_t a_bytes = WHOLE ? kWholeA : g.a_bytes;
  const uint32_t stage_size = WHOLE ? kWholeStage : g.stage_size;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = CG == 2 ? cta_rank() : 0;
  const int first = blockIdx.x / CG, stride = gridDim.x / CG;
  const int tiles = g.m_tiles * g.n_tiles * g.splits;
  // A short sum of both MN major takes stages of less than kBK: rows that do
  // not exist are not copied as zeros.
  const int bk = WHOLE || !(A_MN && B_MN) ? kBK : g.bk;

  if (tid == 0) {
    for (int s = 0; s < stages; ++s) {
      bar_init(full + 8 * s, CG);
      bar_init(empty + 8 * s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      bar_init(acc_full + 8 * s, 1);
      bar_init(acc_empty + 8 * s, CG * kEpiWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 2) tmem_alloc<CG>(tmem_slot, kTmemCols);
  tmem_fence_before();
  if constexpr (CG == 2) cluster_sync();
  __syncthreads();
  tmem_fence_after();
  uint32_t tmem;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(tmem) : "r"(tmem_slot) : "memory");
  pdl_wait_then_release();
  if (warp == 0) {
    if (lane == 0) {
      // what earlier kernels wrote by ordinary stores, before copies by TMA
      asm volatile("fence.proxy.async;" ::: "memory");
      // B's box has g.bn / CG rows.  A's may have less than kBM: the rows of
      // shared memory past it hold anything, and their sums are not used.
      const uint32_t stage_bytes =
          WHOLE ? kWholeStage : (PARTS * (A_MN ? kBM : g.a_rows) +
                                 (B_MN ? kBRows : g.bn / CG)) * bk * 2;
      const uint32_t full0 = CG == 2 ? peer_addr(full, 0) : full;
      int s = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += stride) {
        const Tile tile = tile_of(g, t);
        const int m0 = (tile.m * CG + (int)rank) * kBM;
        const int n0 = tile.n * g.bn + (int)rank * kBRows;
        for (int k = tile.k0; k < tile.k1; ++k) {
          if (!(ok = bar_wait(empty + 8 * s, phase ^ 1))) break;
          const uint32_t at = base + s * stage_size;
          const uint32_t bar = full0 + 8 * s;
          bar_expect(bar, stage_bytes);
#pragma unroll
          for (int p = 0; p < PARTS; ++p) {
            const uint32_t to = at + p * a_bytes;
            if constexpr (A_MN) {
#pragma unroll
              for (int j = 0; j < kBM / 64; ++j)
                tma_load<CG>(to + j * bk * 128, &g.a[p], m0 + 64 * j, k * bk, bar);
            } else {
              tma_load<CG>(to, &g.a[p], k * kBK, m0, bar);
            }
          }
          const uint32_t to = at + PARTS * a_bytes;
          if constexpr (B_MN) {
#pragma unroll
            for (int j = 0; j < kBRows / 64; ++j)
              tma_load<CG>(to + j * bk * 128, &g.b, n0 + 64 * j, g.b_row0 + k * bk, bar);
          } else {
            tma_load<CG>(to, &g.b, k * kBK, g.b_row0 + n0, bar);
          }
          if (++s == stages) {
            s = 0;
            phase ^= 1;
          }
        }
      }
      // Until the products have read them, the copies may still be in flight:
      // the last use of every stage is waited for, so no copy outlives the block.
      for (int i = 0; i < stages; ++i) {
        bar_wait(empty + 8 * s, phase ^ 1);
        if (++s == stages) {
          s = 0;
          phase ^= 1;
        }
      }
    }
  } else if (warp == 1) {
    if (rank == 0 && lane == 0) {
      const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((A_MN ? 1u : 0u) << 15) |
                             ((B_MN ? 1u : 0u) << 16) | ((uint32_t)(g.bn / 8) << 17) |
                             ((uint32_t)(kBM * CG / 16) << 24);
      // descriptors of stage 0; those of stage s are stage_size s / 16 more
      uint64_t desc_a[PARTS];
#pragma unroll
      for (int p = 0; p < PARTS; ++p) desc_a[p] = smem_desc<A_MN>(base + p * a_bytes, bk);
      const uint64_t desc_b = smem_desc<B_MN>(base + PARTS * a_bytes, bk);
      int s = 0, buf = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += stride) {
        const Tile tile = tile_of(g, t);
        for (int k0 = tile.k0; k0 < tile.k1 && ok; k0 += g.chunk) {
          const int k1 = min(k0 + g.chunk, tile.k1);
          if (!(ok = bar_wait(acc_empty + 8 * buf, acc_phase ^ 1))) break;
          tmem_fence_after();
          const uint32_t d = tmem + buf * kBN;
          for (int k = k0; k < k1; ++k) {
            if (!(ok = bar_wait(full + 8 * s, phase))) break;
            tmem_fence_after();
            const uint32_t at = s * (stage_size >> 4);
            const uint64_t b = desc_b + at;
#pragma unroll
            for (int p = 0; p < PARTS; ++p) {
              const uint64_t a = desc_a[p] + at;
#pragma unroll
              for (int i = 0; i < kBK / 16; ++i) {
                if (!WHOLE && A_MN && B_MN && i * 16 >= bk) break;
                // 16 of the sum: 32 bytes along a row, or 16 rows of 128 bytes
                mma<CG>(d, a + i * ((A_MN ? 2048 : 32) >> 4), b + i * ((B_MN ? 2048 : 32) >> 4),
                        idesc, k > k0 || p > 0 || i > 0);
              }
            }
            mma_commit<CG>(empty + 8 * s);
            if (++s == stages) {
              s = 0;
              phase ^= 1;
            }
          }
          if (ok) mma_commit<CG>(acc_full + 8 * buf);
          if ((buf ^= 1) == 0) acc_phase ^= 1;
        }
      }
    }
  } else if (warp >= 4) {
    const int quarter = warp & 3;  // the 32 rows of tensor memory this warp may read
    const int half = (warp - 4) >> 2;
    const uint32_t box = bars + kBarBytes + (warp - 4) * kOutBytes;
    float scale = 1.f;
    if constexpr (EPI != kEpiStats) scale = common_factor(g, tid - 128, factor);
    int buf = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int t = first; t < tiles; t += stride) {
      const Tile tile = tile_of(g, t);
      float v[kHalf];
      for (int k0 = tile.k0; k0 < tile.k1; k0 += g.chunk) {
        // A wait that ran out leaves NaN in everything this block still owes.
        ok = ok && bar_wait(acc_full + 8 * buf, acc_phase);
        ok = __all_sync(0xFFFFFFFFu, ok);
        tmem_fence_after();
        const uint32_t acc = tmem + buf * kBN + half * kHalf + ((uint32_t)(quarter * 32) << 16);
        if (k0 == tile.k0) {
          tmem_load128(acc, v);
        } else {
#pragma unroll
          for (int c = 0; c < kHalf; c += 32) tmem_add32(acc + c, v + c);
        }
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) {
          const uint32_t bar = acc_empty + 8 * buf;
          bar_arrive(CG == 2 ? peer_addr(bar, 0) : bar);
        }
        if ((buf ^= 1) == 0) acc_phase ^= 1;
      }
      const int row = (tile.m * CG + (int)rank) * kBM + quarter * 32 + lane;
      const int col0 = tile.n * g.bn + half * kHalf;
      // columns of this half that are the tile's and exist
      const int left = min(g.n - tile.n * g.bn, g.bn) - half * kHalf;
      if constexpr (EPI == kEpiStats) {
        epilogue_stats(g, v, row, col0, left, 2 * tile.n + half, !ok);
      } else if constexpr (EPI == kEpiDz) {
        if (CG == 2 && row - lane + 32 <= g.m)
          epilogue_dz<CG == 2>(g, v, row, col0, left, scale, !ok, box);
        else
          epilogue_dz<false>(g, v, row, col0, left, scale, !ok, box);
      } else {
        if (g.c_type == RCC_F32)
          epilogue_out<float>(g, v, row, col0, left, tile.split, scale, !ok, box);
        else
          epilogue_out<__nv_bfloat16>(g, v, row, col0, left, tile.split, scale, !ok, box);
      }
      __syncwarp();
    }
    if (EPI != kEpiStats && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  } else if (EPI == kEpiDz && g.x_copy) {
    copy_counted(g, (size_t)blockIdx.x * 2 + (warp - 2), (size_t)gridDim.x * 2, lane);
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  tmem_fence_after();
  if (warp == 2) tmem_free<CG>(tmem, kTmemCols);
}

// ---- joins ---------------------------------------------------------------------------

constexpr int kJoinRows = 8;

// (max, sum of exp) of two sets of scores; (-inf, 0): an empty set.  A NaN in
// either sum stays.
__device__ __forceinline__ float2 join_pair(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x), from = m == -INFINITY ? 0.f : m;
  return make_float2(m, a.y * exp2_fast((a.x - from) * kLog2e) +
                            b.y * exp2_fast((b.x - from) * kLog2e));
}

// lse and loss of a row from its (max, sum) pairs: PARTS threads take them in
// turn, eight loads under way; then a warp joins a row's threads.
template <int PARTS>
__global__ void __launch_bounds__(kJoinRows* PARTS)
    join_stats_kernel(const float2* part, int parts, const float* zlab, const void* labels,
                      int labels64, size_t tokens, size_t vocab, float* loss, float* lse) {
  __shared__ float2 red[kJoinRows][PARTS + 1];
  pdl_wait_then_release();
  const int x = threadIdx.x % kJoinRows, y = threadIdx.x / kJoinRows;
  const size_t row = (size_t)blockIdx.x * kJoinRows + x;
  float2 all = make_float2(-INFINITY, 0.f);
  if (row < tokens) {
    for (int j = y; j < parts; j += 8 * PARTS) {
      float2 p[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        p[i] = j + i * PARTS < parts ? part[(size_t)(j + i * PARTS) * tokens + row]
                                     : make_float2(-INFINITY, 0.f);
      float m = all.x;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, p[i].x);
      const float from = m == -INFINITY ? 0.f : m;
      float sum = all.y * exp2_fast((all.x - from) * kLog2e);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (j + i * PARTS < parts) sum = fmaf(p[i].y, exp2_fast((p[i].x - from) * kLog2e), sum);
      all = make_float2(m, sum);
    }
  }
  red[x][y] = all;
  __syncthreads();
  const int of = threadIdx.x / 32, lane = threadIdx.x % 32;  // warp `of`: row `of`
  const size_t t = (size_t)blockIdx.x * kJoinRows + of;
  if (of >= kJoinRows || t >= tokens) return;
  float z = 0.f;
  bool hit = false;
  if (lane == 0) {
    hit = load_id(labels, labels64, t, vocab) >= 0;
    if (hit) z = zlab[t];
  }
  all = red[of][lane];
#pragma unroll
  for (int i = 32; i < PARTS; i += 32) all = join_pair(all, red[of][lane + i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float2 b = make_float2(__shfl_xor_sync(0xFFFFFFFFu, all.x, o),
                                 __shfl_xor_sync(0xFFFFFFFFu, all.y, o));
    all = lane & o ? join_pair(b, all) : join_pair(all, b);  // the same order in both lanes
  }
  if (lane == 0) {
    const float rest = logf(all.y);
    lse[t] = all.x + rest;
    loss[t] = hit ? all.x - z + rest : 0.f;  // without the rounding of lse, which is far larger
  }
}

constexpr int kSliceThreads = 256, kSliceParts = 8;

// out = the sum of the slices: `parts` sums of eight elements each, a power of
// two up to kSliceParts, which the first one adds up
template <typename T>
__global__ void __launch_bounds__(kSliceThreads)
    join_slices_kernel(const float* part, int slices, size_t n, T* out, bool wide, int parts) {
  __shared__ float red[kSliceThreads * 8 + 8 * kSliceParts];
  pdl_wait_then_release();
  const int across = kSliceThreads / parts;
  const int x = threadIdx.x % across, y = threadIdx.x / across;
  const size_t i = ((size_t)blockIdx.x * across + x) * 8;
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (i < n) {
    for (int k = y; k < slices; k += 4 * parts) {
      float v[4][8];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (k + u * parts < slices) load8(part + (size_t)(k + u * parts) * n + i, v[u]);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (k + u * parts < slices) {
#pragma unroll
          for (int e = 0; e < 8; ++e) s[e] += v[u][e];
        }
    }
  }
  if (parts > 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) red[(y * 8 + e) * (across + 1) + x] = s[e];
    __syncthreads();
    if (y != 0) return;
    for (int k = 1; k < parts; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] += red[(k * 8 + e) * (across + 1) + x];
  }
  if (i >= n) return;
  if (wide || sizeof(T) == 2) {
    store8(out + i, s);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) from_f32(s[e], out[i + e]);
  }
}

// ---- host ------------------------------------------------------------------------------

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                             const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                             const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static std::atomic<EncodeFn> fn{nullptr};
  EncodeFn f = fn.load(std::memory_order_acquire);
  if (!f) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult got;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &got) != cudaSuccess ||
        got != cudaDriverEntryPointSuccess)
      return nullptr;
    f = reinterpret_cast<EncodeFn>(p);
    fn.store(f, std::memory_order_release);
  }
  return f;
}

// A matrix of `rows` rows of `cols` elements of `size` bytes in boxes of 128
// bytes (swizzled) by `box_rows`; what lies outside reads as zero and is not
// written.
bool make_map(CUtensorMap* map, const void* p, size_t cols, size_t rows, size_t ld, int box_rows,
              size_t size = 2) {
  const EncodeFn encode = encode_fn();
  if (!encode) return false;
  const cuuint64_t dims[2] = {cols, rows}, strides[1] = {ld * size};
  const cuuint32_t box[2] = {(cuuint32_t)(128 / size), (cuuint32_t)box_rows}, step[2] = {1, 1};
  return encode(map, size == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                2, const_cast<void*>(p), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t ceil_div(size_t a, size_t b) { return (a + b - 1) / b; }

template <int CG, int PARTS, bool A_MN, bool B_MN, int EPI, bool WHOLE>
cudaError_t launch_gemm_of(GemmArgs& g, cudaStream_t stream) {
  // a block's boxes, on boundaries of 1,024 bytes
  const int a_rows = A_MN ? kBM : g.a_rows, b_rows = B_MN ? kBN / CG : g.bn / CG;
  const auto up = [](int n) { return (n + 1023) / 1024 * 1024; };
  g.a_bytes = up(a_rows * g.bk * 2);
  g.stage_size = PARTS * g.a_bytes + up(b_rows * g.bk * 2);
  g.stages = std::min(kMaxStages, kStageMemory / g.stage_size);
  auto kernel = gemm_kernel<CG, PARTS, A_MN, B_MN, EPI, WHOLE>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_shared(kernel, kGemmShared, allowed);
  if (e != cudaSuccess) return e;
  const int tiles = g.m_tiles * g.n_tiles * g.splits;
  const int units = std::min(tiles, sm_count() / CG);
  return launch_cluster(kernel, dim3(units * CG), dim3(kGemmThreads), kGemmShared, CG, stream, g);
}

// Rows of A's box: those that exist, in whole swizzle atoms.  A box that is
// mostly filled with zeros is slow: one token against 131,072 x 4,096 took
// 254 us with 128 rows, 64 tokens 169.
int box_rows(size_t rows) { return (int)std::min<size_t>(kBM, (rows + 7) / 8 * 8); }

// Of a sum of k per stage: as even as multiples of 16 allow
int stage_rows(size_t k) {
  const size_t stages = ceil_div(k, kBK);
  return (int)(ceil_div(ceil_div(k, stages), 16) * 16);
}

// Rows of C, columns, and the extent of the sum; the maps are the caller's.
template <int PARTS, bool A_MN, bool B_MN, int EPI>
cudaError_t launch_gemm(GemmArgs& g, bool pair, size_t m, size_t n, size_t k, int bn, int splits,
                        int group, cudaStream_t stream) {
  g.m = (int)m;
  g.n = (int)n;
  g.m_tiles = (int)ceil_div(m, kBM * (pair ? 2 : 1));
  g.bn = bn;
  g.a_rows = box_rows(m);
  g.n_tiles = (int)ceil_div(n, bn);
  g.bk = A_MN && B_MN ? stage_rows(k) : kBK;
  g.k_blocks = (int)ceil_div(k, g.bk);
  g.splits = splits;
  g.group = group;
  const int mmas = EPI == kEpiOut ? kOutMmas : pair ? kScoreMmas : kScoreMmasFew;
  g.chunk = EPI == kEpiOut && g.c_type == RCC_BF16 ? g.k_blocks : mmas / (PARTS * (kBK / 16));
  // whole boxes: of a pair, unless the sum is short; what one block does alone
  // is bound by memory
  if (!pair) return launch_gemm_of<1, PARTS, A_MN, B_MN, EPI, false>(g, stream);
  if constexpr (A_MN && B_MN)
    if (g.bk < kBK) return launch_gemm_of<2, PARTS, A_MN, B_MN, EPI, false>(g, stream);
  return launch_gemm_of<2, PARTS, A_MN, B_MN, EPI, true>(g, stream);
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Two SMs share a tile of 256 rows unless 128 rows are all there are.
bool paired(size_t rows) { return rows > (size_t)kBM; }

// Columns of a tile of scores.  With few tokens a pass is bound by reading W,
// so its rows are shared out evenly: the same number of tiles for every SM.
int score_width(size_t tokens, size_t vocab) {
  if (paired(tokens)) return kBN;
  const size_t sms = sm_count(), turns = ceil_div(vocab, sms * kBN);
  return (int)(ceil_div(ceil_div(vocab, sms * turns), 16) * 16);
}

// Tiles of rows that share a run over the columns: what a turn of all SMs reads
// of A and B stays in L2.  Scores of 8,192 x 131,072 x 4,096 under the power
// limit: 16 tiles 4.86 to 4.92 ms, 12 4.98, 20 5.04, 32 5.21 to 5.24; the
// gradients' products do not tell 4, 8 and 16 apart.
constexpr int kScoreGroup = 16, kGradGroup = 8;

// Rows of whole 32-byte sectors
bool wide_rows(const void* c, size_t dim, size_t size) {
  return (reinterpret_cast<uintptr_t>(c) & 31u) == 0 && dim * size % 32 == 0;
}

// The backward pass's pieces of the vocabulary and what it keeps of each.
struct Pieces {
  size_t width;      // vocabulary entries of a piece, a multiple of kBN
  size_t count;
  int parts;         // bf16 numbers that make one dz
  int splits;        // of the sum of dx
  size_t dz_bytes;   // of one part
  size_t dx_bytes;   // of the fp32 slices of dx, 0: summed in dx itself
  size_t x_bytes;    // of x without its padding rows
};
constexpr size_t kDzBytes = (size_t)512 << 20;

Pieces pieces_of(size_t tokens, size_t vocab, size_t dim, int grad_type) {
  Pieces p;
  p.parts = grad_type == RCC_F32 ? kMaxParts : 1;
  const size_t most = std::max<size_t>(kBN, kDzBytes / (tokens * 2 * p.parts) / kBN * kBN);
  p.count = ceil_div(vocab, most);
  p.width = ceil_div(ceil_div(vocab, p.count), kBN) * kBN;
  p.count = ceil_div(vocab, p.width);
  p.dz_bytes = up256(tokens * p.width * 2);
  const int cg = paired(tokens) ? 2 : 1;
  const size_t tiles = ceil_div(tokens, kBM * cg) * ceil_div(dim, kBN);
  const size_t units = sm_count() / cg, k_blocks = p.width / kBK;
  // Pieces of the sum of dx, each added up by itself: the fewest turns of all
  // SMs, at 0.27 us for a stage's products, against writing and reading a
  // slice more, at 6 TB/s.
  p.splits = 1;
  double best = 0;
  for (size_t s = 1; s <= 64 && s <= std::max<size_t>(1, k_blocks / 8); ++s) {
    const double turns = (double)ceil_div(tiles * s, units);
    const double us = turns * (double)ceil_div(k_blocks, s) * 0.27 * p.parts +
                      (s > 1 ? (double)(s * tokens * dim) * 8 / 6e6 + 4 : 0);
    if (s == 1 || us < best) {
      best = us;
      p.splits = (int)s;
    }
  }
  const bool direct = p.splits == 1 && (p.count == 1 || grad_type == RCC_F32);
  p.dx_bytes = direct ? 0 : up256(p.splits * tokens * dim * 4);
  p.x_bytes = up256(tokens * dim * 2);
  return p;
}

}  // namespace

size_t linear_ce_workspace(size_t tokens, size_t vocab, size_t dim, bool backward, int grad_type) {
  if (!backward)
    return up256(2 * ceil_div(vocab, score_width(tokens, vocab)) * tokens * sizeof(float2)) +
           up256(tokens * 4);
  const Pieces p = pieces_of(tokens, vocab, dim, grad_type);
  return p.parts * p.dz_bytes + p.dx_bytes + p.x_bytes;
}

cudaError_t launch_linear_ce_forward(const CeArgs& a, cudaStream_t stream, uint64_t* launches) {
  const bool pair = paired(a.tokens);
  const int bn = score_width(a.tokens, a.vocab);
  const int parts = 2 * (int)ceil_div(a.vocab, bn);  // one for each half of a tile's columns
  GemmArgs g = {};
  g.part = static_cast<float2*>(a.workspace);
  g.zlab = reinterpret_cast<float*>(static_cast<char*>(a.workspace) +
                                    up256((size_t)parts * a.tokens * sizeof(float2)));
  g.labels = a.labels;
  g.labels64 = a.labels64;
  g.vocab = (int)a.vocab;
  if (!make_map(&g.a[0], a.x, a.dim, a.tokens, a.ld_x, box_rows(a.tokens)) ||
      !make_map(&g.b, a.w, a.dim, a.vocab, a.ld_w, bn / (pair ? 2 : 1)))
    return cudaErrorInvalidValue;
  cudaError_t e = launch_gemm<1, false, false, kEpiStats>(g, pair, a.tokens, a.vocab, a.dim, bn, 1,
                                                          kScoreGroup, stream);
  if (e != cudaSuccess) return e;
  // few rows: more threads to each
  const auto join = [&](auto threads) {
    constexpr int kParts = decltype(threads)::value;
    return launch_kernel(join_stats_kernel<kParts>, dim3((unsigned)ceil_div(a.tokens, kJoinRows)),
                         dim3(kJoinRows * kParts), 0, stream, (const float2*)g.part, parts,
                         (const float*)g.zlab, a.labels, a.labels64, a.tokens, a.vocab, a.loss,
                         a.lse);
  };
  e = a.tokens <= 1024 ? join(std::integral_constant<int, 128>())
                       : join(std::integral_constant<int, 32>());
  if (e == cudaSuccess) *launches = 2;
  return e;
}

namespace {
// what all products of the backward pass need for the common factor
GemmArgs grad_args(const CeArgs& a) {
  GemmArgs g = {};
  g.labels = a.labels;
  g.labels64 = a.labels64;
  g.vocab = (int)a.vocab;
  g.tokens = (int)a.tokens;
  g.dloss = a.dloss;
  return g;
}
}  // namespace

cudaError_t launch_linear_ce_backward(const CeArgs& a, cudaStream_t stream, uint64_t* launches) {
  const Pieces p = pieces_of(a.tokens, a.vocab, a.dim, a.grad_type);
  char* ws = static_cast<char*>(a.workspace);
  __nv_bfloat16* dz[kMaxParts] = {};
  for (int k = 0; k < p.parts; ++k)
    dz[k] = reinterpret_cast<__nv_bfloat16*>(ws + k * p.dz_bytes);
  float* slices = p.dx_bytes ? reinterpret_cast<float*>(ws + p.parts * p.dz_bytes) : nullptr;
  uint4* x_copy = reinterpret_cast<uint4*>(ws + p.parts * p.dz_bytes + p.dx_bytes);
  const size_t grad_size = a.grad_type == RCC_F32 ? 4 : 2;
  const bool pair = paired(a.tokens);
  cudaError_t e;
  for (size_t i = 0; i < p.count; ++i) {
    const size_t v0 = i * p.width, width = std::min(p.width, a.vocab - v0);
    {  // dz of the piece
      GemmArgs g = grad_args(a);
      g.b_row0 = (int)v0;
      g.lse = a.lse;
      for (int k = 0; k < p.parts; ++k) g.dz[k] = dz[k];
      for (int k = 0; k < p.parts && pair; ++k)  // tiles of whole boxes
        if (!make_map(&g.c[k], dz[k], width, a.tokens, p.width, 32)) return cudaErrorInvalidValue;
      g.ld_dz = p.width;
      if (a.dw && i == 0) {  // rows are whole words of 16 bytes
        g.x = static_cast<const uint4*>(a.x);
        g.x_copy = x_copy;
        g.ld_x = a.ld_x / 8;
        g.x_words = a.dim / 8;
      }
      const int bn = score_width(a.tokens, width);
      if (!make_map(&g.a[0], a.x, a.dim, a.tokens, a.ld_x, box_rows(a.tokens)) ||
          !make_map(&g.b, a.w, a.dim, a.vocab, a.ld_w, bn / (pair ? 2 : 1)))
        return cudaErrorInvalidValue;
      e = launch_gemm<1, false, false, kEpiDz>(g, pair, a.tokens, width, a.dim, bn, 1, kScoreGroup,
                                               stream);
      if (e != cudaSuccess) return e;
      ++*launches;
    }
    if (a.dx) {  // dx (+)= dz W
      GemmArgs g = grad_args(a);
      g.b_row0 = (int)v0;
      g.out = slices ? slices : a.dx;
      g.c_type = slices ? RCC_F32 : a.grad_type;
      g.ld_c = a.dim;
      g.split_stride = a.tokens * a.dim;
      g.add = i > 0;
      g.wide = wide_rows(g.out, a.dim, slices ? 4 : grad_size);
      g.copy_out = !g.add;
      if (g.copy_out && !make_map(&g.c[0], g.out, a.dim, a.tokens * (slices ? p.splits : 1), a.dim,
                                  32, slices ? 4 : grad_size))
        return cudaErrorInvalidValue;
      for (int k = 0; k < p.parts; ++k)
        if (!make_map(&g.a[k], dz[k], width, a.tokens, p.width, box_rows(a.tokens))) return cudaErrorInvalidValue;
      if (!make_map(&g.b, a.w, a.dim, a.vocab, a.ld_w, kBK)) return cudaErrorInvalidValue;
      const int splits = (int)std::min<size_t>(p.splits, ceil_div(width, kBK));
      e = p.parts > 1 ? launch_gemm<kMaxParts, false, true, kEpiOut>(g, pair, a.tokens, a.dim, width,
                                                              kBN, splits, kGradGroup, stream)
                       : launch_gemm<1, false, true, kEpiOut>(g, pair, a.tokens, a.dim, width,
                                                              kBN, splits, kGradGroup, stream);
      if (e != cudaSuccess) return e;
      ++*launches;
    }
    if (a.dw) {  // the piece's rows of dW (+)= dz^T x
      GemmArgs g = grad_args(a);
      g.out = static_cast<char*>(a.dw) + v0 * a.dim * grad_size;
      g.c_type = a.grad_type;
      g.ld_c = a.dim;
      g.add = a.accumulate;
      g.wide = wide_rows(g.out, a.dim, grad_size);
      g.copy_out = !g.add;
      if (g.copy_out && !make_map(&g.c[0], g.out, a.dim, width, a.dim, 32, grad_size))
        return cudaErrorInvalidValue;
      for (int k = 0; k < p.parts; ++k)
        if (!make_map(&g.a[k], dz[k], width, a.tokens, p.width, stage_rows(a.tokens))) return cudaErrorInvalidValue;
      if (!make_map(&g.b, x_copy, a.dim, a.tokens, a.dim, stage_rows(a.tokens))) return cudaErrorInvalidValue;
      const bool wide = paired(width);
      e = p.parts > 1 ? launch_gemm<kMaxParts, true, true, kEpiOut>(g, wide, width, a.dim, a.tokens, kBN, 1,
                                                             kGradGroup, stream)
                       : launch_gemm<1, true, true, kEpiOut>(g, wide, width, a.dim, a.tokens, kBN, 1,
                                                             kGradGroup, stream);
      if (e != cudaSuccess) return e;
      ++*launches;
    }
  }
  if (a.dx && slices) {
    const size_t n = a.tokens * a.dim;
    int parts = 1;
    while (parts < kSliceParts && 2 * parts <= p.splits) parts *= 2;
    const dim3 grid((unsigned)ceil_div(n, kSliceThreads / parts * 8)), block(kSliceThreads);
    e = a.grad_type == RCC_F32
            ? launch_kernel(join_slices_kernel<float>, grid, block, 0, stream,
                            (const float*)slices, p.splits, n, static_cast<float*>(a.dx),
                            (reinterpret_cast<uintptr_t>(a.dx) & 31u) == 0, parts)
            : launch_kernel(join_slices_kernel<__nv_bfloat16>, grid, block, 0, stream,
                            (const float*)slices, p.splits, n, static_cast<__nv_bfloat16*>(a.dx),
                            true, parts);
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  return cudaSuccess;
}

}  // namespace lm
}  // namespace rcc
