// rmsnorm.cu -- RMS norm that keeps its input in 8 bits, and its backward pass
// from the 8 bits.
//
//   forward   r = 1/sqrt(mean(x^2) + eps);  y = x r w
//             kept: q = rint(x (127 (1/a))), s = a (1/127) with a = max|x| of 128
//             columns, every operation rounded to fp32
//   backward  x' = q s;  r = 1/sqrt(mean(x'^2) + eps);  n = x' r
//             dx = r (dy w - n mean(dy w n));  dw = sum over tokens of dy n
//
// The backward pass is the exact gradient of the norm at the kept input x', so
// nothing but q and s (1.03 bytes an element) has to survive from the forward
// pass.
#include <algorithm>

#include "lm_common.cuh"
#include "lm_internal.h"

namespace rcc {
namespace lm {
namespace {

// A group whose largest magnitude is below this is kept as zeros (1/a stays
// finite for the others).
constexpr float kTiny = 7.52316385e-37f;  // 2^-120

// Sums over the G threads (a power of two) that share a row; G > 32 goes
// through `red`, which the caller alternates from row to row, so that one
// barrier a row is enough.  Every thread of the block calls it.
template <int G, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*red)[N], int tid) {
#pragma unroll
  for (int o = (G < 32 ? G : 32) / 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
  if constexpr (G > 32) {
    if ((tid & 31) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) red[tid >> 5][i] = v[i];
    __syncthreads();
    const int w0 = (tid / G) * (G / 32);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.f;
#pragma unroll
    for (int w = 0; w < G / 32; ++w)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += red[w0 + w][i];
  }
}

__device__ __forceinline__ float max_nan(float a, float b) {  // a NaN wins
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// 1.5 2^23: adding it leaves a value below 2^22 rounded to a whole number,
// ties to even, in the low bits of the sum.
constexpr float kWhole = 12582912.f;

// rint(x inv) of two values, in the low bytes.  Two roundings, the product's
// and the whole number's: never one fused operation.
__device__ __forceinline__ uint32_t quantize2(float2 a, float inv) {
  a = mul2(a, both(inv));
  return __byte_perm(__float_as_uint(__fadd_rn(a.x, kWhole)),
                     __float_as_uint(__fadd_rn(a.y, kWhole)), 0x0040);
}
// and back: four signed bytes as floats (2^23 + 128 + q has q + 128 in its low bits)
__device__ __forceinline__ void widen4(uint32_t q, float2& a, float2& b) {
  q ^= 0x80808080u;
  constexpr uint32_t k = 0x4B000000u;
  constexpr float c = -8388736.f;
  a = add2(make_float2(__uint_as_float(__byte_perm(q, k, 0x7540)),
                       __uint_as_float(__byte_perm(q, k, 0x7541))), both(c));
  b = add2(make_float2(__uint_as_float(__byte_perm(q, k, 0x7542)),
                       __uint_as_float(__byte_perm(q, k, 0x7543))), both(c));
}

// threads of a block whose rows take G threads each
template <int G>
constexpr int kBlock = G > 256 ? G : 256;

// A thread holds parts of 16 bytes, kE elements, as they lie in memory or as
// kE / 2 fp32 pairs; a part's columns are p G kE after those of part 0.
//   VEC (aligned rows of whole parts): kE neighbouring columns from t kE of
//   thread t of the G that share a row, so that 128 / kE threads hold a group
//   of 128 columns.
//   else (any alignment and width): every 32nd column of the warp's 32 kE, so
//   that a warp's single elements lie side by side; four of them on all lanes
//   are a group, so a part has kE / 4 groups.
template <typename T, bool VEC>
struct Part {
  static constexpr int kE = 16 / (int)sizeof(T);
  static constexpr int kPairs = kE / 2;
  static constexpr int kBytes8 = kE / 4;  // words of the 8-bit form
  static constexpr int kScales = VEC ? 1 : kE / 4;
  static constexpr int kLanes = VEC ? (int)kKeepGroup / kE : 32;  // that share a group
  static constexpr int kStep = VEC ? 1 : 32;  // columns from an element to the next
  static __device__ __forceinline__ int first_column(int t) {
    return VEC ? t * kE : t / 32 * 32 * kE + t % 32;
  }
};
__device__ __forceinline__ void widen(const uint4& r, float2 (&v)[4], __nv_bfloat16) {
  widen2(r.x, v[0].x, v[0].y);
  widen2(r.y, v[1].x, v[1].y);
  widen2(r.z, v[2].x, v[2].y);
  widen2(r.w, v[3].x, v[3].y);
}
__device__ __forceinline__ void widen(const uint4& r, float2 (&v)[2], float) {
  v[0] = make_float2(__uint_as_float(r.x), __uint_as_float(r.y));
  v[1] = make_float2(__uint_as_float(r.z), __uint_as_float(r.w));
}
__device__ __forceinline__ uint4 narrow(const float2 (&v)[4], __nv_bfloat16) {
  return make_uint4(pack2(v[0].x, v[0].y), pack2(v[1].x, v[1].y), pack2(v[2].x, v[2].y),
                    pack2(v[3].x, v[3].y));
}
__device__ __forceinline__ uint4 narrow(const float2 (&v)[2], float) {
  return make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x),
                    __float_as_uint(v[1].y));
}
// A part at p; past `left` columns its elements are zeros and not written
template <bool VEC, typename T>
__device__ __forceinline__ uint4 load_part(const T* p, int left) {
  if constexpr (VEC) {
    return *reinterpret_cast<const uint4*>(p);
  } else {
    float2 v[Part<T, VEC>::kPairs];
#pragma unroll
    for (int e = 0; e < Part<T, VEC>::kPairs; ++e) {
      v[e].x = 64 * e < left ? to_f32(p[64 * e]) : 0.f;
      v[e].y = 64 * e + 32 < left ? to_f32(p[64 * e + 32]) : 0.f;
    }
    return narrow(v, T());
  }
}
template <bool VEC, typename T, int PAIRS>
__device__ __forceinline__ void store_part(T* p, int left, const float2 (&v)[PAIRS]) {
  if constexpr (VEC) {
    *reinterpret_cast<uint4*>(p) = narrow(v, T());
  } else {
#pragma unroll
    for (int e = 0; e < PAIRS; ++e) {
      if (64 * e < left) from_f32(v[e].x, p[64 * e]);
      if (64 * e + 32 < left) from_f32(v[e].y, p[64 * e + 32]);
    }
  }
}
// The weight of a part's columns
template <bool VEC, int PAIRS>
__device__ __forceinline__ void load_weight(const float* w, int left, float2 (&v)[PAIRS]) {
#pragma unroll
  for (int e = 0; e < PAIRS; e += 2) {  // four columns at a time: a part of fp32
    const int at = VEC ? 2 * e : 64 * e;
    const uint4 f = load_part<VEC>(w + at, left - at);
    v[e] = make_float2(__uint_as_float(f.x), __uint_as_float(f.y));
    v[e + 1] = make_float2(__uint_as_float(f.z), __uint_as_float(f.w));
  }
}
// The bytes of a part: kBytes8 words, whatever the layout
template <bool VEC, int WORDS>
__device__ __forceinline__ void load_bytes(const int8_t* p, int left, uint32_t (&q)[WORDS]) {
  if constexpr (!VEC) {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
      q[i] = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if ((4 * i + e) * 32 < left)
          q[i] |= (uint32_t)(uint8_t)p[(4 * i + e) * 32] << (8 * e);
    }
  } else if constexpr (WORDS == 2) {
    const uint2 two = *reinterpret_cast<const uint2*>(p);
    q[0] = two.x;
    q[1] = two.y;
  } else {
    q[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}
template <bool VEC, int WORDS>
__device__ __forceinline__ void store_bytes(int8_t* p, int left, const uint32_t (&q)[WORDS]) {
  if constexpr (!VEC) {
#pragma unroll
    for (int i = 0; i < WORDS; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if ((4 * i + e) * 32 < left) p[(4 * i + e) * 32] = (int8_t)(q[i] >> (8 * e));
  } else if constexpr (WORDS == 2) {
    *reinterpret_cast<uint2*>(p) = make_uint2(q[0], q[1]);
  } else {
    *reinterpret_cast<uint32_t*>(p) = q[0];
  }
}

// `n` (4, 8 or 16) bytes of global memory into shared memory, asynchronously
template <int N>
__device__ __forceinline__ void copy_async(void* to, const void* from) {
  const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at), "l"(from), "n"(N)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {  // all but the newest N groups
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Threads of all blocks of one SM (those waiting to start included) and rows
// held in shared memory.  Measured at 16,384 rows of 4,096 bf16 (fp32) columns,
// where 6.78 TB/s would take 50 (89) us each way:
//   forward   2,048 threads, 2 rows held              54.2 (98.9) us
//             1,024 threads, 2 rows held              58.3 (105)
//             1,024 threads, 3 rows held              62.6 (106)
//             4,096 threads, nothing copied ahead     63.2 (92.4)
//             1,024 threads, nothing copied ahead     63.5 (93.4)
//   backward  512 threads, 3 rows held                61.4 (97.7)
//             512 threads, 4 rows held                62.2 (96.0)
//             768 threads, 3 rows held                62.3 (96.9)
//             768 threads, 2 rows held                62.1 (99.7)
//             1,024 threads, 2 rows held              73.1 (99.6)
// and of 2,048 bf16 columns backward 35.2 with 512 threads, 36.4 with 768.  Of
// 4,095 columns, not copied ahead: 512 threads 137 (198), 768 108 (154), 1,024
// 111 (152).
// So the forward pass copies rows of 2-byte types ahead; an fp32 row is as many
// loads in flight by itself.
constexpr int kForeThreads = 2048, kForeStages = 2, kForeDirect = 4096;
constexpr int kBackThreads = 512, kBackStages = 3, kBackDirect = 768;
constexpr int kSharedMost = 220 * 1024;   // of all blocks of one SM

// blocks of `threads` that one SM takes, of `shared` bytes each, for `all` threads
constexpr int blocks_per_sm(int all, int threads, int shared) {
  return shared && kSharedMost / shared < all / threads ? (kSharedMost / shared > 0 ? kSharedMost / shared : 1)
                                                        : (all / threads > 0 ? all / threads : 1);
}

// Rows copied ahead into shared memory (aligned rows, VEC).  A thread writes
// and reads its own parts alone, so the copies need no barrier; a group's scale
// is one lane's copy, for the lanes of its warp.
template <typename T, int G, int NV, bool VEC>
struct NormFore {
  static constexpr int kThreads = kBlock<G>;
  static constexpr int kParts = NV * 8 / Part<T, VEC>::kE;
  static constexpr int kStage = kThreads * kParts * 16;
  static constexpr int kFit = kSharedMost / kStage;
  static constexpr int kStages = VEC && sizeof(T) == 2 && kFit >= kForeStages ? kForeStages : 0;
  static constexpr int kShared = kStages * kStage;
  static constexpr int kPerSm = blocks_per_sm(kStages ? kForeThreads : kForeDirect, kThreads, kShared);
};

// One row for each group of G threads at a time; a thread keeps its part of
// the weight over all its rows.
template <typename T, int G, int NV, bool VEC>
__global__ void __launch_bounds__(kBlock<G>) norm_forward_kernel(const NormArgs a) {
  using F = NormFore<T, G, NV, VEC>;
  using P = Part<T, VEC>;
  constexpr int kThreads = F::kThreads, kRows = kThreads / G, kStages = F::kStages;
  constexpr int kParts = F::kParts;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float red[2][kThreads / 32][1];
  pdl_wait_then_release();
  const int tid = threadIdx.x, t = tid % G;
  constexpr int kSpan = G * P::kE;  // columns from a thread's part to its next
  const int col = P::first_column(t);
  const int dim = (int)a.dim, left = dim - col;
  const int groups = (dim + (int)kKeepGroup - 1) / (int)kKeepGroup;
  const int kept_left = groups * (int)kKeepGroup - col;
  const float inv_dim = 1.f / (float)dim;
  // this thread's first part of its row, here and in the row that is copied ahead
  size_t row = (size_t)blockIdx.x * kRows + tid / G;
  const size_t step = (size_t)gridDim.x * kRows;
  const T* ahead = static_cast<const T*>(a.x) + row * a.ld_x + col;
  T* y = static_cast<T*>(a.y) + row * a.ld_y + col;
  int8_t* kept = a.kept + row * groups * kKeepGroup + col;
  float* scales = a.scales + row * groups + col / (int)kKeepGroup;
  size_t ahead_row = row;
  auto x_at = [&](int s, int p) {
    return reinterpret_cast<uint4*>(smem + s * F::kStage) + p * kThreads + tid;
  };
  auto copy_row = [&](int s) {
    if (ahead_row < a.tokens) {
#pragma unroll
      for (int p = 0; p < kParts; ++p)
        if (left > p * kSpan) copy_async<16>(x_at(s, p), ahead + p * kSpan);
    }
    copies_commit();  // one group a row, also when there is none
    ahead += step * a.ld_x;
    ahead_row += step;
  };
  for (int s = 0; s < kStages - 1; ++s) copy_row(s);
  float2 w[kParts][P::kPairs];
#pragma unroll
  for (int p = 0; p < kParts; ++p)
    if (left > p * kSpan)
      load_weight<VEC>(a.weight + col + p * kSpan, left - p * kSpan, w[p]);
  int stage = 0, flip = 0;
  for (size_t first = (size_t)blockIdx.x * kRows; first < a.tokens; first += step, row += step) {
    const bool live = kRows == 1 || row < a.tokens;
    if constexpr (kStages > 0) {
      copy_row(stage == 0 ? kStages - 1 : stage - 1);
      copies_wait<kStages - 1>();
    }
    float2 v[kParts][P::kPairs];
    float2 sq = both(0.f);
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      uint4 raw = make_uint4(0u, 0u, 0u, 0u);
      if (live && left > p * kSpan) {
        if constexpr (kStages > 0)
          raw = *x_at(stage, p);
        else
          raw = load_part<VEC>(ahead + p * kSpan, left - p * kSpan);
      }
      widen(raw, v[p], T());
#pragma unroll
      for (int e = 0; e < P::kPairs; ++e) sq = fma2(v[p][e], v[p][e], sq);
    }
    float sum[1] = {sq.x + sq.y};
    row_sum<G>(sum, red[flip], tid);
    const float r = rsqrtf(fmaf(sum[0], inv_dim, a.eps));
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      if (a.kept) {
        constexpr int kOf = P::kPairs / P::kScales;  // pairs of one group
        float amax[P::kScales];
#pragma unroll
        for (int i = 0; i < P::kScales; ++i) {
          amax[i] = 0.f;
#pragma unroll
          for (int e = i * kOf; e < (i + 1) * kOf; ++e)
            amax[i] = max_nan(max_nan(amax[i], fabsf(v[p][e].x)), fabsf(v[p][e].y));
#pragma unroll
          for (int o = P::kLanes / 2; o > 0; o >>= 1)
            amax[i] = max_nan(amax[i], __shfl_xor_sync(0xFFFFFFFFu, amax[i], o));
        }
        if (live && kept_left > p * kSpan) {
          uint32_t q[P::kBytes8];
#pragma unroll
          for (int i = 0; i < P::kScales; ++i) {
            // a NaN or infinity: zeros and a NaN scale; next to nothing: zeros
            const bool fine = amax[i] >= kTiny && amax[i] < INFINITY;
            const float inv = fine ? 127.f * __frcp_rn(amax[i]) : 0.f;
            constexpr int kWords = P::kBytes8 / P::kScales;
#pragma unroll
            for (int k = i * kWords; k < (i + 1) * kWords; ++k) {
              q[k] = __byte_perm(quantize2(v[p][2 * k], inv), quantize2(v[p][2 * k + 1], inv),
                                 0x5410);
              if (!fine) q[k] = 0u;
            }
            if (t % P::kLanes == 0 && kept_left > p * kSpan + i * (int)kKeepGroup)
              scales[p * (kSpan / (int)kKeepGroup) + i] =
                  fine ? amax[i] * (1.f / 127.f)
                       : amax[i] < kTiny ? 0.f : __uint_as_float(0x7FC00000u);
          }
          store_bytes<VEC>(kept + p * kSpan, kept_left - p * kSpan, q);
        }
      }
      if (live && left > p * kSpan) {
#pragma unroll
        for (int e = 0; e < P::kPairs; ++e) v[p][e] = mul2(mul2(v[p][e], both(r)), w[p][e]);
        store_part<VEC>(y + p * kSpan, left - p * kSpan, v[p]);
      }
    }
    y += step * a.ld_y;
    kept += step * groups * kKeepGroup;
    scales += step * groups;
    if constexpr (kStages == 0) ahead += step * a.ld_x;
    stage = stage + 1 >= kStages ? 0 : stage + 1;
    flip ^= 1;
  }
}

// ---- backward ------------------------------------------------------------------

// What a block of the backward pass holds in shared memory: the weight, and
// rows of dy, the 8-bit input and its scales copied ahead.  Where not even two
// rows fit (fp32 rows of more than 16,384) nothing is copied ahead.
template <typename T, int G, int NV, bool VEC>
struct NormBack {
  static constexpr int kThreads = kBlock<G>;
  static constexpr int kParts = NV * 8 / Part<T, VEC>::kE;
  static constexpr int kScaled = kThreads / Part<T, VEC>::kLanes;  // groups of one part
  static constexpr int kStage = kThreads * kParts * (16 + Part<T, VEC>::kE) + kParts * kScaled * 4;
  static constexpr bool kHoldWeight = kThreads * NV * 32 + 2 * kStage <= kSharedMost;
  static constexpr int kWeight = kHoldWeight ? kThreads * NV * 32 : 0;
  static constexpr int kFit = (kSharedMost - kWeight) / kStage;
  static constexpr int kStages = VEC && kFit >= 2 ? (kFit < kBackStages ? kFit : kBackStages) : 0;
  static constexpr int kShared = kWeight + kStages * kStage;
  static constexpr int kPerSm = blocks_per_sm(kStages ? kBackThreads : kBackDirect, kThreads, kShared);
};

// Rows are dealt to the blocks in turn; a thread keeps the weight gradient of
// its columns in registers over all of its rows, and each block writes one
// row of partial sums, which norm_dweight_kernel adds in a fixed order.
// Bandwidth bound: rows are copied ahead into shared memory (aligned rows,
// VEC) while the current one is reduced.
template <typename T, int G, int NV, bool VEC>
__global__ void __launch_bounds__(kBlock<G>, NormBack<T, G, NV, VEC>::kPerSm)
    norm_backward_kernel(const NormGradArgs a) {
  using B = NormBack<T, G, NV, VEC>;
  using P = Part<T, VEC>;
  constexpr int kThreads = B::kThreads, kRows = kThreads / G, kStages = B::kStages;
  constexpr int kParts = B::kParts;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float red[2][kThreads / 32][2];
  pdl_wait_then_release();
  const int tid = threadIdx.x, t = tid % G;
  constexpr int kSpan = G * P::kE;  // columns from a thread's part to its next
  const int col = P::first_column(t);
  const int dim = (int)a.dim, left = dim - col;
  const int groups = (dim + (int)kKeepGroup - 1) / (int)kKeepGroup;
  const float inv_dim = 1.f / (float)dim;
  size_t row = (size_t)blockIdx.x * kRows + tid / G;
  const size_t step = (size_t)gridDim.x * kRows;
  // this thread's first part of the row that is copied ahead, and of its output
  const T* dy = static_cast<const T*>(a.dy) + row * a.ld_dy + col;
  const int8_t* kept = a.kept + row * groups * kKeepGroup + col;
  const float* scales = a.scales + row * groups + col / (int)kKeepGroup;
  T* dx_out = static_cast<T*>(a.dx) + row * a.ld_dx + col;
  size_t ahead_row = row;
  // what neighbouring threads hold of one kind lies side by side
  auto weight_at = [&](int p, int h) {
    return reinterpret_cast<float4*>(smem) + (p * P::kBytes8 + h) * kThreads + tid;
  };
  auto dy_at = [&](int s, int p) {
    return reinterpret_cast<uint4*>(smem + B::kWeight + s * B::kStage) + p * kThreads + tid;
  };
  auto q_at = [&](int s, int p) {
    return reinterpret_cast<uint32_t*>(smem + B::kWeight + s * B::kStage +
                                       kThreads * kParts * 16) +
           (p * kThreads + tid) * P::kBytes8;
  };
  auto scale_at = [&](int s, int p) {
    return reinterpret_cast<float*>(smem + B::kWeight + s * B::kStage +
                                    kThreads * kParts * (16 + P::kE)) +
           p * B::kScaled + tid / P::kLanes;
  };
  auto weight = [&](int p, float2 (&w)[P::kPairs]) {
    if constexpr (B::kHoldWeight) {
#pragma unroll
      for (int h = 0; h < P::kBytes8; ++h) {
        const float4 f = *weight_at(p, h);
        w[2 * h] = make_float2(f.x, f.y);
        w[2 * h + 1] = make_float2(f.z, f.w);
      }
    } else {
      load_weight<VEC>(a.weight + col + p * kSpan, left - p * kSpan, w);
    }
  };
  auto next_row = [&]() {
    dy += step * a.ld_dy;
    kept += step * groups * kKeepGroup;
    scales += step * groups;
    ahead_row += step;
  };
  auto copy_row = [&](int s) {
    if (ahead_row < a.tokens) {
#pragma unroll
      for (int p = 0; p < kParts; ++p) {
        if (left > p * kSpan) {
          copy_async<16>(dy_at(s, p), dy + p * kSpan);
          copy_async<P::kE>(q_at(s, p), kept + p * kSpan);
          if (t % P::kLanes == 0)
            copy_async<4>(scale_at(s, p), scales + p * (kSpan / (int)kKeepGroup));
        }
      }
    }
    copies_commit();  // one group a row, also when there is none
    next_row();
  };

  for (int s = 0; s < kStages - 1; ++s) copy_row(s);
  float2 acc[kParts][P::kPairs];
#pragma unroll
  for (int p = 0; p < kParts; ++p) {
    if (B::kHoldWeight && left > p * kSpan) {
      float2 w[P::kPairs];
      load_weight<VEC>(a.weight + col + p * kSpan, left - p * kSpan, w);
#pragma unroll
      for (int h = 0; h < P::kBytes8; ++h)
        *weight_at(p, h) = make_float4(w[2 * h].x, w[2 * h].y, w[2 * h + 1].x, w[2 * h + 1].y);
    }
#pragma unroll
    for (int e = 0; e < P::kPairs; ++e) acc[p][e] = both(0.f);
  }
  int stage = 0, flip = 0;
  for (size_t first = (size_t)blockIdx.x * kRows; first < a.tokens; first += step, row += step) {
    const bool live = kRows == 1 || row < a.tokens;
    if constexpr (kStages > 0) {
      copy_row(stage == 0 ? kStages - 1 : stage - 1);
      copies_wait<kStages - 1>();
      __syncwarp();  // a group's scale is one lane's copy
    }
    // kept over the reduction: dy w, and dy and the bytes as they came
    uint4 raw[kParts];
    uint32_t q[kParts][P::kBytes8];
    float2 dw[kParts][P::kPairs];
    float scale[kParts][P::kScales];
    float2 xx = both(0.f), dx = both(0.f);  // sums of x'^2, of dy w x'
    constexpr int kOf = P::kPairs / P::kScales;  // pairs of one scale
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      if (live && left > p * kSpan) {
        if constexpr (kStages > 0) {
          raw[p] = *dy_at(stage, p);
          load_bytes<VEC>(reinterpret_cast<const int8_t*>(q_at(stage, p)), P::kE, q[p]);
          scale[p][0] = *scale_at(stage, p);
        } else {
          raw[p] = load_part<VEC>(dy + p * kSpan, left - p * kSpan);
          load_bytes<VEC>(kept + p * kSpan, left - p * kSpan, q[p]);
#pragma unroll
          for (int i = 0; i < P::kScales; ++i)
            scale[p][i] = left > p * kSpan + i * (int)kKeepGroup
                              ? scales[p * (kSpan / (int)kKeepGroup) + i] : 0.f;
        }
        float2 x[P::kPairs], d[P::kPairs], w[P::kPairs];
        weight(p, w);
        widen(raw[p], d, T());
#pragma unroll
        for (int i = 0; i < P::kBytes8; ++i) widen4(q[p][i], x[2 * i], x[2 * i + 1]);
#pragma unroll
        for (int i = 0; i < P::kScales; ++i) {
          float2 qq = both(0.f), dq = both(0.f);
#pragma unroll
          for (int e = i * kOf; e < (i + 1) * kOf; ++e) {  // of whole numbers; their scale after
            dw[p][e] = mul2(d[e], w[e]);
            qq = fma2(x[e], x[e], qq);
            dq = fma2(dw[p][e], x[e], dq);
          }
          xx = fma2(qq, both(scale[p][i] * scale[p][i]), xx);
          dx = fma2(dq, both(scale[p][i]), dx);
        }
      }
    }
    float sum[2] = {xx.x + xx.y, dx.x + dx.y};
    row_sum<G>(sum, red[flip], tid);
    const float r = rsqrtf(fmaf(sum[0], inv_dim, a.eps));
    const float m = sum[1] * r * inv_dim;  // mean of dy w n
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      if (live && left > p * kSpan) {
        float2 x[P::kPairs], d[P::kPairs], out[P::kPairs];
        widen(raw[p], d, T());
#pragma unroll
        for (int i = 0; i < P::kBytes8; ++i) widen4(q[p][i], x[2 * i], x[2 * i + 1]);
#pragma unroll
        for (int e = 0; e < P::kPairs; ++e) {
          const float2 n = mul2(x[e], both(r * scale[p][e / kOf]));
          acc[p][e] = fma2(d[e], n, acc[p][e]);
          out[e] = mul2(fma2(n, both(-m), dw[p][e]), both(r));
        }
        store_part<VEC>(dx_out + p * kSpan, left - p * kSpan, out);
      }
    }
    dx_out += step * a.ld_dx;
    if constexpr (kStages == 0) next_row();
    stage = stage + 1 >= kStages ? 0 : stage + 1;
    flip ^= 1;
  }
  // one row of partial sums for each group of threads
  const int ld = groups * (int)kKeepGroup;
  float* part = static_cast<float*>(a.workspace) + ((size_t)blockIdx.x * kRows + tid / G) * ld + col;
#pragma unroll
  for (int p = 0; p < kParts; ++p) {
    if (left <= p * kSpan) continue;
#pragma unroll
    for (int e = 0; e < P::kPairs; e += 2) {  // four columns at a time: a part of fp32
      const int at = p * kSpan + 2 * e * P::kStep;
      const float2 four[2] = {acc[p][e], acc[p][e + 1]};
      store_part<VEC>(part + at, left - at, four);
    }
  }
}

constexpr int kSumCols = 32, kSumRows = 32;

// dw[c] (+)= sum over the rows of partial sums, 32 of them at a time
__global__ void __launch_bounds__(kSumCols* kSumRows)
    norm_dweight_kernel(const float* part, size_t rows, size_t ld, float* dweight, size_t dim,
                        bool accumulate) {
  __shared__ float red[kSumRows][kSumCols + 1];
  pdl_wait_then_release();
  const int c = threadIdx.x % kSumCols, y = threadIdx.x / kSumCols;
  const size_t col = (size_t)blockIdx.x * kSumCols + c;
  float s = 0.f;
  if (col < dim) {
    const float* p = part + y * ld + col;
    size_t r = y;
    for (; r + 7 * kSumRows < rows; r += 8 * kSumRows) {  // eight loads under way
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = p[i * kSumRows * ld];
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i];
      p += 8 * kSumRows * ld;
    }
    for (; r < rows; r += kSumRows, p += kSumRows * ld) s += *p;
  }
  red[y][c] = s;
  __syncthreads();
  if (y == 0 && col < dim) {
#pragma unroll
    for (int i = 1; i < kSumRows; ++i) s += red[i][c];
    dweight[col] = accumulate ? dweight[col] + s : s;
  }
}

// Threads that share a row, and how often eight columns each of them holds
struct NormShape {
  int g, nv;
};
NormShape norm_shape(size_t dim) {
  const size_t vecs = (dim + 7) / 8;
  int g = 32;
  while (g < 1024 && (size_t)g * 2 < vecs) g *= 2;
  return {g, (size_t)g >= vecs ? 1 : (size_t)g * 2 >= vecs ? 2 : 4};
}

int norm_threads(const NormShape& s) { return s.g > 256 ? s.g : 256; }
int norm_rows_per_block(const NormShape& s) { return norm_threads(s) / s.g; }

// blocks that the rows need, at most what fills every SM once
size_t norm_blocks(size_t tokens, const NormShape& s, int per_sm) {
  const size_t rows = norm_rows_per_block(s);
  const size_t need = (tokens + rows - 1) / rows, fill = (size_t)sm_count() * per_sm;
  return need < fill ? need : fill;
}

template <typename F>
cudaError_t with_shape(const NormShape& s, F f) {
  using Two = std::integral_constant<int, 2>;
  switch (s.g) {
    case 32:
      if (s.nv == 1)
        return f(std::integral_constant<int, 32>(), std::integral_constant<int, 1>());
      return f(std::integral_constant<int, 32>(), Two());
    case 64: return f(std::integral_constant<int, 64>(), Two());
    case 128: return f(std::integral_constant<int, 128>(), Two());
    case 256: return f(std::integral_constant<int, 256>(), Two());
    case 512: return f(std::integral_constant<int, 512>(), Two());
  }
  if (s.nv == 2) return f(std::integral_constant<int, 1024>(), Two());
  return f(std::integral_constant<int, 1024>(), std::integral_constant<int, 4>());
}

template <typename T, bool VEC>
cudaError_t forward_of(const NormArgs& a, cudaStream_t stream) {
  const NormShape s = norm_shape(a.dim);
  return with_shape(s, [&](auto g, auto nv) {
    using F = NormFore<T, decltype(g)::value, decltype(nv)::value, VEC>;
    auto kernel = norm_forward_kernel<T, decltype(g)::value, decltype(nv)::value, VEC>;
    if (F::kShared > 40 * 1024) {  // with what is static, more than every kernel may have
      static std::atomic<uint64_t> allowed{0};
      const cudaError_t e = allow_shared(kernel, F::kShared, allowed);
      if (e != cudaSuccess) return e;
    }
    return launch_kernel(kernel, dim3((unsigned)norm_blocks(a.tokens, s, F::kPerSm)),
                         dim3(F::kThreads), F::kShared, stream, a);
  });
}

// *blocks: blocks launched, each of which leaves its rows of partial sums
template <typename T, bool VEC>
cudaError_t backward_of(const NormGradArgs& a, cudaStream_t stream, size_t* blocks) {
  const NormShape s = norm_shape(a.dim);
  return with_shape(s, [&](auto g, auto nv) {
    constexpr int G = decltype(g)::value;
    using B = NormBack<T, G, decltype(nv)::value, VEC>;
    auto kernel = norm_backward_kernel<T, G, decltype(nv)::value, VEC>;
    if (B::kShared > 40 * 1024) {  // with what is static, more than every kernel may have
      static std::atomic<uint64_t> allowed{0};
      const cudaError_t e = allow_shared(kernel, B::kShared, allowed);
      if (e != cudaSuccess) return e;
    }
    *blocks = norm_blocks(a.tokens, s, B::kPerSm);
    return launch_kernel(kernel, dim3((unsigned)*blocks), dim3(B::kThreads), B::kShared, stream, a);
  });
}

}  // namespace

cudaError_t launch_rmsnorm_forward(const NormArgs& a, cudaStream_t stream) {
  if (a.type == RCC_F32) return a.vec ? forward_of<float, true>(a, stream) : forward_of<float, false>(a, stream);
  return a.vec ? forward_of<__nv_bfloat16, true>(a, stream)
               : forward_of<__nv_bfloat16, false>(a, stream);
}

size_t rmsnorm_backward_workspace(size_t tokens, size_t dim) {
  const NormShape s = norm_shape(dim);
  const size_t ld = (dim + kKeepGroup - 1) / kKeepGroup * kKeepGroup;
  const int most = std::max(1, std::max(kBackThreads, kBackDirect) / norm_threads(s));
  return norm_blocks(tokens, s, most) * norm_rows_per_block(s) * ld * sizeof(float);
}

cudaError_t launch_rmsnorm_backward(const NormGradArgs& a, cudaStream_t stream,
                                    uint64_t* launches) {
  cudaError_t e;
  size_t blocks = 0;
  if (a.type == RCC_F32)
    e = a.vec ? backward_of<float, true>(a, stream, &blocks)
              : backward_of<float, false>(a, stream, &blocks);
  else
    e = a.vec ? backward_of<__nv_bfloat16, true>(a, stream, &blocks)
              : backward_of<__nv_bfloat16, false>(a, stream, &blocks);
  if (e != cudaSuccess) return e;
  const NormShape s = norm_shape(a.dim);
  const size_t ld = (a.dim + kKeepGroup - 1) / kKeepGroup * kKeepGroup;
  e = launch_kernel(norm_dweight_kernel, dim3((unsigned)((a.dim + kSumCols - 1) / kSumCols)),
                    dim3(kSumCols * kSumRows), 0, stream,
                    static_cast<const float*>(a.workspace),
                    blocks * norm_rows_per_block(s), ld,
                    a.dweight, a.dim, a.accumulate);
  if (e == cudaSuccess) *launches = 2;
  return e;
}

}  // namespace lm
}  // namespace rcc
