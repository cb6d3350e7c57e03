// rmsnorm.cuh -- RMS norm that keeps its input in 8 bits, and its backward pass
// from the 8 bits: the kernels of rmsnorm.cu, and of add_rmsnorm.cu with kAdd
// and kEight.
//
//   forward   r = 1/sqrt(mean(x^2) + eps);  y = x r w
//             kept: q = rint(x (127 (1/a))), s = a (1/127) with a = max|x| of 128
//             columns, every operation rounded to fp32
//   backward  x' = q s;  r = 1/sqrt(mean(x'^2) + eps);  n = x' r
//             dx = r (dy w - n mean(dy w n));  dw = sum over tokens of dy n
//   kAdd      forward: x is the sum of two inputs, rounded once to their type and
//             written; backward: the sum's own gradient is added to dx
//   kEight    y leaves as e4m3: y (448 (1/a)), s = a (1/448) with a = max|y| of 128
//             columns
//
// The backward pass is the exact gradient of the norm at the kept input x', so
// nothing but q and s (1.03 bytes an element) has to survive from the forward
// pass.
#pragma once

#include <algorithm>

#include "lm_common.cuh"
#include "lm_internal.h"

namespace rcc {
namespace lm {
namespace {

// What a kernel does beside the norm
constexpr int kAdd = 1, kEight = 2;

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
// Two values as e4m3, to nearest even, a in the low byte
__device__ __forceinline__ uint32_t e4m3_pair(float2 v) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(v.y), "f"(v.x));
  return d;
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

// A row of `dim` elements, and what else is in its first and last 16 bytes, into
// shared memory by the G threads that share it (t of them); nothing outside of
// [lo, hi), which holds all rows, is read.  The row then begins at `to` plus its
// address modulo 16.
template <int G, typename T>
__device__ __forceinline__ void copy_window(unsigned char* to, const T* row, int dim, const T* lo,
                                            const T* hi, int t) {
  const uintptr_t begin = reinterpret_cast<uintptr_t>(row);
  const uintptr_t end = begin + dim * sizeof(T), from = begin & ~uintptr_t{15};
  const int n = (int)((end - from + 15) / 16);
  for (int c = t; c < n; c += G) {
    const uintptr_t at = from + 16 * c;
    if (at >= reinterpret_cast<uintptr_t>(lo) && at + 16 <= reinterpret_cast<uintptr_t>(hi)) {
      copy_async<16>(to + 16 * c, reinterpret_cast<const void*>(at));
    } else {
      for (int e = 0; e < 16; e += (int)sizeof(T))
        if (at + e >= begin && at + e < end)
          *reinterpret_cast<T*>(to + 16 * c + e) = *reinterpret_cast<const T*>(at + e);
    }
  }
}
template <typename T>
__device__ __forceinline__ const T* in_window(const unsigned char* to, const T* row) {
  return reinterpret_cast<const T*>(to + (reinterpret_cast<uintptr_t>(row) & 15));
}
// What the threads of a row wrote is there for all of them.  G > 32: every
// thread of the block.
template <int G>
__device__ __forceinline__ void sync_row() {
  if constexpr (G > 32)
    __syncthreads();
  else
    __syncwarp();
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
// loads in flight by itself.  With an output in 8 bits there is more to do between
// a row's loads and its last store, and fp32 rows are copied ahead too: with the
// residual 150 us (5.8 TB/s; 143 of 8,192 columns) instead of 182 (234).  The
// residual alone, kept in 8 bits: 180 us as they are (6.3 TB/s), 186 copied ahead;
// bf16 97 us (6.3 TB/s), and 76 with the output in 8 bits.
constexpr int kForeThreads = 2048, kForeStages = 2, kForeDirect = 4096;
constexpr int kBackThreads = 512, kBackStages = 3, kBackDirect = 768;
constexpr int kSharedMost = 220 * 1024;   // of all blocks of one SM

// blocks of `threads` that one SM takes, of `shared` bytes each, for `all` threads
constexpr int blocks_per_sm(int all, int threads, int shared) {
  return shared && kSharedMost / shared < all / threads ? (kSharedMost / shared > 0 ? kSharedMost / shared : 1)
                                                        : (all / threads > 0 ? all / threads : 1);
}

// Rows copied ahead into shared memory.  Aligned rows (VEC): a thread writes and
// reads its own parts alone, so the copies need no barrier; a group's scale is one
// lane's copy, for the lanes of its warp.  Others: in whole 16 bytes that reach
// into the neighbouring rows, read back element by element behind a barrier, with
// another one between the last of that and the next copies into the same stage
// (16,384 x 4,095 bf16: 85 us instead of 102, with the residual 125 instead of 198,
// backward with kAdd 120 instead of 211; the backward pass without it stays as it
// was: its dweight would be summed in another order).
constexpr int kWindow = 32;  // bytes that a row's copy may be longer than the row
template <typename T, int G, int NV, bool VEC, int MORE>
struct NormFore {
  static constexpr int kThreads = kBlock<G>;
  static constexpr int kParts = NV * 8 / Part<T, VEC>::kE;
  static constexpr int kOne = NV * 8 * G * (int)sizeof(T) + (VEC ? 0 : kWindow);  // a row
  static constexpr int kRow = kThreads / G * kOne;  // the rows of one input
  static constexpr int kStage = MORE & kAdd ? 2 * kRow : kRow;
  static constexpr int kFit = kSharedMost / kStage;
  static constexpr int kStages =
      (!VEC || sizeof(T) == 2 || (MORE & kEight)) && kFit >= kForeStages ? kForeStages : 0;
  static constexpr int kShared = kStages * kStage;
  static constexpr int kPerSm = blocks_per_sm(kStages ? kForeThreads : kForeDirect, kThreads, kShared);
};

// One row for each group of G threads at a time; a thread keeps its part of
// the weight over all its rows.
template <typename T, int G, int NV, bool VEC, int MORE>
__global__ void __launch_bounds__(kBlock<G>) norm_forward_kernel(const NormArgs a) {
  using F = NormFore<T, G, NV, VEC, MORE>;
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
  [[maybe_unused]] const T* other = static_cast<const T*>(a.residual) + row * a.ld_residual + col;
  [[maybe_unused]] T* sum_out = static_cast<T*>(a.sum) + row * a.dim + col;
  [[maybe_unused]] T* y = static_cast<T*>(a.y) + row * a.ld_y + col;
  [[maybe_unused]] int8_t* y8 = static_cast<int8_t*>(a.y) + row * a.ld_y + col;
  [[maybe_unused]] float* y_scales = a.y_scales + row * groups + col / (int)kKeepGroup;
  int8_t* kept = a.kept + row * groups * kKeepGroup + col;
  float* scales = a.scales + row * groups + col / (int)kKeepGroup;
  size_t ahead_row = row;
  auto x_at = [&](int s, int p) {
    return reinterpret_cast<uint4*>(smem + s * F::kStage) + p * kThreads + tid;
  };
  // rows that are not aligned: where the group's lies in a stage
  [[maybe_unused]] auto window = [&](int s) {
    return smem + s * F::kStage + tid / G * F::kOne;
  };
  auto copy_row = [&](int s) {
    if (ahead_row < a.tokens) {
      if constexpr (!VEC) {
        const T* x = static_cast<const T*>(a.x);
        copy_window<G>(window(s), ahead - col, dim, x, x + (a.tokens - 1) * a.ld_x + dim, t);
        if constexpr ((MORE & kAdd) != 0) {
          const T* r = static_cast<const T*>(a.residual);
          copy_window<G>(window(s) + F::kRow, other - col, dim, r,
                         r + (a.tokens - 1) * a.ld_residual + dim, t);
        }
      } else {
#pragma unroll
        for (int p = 0; p < kParts; ++p)
          if (left > p * kSpan) {
            copy_async<16>(x_at(s, p), ahead + p * kSpan);
            if constexpr ((MORE & kAdd) != 0)
              copy_async<16>(x_at(s, p) + F::kRow / 16, other + p * kSpan);
          }
      }
    }
    copies_commit();  // one group a row, also when there is none
    ahead += step * a.ld_x;
    if constexpr ((MORE & kAdd) != 0) other += step * a.ld_residual;
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
    // this row's elements, where they are not copied by the threads that use them
    [[maybe_unused]] const T* here = ahead;
    [[maybe_unused]] const T* there = other;
    if constexpr (kStages > 0) {
      if constexpr (!VEC && G == 32) __syncwarp();  // all lanes are through with the stage
      copy_row(stage == 0 ? kStages - 1 : stage - 1);
      copies_wait<kStages - 1>();
      if constexpr (!VEC) {
        sync_row<G>();
        here = in_window(window(stage), static_cast<const T*>(a.x) + row * a.ld_x) + col;
        if constexpr ((MORE & kAdd) != 0)
          there = in_window(window(stage) + F::kRow,
                            static_cast<const T*>(a.residual) + row * a.ld_residual) + col;
      }
    }
    float2 v[kParts][P::kPairs];
    float2 sq = both(0.f);
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      uint4 raw = make_uint4(0u, 0u, 0u, 0u);
      if (live && left > p * kSpan) {
        if constexpr (VEC && kStages > 0)
          raw = *x_at(stage, p);
        else
          raw = load_part<VEC>(here + p * kSpan, left - p * kSpan);
      }
      widen(raw, v[p], T());
      if constexpr ((MORE & kAdd) != 0) {
        // the sum as it is written: the norm is taken of what the next layer reads
        if (live && left > p * kSpan) {
          float2 r[P::kPairs];
          widen(VEC && kStages > 0 ? x_at(stage, p)[F::kRow / 16]
                                   : load_part<VEC>(there + p * kSpan, left - p * kSpan), r, T());
#pragma unroll
          for (int e = 0; e < P::kPairs; ++e) v[p][e] = add2(v[p][e], r[e]);
          store_part<VEC>(sum_out + p * kSpan, left - p * kSpan, v[p]);
          if constexpr (sizeof(T) == 2) widen(narrow(v[p], T()), v[p], T());
        }
      }
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
        if constexpr ((MORE & kEight) == 0)
          store_part<VEC>(y + p * kSpan, left - p * kSpan, v[p]);
      }
      if constexpr ((MORE & kEight) != 0) {
        constexpr int kOf = P::kPairs / P::kScales;
        uint32_t q[P::kBytes8];
#pragma unroll
        for (int i = 0; i < P::kScales; ++i) {
          // lanes past the row hold zeros
          float top = 0.f;
#pragma unroll
          for (int e = i * kOf; e < (i + 1) * kOf; ++e)
            top = max_nan(max_nan(top, fabsf(v[p][e].x)), fabsf(v[p][e].y));
#pragma unroll
          for (int o = P::kLanes / 2; o > 0; o >>= 1)
            top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
          const bool fine = top >= kTiny && top < INFINITY;
          const float inv = fine ? 448.f * __frcp_rn(top) : 0.f;
          constexpr int kWords = P::kBytes8 / P::kScales;
#pragma unroll
          for (int k = i * kWords; k < (i + 1) * kWords; ++k)
            q[k] = fine ? e4m3_pair(mul2(v[p][2 * k], both(inv))) |
                              e4m3_pair(mul2(v[p][2 * k + 1], both(inv))) << 16
                        : 0u;
          if (live && t % P::kLanes == 0 && left > p * kSpan + i * (int)kKeepGroup)
            y_scales[p * (kSpan / (int)kKeepGroup) + i] =
                fine ? top * (1.f / 448.f)
                     : top < kTiny ? 0.f : __uint_as_float(0x7FC00000u);
        }
        if (live && left > p * kSpan) store_bytes<VEC>(y8 + p * kSpan, left - p * kSpan, q);
      }
    }
    if constexpr ((MORE & kAdd) != 0) sum_out += step * a.dim;
    if constexpr ((MORE & kEight) != 0) {
      y8 += step * a.ld_y;
      y_scales += step * groups;
    }
    y += step * a.ld_y;
    kept += step * groups * kKeepGroup;
    scales += step * groups;
    if constexpr (kStages == 0) {
      ahead += step * a.ld_x;
      if constexpr ((MORE & kAdd) != 0) other += step * a.ld_residual;
    }
    stage = stage + 1 >= kStages ? 0 : stage + 1;
    flip ^= 1;
  }
}

// ---- backward ------------------------------------------------------------------

// What a block of the backward pass holds in shared memory: the weight, and
// rows of dy, the 8-bit input and its scales copied ahead.  Where not even two
// rows fit (fp32 rows of more than 16,384; with kAdd, two inputs, fp32 of more than
// 8,192 and bf16 of more than 16,384) nothing is copied ahead and one block an SM
// loads as it goes.  With kAdd (without), 67 M elements: fp32 of 8,192 columns 134 us
// (98), of 12,288 217 (159), of 20,480 385 (241); bf16 of 8,192 74 (69), of 16,384
// 120 (93), of 20,480 205 (181).
template <typename T, int G, int NV, bool VEC, int MORE>
struct NormBack {
  static constexpr int kThreads = kBlock<G>;
  static constexpr int kParts = NV * 8 / Part<T, VEC>::kE;
  static constexpr int kScaled = kThreads / Part<T, VEC>::kLanes;  // groups of one part
  static constexpr int kOne = NV * 8 * G * (int)sizeof(T) + (VEC ? 0 : kWindow);  // a row
  static constexpr int kRow = kThreads / G * kOne;  // of dy, and of the sum's gradient
  static constexpr int kStage = kRow + kThreads * NV * 8 +
                                (VEC ? kParts * kScaled : kThreads * NV * 8 / (int)kKeepGroup) * 4 +
                                (MORE & kAdd ? kRow : 0);
  static constexpr bool kHoldWeight = kThreads * NV * 32 + 2 * kStage <= kSharedMost;
  static constexpr int kWeight = kHoldWeight ? kThreads * NV * 32 : 0;
  static constexpr int kFit = (kSharedMost - kWeight) / kStage;
  static constexpr int kStages = (VEC || (MORE & kAdd)) && kFit >= 2
                                     ? (kFit < kBackStages ? kFit : kBackStages) : 0;
  static constexpr int kShared = kWeight + kStages * kStage;
  static constexpr int kPerSm = blocks_per_sm(kStages ? kBackThreads : kBackDirect, kThreads, kShared);
  // Rows that are not aligned: dsum is read from its stage in front of the row's
  // reduction, whose barrier then stands between it and the next copies into that
  // stage; or, where a thread has no registers to hold it in, behind the reduction,
  // and a barrier of its own stands in front of the copies.  16,384 x 4,095 bf16 120 us
  // against 124, 8,190 x 8,191 131 against 137; fp32 4,095 183 against 182, 8,191 165
  // against 152; 4,095 x 16,383 bf16 198 against 184.
  static constexpr bool kEarly = kStages > 0 && !VEC && (MORE & kAdd) != 0 &&
                                 kThreads * (int)sizeof(T) <= 1024;
  // a block's rows of partial sums are added up where the weight was
  static constexpr bool kJoin = (MORE & kAdd) != 0 && kThreads > G && kHoldWeight;
};

// Rows are dealt to the blocks in turn; a thread keeps the weight gradient of
// its columns in registers over all of its rows, and each block writes one
// row of partial sums, which norm_dweight_kernel adds in a fixed order.
// Bandwidth bound: rows are copied ahead into shared memory (aligned rows, VEC;
// with kAdd others too) while the current one is reduced, where two of them fit.
template <typename T, int G, int NV, bool VEC, int MORE>
__global__ void __launch_bounds__(kBlock<G>, NormBack<T, G, NV, VEC, MORE>::kPerSm)
    norm_backward_kernel(const NormGradArgs a) {
  using B = NormBack<T, G, NV, VEC, MORE>;
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
  // the sum's own gradient, of the row that is copied ahead
  [[maybe_unused]] const T* dh = static_cast<const T*>(a.dsum) + row * a.ld_dsum + col;
  T* dx_out = static_cast<T*>(a.dx) + row * a.ld_dx + col;
  size_t ahead_row = row;
  // what neighbouring threads hold of one kind lies side by side
  auto weight_at = [&](int p, int h) {
    return reinterpret_cast<float4*>(smem) + (p * P::kBytes8 + h) * kThreads + tid;
  };
  auto dy_at = [&](int s, int p) {
    return reinterpret_cast<uint4*>(smem + B::kWeight + s * B::kStage) + p * kThreads + tid;
  };
  [[maybe_unused]] auto dh_at = [&](int s, int p) {  // behind the scales
    return reinterpret_cast<uint4*>(smem + B::kWeight + s * B::kStage + B::kStage - B::kRow) +
           p * kThreads + tid;
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
    if constexpr ((MORE & kAdd) != 0) dh += step * a.ld_dsum;
    kept += step * groups * kKeepGroup;
    scales += step * groups;
    ahead_row += step;
  };
  // rows that are not aligned: dy, the sum's gradient, bytes and scales of the
  // group's row, each kind's rows one after the other
  [[maybe_unused]] auto window = [&](int s, int input) {
    return smem + B::kWeight + s * B::kStage + input * B::kRow + tid / G * B::kOne;
  };
  constexpr int kInputs = MORE & kAdd ? 2 : 1;
  [[maybe_unused]] auto bytes_at = [&](int s) {
    return reinterpret_cast<int8_t*>(smem + B::kWeight + s * B::kStage + kInputs * B::kRow +
                                     tid / G * (NV * 8 * G));
  };
  [[maybe_unused]] auto scales_at = [&](int s) {
    return reinterpret_cast<float*>(smem + B::kWeight + s * B::kStage + kInputs * B::kRow +
                                    kThreads * NV * 8) + tid / G * (NV * 8 * G / (int)kKeepGroup);
  };
  auto copy_row = [&](int s) {
    if (!VEC && ahead_row < a.tokens) {
      const T* base = static_cast<const T*>(a.dy);
      copy_window<G>(window(s, 0), dy - col, dim, base, base + (a.tokens - 1) * a.ld_dy + dim, t);
      if constexpr ((MORE & kAdd) != 0) {
        base = static_cast<const T*>(a.dsum);
        copy_window<G>(window(s, 1), dh - col, dim, base,
                       base + (a.tokens - 1) * a.ld_dsum + dim, t);
      }
      for (int c = t; c < groups * (int)kKeepGroup / 16; c += G)
        copy_async<16>(bytes_at(s) + 16 * c, kept - col + 16 * c);
      for (int c = t; c < groups; c += G)
        copy_async<4>(scales_at(s) + c, scales - col / (int)kKeepGroup + c);
    } else if (ahead_row < a.tokens) {
#pragma unroll
      for (int p = 0; p < kParts; ++p) {
        if (left > p * kSpan) {
          copy_async<16>(dy_at(s, p), dy + p * kSpan);
          if constexpr ((MORE & kAdd) != 0) copy_async<16>(dh_at(s, p), dh + p * kSpan);
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
    // this row's elements, where they are not copied by the threads that use them
    [[maybe_unused]] const T* dy_here = dy;
    [[maybe_unused]] const T* dh_here = dh;
    [[maybe_unused]] const int8_t* kept_here = kept;
    [[maybe_unused]] const float* scales_here = scales;
    if constexpr (kStages > 0) {
      // Other threads' copies go into the stage that this one has read.  Of G > 32 the
      // barrier of row_sum is between all that is read in front of it and them.
      if constexpr (!VEC && (G == 32 || !B::kEarly)) sync_row<G>();
      copy_row(stage == 0 ? kStages - 1 : stage - 1);
      copies_wait<kStages - 1>();
      if constexpr (VEC) {
        __syncwarp();  // a group's scale is one lane's copy
      } else {
        sync_row<G>();
        dy_here = in_window(window(stage, 0), static_cast<const T*>(a.dy) + row * a.ld_dy) + col;
        if constexpr ((MORE & kAdd) != 0)
          dh_here =
              in_window(window(stage, 1), static_cast<const T*>(a.dsum) + row * a.ld_dsum) + col;
        kept_here = bytes_at(stage) + col;
        scales_here = scales_at(stage) + col / (int)kKeepGroup;
      }
    }
    // kept over the reduction: dy w, and dy and the bytes as they came
    uint4 raw[kParts];
    [[maybe_unused]] uint4 raw_dh[kParts];  // kEarly
    uint32_t q[kParts][P::kBytes8];
    float2 dw[kParts][P::kPairs];
    float scale[kParts][P::kScales];
    float2 xx = both(0.f), dx = both(0.f);  // sums of x'^2, of dy w x'
    constexpr int kOf = P::kPairs / P::kScales;  // pairs of one scale
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      if (live && left > p * kSpan) {
        if constexpr (VEC && kStages > 0) {
          raw[p] = *dy_at(stage, p);
          load_bytes<VEC>(reinterpret_cast<const int8_t*>(q_at(stage, p)), P::kE, q[p]);
          scale[p][0] = *scale_at(stage, p);
        } else {
          raw[p] = load_part<VEC>(dy_here + p * kSpan, left - p * kSpan);
          load_bytes<VEC>(kept_here + p * kSpan, left - p * kSpan, q[p]);
          if constexpr (B::kEarly) raw_dh[p] = load_part<VEC>(dh_here + p * kSpan, left - p * kSpan);
#pragma unroll
          for (int i = 0; i < P::kScales; ++i)
            scale[p][i] = left > p * kSpan + i * (int)kKeepGroup
                              ? scales_here[p * (kSpan / (int)kKeepGroup) + i] : 0.f;
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
        if constexpr ((MORE & kAdd) != 0) {
          float2 more[P::kPairs];
          if constexpr (B::kEarly)
            widen(raw_dh[p], more, T());
          else
            widen(VEC && kStages > 0 ? *dh_at(stage, p)
                                     : load_part<VEC>(dh_here + p * kSpan, left - p * kSpan),
                  more, T());
#pragma unroll
          for (int e = 0; e < P::kPairs; ++e) out[e] = add2(out[e], more[e]);
        }
        store_part<VEC>(dx_out + p * kSpan, left - p * kSpan, out);
      }
    }
    dx_out += step * a.ld_dx;
    if constexpr (kStages == 0) next_row();
    stage = stage + 1 >= kStages ? 0 : stage + 1;
    flip ^= 1;
  }
  // one row of partial sums for each group of threads; with kAdd for each block,
  // whose groups' sums are added first (1,023 rows of 1,000 fp32 columns: 256 rows
  // left to norm_dweight_kernel instead of 1,024)
  const int ld = groups * (int)kKeepGroup;
  float* part = static_cast<float*>(a.workspace) + ((size_t)blockIdx.x * kRows + tid / G) * ld + col;
  if constexpr (B::kJoin) {
    __syncthreads();  // the weight is read no more
    auto held = [&](int group, int p, int e) {
      return reinterpret_cast<float2*>(smem) + ((group * kParts + p) * P::kPairs + e) * G + t;
    };
#pragma unroll
    for (int p = 0; p < kParts; ++p)
#pragma unroll
      for (int e = 0; e < P::kPairs; ++e) *held(tid / G, p, e) = acc[p][e];
    __syncthreads();
    if (tid >= G) return;
    for (int r = 1; r < kRows; ++r)
#pragma unroll
      for (int p = 0; p < kParts; ++p)
#pragma unroll
        for (int e = 0; e < P::kPairs; ++e) acc[p][e] = add2(acc[p][e], *held(r, p, e));
    part = static_cast<float*>(a.workspace) + (size_t)blockIdx.x * ld + col;
  }
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

template <typename T, bool VEC, int MORE>
cudaError_t forward_of(const NormArgs& a, cudaStream_t stream) {
  const NormShape s = norm_shape(a.dim);
  return with_shape(s, [&](auto g, auto nv) {
    using F = NormFore<T, decltype(g)::value, decltype(nv)::value, VEC, MORE>;
    auto kernel = norm_forward_kernel<T, decltype(g)::value, decltype(nv)::value, VEC, MORE>;
    if (F::kShared > 40 * 1024) {  // with what is static, more than every kernel may have
      static std::atomic<uint64_t> allowed{0};
      const cudaError_t e = allow_shared(kernel, F::kShared, allowed);
      if (e != cudaSuccess) return e;
    }
    return launch_kernel(kernel, dim3((unsigned)norm_blocks(a.tokens, s, F::kPerSm)),
                         dim3(F::kThreads), F::kShared, stream, a);
  });
}

// *rows: rows of partial sums that the blocks leave
template <typename T, bool VEC, int MORE>
cudaError_t backward_of(const NormGradArgs& a, cudaStream_t stream, size_t* rows) {
  const NormShape s = norm_shape(a.dim);
  return with_shape(s, [&](auto g, auto nv) {
    constexpr int G = decltype(g)::value;
    using B = NormBack<T, G, decltype(nv)::value, VEC, MORE>;
    auto kernel = norm_backward_kernel<T, G, decltype(nv)::value, VEC, MORE>;
    if (B::kShared > 40 * 1024) {  // with what is static, more than every kernel may have
      static std::atomic<uint64_t> allowed{0};
      const cudaError_t e = allow_shared(kernel, B::kShared, allowed);
      if (e != cudaSuccess) return e;
    }
    const size_t blocks = norm_blocks(a.tokens, s, B::kPerSm);
    *rows = B::kJoin ? blocks : blocks * norm_rows_per_block(s);
    return launch_kernel(kernel, dim3((unsigned)blocks), dim3(B::kThreads), B::kShared, stream, a);
  });
}


template <int MORE>
cudaError_t forward_with(const NormArgs& a, cudaStream_t stream) {
  if (a.type == RCC_F32)
    return a.vec ? forward_of<float, true, MORE>(a, stream)
                 : forward_of<float, false, MORE>(a, stream);
  return a.vec ? forward_of<__nv_bfloat16, true, MORE>(a, stream)
               : forward_of<__nv_bfloat16, false, MORE>(a, stream);
}

// dx, then dweight from the blocks' rows of partial sums
template <int MORE>
cudaError_t backward_with(const NormGradArgs& a, cudaStream_t stream, uint64_t* launches) {
  cudaError_t e;
  size_t rows = 0;
  if (a.type == RCC_F32)
    e = a.vec ? backward_of<float, true, MORE>(a, stream, &rows)
              : backward_of<float, false, MORE>(a, stream, &rows);
  else
    e = a.vec ? backward_of<__nv_bfloat16, true, MORE>(a, stream, &rows)
              : backward_of<__nv_bfloat16, false, MORE>(a, stream, &rows);
  if (e != cudaSuccess) return e;
  const size_t ld = (a.dim + kKeepGroup - 1) / kKeepGroup * kKeepGroup;
  e = launch_kernel(norm_dweight_kernel, dim3((unsigned)((a.dim + kSumCols - 1) / kSumCols)),
                    dim3(kSumCols * kSumRows), 0, stream,
                    static_cast<const float*>(a.workspace), rows, ld, a.dweight, a.dim,
                    a.accumulate);
  if (e == cudaSuccess) *launches = 2;
  return e;
}

}  // namespace
}  // namespace lm
}  // namespace rcc
