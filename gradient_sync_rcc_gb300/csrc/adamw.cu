// adamw.cu -- AdamW over many tensors, its states in fp32 or in 8 bits.
//
//   g = grad (1/scale) coef,  coef = max_grad_norm / |g| where that is less than 1
//   m = b1 m + (1-b1) g;  v = b2 v + (1-b2) g^2
//   p = p (1 - lr wd) - lr/(1-b1^t) m / (sqrt(v) / sqrt(1-b2^t) + eps)
// every operation rounded to fp32 in this order, as rcc_grad_sync_adamw's.
//
// States in 8 bits: m and sqrt(v) (half the range of v, and what is divided by)
// as e4m3 with one scale for 128 elements, the smallest power of two that holds
// the largest of them.  A scale of another form would move every value off the
// grid at every step; so a value that does not change is held as it was.  A
// value between two of the grid is rounded up with the chance of its distance:
// a second moment moves by 0.1% a step where the grid's steps are 6 to 12%, and
// rounding to nearest would hold it where it is.  The numbers are a hash of
// seed, step, tensor and place: the same call gives the same bits.  A sqrt(v)
// above zero is never held as zero, which would let m / sqrt(v) grow without
// bound.
//
// One pass over the gradients for their norm, one that updates.  Both are bound
// by memory: a block takes a range of neighbouring items (4,096 elements of a
// tensor), the update from its end, where the gradients are still in L2.
#include "lm_common.cuh"
#include "lm_internal.h"

namespace rcc {
namespace lm {
namespace {

constexpr int kThreads = 256;
constexpr int kUnit = 8;                             // elements of a thread at a time
constexpr int kUnits = kAdamWItem / (kThreads * kUnit);  // of them in an item
constexpr int kGroup = 128;                          // elements that share a scale
constexpr int kLanes = kGroup / kUnit;               // threads that share one
constexpr uint32_t kGolden = 0x9E3779B9u;            // the golden ratio's fraction
constexpr uint32_t kRootTwo = 0x6A09E667u, kRootThree = 0xBB67AE85u;  // the roots' fractions

static_assert(kAdamWItem % (kThreads * kUnit) == 0 && kLanes == 16, "whole units and groups");

__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= kRootTwo;
  x ^= x >> 15;
  x *= kRootThree;
  return x ^ (x >> 16);
}

// Items [lo, hi) of block b of n
__device__ __forceinline__ void range_of(uint64_t items, uint64_t& lo, uint64_t& hi) {
  const uint64_t n = gridDim.x, b = blockIdx.x;
  lo = items / n * b + min(b, items % n);
  hi = lo + items / n + (b < items % n ? 1 : 0);
}

// ---- the gradients' norm --------------------------------------------------------

__device__ __forceinline__ float grad_at(const AdamWTensor& t, uint64_t i) {
  return t.bf16 ? to_f32(static_cast<const __nv_bfloat16*>(t.grad)[i])
                : static_cast<const float*>(t.grad)[i];
}

// A thread's sum of squares as a value and the error it has run up, two of each:
// sum' = fl(sum + g^2) is one fused operation, and what it dropped is exact but
// for u^2 of it, so n squares are good to n 2^-48, without GB300's few fp64
// units.  Seven instructions for two elements.
struct Squares {
  float2 sum = both(0.f), rest = both(0.f);
  uint32_t seen = 0;  // bits of the elements but their signs
  __device__ __forceinline__ void add(float2 g) {
    const float2 t = fma2(g, g, sum);
    const float2 d = add2(t, neg(sum));  // near g^2
    const float2 of_sum = add2(sum, neg(add2(t, neg(d))));
    rest = add2(rest, add2(of_sum, fma2(g, g, neg(d))));
    sum = t;
  }
  static __device__ __forceinline__ float2 neg(float2 v) { return make_float2(-v.x, -v.y); }
  // Neither overflown nor among the smallest numbers, where errors are lost
  __device__ __forceinline__ bool sound() const {
    const float s = sum.x + sum.y;
    return seen == 0 || (s > 0x1p-60f && s < 0x1p100f);
  }
  __device__ __forceinline__ double value() const {
    return ((double)sum.x + (double)rest.x) + ((double)sum.y + (double)rest.y);
  }
};

// fp64, for gradients that Squares cannot sum; counts what is not finite
struct WideSquares {
  double sum = 0.0;
  uint32_t bad = 0;
  __device__ __forceinline__ void add(float g) {
    if (!(fabsf(g) < INFINITY))
      ++bad;
    else if (g != 0.f)
      sum += (double)g * (double)g;
  }
};

// Eight gradients as they lie in memory
struct Raw {
  uint32_t w[8];
};
__device__ __forceinline__ void load_raw(const AdamWTensor& t, uint64_t i, Raw& r) {
  if (t.bf16) {
    const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(t.grad) + i);
    r.w[0] = v.x;
    r.w[1] = v.y;
    r.w[2] = v.z;
    r.w[3] = v.w;
  } else {
    float f[8];
    load8(static_cast<const float*>(t.grad) + i, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) r.w[e] = __float_as_uint(f[e]);
  }
}
__device__ __forceinline__ float2 pair_of(const AdamWTensor& t, const Raw& r, int i) {
  if (!t.bf16) return make_float2(__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1]));
  float2 v;
  widen2(r.w[i], v.x, v.y);
  return v;
}

// Elements [begin, end) of a tensor, begin on a whole item
__device__ __forceinline__ void add_range(const AdamWTensor& t, uint64_t begin, uint64_t end,
                                          Squares& s) {
  constexpr int kAhead = 4;  // vectors of a thread under way
  uint64_t from = begin;
  if (t.vec) {
    const uint64_t vectors = (end - begin) / kUnit;
    for (uint64_t v = threadIdx.x; v < vectors; v += kAhead * kThreads) {
      Raw r[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (v + k * kThreads < vectors) load_raw(t, begin + (v + k * kThreads) * kUnit, r[k]);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (v + k * kThreads >= vectors) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s.seen |= t.bf16 ? r[k].w[i] & 0x7FFF7FFFu
                           : (r[k].w[2 * i] | r[k].w[2 * i + 1]) & 0x7FFFFFFFu;
          s.add(pair_of(t, r[k], i));
        }
      }
    }
    from = begin + vectors * kUnit;
  }
  for (uint64_t i = from + threadIdx.x; i < end; i += kThreads) {
    const float g = grad_at(t, i);
    s.seen |= __float_as_uint(g) & 0x7FFFFFFFu;
    s.add(make_float2(g, 0.f));
  }
}

// The tensors' pieces within the block's items, one after the other
template <typename F>
__device__ __forceinline__ void for_each_range(const AdamWArgs& a, F f) {
  uint64_t lo, hi;
  range_of(a.num_items, lo, hi);
  AdamWItem it = a.items[lo];
  while (lo < hi) {
    const AdamWTensor t = a.tensors[it.tensor];
    const uint64_t begin = (uint64_t)it.chunk * kAdamWItem;
    const uint64_t left = (t.numel - begin + kAdamWItem - 1) / kAdamWItem;  // items of the tensor
    const uint64_t take = min(left, hi - lo);
    f(t, begin, min(begin + take * kAdamWItem, t.numel));
    lo += take;
    it = {it.tensor + 1, 0};
  }
}

// Sums over the block, for thread 0; `sums` and `bads` are free again after the
// next barrier
__device__ __forceinline__ void block_sum(double& sum, unsigned long long& bad, double* sums,
                                          unsigned long long* bads) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    bad += __shfl_xor_sync(0xFFFFFFFFu, bad, o);
  }
  if (threadIdx.x % 32 == 0) {
    sums[threadIdx.x / 32] = sum;
    bads[threadIdx.x / 32] = bad;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) {
      sum += sums[w];
      bad += bads[w];
    }
  }
}

// Whether and how the step is taken: one thread, once a step
__device__ __forceinline__ void decide(const AdamWArgs& a, double sum, unsigned long long bad) {
  rcc_adamw_status s = *a.status;
  AdamWDecision d = {};
  const double norm = sqrt(sum) / a.scale;
  d.skip = bad > 0 || !(norm < INFINITY);
  d.coef = !d.skip && a.max_norm > 0.0 && norm > a.max_norm ? (float)(a.max_norm / norm) : 1.f;
  d.step = (uint32_t)s.step;
  s.grad_norm = norm;
  s.nonfinite = bad > 0xFFFFFFFFull ? 0xFFFFFFFFu : (uint32_t)bad;
  s.skipped = d.skip;
  s.clip_coef = d.coef;
  if (!d.skip) {
    s.step += 1;
    s.beta1_power *= a.beta1;
    s.beta2_power *= a.beta2;
    d.step_size = (float)(a.lr / (1.0 - s.beta1_power));
    d.inv_root = (float)(1.0 / sqrt(1.0 - s.beta2_power));
  }
  *a.status = s;
  *a.decision = d;
}

// Each block leaves one row; the last one to do so adds them up, in the rows'
// order, and decides.
__global__ void __launch_bounds__(kThreads) adamw_norm_kernel(const AdamWArgs a) {
  __shared__ double sums[kThreads / 32];
  __shared__ unsigned long long bads[kThreads / 32];
  __shared__ bool last;
  pdl_wait_then_release();
  Squares s;
  for_each_range(a, [&](const AdamWTensor& t, uint64_t begin, uint64_t end) {
    add_range(t, begin, end, s);
  });
  double sum = s.value();
  unsigned long long bad = 0;
  if (!s.sound()) {
    WideSquares w;
    for_each_range(a, [&](const AdamWTensor& t, uint64_t begin, uint64_t end) {
      // the same elements of this thread
      uint64_t from = begin;
      if (t.vec) {
        const uint64_t vectors = (end - begin) / kUnit;
        for (uint64_t v = threadIdx.x; v < vectors; v += kThreads)
          for (int e = 0; e < kUnit; ++e) w.add(grad_at(t, begin + v * kUnit + e));
        from = begin + vectors * kUnit;
      }
      for (uint64_t i = from + threadIdx.x; i < end; i += kThreads) w.add(grad_at(t, i));
    });
    sum = w.sum;
    bad = w.bad;
  }
  block_sum(sum, bad, sums, bads);
  if (threadIdx.x == 0) {
    a.rows[blockIdx.x] = {sum, (uint32_t)min(bad, 0xFFFFFFFFull), 0u};
    __threadfence();
    last = atomicAdd(a.arrived, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  sum = 0.0;
  bad = 0;
  for (uint32_t r = threadIdx.x; r < gridDim.x; r += kThreads) {
    sum += __ldcg(&a.rows[r].sum);
    bad += __ldcg(&a.rows[r].bad);
  }
  block_sum(sum, bad, sums, bads);
  if (threadIdx.x == 0) {
    *a.arrived = 0;
    decide(a, sum, bad);
  }
}

// ---- the update -----------------------------------------------------------------

struct Unit {
  float g[kUnit], p[kUnit], m[kUnit], v[kUnit];
};

__device__ __forceinline__ void widen_e4m3(uint2 q, float (&v)[kUnit]) {
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h;  // two halves: e4m3 is exact in them
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(w[i / 2] >> (16 * (i % 2)))));
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\t"
        "cvt.f32.f16 %1, b;\n\t}" : "=f"(v[2 * i]), "=f"(v[2 * i + 1]) : "r"(h));
  }
}
__device__ __forceinline__ uint2 narrow_e4m3(const float (&v)[kUnit]) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(v[4 * i + 1]), "f"(v[4 * i]));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(v[4 * i + 3]), "f"(v[4 * i + 2]));
    w[i] = lo | (uint32_t)hi << 16;
  }
  return make_uint2(w[0], w[1]);
}

// The smallest power of two s with top <= 448 s: 448 is 1.75 2^8, so a fraction
// above 0.75 carries into the exponent.  0 for next to nothing, NaN for a NaN.
__device__ __forceinline__ float power_for(uint32_t top_bits) {
  const float top = __uint_as_float(top_bits);
  if (top < kAdamWNothing) return 0.f;
  if (!(top <= INFINITY)) return top;
  const uint32_t b = min(top_bits, 0x7F7FFFFFu);
  return __uint_as_float(((b + 0x1FFFFFu) & 0x7F800000u) - (8u << 23));
}

// y >= 0 on the grid of e4m3, up with a chance of its distance over a step:
// `number` of 2^16.  Below 2^-6 the grid is even, as it is from 2^-6 to 2^-5.
__device__ __forceinline__ float round_e4m3(float y, uint32_t number) {
  const float low = y < 0x1p-6f ? 0x1p-6f : 0.f;
  const uint32_t b = (__float_as_uint(__fadd_rn(y, low)) + (number << 4)) & 0xFFF00000u;
  return fminf(__uint_as_float(b) - low, 448.f);
}

// The largest of the 16 threads of a group, as bits: a NaN is the largest of all
__device__ __forceinline__ uint32_t group_max(uint32_t bits) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1)
    bits = max(bits, __shfl_xor_sync(0xFFFFFFFFu, bits, o));
  return bits;
}

// Values to hold: |v| by their scale, rounded, with their sign
template <bool ROOT>
__device__ __forceinline__ float hold(float (&v)[kUnit], const uint32_t (&numbers)[kUnit]) {
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < kUnit; ++e) top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
  const float scale = power_for(group_max(top));
  const float inv = scale > 0.f ? __uint_as_float((254u << 23) - __float_as_uint(scale)) : 0.f;
#pragma unroll
  for (int e = 0; e < kUnit; ++e) {
    const float y = fabsf(v[e]) * inv;
    float w = round_e4m3(y, numbers[e]);
    if (ROOT) w = y > 0.f ? fmaxf(w, 0x1p-9f) : 0.f;
    v[e] = copysignf(w, v[e]);
  }
  return scale;
}

// Up to eight elements from the i-th on; zeros past the tensor
template <bool EIGHT>
__device__ __forceinline__ void load_unit(const AdamWTensor& t, uint64_t i, bool whole, Unit& u) {
  if (whole) {
    if (t.bf16)
      load8(static_cast<const __nv_bfloat16*>(t.grad) + i, u.g);
    else
      load8(static_cast<const float*>(t.grad) + i, u.g);
    load8(t.param + i, u.p);
    if constexpr (EIGHT) {
      widen_e4m3(*reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.m) + i), u.m);
      widen_e4m3(*reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.v) + i), u.v);
    } else {
      load8(static_cast<const float*>(t.m) + i, u.m);
      load8(static_cast<const float*>(t.v) + i, u.v);
    }
    return;
  }
  uint32_t q[2][2] = {};
#pragma unroll
  for (int e = 0; e < kUnit; ++e) {
    const bool live = i + e < t.numel;
    u.g[e] = live ? grad_at(t, i + e) : 0.f;
    u.p[e] = live ? t.param[i + e] : 0.f;
    if constexpr (EIGHT) {
      q[0][e / 4] |= (live ? static_cast<const uint8_t*>(t.m)[i + e] : 0u) << (8 * (e % 4));
      q[1][e / 4] |= (live ? static_cast<const uint8_t*>(t.v)[i + e] : 0u) << (8 * (e % 4));
    } else {
      u.m[e] = live ? static_cast<const float*>(t.m)[i + e] : 0.f;
      u.v[e] = live ? static_cast<const float*>(t.v)[i + e] : 0.f;
    }
  }
  if constexpr (EIGHT) {
    widen_e4m3(make_uint2(q[0][0], q[0][1]), u.m);
    widen_e4m3(make_uint2(q[1][0], q[1][1]), u.v);
  }
}

template <bool EIGHT>
__device__ __forceinline__ void store_unit(const AdamWTensor& t, uint64_t i, bool whole,
                                           const Unit& u) {
  uint2 m8 = {}, v8 = {};
  if constexpr (EIGHT) {
    m8 = narrow_e4m3(u.m);
    v8 = narrow_e4m3(u.v);
  }
  if (whole) {
    store8(t.param + i, u.p);
    if (t.copy) store8(t.copy + i, u.p);
    if constexpr (EIGHT) {
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.m) + i) = m8;
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.v) + i) = v8;
    } else {
      store8(static_cast<float*>(t.m) + i, u.m);
      store8(static_cast<float*>(t.v) + i, u.v);
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < kUnit; ++e) {
    if (i + e >= t.numel) continue;
    t.param[i + e] = u.p[e];
    if (t.copy) from_f32(u.p[e], t.copy[i + e]);
    if constexpr (EIGHT) {
      static_cast<uint8_t*>(t.m)[i + e] = (uint8_t)((e < 4 ? m8.x : m8.y) >> (8 * (e % 4)));
      static_cast<uint8_t*>(t.v)[i + e] = (uint8_t)((e < 4 ? v8.x : v8.y) >> (8 * (e % 4)));
    } else {
      static_cast<float*>(t.m)[i + e] = u.m[e];
      static_cast<float*>(t.v)[i + e] = u.v[e];
    }
  }
}

template <bool EIGHT>
__global__ void __launch_bounds__(kThreads) adamw_update_kernel(const AdamWArgs a) {
  pdl_wait_then_release();
  const AdamWDecision d = *a.decision;
  if (d.skip) return;
  uint64_t lo, hi;
  range_of(a.num_items, lo, hi);
  const uint32_t key = mix(a.seed ^ mix(d.step));
  for (uint64_t item = hi; item-- > lo;) {
    const AdamWItem it = a.items[item];
    const AdamWTensor t = a.tensors[it.tensor];
    const uint32_t block_key = mix(mix(key + it.tensor * kGolden) ^ it.chunk);
    for (int k = 0; k < kUnits; ++k) {
      const uint32_t inside = (k * kThreads + threadIdx.x) * kUnit;
      const uint64_t i = (uint64_t)it.chunk * kAdamWItem + inside;
      const bool whole = t.vec && i + kUnit <= t.numel;
      Unit u;
      load_unit<EIGHT>(t, i, whole, u);
      if constexpr (EIGHT) {
        const bool live = i < t.numel;
        const float ms = live ? t.m_scales[i / kGroup] : 0.f;
        const float vs = live ? t.v_scales[i / kGroup] : 0.f;
#pragma unroll
        for (int e = 0; e < kUnit; ++e) {
          u.m[e] = __fmul_rn(u.m[e], ms);
          u.v[e] = __fmul_rn(u.v[e], vs);
          u.v[e] = __fmul_rn(u.v[e], u.v[e]);
        }
      }
#pragma unroll
      for (int e = 0; e < kUnit; ++e) {
        const float g = __fmul_rn(__fmul_rn(u.g[e], a.inv_scale), d.coef);
        u.m[e] = __fadd_rn(__fmul_rn(a.b1, u.m[e]), __fmul_rn(a.one_minus_b1, g));
        u.v[e] = __fadd_rn(__fmul_rn(a.b2, u.v[e]), __fmul_rn(a.one_minus_b2, __fmul_rn(g, g)));
        const float root = __fsqrt_rn(u.v[e]);
        const float denom = __fadd_rn(__fmul_rn(root, d.inv_root), a.eps);
        u.p[e] = __fsub_rn(__fmul_rn(u.p[e], a.decay),
                           __fmul_rn(d.step_size, __fdiv_rn(u.m[e], denom)));
        if (EIGHT) u.v[e] = root;
      }
      if constexpr (EIGHT) {
        uint32_t numbers[kUnit];
#pragma unroll
        for (int e = 0; e < kUnit; e += 2) {
          const uint32_t h = mix(block_key + (inside + e) / 2);
          numbers[e] = h & 0xFFFFu;
          numbers[e + 1] = h >> 16;
        }
        const float ms = hold<false>(u.m, numbers), vs = hold<true>(u.v, numbers);
        if (threadIdx.x % kLanes == 0 && i < t.numel) {
          t.m_scales[i / kGroup] = ms;
          t.v_scales[i / kGroup] = vs;
        }
      }
      store_unit<EIGHT>(t, i, whole, u);
    }
  }
}

}  // namespace

cudaError_t launch_adamw(const AdamWArgs& a, bool eight, cudaStream_t stream,
                         uint64_t* launches) {
  const uint64_t fill = (uint64_t)a.num_rows;
  const unsigned blocks = (unsigned)(a.num_items < fill ? a.num_items : fill);
  cudaError_t e = launch_kernel(adamw_norm_kernel, dim3(blocks), dim3(kThreads), 0, stream, a);
  if (e != cudaSuccess) return e;
  e = launch_kernel(eight ? adamw_update_kernel<true> : adamw_update_kernel<false>, dim3(blocks),
                    dim3(kThreads), 0, stream, a);
  if (e == cudaSuccess) *launches = 2;
  return e;
}

int adamw_rows() { return sm_count() * 8; }

}  // namespace lm
}  // namespace rcc
