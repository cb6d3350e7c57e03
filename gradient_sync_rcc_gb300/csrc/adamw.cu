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

#ifndef NORM_AHEAD
#define NORM_AHEAD 2
#define NORM_PER_SM 4
#define UPD_AHEAD 1
#define UPD_PER_SM 4
#endif
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
template <bool BF16>
struct Raw {
  static constexpr int kWords = BF16 ? 4 : 8;
  uint32_t w[kWords];
};
__device__ __forceinline__ void load_raw(const void* grad, uint64_t i, Raw<true>& r) {
  const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(grad) + i);
  r.w[0] = v.x;
  r.w[1] = v.y;
  r.w[2] = v.z;
  r.w[3] = v.w;
}
__device__ __forceinline__ void load_raw(const void* grad, uint64_t i, Raw<false>& r) {
  float f[8];
  load8(static_cast<const float*>(grad) + i, f);
#pragma unroll
  for (int e = 0; e < 8; ++e) r.w[e] = __float_as_uint(f[e]);
}
__device__ __forceinline__ float2 pair_of(const Raw<true>& r, int i) {
  float2 v;
  widen2(r.w[i], v.x, v.y);
  return v;
}
__device__ __forceinline__ float2 pair_of(const Raw<false>& r, int i) {
  return make_float2(__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1]));
}

// Elements [begin, end) of a tensor, begin on a whole item
template <bool BF16>
__device__ __forceinline__ void add_vectors(const void* grad, uint64_t begin, uint64_t vectors,
                                            Squares& s) {
  constexpr int kAhead = BF16 ? 2 * NORM_AHEAD : NORM_AHEAD;  // vectors of a thread under way
  for (uint64_t v = threadIdx.x; v < vectors; v += kAhead * kThreads) {
    Raw<BF16> r[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
#pragma unroll
      for (int e = 0; e < Raw<BF16>::kWords; ++e) r[k].w[e] = 0u;
      if (v + k * kThreads < vectors) load_raw(grad, begin + (v + k * kThreads) * kUnit, r[k]);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
#pragma unroll
      for (int e = 0; e < Raw<BF16>::kWords; ++e)
        s.seen |= r[k].w[e] & (BF16 ? 0x7FFF7FFFu : 0x7FFFFFFFu);
#pragma unroll
      for (int i = 0; i < 4; ++i) s.add(pair_of(r[k], i));
    }
  }
}
__device__ __forceinline__ void add_range(const AdamWTensor& t, uint64_t begin, uint64_t end,
                                          Squares& s) {
  uint64_t from = begin;
  if (t.vec) {
    const uint64_t vectors = (end - begin) / kUnit;
    if (t.bf16)
      add_vectors<true>(t.grad, begin, vectors, s);
    else
      add_vectors<false>(t.grad, begin, vectors, s);
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
    d.factor = (float)((double)d.coef / a.scale);
    d.step_size = (float)(a.lr / (1.0 - s.beta1_power));
    d.inv_root = (float)(1.0 / sqrt(1.0 - s.beta2_power));
  }
  *a.status = s;
  *a.decision = d;
}

// Each block leaves one row; the last one to do so adds them up, in the rows'
// order, and decides.
__global__ void __launch_bounds__(kThreads, NORM_PER_SM) adamw_norm_kernel(const AdamWArgs a) {
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

// Eight neighbours as they lie in memory, and their group's scales
template <bool EIGHT, bool BF16>
struct Unit {
  Raw<BF16> g;
  float p[kUnit];
  float m[EIGHT ? 1 : kUnit], v[EIGHT ? 1 : kUnit];
  uint2 m8, v8;
  float ms, vs;
};

__device__ __forceinline__ void widen_e4m3(uint2 q, float2 (&v)[4]) {
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h;  // two halves: e4m3 is exact in them
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(w[i / 2] >> (16 * (i % 2)))));
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\t"
        "cvt.f32.f16 %1, b;\n\t}" : "=f"(v[i].x), "=f"(v[i].y) : "r"(h));
  }
}
__device__ __forceinline__ uint2 narrow_e4m3(const float2 (&v)[4]) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(v[2 * i].y), "f"(v[2 * i].x));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(hi) : "f"(v[2 * i + 1].y), "f"(v[2 * i + 1].x));
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
// `chance`, of 2^20.  Below 2^-6 the grid is even, as it is from 2^-6 to 2^-5.
// Over 448 is left to the conversion, which saturates.
__device__ __forceinline__ float round_e4m3(float y, uint32_t chance) {
  const float low = y < 0x1p-6f ? 0x1p-6f : 0.f;
  const uint32_t b = (__float_as_uint(__fadd_rn(y, low)) + chance) & 0xFFF00000u;
  return __fsub_rn(__uint_as_float(b), low);
}

// What eight values of a group are held as, and its scale
template <bool ROOT>
__device__ __forceinline__ uint2 hold(const float2 (&v)[4], const uint32_t (&chance)[kUnit],
                                      float& scale) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    top = max(max(top, __float_as_uint(v[i].x) & 0x7FFFFFFFu), __float_as_uint(v[i].y) & 0x7FFFFFFFu);
  // over the 16 threads of a group; a NaN's bits are the largest of all
  top = __reduce_max_sync(threadIdx.x & 16 ? 0xFFFF0000u : 0x0000FFFFu, top);
  scale = power_for(top);
  const float inv = scale > 0.f ? __uint_as_float((254u << 23) - __float_as_uint(scale)) : 0.f;
  float2 w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = mul2(v[i], both(inv));
    w[i].x = round_e4m3(ROOT ? y.x : fabsf(y.x), chance[2 * i]);
    w[i].y = round_e4m3(ROOT ? y.y : fabsf(y.y), chance[2 * i + 1]);
    if (ROOT) {
      if (y.x > 0.f) w[i].x = fmaxf(w[i].x, 0x1p-9f);
      if (y.y > 0.f) w[i].y = fmaxf(w[i].y, 0x1p-9f);
    } else {
      w[i] = make_float2(copysignf(w[i].x, y.x), copysignf(w[i].y, y.y));
    }
  }
  return narrow_e4m3(w);
}

// Up to eight elements from the i-th on; zeros past the tensor
template <bool EIGHT, bool BF16>
__device__ __forceinline__ void load_unit(const AdamWTensor& t, uint64_t i,
                                          Unit<EIGHT, BF16>& u) {
  if constexpr (EIGHT) {
    const bool live = i < t.numel;
    u.ms = live ? t.m_scales[i / kGroup] : 0.f;
    u.vs = live ? t.v_scales[i / kGroup] : 0.f;
  }
  if (t.vec && i + kUnit <= t.numel) {
    load_raw(t.grad, i, u.g);
    load8(t.param + i, u.p);
    if constexpr (EIGHT) {
      u.m8 = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.m) + i);
      u.v8 = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.v) + i);
    } else {
      load8(static_cast<const float*>(t.m) + i, u.m);
      load8(static_cast<const float*>(t.v) + i, u.v);
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < Raw<BF16>::kWords; ++e) u.g.w[e] = 0u;
  uint32_t q[2][2] = {};
#pragma unroll
  for (int e = 0; e < kUnit; ++e) {
    const bool live = i + e < t.numel;
    if constexpr (BF16)
      u.g.w[e / 2] |= (live ? static_cast<const uint16_t*>(t.grad)[i + e] : 0u) << (16 * (e % 2));
    else
      u.g.w[e] = live ? static_cast<const uint32_t*>(t.grad)[i + e] : 0u;
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
    u.m8 = make_uint2(q[0][0], q[0][1]);
    u.v8 = make_uint2(q[1][0], q[1][1]);
  }
}

template <bool EIGHT, bool BF16>
__device__ __forceinline__ void store_unit(const AdamWTensor& t, uint64_t i,
                                           const Unit<EIGHT, BF16>& u) {
  if constexpr (EIGHT) {
    if (threadIdx.x % kLanes == 0 && i < t.numel) {
      t.m_scales[i / kGroup] = u.ms;
      t.v_scales[i / kGroup] = u.vs;
    }
  }
  if (t.vec && i + kUnit <= t.numel) {
    store8(t.param + i, u.p);
    if (t.copy) store8(t.copy + i, u.p);
    if constexpr (EIGHT) {
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.m) + i) = u.m8;
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.v) + i) = u.v8;
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
      static_cast<uint8_t*>(t.m)[i + e] = (uint8_t)((e < 4 ? u.m8.x : u.m8.y) >> (8 * (e % 4)));
      static_cast<uint8_t*>(t.v)[i + e] = (uint8_t)((e < 4 ? u.v8.x : u.v8.y) >> (8 * (e % 4)));
    } else {
      static_cast<float*>(t.m)[i + e] = u.m[e];
      static_cast<float*>(t.v)[i + e] = u.v[e];
    }
  }
}

// fp32 states: every operation rounded, as rcc_grad_sync_adamw's update
template <bool BF16>
__device__ __forceinline__ void update_unit(const AdamWArgs& a, const AdamWDecision& d,
                                            uint32_t, Unit<false, BF16>& u) {
#pragma unroll
  for (int e = 0; e < kUnit; ++e) {
    const float2 two = pair_of(u.g, e / 2);
    const float g = __fmul_rn(__fmul_rn(e % 2 ? two.y : two.x, a.inv_scale), d.coef);
    const float m = __fadd_rn(__fmul_rn(a.b1, u.m[e]), __fmul_rn(a.one_minus_b1, g));
    const float v = __fadd_rn(__fmul_rn(a.b2, u.v[e]), __fmul_rn(a.one_minus_b2, __fmul_rn(g, g)));
    const float denom = __fadd_rn(__fmul_rn(__fsqrt_rn(v), d.inv_root), a.eps);
    u.p[e] = __fsub_rn(__fmul_rn(u.p[e], a.decay), __fmul_rn(d.step_size, __fdiv_rn(m, denom)));
    u.m[e] = m;
    u.v[e] = v;
  }
}

__device__ __forceinline__ float root_of(float v) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float inverse_of(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// 8-bit states: two elements an operation, products fused into sums, root and
// quotient to 2^-22: what is held keeps four bits of it.
template <bool BF16>
__device__ __forceinline__ void update_unit(const AdamWArgs& a, const AdamWDecision& d,
                                            uint32_t first, Unit<true, BF16>& u) {
  float2 m[4], v[4];
  widen_e4m3(u.m8, m);
  widen_e4m3(u.v8, v);
  uint32_t chance[kUnit];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 g = mul2(pair_of(u.g, i), both(d.factor));
    m[i] = fma2(m[i], both(u.ms * a.b1), mul2(g, both(a.one_minus_b1)));
    const float2 root = mul2(v[i], both(u.vs));
    v[i] = fma2(mul2(root, root), both(a.b2), mul2(mul2(g, g), both(a.one_minus_b2)));
    v[i] = make_float2(root_of(v[i].x), root_of(v[i].y));
    const float2 denom = fma2(v[i], both(d.inv_root), both(a.eps));
    const float2 change = mul2(m[i], make_float2(inverse_of(denom.x), inverse_of(denom.y)));
    const float2 p = fma2(change, both(-d.step_size),
                          mul2(make_float2(u.p[2 * i], u.p[2 * i + 1]), both(a.decay)));
    u.p[2 * i] = p.x;
    u.p[2 * i + 1] = p.y;
    const uint32_t h = mix(first + i);
    chance[2 * i] = (h & 0xFFFFu) << 4;
    chance[2 * i + 1] = h >> 16 << 4;
  }
  u.m8 = hold<false>(m, chance, u.ms);
  u.v8 = hold<true>(v, chance, u.vs);
}

template <bool EIGHT, bool BF16>
__device__ __forceinline__ void update_item(const AdamWArgs& a, const AdamWDecision& d,
                                            const AdamWTensor& t, uint32_t chunk, uint32_t key) {
  const uint64_t i = (uint64_t)chunk * kAdamWItem + threadIdx.x * kUnit;
#pragma unroll 1
  for (int k0 = 0; k0 < kUnits; k0 += UPD_AHEAD) {
    Unit<EIGHT, BF16> u[UPD_AHEAD];
#pragma unroll
    for (int k = 0; k < UPD_AHEAD; ++k) load_unit(t, i + (k0 + k) * kThreads * kUnit, u[k]);
#pragma unroll
    for (int k = 0; k < UPD_AHEAD; ++k) {
      update_unit(a, d, key + ((k0 + k) * kThreads + threadIdx.x) * (kUnit / 2), u[k]);
      store_unit(t, i + (k0 + k) * kThreads * kUnit, u[k]);
    }
  }
}

template <bool EIGHT>
__global__ void __launch_bounds__(kThreads, UPD_PER_SM) adamw_update_kernel(const AdamWArgs a) {
  __shared__ AdamWTensor t;
  pdl_wait_then_release();
  const AdamWDecision d = *a.decision;
  if (d.skip) return;
  uint64_t lo, hi;
  range_of(a.num_items, lo, hi);
  const uint32_t step_key = mix(a.seed ^ mix(d.step));
  AdamWItem next = a.items[hi - 1];
  uint32_t tensor = ~0u;
  for (uint64_t item = hi; item-- > lo;) {
    const AdamWItem it = next;
    if (item > lo) next = a.items[item - 1];
    if (it.tensor != tensor) {
      __syncthreads();
      tensor = it.tensor;
      if (threadIdx.x < sizeof(AdamWTensor) / 8)
        reinterpret_cast<uint64_t*>(&t)[threadIdx.x] =
            reinterpret_cast<const uint64_t*>(a.tensors + tensor)[threadIdx.x];
      __syncthreads();
    }
    const uint32_t key = mix(mix(step_key + tensor * kGolden) ^ it.chunk);
    if (t.bf16)
      update_item<EIGHT, true>(a, d, t, it.chunk, key);
    else
      update_item<EIGHT, false>(a, d, t, it.chunk, key);
  }
}

}  // namespace

cudaError_t launch_adamw(const AdamWArgs& a, bool eight, cudaStream_t stream,
                         uint64_t* launches) {
  // every SM full once, ranges of items as long as that makes them
  auto blocks_for = [&](int per_sm) {
    const uint64_t fill = (uint64_t)a.sms * per_sm;
    return dim3((unsigned)(a.num_items < fill ? a.num_items : fill));
  };
  cudaError_t e = launch_kernel(adamw_norm_kernel, blocks_for(NORM_PER_SM), dim3(kThreads), 0, stream, a);
  if (e != cudaSuccess) return e;
  e = launch_kernel(eight ? adamw_update_kernel<true> : adamw_update_kernel<false>,
                    blocks_for(UPD_PER_SM), dim3(kThreads), 0, stream, a);
  if (e == cudaSuccess) *launches = 2;
  return e;
}

int adamw_sms() { return sm_count(); }
int adamw_rows(int sms) { return sms * NORM_PER_SM; }

}  // namespace lm
}  // namespace rcc
