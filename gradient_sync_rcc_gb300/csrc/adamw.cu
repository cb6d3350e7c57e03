// adamw.cu -- AdamW over many tensors, its states in fp32 or in 8 bits.
//
//   g = grad (1/scale) coef,  coef = max_grad_norm / |g| where that is less than 1
//   m = b1 m + (1-b1) g;  v = b2 v + (1-b2) g^2
//   p = p (1 - lr wd) - lr/(1-b1^t) m / (sqrt(v) / sqrt(1-b2^t) + eps)
// Every operation is rounded to fp32, in the order of rcc_grad_sync_adamw's, whose
// bits these are with fp32 states.
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
// by memory: a block takes a range of neighbouring items (2,048 elements of a
// tensor), the update from its end, where the gradients are still in L2.
#include "lm_common.cuh"
#include "lm_internal.h"
#include "rounded.cuh"

namespace rcc {
namespace lm {
namespace {

constexpr int kThreads = 256;
constexpr int kUnit = 8;                 // elements of a thread in an item
constexpr int kGroup = 128;              // elements that share a scale
constexpr int kLanes = kGroup / kUnit;   // threads that share one
constexpr int kNumbered = 4096;          // elements whose rounding numbers share a key
constexpr uint32_t kGolden = 0x9E3779B9u;            // the golden ratio's fraction
constexpr uint32_t kRootTwo = 0x6A09E667u, kRootThree = 0xBB67AE85u;  // the roots' fractions
constexpr uint32_t kNothingBits = 27u << 23;  // 2^-100: a group below it is held as zeros

// Blocks that an SM holds, of each kernel, vectors of eight fp32 gradients that a
// thread of the norm has under way (bf16: twice as many), stages of the 8-bit
// update.  A step of 544 M elements of 1,024 tensors, bf16 gradients, in 8-bit
// states: 1,748 us (102 M in one tensor, fp32 gradients: 369).  With three blocks of
// the norm 16 us more, with eight of 32 registers 34.  Update: two stages 1,777 (376),
// four 1,752 (403); two blocks of four stages 1,822 (386), four blocks of two 1,834
// (380).  With fused arithmetic, 1,562: loaded by its threads instead of copied ahead
// 190 us more, with a block barrier for each stage 290.
constexpr int kNormPerSm = 4, kNormAhead = 2, kUpdatePerSm = 4;
constexpr int kEightPerSm = 3, kStages = 3;

static_assert(kAdamWItem == kThreads * kUnit && kNumbered % kAdamWItem == 0 && kLanes == 16,
              "whole units and groups");

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

// A thread's sum of squares without GB300's few fp64 units, as a value and the error
// it has run up, two of each: sum' = fl(sum + g^2) is one fused operation, and what it
// dropped is exact but for 2 u^2 of the sum (u = 2^-24).  Seven instructions for two
// elements.
// The errors themselves are added in fp32: i of them come to i u of the sum at most,
// so n squares are good to (n^2 / 6 + 2 n) u^2 of their sum.  So after kFold of them
// sum and error go into a second pair in the same manner, and that one after kFolds
// times into fp64: 235 u^2 and 149 u^2, 2^-40.4 of the norm together.
// (bf16 gradients, 544 M elements, a step in 8-bit states: 1,773 us; 1,753 without the
// second pair and fp64, 1,859 with fp64 alone, after 32 squares.)
constexpr int kFold = 32, kFolds = 8;
struct Squares {
  float2 sum = both(0.f), rest = both(0.f);
  float2 high = both(0.f), low = both(0.f);
  double settled = 0.0;
  int added = 0, folded = 0;
  bool more = false;  // than sum and rest (a few elements: 9.3 us a step, 10.1 without)
  uint32_t seen = 0;  // bits of the elements but their signs
  __device__ __forceinline__ void add(float2 g) {
    const float2 t = fma2(g, g, sum);
    const float2 d = add2(t, neg(sum));  // near g^2
    const float2 of_sum = add2(sum, neg(add2(t, neg(d))));
    rest = add2(rest, add2(of_sum, fma2(g, g, neg(d))));
    sum = t;
  }
  // In front of n more of each
  __device__ __forceinline__ void room(int n) {
    if (added + n > kFold) {
      fold();
      added = 0;
    }
    added += n;
  }
  __device__ __forceinline__ void fold() {
    const float2 t = add2(high, sum);
    const float2 d = add2(t, neg(high));
    const float2 error = add2(add2(high, neg(add2(t, neg(d)))), add2(sum, neg(d)));
    low = add2(low, add2(error, rest));
    high = t;
    sum = rest = both(0.f);
    more = true;
    if (++folded == kFolds) {
      settled += wide(high, low);
      high = low = both(0.f);
      folded = 0;
    }
  }
  static __device__ __forceinline__ float2 neg(float2 v) { return make_float2(-v.x, -v.y); }
  static __device__ __forceinline__ double wide(float2 value, float2 error) {
    return ((double)value.x + (double)error.x) + ((double)value.y + (double)error.y);
  }
  // Neither overflown nor among the smallest numbers, where errors are lost
  __device__ __forceinline__ bool sound() const {
    float s = sum.x + sum.y;
    if (more) s += (high.x + high.y) + (float)settled;
    return seen == 0 || (s > 0x1p-60f && s < 0x1p100f);
  }
  __device__ __forceinline__ double value() const {
    const double s = wide(sum, rest);
    return more ? s + (settled + wide(high, low)) : s;
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

// Eight fp32 values, on a boundary of 32 bytes (wide) or 16
__device__ __forceinline__ void load_eight(const float* p, bool wide, float (&v)[kUnit]) {
  if (wide) {
    load8(p, v);
    return;
  }
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x;
  v[1] = a.y;
  v[2] = a.z;
  v[3] = a.w;
  v[4] = b.x;
  v[5] = b.y;
  v[6] = b.z;
  v[7] = b.w;
}
__device__ __forceinline__ void store_eight(float* p, bool wide, const float (&v)[kUnit]) {
  if (wide) {
    store8(p, v);
    return;
  }
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// Eight gradients as they lie in memory
template <bool BF16>
struct Raw {
  static constexpr int kWords = BF16 ? 4 : 8;
  uint32_t w[kWords];
};
template <bool BF16>
__device__ __forceinline__ void set_words(Raw<BF16>& r, int at, const uint4& v) {
  r.w[at] = v.x;
  r.w[at + 1] = v.y;
  r.w[at + 2] = v.z;
  r.w[at + 3] = v.w;
}
__device__ __forceinline__ void set_wide(Raw<false>& r, const uint4& v) {  // of bf16
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.w[2 * i] = w[i] << 16;
    r.w[2 * i + 1] = w[i] & 0xFFFF0000u;
  }
}
__device__ __forceinline__ void load_raw(const void* grad, uint64_t i, bool, Raw<true>& r) {
  set_words(r, 0, *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(grad) + i));
}
__device__ __forceinline__ void load_raw(const void* grad, uint64_t i, bool wide, Raw<false>& r) {
  float f[8];
  load_eight(static_cast<const float*>(grad) + i, wide, f);
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
__device__ __forceinline__ void add_vectors(const void* grad, bool wide, uint64_t begin,
                                            uint64_t vectors, Squares& s) {
  constexpr int kAhead = BF16 ? 2 * kNormAhead : kNormAhead;  // vectors of a thread under way
  for (uint64_t v = threadIdx.x; v < vectors; v += kAhead * kThreads) {
    Raw<BF16> r[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
#pragma unroll
      for (int e = 0; e < Raw<BF16>::kWords; ++e) r[k].w[e] = 0u;
      if (v + k * kThreads < vectors) load_raw(grad, begin + (v + k * kThreads) * kUnit, wide, r[k]);
    }
    s.room(kAhead * kUnit / 2);
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
      add_vectors<true>(t.grad, true, begin, vectors, s);
    else
      add_vectors<false>(t.grad, t.wide, begin, vectors, s);
    from = begin + vectors * kUnit;
  }
  for (uint64_t i = from + threadIdx.x; i < end; i += 8 * kThreads) {
    float g[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) g[k] = i + k * kThreads < end ? grad_at(t, i + k * kThreads) : 0.f;
    s.room(4);
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      s.seen |= (__float_as_uint(g[k]) | __float_as_uint(g[k + 1])) & 0x7FFFFFFFu;
      s.add(make_float2(g[k], g[k + 1]));
    }
  }
}

// Where a block's items begin.  The tables do not change between steps, so they
// are read before the kernel ahead is through.
struct Start {
  uint64_t items;
  AdamWItem item;
  AdamWTensor tensor;
};
__device__ __forceinline__ Start start_of(const AdamWArgs& a) {
  Start s;
  uint64_t lo, hi;
  range_of(a.num_items, lo, hi);
  s.items = hi - lo;
  s.item = a.items[lo];
  s.tensor = a.tensors[s.item.tensor];
  return s;
}
// The tensors' pieces within the block's items, one after the other
template <typename F>
__device__ __forceinline__ void for_each_range(const AdamWArgs& a, const Start& s, F f) {
  AdamWItem it = s.item;
  AdamWTensor t = s.tensor;
  for (uint64_t items = s.items;;) {
    const uint64_t begin = (uint64_t)it.chunk * kAdamWItem;
    const uint64_t left = (t.numel - begin + kAdamWItem - 1) / kAdamWItem;  // items of the tensor
    const uint64_t take = min(left, items);
    f(t, begin, min(begin + take * kAdamWItem, t.numel));
    items -= take;
    if (items == 0) return;
    it = {it.tensor + 1, 0};
    t = a.tensors[it.tensor];
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
  if (threadIdx.x < kThreads / 32) {
    sum = sums[threadIdx.x];
    bad = bads[threadIdx.x];
#pragma unroll
    for (int o = kThreads / 64; o > 0; o >>= 1) {
      sum += __shfl_xor_sync((1u << kThreads / 32) - 1, sum, o);
      bad += __shfl_xor_sync((1u << kThreads / 32) - 1, bad, o);
    }
  }
}

// What the step would be, from the status before it: one thread, once a step
struct Powers {
  double beta1, beta2;
  float step_size, inv_root;
  int64_t step;
};
__device__ __forceinline__ Powers powers_of(const AdamWArgs& a) {
  Powers p;
  p.step = a.status->step;
  p.beta1 = a.status->beta1_power * a.beta1;
  p.beta2 = a.status->beta2_power * a.beta2;
  p.step_size = (float)(a.lr / (1.0 - p.beta1));
  p.inv_root = (float)(1.0 / sqrt(1.0 - p.beta2));
  return p;
}

// Whether and how it is taken
__device__ __forceinline__ void decide(const AdamWArgs& a, const Powers& p, double sum,
                                       unsigned long long bad) {
  const double norm = sqrt(sum) * a.inv_scale64;
  AdamWDecision d;
  d.skip = bad > 0 || !(norm < INFINITY);
  const double coef = !d.skip && a.max_norm > 0.0 && norm > a.max_norm ? a.max_norm / norm : 1.0;
  d.coef = (float)coef;
  d.step = (uint32_t)p.step;
  d.step_size = p.step_size;
  d.inv_root = p.inv_root;
  *a.decision = d;
  a.status->grad_norm = norm;
  a.status->nonfinite = bad > 0xFFFFFFFFull ? 0xFFFFFFFFu : (uint32_t)bad;
  a.status->skipped = d.skip;
  a.status->clip_coef = d.coef;
  if (d.skip) return;
  a.status->step = p.step + 1;
  a.status->beta1_power = p.beta1;
  a.status->beta2_power = p.beta2;
}

// Whether the block is the last to arrive: its writes before are there for the
// last one to read
__device__ __forceinline__ bool arrive_last(uint32_t* arrived) {
  uint32_t before;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(arrived)
               : "memory");
  return before == gridDim.x - 1;
}

// Each block leaves one row; the last one to do so adds them up, in the rows'
// order, and decides.
__global__ void __launch_bounds__(kThreads, kNormPerSm) adamw_norm_kernel(const AdamWArgs a) {
  __shared__ double sums[kThreads / 32];
  __shared__ unsigned long long bads[kThreads / 32];
  __shared__ Powers powers;
  __shared__ bool last;
  const Start start = start_of(a);
  pdl_wait_then_release();
  Squares s;
  for_each_range(a, start, [&](const AdamWTensor& t, uint64_t begin, uint64_t end) {
    add_range(t, begin, end, s);
  });
  double sum = s.value();
  unsigned long long bad = 0;
  if (!s.sound()) {
    WideSquares w;
    for_each_range(a, start_of(a), [&](const AdamWTensor& t, uint64_t begin, uint64_t end) {
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
    last = arrive_last(a.arrived);
  }
  __syncthreads();
  if (!last) return;
  if (threadIdx.x == kThreads - 1) powers = powers_of(a);  // beside the sum
  sum = 0.0;
  bad = 0;
  for (uint32_t r = threadIdx.x; r < gridDim.x; r += kThreads) {
    sum += __ldcg(&a.rows[r].sum);
    bad += __ldcg(&a.rows[r].bad);
  }
  block_sum(sum, bad, sums, bads);
  if (threadIdx.x == 0) {
    *a.arrived = 0;
    decide(a, powers, sum, bad);
  }
}

// ---- the update -----------------------------------------------------------------

// Eight elements as they lie in memory, and the scales of the first and the last
// four: neighbours, of one group; or (buffers on no boundary, the end of a tensor)
// every 32nd of the warp's 256, so that a warp's accesses lie side by side and its
// two groups are the first and the last four of all lanes.  100 M elements one
// element off their boundaries, fp32 gradients: fp32 states 558 us a step (506 on
// them; 1,362 as neighbours, element by element), 8-bit states 677 (360).
template <bool EIGHT, bool BF16>
struct Unit {
  Raw<BF16> g;
  float p[kUnit];
  float m[EIGHT ? 1 : kUnit], v[EIGHT ? 1 : kUnit];
  uint2 m8, v8;
  float ms[2], vs[2];
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

// y >= 0 on the grid of e4m3, up with a chance of its distance over a step:
// `number` of 2^20, in steps of 16.  Below 2^-6 the grid is even, as it is from 2^-6
// to 2^-5.  Over 448 is left to the conversion, which saturates.
__device__ __forceinline__ float round_e4m3(float y, uint32_t number) {
  const float low = y < 0x1p-6f ? 0x1p-6f : 0.f;
  const uint32_t b = (__float_as_uint(__fadd_rn(y, low)) + number) & 0xFFF00000u;
  return __fsub_rn(__uint_as_float(b), low);
}

// The scale s of a group by the bits of its largest value: the smallest power of
// two with max <= 448 s.  448 is 1.75 2^8, so a fraction above 0.75 carries into
// the exponent.  0 for next to nothing, NaN for a NaN.  `inv`: 1 / s, or 0.
__device__ __forceinline__ float scale_for(uint32_t top, float& inv) {
  const uint32_t s = ((min(top, 0x7F7FFFFFu) + 0x1FFFFFu) & 0x7F800000u) - (8u << 23);
  const bool some = top >= kNothingBits;
  inv = some ? __uint_as_float((254u << 23) - s) : 0.f;
  return some ? __uint_as_float(top > 0x7F800000u ? top : s) : 0.f;
}

// The bits of the largest of a thread's values (ROOT: none is negative), of each group
template <bool ROOT, bool STRIDED>
__device__ __forceinline__ void top_of(const float2 (&v)[4], uint32_t (&top)[2]) {
#pragma unroll
  for (int half = 0; half < (STRIDED ? 2 : 1); ++half) {
    top[half] = 0;
#pragma unroll
    for (int i = 2 * half; i < (STRIDED ? 2 * half + 2 : 4); ++i) {
      const uint32_t x = __float_as_uint(v[i].x), y = __float_as_uint(v[i].y);
      top[half] = ROOT ? max(max(top[half], x), y) : max(max(top[half], x << 1), y << 1);
    }
    if (!ROOT) top[half] >>= 1;
  }
}

// What eight values are held as, and their scales.  `top`: of the thread's values.
// `number`: of two elements each, 16 bits of them.
template <bool ROOT, bool STRIDED>
__device__ __forceinline__ uint2 hold(const float2 (&v)[4], const uint32_t (&top)[2],
                                      const uint32_t (&number)[4], float (&scale)[2]) {
  float inv[2];
#pragma unroll
  for (int half = 0; half < (STRIDED ? 2 : 1); ++half) {
    // over the threads of the group; a NaN's bits are the largest of all
    const uint32_t lanes = STRIDED ? 0xFFFFFFFFu : threadIdx.x & 16 ? 0xFFFF0000u : 0x0000FFFFu;
    scale[half] = scale_for(__reduce_max_sync(lanes, top[half]), inv[half]);
  }
  float2 w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = mul2(v[i], both(inv[STRIDED ? i / 2 : 0]));
    w[i].x = round_e4m3(ROOT ? y.x : fabsf(y.x), number[i] << 4 & 0xFFFF0u);
    w[i].y = round_e4m3(ROOT ? y.y : fabsf(y.y), number[i] >> 12 & 0xFFFF0u);
    if (ROOT) {
      if (y.x > 0.f) w[i].x = fmaxf(w[i].x, 0x1p-9f);
      if (y.y > 0.f) w[i].y = fmaxf(w[i].y, 0x1p-9f);
    } else {
      w[i] = make_float2(copysignf(w[i].x, y.x), copysignf(w[i].y, y.y));
    }
  }
  return narrow_e4m3(w);
}

// Whether the warp's 256 elements from the i-th on are loaded in vectors
__device__ __forceinline__ bool vectors(const AdamWTensor& t, uint64_t warp_first) {
  return t.vec && warp_first + 32 * kUnit <= t.numel;
}
__device__ __forceinline__ uint64_t warp_first(uint64_t item_first) {
  return item_first + threadIdx.x / 32 * 32 * kUnit;
}
// The first of a thread's neighbours, and the first of its strided elements
__device__ __forceinline__ uint64_t neighbours(uint64_t warp) {
  return warp + threadIdx.x % 32 * kUnit;
}
__device__ __forceinline__ uint64_t strided(uint64_t warp) { return warp + threadIdx.x % 32; }

template <bool EIGHT, bool BF16>
__device__ __forceinline__ void load_vectors(const AdamWTensor& t, uint64_t warp,
                                             Unit<EIGHT, BF16>& u) {
  const uint64_t i = neighbours(warp);
  if constexpr (BF16) {
    load_raw(t.grad, i, t.wide, u.g);
  } else if (t.bf16) {
    set_wide(u.g, *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(t.grad) + i));
  } else {
    load_raw(t.grad, i, t.wide, u.g);
  }
  load_eight(t.param + i, t.wide, u.p);
  if constexpr (EIGHT) {
    u.m8 = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.m) + i);
    u.v8 = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.v) + i);
    u.ms[0] = t.m_scales[i / kGroup];
    u.vs[0] = t.v_scales[i / kGroup];
  } else {
    load_eight(static_cast<const float*>(t.m) + i, t.wide, u.m);
    load_eight(static_cast<const float*>(t.v) + i, t.wide, u.v);
  }
}

// Elements past the tensor are zeros
template <bool EIGHT, bool BF16>
__device__ __forceinline__ void load_strided(const AdamWTensor& t, uint64_t warp,
                                             Unit<EIGHT, BF16>& u) {
#pragma unroll
  for (int e = 0; e < Raw<BF16>::kWords; ++e) u.g.w[e] = 0u;
  uint32_t q[2][2] = {};
#pragma unroll
  for (int e = 0; e < kUnit; ++e) {
    const uint64_t i = strided(warp) + 32 * e;
    const bool live = i < t.numel;
    if constexpr (BF16)
      u.g.w[e / 2] |= (live ? static_cast<const uint16_t*>(t.grad)[i] : 0u) << (16 * (e % 2));
    else
      u.g.w[e] = live ? __float_as_uint(grad_at(t, i)) : 0u;
    u.p[e] = live ? t.param[i] : 0.f;
    if constexpr (EIGHT) {
      q[0][e / 4] |= (live ? static_cast<const uint8_t*>(t.m)[i] : 0u) << (8 * (e % 4));
      q[1][e / 4] |= (live ? static_cast<const uint8_t*>(t.v)[i] : 0u) << (8 * (e % 4));
    } else {
      u.m[e] = live ? static_cast<const float*>(t.m)[i] : 0.f;
      u.v[e] = live ? static_cast<const float*>(t.v)[i] : 0.f;
    }
  }
  if constexpr (EIGHT) {
    u.m8 = make_uint2(q[0][0], q[0][1]);
    u.v8 = make_uint2(q[1][0], q[1][1]);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint64_t at = warp + half * kGroup;
      u.ms[half] = at < t.numel ? t.m_scales[at / kGroup] : 0.f;
      u.vs[half] = at < t.numel ? t.v_scales[at / kGroup] : 0.f;
    }
  }
}

template <bool EIGHT, bool BF16>
__device__ __forceinline__ void store_vectors(const AdamWTensor& t, uint64_t warp,
                                              const Unit<EIGHT, BF16>& u) {
  const uint64_t i = neighbours(warp);
  store_eight(t.param + i, t.wide, u.p);
  if (t.copy) store8(t.copy + i, u.p);
  if constexpr (EIGHT) {
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.m) + i) = u.m8;
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.v) + i) = u.v8;
    if (threadIdx.x % kLanes == 0) {
      t.m_scales[i / kGroup] = u.ms[0];
      t.v_scales[i / kGroup] = u.vs[0];
    }
  } else {
    store_eight(static_cast<float*>(t.m) + i, t.wide, u.m);
    store_eight(static_cast<float*>(t.v) + i, t.wide, u.v);
  }
}

template <bool EIGHT, bool BF16>
__device__ __forceinline__ void store_strided(const AdamWTensor& t, uint64_t warp,
                                              const Unit<EIGHT, BF16>& u) {
#pragma unroll
  for (int e = 0; e < kUnit; ++e) {
    const uint64_t i = strided(warp) + 32 * e;
    if (i >= t.numel) continue;
    t.param[i] = u.p[e];
    if (t.copy) from_f32(u.p[e], t.copy[i]);
    if constexpr (EIGHT) {
      static_cast<uint8_t*>(t.m)[i] = (uint8_t)((e < 4 ? u.m8.x : u.m8.y) >> (8 * (e % 4)));
      static_cast<uint8_t*>(t.v)[i] = (uint8_t)((e < 4 ? u.v8.x : u.v8.y) >> (8 * (e % 4)));
    } else {
      static_cast<float*>(t.m)[i] = u.m[e];
      static_cast<float*>(t.v)[i] = u.v[e];
    }
  }
  if constexpr (EIGHT) {
    const int half = threadIdx.x % 32;  // lane 0 the first group's, lane 1 the second's
    const uint64_t at = warp + half * kGroup;
    if (half < 2 && at < t.numel) {
      t.m_scales[at / kGroup] = half ? u.ms[1] : u.ms[0];
      t.v_scales[at / kGroup] = half ? u.vs[1] : u.vs[0];
    }
  }
}

// fp32 states: every operation rounded, as rcc_grad_sync_adamw's update
template <bool BF16>
__device__ __forceinline__ void update_unit(const AdamWArgs& a, const AdamWDecision& d,
                                            Unit<false, BF16>& u) {
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

// Whether denominators are in quotient2's range for all v <= kMostSquare (sqrt(v) <=
// 2^15), and the step size over 2^64 is exact.  Else, and for larger v and m, CUDA's
// rounded operations one by one: 544 M elements 1,742 us, with an eps of 1e-20 2,939.
__device__ __forceinline__ bool in_range(const AdamWArgs& a, const AdamWDecision& d) {
  return a.eps >= kLeastBelow && a.eps <= 1.f && d.inv_root <= 0x1p8f &&
         (d.step_size >= 0x1p-62f || d.step_size == 0.f);
}

// 8-bit states: what they stand for (value times scale; a root's square is v), then
// the same operations, each rounded, two elements at a time.  So the bytes are the
// definition's, step after step: a value that one last place moves across its
// rounding number is held a whole step of the grid off, and its parameter goes
// another way from there on.  (Products fused into sums and roots to 2^-22: 1,562 us
// where this took 1,754, 450 of 544 M values off after one step, and after twelve
// parameters by 0.1 of their root mean square.)
// `key`: of the rounding numbers of the block of kNumbered elements, `first`: the
// thread's first element in it.  `usual`: in_range.
template <bool STRIDED, bool BF16>
__device__ __forceinline__ void update_unit(const AdamWArgs& a, const AdamWDecision& d,
                                            uint32_t key, uint32_t first, bool usual,
                                            Unit<true, BF16>& u) {
  float2 m[4], v[4];
  widen_e4m3(u.m8, m);
  widen_e4m3(u.v8, v);
  uint32_t most_square = 0;  // of v, its bits
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 g = mul2(mul2(pair_of(u.g, i), both(a.inv_scale)), both(d.coef));
    constexpr int kHalf = STRIDED ? 2 : 4;  // pairs of one scale
    m[i] = mul2(m[i], both(u.ms[i / kHalf]));
    m[i] = sum2(mul2(m[i], both(a.b1)), mul2(g, both(a.one_minus_b1)), a.one);
    const float2 root = mul2(v[i], both(u.vs[i / kHalf]));
    v[i] = sum2(mul2(mul2(root, root), both(a.b2)), mul2(mul2(g, g), both(a.one_minus_b2)), a.one);
    most_square = max(most_square, max(__float_as_uint(v[i].x), __float_as_uint(v[i].y)));
  }
  uint32_t top[2];
  top_of<false, STRIDED>(m, top);
  const uint32_t most = STRIDED ? max(top[0], top[1]) : top[0];  // a NaN's bits are more
  if (usual && most <= __float_as_uint(kMost) && most_square <= __float_as_uint(kMostSquare)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = root2(v[i]);
      const float2 denom = sum2(mul2(v[i], both(d.inv_root)), both(a.eps), a.one);
      const float2 p = sum2(mul2(make_float2(u.p[2 * i], u.p[2 * i + 1]), both(a.decay)),
                            mul2(quotient2(m[i], denom), both(d.step_size * -0x1p-64f)), a.one);
      u.p[2 * i] = p.x;
      u.p[2 * i + 1] = p.y;
    }
  } else {  // a loop: where it is not taken, it costs no registers
    float mm[kUnit], vv[kUnit], pp[kUnit];
#pragma unroll
    for (int e = 0; e < kUnit; ++e) {
      mm[e] = e % 2 ? m[e / 2].y : m[e / 2].x;
      vv[e] = e % 2 ? v[e / 2].y : v[e / 2].x;
      pp[e] = u.p[e];
    }
#pragma unroll 1
    for (int e = 0; e < kUnit; ++e) {
      vv[e] = __fsqrt_rn(vv[e]);
      const float denom = __fadd_rn(__fmul_rn(vv[e], d.inv_root), a.eps);
      const float change = __fdiv_rn(mm[e], denom);
      pp[e] = __fsub_rn(__fmul_rn(pp[e], a.decay), __fmul_rn(d.step_size, change));
    }
#pragma unroll
    for (int e = 0; e < kUnit; ++e) {
      (e % 2 ? v[e / 2].y : v[e / 2].x) = vv[e];
      u.p[e] = pp[e];
    }
  }
  uint32_t number[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (STRIDED) {  // both elements are the first, or the second, of their two
      const uint32_t at = first + 64 * i;
      number[i] = __byte_perm(mix(key + at / 2), mix(key + at / 2 + 16),
                              at % 2 ? 0x7632 : 0x5410);
    } else {
      number[i] = mix(key + first / 2 + i);
    }
  }
  u.m8 = hold<false, STRIDED>(m, top, number, u.ms);
  top_of<true, STRIDED>(v, top);
  u.v8 = hold<true, STRIDED>(v, top, number, u.vs);
}

// fp32 states: a thread's loads are bytes enough by themselves.
template <bool BF16>
__device__ __forceinline__ void update_item(const AdamWArgs& a, const AdamWDecision& d,
                                            const AdamWTensor& t, uint32_t chunk) {
  const uint64_t warp = warp_first((uint64_t)chunk * kAdamWItem);
  Unit<false, BF16> u;
  if (vectors(t, warp)) {
    load_vectors(t, warp, u);
    update_unit(a, d, u);
    store_vectors(t, warp, u);
  } else {
    load_strided(t, warp, u);
    update_unit(a, d, u);
    store_strided(t, warp, u);
  }
}
__global__ void __launch_bounds__(kThreads, kUpdatePerSm) adamw_update_kernel(const AdamWArgs a) {
  __shared__ AdamWTensor t;
  uint64_t lo, hi;
  range_of(a.num_items, lo, hi);
  AdamWItem next = a.items[hi - 1];
  uint32_t tensor = next.tensor;
  auto load_tensor = [&] {
    if (threadIdx.x < sizeof(AdamWTensor) / 8)
      reinterpret_cast<uint64_t*>(&t)[threadIdx.x] =
          reinterpret_cast<const uint64_t*>(a.tensors + tensor)[threadIdx.x];
    __syncthreads();
  };
  load_tensor();
  pdl_wait_then_release();
  const AdamWDecision d = *a.decision;
  if (d.skip) return;
  for (uint64_t item = hi; item-- > lo;) {
    const AdamWItem it = next;
    if (item > lo) next = a.items[item - 1];
    if (it.tensor != tensor) {
      __syncthreads();
      tensor = it.tensor;
      load_tensor();
    }
    if (t.bf16)
      update_item<true>(a, d, t, it.chunk);
    else
      update_item<false>(a, d, t, it.chunk);
  }
}

// 8-bit states: half the bytes for the same threads, so what a block reads is
// copied into shared memory ahead, item by item.  One more warp does that; an
// item's stage is full when its bytes are there and empty when all other warps are
// through, which no block barrier holds together.
constexpr int kEightThreads = kThreads + 32;

struct Entry {  // an item and its tensor
  AdamWTensor t;
  AdamWItem item;
};
constexpr int kEntryWords = sizeof(Entry) / 8;

// A stage: parameters, gradients, the two states, their scales, the entry
template <bool BF16>
struct Stage {
  static constexpr int kGrad = kAdamWItem * 4, kM = kGrad + kAdamWItem * (BF16 ? 2 : 4);
  static constexpr int kV = kM + kAdamWItem, kMs = kV + kAdamWItem, kVs = kMs + kAdamWItem / kGroup * 4;
  static constexpr int kEntry = kVs + kAdamWItem / kGroup * 4;
  static constexpr int kBytes = (kEntry + (int)sizeof(Entry) + 127) / 128 * 128;
};

// `bytes` (a multiple of 16, from a boundary of 16) into shared memory
__device__ __forceinline__ void copy_bulk(uint32_t to, const void* from, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          to), "l"(from), "r"(bytes), "r"(bar) : "memory");
}

// Whether the item at `first` is whole and on boundaries that bulk copies take
__device__ __forceinline__ bool whole_item(const AdamWTensor& t, uint64_t first) {
  return t.bulk && first + kAdamWItem <= t.numel;
}

template <bool BF16>
__device__ __forceinline__ void copy_item(const AdamWTensor& t, uint64_t first, uint32_t to,
                                           uint32_t bar) {
  using S = Stage<BF16>;
  const uint32_t size = BF16 || t.bf16 ? 2 : 4;
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar),
               "r"(kAdamWItem * (4 + size + 2)) : "memory");
  copy_bulk(to, t.param + first, kAdamWItem * 4, bar);
  copy_bulk(to + S::kGrad, static_cast<const char*>(t.grad) + first * size, kAdamWItem * size, bar);
  copy_bulk(to + S::kM, static_cast<const char*>(t.m) + first, kAdamWItem, bar);
  copy_bulk(to + S::kV, static_cast<const char*>(t.v) + first, kAdamWItem, bar);
}
// The scales, which may lie anywhere: one a lane, whose arrival follows its copy
template <bool BF16>
__device__ __forceinline__ void copy_scale(const AdamWTensor& t, uint64_t first,
                                           unsigned char* stage, int lane, uint32_t bar) {
  static_assert(kAdamWItem / kGroup == 16, "a half warp each");
  const float* from = (lane < 16 ? t.m_scales : t.v_scales) + first / kGroup + lane % 16;
  copy_async<4>(stage + Stage<BF16>::kMs + lane * 4, from);
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// A thread's unit out of a stage
template <bool BF16>
__device__ __forceinline__ void take_unit(const unsigned char* stage, bool bf16,
                                          Unit<true, BF16>& u) {
  using S = Stage<BF16>;
  const int tid = threadIdx.x;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint4 q = reinterpret_cast<const uint4*>(stage)[2 * tid + h];
    u.p[4 * h] = __uint_as_float(q.x);
    u.p[4 * h + 1] = __uint_as_float(q.y);
    u.p[4 * h + 2] = __uint_as_float(q.z);
    u.p[4 * h + 3] = __uint_as_float(q.w);
  }
  const uint4* g = reinterpret_cast<const uint4*>(stage + S::kGrad);
  if constexpr (BF16) {
    set_words(u.g, 0, g[tid]);
  } else if (bf16) {
    set_wide(u.g, g[tid]);
  } else {
    set_words(u.g, 0, g[2 * tid]);
    set_words(u.g, 4, g[2 * tid + 1]);
  }
  u.m8 = reinterpret_cast<const uint2*>(stage + S::kM)[tid];
  u.v8 = reinterpret_cast<const uint2*>(stage + S::kV)[tid];
  u.ms[0] = reinterpret_cast<const float*>(stage + S::kMs)[tid / kLanes];
  u.vs[0] = reinterpret_cast<const float*>(stage + S::kVs)[tid / kLanes];
}

__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// BF16: every gradient of the plan is; else they may be mixed, and are widened where
// they are taken (1,024 tensors of 544 M elements, all bf16: 1,748 us a step, 1,775 by
// the mixed form).
template <bool BF16>
__global__ void __launch_bounds__(kEightThreads, kEightPerSm)
    adamw_update_eight_kernel(const AdamWArgs a) {
  using S = Stage<BF16>;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) uint64_t bars[2][kStages];
  const int tid = threadIdx.x;
  const uint32_t full = (uint32_t)__cvta_generic_to_shared(bars[0]), empty = full + 8 * kStages;
  const uint32_t stages = (uint32_t)__cvta_generic_to_shared(smem);
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      bar_init(full + 8 * s, 33);  // the bulk copies', and each lane's
      bar_init(empty + 8 * s, kThreads / 32);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  uint64_t lo, hi;
  range_of(a.num_items, lo, hi);
  const uint64_t items = hi - lo;  // the n-th is the one at hi - 1 - n
  int s = 0;
  uint32_t parity = 0;
  auto next = [&] {
    if (++s == kStages) {
      s = 0;
      parity ^= 1;
    }
  };
  if (tid >= kThreads) {
    const int lane = tid - kThreads;
    auto item_at = [&](uint64_t n) { return a.items[hi - 1 - min(n, items - 1)]; };
    auto entry_word = [&](const AdamWItem& it) {  // of the first kEntryWords lanes
      if (lane >= kEntryWords) return uint64_t{0};
      if (lane == kEntryWords - 1) return (uint64_t)it.chunk << 32 | it.tensor;
      return reinterpret_cast<const uint64_t*>(a.tensors + it.tensor)[lane];
    };
    // words of the next item, and the one after that (tables that do not change)
    uint64_t word = entry_word(item_at(0));
    AdamWItem far = item_at(1);
    pdl_wait_then_release();
    if (a.decision->skip) return;
    uint64_t n = 0;
    for (; n < items; ++n, next()) {
      const uint64_t word_next = entry_word(far);
      far = item_at(n + 2);
      if (n >= kStages && !bar_wait(empty + 8 * s, parity ^ 1)) break;
      unsigned char* stage = smem + s * S::kBytes;
      const Entry& e = *reinterpret_cast<const Entry*>(stage + S::kEntry);
      if (lane < kEntryWords) reinterpret_cast<uint64_t*>(stage + S::kEntry)[lane] = word;
      __syncwarp();
      const uint64_t first = (uint64_t)e.item.chunk * kAdamWItem;
      if (whole_item(e.t, first)) {
        copy_scale<BF16>(e.t, first, stage, lane, full + 8 * s);
        if (lane == 0) copy_item<BF16>(e.t, first, stages + s * S::kBytes, full + 8 * s);
      } else {
        arrive(full + 8 * s);
        if (lane == 0) arrive(full + 8 * s);
      }
      word = word_next;
    }
    if (n < items) {  // a wait ran out: the copies under way end before the block does
      if (lane == 0) a.status->skipped = -1;
      for (uint64_t m = n >= kStages ? n - kStages : 0; m < n; ++m)
        bar_wait(full + 8 * (int)(m % kStages), (uint32_t)(m / kStages) & 1);
    }
    return;
  }
  pdl_wait_then_release();
  const AdamWDecision d = *a.decision;
  if (d.skip) return;
  const bool usual = in_range(a, d);
  const uint32_t step_key = mix(a.seed ^ mix(d.step));
  for (uint64_t n = 0; n < items; ++n, next()) {
    if (!bar_wait(full + 8 * s, parity)) {
      a.status->skipped = -1;
      return;
    }
    const unsigned char* stage = smem + s * S::kBytes;
    const Entry& e = *reinterpret_cast<const Entry*>(stage + S::kEntry);
    const uint64_t first = (uint64_t)e.item.chunk * kAdamWItem, warp = warp_first(first);
    const uint32_t key =
        mix(mix(step_key + e.item.tensor * kGolden) ^ (uint32_t)(first / kNumbered));
    Unit<true, BF16> u;
    if (vectors(e.t, warp)) {
      if (whole_item(e.t, first))
        take_unit<BF16>(stage, e.t.bf16, u);
      else
        load_vectors(e.t, warp, u);
      update_unit<false>(a, d, key, (uint32_t)(neighbours(warp) % kNumbered), usual, u);
      store_vectors(e.t, warp, u);
    } else {
      load_strided(e.t, warp, u);
      update_unit<true>(a, d, key, (uint32_t)(strided(warp) % kNumbered), usual, u);
      store_strided(e.t, warp, u);
    }
    __syncwarp();
    if (tid % 32 == 0) arrive(empty + 8 * s);
  }
}

// Every SM full once, ranges of items as long as that makes them
dim3 blocks_for(const AdamWArgs& a, int per_sm) {
  const uint64_t fill = (uint64_t)a.sms * per_sm;
  return dim3((unsigned)(a.num_items < fill ? a.num_items : fill));
}

template <bool BF16>
cudaError_t launch_eight(const AdamWArgs& a, cudaStream_t stream) {
  constexpr int kShared = kStages * Stage<BF16>::kBytes;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_shared(adamw_update_eight_kernel<BF16>, kShared, allowed);
  if (e != cudaSuccess) return e;
  return launch_kernel(adamw_update_eight_kernel<BF16>, blocks_for(a, kEightPerSm),
                       dim3(kEightThreads), kShared, stream, a);
}

}  // namespace

cudaError_t launch_adamw(const AdamWArgs& a, bool eight, cudaStream_t stream,
                         uint64_t* launches) {
  cudaError_t e =
      launch_kernel(adamw_norm_kernel, blocks_for(a, kNormPerSm), dim3(kThreads), 0, stream, a);
  if (e != cudaSuccess) return e;
  if (eight) {
    e = a.all_bf16 ? launch_eight<true>(a, stream) : launch_eight<false>(a, stream);
  } else {
    e = launch_kernel(adamw_update_kernel, blocks_for(a, kUpdatePerSm), dim3(kThreads), 0, stream, a);
  }
  if (e == cudaSuccess) *launches = 2;
  return e;
}

int adamw_sms() { return sm_count(); }
int adamw_rows(int sms) { return sms * kNormPerSm; }

}  // namespace lm
}  // namespace rcc
