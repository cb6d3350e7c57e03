// rotary.cu -- rotary positions on queries and keys.
//
// A pair (a, b) of a head's columns at position p becomes
//   (a c - b s, a s + b c),  c = scale cos(2 pi p f), s = scale sin(2 pi p f)
// with its frequency f in turns a position; the inverse turns by -p f, which is
// also the gradient.  f comes as a 64-bit fraction of a turn, so that p f modulo
// 2^64 is the fraction left of the turns, exact for every position: no angle is
// reduced, and a far position is as good as a near one.  Its upper 32 bits are
// the argument of the sine and cosine (2^-25 of half a turn off as a float).
//
// Memory bound: queries and keys are read and written once, in one launch.  A
// block takes a few tokens with all their heads (or, where there are few tokens,
// some heads of one), makes their sines and cosines once, in shared memory, while
// its first loads are under way, and turns unit after unit: W pairs, two vectors
// of W elements.
#include <algorithm>

#include "lm_common.cuh"
#include "lm_internal.h"

namespace rcc {
namespace lm {
namespace {

constexpr int kThreads = 256;
// Blocks an SM, units of a block for each thread, units that a thread has under
// way (32-byte vectors: half).  16,384 tokens of 40 heads of 128 in bf16, forward
// and backward (671 MB): 104.9 us (6.4 TB/s); with four units under way and three
// blocks 106.8, four units a block 104.4, two 131.  Sines made by each thread for
// four heads instead: 177.
constexpr int kPerSm = 4, kShare = 8, kUnderWay = 2;
constexpr int kTableBytes = 32 * 1024;  // of sines and cosines, at most

// W elements as they lie in memory
template <typename T, int W>
struct Vector {
  static constexpr int kBytes = W * (int)sizeof(T);
  static constexpr int kWords = kBytes < 4 ? 1 : kBytes / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kBytes == 32) {
      asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                     "=r"(w[6]), "=r"(w[7]) : "l"(p) : "memory");
    } else if constexpr (kBytes == 16) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x;
      w[1] = v.y;
      w[2] = v.z;
      w[3] = v.w;
    } else if constexpr (kBytes == 8) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x;
      w[1] = v.y;
    } else if constexpr (kBytes == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (kBytes == 32)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
                   "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                   : "memory");
    else if constexpr (kBytes == 16)
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (kBytes == 8)
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else if constexpr (kBytes == 4)
      *reinterpret_cast<uint32_t*>(p) = w[0];
    else
      *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    return __uint_as_float(i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
  }
  __device__ __forceinline__ void set(const float (&v)[W]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = __float_as_uint(v[i]);
    } else if constexpr (W == 1) {
      w[0] = pack2(v[0], 0.f) & 0xFFFFu;
    } else {
#pragma unroll
      for (int i = 0; i < W; i += 2) w[i / 2] = pack2(v[i], v[i + 1]);
    }
  }
};

__device__ __forceinline__ uint64_t position_of(const RotaryArgs& a, size_t token) {
  int64_t p = (int64_t)token;
  if (a.positions)
    p = a.index64 ? static_cast<const int64_t*>(a.positions)[token]
                  : static_cast<const int32_t*>(a.positions)[token];
  return p < 0 ? 0 : (uint64_t)p + (uint64_t)a.offset;
}

// Cosine and sine of a token's pairs, with the scale.  The pairs of a unit lie
// a column of `units` float4 (of two pairs) apart, so that neighbouring units'
// reads fall on neighbouring banks; W of 1 has one pair in a float2.
template <int W>
__device__ __forceinline__ int table_at(int pair, int units) {
  if constexpr (W == 1) return pair;
  return ((pair % W) / 2 * units + pair / W) * 2 + pair % 2;
}

// A unit of a head, at two columns; `turned` of its pairs turn
template <typename T, int W>
struct Unit {
  Vector<T, W> x, y;
  T* out;
  int first, second;  // columns; -1: none
  int table;          // of its token and unit
  int turned;
};

template <typename T, int W, bool HALF>
__global__ void __launch_bounds__(kThreads, kPerSm) rotary_kernel(const RotaryArgs a) {
  extern __shared__ __align__(16) float2 table[];
  constexpr int kAhead = W * sizeof(T) >= 32 ? kUnderWay / 2 : kUnderWay;  // units of a thread under way
  pdl_wait_then_release();
  const int units = a.units, pairs = (int)a.pairs, dim = (int)a.head_dim;
  const int turned_units = (pairs + W - 1) / W, held = turned_units * W;  // pairs in the table
  // tokens [t0, t0 + tokens), heads [h0, h0 + heads) of the queries' and then the keys'
  const size_t t0 = (size_t)blockIdx.x * a.block_tokens;
  const int tokens = (int)min((size_t)a.block_tokens, a.tokens - t0);
  const int h0 = blockIdx.y * a.block_heads;
  const int heads = min(a.block_heads, (int)(a.q.heads + a.k.heads) - h0);
  const int all = tokens * heads * units;

  // the thread's unit, and the step to its next one
  int u = threadIdx.x % units, h = threadIdx.x / units, t = h / heads;
  h -= t * heads;
  const int du = kThreads % units, dh = kThreads / units % heads,
            dt = kThreads / units / heads;
  auto advance = [&] {
    u += du;
    h += dh;
    t += dt;
    if (u >= units) {
      u -= units;
      ++h;
    }
    if (h >= heads) {
      h -= heads;
      ++t;
    }
  };
  auto begin = [&](Unit<T, W>& w) {
    const int head = h0 + h;
    const bool key = head >= (int)a.q.heads;
    const RotaryRows& r = key ? a.k : a.q;
    const size_t at = key ? head - (int)a.q.heads : head;
    const T* in = static_cast<const T*>(r.in) + (t0 + t) * r.in_token + at * r.in_head;
    w.out = static_cast<T*>(r.out) + (t0 + t) * r.out_token + at * r.out_head;
    w.turned = min(W, pairs - u * W);
    w.table = t * held + (W == 1 ? u : 2 * u);
    if (HALF) {
      w.first = w.turned > 0 ? u * W : 2 * pairs + (u - turned_units) * 2 * W;
      w.second = w.turned > 0 ? w.first + pairs : w.first + W;
    } else {
      w.first = u * 2 * W;
      w.second = w.first + W;
    }
    w.x.load(in + w.first);
    if (w.second < dim) w.y.load(in + w.second);
  };
  auto finish = [&](Unit<T, W>& w) {
    if (w.turned > 0) {
      float c[W], s[W];
      if constexpr (W == 1) {
        c[0] = table[w.table].x;
        s[0] = table[w.table].y;
      } else {
#pragma unroll
        for (int e = 0; e < W; e += 2) {
          const float4 f = *reinterpret_cast<const float4*>(&table[w.table + e * turned_units]);
          c[e] = f.x;
          s[e] = f.y;
          c[e + 1] = f.z;
          s[e + 1] = f.w;
        }
      }
      float x[W], y[W];
      if constexpr (HALF) {
#pragma unroll
        for (int e = 0; e < W; ++e) {
          const float p = w.x.get(e), q = w.y.get(e);
          x[e] = p * c[e] - q * s[e];
          y[e] = p * s[e] + q * c[e];
        }
      } else {  // x and y are neighbours; their pairs past the last stay
#pragma unroll
        for (int e = 0; e < W; ++e) {
          const int i = 2 * e % W, j = (2 * e + 1) % W;
          const bool lower = 2 * e < W, low_j = 2 * e + 1 < W;
          const float p = lower ? w.x.get(i) : w.y.get(i), q = low_j ? w.x.get(j) : w.y.get(j);
          const float up = e < w.turned ? p * c[e] - q * s[e] : p;
          const float uq = e < w.turned ? p * s[e] + q * c[e] : q;
          if (lower) x[i] = up;
          else y[i] = up;
          if (low_j) x[j] = uq;
          else y[j] = uq;
        }
      }
      w.x.set(x);
      w.y.set(y);
    }
    w.x.store(w.out + w.first);
    if (w.second < dim) w.y.store(w.out + w.second);
  };

  bool made = false;
  for (int n = threadIdx.x; n - (int)threadIdx.x < all; n += kAhead * kThreads) {
    Unit<T, W> w[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (n + k * kThreads < all) begin(w[k]);
      advance();
    }
    if (!made) {
      for (int i = threadIdx.x; i < tokens * held; i += kThreads) {
        const int token = i / held, pair = i - token * held;
        float s = 0.f, c = 1.f;
        if (pair < pairs) {
          // half turns in [-1, 1)
          const uint64_t left = position_of(a, t0 + token) * a.turns[pair];
          sincospif((float)(int32_t)(left >> 32) * 0x1p-31f, &s, &c);
        }
        table[token * held + table_at<W>(pair, turned_units)] =
            make_float2(a.scale * c, a.inverse ? -a.scale * s : a.scale * s);
      }
      __syncthreads();
      made = true;
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (n + k * kThreads < all) finish(w[k]);
  }
}

// A block has one unit for each thread where that is what fills the card, up to
// kShare where there are enough.
template <typename T, int W, bool HALF>
cudaError_t launch_of(RotaryArgs& a, cudaStream_t stream) {
  const size_t heads = a.q.heads + a.k.heads, pairs = a.pairs;
  const size_t turned = (pairs + W - 1) / W, rest = a.head_dim - 2 * pairs;
  a.units = (int)(!a.copies ? turned
                  : HALF    ? turned + (rest + 2 * W - 1) / (2 * W)
                            : (a.head_dim + 2 * W - 1) / (2 * W));
  const size_t per_token = heads * a.units;
  const size_t want = std::min<size_t>(
      kShare * kThreads, std::max<size_t>(kThreads, a.tokens * per_token / (sm_count() * 6)));
  size_t most = std::max<size_t>(1, kTableBytes / (turned * W * sizeof(float2)));
  a.block_tokens = (int)std::min(most, std::max<size_t>(1, want / per_token));
  a.block_heads = (int)heads;
  size_t splits = 1;
  if (per_token > want) {
    splits = std::min<size_t>(65535, std::min(heads, (per_token + want - 1) / want));
    a.block_heads = (int)((heads + splits - 1) / splits);
    splits = (heads + a.block_heads - 1) / a.block_heads;
  }
  const dim3 grid((unsigned)((a.tokens + a.block_tokens - 1) / a.block_tokens), (unsigned)splits);
  const size_t shared = a.block_tokens * turned * W * sizeof(float2);
  return launch_kernel(rotary_kernel<T, W, HALF>, grid, dim3(kThreads), shared, stream, a);
}
template <typename T, int W>
cudaError_t launch_wide(RotaryArgs& a, cudaStream_t stream) {
  return a.half ? launch_of<T, W, true>(a, stream) : launch_of<T, W, false>(a, stream);
}
// Vectors as wide as the rows allow (the halves' lengths, strides, boundaries): 32 + 8
// heads of bf16, 168 MB both ways in 8,192 x 128 / head_dim tokens: 29 us eight wide,
// 36 four (40 turned of 80), 58 two (20 of 80), 105 one (6 of 64).
template <typename T>
cudaError_t launch_type(RotaryArgs& a, cudaStream_t stream) {
  switch (a.wide) {
    case 8: return launch_wide<T, 8>(a, stream);
    case 4: return launch_wide<T, 4>(a, stream);
    case 2: return launch_wide<T, 2>(a, stream);
  }
  return launch_wide<T, 1>(a, stream);
}

}  // namespace

cudaError_t launch_rotary(RotaryArgs a, cudaStream_t stream) {
  return a.type == RCC_F32 ? launch_type<float>(a, stream) : launch_type<__nv_bfloat16>(a, stream);
}

}  // namespace lm
}  // namespace rcc
