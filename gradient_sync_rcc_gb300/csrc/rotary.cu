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
// thread makes the sines and cosines of eight pairs of a token and turns those
// pairs in kHeads heads, so that 16 (32) bytes a pair of accesses stand against
// an eighth of the sines; its loads are all under way before the first is used.
#include "lm_common.cuh"
#include "lm_internal.h"

namespace rcc {
namespace lm {
namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 4;  // heads of one token that a thread turns

struct Rows {
  const char* in;
  char* out;
};

// The head `h` of a token among the queries' and then the keys'
__device__ __forceinline__ Rows head_rows(const RotaryArgs& a, size_t token, int h, int size) {
  const bool key = h >= (int)a.q.heads;
  const RotaryRows& r = key ? a.k : a.q;
  const size_t head = key ? h - (int)a.q.heads : h;
  Rows s;
  s.in = static_cast<const char*>(r.in) + (token * r.in_token + head * r.in_head) * size;
  s.out = static_cast<char*>(r.out) + (token * r.out_token + head * r.out_head) * size;
  return s;
}

__device__ __forceinline__ uint64_t position_of(const RotaryArgs& a, size_t token) {
  int64_t p = (int64_t)token;
  if (a.positions)
    p = a.index64 ? static_cast<const int64_t*>(a.positions)[token]
                  : static_cast<const int32_t*>(a.positions)[token];
  return p < 0 ? 0 : (uint64_t)p + (uint64_t)a.offset;
}

__device__ __forceinline__ void sine_cosine(uint64_t position, uint64_t turns, float scale,
                                            float& s, float& c) {
  // half turns in [-1, 1)
  const float half = (float)(int32_t)((position * turns) >> 32) * 0x1p-31f;
  sincospif(half, &s, &c);
  s *= scale;
  c *= scale;
}

// A unit of VEC: eight pairs (16 elements), or eight elements that are only
// copied; else one pair or one element.
template <typename T, bool VEC, bool HALF>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs a) {
  pdl_wait_then_release();
  constexpr int kWide = VEC ? 8 : 1;
  const uint64_t at = (uint64_t)blockIdx.x * kThreads + threadIdx.x;
  const uint32_t units = a.turned_units + a.copied_units;
  const uint32_t each = units * a.chunks;  // threads of a token
  const uint64_t token = at / each;
  if (token >= a.tokens) return;
  const uint32_t rest = (uint32_t)(at - token * each);
  const uint32_t chunk = rest / units, unit = rest - chunk * units;
  const int h0 = (int)chunk * kHeads;
  const int live = min(kHeads, (int)(a.q.heads + a.k.heads) - h0);
  if (unit >= a.turned_units) {
    const uint32_t col = 2 * a.pairs + (unit - a.turned_units) * kWide;
    for (int i = 0; i < live; ++i) {
      const Rows r = head_rows(a, token, h0 + i, sizeof(T));
      const T* in = reinterpret_cast<const T*>(r.in) + col;
      T* out = reinterpret_cast<T*>(r.out) + col;
      if constexpr (VEC) {
        float v[8];
        load8(in, v);
        store8(out, v);
      } else {
        *out = *in;
      }
    }
    return;
  }
  // first and second elements of the unit's pairs
  const uint32_t first = HALF ? unit * kWide : 2 * unit * kWide;
  const uint32_t second = HALF ? first + a.pairs : first + kWide;
  float x[kHeads][kWide], y[kHeads][kWide];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    if (i < live) {
      const T* in = reinterpret_cast<const T*>(head_rows(a, token, h0 + i, sizeof(T)).in);
      if constexpr (VEC) {
        load8(in + first, x[i]);
        load8(in + second, y[i]);
      } else {
        x[i][0] = to_f32(in[first]);
        y[i][0] = to_f32(in[second]);
      }
    }
  }
  float s[kWide], c[kWide];
  const uint64_t position = position_of(a, token);
#pragma unroll
  for (int e = 0; e < kWide; ++e)
    sine_cosine(position, a.turns[unit * kWide + e], a.scale, s[e], c[e]);
  if (a.inverse)
#pragma unroll
    for (int e = 0; e < kWide; ++e) s[e] = -s[e];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    if (i < live) {
      T* out = reinterpret_cast<T*>(head_rows(a, token, h0 + i, sizeof(T)).out);
      float u[kWide], v[kWide];
      if constexpr (HALF || !VEC) {
#pragma unroll
        for (int e = 0; e < kWide; ++e) {
          u[e] = x[i][e] * c[e] - y[i][e] * s[e];
          v[e] = x[i][e] * s[e] + y[i][e] * c[e];
        }
      } else {  // neighbours: x holds the first four pairs, y the others
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          u[2 * e] = x[i][2 * e] * c[e] - x[i][2 * e + 1] * s[e];
          u[2 * e + 1] = x[i][2 * e] * s[e] + x[i][2 * e + 1] * c[e];
          v[2 * e] = y[i][2 * e] * c[4 + e] - y[i][2 * e + 1] * s[4 + e];
          v[2 * e + 1] = y[i][2 * e] * s[4 + e] + y[i][2 * e + 1] * c[4 + e];
        }
      }
      if constexpr (VEC) {
        store8(out + first, u);
        store8(out + second, v);
      } else {
        from_f32(u[0], out[first]);
        from_f32(v[0], out[second]);
      }
    }
  }
}

template <typename T>
cudaError_t launch_of(RotaryArgs& a, cudaStream_t stream) {
  const size_t wide = a.vec ? 8 : 1;
  a.turned_units = (uint32_t)(a.pairs / wide);
  a.copied_units = a.copies ? (uint32_t)((a.head_dim - 2 * a.pairs) / wide) : 0;
  a.chunks = (uint32_t)((a.q.heads + a.k.heads + kHeads - 1) / kHeads);
  const size_t threads = a.tokens * (a.turned_units + a.copied_units) * a.chunks;
  const dim3 grid((unsigned)((threads + kThreads - 1) / kThreads));
  auto kernel = a.vec ? a.half ? rotary_kernel<T, true, true> : rotary_kernel<T, true, false>
                      : a.half ? rotary_kernel<T, false, true> : rotary_kernel<T, false, false>;
  return launch_kernel(kernel, grid, dim3(kThreads), 0, stream, a);
}

}  // namespace

cudaError_t launch_rotary(RotaryArgs a, cudaStream_t stream) {
  return a.type == RCC_F32 ? launch_of<float>(a, stream) : launch_of<__nv_bfloat16>(a, stream);
}

}  // namespace lm
}  // namespace rcc
