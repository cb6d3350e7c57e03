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
#include "lm_common.cuh"
#include "lm_internal.h"

namespace rcc {
namespace lm {
namespace {

// A group whose largest magnitude is below this is kept as zeros (1/a stays
// finite for the others).
constexpr float kTiny = 7.52316385e-37f;  // 2^-120

// Sums over the G threads (a power of two) that share a row; G > 32 goes
// through shared memory.  Every thread of the block calls it.
template <int G, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*red)[N], int tid) {
#pragma unroll
  for (int o = (G < 32 ? G : 32) / 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
  if constexpr (G > 32) {
    __syncthreads();  // the previous row's sums have been read
    if ((tid & 31) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) red[tid >> 5][i] = v[i];
    __syncthreads();
    const int w0 = (tid / G) * (G / 32);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.f;
    for (int w = 0; w < G / 32; ++w)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += red[w0 + w][i];
  }
}

// threads of a block whose rows take G threads each
template <int G>
constexpr int kBlock = G > 256 ? G : 256;

// One row for each group of G threads; a thread holds NV vectors of eight
// columns, vector k at (k G + t) 8, so 16 neighbouring threads hold one group
// of 128 columns.
template <typename T, int G, int NV, bool VEC>
__global__ void __launch_bounds__(kBlock<G>) norm_forward_kernel(const NormArgs a) {
  constexpr int kRows = kBlock<G> / G;
  __shared__ float red[kBlock<G> / 32][1];
  pdl_wait_then_release();
  const int tid = threadIdx.x, t = tid % G;
  const size_t row = (size_t)blockIdx.x * kRows + tid / G;
  const bool live = row < a.tokens;
  const T* x = static_cast<const T*>(a.x) + (live ? row : 0) * a.ld_x;
  float v[NV][8];
  float sum[1] = {0.f};
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const size_t col = (size_t)(k * G + t) * 8;
    if (live && col < a.dim) {
      load_row8<VEC>(x, col, a.dim, v[k]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[k][e] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[0] = fmaf(v[k][e], v[k][e], sum[0]);
  }
  row_sum<G>(sum, red, tid);
  const float r = __frsqrt_rn(sum[0] / (float)a.dim + a.eps);
  const size_t groups = (a.dim + kKeepGroup - 1) / kKeepGroup;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const size_t col = (size_t)(k * G + t) * 8;
    if (a.kept) {
      // |x| as its bits: ordered like the values, infinity and NaN above them
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[k][e]) & 0x7FFFFFFFu);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
      if (live && col < groups * kKeepGroup) {
        const float amax = __uint_as_float(top);
        const bool bad = top >= 0x7F800000u, small = amax < kTiny;
        const float inv = bad || small ? 0.f : 127.f * __frcp_rn(amax);
        uint32_t w[2] = {0u, 0u};
        if (!bad) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int q = __float2int_rn(v[k][e] * inv);
            w[e >> 2] |= (uint32_t)(q & 0xFF) << (8 * (e & 3));
          }
        }
        *reinterpret_cast<uint2*>(a.kept + row * groups * kKeepGroup + col) =
            make_uint2(w[0], w[1]);
        if ((t & 15) == 0)
          a.scales[row * groups + col / kKeepGroup] =
              bad ? __uint_as_float(0x7FC00000u) : small ? 0.f : amax * (1.f / 127.f);
      }
    }
    if (live && col < a.dim) {
      float w8[8];
      load_row8<VEC>(a.weight, col, a.dim, w8);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[k][e] = v[k][e] * r * w8[e];
      store_row8<VEC>(static_cast<T*>(a.y) + row * a.ld_y, col, a.dim, v[k]);
    }
  }
}

// Rows are dealt to the blocks in turn; a thread keeps the weight gradient of
// its columns in registers over all of its rows, and each block writes one
// row of partial sums, which norm_dweight_kernel adds in a fixed order.
template <typename T, int G, int NV, bool VEC>
__global__ void __launch_bounds__(kBlock<G>) norm_backward_kernel(const NormGradArgs a) {
  constexpr int kRows = kBlock<G> / G;
  __shared__ float red[kBlock<G> / 32][2];
  pdl_wait_then_release();
  const int tid = threadIdx.x, t = tid % G;
  const size_t groups = (a.dim + kKeepGroup - 1) / kKeepGroup;
  float acc[NV][8];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[k][e] = 0.f;
  for (size_t first = (size_t)blockIdx.x * kRows; first < a.tokens;
       first += (size_t)gridDim.x * kRows) {
    const size_t row = first + tid / G;
    const bool live = row < a.tokens;
    const T* dy = static_cast<const T*>(a.dy) + (live ? row : 0) * a.ld_dy;
    float x[NV][8], d[NV][8];
    float sum[2] = {0.f, 0.f};  // of x'^2, of dy w x'
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const size_t col = (size_t)(k * G + t) * 8;
      if (live && col < a.dim) {
        load_row8<VEC>(dy, col, a.dim, d[k]);
        const uint2 q = *reinterpret_cast<const uint2*>(
            a.kept + row * groups * kKeepGroup + col);
        const float s = a.scales[row * groups + col / kKeepGroup];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          x[k][e] = (float)(int8_t)((e < 4 ? q.x : q.y) >> (8 * (e & 3))) * s;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[k][e] = d[k][e] = 0.f;
      }
      float w[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (col < a.dim) load_row8<VEC>(a.weight, col, a.dim, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sum[0] = fmaf(x[k][e], x[k][e], sum[0]);
        sum[1] = fmaf(d[k][e] * w[e], x[k][e], sum[1]);
      }
    }
    row_sum<G>(sum, red, tid);
    const float r = __frsqrt_rn(sum[0] / (float)a.dim + a.eps);
    const float m = sum[1] * r / (float)a.dim;  // mean of dy w n
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const size_t col = (size_t)(k * G + t) * 8;
      if (live && col < a.dim) {
        float w[8];
        load_row8<VEC>(a.weight, col, a.dim, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float n = x[k][e] * r;
          acc[k][e] = fmaf(d[k][e], n, acc[k][e]);
          d[k][e] = r * (d[k][e] * w[e] - n * m);
        }
        store_row8<VEC>(static_cast<T*>(a.dx) + row * a.ld_dx, col, a.dim, d[k]);
      }
    }
  }
  // one row of partial sums for each group of threads
  float* part = static_cast<float*>(a.workspace) +
                ((size_t)blockIdx.x * kRows + tid / G) * groups * kKeepGroup;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const size_t col = (size_t)(k * G + t) * 8;
    if (col < groups * kKeepGroup) store8(part + col, acc[k]);
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
  if (col < dim)
    for (size_t r = y; r < rows; r += kSumRows) s += part[r * ld + col];
  red[y][c] = s;
  __syncthreads();
  if (y == 0 && col < dim) {
    for (int i = 1; i < kSumRows; ++i) s += red[i][c];
    dweight[col] = accumulate ? dweight[col] + s : s;
  }
}

// Threads that share a row, and vectors of eight columns for each
struct NormShape {
  int g, nv;
};
NormShape norm_shape(size_t dim) {
  const size_t vecs = (dim + 7) / 8;
  if (vecs <= 32) return {32, 1};
  if (vecs <= 64) return {32, 2};
  if (vecs <= 128) return {64, 2};
  if (vecs <= 256) return {128, 2};
  if (vecs <= 512) return {256, 2};
  if (vecs <= 1024) return {256, 4};
  if (vecs <= 2048) return {512, 4};
  return {1024, 4};
}

int norm_threads(const NormShape& s) { return s.g > 256 ? s.g : 256; }
int norm_rows_per_block(const NormShape& s) { return norm_threads(s) / s.g; }

// blocks of the backward pass: every SM filled once with 1,024 threads
size_t norm_backward_blocks(size_t tokens, const NormShape& s) {
  const size_t rows = norm_rows_per_block(s);
  const size_t need = (tokens + rows - 1) / rows;
  const size_t fill = (size_t)sm_count() * (1024 / norm_threads(s));
  return need < fill ? need : fill;
}

template <typename F>
cudaError_t with_shape(const NormShape& s, F f) {
  if (s.g == 32 && s.nv == 1) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 1>());
  if (s.g == 32) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 2>());
  if (s.g == 64) return f(std::integral_constant<int, 64>(), std::integral_constant<int, 2>());
  if (s.g == 128) return f(std::integral_constant<int, 128>(), std::integral_constant<int, 2>());
  if (s.g == 256 && s.nv == 2) return f(std::integral_constant<int, 256>(), std::integral_constant<int, 2>());
  if (s.g == 256) return f(std::integral_constant<int, 256>(), std::integral_constant<int, 4>());
  if (s.g == 512) return f(std::integral_constant<int, 512>(), std::integral_constant<int, 4>());
  return f(std::integral_constant<int, 1024>(), std::integral_constant<int, 4>());
}

template <typename T, bool VEC>
cudaError_t forward_of(const NormArgs& a, cudaStream_t stream) {
  const NormShape s = norm_shape(a.dim);
  const size_t rows = norm_rows_per_block(s);
  return with_shape(s, [&](auto g, auto nv) {
    constexpr int G = decltype(g)::value, NV = decltype(nv)::value;
    return launch_kernel(norm_forward_kernel<T, G, NV, VEC>,
                         dim3((unsigned)((a.tokens + rows - 1) / rows)), dim3(kBlock<G>), 0,
                         stream, a);
  });
}

template <typename T, bool VEC>
cudaError_t backward_of(const NormGradArgs& a, cudaStream_t stream) {
  const NormShape s = norm_shape(a.dim);
  return with_shape(s, [&](auto g, auto nv) {
    constexpr int G = decltype(g)::value, NV = decltype(nv)::value;
    return launch_kernel(norm_backward_kernel<T, G, NV, VEC>,
                         dim3((unsigned)norm_backward_blocks(a.tokens, s)), dim3(kBlock<G>), 0,
                         stream, a);
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
  return norm_backward_blocks(tokens, s) * norm_rows_per_block(s) * ld * sizeof(float);
}

cudaError_t launch_rmsnorm_backward(const NormGradArgs& a, cudaStream_t stream,
                                    uint64_t* launches) {
  cudaError_t e;
  if (a.type == RCC_F32)
    e = a.vec ? backward_of<float, true>(a, stream) : backward_of<float, false>(a, stream);
  else
    e = a.vec ? backward_of<__nv_bfloat16, true>(a, stream)
              : backward_of<__nv_bfloat16, false>(a, stream);
  if (e != cudaSuccess) return e;
  const NormShape s = norm_shape(a.dim);
  const size_t ld = (a.dim + kKeepGroup - 1) / kKeepGroup * kKeepGroup;
  e = launch_kernel(norm_dweight_kernel, dim3((unsigned)((a.dim + kSumCols - 1) / kSumCols)),
                    dim3(kSumCols * kSumRows), 0, stream,
                    static_cast<const float*>(a.workspace),
                    norm_backward_blocks(a.tokens, s) * (size_t)norm_rows_per_block(s), ld,
                    a.dweight, a.dim, a.accumulate);
  if (e == cudaSuccess) *launches = 2;
  return e;
}

}  // namespace lm
}  // namespace rcc
