// quantize.cu -- rows of floating-point numbers to 8-bit integers with one
// scale a row (include/rbf_ops.h, quantize_rows_i8_dev).
//
// With t = max_j |x_j|: scale = t * (1 / 127), q_j = x_j * ((1 / t) * 127)
// rounded to nearest even, all in fp32 (one division a row, one product a
// value, each rounded as IEEE says, so that the integers are the same wherever
// they are computed). |q| <= 127: x_j times the factor is at most
// 127 (1 + 2^-22), which rounds to 127.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "ops_internal.h"
#include "rbf_device.cuh"

namespace rbf {
namespace {

constexpr int kQuantThreads = 256;

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }

// What a row's values are multiplied by: first by `pre` (a power of two: 1,
// or 2^100 for a row so small that 1 / t could overflow), then by `inv`.
struct RowScale {
  float scale, pre, inv;
};

// `code`: the largest |x| of the row as its fp32 pattern, which orders
// magnitudes as unsigned integers with the infinities and the NaNs on top.
__device__ __forceinline__ RowScale row_scale(uint32_t code) {
  RowScale r;
  if (code >= 0x7F800000u) {  // a NaN or an infinity: zeros, and a scale that makes every product NaN
    r.scale = __uint_as_float(0x7FC00000u);
    r.pre = 0.0f;
    r.inv = 0.0f;
    return r;
  }
  const float t = __uint_as_float(code);
  r.scale = __fmul_rn(t, 1.0f / 127.0f);
  r.pre = t < 0x1p-100f ? 0x1p100f : 1.0f;
  r.inv = t > 0.0f ? __fmul_rn(__fdiv_rn(1.0f, __fmul_rn(t, r.pre)), 127.0f) : 0.0f;
  return r;
}

__device__ __forceinline__ int quantize_one(float x, const RowScale& r) {
  if (r.inv == 0.0f) return 0;  // also keeps 0 * infinity out
  return __float2int_rn(__fmul_rn(__fmul_rn(x, r.pre), r.inv));
}

__device__ __forceinline__ uint32_t block_max(uint32_t v) {
  __shared__ uint32_t part[kQuantThreads / 32];
  __shared__ uint32_t whole;
  v = __reduce_max_sync(kFullMask, v);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    const uint32_t w = __reduce_max_sync(kFullMask, threadIdx.x < kQuantThreads / 32 ? part[threadIdx.x] : 0u);
    if (threadIdx.x == 0) whole = w;
  }
  __syncthreads();
  return whole;
}

// One CTA per row, any strides and alignments: two reads of the row, the
// second from cache.
template <typename T>
__global__ void __launch_bounds__(kQuantThreads)
    quantize_rows_kernel(const T* __restrict__ x, int64_t ld_x, int64_t rows, int cols, int8_t* __restrict__ q,
                         int64_t ld_q, float* __restrict__ scale) {
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const T* row = x + r * ld_x;
    uint32_t top = 0;
    for (int j = threadIdx.x; j < cols; j += kQuantThreads)
      top = max(top, __float_as_uint(to_f32(row[j])) & 0x7FFFFFFFu);
    const RowScale s = row_scale(block_max(top));
    for (int j = threadIdx.x; j < cols; j += kQuantThreads)
      q[r * ld_q + j] = static_cast<int8_t>(quantize_one(to_f32(row[j]), s));
    if (threadIdx.x == 0) scale[r] = s.scale;
    __syncthreads();  // block_max's shared words are used again
  }
}

template <typename T>
cudaError_t launch_t(const QuantizeLaunch& a, cudaStream_t st) {
  const int64_t grid = std::min<int64_t>(a.rows, int64_t(1) << 20);
  quantize_rows_kernel<T><<<static_cast<unsigned>(grid), kQuantThreads, 0, st>>>(
      static_cast<const T*>(a.x), a.ld_x, a.rows, a.cols, a.q, a.ld_q, a.scale);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize_rows(const QuantizeLaunch& a, cudaStream_t st) {
  if (a.dtype == kF32) return launch_t<float>(a, st);
  if (a.dtype == kBF16) return launch_t<__nv_bfloat16>(a, st);
  return launch_t<__half>(a, st);
}

}  // namespace rbf
