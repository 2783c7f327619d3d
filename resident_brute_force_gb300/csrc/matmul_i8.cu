// matmul_i8.cu -- what the products of 8-bit matrices (include/rbf_ops.h,
// matmul_i8_dev) need beside their two kernels: rows put on 16-byte boundaries,
// and the result of a depth of zero.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "ops_internal.h"
#include "rbf_device.cuh"

namespace rbf {
namespace {

struct Epilogue {
  const float* a_scale;
  const float* b_scale;
  const float* bias;
  void* out;
  int out_dtype;
  int64_t ld_out;
};

__device__ __forceinline__ void store_out(const Epilogue& e, int64_t i, int64_t j, int sum) {
  const int64_t at = i * e.ld_out + j;
  if (e.out_dtype == kI32) {
    static_cast<int*>(e.out)[at] = sum;
    return;
  }
  float v = __int2float_rn(sum);
  if (e.a_scale) v = __fmul_rn(v, e.a_scale[i]);
  v = __fmaf_rn(v, e.b_scale ? e.b_scale[j] : 1.0f, e.bias ? e.bias[j] : 0.0f);
  if (e.out_dtype == kF32)
    static_cast<float*>(e.out)[at] = v;
  else if (e.out_dtype == kBF16)
    static_cast<__nv_bfloat16*>(e.out)[at] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(e.out)[at] = __float2half_rn(v);
}

// ------------------------------------------------------------ a depth of zero

__global__ void __launch_bounds__(256) matmul_i8_empty_kernel(int64_t m, int64_t n, const Epilogue e) {
  for (int64_t g = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; g < m * n; g += static_cast<int64_t>(gridDim.x) * 256)
    store_out(e, g / n, g % n, 0);
}

// ------------------------------------------------- rows to 16-byte boundaries
//
// Sixteen bytes a thread, from the four or five aligned words that hold them:
// each of those has a byte of the row in it. The product then runs as for such
// rows, a part of b that L2 holds at a time. Measured with a dp4a kernel of any
// strides in its place: 256 x 100,000 x 1,001 111 us and 701, 37 x 10,007 x
// 1,001 18.6 and 44.7, 1 x 1M x 770 533 and 1,173 (aligned: 115), 1 x 1,000 x
// 383 10.3 and 14.5.
__global__ void __launch_bounds__(256)
    pitch_rows_kernel(const int8_t* __restrict__ b, int64_t ld_b, int64_t rows, int k, int8_t* __restrict__ out, int pitch) {
  const int per = pitch / 16;
  const int64_t all = rows * per;
  for (int64_t g = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; g < all; g += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t i = g / per;
    const int c = static_cast<int>(g - i * per) * 16;
    const int8_t* row = b + i * ld_b;
    const uintptr_t from = reinterpret_cast<uintptr_t>(row + c), end = reinterpret_cast<uintptr_t>(row + k);
    const uint32_t* word = reinterpret_cast<const uint32_t*>(from & ~uintptr_t(3));
    const int shift = static_cast<int>(from & 3) * 8;
    uint32_t w[5];
#pragma unroll
    for (int j = 0; j < 5; ++j) w[j] = reinterpret_cast<uintptr_t>(word + j) < end ? word[j] : 0u;
    uint4 v;
    v.x = __funnelshift_r(w[0], w[1], shift);
    v.y = __funnelshift_r(w[1], w[2], shift);
    v.z = __funnelshift_r(w[2], w[3], shift);
    v.w = __funnelshift_r(w[3], w[4], shift);
    *reinterpret_cast<uint4*>(out + i * pitch + c) = v;
  }
}

}  // namespace

cudaError_t launch_pitch_rows(const int8_t* b, int64_t ld_b, int64_t rows, int k, int8_t* out, int pitch, int num_sms,
                              cudaStream_t st) {
  const int64_t blocks = std::min<int64_t>((rows * (pitch / 16) + 255) / 256, int64_t(num_sms) * 8);
  pitch_rows_kernel<<<static_cast<unsigned>(blocks), 256, 0, st>>>(b, ld_b, rows, k, out, pitch);
  return cudaGetLastError();
}

cudaError_t launch_matmul_i8_empty(const MatmulI8Launch& a, int num_sms, cudaStream_t st) {
  const Epilogue e{a.a_scale, a.b_scale, a.bias, a.out, a.out_dtype, a.ld_out};
  const int64_t blocks = std::min<int64_t>((a.m * a.n + 255) / 256, int64_t(num_sms) * 8);
  matmul_i8_empty_kernel<<<static_cast<unsigned>(blocks), 256, 0, st>>>(a.m, a.n, e);
  return cudaGetLastError();
}

}  // namespace rbf
