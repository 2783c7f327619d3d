// matmul_i8.cu -- product of two matrices of 8-bit integers with a scale for
// each row of either (include/rbf_ops.h, matmul_i8_dev):
//
//   out[i, j] = a_scale[i] * b_scale[j] * sum_k a[i, k] b[j, k] + bias[j]
//
// The sums are exact 32-bit integers, converted to fp32 once; the scales and
// the bias are applied in fp32 and the result is rounded once to the output's
// type.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

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

// --------------------------------------------------- any strides, dp4a
//
// A 64 x 64 tile a CTA of 256 threads, 4 x 4 sums a thread, 64 values of
// depth a step through shared memory, four products an instruction (dp4a). For
// operands that no tensor map can describe (b off 16-byte boundaries) and for a
// depth of zero: bound by the dp4a rate and by the loads' instructions.

constexpr int kAnyTile = 64;
constexpr int kAnyWords = 16;  // 4-byte words of one row and step

// Four values of a row from `c` on, zero past the end.
__device__ __forceinline__ int word_at(const int8_t* row, int c, int k, bool wide) {
  if (wide && c + 4 <= k) return *reinterpret_cast<const int*>(row + c);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (c + i < k) w |= static_cast<uint32_t>(static_cast<uint8_t>(row[c + i])) << (8 * i);
  return static_cast<int>(w);
}

__global__ void __launch_bounds__(256)
    matmul_i8_any_kernel(const int8_t* __restrict__ a, int64_t ld_a, const int8_t* __restrict__ b, int64_t ld_b,
                         int64_t m, int64_t n, int k, const Epilogue e) {
  __shared__ int sa[kAnyTile][kAnyWords + 1];
  __shared__ int sb[kAnyTile][kAnyWords + 1];
  const int64_t j0 = static_cast<int64_t>(blockIdx.x) * kAnyTile;
  const int64_t i0 = static_cast<int64_t>(blockIdx.y) * kAnyTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const bool wide_a = (reinterpret_cast<uintptr_t>(a) & 3) == 0 && ld_a % 4 == 0;
  const bool wide_b = (reinterpret_cast<uintptr_t>(b) & 3) == 0 && ld_b % 4 == 0;
  int sum[4][4] = {};
  for (int k0 = 0; k0 < k; k0 += 4 * kAnyWords) {
    for (int w = threadIdx.x; w < kAnyTile * kAnyWords; w += 256) {
      const int r = w / kAnyWords, c = w % kAnyWords;
      sa[r][c] = i0 + r < m ? word_at(a + (i0 + r) * ld_a, k0 + 4 * c, k, wide_a) : 0;
      sb[r][c] = j0 + r < n ? word_at(b + (j0 + r) * ld_b, k0 + 4 * c, k, wide_b) : 0;
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kAnyWords; ++c) {
      int va[4], vb[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        va[x] = sa[ty + 16 * x][c];
        vb[x] = sb[tx + 16 * x][c];
      }
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) sum[x][y] = __dp4a(va[x], vb[y], sum[x][y]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int x = 0; x < 4; ++x)
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const int64_t i = i0 + ty + 16 * x, j = j0 + tx + 16 * y;
      if (i < m && j < n) store_out(e, i, j, sum[x][y]);
    }
}

Epilogue epilogue_of(const MatmulI8Launch& a) {
  Epilogue e;
  e.a_scale = a.a_scale;
  e.b_scale = a.b_scale;
  e.bias = a.bias;
  e.out = a.out;
  e.out_dtype = a.out_dtype;
  e.ld_out = a.ld_out;
  return e;
}

}  // namespace

cudaError_t launch_matmul_i8_any(const MatmulI8Launch& a, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>((a.n + kAnyTile - 1) / kAnyTile),
                  static_cast<unsigned>((a.m + kAnyTile - 1) / kAnyTile));
  matmul_i8_any_kernel<<<grid, 256, 0, st>>>(a.a, a.ld_a, a.b, a.ld_b, a.m, a.n, a.k, epilogue_of(a));
  return cudaGetLastError();
}

}  // namespace rbf
