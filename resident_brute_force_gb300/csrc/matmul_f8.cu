// matmul_f8.cu -- product of two 8-bit floating-point matrices with a scale for
// each 128 values of a row of a, and for each 128 values of a row or of 128 rows
// of b (include/rbf_ops.h, matmul_f8_dev):
//
//   out[i, j] = sum_c a_scale[i, c] b_scale[j / block_rows, c] sum_{k in block c} a[i, k] b[j, k] + bias[j]
//
// A tile of 64 x 64 outputs a CTA, sixteen a thread; a block of 128 values of
// depth at a time, as fp32 numbers in shared memory, summed in fp32 and added to
// the outputs' sums with its scales. It takes any strides and alignment.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "ops_internal.h"
#include "rbf_device.cuh"

namespace rbf {
namespace {

constexpr int kBlock = 128;
constexpr int kTile = 64;
constexpr int kThreads = 256;
constexpr int kPitch = kTile + 4;

__device__ __forceinline__ float from_f8(uint8_t v, bool e4m3) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(v, e4m3 ? __NV_E4M3 : __NV_E5M2)));
}

__device__ __forceinline__ void store_out(const MatmulF8Launch& p, int64_t i, int64_t j, float v) {
  const int64_t at = i * p.ld_out + j;
  if (p.bias) v = __fadd_rn(v, p.bias[j]);
  if (p.out_dtype == kF32)
    static_cast<float*>(p.out)[at] = v;
  else if (p.out_dtype == kBF16)
    static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(p.out)[at] = __float2half_rn(v);
}

__global__ void __launch_bounds__(kThreads) matmul_f8_kernel(const MatmulF8Launch p) {
  __shared__ float as[32][kPitch], bs[32][kPitch];
  const int64_t j_tiles = (p.n + kTile - 1) / kTile;
  const int64_t i0 = blockIdx.x / j_tiles * kTile, j0 = blockIdx.x % j_tiles * kTile;
  const int ty = threadIdx.x / 16 * 4, tx = threadIdx.x % 16 * 4;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < p.k; k0 += kBlock) {
    float part[4][4] = {};
    for (int kk = k0; kk < min(p.k, k0 + kBlock); kk += 32) {
      for (int e = threadIdx.x; e < kTile * 32; e += kThreads) {
        const int r = e / 32, c = e % 32;
        const bool in = kk + c < p.k;
        as[c][r] = in && i0 + r < p.m ? from_f8(p.a[(i0 + r) * p.ld_a + kk + c], p.a_dtype == kE4M3) : 0.0f;
        bs[c][r] = in && j0 + r < p.n ? from_f8(p.b[(j0 + r) * p.ld_b + kk + c], p.b_dtype == kE4M3) : 0.0f;
      }
      __syncthreads();
#pragma unroll 8
      for (int c = 0; c < 32; ++c)
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
          for (int x = 0; x < 4; ++x) part[y][x] = __fmaf_rn(as[c][ty + y], bs[c][tx + x], part[y][x]);
      __syncthreads();
    }
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const int64_t i = i0 + ty + y;
      const float sa = i < p.m ? p.a_scale[i * p.ld_a_scale + k0 / kBlock] : 0.0f;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int64_t j = j0 + tx + x;
        const float sb = j < p.n ? p.b_scale[j / p.block_rows * p.ld_b_scale + k0 / kBlock] : 0.0f;
        acc[y][x] = __fmaf_rn(part[y][x], __fmul_rn(sa, sb), acc[y][x]);
      }
    }
  }
#pragma unroll
  for (int y = 0; y < 4; ++y)
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (i0 + ty + y < p.m && j0 + tx + x < p.n) store_out(p, i0 + ty + y, j0 + tx + x, acc[y][x]);
}

}  // namespace

cudaError_t launch_matmul_f8(const MatmulF8Launch& a, cudaStream_t st) {
  const int64_t tiles = ((a.m + kTile - 1) / kTile) * ((a.n + kTile - 1) / kTile);
  matmul_f8_kernel<<<static_cast<unsigned>(tiles), kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace rbf
