// matmul_i8_few.cu -- the 8-bit integer product for up to four tokens
// (include/rbf_ops.h, matmul_i8_dev and linear_i8_dev), in one launch.
//
//   out[i, j] = a_scale[i] * b_scale[j] * sum_k a[i, k] b[j, k] + bias[j]
//
// So few tokens leave b's bytes to be read once and 4 m operations on each, a
// matter of memory bandwidth (dp4a, four products an instruction).
// The tokens are put into shared memory by every CTA, as bytes; rows of
// floating-point numbers (linear_i8_dev) are quantised there, each CTA for
// itself, which costs less than a launch of its own and a wait for it.
//
// Eight lanes share a row of b, 128 contiguous bytes a step, and a warp has
// four such groups; a group takes kRows rows at once, so that a lane has that
// many 16-byte loads under way and every 16 bytes of the tokens that it reads
// serve kRows rows. The sums are exact integers; three shuffles join a group's.
//
// 1 x 1M x 768 to fp32: 114 us = 6.8 TB/s, the copy rate; 1 x 10,000 x 384,
// which L2 holds, 6.2 us: a launch, the tokens' way to shared memory and one
// round of loads.
#include <algorithm>

#include "ops_internal.h"
#include "quantize.cuh"
#include "rbf_device.cuh"
#include "rbf_internal.h"

namespace rbf {
namespace {

constexpr int kFewThreads = 256;
constexpr int kGroup = 8;  // lanes of a row

struct FewParams {
  const void* a;
  int64_t ld_a;
  const float* a_scale;
  const int8_t* b;
  int64_t ld_b;
  const float* b_scale;
  const float* bias;
  void* out;
  int64_t ld_out;
  int64_t n;
  int m, k;
  int out_dtype;
};

__device__ __forceinline__ uint32_t few_block_max(uint32_t v) {
  __shared__ uint32_t part[kFewThreads / 32];
  v = __reduce_max_sync(kFullMask, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kFewThreads / 32; ++w) v = max(v, part[w]);
  return v;
}

// 16 bytes of a row of b; past its end (the row's last ones may be the
// memory's) they are read one by one, zero beyond.
__device__ __forceinline__ int4 load16(const int8_t* row, int c, int k) {
  if (c + 16 <= k) return __ldg(reinterpret_cast<const int4*>(row + c));
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (c + i < k) w[i >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(row[c + i])) << (8 * (i & 3));
  return make_int4(static_cast<int>(w[0]), static_cast<int>(w[1]), static_cast<int>(w[2]), static_cast<int>(w[3]));
}

// X: the tokens' type, int8_t or a floating-point type that is quantised here.
// kAhead: steps whose loads are under way. STREAM: b is larger than what L2
// would keep for the next call, and its lines are marked to leave first.
template <typename X, int M, int kRows, int kAhead, bool STREAM>
__global__ void __launch_bounds__(kFewThreads) matmul_i8_few_kernel(const FewParams p) {
  extern __shared__ __align__(16) int8_t tokens[];  // [m][pitch], zero past k
  __shared__ float scales[M];
  const int pitch = (p.k + 15) / 16 * 16;
  if constexpr (sizeof(X) == 1) {
    for (int i = 0; i < p.m; ++i) {
      const int8_t* row = static_cast<const int8_t*>(p.a) + i * p.ld_a;
      for (int c = threadIdx.x; c < pitch; c += kFewThreads) tokens[i * pitch + c] = c < p.k ? row[c] : static_cast<int8_t>(0);
    }
    if (threadIdx.x < p.m) scales[threadIdx.x] = p.a_scale ? p.a_scale[threadIdx.x] : 1.0f;
  } else {
    for (int i = 0; i < p.m; ++i) {
      const X* row = static_cast<const X*>(p.a) + i * p.ld_a;
      uint32_t top = 0;
      for (int c = threadIdx.x; c < p.k; c += kFewThreads) top = max(top, __float_as_uint(to_f32(row[c])) & 0x7FFFFFFFu);
      const RowScale s = row_scale(few_block_max(top));
      for (int c = threadIdx.x; c < pitch; c += kFewThreads)
        tokens[i * pitch + c] = c < p.k ? static_cast<int8_t>(__float_as_uint(quantize_sum(to_f32(row[c]), s))) : static_cast<int8_t>(0);
      if (threadIdx.x == 0) scales[i] = s.scale;
    }
  }
  __syncthreads();

  const int lane = threadIdx.x & 31;
  const int part = lane % kGroup;
  const int64_t groups = static_cast<int64_t>(gridDim.x) * (kFewThreads / kGroup);
  const int64_t blocks = (p.n + kRows - 1) / kRows;
  // All lanes of a warp run the same number of steps: the shuffles need them.
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kFewThreads / kGroup) + threadIdx.x / kGroup;
  const int64_t rounds = (blocks - (first - lane / kGroup) + groups - 1) / groups;
  for (int64_t t = 0; t < rounds; ++t) {
    const int64_t j0 = (first + t * groups) * kRows;
    const int8_t* row[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) row[r] = p.b + min(j0 + r, p.n - 1) * p.ld_b;
    int sum[kRows][M] = {};
    auto multiply = [&](const int4 (&w)[kRows], int c) {
#pragma unroll
      for (int i = 0; i < M; ++i) {
        if (M > 1 && i >= p.m) break;
        const int4 x = *reinterpret_cast<const int4*>(tokens + i * pitch + c);
#pragma unroll
        for (int r = 0; r < kRows; ++r)
          sum[r][i] = __dp4a(w[r].x, x.x, __dp4a(w[r].y, x.y, __dp4a(w[r].z, x.z, __dp4a(w[r].w, x.w, sum[r][i]))));
      }
    };
    constexpr int kStep = 16 * kGroup;
    int c = 16 * part;
    const int whole = p.k - p.k % 16;  // no 16 bytes of a row reach past this
    for (; c + (kAhead - 1) * kStep < whole; c += kAhead * kStep) {
      int4 w[kAhead][kRows];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          const int4* at = reinterpret_cast<const int4*>(row[r] + c + u * kStep);
          w[u][r] = STREAM ? __ldcs(at) : __ldg(at);
        }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) multiply(w[u], c + u * kStep);
    }
    for (; c < p.k; c += kStep) {
      int4 w[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) w[r] = load16(row[r], c, p.k);
      multiply(w, c);
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int i = 0; i < M; ++i)
#pragma unroll
        for (int d = kGroup / 2; d > 0; d >>= 1) sum[r][i] += __shfl_xor_sync(kFullMask, sum[r][i], d);
    // Lane `part` of the group stores the results part, part + 8 ..
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
#pragma unroll
      for (int i = 0; i < M; ++i) {
        const int64_t j = j0 + r;
        if ((r * M + i) % kGroup != part || i >= p.m || j >= p.n) continue;
        const int64_t at = i * p.ld_out + j;
        if (p.out_dtype == kI32) {
          static_cast<int*>(p.out)[at] = sum[r][i];
          continue;
        }
        const float v = __fmaf_rn(__fmul_rn(__int2float_rn(sum[r][i]), scales[i]), p.b_scale ? p.b_scale[j] : 1.0f, p.bias ? p.bias[j] : 0.0f);
        if (p.out_dtype == kF32)
          static_cast<float*>(p.out)[at] = v;
        else if (p.out_dtype == kBF16)
          static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
        else
          static_cast<__half*>(p.out)[at] = __float2half_rn(v);
      }
    }
  }
}

template <typename X, int M, int kRows, int kAhead, bool STREAM>
cudaError_t launch_rows(const FewParams& p, int num_sms, cudaStream_t st) {
  auto fn = matmul_i8_few_kernel<X, M, kRows, kAhead, STREAM>;
  static PerDeviceOnce once;
  const cudaError_t ready = once.run(
      [fn] { return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewMaxTokenBytes); });
  if (ready != cudaSuccess) return ready;
  const int smem = p.m * ((p.k + 15) / 16 * 16);
  const int64_t rows = static_cast<int64_t>(kFewThreads / kGroup) * kRows;  // of a CTA at a time
  const int64_t grid = std::min<int64_t>((p.n + rows - 1) / rows, int64_t(num_sms) * (smem > 48 * 1024 ? 2 : 4));
  fn<<<static_cast<unsigned>(grid), kFewThreads, smem, st>>>(p);
  return cudaGetLastError();
}

constexpr int64_t kL2Bytes = int64_t(64) << 20;
// Rows of a group and steps under way, measured at 1M x 768 for 1, 2 and 4
// tokens: 2 x 6 114, 138 and 147 us; 1 x 6 129, 116 and 148; 4 x 3 135, 146
// and 134.
template <int M>
constexpr int kRowsOf = M == 1 ? 2 : M == 2 ? 1 : 4;
template <int M>
constexpr int kAheadOf = M <= 2 ? 6 : 3;

template <typename X, int M>
cudaError_t launch_m(const FewParams& p, int num_sms, cudaStream_t st) {
  // One row a group where that is what gives every SM work.
  if (p.n < int64_t(num_sms) * 4 * (kFewThreads / kGroup)) return launch_rows<X, M, 1, 6, false>(p, num_sms, st);
  if (p.n * p.k <= kL2Bytes) return launch_rows<X, M, kRowsOf<M>, kAheadOf<M>, false>(p, num_sms, st);
  return launch_rows<X, M, kRowsOf<M>, kAheadOf<M>, true>(p, num_sms, st);
}

template <typename X>
cudaError_t launch_x(const FewParams& p, int num_sms, cudaStream_t st) {
  if (p.m == 1) return launch_m<X, 1>(p, num_sms, st);
  if (p.m == 2) return launch_m<X, 2>(p, num_sms, st);
  return launch_m<X, 4>(p, num_sms, st);
}

}  // namespace

bool matmul_i8_few_fits(const MatmulI8Launch& a) {
  return a.m <= 4 && a.k > 0 && (reinterpret_cast<uintptr_t>(a.b) & 15) == 0 && a.ld_b % 16 == 0 &&
         a.m * ((a.k + 15) / 16 * 16) <= kFewMaxTokenBytes;
}

cudaError_t launch_matmul_i8_few(const MatmulI8Launch& a, const void* tokens, int64_t ld, int dtype, int num_sms, cudaStream_t st) {
  FewParams p;
  p.a = tokens;
  p.ld_a = ld;
  p.a_scale = a.a_scale;
  p.b = a.b;
  p.ld_b = a.ld_b;
  p.b_scale = a.b_scale;
  p.bias = a.bias;
  p.out = a.out;
  p.ld_out = a.ld_out;
  p.n = a.n;
  p.m = static_cast<int>(a.m);
  p.k = a.k;
  p.out_dtype = a.out_dtype;
  if (dtype == kI8) return launch_x<int8_t>(p, num_sms, st);
  if (dtype == kF32) return launch_x<float>(p, num_sms, st);
  if (dtype == kBF16) return launch_x<__nv_bfloat16>(p, num_sms, st);
  return launch_x<__half>(p, num_sms, st);
}

}  // namespace rbf
