// quantize.cu -- rows of floating-point numbers to 8-bit integers with one
// scale a row (include/rbf_ops.h, quantize_rows_i8_dev).
// The arithmetic is quantize.cuh's.
#include <algorithm>

#include "ops_internal.h"
#include "quantize.cuh"
#include "rbf_device.cuh"

namespace rbf {
namespace {

constexpr int kQuantThreads = 256;

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

// Where a row goes: bytes, or (f16 set) the fp16 rows of a product's
// workspace, which are zero from the row's end to their pitch.
struct Out {
  int8_t* q;
  int64_t ld_q;
  __half* f16;
  int pitch;
  unsigned* block_l1;  // with f16: the largest sum of |q| over 128 values
  float* scale;
};

// Any strides, alignments and lengths, THREADS threads a row: two reads of it,
// the second from cache. 200,000 x 65 bf16: 205 us with a CTA a row, 35 with a
// warp; 100,000 x 333: 131 and 33. 30,000 x 2,500 (rows on 8-byte boundaries):
// 84 us, 82 with a row's values kept in registers, which leaves fewer CTAs an
// SM and costs longer and shorter rows a quarter. 8,192 x 14,336, too wide for
// the kernel below: 93 us, 52 for its bytes once.
// J holds a column's number plus a step: unsigned for rows that end within a
// step of 2^31, int for all others (as unsigned numbers 30,000 x 2,500 takes 96).
template <typename T, int THREADS, typename J>
__global__ void __launch_bounds__(kQuantThreads)
    quantize_rows_any_kernel(const T* __restrict__ x, int64_t ld_x, int64_t rows, int cols, const Out o) {
  pdl_launch_dependents();  // a product may become resident now; it waits for these rows
  constexpr int kRows = kQuantThreads / THREADS;
  const J t = threadIdx.x % THREADS, n = cols, pitch = o.pitch;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / THREADS; r < rows; r += static_cast<int64_t>(gridDim.x) * kRows) {
    const T* row = x + r * ld_x;
    uint32_t top = 0;
    for (J j = t; j < n; j += THREADS) top = max(top, __float_as_uint(to_f32(row[j])) & 0x7FFFFFFFu);
    const RowScale s = row_scale(THREADS == 32 ? __reduce_max_sync(kFullMask, top) : block_max(top));
    if (o.f16) {
      for (J j = t; j < pitch; j += THREADS)
        o.f16[r * o.pitch + j] = __float2half_rn(j < n ? quantize_sum(to_f32(row[j]), s) - kRounder : 0.0f);
      if (t == 0) atomicMax(o.block_l1, 128u * 127u);  // the bound of any row: not worth a reduction here
    } else {
      for (J j = t; j < n; j += THREADS)
        o.q[r * o.ld_q + j] = static_cast<int8_t>(__float_as_uint(quantize_sum(to_f32(row[j]), s)));
    }
    if (t == 0) o.scale[r] = s.scale;
    if (THREADS > 32) __syncthreads();  // block_max's shared words are used again
  }
}

// THREADS threads a row (a warp up to 1,024 values, else the CTA up to 8,192),
// which stays in registers: one read of it and one write, eight values a
// thread at a time. Rows start on 16-byte boundaries, int8 rows on 8-byte ones.
// Bound by memory now that a value costs ten instructions (the magnitudes are
// compared as T's own patterns, two a word): 16,384 x 8,192 bf16 60 us =
// 6.73 TB/s, 0.99 of the copy rate (87.7 with fourteen instructions a value);
// 200,000 x 1,024 89; 200,000 x 768 fp32 113; 65,536 x 4,096 bf16 131 (139 with
// six CTAs an SM, the eight need 32 registers).
constexpr int kHeld = 4;  // groups of eight values a thread holds

template <typename T, int THREADS, bool F16>
__global__ void __launch_bounds__(kQuantThreads, sizeof(T) == 2 && THREADS > 32 ? 8 : 1)
    quantize_rows_held_kernel(const T* __restrict__ x, int64_t ld_x, int64_t rows, int cols, const Out o) {
  pdl_launch_dependents();
  constexpr int kRows = kQuantThreads / THREADS;
  const int t = threadIdx.x % THREADS;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / THREADS;
  if (kRows > 1 && r >= rows) return;  // whole warps
  const T* row = x + r * ld_x;
  Eight<T> v[kHeld];
  uint32_t top = 0;
#pragma unroll
  for (int g = 0; g < kHeld; ++g) {
    const int c = (g * THREADS + t) * 8;
    v[g].clear();
    if (c < cols) v[g].load(row + c, cols - c);
  }
#pragma unroll
  for (int g = 0; g < kHeld; ++g) top = v[g].top(top);
  top = Eight<T>::code(top);
  const RowScale s = row_scale(THREADS == 32 ? __reduce_max_sync(kFullMask, top) : block_max(top));
  if (s.pre != 1.0f) {  // few rows: the values are scaled up, or the row has none (inv is 0) and they are zeros
#pragma unroll
    for (int g = 0; g < kHeld; ++g) {
      if (s.inv == 0.0f)
        v[g].clear();
      else
        v[g].scale_by(s.pre);
    }
  }
  if (t == 0) o.scale[r] = s.scale;
  const int end = F16 ? o.pitch : cols;
  float l1_top = 0.0f;
#pragma unroll
  for (int g = 0; g < kHeld; ++g) {
    const int c = (g * THREADS + t) * 8;
    if (c >= end) break;  // whole groups of 16 threads: the pitch is a multiple of 128
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __fadd_rn(__fmul_rn(v[g][i], s.inv), kRounder);
    if constexpr (F16) {
      __half2 h[4];
      float l1 = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float lo = __fsub_rn(q[2 * i], kRounder), hi = __fsub_rn(q[2 * i + 1], kRounder);
        h[i] = __floats2half2_rn(lo, hi);
        l1 += fabsf(lo) + fabsf(hi);
      }
      *reinterpret_cast<uint4*>(o.f16 + r * o.pitch + c) = *reinterpret_cast<const uint4*>(h);
      // 16 threads hold the 128 values of a stage.
      const unsigned half = 0xFFFFu << (threadIdx.x & 16);
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) l1 += __shfl_xor_sync(half, l1, d);
      l1_top = fmaxf(l1_top, l1);
    } else {
      const uint32_t w[2] = {pack_bytes(q[0], q[1], q[2], q[3]), pack_bytes(q[4], q[5], q[6], q[7])};
      int8_t* dst = o.q + r * o.ld_q + c;
      if (c + 8 <= cols) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c + i < cols) dst[i] = static_cast<int8_t>(w[i >> 2] >> (8 * (i & 3)));
      }
    }
  }
  if constexpr (F16) {
    const unsigned l1 = THREADS == 32 ? __reduce_max_sync(kFullMask, static_cast<unsigned>(l1_top))
                                      : block_max(static_cast<unsigned>(l1_top));
    if (t == 0) atomicMax(o.block_l1, l1);
  }
}

template <typename T, bool F16>
cudaError_t launch_t(const QuantizeLaunch& a, cudaStream_t st) {
  Out o;
  o.q = a.q;
  o.ld_q = a.ld_q;
  o.f16 = static_cast<__half*>(a.f16);
  o.pitch = a.f16_pitch;
  o.block_l1 = a.block_l1;
  o.scale = a.scale;
  const T* x = static_cast<const T*>(a.x);
  const bool aligned = (reinterpret_cast<uintptr_t>(a.x) & 15) == 0 && (a.ld_x * sizeof(T)) % 16 == 0 &&
                       (F16 || ((reinterpret_cast<uintptr_t>(a.q) & 7) == 0 && a.ld_q % 8 == 0));
  const int width = F16 ? a.f16_pitch : a.cols;
  if (aligned && width <= 32 * 8 * kHeld) {
    const int64_t grid = (a.rows + kQuantThreads / 32 - 1) / (kQuantThreads / 32);
    quantize_rows_held_kernel<T, 32, F16><<<static_cast<unsigned>(grid), kQuantThreads, 0, st>>>(x, a.ld_x, a.rows, a.cols, o);
  } else if (aligned && width <= kQuantThreads * 8 * kHeld) {
    quantize_rows_held_kernel<T, kQuantThreads, F16><<<static_cast<unsigned>(a.rows), kQuantThreads, 0, st>>>(x, a.ld_x, a.rows, a.cols, o);
  } else if (width <= 32 * 8 * kHeld) {
    const int64_t grid = std::min<int64_t>((a.rows + kQuantThreads / 32 - 1) / (kQuantThreads / 32), int64_t(1) << 20);
    quantize_rows_any_kernel<T, 32, int><<<static_cast<unsigned>(grid), kQuantThreads, 0, st>>>(x, a.ld_x, a.rows, a.cols, o);
  } else {
    const int64_t grid = std::min<int64_t>(a.rows, int64_t(1) << 20);
    auto fn = a.cols > INT32_MAX - kQuantThreads ? quantize_rows_any_kernel<T, kQuantThreads, unsigned> : quantize_rows_any_kernel<T, kQuantThreads, int>;
    fn<<<static_cast<unsigned>(grid), kQuantThreads, 0, st>>>(x, a.ld_x, a.rows, a.cols, o);
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_to(const QuantizeLaunch& a, cudaStream_t st) {
  return a.f16 ? launch_t<T, true>(a, st) : launch_t<T, false>(a, st);
}

}  // namespace

cudaError_t launch_quantize_rows(const QuantizeLaunch& a, cudaStream_t st) {
  if (a.dtype == kF32) return launch_to<float>(a, st);
  if (a.dtype == kBF16) return launch_to<__nv_bfloat16>(a, st);
  return launch_to<__half>(a, st);
}

}  // namespace rbf
