// quantize_f8.cu -- rows to 8-bit floating point with a scale for each block of
// 128 values of a row, or of 128 x 128 (include/rbf_ops.h, quantize_f8_dev).
//
// With t = max |x| over the block and MAX the type's largest number:
//   scale = t * (1 / MAX),  q = x * ((1 / t) * MAX) rounded to the nearest 8-bit number,
// in fp32, each step rounded as IEEE says, so that the bytes are the same
// wherever they are computed. |x| times the factor is at most MAX (1 + 2^-22), which
// rounds to MAX. A block so small that the factor passes 2^127 takes that and 2^-127.
//
// One pass: a block is held between its maximum and its rounding.
// Blocks of a row: 16 lanes (fp32: 32) a block, 16 bytes a lane, four blocks a
// lane under way in registers, and no division but the scales'. Blocks of 128 x 128: a CTA each,
// 32 KB (fp32: 64) in its threads' registers and, as six CTAs of 256 threads an SM leave 40
// of those a thread and two of 512 leave 64, partly in local memory: bf16 stores 80 bytes a
// thread there, fp16, whose values are unpacked by conversions, 384, fp32 24.
// What bounds it: HBM, and for fp16's blocks that local memory. 8192 x 8192 bf16 and fp16: 40.0 and
// 39.5 us by rows, 37.5 and 44.8 by blocks (30 for the bytes at the copy rate); fp32 4096 x 8192
// 33.1 and 29.5 (25).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "ops_internal.h"
#include "rbf_device.cuh"

namespace rbf {
namespace {

constexpr int kBlock = 128;

template <typename T>
constexpr int kLen = 16 / sizeof(T);  // values of a lane's 16 bytes

// Magnitudes as their fp32 patterns: ordered as unsigned integers, the
// infinities and the NaNs on top.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

struct BlockScale {
  float scale, inv;
};
template <__nv_fp8_interpretation_t F8>
__device__ __forceinline__ BlockScale block_scale(uint32_t code) {
  constexpr float top = F8 == __NV_E4M3 ? 448.0f : 57344.0f;
  BlockScale s;
  if (code >= 0x7F800000u) {  // a NaN or an infinity: zeros, and a scale that makes every product NaN
    s.scale = __uint_as_float(0x7FC00000u);
    s.inv = 0.0f;
  } else if (code == 0) {
    s.scale = s.inv = 0.0f;
  } else {
    const float t = __uint_as_float(code);
    s.inv = __fmul_rn(__fdiv_rn(1.0f, t), top);
    s.scale = __fmul_rn(t, 1.0f / top);
    if (s.inv > 0x1p127f) {
      s.inv = 0x1p127f;
      s.scale = 0x1p-127f;
    }
  }
  return s;
}

template <typename T>
__device__ __forceinline__ void unpack(const uint4& v, float (&x)[kLen<T>]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      x[i] = __uint_as_float(w[i]);
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

// kLen values from column c on of a row of `cols` (0 past it).
// WHOLE: every piece lies within the row and on its boundary. (Column numbers are
// unsigned: a row's last block may reach past 2^31.)
template <bool WHOLE, typename T>
__device__ __forceinline__ uint4 load_piece(const T* row, uint32_t c, uint32_t cols, bool wide) {
  if (WHOLE || (wide && c + kLen<T> <= cols)) return __ldcs(reinterpret_cast<const uint4*>(row + c));
  uint4 r = make_uint4(0u, 0u, 0u, 0u);
  T* e = reinterpret_cast<T*>(&r);
#pragma unroll
  for (int i = 0; i < kLen<T>; ++i)
    if (c + i < cols) e[i] = row[c + i];
  return r;
}

template <typename T>
__device__ __forceinline__ uint32_t piece_top(const uint4& v) {
  float x[kLen<T>];
  unpack<T>(v, x);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kLen<T>; ++i) m = max(m, magnitude(x[i]));
  return m;
}

template <bool WHOLE, typename T, __nv_fp8_interpretation_t F8>
__device__ __forceinline__ void store_piece(uint8_t* row, uint32_t c, uint32_t cols, bool wide, const uint4& v, float inv) {
  float x[kLen<T>];
  unpack<T>(v, x);
  uint16_t h[kLen<T> / 2];
#pragma unroll
  for (int i = 0; i < kLen<T> / 2; ++i) {
    const float a = inv != 0.0f ? __fmul_rn(x[2 * i], inv) : 0.0f, b = inv != 0.0f ? __fmul_rn(x[2 * i + 1], inv) : 0.0f;
    h[i] = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, F8);
  }
  if (WHOLE || (wide && c + kLen<T> <= cols)) {
    if constexpr (kLen<T> == 8)
      *reinterpret_cast<uint2*>(row + c) = make_uint2(h[0] | static_cast<uint32_t>(h[1]) << 16, h[2] | static_cast<uint32_t>(h[3]) << 16);
    else
      *reinterpret_cast<uint32_t*>(row + c) = h[0] | static_cast<uint32_t>(h[1]) << 16;
    return;
  }
#pragma unroll
  for (int i = 0; i < kLen<T>; ++i)
    if (c + i < cols) row[c + i] = static_cast<uint8_t>(h[i / 2] >> (8 * (i & 1)));
}

// Whether a matrix' rows start on boundaries of `bytes`.
__device__ __forceinline__ bool rows_on(const void* p, int64_t ld_bytes, int bytes) {
  return ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld_bytes)) & static_cast<uintptr_t>(bytes - 1)) == 0;
}

constexpr int kThreads = 256;
constexpr int kRowCtas = 4;  // an SM: rounds of warps that go on, not of new CTAs

template <typename T>
constexpr int kGroup = 4 * 32 / (kBlock / kLen<T>);  // blocks of a warp: four a lane

// A warp takes a group of blocks of one row at a time; a row has 2^bits of them.
// The next group's values are on their way while this one's are rounded.
template <typename T, __nv_fp8_interpretation_t F8>
__global__ void __launch_bounds__(kThreads) quantize_f8_rows_kernel(const QuantizeF8Launch a, int bits) {
  constexpr int kLanes = kBlock / kLen<T>;  // of a block
  constexpr int kAhead = 4;                 // blocks a lane
  const T* x = static_cast<const T*>(a.x);
  uint8_t* q = static_cast<uint8_t*>(a.q);
  const bool wide_x = rows_on(x, a.ld_x * static_cast<int64_t>(sizeof(T)), 16), wide_q = rows_on(q, a.ld_q, kLen<T>);
  const int per = (a.cols - 1) / kBlock + 1;
  const int lane = threadIdx.x & 31, sub = lane % kLanes;
  const int64_t all = a.rows << bits, step = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  struct Group {
    int64_t r;
    int b0;  // this lane's first block
    bool whole;
  };
  auto group_of = [&](int64_t u) {
    Group g;
    g.r = u >> bits;
    const int b0 = static_cast<int>(u & ((int64_t(1) << bits) - 1)) * kGroup<T>;
    g.b0 = b0 + lane / kLanes;
    g.whole = wide_x && wide_q && static_cast<uint32_t>(b0 + kGroup<T>) * kBlock <= static_cast<uint32_t>(a.cols);
    return g;
  };
  auto load = [&](const Group& g, uint4 (&v)[kAhead]) {
    const T* row = x + g.r * a.ld_x;
    if (g.whole) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) v[j] = load_piece<true>(row, static_cast<uint32_t>(g.b0 + j * (32 / kLanes)) * kBlock + sub * kLen<T>, a.cols, true);
    } else {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int b = g.b0 + j * (32 / kLanes);
        v[j] = b < per ? load_piece<false>(row, static_cast<uint32_t>(b) * kBlock + sub * kLen<T>, a.cols, wide_x) : make_uint4(0u, 0u, 0u, 0u);
      }
    }
  };
  int64_t u = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  if (u >= all) return;
  Group g = group_of(u);
  uint4 v[kAhead];
  load(g, v);
  for (;;) {
    u += step;
    const bool more = u < all;
    Group next = g;
    uint4 ahead[kAhead];
    if (more) {
      next = group_of(u);
      load(next, ahead);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int b = g.b0 + j * (32 / kLanes);
      const uint32_t c = static_cast<uint32_t>(b) * kBlock + sub * kLen<T>;
      uint32_t m = piece_top<T>(v[j]);
#pragma unroll
      for (int d = kLanes / 2; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(kFullMask, m, d));
      const BlockScale s = block_scale<F8>(m);
      if (g.whole)
        store_piece<true, T, F8>(q + g.r * a.ld_q, c, a.cols, true, v[j], s.inv);
      else if (b < per)
        store_piece<false, T, F8>(q + g.r * a.ld_q, c, a.cols, wide_q, v[j], s.inv);
      if (sub == 0 && b < per) a.scale[g.r * a.ld_scale + b] = s.scale;
    }
    if (!more) break;
    g = next;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) v[j] = ahead[j];
  }
}

template <typename T>
constexpr int kTileThreads = sizeof(T) == 2 ? 256 : 512;

template <typename T, __nv_fp8_interpretation_t F8>
__global__ void __launch_bounds__(kTileThreads<T>, sizeof(T) == 2 ? 6 : 2) quantize_f8_blocks_kernel(const QuantizeF8Launch a) {
  constexpr int kLanes = kBlock / kLen<T>;
  constexpr int kRows = kTileThreads<T> / kLanes;  // of a pass
  constexpr int kPasses = kBlock / kRows;
  __shared__ uint32_t part[kTileThreads<T> / 32];
  const T* x = static_cast<const T*>(a.x);
  uint8_t* q = static_cast<uint8_t*>(a.q);
  const bool wide_x = rows_on(x, a.ld_x * static_cast<int64_t>(sizeof(T)), 16), wide_q = rows_on(q, a.ld_q, kLen<T>);
  const int per = (a.cols - 1) / kBlock + 1;
  const int bi = static_cast<int>(blockIdx.x) / per, bj = static_cast<int>(blockIdx.x) - bi * per;
  const bool whole = wide_x && wide_q && static_cast<uint32_t>(bj + 1) * kBlock <= static_cast<uint32_t>(a.cols) && int64_t(bi + 1) * kBlock <= a.rows;
  const int64_t r0 = static_cast<int64_t>(bi) * kBlock + threadIdx.x / kLanes;
  const uint32_t c = static_cast<uint32_t>(bj) * kBlock + threadIdx.x % kLanes * kLen<T>;
  auto tile = [&](auto is_whole) {
    constexpr bool kWhole = decltype(is_whole)::value;
    uint4 v[kPasses];
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int64_t r = r0 + p * kRows;
      v[p] = kWhole || r < a.rows ? load_piece<kWhole>(x + r * a.ld_x, c, a.cols, wide_x) : make_uint4(0u, 0u, 0u, 0u);
    }
    uint32_t m = 0;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) m = max(m, piece_top<T>(v[p]));
    m = __reduce_max_sync(kFullMask, m);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
    m = __reduce_max_sync(kFullMask, part[(threadIdx.x & 31) % (kTileThreads<T> / 32)]);
    const BlockScale s = block_scale<F8>(m);
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int64_t r = r0 + p * kRows;
      if (kWhole || r < a.rows) store_piece<kWhole, T, F8>(q + r * a.ld_q, c, a.cols, wide_q, v[p], s.inv);
    }
    if (threadIdx.x == 0) a.scale[static_cast<int64_t>(bi) * a.ld_scale + bj] = s.scale;
  };
  if (whole)
    tile(std::true_type{});
  else
    tile(std::false_type{});
}

template <typename T, __nv_fp8_interpretation_t F8>
cudaError_t launch_t(const QuantizeF8Launch& a, int num_sms, cudaStream_t st) {
  const int per = (a.cols - 1) / kBlock + 1;
  if (a.block_rows == 1) {
    int bits = 0;
    while (int64_t(kGroup<T>) << bits < per) ++bits;
    const int64_t ctas = std::min<int64_t>(((a.rows << bits) + kThreads / 32 - 1) / (kThreads / 32), int64_t(num_sms) * kRowCtas);
    quantize_f8_rows_kernel<T, F8><<<static_cast<unsigned>(ctas), kThreads, 0, st>>>(a, bits);
  } else {
    // Rows past what one grid takes go in parts of whole blocks.
    const int64_t most = (int64_t(1) << 30) / per * kBlock;
    for (int64_t r = 0; r < a.rows; r += most) {
      QuantizeF8Launch p = a;
      p.rows = std::min(most, a.rows - r);
      p.x = static_cast<const T*>(a.x) + r * a.ld_x;
      p.q = static_cast<uint8_t*>(a.q) + r * a.ld_q;
      p.scale = a.scale + r / kBlock * a.ld_scale;
      quantize_f8_blocks_kernel<T, F8><<<static_cast<unsigned>((p.rows + kBlock - 1) / kBlock * per), kTileThreads<T>, 0, st>>>(p);
    }
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_f8(const QuantizeF8Launch& a, int num_sms, cudaStream_t st) {
  return a.q_dtype == kE4M3 ? launch_t<T, __NV_E4M3>(a, num_sms, st) : launch_t<T, __NV_E5M2>(a, num_sms, st);
}

}  // namespace

cudaError_t launch_quantize_f8(const QuantizeF8Launch& a, int num_sms, cudaStream_t st) {
  if (a.dtype == kF32) return launch_f8<float>(a, num_sms, st);
  if (a.dtype == kBF16) return launch_f8<__nv_bfloat16>(a, num_sms, st);
  return launch_f8<__half>(a, num_sms, st);
}

}  // namespace rbf
