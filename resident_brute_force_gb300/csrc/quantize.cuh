// quantize.cuh -- the arithmetic of the 8-bit row quantisation, shared by the
// kernels that quantise.
//
// With t = max_j |x_j|: scale = t * (1 / 127), q_j = x_j * ((1 / t) * 127)
// rounded to nearest even, all in fp32 (one division a row, one product a
// value, each rounded as IEEE says, so that the integers are the same wherever
// they are computed). |q| <= 127: x_j times the factor is at most
// 127 (1 + 2^-22), which rounds to 127.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

namespace rbf {

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

// The quantised value plus 1.5 * 2^23: adding that rounds to a whole number
// (halves to even), whose two's complement is the sum's low byte.
constexpr float kRounder = 12582912.0f;
__device__ __forceinline__ float quantize_sum(float x, const RowScale& r) {
  return r.inv != 0.0f ? __fadd_rn(__fmul_rn(__fmul_rn(x, r.pre), r.inv), kRounder) : kRounder;  // no 0 * infinity
}

// The low bytes of four such sums.
__device__ __forceinline__ uint32_t pack_bytes(float a, float b, float c, float d) {
  const uint32_t lo = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040);
  const uint32_t hi = __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}

// Eight values as they are in memory, read from a 16-byte boundary, zero from
// `live` on.
template <typename T>
struct Eight {
  uint4 raw[sizeof(T) / 2];

  __device__ __forceinline__ void load(const T* p, int live) {
    if (live >= 8) {
#pragma unroll
      for (unsigned i = 0; i < sizeof(T) / 2; ++i) raw[i] = reinterpret_cast<const uint4*>(p)[i];
    } else {
      clear();
      T* e = reinterpret_cast<T*>(raw);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < live) e[i] = p[i];
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (unsigned i = 0; i < sizeof(T) / 2; ++i) raw[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  // Words 0 .. 2 sizeof(T) - 1 as they are in memory.
  __device__ __forceinline__ uint32_t& word(int i) { return reinterpret_cast<uint32_t*>(raw)[i]; }
  __device__ __forceinline__ float operator[](int i) const { return to_f32(reinterpret_cast<const T*>(raw)[i]); }
  // The largest magnitude so far as T's own pattern (16-bit types: in each
  // half), and that as the fp32 pattern that row_scale takes.
  __device__ __forceinline__ uint32_t top(uint32_t t) {
#pragma unroll
    for (unsigned i = 0; i < 2 * sizeof(T); ++i)
      t = sizeof(T) == 4 ? max(t, word(i) & 0x7FFFFFFFu) : __vmaxu2(t, word(i) & 0x7FFF7FFFu);
    return t;
  }
  static __device__ __forceinline__ uint32_t code(uint32_t t) {
    if constexpr (sizeof(T) == 4) return t;
    const uint32_t one = max(t >> 16, t & 0xFFFFu);
    if constexpr (std::is_same_v<T, __nv_bfloat16>) return one << 16;
    return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(one))));
  }
  // The values times `pre`, a power of two that leaves them within T (exact).
  __device__ __forceinline__ void scale_by(float pre) {
    T* e = reinterpret_cast<T*>(raw);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (sizeof(T) == 4) e[i] *= pre;
      if constexpr (std::is_same_v<T, __nv_bfloat16>) e[i] = __float2bfloat16_rn(__bfloat162float(e[i]) * pre);
    }
  }
};

}  // namespace rbf
