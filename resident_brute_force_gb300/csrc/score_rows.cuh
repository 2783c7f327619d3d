// score_rows.cuh -- rows of scores as the kernels that read whole rows see
// them: 16-byte vectors of any of the three types, arithmetic on pairs of fp32
// numbers, sums of 64-bit integers over a warp, and words sent to another CTA
// of a cluster.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "f32x2.cuh"
#include "rbf_device.cuh"

namespace rbf {

template <typename T>
struct Vec;  // 16 bytes of scores
template <>
struct Vec<float> {
  static constexpr int kLen = 4;
  static constexpr int kSame = 0;  // low bits of a score's code that its type leaves equal
  static constexpr uint32_t kNone = 0xFF800000u;  // -infinity
  static __device__ __forceinline__ void unpack(const uint4& v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ float one(float e) { return e; }
  // Elementwise maximum; a NaN loses to any number.
  static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kLen = 8;
  static constexpr int kSame = 16;
  static constexpr uint32_t kNone = 0xFF80FF80u;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ float one(__nv_bfloat16 e) { return __bfloat162float(e); }
  static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};
template <>
struct Vec<__half> {
  static constexpr int kLen = 8;
  static constexpr int kSame = 13;
  static constexpr uint32_t kNone = 0xFC00FC00u;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ float one(__half e) { return __half2float(e); }
  static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b) {
    const __half2 r = __hmax2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};

template <typename T>
__device__ __forceinline__ uint4 vec_max(const uint4& a, const uint4& b) {
  return make_uint4(Vec<T>::max(a.x, b.x), Vec<T>::max(a.y, b.y), Vec<T>::max(a.z, b.z), Vec<T>::max(a.w, b.w));
}
template <typename T>
__device__ __forceinline__ uint4 vec_none() {
  return make_uint4(Vec<T>::kNone, Vec<T>::kNone, Vec<T>::kNone, Vec<T>::kNone);
}

// The largest score of a vector.
template <typename T>
__device__ __forceinline__ float vec_top(const uint4& v) {
  float x[Vec<T>::kLen];
  if constexpr (sizeof(T) == 2) {
    const uint32_t m = Vec<T>::max(Vec<T>::max(v.x, v.y), Vec<T>::max(v.z, v.w));
    Vec<T>::unpack(make_uint4(m, m, m, m), x);
    return fmaxf(x[0], x[1]);
  } else {
    Vec<T>::unpack(v, x);
    return fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
  }
}

// Scores i0 .. i0 + kLen - 1 of a row of n, -infinity where there are none; out
// of line, for the one or two vectors of a row that reach past it.
template <typename T>
__device__ __noinline__ uint4 load_edge(const T* p, int i0, int n) {
  uint4 r = vec_none<T>();
  T* e = reinterpret_cast<T*>(&r);
#pragma unroll 1
  for (int i = 0; i < Vec<T>::kLen; ++i)
    if (i0 + i >= 0 && i0 + i < n) e[i] = p[i0 + i];
  return r;
}

// A row as 16-byte vectors on 16-byte boundaries: vector v holds the elements
// v * kLen - lead .. of it. The vectors at either end may reach past the row;
// those are read element by element, -infinity outside. A NaN becomes -infinity.
template <typename T>
struct Row {
  const T* p;
  int n, lead, vecs;

  __device__ __forceinline__ Row(const T* row, int len) : p(row), n(len) {
    lead = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    vecs = (n + lead + Vec<T>::kLen - 1) / Vec<T>::kLen;
  }
  __device__ __forceinline__ uint4 load(int v) const {
    const int i0 = v * Vec<T>::kLen - lead;
    if (i0 >= 0 && i0 + Vec<T>::kLen <= n) return vec_max<T>(*reinterpret_cast<const uint4*>(p + i0), vec_none<T>());
    return vec_max<T>(load_edge(p, i0, n), vec_none<T>());
  }
};

__device__ __forceinline__ float ex2(float z) {  // exp2f where the result is not subnormal, 0 there
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(z));
  return r;
}

// total * part / 2^30, rounded down.
__device__ __forceinline__ u64 share(u64 total, u64 part) {
  return (__umul64hi(total, part) << 34) | ((total * part) >> 30);
}

// Sum over the warp, in three parts of 26 bits: 32 of each stay under 2^31.
__device__ __forceinline__ u64 warp_sum(u64 v) {
  constexpr u64 kPart = (u64(1) << 26) - 1;
  const u64 a = __reduce_add_sync(kFullMask, static_cast<unsigned>(v & kPart));
  const u64 b = __reduce_add_sync(kFullMask, static_cast<unsigned>(v >> 26 & kPart));
  const u64 c = __reduce_add_sync(kFullMask, static_cast<unsigned>(v >> 52));
  return a + (b << 26) + (c << 52);
}
__device__ __forceinline__ u64 warp_max(u64 v) {
  const unsigned hi = __reduce_max_sync(kFullMask, static_cast<unsigned>(v >> 32));
  const unsigned lo = __reduce_max_sync(kFullMask, static_cast<unsigned>(v >> 32) == hi ? static_cast<unsigned>(v) : 0u);
  return static_cast<u64>(hi) << 32 | lo;
}
template <typename V>
__device__ __forceinline__ V warp_scan(V v, int lane) {  // inclusive
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const V o = __shfl_up_sync(kFullMask, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void remote_store(uint32_t a, u64 v) {
  asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}

}  // namespace rbf
