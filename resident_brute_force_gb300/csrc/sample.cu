// sample.cu -- one index a row, drawn from its scores with temperature, top-k,
// top-p and min-p (include/rbf_ops.h, sample_dev).
//
// Weights. e_j = 2^((x_j - max x) log2(e) / T) in fp32, held as w_j = e_j
// rounded to a whole multiple of 2^-36 (halves to even). Every sum of weights
// is then a sum of 64-bit integers: exact, and the same for every split of the
// row over threads. The rounding is 2^-37 of the largest weight at most; all
// of a row of 2^26 scores stays below 2^62.
//
// Order. The 64-bit keys of rbf_device.cuh put a row in the order of the
// search (higher score first, lower index on a tie). top_k keeps the keys from
// K_k = max{K : #(key >= K) >= k} on; top_p those from
// K_p = max{K : w(key >= K, key >= K_k) >= top_p * w(key >= K_k)} on (the
// shortest prefix that reaches top_p); both are found by halving the interval
// of keys, one pass over the row a step. min_p is a test on e itself.
//
// Choice. With W the kept sum and r = floor(W * u), the index is the first one
// whose running kept sum exceeds r. Each warp owns a contiguous part of the
// row, so its sum says whether r falls into it; the part that holds r is
// divided among the warps again until one warp has it in its lanes.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "ops_internal.h"
#include "rbf_device.cuh"

namespace rbf {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kOne = 68719476736.0f;  // 2^36: the largest weight

using u64 = unsigned long long;

template <typename T>
struct Vec;  // 16 bytes of scores
template <>
struct Vec<float> {
  static constexpr int kLen = 4;
  static constexpr uint32_t kNone = 0xFF800000u;  // -infinity
  static __device__ __forceinline__ void unpack(const uint4& v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kLen = 8;
  static constexpr uint32_t kNone = 0xFF80FF80u;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct Vec<__half> {
  static constexpr int kLen = 8;
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
};

// A row as 16-byte vectors on 16-byte boundaries: vector v holds the elements
// v * kLen - lead .. of it. The vectors at either end may reach past the row;
// those are read element by element, -infinity outside.
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
    if (i0 >= 0 && i0 + Vec<T>::kLen <= n) return *reinterpret_cast<const uint4*>(p + i0);
    uint4 r = make_uint4(Vec<T>::kNone, Vec<T>::kNone, Vec<T>::kNone, Vec<T>::kNone);
    T* e = reinterpret_cast<T*>(&r);
#pragma unroll
    for (int i = 0; i < Vec<T>::kLen; ++i)
      if (i0 + i >= 0 && i0 + i < n) e[i] = p[i0 + i];
    return r;
  }
};

// What a row asks for.
struct Ask {
  float rate;    // log2(e) / T
  int k;         // indices that top_k keeps
  u64 part_p;    // top_p in 2^-30ths (2^30: all)
  float min_p;
  u64 part_u;    // u in 2^-30ths
};

__device__ __forceinline__ Ask read_ask(const SampleLaunch& a, int64_t r) {
  Ask q;
  const float t = a.temperature ? a.temperature[r] : 1.0f;
  const bool warm = t > 0.0f;  // also false for a NaN
  // An infinite temperature would make (-infinity) * 0 of a masked score.
  q.rate = warm ? fmaxf(__fdiv_rn(kLog2e, t), 1.17549435e-38f) : kLog2e;
  const int k = a.top_k ? a.top_k[r] : 0;
  q.k = !warm ? 1 : (k > 0 && k < a.vocab ? k : a.vocab);
  const float p = a.top_p ? a.top_p[r] : 1.0f;
  q.part_p = p < 1.0f ? static_cast<u64>(rintf(fmaxf(p, 0.0f) * 0x1p30f)) : u64(1) << 30;
  const float mp = a.min_p ? a.min_p[r] : 0.0f;
  q.min_p = mp > 0.0f ? mp : 0.0f;
  const float u = a.u[r];
  const float uf = u > 0.0f ? fminf(floorf(u * 0x1p30f), 1073741824.0f) : 0.0f;
  q.part_u = min(static_cast<u64>(uf), (u64(1) << 30) - 1);
  return q;
}

// total * part / 2^30, rounded down.
__device__ __forceinline__ u64 share(u64 total, u64 part) {
  return (__umul64hi(total, part) << 34) | ((total * part) >> 30);
}

__device__ __forceinline__ float weight_f(float x, float top, float rate) {
  if (x == top) return 1.0f;
  return x > top || x < top ? exp2f(__fmul_rn(__fsub_rn(x, top), rate)) : 0.0f;  // a NaN has no weight
}
__device__ __forceinline__ u64 fixed(float e) { return static_cast<u64>(__float2ll_rn(__fmul_rn(e, kOne))); }

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(kFullMask, v, m);
  return v;
}
__device__ __forceinline__ u64 warp_max(u64 v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v = umax64(v, __shfl_xor_sync(kFullMask, v, m));
  return v;
}

struct Shared {
  u64 part[kWarps];
  u64 warp[kWarps];  // the warps' kept sums
  int lo, hi;        // the vectors that still may hold the choice
  u64 before;        // kept sum ahead of them
};

template <bool MAX>
__device__ __forceinline__ u64 block_reduce(u64 v, Shared& s) {
  v = MAX ? warp_max(v) : warp_sum(v);
  __syncthreads();  // the words of the last reduction have been read
  if ((threadIdx.x & 31) == 0) s.part[threadIdx.x >> 5] = v;
  __syncthreads();
  u64 r = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) r = MAX ? umax64(r, s.part[w]) : r + s.part[w];
  return r;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleLaunch a) {
  constexpr int E = Vec<T>::kLen;
  __shared__ Shared s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const Row<T> row(static_cast<const T*>(a.logits) + r * a.ld, a.vocab);
    const Ask q = read_ask(a, r);
    // f(key, score) of every element of vectors [v0, v1), lane by lane.
    auto each = [&](int v0, int v1, auto&& f) {
      for (int v = v0 + lane; v < v1; v += 32) {
        const uint4 raw = row.load(v);
        float x[E];
        Vec<T>::unpack(raw, x);
#pragma unroll
        for (int i = 0; i < E; ++i) f(make_key(x[i], static_cast<uint32_t>(v * E - row.lead + i)), x[i]);
      }
    };
    const int v0 = static_cast<int>(int64_t(row.vecs) * warp / kWarps);
    const int v1 = static_cast<int>(int64_t(row.vecs) * (warp + 1) / kWarps);

    u64 best = 0;
    each(v0, v1, [&](u64 key, float x) {
      if (x > -INFINITY) best = umax64(best, key);
    });
    const u64 top_key = block_reduce<true>(best, s);
    if (top_key == 0) {  // nothing but -infinity
      if (threadIdx.x == 0) {
        a.token[r] = -1;
        if (a.logprob) a.logprob[r] = -INFINITY;
      }
      continue;
    }
    const float top = key_score(top_key);

    u64 cut = 0;
    if (q.k < a.vocab) {
      u64 lo = 0, hi = top_key + 1;
      while (hi - lo > 1) {
        const u64 mid = lo + (hi - lo) / 2;
        u64 c = 0;
        each(v0, v1, [&](u64 key, float) { c += key >= mid; });
        if (block_reduce<false>(c, s) >= static_cast<u64>(q.k))
          lo = mid;
        else
          hi = mid;
      }
      cut = lo;
    }
    auto mass_from = [&](u64 from) {
      u64 w = 0;
      each(v0, v1, [&](u64 key, float x) {
        if (key >= from) w += fixed(weight_f(x, top, q.rate));
      });
      return block_reduce<false>(w, s);
    };
    if (q.part_p < (u64(1) << 30)) {
      const u64 target = share(mass_from(cut), q.part_p);
      u64 lo = cut, hi = top_key + 1;
      if (target == 0) lo = top_key;
      while (hi - lo > 1) {
        const u64 mid = lo + (hi - lo) / 2;
        if (mass_from(mid) >= target)
          lo = mid;
        else
          hi = mid;
      }
      cut = lo;
    }

    // The kept weight of an element.
    auto kept = [&](u64 key, float x) -> u64 {
      const float e = weight_f(x, top, q.rate);
      return key >= cut && (e >= q.min_p || key == top_key) ? fixed(e) : 0ull;
    };
    u64 w = 0;
    each(v0, v1, [&](u64 key, float x) { w += kept(key, x); });
    const u64 total = block_reduce<false>(w, s);
    const u64 aim = share(total, q.part_u);
    // Narrow the vectors that hold the choice: s.part has the warps' sums over
    // the 16 equal parts of [lo, hi).
    if (threadIdx.x == 0) {
      s.lo = 0;
      s.hi = row.vecs;
      s.before = 0;
    }
    __syncthreads();
    for (;;) {
      const int lo = s.lo, len = s.hi - s.lo;
      const u64 before = s.before;
      u64 upto = before;
      int in = 0;
      while (in < kWarps - 1 && upto + s.part[in] <= aim) upto += s.part[in++];
      const int n0 = lo + static_cast<int>(int64_t(len) * in / kWarps);
      const int n1 = lo + static_cast<int>(int64_t(len) * (in + 1) / kWarps);
      __syncthreads();
      if (threadIdx.x == 0) {
        s.lo = n0;
        s.hi = n1;
        s.before = upto;
      }
      if (n1 - n0 <= 32) break;
      u64 part = 0;
      each(n0 + static_cast<int>(int64_t(n1 - n0) * warp / kWarps), n0 + static_cast<int>(int64_t(n1 - n0) * (warp + 1) / kWarps),
           [&](u64 key, float x) { part += kept(key, x); });
      part = warp_sum(part);
      if (lane == 0) s.part[warp] = part;
      __syncthreads();
    }
    __syncthreads();
    if (warp == 0) {
      const int v = s.lo + lane;
      u64 mine[E];
      u64 sum = 0;
      if (v < s.hi) {
        float x[E];
        Vec<T>::unpack(row.load(v), x);
#pragma unroll
        for (int i = 0; i < E; ++i) {
          mine[i] = kept(make_key(x[i], static_cast<uint32_t>(v * E - row.lead + i)), x[i]);
          sum += mine[i];
        }
      }
      u64 upto = sum;  // inclusive over the lanes
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const u64 o = __shfl_up_sync(kFullMask, upto, d);
        if (lane >= d) upto += o;
      }
      u64 run = s.before + upto - sum;
      if (sum > 0 && run <= aim && aim < run + sum) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
          if (run <= aim && aim < run + mine[i]) {
            a.token[r] = v * E - row.lead + i;
            if (a.logprob) {
              const float share_of = __fdiv_rn(__ull2float_rn(mine[i]), __ull2float_rn(total));
              const float rest = __fdiv_rn(__ull2float_rn(total - mine[i]), __ull2float_rn(total));
              a.logprob[r] = 2 * mine[i] < total ? logf(share_of) : log1pf(-rest);
            }
          }
          run += mine[i];
        }
      }
    }
    __syncthreads();
  }
}

template <typename T>
cudaError_t launch_t(const SampleLaunch& a, cudaStream_t st) {
  const int64_t grid = std::min<int64_t>(a.rows, int64_t(1) << 20);
  sample_kernel<T><<<static_cast<unsigned>(grid), kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_sample(const SampleLaunch& a, cudaStream_t st) {
  if (a.dtype == kF32) return launch_t<float>(a, st);
  if (a.dtype == kBF16) return launch_t<__nv_bfloat16>(a, st);
  return launch_t<__half>(a, st);
}

}  // namespace rbf
