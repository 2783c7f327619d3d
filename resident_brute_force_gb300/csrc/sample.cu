// sample.cu -- one index a row, drawn from its scores with temperature, top-k,
// top-p and min-p (include/rbf_ops.h, sample_dev).
//
// Weights. e_j = 2^z_j, z_j = (x_j - max x) log2(e) / T in fp32, held as w_j =
// e_j rounded to a whole multiple of 2^-36 (halves to even). Every sum of
// weights is then a sum of 64-bit integers: exact, and the same for every split
// of the row over threads and every order of atomics. The rounding is 2^-37 of
// the largest weight at most; a row of 2^26 scores stays below 2^62. An index
// with z < -37 has no weight.
//
// Order. The 64-bit keys of rbf_device.cuh put a row in the order of the search
// (higher score first, lower index on a tie). top_k and top_p keep a prefix of
// that order, which ends at a key K:
//   top_k  K = max{K : #(key >= K) >= k}
//   top_p  K = max{K : w(key >= K) >= top_p * w(what top_k kept)}
// min_p is a test on e itself.
//
// Choice. With W the kept sum and r = floor(W * u), the index is the first one
// whose running kept sum exceeds r.
//
// How. A cluster of 1 to 16 CTAs takes a row; each CTA holds its part in
// shared memory where that fits (else it reads it again, from L2) and each
// warp owns a contiguous part of that.
//   1. One read from memory finds the largest score.
//   2. Without top_k and top_p a second pass sums the weights, per warp.
//   3. Else the second pass counts the scores in bins of 2^(1/64) in weight.
//      The counts give the bin in which top_k ends, and bounds on the sum of
//      weights above each bin edge that leave two or three bins in which top_p
//      can end; if these hold more than a list, they are divided again.
//      a. If all indices down to there fit a list (kListCap), they are
//         gathered and one CTA finishes the row in it: sorted by key it knows
//         the kept prefix, sorted again by index the choice.
//      b. Else a third pass sums the weights above those bins, per warp, and
//         gathers the scores in them; sorted, they give the key K.
//   4. The warps' kept sums say which warp's part holds r; that part is divided
//      among the warps again until one warp has it in its lanes.
// Rows whose scores coincide so often that no bins divide them (thousands of
// equal ones around the end of the prefix) find K by halving the interval of
// keys, one pass over the row a step.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "ops_internal.h"
#include "rbf_device.cuh"
#include "rbf_internal.h"

namespace rbf {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kOne = 68719476736.0f;  // 2^36: the largest weight
constexpr int kBinsPerOctave = 64;
constexpr int kBins = 37 * kBinsPerOctave + 1;  // z = 0 .. -37, rounded
constexpr int kBinsPerThread = (kBins + kThreads - 1) / kThreads;
constexpr int kListCap = 2048;

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
  // Elementwise maximum; a NaN loses to any number.
  static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
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
  static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
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
    uint4 r = vec_none<T>();
    T* e = reinterpret_cast<T*>(&r);
#pragma unroll
    for (int i = 0; i < Vec<T>::kLen; ++i)
      if (i0 + i >= 0 && i0 + i < n) e[i] = p[i0 + i];
    return vec_max<T>(r, vec_none<T>());
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
constexpr u64 kAll = u64(1) << 30;

__device__ __forceinline__ Ask read_ask(const SampleLaunch& a, int64_t r) {
  Ask q;
  const float t = a.temperature ? a.temperature[r] : 1.0f;
  const bool warm = t > 0.0f;  // also false for a NaN
  // An infinite temperature would make (-infinity) * 0 of a masked score.
  q.rate = warm ? fmaxf(__fdiv_rn(kLog2e, t), 1.17549435e-38f) : kLog2e;
  const int k = a.top_k ? a.top_k[r] : 0;
  q.k = !warm ? 1 : (k > 0 && k < a.vocab ? k : a.vocab);
  const float p = a.top_p ? a.top_p[r] : 1.0f;
  q.part_p = p < 1.0f ? static_cast<u64>(rintf(fmaxf(p, 0.0f) * 0x1p30f)) : kAll;
  const float mp = a.min_p ? a.min_p[r] : 0.0f;
  q.min_p = mp > 0.0f ? mp : 0.0f;
  // Where only the best index can stay, it is the one that top_k = 1 keeps.
  if (q.part_p == 0 || q.min_p > 1.0f) q.k = 1;
  const float u = a.u[r];
  const float uf = u > 0.0f ? fminf(floorf(u * 0x1p30f), 1073741824.0f) : 0.0f;
  q.part_u = min(static_cast<u64>(uf), kAll - 1);
  return q;
}

// total * part / 2^30, rounded down.
__device__ __forceinline__ u64 share(u64 total, u64 part) {
  return (__umul64hi(total, part) << 34) | ((total * part) >> 30);
}

// ---------------------------------------------------------------- weights

// Two fp32 numbers in a register pair, one instruction for both, each rounded
// as the single instruction rounds.
__device__ __forceinline__ u64 pack2(float a, float b) {
  u64 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float low2(u64 v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float high2(u64 v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
  u64 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ u64 mul2(u64 a, u64 b) {
  u64 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) {
  u64 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float ex2(float z) {  // exp2f where the result is not subnormal, 0 there
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(z));
  return r;
}

// The scale of a row's weights. A largest score of +infinity leaves only the
// scores that equal it: they become 0 and the others -infinity.
struct Scale {
  float top, rate;
  bool inf;
  u64 ntop2, rate2;
  __device__ __forceinline__ Scale(float t, float r) : top(t), rate(r), inf(t == INFINITY) {
    if (inf) top = 0.0f;
    ntop2 = pack2(-top, -top);
    rate2 = pack2(rate, rate);
  }
  __device__ __forceinline__ float shift(float x) const { return inf ? (x == INFINITY ? 0.0f : -INFINITY) : x; }
  // z of two scores.
  __device__ __forceinline__ u64 z2(float a, float b) const { return mul2(add2(pack2(shift(a), shift(b)), ntop2), rate2); }
  __device__ __forceinline__ float z(float x) const { return __fmul_rn(__fsub_rn(shift(x), top), rate); }
};

__device__ __forceinline__ u64 fixed(float e) { return static_cast<u64>(__float2ll_rn(__fmul_rn(e, kOne))); }
__device__ __forceinline__ u64 weight(float x, const Scale& s) { return fixed(ex2(s.z(x))); }

// A sum of weights. e is divided into a multiple of 2^-18 and a rest that is
// rounded to a multiple of 2^-36 (adding and subtracting 1.5 * 2^23 units
// rounds to units, halves to even); both parts are summed in fp32, exactly, for
// up to 64 weights a lane of the pair, then moved into the integer.
struct Mass {
  u64 hi, lo, total;
  __device__ __forceinline__ Mass() : hi(0), lo(0), total(0) {}
  __device__ __forceinline__ void add(u64 e2) {
    const u64 c1 = pack2(0x1.8p5f, 0x1.8p5f), n1 = pack2(-0x1.8p5f, -0x1.8p5f);
    const u64 c2 = pack2(0x1.8p-13f, 0x1.8p-13f), n2 = pack2(-0x1.8p-13f, -0x1.8p-13f);
    const u64 minus = pack2(-1.0f, -1.0f);
    const u64 h = add2(add2(e2, c1), n1);
    const u64 l = add2(add2(fma2(h, minus, e2), c2), n2);
    hi = add2(hi, h);
    lo = add2(lo, l);
  }
  __device__ __forceinline__ void flush() {
    total += static_cast<u64>(__float2int_rn(low2(hi) * 0x1p18f) + __float2int_rn(high2(hi) * 0x1p18f)) << 18;
    total += static_cast<u64>(static_cast<long long>(__float2int_rn(low2(lo) * 0x1p36f) + __float2int_rn(high2(lo) * 0x1p36f)));
    hi = 0;
    lo = 0;
  }
};

// ------------------------------------------------------ warps and clusters

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
__device__ __forceinline__ u64 warp_scan(u64 v, int lane) {  // inclusive
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const u64 o = __shfl_up_sync(kFullMask, v, d);
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
__device__ __forceinline__ u64 remote_load(uint32_t a) {
  u64 v;
  asm volatile("ld.shared::cluster.b64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void remote_add(uint32_t a, unsigned v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

struct Shared {
  u64 part[kWarps];
  u64 slot[2][kMaxCluster];  // one word per CTA, written by all of them; two turns
  u64 kept[kWarps];          // the warps' kept sums
  u64 say[8];                // what CTA 0 has decided
  u64 scan[3][kWarps];
  int lo, hi;                // the vectors that still may hold the choice
  u64 before;                // kept sum ahead of them
  unsigned list_len;
};

// The CTAs of a row's cluster, and this one in it.
struct Cta {
  Shared& s;
  uint32_t rank, size;
  int warp, lane;
  int turn = 0;

  __device__ __forceinline__ Cta(Shared& sh) : s(sh) {
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(size));
    warp = threadIdx.x >> 5;
    lane = threadIdx.x & 31;
  }
  __device__ __forceinline__ void sync() const {
    if (size > 1)
      asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    else
      __syncthreads();
  }
  // Sum (or largest) of every thread's v over the cluster; s.slot[turn ^ 1]
  // keeps the CTAs' own until the reduction after the next.
  template <bool MAX>
  __device__ __forceinline__ u64 reduce(u64 v) {
    v = MAX ? warp_max(v) : warp_sum(v);
    __syncthreads();  // the words of the last reduction have been read
    if (lane == 0) s.part[warp] = v;
    __syncthreads();
    u64 r = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) r = MAX ? umax64(r, s.part[w]) : r + s.part[w];
    if (size == 1) return r;
    if (threadIdx.x < size) remote_store(remote(&s.slot[turn][rank], threadIdx.x), r);
    sync();
    r = 0;
    for (uint32_t c = 0; c < size; ++c) r = MAX ? umax64(r, s.slot[turn][c]) : r + s.slot[turn][c];
    turn ^= 1;
    return r;
  }
};

// Descending bitonic sort of n (a power of two) words in shared memory.
__device__ __forceinline__ void block_sort_desc(u64* list, int n) {
  for (int k = 2; k <= n; k <<= 1) {
    for (int j = k >> 1; j > 0; j >>= 1) {
      __syncthreads();
      for (int i = threadIdx.x; i < n / 2; i += kThreads) {
        const int lo = 2 * i - (i & (j - 1)), hi = lo + j;
        const u64 a = list[lo], b = list[hi];
        if (((lo & k) == 0) == (a < b)) {
          list[lo] = b;
          list[hi] = a;
        }
      }
    }
  }
  __syncthreads();
}

__device__ __forceinline__ int pow2_at_least(int n) {
  int p = 32;
  while (p < n) p <<= 1;
  return p;
}

__device__ __forceinline__ float log_share(u64 w, u64 total) {
  return 2 * w < total ? logf(__fdiv_rn(__ull2float_rn(w), __ull2float_rn(total)))
                       : log1pf(-__fdiv_rn(__ull2float_rn(total - w), __ull2float_rn(total)));
}

// Which part of the row a score is in: bins of z, and within a range of them
// [v0, v1] finer ones. `from` .. `to` are the positions in question.
struct Bracket {
  bool fine = false;
  int v0 = 0, v1 = 0;
  float origin = 0.0f, scale = 0.0f;
  int from = 0, to = kBins - 1;

  // The position of a score (its order never decreases as z falls): below 0
  // for one above the finer bins, kBins or more for one that is past all.
  __device__ __forceinline__ int at(float z) const {
    const float y = __fmaf_rn(z, -static_cast<float>(kBinsPerOctave), 8388608.0f);
    if (!(y < 8388608.0f + kBins)) return kBins;
    const int v = static_cast<int>(__float_as_uint(y) - 0x4B000000u);
    if (!fine) return v;
    if (v < v0) return -1;
    if (v > v1) return kBins;
    return min(max(static_cast<int>((-z - origin) * scale), 0), kBins - 1);
  }
  // Bounds on the weight at a position of a bin that is not fine.
  static __device__ __forceinline__ void bounds(int v, unsigned count, bool fine, const Bracket& b, u64& lower, u64& upper) {
    const float zl = fine ? -(b.origin + static_cast<float>(v + 1) / b.scale) : -(v + 0.5f) / kBinsPerOctave;
    const float zu = fine ? -(b.origin + static_cast<float>(v) / b.scale) : -(v - 0.5f) / kBinsPerOctave;
    // 2^-14 covers the rounding of z and of the bins' edges, one unit the weight's own.
    const float l = exp2f(zl) * kOne * (1.0f - 0x1p-14f), u = exp2f(zu) * kOne * (1.0f + 0x1p-14f);
    const u64 lu = static_cast<u64>(l);
    lower = lu > 0 ? (lu - 1) * count : 0;
    upper = (static_cast<u64>(u) + 2) * count;
  }
};

template <typename T, bool HELD>
__global__ void __launch_bounds__(kThreads, 4) sample_kernel(const SampleLaunch a) {
  constexpr int E = Vec<T>::kLen;
  constexpr int kFlush = 64 / (E / 2);  // vectors that Mass sums before a flush
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ Shared s;
  unsigned* hist = reinterpret_cast<unsigned*>(dyn);  // kBins counts, or
  u64* list = reinterpret_cast<u64*>(dyn);            // kListCap keys
  uint4* held = reinterpret_cast<uint4*>(dyn + kListCap * sizeof(u64));

  Cta cta(s);
  const int lane = cta.lane;
  const int64_t r = blockIdx.x / cta.size;
  const Row<T> row(static_cast<const T*>(a.logits) + r * a.ld, a.vocab);
  const Ask q = read_ask(a, r);
  // This CTA's vectors [c0, c1), this warp's [v0, v1).
  const int c0 = static_cast<int>(int64_t(row.vecs) * cta.rank / cta.size);
  const int c1 = static_cast<int>(int64_t(row.vecs) * (cta.rank + 1) / cta.size);
  auto part_of = [](int lo, int hi, int w) { return lo + static_cast<int>(int64_t(hi - lo) * w / kWarps); };
  const int v0 = part_of(c0, c1, cta.warp), v1 = part_of(c0, c1, cta.warp + 1);
  auto get = [&](int v) -> uint4 {
    if constexpr (HELD)
      return held[v - c0];
    else
      return row.load(v);
  };
  auto index_of = [&](int v, int i) { return v * E - row.lead + i; };

  // ------------------------------------------------------ 1. largest score
  uint4 best = vec_none<T>();
  {
    // Whole vectors, four loads under way a lane; then the row's ragged ends.
    const int f0 = max(v0, row.lead > 0 ? 1 : 0), f1 = min(v1, (row.n + row.lead) / E);
    const uint4* src = reinterpret_cast<const uint4*>(row.p - row.lead);
    int v = f0 + lane;
    for (; v + 96 < f1; v += 128) {
      uint4 raw[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) raw[i] = src[v + 32 * i];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        raw[i] = vec_max<T>(raw[i], vec_none<T>());
        if constexpr (HELD) held[v + 32 * i - c0] = raw[i];
        best = vec_max<T>(best, raw[i]);
      }
    }
    for (; v < f1; v += 32) {
      const uint4 raw = vec_max<T>(src[v], vec_none<T>());
      if constexpr (HELD) held[v - c0] = raw;
      best = vec_max<T>(best, raw);
    }
    for (int e = lane; e < 2; e += 32) {
      const int w = e == 0 ? v0 : v1 - 1;
      if (w < v0 || w >= v1 || (w >= f0 && w < f1)) continue;
      const uint4 raw = row.load(w);
      if constexpr (HELD) held[w - c0] = raw;
      best = vec_max<T>(best, raw);
    }
  }
  float x0[E];
  Vec<T>::unpack(best, x0);
#pragma unroll
  for (int i = 1; i < E; ++i) x0[0] = fmaxf(x0[0], x0[i]);
  const float top = score_from_code(static_cast<uint32_t>(cta.reduce<true>(score_code(x0[0]))));
  if (top == -INFINITY) {  // nothing else
    if (cta.rank == 0 && threadIdx.x == 0) {
      a.token[r] = -1;
      if (a.logprob) a.logprob[r] = -INFINITY;
    }
    return;
  }
  const Scale sc(top, q.rate);

  // The best index alone: the first one at the largest score.
  if (q.k == 1) {
    u64 first = 0;
    for (int v = v0 + lane; v < v1; v += 32) {
      float x[E];
      Vec<T>::unpack(get(v), x);
#pragma unroll
      for (int i = E - 1; i >= 0; --i)
        if (x[i] == top) first = umax64(first, ~static_cast<u64>(index_of(v, i)));
    }
    first = cta.reduce<true>(first);
    if (cta.rank == 0 && threadIdx.x == 0) {
      a.token[r] = static_cast<int32_t>(~first);
      if (a.logprob) a.logprob[r] = 0.0f;
    }
    return;
  }

  // f(z pair, vector, first of the two) for this warp's scores; after every
  // kFlush vectors, g().
  auto each_pair = [&](int from, int to, auto&& f, auto&& g) {
    int since = 0;
    for (int v = from + lane; v < to; v += 32) {
      float x[E];
      Vec<T>::unpack(get(v), x);
#pragma unroll
      for (int i = 0; i < E; i += 2) f(sc.z2(x[i], x[i + 1]), v, i, x[i], x[i + 1]);
      if (++since == kFlush) {
        g();
        since = 0;
      }
    }
    g();
  };

  const bool by_k = q.k < a.vocab, by_p = q.part_p < kAll;
  u64 cut = 0;         // keys from here on are kept

  // Kept weight of a score, once the cut is known.
  auto kept = [&](float x, int index) -> u64 {
    const float e = ex2(sc.z(x));
    return e >= q.min_p && make_key(x, static_cast<uint32_t>(index)) >= cut ? fixed(e) : 0ull;
  };

  if (by_k || by_p) {
    // ---------------------------------------------------- 3. count by bins
    Bracket br;
    u64 above = 0;        // cluster-wide sum of weights ahead of the bracket
    u64 count_above = 0;  // and number of scores
    u64 sum_all = 0;      // sum of what top_k kept, once known
    bool know_sum = !by_k;
    bool for_k = by_k;    // which of the two ends is looked for
    u64 kcut = 0;
    u64 last_key = 0;     // the key at which the end that is looked for lies
    for (;;) {
      // Positions of all scores that may be kept: counts of the ones in the
      // bracket's range, sum of the weights ahead of it.
      for (int i = threadIdx.x; i < kBins; i += kThreads) hist[i] = 0;
      if (threadIdx.x == 0) s.list_len = 0;
      cta.sync();
      const bool sum_it = by_p && !for_k && (br.fine || !know_sum || sum_all == 0);
      Mass m;
      each_pair(
          v0, v1,
          [&](u64 z2, int v, int i, float xa, float xb) {
            const float za = low2(z2), zb = high2(z2);
            const int pa = br.at(za), pb = br.at(zb);
            const bool ka = kcut == 0 || make_key(xa, index_of(v, i)) >= kcut;
            const bool kb = kcut == 0 || make_key(xb, index_of(v, i + 1)) >= kcut;
            if (ka && pa >= 0 && pa < kBins) atomicAdd(&hist[pa], 1u);
            if (kb && pb >= 0 && pb < kBins) atomicAdd(&hist[pb], 1u);
            if (sum_it) m.add(pack2(ka && (!br.fine || pa < 0) ? ex2(za) : 0.0f, kb && (!br.fine || pb < 0) ? ex2(zb) : 0.0f));
          },
          [&] { m.flush(); });
      const u64 sum = sum_it ? cta.reduce<false>(m.total) : 0;  // of all, or of the ones ahead of the finer bins
      if (sum_it && !br.fine) sum_all = sum;
      if (sum_it && br.fine) above = sum;
      // CTA 0 collects the counts.
      __syncthreads();
      if (cta.size > 1) {
        if (cta.rank != 0)
          for (int i = threadIdx.x; i < kBins; i += kThreads)
            if (hist[i]) remote_add(remote(&hist[i], 0), hist[i]);
        cta.sync();
      }
      const u64 target = for_k ? static_cast<u64>(q.k) : share(sum_all, q.part_p);
      if (cta.rank == 0) {
        // Running counts and bounds: a thread has kBinsPerThread bins.
        u64 n = 0, lower = 0, upper = 0;
        unsigned c[kBinsPerThread];
#pragma unroll
        for (int i = 0; i < kBinsPerThread; ++i) {
          const int b = threadIdx.x * kBinsPerThread + i;
          c[i] = b < kBins ? hist[b] : 0u;
          n += c[i];
          if (!for_k && c[i]) {
            u64 l, u;
            Bracket::bounds(b, c[i], br.fine, br, l, u);
            lower += l;
            upper += u;
          }
        }
        const u64 sn = warp_scan(n, lane), sl = warp_scan(lower, lane), su = warp_scan(upper, lane);
        if (lane == 31) {
          s.scan[0][cta.warp] = sn;
          s.scan[1][cta.warp] = sl;
          s.scan[2][cta.warp] = su;
        }
        if (threadIdx.x == 0) {
          s.say[0] = kBins - 1;  // first position at which the end may lie
          s.say[1] = kBins - 1;  // last one
        }
        __syncthreads();
        u64 bn = count_above, bl = above, bu = above;
        u64 all = 0;
        for (int w = 0; w < kWarps; ++w) {
          if (w < cta.warp) {
            bn += s.scan[0][w];
            bl += s.scan[1][w];
            bu += s.scan[2][w];
          }
          all += s.scan[0][w];
        }
        bn += sn - n;
        bl += sl - lower;
        bu += su - upper;
        // The thread in whose bins a running value passes the target.
        u64 fn = bn, fl = bl, fu = bu;
        for (int i = 0; i < kBinsPerThread; ++i) {
          const int b = threadIdx.x * kBinsPerThread + i;
          if (b >= kBins) break;
          u64 l = 0, u = 0;
          if (!for_k && c[i]) Bracket::bounds(b, c[i], br.fine, br, l, u);
          if (for_k) {
            if (fn < target && fn + c[i] >= target) s.say[0] = s.say[1] = b;
          } else {
            if (fu < target && fu + u >= target) s.say[0] = b;
            if (fl < target && fl + l >= target) s.say[1] = b;
          }
          fn += c[i];
          fl += l;
          fu += u;
        }
        __syncthreads();
        // Counts ahead of the bracket, and in it.
        const int from = static_cast<int>(s.say[0]), to = static_cast<int>(s.say[1]);
        u64 ahead = 0, in = 0;
#pragma unroll
        for (int i = 0; i < kBinsPerThread; ++i) {
          const int b = threadIdx.x * kBinsPerThread + i;
          if (b < from) ahead += c[i];
          if (b >= from && b <= to) in += c[i];
        }
        ahead = warp_sum(ahead);
        in = warp_sum(in);
        __syncthreads();
        if (lane == 0) {
          s.scan[0][cta.warp] = ahead;
          s.scan[1][cta.warp] = in;
        }
        __syncthreads();
        if (threadIdx.x == 0) {
          ahead = count_above;
          in = 0;
          for (int w = 0; w < kWarps; ++w) {
            ahead += s.scan[0][w];
            in += s.scan[1][w];
          }
          s.say[2] = ahead;
          s.say[3] = in;
          s.say[4] = count_above + all;  // scores down to the last position
        }
        __syncthreads();
        if (cta.size > 1 && threadIdx.x >= 1 && threadIdx.x < cta.size)
          for (int i = 0; i < 5; ++i) remote_store(remote(&s.say[i], threadIdx.x), s.say[i]);
      }
      cta.sync();
      br.from = static_cast<int>(s.say[0]);
      br.to = static_cast<int>(s.say[1]);
      const u64 ahead = s.say[2], in = s.say[3], reach = s.say[4];
      if (for_k && !br.fine && reach <= target) {
        // Everything that has a weight is among the top_k.
        for_k = false;
        if (!by_p) break;  // nothing is cut
        br = Bracket();
        cta.sync();
        continue;
      }
      const bool whole = ahead + in <= kListCap && !br.fine;  // all down to the bracket's end
      if (!whole && in > kListCap && !br.fine) {
        // Divide the bracket's bins again.
        Bracket f;
        f.fine = true;
        f.v0 = br.from;
        f.v1 = br.to;
        f.origin = (br.from - 0.5f) / kBinsPerOctave;
        f.scale = static_cast<float>(kBins) * kBinsPerOctave / static_cast<float>(br.to - br.from + 1);
        br = f;
        count_above = ahead;
        cta.sync();  // CTA 0's words have been read
        continue;
      }
      if (in <= kListCap || whole) {
        // ------------------------------------------------------- gather
        cta.sync();  // the counts are no longer needed
        const int from = whole ? 0 : br.from;
        Mass m2;
        each_pair(
            v0, v1,
            [&](u64 z2, int v, int i, float xa, float xb) {
              const float za = low2(z2), zb = high2(z2);
              const int pa = br.at(za), pb = br.at(zb);
              const u64 key_a = make_key(xa, index_of(v, i)), key_b = make_key(xb, index_of(v, i + 1));
              if (pa >= from && pa <= br.to && key_a >= kcut) {
                const unsigned n = atomicAdd(&s.list_len, 1u);
                if (n < kListCap) list[n] = key_a;
              }
              if (pb >= from && pb <= br.to && key_b >= kcut) {
                const unsigned n = atomicAdd(&s.list_len, 1u);
                if (n < kListCap) list[n] = key_b;
              }
              if (!whole && by_p) m2.add(pack2(pa < from ? ex2(za) : 0.0f, pb < from ? ex2(zb) : 0.0f));
            },
            [&] { m2.flush(); });
        if (!whole && by_p) above = cta.reduce<false>(m2.total);
        cta.sync();
        if (cta.rank == 0) {
          // Append the other CTAs' keys.
          int len = static_cast<int>(s.list_len);
          for (uint32_t c = 1; c < cta.size; ++c) {
            unsigned n;
            asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(n) : "r"(remote(&s.list_len, c)) : "memory");
            for (unsigned i = threadIdx.x; i < n; i += kThreads)
              if (len + static_cast<int>(i) < kListCap) list[len + i] = remote_load(remote(&list[i], c));
            len += static_cast<int>(n);
          }
          len = min(len, kListCap);
          const int size = pow2_at_least(len);
          for (int i = len + threadIdx.x; i < size; i += kThreads) list[i] = 0;
          block_sort_desc(list, size);
          // Running weights in the order of the search: a thread has `per` keys.
          const int per = (size + kThreads - 1) / kThreads;
          u64 sum_here = 0;
          for (int i = 0; i < per; ++i) {
            const int j = threadIdx.x * per + i;
            if (j < len) sum_here += weight(key_score(list[j]), sc);
          }
          const u64 incl = warp_scan(sum_here, lane);
          if (lane == 31) s.scan[0][cta.warp] = incl;
          __syncthreads();
          u64 run = incl - sum_here;
          for (int w = 0; w < cta.warp; ++w) run += s.scan[0][w];
          if (whole) {
            // Finish the row here. top_k's sum, then the kept prefix.
            const int nk = for_k ? min(q.k, len) : len;
            if (threadIdx.x == 0) {
              s.say[5] = 0;
              s.say[6] = 0;
              s.say[7] = 1;
            }
            __syncthreads();
            if (by_p && for_k) {
              u64 t = run;
              for (int i = 0; i < per; ++i) {
                const int j = threadIdx.x * per + i;
                if (j < len) t += weight(key_score(list[j]), sc);
                if (j == nk - 1) s.say[5] = t;
              }
              __syncthreads();
            }
            const u64 goal = by_p ? share(for_k ? s.say[5] : sum_all, q.part_p) : ~0ull;
            {
              u64 t = run;
              int mine = 0;
              for (int i = 0; i < per; ++i) {
                const int j = threadIdx.x * per + i;
                if (j >= nk) break;
                const float e = ex2(sc.z(key_score(list[j])));
                if (j == 0 || (t < goal && e >= q.min_p)) ++mine;
                t += fixed(e);
              }
              mine = __reduce_add_sync(kFullMask, mine);
              if (lane == 0) atomicAdd(reinterpret_cast<unsigned*>(&s.say[6]), static_cast<unsigned>(mine));
            }
            __syncthreads();
            const int nkeep = static_cast<int>(s.say[6]);
            // In index order: the key's low word falls as the index rises.
            const int size2 = pow2_at_least(nkeep);
            for (int i = threadIdx.x; i < size2; i += kThreads) {
              const u64 key = i < nkeep ? list[i] : 0ull;
              list[i] = (key << 32) | (key >> 32);
            }
            block_sort_desc(list, size2);
            const int per2 = (size2 + kThreads - 1) / kThreads;
            u64 here = 0;
            for (int i = 0; i < per2; ++i) {
              const int j = threadIdx.x * per2 + i;
              if (j < nkeep) here += weight(score_from_code(static_cast<uint32_t>(list[j])), sc);
            }
            const u64 in2 = warp_scan(here, lane);
            __syncthreads();
            if (lane == 31) s.scan[0][cta.warp] = in2;
            __syncthreads();
            u64 t = in2 - here, w_all = 0;
            for (int w = 0; w < kWarps; ++w) {
              if (w < cta.warp) t += s.scan[0][w];
              w_all += s.scan[0][w];
            }
            const u64 aim = share(w_all, q.part_u);
            for (int i = 0; i < per2; ++i) {
              const int j = threadIdx.x * per2 + i;
              if (j >= nkeep) break;
              const u64 w = weight(score_from_code(static_cast<uint32_t>(list[j])), sc);
              if (t <= aim && aim < t + w) {
                a.token[r] = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(list[j] >> 32));
                if (a.logprob) a.logprob[r] = log_share(w, w_all);
              }
              t += w;
            }
          } else {
            // The key at which the prefix ends.
            if (threadIdx.x == 0) s.say[5] = list[len > 0 ? len - 1 : 0];
            __syncthreads();
            u64 t = above + run;
            for (int i = 0; i < per; ++i) {
              const int j = threadIdx.x * per + i;
              if (j >= len) break;
              const u64 w = weight(key_score(list[j]), sc);
              if (for_k ? ahead + j + 1 == target : (t < target && t + w >= target)) {
                s.say[5] = list[j];
                s.say[6] = t + w;
              }
              t += w;
            }
            __syncthreads();
            if (threadIdx.x >= 1 && threadIdx.x < cta.size)
              for (int i = 5; i < 7; ++i) remote_store(remote(&s.say[i], threadIdx.x), s.say[i]);
          }
        }
        cta.sync();
        if (whole) return;  // CTA 0 has finished the row, and nobody reads another's memory any more
        last_key = s.say[5];
      } else {
        // Equal scores by the thousand: halve the interval of keys.
        u64 lo = kcut, hi = make_key(top, 0) + 1;
        while (hi - lo > 1) {
          const u64 mid = lo + (hi - lo) / 2;
          u64 c = 0;
          for (int v = v0 + lane; v < v1; v += 32) {
            float x[E];
            Vec<T>::unpack(get(v), x);
#pragma unroll
            for (int i = 0; i < E; ++i)
              if (make_key(x[i], index_of(v, i)) >= mid) c += for_k ? 1ull : weight(x[i], sc);
          }
          if (cta.reduce<false>(c) >= target)
            lo = mid;
          else
            hi = mid;
        }
        last_key = lo;
        cta.sync();
      }
      if (!for_k) {
        cut = last_key;
        break;
      }
      kcut = cut = last_key;
      for_k = false;
      if (!by_p) break;
      // Now top_p, among what top_k kept.
      know_sum = false;
      sum_all = 0;
      above = 0;
      count_above = 0;
      br = Bracket();
      cta.sync();
    }
  }

  // ------------------------------------------------- the warps' kept sums
  Mass m;
  each_pair(
      v0, v1,
      [&](u64 z2, int v, int i, float xa, float xb) {
        float ea = ex2(low2(z2)), eb = ex2(high2(z2));
        if (ea < q.min_p || (cut != 0 && make_key(xa, index_of(v, i)) < cut)) ea = 0.0f;
        if (eb < q.min_p || (cut != 0 && make_key(xb, index_of(v, i + 1)) < cut)) eb = 0.0f;
        m.add(pack2(ea, eb));
      },
      [&] { m.flush(); });
  const u64 total = cta.reduce<false>(m.total);
  const u64 own = warp_sum(m.total);
  if (lane == 0) s.kept[cta.warp] = own;
  const u64 aim = share(total, q.part_u);
  u64 before = 0;
  u64 mine_all = total;
  if (cta.size > 1) {
    for (uint32_t c = 0; c < cta.rank; ++c) before += s.slot[cta.turn ^ 1][c];
    mine_all = s.slot[cta.turn ^ 1][cta.rank];
  }
  if (aim < before || aim >= before + mine_all) return;  // another CTA's part

  // Narrow the vectors that hold the choice: s.kept has the sums over the equal
  // parts of [lo, hi), one a warp.
  if (threadIdx.x == 0) {
    s.lo = c0;
    s.hi = c1;
    s.before = before;
  }
  __syncthreads();
  for (;;) {
    const int lo = s.lo, hi = s.hi;
    u64 upto = s.before;
    int in = 0;
    while (in < kWarps - 1 && upto + s.kept[in] <= aim) upto += s.kept[in++];
    const int n0 = part_of(lo, hi, in), n1 = part_of(lo, hi, in + 1);
    __syncthreads();
    if (threadIdx.x == 0) {
      s.lo = n0;
      s.hi = n1;
      s.before = upto;
    }
    if (n1 - n0 <= 32) break;
    u64 part = 0;
    const int m1 = part_of(n0, n1, cta.warp + 1);
    for (int v = part_of(n0, n1, cta.warp) + lane; v < m1; v += 32) {
      float x[E];
      Vec<T>::unpack(get(v), x);
#pragma unroll
      for (int i = 0; i < E; ++i) part += kept(x[i], index_of(v, i));
    }
    part = warp_sum(part);
    if (lane == 0) s.kept[cta.warp] = part;
    __syncthreads();
  }
  __syncthreads();
  if (cta.warp == 0) {
    const int v = s.lo + lane;
    u64 mine[E];
    u64 sum = 0;
    if (v < s.hi) {
      float x[E];
      Vec<T>::unpack(get(v), x);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        mine[i] = kept(x[i], index_of(v, i));
        sum += mine[i];
      }
    }
    u64 run = s.before + warp_scan(sum, lane) - sum;
    if (sum > 0 && run <= aim && aim < run + sum) {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        if (run <= aim && aim < run + mine[i]) {
          a.token[r] = index_of(v, i);
          if (a.logprob) a.logprob[r] = log_share(mine[i], total);
        }
        run += mine[i];
      }
    }
  }
}

template <typename T, bool HELD>
cudaError_t launch_t(const SampleLaunch& a, int cluster, int held_bytes, cudaStream_t st) {
  auto fn = sample_kernel<T, HELD>;
  static PerDeviceOnce once;
  const cudaError_t ready = once.run([fn] {
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, max_dynamic_smem() - 2048);
    return e != cudaSuccess ? e : cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  });
  if (ready != cudaSuccess) return ready;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.rows * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kListCap * sizeof(u64) + static_cast<size_t>(held_bytes);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, a);
}

template <typename T>
cudaError_t launch_rows(const SampleLaunch& a, cudaStream_t st) {
  const int64_t bytes = int64_t(a.vocab) * sizeof(T) + 32;
  // A CTA's part in shared memory: 32 KB leaves room for four CTAs an SM, whose
  // reads overlap the others' passes.
  int cluster = 1;
  while (cluster < kMaxCluster && bytes / cluster > 32 * 1024) cluster *= 2;
  const int64_t held = (bytes + cluster - 1) / cluster / 16 * 16 + 32;
  if (held <= 64 * 1024) return launch_t<T, true>(a, cluster, static_cast<int>(held), st);
  return launch_t<T, false>(a, cluster, 0, st);
}

}  // namespace

cudaError_t launch_sample(const SampleLaunch& a, cudaStream_t st) {
  // A grid has 2^31 - 1 CTAs; more rows than that times the cluster go in parts.
  SampleLaunch part = a;
  for (int64_t r = 0; r < a.rows; r += int64_t(1) << 26) {
    part.rows = std::min<int64_t>(a.rows - r, int64_t(1) << 26);
    part.logits = static_cast<const char*>(a.logits) + r * a.ld * dtype_bytes(a.dtype);
    part.u = a.u + r;
    part.temperature = a.temperature ? a.temperature + r : nullptr;
    part.top_k = a.top_k ? a.top_k + r : nullptr;
    part.top_p = a.top_p ? a.top_p + r : nullptr;
    part.min_p = a.min_p ? a.min_p + r : nullptr;
    part.token = a.token + r;
    part.logprob = a.logprob ? a.logprob + r : nullptr;
    const cudaError_t e = a.dtype == kF32    ? launch_rows<float>(part, st)
                          : a.dtype == kBF16 ? launch_rows<__nv_bfloat16>(part, st)
                                             : launch_rows<__half>(part, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace rbf
