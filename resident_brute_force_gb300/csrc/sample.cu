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
//   3. top_k: of the threads' largest scores (distinct scores of the row), the
//      k-th largest bounds the row's k-th from below, so one pass gathers
//      little more than the k best into a list, from which top_p is found
//      too. top_p, and a top_k past half of the threads: a pass counts the
//      scores in bins of 2^(1/128) in weight and sums the weights; the counts
//      bound the sums above each bin edge, which leaves one to three bins in
//      which the prefix can end. With such a top_k, top_p takes two more
//      passes, for its share of the weight that top_k kept.
//   4. Few candidates (kSmall): one CTA finishes the row, every thread finding
//      the rank and the running weight of its candidate by looking at all.
//      Else the scores of those bins are gathered in a list, where K is found
//      by halving, while the weights above them are summed, per warp.
//   5. The warps' kept sums say which warp's part holds r; that part is divided
//      among the warps again until one warp has it in its lanes.
// Where a list does not hold the bins' scores they are divided into finer
// bins; scores that coincide by the thousand (no bins divide them) leave K to
// be found by halving the interval of keys, one pass over the row a step.
//
// What bounds it: with top_p, instructions for half of the time (256 x 128,000:
// 73 a score, of which the passes over scores that are on chip are about half,
// the rest the fixed part of a CTA) and barriers for most of the other half;
// with no filter and with top_k (27 and 29 a score, 52 and 42 % of the issue
// slots) the first read, whose waves have nothing else under way, and barriers;
// with few rows latency (1 x 10,000: 22 % of the issue slots of two SMs; 8 x
// 1,000,000 min_p, read again from L2: 27 %). The shared-memory atomics of the
// counts go at 11 to 14 lanes a clock and SM, and there are
// per row some ten exchanges across the cluster at 450 clocks each. The text
// counts too: the kernel is 150 to 177 KB, more than the instruction cache, and
// passes that few rows take are loops over single scores (with every loop
// unrolled it was 296 to 432 KB; 256 x 128,000 top_p from cold 143 us, now 133,
// top_k 700 with top_p 230, now 124).
// Measured (us, the bytes alone at the copy rate in brackets): 1 x 10,000 fp32
// top_k + top_p 12 to 14 (0.006); 61 x 100,003 bf16 top_p 39 (1.8); 256 x 128,000
// bf16 top_p 124, top_k <= 100 62, top_k 5,000-9,000 115, neither 43.5, best index
// 35 (9.6); 8 x 1,000,000 fp32 min_p 25, top_p 66 (4.7).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "ops_internal.h"
#include "rbf_device.cuh"
#include "rbf_internal.h"

namespace rbf {
namespace {

constexpr int kMaxCluster = 16;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kOne = 68719476736.0f;  // 2^36: the largest weight
constexpr int kBinsPerOctave = 128;
constexpr int kBins = 37 * kBinsPerOctave + 1;  // z = 0 .. -37, rounded
constexpr int kQuads = (kBins + 3) / 4;  // the counts are read four at a time
// Keys of a list: as many as fit where the counts of all bins are, more where
// the row is not in shared memory.
template <bool HELD>
constexpr int kListCap = HELD ? kQuads * 2 : 8192;
constexpr int kMaxHeld = 64 * 1024;  // of a row's scores in one CTA's shared memory
constexpr int kMaxSmem = kMaxHeld + kListCap<true> * 8;
constexpr int kSmall = 256;              // candidates of a row that one CTA finishes

using u64 = unsigned long long;

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
  // A finite rate above 0: an infinite temperature would make (-infinity) * 0 of
  // a masked score, and one under 4.24e-39 0 * infinity of the best score. The
  // smallest float leaves every finite score the weight 1, to 2^-20.
  q.rate = warm ? fminf(fmaxf(__fdiv_rn(kLog2e, t), 1.4e-45f), 3.40282347e38f) : kLog2e;
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
  static __device__ __forceinline__ float shift(float x) { return x == INFINITY ? 0.0f : -INFINITY; }
  // z of two scores that have been shifted where that is due.
  __device__ __forceinline__ u64 z2(float a, float b) const { return mul2(add2(pack2(a, b), ntop2), rate2); }
  __device__ __forceinline__ float z(float x) const { return __fmul_rn(__fsub_rn(inf ? shift(x) : x, top), rate); }
};

__device__ __forceinline__ u64 fixed(float e) { return static_cast<u64>(__float2ll_rn(__fmul_rn(e, kOne))); }
__device__ __forceinline__ u64 weight(float x, const Scale& s) { return fixed(ex2(s.z(x))); }

// A sum of weights. e is divided into a multiple of 2^-18 and a rest that is
// rounded to a multiple of 2^-36: adding 1.5 * 2^23 units rounds to units
// (halves to even) and leaves their number, plus that of the constant, in the
// low bits of the fp32 pattern. The patterns are summed as integers, modulo
// 2^32, and the constants' share is taken out at the end: exact for up to 2^13
// weights a thread, then moved into 64 bits.
struct Mass {
  unsigned hi = 0, lo = 0;
  u64 total = 0;
  static constexpr float kHi = 0x1.8p5f, kLo = 0x1.8p-13f;
  __device__ __forceinline__ void add(float a, float b) {
    const float ta = __fadd_rn(a, kHi), tb = __fadd_rn(b, kHi);
    hi += __float_as_uint(ta) + __float_as_uint(tb);
    const float la = __fadd_rn(a, __fsub_rn(kHi, ta)), lb = __fadd_rn(b, __fsub_rn(kHi, tb));
    lo += __float_as_uint(__fadd_rn(la, kLo)) + __float_as_uint(__fadd_rn(lb, kLo));
  }
  // `n`: weights added since the last flush.
  __device__ __forceinline__ void flush(unsigned n) {
    total += static_cast<u64>(hi - n * 0x42400000u) << 18;
    total += static_cast<u64>(static_cast<long long>(static_cast<int>(lo - n * 0x39400000u)));
    hi = 0;
    lo = 0;
  }
};

// ------------------------------------------------------ warps and clusters

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

template <int WARPS>
struct Shared {
  u64 part[WARPS];
  u64 slot[2][kMaxCluster];  // one word per CTA, written by all of them; two turns
  u64 kept[WARPS];          // the warps' kept sums
  u64 say[8];                // what CTA 0 has decided
  u64 words[4][kMaxCluster]; // words that every CTA has sent to every other
  u64 small_key[kSmall];     // candidates, and what they keep
  u64 small_w[kSmall];
  unsigned add_lo[WARPS], add_hi[WARPS];
  u64 scan[4][WARPS];
  u64 found[4];              // this CTA's part of say[0] .. say[3]
  int lo, hi;                // the vectors that still may hold the choice
  u64 before;                // kept sum ahead of them
  unsigned list_len;
};

// The CTAs of a row's cluster, and this one in it.
template <int WARPS>
struct Cta {
  Shared<WARPS>& s;
  uint32_t rank, size;
  int warp, lane;
  int turn = 0;

  __device__ __forceinline__ Cta(Shared<WARPS>& sh) : s(sh) {
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
  // A CTA's shared memory may be written by others once it has started: all
  // arrive at the kernel's start and wait ahead of the first remote store (at
  // `reduce`), with the read of the row in between. The arrival has nothing to
  // release: a relaxed one saves 0.6 to 1.7 us of 15 to 45.
  __device__ __forceinline__ void started() const {
    if (size > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  }
  __device__ __forceinline__ void all_started() const {
    if (size > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  // Sum (or largest) of every thread's v over the cluster; s.slot[turn ^ 1]
  // keeps the CTAs' own until the reduction after the next.
  template <bool MAX>
  __device__ __forceinline__ u64 reduce(u64 v) {
    v = MAX ? warp_max(v) : warp_sum(v);
    __syncthreads();  // the words of the last reduction have been read
    if (lane == 0) s.part[warp] = v;
    __syncthreads();
    u64 r = lane < WARPS ? s.part[lane] : 0ull;
    r = MAX ? warp_max(r) : warp_sum(r);
    if (size == 1) return r;
    if (threadIdx.x < size) remote_store(remote(&s.slot[turn][rank], threadIdx.x), r);
    sync();
    r = lane < static_cast<int>(size) ? s.slot[turn][lane] : 0ull;
    turn ^= 1;
    return MAX ? warp_max(r) : warp_sum(r);
  }
};

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

  // A bin is the rounding of -128 z to a whole number, which adding 2^23 leaves in the low bits of the fp32 pattern.
  static constexpr uint32_t kPattern = 0x4B000000u;
  static __device__ __forceinline__ float pattern(float z) { return __fmaf_rn(z, -static_cast<float>(kBinsPerOctave), 8388608.0f); }
  // The bin of a pattern; kBins or more for z under -37 (infinities have larger patterns).
  static __device__ __forceinline__ uint32_t bin(float y) { return __float_as_uint(y) - kPattern; }
  // The position of a score (its order never decreases as z falls): below 0
  // for one above the finer bins, kBins or more for one that is past all.
  __device__ __forceinline__ int at(float z, float y) const {
    const uint32_t v = bin(y);
    if (v >= static_cast<uint32_t>(kBins)) return kBins;
    if (!fine) return static_cast<int>(v);
    if (static_cast<int>(v) < v0) return -1;
    if (static_cast<int>(v) > v1) return kBins;
    return min(max(static_cast<int>((-z - origin) * scale), 0), kBins - 1);
  }
  // z at the lower-weight edge of position p, and the step to the next one.
  __device__ __forceinline__ float edge(int p) const {
    return fine ? -(origin + static_cast<float>(p + 1) / scale) : -(static_cast<float>(p) + 0.5f) / kBinsPerOctave;
  }
  __device__ __forceinline__ float step() const { return fine ? -1.0f / scale : -1.0f / kBinsPerOctave; }
};
// Sums of counts times the weights at the bins' edges bound the sums of weights;
// a thread makes them in fp32, in units of the largest weight: 2^-14 covers the
// rounding of z (under 2^-18), of the edges and of its few dozen additions,
// 2^-36 a score the weights' own.
constexpr float kBelow = 1.0f - 0x1p-14f, kAbove = 1.0f + 0x1p-14f;

// HELD: a CTA's part of the row is in shared memory.
template <typename T, bool HELD, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) sample_kernel(const SampleLaunch a) {
  constexpr int kWarps = kThreads / 32;
  constexpr int kCap = kListCap<HELD>;
  constexpr int E = Vec<T>::kLen;
  constexpr int kFlush = 8192 / E;  // vectors that Mass sums before a flush
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ Shared<kWarps> s;
  unsigned* hist = reinterpret_cast<unsigned*>(dyn);  // kBins counts, or
  u64* list = reinterpret_cast<u64*>(dyn);            // kCap keys
  uint4* held = reinterpret_cast<uint4*>(dyn + kCap * sizeof(u64));

  Cta<kWarps> cta(s);
  cta.started();
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
#pragma unroll 1
    for (; v < f1; v += 32) {
      const uint4 raw = vec_max<T>(src[v], vec_none<T>());
      if constexpr (HELD) held[v - c0] = raw;
      best = vec_max<T>(best, raw);
    }
#pragma unroll 1
    for (int e = lane; e < 2; e += 32) {
      const int w = e == 0 ? v0 : v1 - 1;
      if (v0 >= v1 || (e == 1 && w == v0) || (w >= f0 && w < f1)) continue;
      const uint4 raw = row.load(w);
      if constexpr (HELD) held[w - c0] = raw;
      best = vec_max<T>(best, raw);
    }
  }
  float x0[E];
  Vec<T>::unpack(best, x0);
#pragma unroll
  for (int i = 1; i < E; ++i) x0[0] = fmaxf(x0[0], x0[i]);
  __syncwarp();  // the barrier is for converged warps
  cta.all_started();
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
#pragma unroll 1
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

  // f(the scores' z, vector) for this warp's vectors, some loads under way a
  // lane; after at most kFlush vectors g(number of scores since the last one).
  auto each = [&](auto&& f, auto&& g) {
    auto one = [&](const uint4& raw, int v) {
      float x[E], z[E];
      Vec<T>::unpack(raw, x);
      if (sc.inf) {
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = Scale::shift(x[i]);
      }
#pragma unroll
      for (int i = 0; i < E; i += 2) {
        const u64 z2 = sc.z2(x[i], x[i + 1]);
        z[i] = low2(z2);
        z[i + 1] = high2(z2);
      }
      f(z, v);
    };
    constexpr int kBatch = HELD ? 1 : 4;
    int v = v0 + lane, since = 0;
    for (; v + 32 * (kBatch - 1) < v1; v += 32 * kBatch) {
      uint4 raw[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) raw[i] = get(v + 32 * i);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) one(raw[i], v + 32 * i);
      if ((since += kBatch) == kFlush) {
        g(static_cast<unsigned>(since * E));
        since = 0;
      }
    }
    g(static_cast<unsigned>(since * E));
    since = 0;
#pragma unroll 1
    for (; v < v1; v += 32, ++since) one(get(v), v);
    g(static_cast<unsigned>(since * E));
  };
  // One score, read again (its index is one of the row's).
  auto score_at = [&](int v, int i) -> float {
    if constexpr (HELD)
      return Vec<T>::one(reinterpret_cast<const T*>(held + (v - c0))[i]);
    else
      return fmaxf(Vec<T>::one(row.p[index_of(v, i)]), -INFINITY);
  };
  // f(score, key) for this warp's scores, one at a time: for the passes that few
  // rows take, in a twentieth of the code.
  auto each_one = [&](auto&& f) {
#pragma unroll 1
    for (int v = v0 + lane; v < v1; v += 32) {
#pragma unroll 1
      for (int i = 0; i < E; ++i) {
        const int index = index_of(v, i);
        if (index < 0 || index >= row.n) continue;
        const float x = score_at(v, i);
        f(x, make_key(x, static_cast<uint32_t>(index)));
      }
    }
  };
  // Put the scores of a vector that `mask` names into this CTA's list.
  auto append = [&](unsigned mask, int v) {
    if (mask == 0) return;
    unsigned at = atomicAdd(&s.list_len, static_cast<unsigned>(__popc(mask)));
    for (; mask != 0; mask &= mask - 1, ++at) {
      const int i = __ffs(static_cast<int>(mask)) - 1;
      if (at < kCap) list[at] = make_key(score_at(v, i), static_cast<uint32_t>(index_of(v, i)));
    }
  };
  // Sum over CTA 0's threads of a value each, for all of them; `t` names one of three words a warp.
  auto block_sum = [&](u64 v, int t) {
    v = warp_sum(v);
    if (lane == 0) s.scan[t][cta.warp] = v;
    __syncthreads();
    return warp_sum(lane < kWarps ? s.scan[t][lane] : 0ull);
  };
  // CTA 0's words [i0, i1) to the others.
  auto tell = [&](int i0, int i1) {
    __syncthreads();
    if (cta.rank == 0 && threadIdx.x >= 1 && threadIdx.x < cta.size)
      for (int i = i0; i < i1; ++i) remote_store(remote(&s.say[i], threadIdx.x), s.say[i]);
    cta.sync();
  };

  const bool by_k = q.k < a.vocab, by_p = q.part_p < kAll;
  u64 cut = 0;           // keys from here on are kept
  bool summed = false;   // s.kept has the warps' kept sums

  // Kept weight of a score, once the cut is known, and of a vector's scores.
  auto kept = [&](int v, int i) -> u64 {
    const int index = index_of(v, i);
    if (index < 0 || index >= row.n) return 0;
    const float x = score_at(v, i), e = ex2(sc.z(x));
    return e >= q.min_p && make_key(x, static_cast<uint32_t>(index)) >= cut ? fixed(e) : 0ull;
  };
  auto kept_of = [&](int v) {
    u64 sum = 0;
#pragma unroll 2
    for (int i = 0; i < E; ++i) sum += kept(v, i);
    return sum;
  };

  // Counts of the scores by position, and where a prefix ends that has `target`
  // scores (for_k) or weight: say[0], say[1] the first and last position, say[2]
  // scores ahead of the first, say[3] scores down to the last one, say[4] all.
  // Each CTA adds up the cluster's counts for an equal part of the positions.
  // For weights `mine` is the thread's sum of all of them or, with finer bins, of
  // the ones ahead; the row's goes to sum_all or above, and the target follows.
  // Where all are summed the bounds are taken from the other end too: those of a
  // prefix are the sum less those of the rest, and near top_p = 1 that rest is
  // small, and so is its error.
  auto clear_counts = [&]() {
#pragma unroll 1
    for (int i = threadIdx.x; i < kQuads; i += kThreads) reinterpret_cast<uint4*>(hist)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (threadIdx.x == 0) s.list_len = 0;
    __syncthreads();
  };
  auto decide = [&](const Bracket& br, bool for_k, u64 mine, u64 sum_k, u64& sum_all, u64& above, u64 count_above, u64& target) {
    cta.sync();  // all counts are there
    const int per = (kQuads + static_cast<int>(cta.size) * kThreads - 1) / (static_cast<int>(cta.size) * kThreads);  // a thread's
    const int q0 = (static_cast<int>(cta.rank) * kThreads + static_cast<int>(threadIdx.x)) * per;
    const int q1 = min(q0 + per, kQuads), b0 = 4 * q0;
    // The cluster's counts of four positions, eight CTAs' loads under way at once.
    auto count = [&](int quad) {
      uint4 c = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
      for (uint32_t o0 = 0; o0 < cta.size; o0 += 8) {
        uint4 got[8];
#pragma unroll
        for (uint32_t o = 0; o < 8; ++o) {
          got[o] = make_uint4(0u, 0u, 0u, 0u);
          if (o0 + o < cta.size)
            asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(got[o].x), "=r"(got[o].y), "=r"(got[o].z), "=r"(got[o].w)
                         : "r"(remote(hist + 4 * quad, o0 + o))
                         : "memory");
        }
#pragma unroll
        for (uint32_t o = 0; o < 8; ++o) {
          c.x += got[o].x;
          c.y += got[o].y;
          c.z += got[o].z;
          c.w += got[o].w;
        }
      }
      return c;
    };
    unsigned n = 0;
    float lower = 0.0f, upper = 0.0f;
    const float step = br.step(), ratio = exp2f(step), low0 = exp2f(br.edge(b0)), high0 = exp2f(br.edge(b0) - step);
    float low = low0, high = high0;
    uint4 c4 = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
    for (int quad = q0; quad < q1; ++quad) {
      c4 = count(quad);
      const unsigned c[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        n += c[i];
        const float f = static_cast<float>(c[i]);
        lower += f * fmaxf(low - 0x1p-36f, 0.0f);
        upper += f * (high + 0x1p-36f);
        high = low;
        low *= ratio;
      }
    }
    // As whole numbers from here on, so that one thread's end is the next one's start.
    const u64 wl = static_cast<u64>(lower * (kOne * kBelow)), wu = static_cast<u64>(upper * (kOne * kAbove)) + (n > 0);
    const unsigned sn = warp_scan(n, lane);
    const u64 sl = warp_scan(wl, lane), su = warp_scan(wu, lane);
    if (lane == 31) {
      s.scan[0][cta.warp] = sn;
      s.scan[1][cta.warp] = sl;
      s.scan[2][cta.warp] = su;
    }
    mine = warp_sum(mine);
    if (lane == 0) s.scan[3][cta.warp] = mine;
    if (threadIdx.x == 0) {
      s.say[0] = s.say[1] = kBins - 1;
      s.say[2] = s.say[3] = ~0ull;  // not told
      s.found[0] = s.found[1] = ~0ull;
    }
    __syncthreads();
    // The warps' and the CTAs' totals, and with them the values ahead of this thread's bins.
    const bool warp_there = lane < kWarps, warp_ahead = lane < cta.warp;
    const u64 on = warp_there ? s.scan[0][lane] : 0ull, ol = warp_there ? s.scan[1][lane] : 0ull, ou = warp_there ? s.scan[2][lane] : 0ull;
    u64 fn = count_above + warp_sum(warp_ahead ? on : 0ull) + sn - n;
    u64 fl = warp_sum(warp_ahead ? ol : 0ull) + sl - wl, fu = warp_sum(warp_ahead ? ou : 0ull) + su - wu;
    u64 all = warp_sum(on), all_l = warp_sum(ol), all_u = warp_sum(ou), all_m = warp_sum(warp_there ? s.scan[3][lane] : 0ull);
    if (cta.size > 1) {
      if (threadIdx.x < cta.size) {
        remote_store(remote(&s.words[0][cta.rank], threadIdx.x), all);
        remote_store(remote(&s.words[1][cta.rank], threadIdx.x), all_l);
        remote_store(remote(&s.words[2][cta.rank], threadIdx.x), all_u);
        remote_store(remote(&s.words[3][cta.rank], threadIdx.x), all_m);
      }
      cta.sync();
      const bool there = lane < static_cast<int>(cta.size), ahead = lane < static_cast<int>(cta.rank);
      const u64 cn = there ? s.words[0][lane] : 0ull;
      all = warp_sum(cn);
      fn += warp_sum(ahead ? cn : 0ull);
      const u64 cl = there ? s.words[1][lane] : 0ull, cu = there ? s.words[2][lane] : 0ull;
      all_l = warp_sum(cl);
      all_u = warp_sum(cu);
      fl += warp_sum(ahead ? cl : 0ull);
      fu += warp_sum(ahead ? cu : 0ull);
      all_m = warp_sum(there ? s.words[3][lane] : 0ull);
    }
    if (for_k) {
      target = static_cast<u64>(q.k);
    } else if (br.fine) {
      above = all_m;
    } else {
      sum_all = all_m;
      target = share(sum_k ? sum_k : sum_all, q.part_p);
    }
    const u64 sum = for_k || br.fine ? 0 : sum_all;
    fl += above;
    fu += above;
    // Bounds on the weight down to a point that has the running sums l and u.
    auto at_least = [&](u64 l, u64 u) { return sum ? max(static_cast<long long>(l), static_cast<long long>(sum - all_u + u)) : static_cast<long long>(l); };
    auto at_most = [&](u64 l, u64 u) { return sum ? min(static_cast<long long>(u), static_cast<long long>(sum - all_l + l)) : static_cast<long long>(u); };
    const long long goal = static_cast<long long>(target);
    if (threadIdx.x == 0) s.say[4] = count_above + all;
    // The thread in whose bins a running value reaches the target says so.
    const u64 nl = fl + wl, nu = fu + wu;
    const long long start_l = at_least(fl, fu), start_u = at_most(fl, fu);
    if (n > 0 && (for_k ? fn < target && fn + n >= target
                        : (start_l < goal && at_least(nl, nu) >= goal) || (start_u < goal && at_most(nl, nu) >= goal))) {
      low = low0;
      high = high0;
      float rl = 0.0f, ru = 0.0f;
      long long at_l = start_l, at_u = start_u;
  #pragma unroll 1
    for (int quad = q0; quad < q1; ++quad) {
        if (q1 - q0 > 1) c4 = count(quad);
        const unsigned c[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const u64 b = static_cast<u64>(4 * quad + i);
          const bool end = quad == q1 - 1 && i == 3;
          const float f = static_cast<float>(c[i]);
          rl += f * fmaxf(low - 0x1p-36f, 0.0f);
          ru += f * (high + 0x1p-36f);
          const u64 run_l = end ? nl : fl + static_cast<u64>(rl * (kOne * kBelow)), run_u = end ? nu : fu + static_cast<u64>(ru * (kOne * kAbove)) + 1;
          const long long to_l = at_least(run_l, run_u), to_u = at_most(run_l, run_u);
          const u64 counted = fn;
          const bool first = for_k ? counted < target && counted + c[i] >= target : at_u < goal && to_u >= goal;
          const bool last = for_k ? first : at_l < goal && to_l >= goal;
          if (first) {
            s.found[0] = b;
            s.found[2] = fn;
          }
          fn += c[i];
          if (last) {
            s.found[1] = b;
            s.found[3] = fn;
          }
          at_l = to_l;
          at_u = to_u;
          high = low;
          low *= ratio;
        }
      }
    }
    __syncthreads();
    if (threadIdx.x < 2 * cta.size) {
      const int w = threadIdx.x & 1;
      if (s.found[w] != ~0ull) {
        remote_store(remote(&s.say[w], threadIdx.x >> 1), s.found[w]);
        remote_store(remote(&s.say[2 + w], threadIdx.x >> 1), s.found[2 + w]);
      }
    }
    cta.sync();
  };

  // All CTAs' lists behind CTA 0's; the number of keys (more than kCap:
  // they are not all there). `sum`, a value of each thread, becomes the row's.
  auto merge_lists = [&](u64& sum) -> u64 {
    sum = block_sum(sum, 0);
    const unsigned mine = s.list_len;
    if (cta.size == 1) {
      __syncthreads();  // the next pass may set it back
      return mine;
    }
    if (threadIdx.x < cta.size) {
      remote_store(remote(&s.words[0][cta.rank], threadIdx.x), mine);
      remote_store(remote(&s.words[1][cta.rank], threadIdx.x), sum);
    }
    cta.sync();
    sum = warp_sum(lane < static_cast<int>(cta.size) ? s.words[1][lane] : 0ull);
    u64 all = 0, at = 0;
#pragma unroll 1
    for (uint32_t o = 0; o < cta.size; ++o) {
      if (o < cta.rank) at += s.words[0][o];
      all += s.words[0][o];
    }
    if (cta.rank != 0 && all <= kCap)
#pragma unroll 1
      for (unsigned i = threadIdx.x; i < mine; i += kThreads) remote_store(remote(&list[at + i], 0), list[i]);
    cta.sync();
    return all;
  };

  // The row's end in CTA 0: its n <= kSmall candidates are all that may be
  // kept. Every thread takes one and looks at all of them. sum_all: what top_p
  // is a share of (0: the sum of the q.k best of the candidates).
  auto finish_small = [&](int candidates, u64 sum_all) {
    const int n = min(candidates, kSmall);
    const int t = threadIdx.x;
    const u64 key = t < n ? list[t] : 0ull;
    const float e = t < n ? ex2(sc.z(key_score(key))) : 0.0f;
    const u64 w = fixed(e);
    if (t < kSmall) {
      s.small_key[t] = key;
      s.small_w[t] = w;
    }
    __syncthreads();
    int rank = 0;
    u64 ahead = 0;  // weight of the better candidates
#pragma unroll 8
    for (int j = 0; j < n; ++j) {
      const bool better = s.small_key[j] > key;
      rank += better;
      ahead += better ? s.small_w[j] : 0ull;
    }
    bool keep = t < n && rank < q.k;
    if (by_p) {
      const u64 sum = sum_all ? sum_all : block_sum(keep ? w : 0ull, 0);
      keep = keep && ahead < share(sum, q.part_p);
    }
    keep = t < n && (rank == 0 || (keep && e >= q.min_p));
    const u64 all = block_sum(keep ? w : 0ull, 1);  // also: everyone has read small_w
    if (t < kSmall) s.small_w[t] = keep ? w : 0ull;
    __syncthreads();
    const uint32_t low = static_cast<uint32_t>(key);  // falls as the index rises
    u64 before = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) before += static_cast<uint32_t>(s.small_key[j]) > low ? s.small_w[j] : 0ull;
    const u64 aim = share(all, q.part_u);
    if (keep && before <= aim && aim < before + w) {
      a.token[r] = static_cast<int32_t>(key_index(key));
      if (a.logprob) a.logprob[r] = log_share(w, all);
    }
  };

  // In CTA 0: the largest key K of the list for which `base` plus the number
  // (for_k) or weight of its keys from K on reaches the target. Keys without
  // the bits that are the same for all are divided into kSmall buckets, then the keys of the bucket in which the target is
  // reached again, until a bucket is one key.
  auto list_cut = [&](int len, bool for_k, u64 base, u64 target) -> u64 {
    if (len <= kSmall) {  // every thread has a key and looks at all of them
      const int t = threadIdx.x;
      const u64 key = t < len ? list[t] : 0ull;
      const u64 w = t < len ? (for_k ? 1ull : weight(key_score(key), sc)) : 0ull;
      if (t < kSmall) {
        s.small_key[t] = key;
        s.small_w[t] = w;
      }
      __syncthreads();
      u64 ahead = base;
#pragma unroll 8
      for (int j = 0; j < len; ++j) ahead += s.small_key[j] > key ? s.small_w[j] : 0ull;
      if (t < len && ahead < target && ahead + w >= target) s.found[0] = key;
      __syncthreads();
      return s.found[0];
    }
    constexpr int kSame = Vec<T>::kSame;
    const int index_bits = 32 - __clz(a.vocab);
    const u64 index_mask = (u64(1) << index_bits) - 1;
    auto short_key = [&](u64 key) { return (key >> (32 + kSame)) << index_bits | (key & index_mask); };
    u64 lo = ~0ull, hi = 0;
#pragma unroll 1
    for (int j = threadIdx.x; j < len; j += kThreads) {
      const u64 k = short_key(list[j]);
      lo = umin64(lo, k);
      hi = umax64(hi, k);
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
      lo = umin64(lo, __shfl_xor_sync(kFullMask, lo, m));
      hi = umax64(hi, __shfl_xor_sync(kFullMask, hi, m));
    }
    if (lane == 0) {
      s.scan[0][cta.warp] = lo;
      s.scan[1][cta.warp] = hi;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      lo = umin64(lo, s.scan[0][w]);
      hi = umax64(hi, s.scan[1][w]);
    }
    for (;;) {  // the target is reached within [lo, hi]
      const int width = 64 - __clzll(static_cast<long long>(hi - lo));
      const int shift = max(0, width - 8);  // kSmall = 2^8 buckets
      if (threadIdx.x < kSmall) s.small_w[threadIdx.x] = 0;
      __syncthreads();
#pragma unroll 1
      for (int j = threadIdx.x; j < len; j += kThreads) {
        const u64 key = list[j], k = short_key(key);
        if (k >= lo && k <= hi) atomicAdd(&s.small_w[(k - lo) >> shift], for_k ? 1ull : weight(key_score(key), sc));
      }
      __syncthreads();
      // From the last bucket down: a thread has one.
      const int bucket = kSmall - 1 - static_cast<int>(threadIdx.x);
      const u64 w = bucket >= 0 ? s.small_w[bucket] : 0ull;
      const u64 incl = warp_scan(w, lane);
      if (lane == 31) s.scan[2][cta.warp] = incl;
      __syncthreads();
      u64 ahead = base + incl - w;
#pragma unroll
      for (int o = 0; o < kWarps; ++o)
        if (o < cta.warp) ahead += s.scan[2][o];
      if (ahead < target && ahead + w >= target) {
        s.small_key[0] = static_cast<u64>(bucket);
        s.small_key[1] = ahead;
      }
      __syncthreads();
      lo += s.small_key[0] << shift;
      base = s.small_key[1];
      hi = umin64(hi, lo + ((u64(1) << shift) - 1));
      if (shift == 0) break;
    }
#pragma unroll 1
    for (int j = threadIdx.x; j < len; j += kThreads)
      if (short_key(list[j]) == lo) s.small_key[2] = list[j];
    __syncthreads();
    return s.small_key[2];
  };

  // In CTA 0: the weight of the list's keys from `first` on.
  auto list_sum = [&](int len, u64 first) {
    u64 sum = 0;
#pragma unroll 1
    for (int j = threadIdx.x; j < len; j += kThreads)
      if (list[j] >= first) sum += weight(key_score(list[j]), sc);
    return block_sum(sum, 2);
  };
  // The warps' kept sums: what is ahead of a listed part of the scores (s.kept
  // has it), and this CTA's keys of the list (its first ones, in CTA 0's too).
  auto sum_listed = [&]() {
    const int own_len = static_cast<int>(s.list_len);
    if (threadIdx.x < kWarps) s.add_lo[threadIdx.x] = s.add_hi[threadIdx.x] = 0;
    __syncthreads();
#pragma unroll 1
    for (int j = threadIdx.x; j < own_len; j += kThreads) {
      const u64 key = list[j];
      if (key < cut) continue;
      const float e = ex2(sc.z(key_score(key)));
      if (e < q.min_p) continue;
      const u64 w = fixed(e);
      const int v = (static_cast<int>(key_index(key)) + row.lead) / E;
      int o = static_cast<int>(int64_t(v - c0) * kWarps / (c1 - c0));
      while (v >= part_of(c0, c1, o + 1)) ++o;  // the division may round down across a part's start
      atomicAdd(&s.add_lo[o], static_cast<unsigned>(w & 0x7FFFFu));  // 2^13 of them stay under 2^32
      atomicAdd(&s.add_hi[o], static_cast<unsigned>(w >> 19));
    }
    __syncthreads();
    if (threadIdx.x < kWarps) s.kept[threadIdx.x] += (static_cast<u64>(s.add_hi[threadIdx.x]) << 19) + s.add_lo[threadIdx.x];
    summed = true;
  };

  if (by_k && static_cast<u64>(q.k) <= static_cast<u64>(cta.size) * kThreads / 2) {
    // ----------------------------------------------- 3. the k best, in a list
    Bracket br;
    clear_counts();
    const float z = sc.z(x0[0]), y = Bracket::pattern(z);
    const int at = br.at(z, y);
    if (at < kBins) atomicAdd(&hist[at], 1u);
    u64 none = 0, goal = 0;
    decide(br, true, 0, 0, none, none, 0, goal);
    if (s.say[4] >= static_cast<u64>(q.k)) {
      // Every score down to the bin of the k-th largest of the threads' largest.
      const uint32_t last = static_cast<uint32_t>(s.say[1]) + Bracket::kPattern;
      each(
          [&](const float (&z)[E], int v) {
            uint32_t y[E], near = 0xFFFFFFFFu;
#pragma unroll
            for (int i = 0; i < E; ++i) {
              y[i] = __float_as_uint(Bracket::pattern(z[i]));
              near = min(near, y[i]);
            }
            if (near <= last) {  // few vectors hold any
              unsigned mask = 0;
#pragma unroll
              for (int i = 0; i < E; ++i) mask |= (y[i] <= last ? 1u : 0u) << i;
              append(mask, v);
            }
          },
          [](unsigned) {});
      const u64 n = merge_lists(none);
      if (n <= kSmall) {
        if (cta.rank == 0) finish_small(static_cast<int>(n), 0);
        return;
      }
      if (n <= kCap) {
        if (cta.rank == 0) {
          const int len = static_cast<int>(n);
          u64 key = list_cut(len, true, 0, static_cast<u64>(q.k));
          if (by_p) {  // a share of the list's keys from there on
            key = umax64(key, list_cut(len, false, 0, share(list_sum(len, key), q.part_p)));
          }
          if (threadIdx.x == 0) s.say[6] = key;
        }
        tell(6, 7);
        cut = s.say[6];
        if (lane == 0) s.kept[cta.warp] = 0;
        sum_listed();
      }
    }
    cta.sync();  // what was said has been read
  }
  if ((by_k || by_p) && !summed) {
    // --------------------------------- bins, for a large top_k, then top_p
    Bracket br;
    u64 above = 0;         // sum of weights ahead of the bins in question
    u64 count_above = 0;   // number of scores ahead of the finer bins
    u64 sum_k = 0;         // sum of what top_k kept, if not all
    u64 sum_all = 0;       // sum of all
    u64 target = 0;        // number or weight at which the prefix ends
    bool for_k = by_k;     // which of the two ends is looked for
    for (;;) {
      clear_counts();
      Mass m;
      u64 sum = 0;
      if (!br.fine) {
        const uint32_t counts = smem_addr(hist) - Bracket::kPattern * 4u;  // a pattern's count, modulo 2^32
        each(
            [&](const float (&z)[E], int) {
#pragma unroll
              for (int i = 0; i < E; ++i) {
                const uint32_t y = __float_as_uint(Bracket::pattern(z[i]));
                asm volatile(
                    "{\n\t.reg .pred p;\n\t"
                    "setp.lt.u32 p, %1, %2;\n\t"
                    "@p red.shared.add.u32 [%0], 1;\n\t}" ::"r"(counts + y * 4u),
                    "r"(y), "r"(Bracket::kPattern + kBins)
                    : "memory");
              }
              if (!for_k) {
#pragma unroll
                for (int i = 0; i < E; i += 2) m.add(ex2(z[i]), ex2(z[i + 1]));
              }
            },
            [&](unsigned n) { if (!for_k) m.flush(n); });
        sum = m.total;
      } else {
        each_one([&](float x, u64) {
          const float z = sc.z(x);
          const int at = br.at(z, Bracket::pattern(z));
          if (at >= 0 && at < kBins) atomicAdd(&hist[at], 1u);
          if (!for_k && at < 0) sum += fixed(ex2(z));
        });
      }
      decide(br, for_k, sum, sum_k, sum_all, above, count_above, target);
      const u64 reach = s.say[4];
      const u64 ahead = s.say[2];
      const u64 in = (s.say[3] == ~0ull ? reach : s.say[3]) - ahead;  // a lower bound need not get to the target
      br.from = static_cast<int>(s.say[0]);
      br.to = static_cast<int>(s.say[1]);
      u64 last_key = 0;  // 0: everything that has a weight is among the top_k
      if (br.fine || !for_k || reach > target) {
        const bool small = !for_k && !br.fine && ahead + in <= kSmall;  // all that may be kept
        if (small) br.from = 0;
        const bool listed = small || in <= kCap;
        if (!listed && !br.fine) {
          // Divide the bins again.
          Bracket f;
          f.fine = true;
          f.v0 = br.from;
          f.v1 = br.to;
          f.origin = (br.from - 0.5f) / kBinsPerOctave;
          f.scale = static_cast<float>(kBins) * kBinsPerOctave / static_cast<float>(br.to - br.from + 1);
          br = f;
          count_above = ahead;
          cta.sync();
          continue;
        }
        if (listed) {
          // --------------------------------------------------- 4. gather
          const bool weigh = !small;
          u64 ahead_sum = 0;
          if (!br.fine) {
            const uint32_t first = static_cast<uint32_t>(br.from) + Bracket::kPattern, width = static_cast<uint32_t>(br.to - br.from);
            Mass m2;
            each(
                [&](const float (&z)[E], int v) {
                  uint32_t d[E], near = 0xFFFFFFFFu;
#pragma unroll
                  for (int i = 0; i < E; ++i) {
                    d[i] = __float_as_uint(Bracket::pattern(z[i])) - first;
                    near = min(near, d[i]);
                  }
                  if (weigh) {
#pragma unroll
                    for (int i = 0; i < E; i += 2)
                      m2.add(static_cast<int>(d[i]) < 0 ? ex2(z[i]) : 0.0f, static_cast<int>(d[i + 1]) < 0 ? ex2(z[i + 1]) : 0.0f);
                  }
                  if (near <= width) {  // few vectors hold any
                    unsigned mask = 0;
#pragma unroll
                    for (int i = 0; i < E; ++i) mask |= (d[i] <= width ? 1u : 0u) << i;
                    append(mask, v);
                  }
                },
                [&](unsigned n) { if (weigh) m2.flush(n); });
            ahead_sum = m2.total;
          } else {
            each_one([&](float x, u64 key) {
              const float z = sc.z(x);
              const int at = br.at(z, Bracket::pattern(z));
              if (at >= br.from && at <= br.to) {
                const unsigned n = atomicAdd(&s.list_len, 1u);
                if (n < kCap) list[n] = key;
              }
              if (weigh && at < br.from) ahead_sum += fixed(ex2(z));
            });
          }
          const u64 own = warp_sum(ahead_sum);
          if (lane == 0) s.kept[cta.warp] = own;
          const u64 len = merge_lists(ahead_sum);
          above = ahead_sum;
          if (small) {
            if (cta.rank == 0) finish_small(static_cast<int>(len), sum_k ? sum_k : sum_all);
            return;
          }
          if (cta.rank == 0) {
            const u64 key = list_cut(static_cast<int>(len), for_k, for_k ? ahead : above, target);
            const u64 in_list = for_k && by_p ? list_sum(static_cast<int>(len), key) : 0;
            if (threadIdx.x == 0) {
              s.say[5] = in_list;
              s.say[6] = key;
            }
          }
          tell(5, 7);
          last_key = s.say[6];
          sum_k = above + s.say[5];
          if (!(for_k && by_p) && q.min_p == 0.0f) {
            cut = last_key;
            sum_listed();
          }
        } else {
          // Equal scores by the thousand: halve the interval between the
          // smallest and the largest key of the finer bins.
          u64 lo = 0, hi = 0;  // the complement of the smallest; the largest
          each_one([&](float x, u64 key) {
            const float z = sc.z(x);
            const int at = br.at(z, Bracket::pattern(z));
            if (at >= br.from && at <= br.to) {
              lo = umax64(lo, ~key);
              hi = umax64(hi, key);
            }
          });
          lo = ~cta.template reduce<true>(lo);
          hi = cta.template reduce<true>(hi) + 1;
          while (hi - lo > 1) {
            const u64 mid = lo + (hi - lo) / 2;
            u64 c = 0;
            each_one([&](float x, u64 key) {
              if (key >= mid) c += for_k ? 1ull : weight(x, sc);
            });
            if (cta.template reduce<false>(c) >= target)
              lo = mid;
            else
              hi = mid;
          }
          last_key = lo;
          if (for_k && by_p) {
            each_one([&](float x, u64 key) { sum_k += key >= lo ? weight(x, sc) : 0ull; });
            sum_k = cta.template reduce<false>(sum_k);
          }
        }
      }
      cut = umax64(cut, last_key);
      if (!for_k || !by_p) break;
      // Now top_p, of the weight that top_k kept: it ends no later.
      for_k = false;
      above = 0;
      count_above = 0;
      br = Bracket();
      cta.sync();
    }
  }

  // ------------------------------------------------- the warps' kept sums
  if (!summed) {
    u64 sum = 0;
    if (cut == 0) {
      Mass m;
      each(
          [&](const float (&z)[E], int) {
            const float least = q.min_p;
#pragma unroll
            for (int i = 0; i < E; i += 2) {
              const float ea = ex2(z[i]), eb = ex2(z[i + 1]);
              m.add(ea >= least ? ea : 0.0f, eb >= least ? eb : 0.0f);
            }
          },
          [&](unsigned n) { m.flush(n); });
      sum = m.total;
    } else {
      each_one([&](float x, u64 key) {
        const float e = ex2(sc.z(x));
        if (key >= cut && e >= q.min_p) sum += fixed(e);
      });
    }
    sum = warp_sum(sum);
    if (lane == 0) s.kept[cta.warp] = sum;
  }
  __syncthreads();
  const u64 total = cta.reduce<false>(lane == 0 ? s.kept[cta.warp] : 0ull);
  const u64 aim = share(total, q.part_u);
  u64 before = 0;
  u64 mine_all = total;
  if (cta.size > 1) {
#pragma unroll 1
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
#pragma unroll 1
    for (int v = part_of(n0, n1, cta.warp) + lane; v < m1; v += 32) part += kept_of(v);
    part = warp_sum(part);
    if (lane == 0) s.kept[cta.warp] = part;
    __syncthreads();
  }
  __syncthreads();
  if (cta.warp == 0) {
    const int v = s.lo + lane;
    const u64 sum = v < s.hi ? kept_of(v) : 0ull;
    u64 run = s.before + warp_scan(sum, lane) - sum;
    if (sum > 0 && run <= aim && aim < run + sum) {
#pragma unroll 1
      for (int i = 0; i < E; ++i) {
        const u64 w = kept(v, i);
        if (run <= aim && aim < run + w) {
          a.token[r] = index_of(v, i);
          if (a.logprob) a.logprob[r] = log_share(w, total);
        }
        run += w;
      }
    }
  }
}

template <typename T, bool HELD, int kThreads>
cudaError_t launch_t(const SampleLaunch& a, int cluster, int held_bytes, cudaStream_t st) {
  auto fn = sample_kernel<T, HELD, kThreads>;
  static PerDeviceOnce once;
  const cudaError_t ready = once.run([fn] {
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    return e != cudaSuccess ? e : cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  });
  if (ready != cudaSuccess) return ready;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.rows * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kListCap<HELD> * sizeof(u64) + static_cast<size_t>(held_bytes);
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
  // A CTA's part in shared memory: 32 KB leaves room for four CTAs an SM (of 57
  // KB with the counts), whose reads overlap the others' passes.
  int cluster = 1;
  while (cluster < kMaxCluster && bytes / cluster > 32 * 1024) cluster *= 2;
  const int64_t held = (bytes + cluster - 1) / cluster / 16 * 16 + 32;
  if (held <= kMaxHeld) return launch_t<T, true, 256>(a, cluster, static_cast<int>(held), st);
  // Longer parts are read again from L2, with two CTAs an SM: a cluster of 16
  // CTAs that fill an SM each finds room in few of the GPU's clusters of SMs (8
  // rows of 1M with min_p: 28 us against 37 with 1,024 threads a CTA, half of
  // the rows waiting; 25 since the text is shorter).
  return launch_t<T, false, 512>(a, cluster, 0, st);
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
