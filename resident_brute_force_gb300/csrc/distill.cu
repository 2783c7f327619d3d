// distill.cu -- loss and gradient of a distillation from a teacher's best logits
// (include/rbf_ops.h, distill_dev).
//
// Of a row: p = softmax of the teacher's k logits / T and its remaining mass r
// (if any), q = softmax(scores / T), L the listed indices. With P and Q the masses
// of L and softmax_rest the softmax of the other scores,
//   loss           = T^2 [sum_e p_e log(p_e / q_e) + p_r log(p_r / (1 - Q))]
//   d loss / d s_j = T (q_j - sum of p_e at j)             j in L
//                    T softmax_rest_j ((1 - Q) - p_r)      else
// and (1 - Q) - p_r = P - Q: whichever of the two has the smaller terms is taken.
// The masses of the listed and of the other scores are summed apart, each below its
// own largest score, so that neither is a difference and a small one keeps its bits.
//
// A cluster of CTAs a row. A CTA copies its part of the row into shared memory
// (cp.async.bulk), takes the listed scores out of it (their place is -infinity from
// then on), finds the largest and the sum of the others, and after one exchange
// over the cluster writes the gradient from shared memory: a row is read once. A
// part that does not fit is taken in pieces, which are read twice.
//
// What bounds it: HBM, whose two directions are not both busy all the time: bf16 4096 x
// 128000 458 us (2.1 GB at 4.6 TB/s; 310 at the copy rate), its loss alone 267 (155). Clusters that
// go on to the next row took 340 for that. With long lists, the search for entries of the
// same index, which grows with the square of their number: 2591 us at 1024 entries a row.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "ops_internal.h"
#include "rbf_device.cuh"
#include "rbf_internal.h"
#include "score_rows.cuh"

namespace rbf {
namespace {

constexpr int kMaxCluster = 16;
constexpr int kPiece = 64 * 1024;  // bytes of a row in a CTA's shared memory, at most
// Up to this a CTA takes the row alone: three CTAs an SM, one of which reads while
// another writes. With 32 KB, in us: bf16 4096 x 128000 524 in place of 458 (310 for the
// bytes), fp32 4096 x 10000 95 in place of 64 (49), fp16 509 x 100003 68 in place of 52.
constexpr int kAim = kPiece;
// Up to this a CTA has 64 threads: it is bound by its steps, and many run at once. bf16 4096 x 1000
// takes 21 us, 40 with 256 threads. (512 threads for the others: no gain.)
constexpr int kSmallCta = 8192;
constexpr int kBigThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLn2Low = 0.6931471805599453 - static_cast<double>(kLn2);  // what fp32 leaves out

// The number of a score in shared memory that is not one of the types', as its bits.
template <typename T>
struct Bits {
  using type = uint16_t;
  static constexpr uint16_t kNone = std::is_same<T, __nv_bfloat16>::value ? 0xFF80u : 0xFC00u;
};
template <>
struct Bits<float> {
  using type = uint32_t;
  static constexpr uint32_t kNone = 0xFF800000u;
};

__device__ __forceinline__ float read_float(const void* p, int64_t i, int dtype) {
  if (dtype == kF32) return static_cast<const float*>(p)[i];
  if (dtype == kBF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}

template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }

template <typename T>
__device__ __forceinline__ uint4 pack_vec(const float (&g)[Vec<T>::kLen]) {
  uint4 r;
  T* e = reinterpret_cast<T*>(&r);
#pragma unroll
  for (int i = 0; i < Vec<T>::kLen; ++i) e[i] = from_float<T>(g[i]);
  return r;
}

// A number as the sum of two fp32 ones: a loss is a small difference of sums, and
// 64-bit arithmetic runs at a 64th of fp32's rate here. Pairs are a thread's sum of the
// scores that are not listed over a row's pieces (256 in a row of 2^26, whose roundings may
// all be alike), the sums of p_e and of the products with it, and what follows from
// them. Threads' sums are joined in fp32, up to twelve additions of half a step each (in
// pairs: bf16 4096 x 128000 471 us in place of 458, fp32 1 x 10000 8.3 in place of 7.4), and
// so are the at most 1024 weights of a list; the last addition keeps what it leaves out.
struct Pair {
  float h = 0.0f, l = 0.0f;
};
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb))};
}
__device__ __forceinline__ Pair two_product(float a, float b) {
  const float p = __fmul_rn(a, b);
  return {p, __fmaf_rn(a, b, -p)};
}
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
  const Pair s = two_sum(a.h, b.h);
  return {s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l))};
}

// A loss is summed in units of 2^34: T is 2^-20 at least, so that nothing on the way to
// T^2 weight times it passes fp32's range where the loss itself does not (a listed score at its
// type's lowest value is 3.4e38 away). Powers of two change no bit.
constexpr float kUnit = 0x1p34f, kPerUnit = 0x1p-34f;

// What a CTA says of its part to all of its cluster, two floats a word: the largest
// and the sum of the scores that are not listed, the same of the listed ones, the sum
// of p_e ((t_e - largest t) - (s_e - largest of these)) in units of a loss (infinite where a
// listed score is -infinity), and of p_e.
constexpr int kWords = 4;

// The weight 2^((x - top) rate), 0 where nothing is left.
__device__ __forceinline__ float weight_of(float x, float top, float rate) {
  return x == -INFINITY ? 0.0f : ex2(__fmul_rn(__fsub_rn(x, top), rate));
}

template <typename V, typename F>
__device__ __forceinline__ V warp_fold(V v, F&& f) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = f(v, __shfl_xor_sync(kFullMask, v, d));
  return v;
}

// Shared memory of a CTA behind its piece of the row: five words an entry, and a
// hash table of two words a slot for the first entry of each index.
__host__ __device__ constexpr int table_bits(int k) {
  int b = 5;
  while ((1 << b) < 2 * k) ++b;
  return b;
}
__host__ __device__ constexpr int list_bytes(int k) { return k ? 20 * k + (8 << table_bits(k)) : 0; }

template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads) distill_kernel(const DistillLaunch a, int piece_bytes, int cluster_bits, int bits, float rate, int* err,
                                                                  uint64_t timeout_ns) {
  constexpr int E = Vec<T>::kLen;
  constexpr int kWarps = kThreads / 32;
  using B = typename Bits<T>::type;
  extern __shared__ __align__(16) uint8_t dyn[];
  T* piece = reinterpret_cast<T*>(dyn);                                   // piece_bytes
  int* at = reinterpret_cast<int*>(dyn + piece_bytes);                    // [k] index, -1: not in this CTA's part
  float* logit = reinterpret_cast<float*>(at + a.k);                      // [k] the teacher's, -infinity: no entry
  float* score = logit + a.k;                                             // [k] the student's, at the first entry of an index
  float* prob = score + a.k;                                              // [k] p_e
  int* owner = reinterpret_cast<int*>(prob + a.k);                        // [k] the first entry with the same index
  int* key = owner + a.k;                                                 // the table: an index, and its first entry
  int* first = key + (1 << bits);
  __shared__ uint64_t full;
  __shared__ float red[2][kWarps];
  __shared__ float of_warp[9][32];  // what each warp says of its part; zeros past kWarps
  __shared__ u64 said[kMaxCluster][kWords];

  uint32_t rank;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const uint32_t size = 1u << cluster_bits;
  if (size > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t r = blockIdx.x >> cluster_bits;
  // The row's first entries and its numbers are on their way from here on.
  int j_first = -1;
  float t_first = -INFINITY;
  if (tid < a.k) {
    j_first = a.index[r * a.ld_index + tid];
    t_first = read_float(a.teacher, r * a.ld_teacher + tid, a.teacher_dtype);
  }
  const float w_row = a.weight ? a.weight[r] : 1.0f;
  const float rest_raw = a.rest ? a.rest[r] : -INFINITY;
  const T* row = static_cast<const T*>(a.scores) + r * a.ld_scores;
  const int lead = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
  const int vecs = static_cast<int>((int64_t(a.vocab) + lead + E - 1) / E);
  const int c0 = static_cast<int>(int64_t(vecs) * rank >> cluster_bits), c1 = static_cast<int>(int64_t(vecs) * (rank + 1) >> cluster_bits);
  const int piece_vecs = piece_bytes / 16;
  const int pieces = c1 - c0 <= piece_vecs ? 1 : (c1 - c0 + piece_vecs - 1) / piece_vecs;
  if (tid == 0) {
    mbar_init(&full, 1);
    fence_mbar_init();
  }

  // Vectors [v0, v1) of the row into shared memory, -infinity outside of the row.
  const uint64_t policy = l2_policy_evict_first();
  uint32_t phase = 0;
  bool ok = true;
  auto fetch = [&](int v0, int v1) {
    // The vectors that lie inside of the row.
    const int f0 = max(v0, lead > 0 ? 1 : 0), f1 = max(f0, min(v1, static_cast<int>((int64_t(a.vocab) + lead) / E)));
    if (tid == 0) {
      const uint32_t bytes = static_cast<uint32_t>(f1 - f0) * 16u;
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // what was there has been read and written by threads
      mbar_arrive_expect_tx(&full, bytes);
      if (bytes) bulk_copy_g2s(piece + static_cast<int64_t>(f0 - v0) * E, row - lead + static_cast<int64_t>(f0) * E, bytes, &full, policy);
    }
    if (tid >= 32 && tid < 32 + 2 * E) {  // the one or two others
      const int v = tid < 32 + E ? v0 : v1 - 1, i = (tid - 32) % E;
      if (v0 < v1 && (v < f0 || v >= f1)) {
        const int64_t j = int64_t(v) * E - lead + i;
        if (j >= 0 && j < a.vocab)
          piece[(v - v0) * E + i] = row[j];
        else
          reinterpret_cast<B*>(piece)[(v - v0) * E + i] = Bits<T>::kNone;
      }
    }
  };
  auto arrived = [&]() {
    // One thread looks, the others wait at the barrier: all of them looking takes
    // the issue slots that the SM's other CTAs compute in.
    if (tid == 0 && !mbar_wait(&full, phase, timeout_ns)) {
      ok = false;
      mbar_wait(&full, phase, timeout_ns);  // no copy may be in flight when the CTA exits
    }
    phase ^= 1u;
    ok = __syncthreads_and(ok) != 0;
    if (!ok && tid == 0) atomicOr(err, kErrConsumerTimeout);
  };
  fetch(c0, min(c1, c0 + piece_vecs));  // its barrier is the issuing thread's own so far
  if (a.k)
    for (int s = tid; s < 2 << bits; s += kThreads) key[s] = s < 1 << bits ? -1 : INT32_MAX;
  for (int i = tid; i < 9 * 32; i += kThreads) of_warp[0][i] = i < 64 ? -INFINITY : 0.0f;  // two largest scores, seven sums
  __syncthreads();

  // ------------------------------------------- the teacher, ahead of the scores
  const float rest_t = rest_raw * a.temperature;  // as a logit
  float top_t = rest_t;
  for (int e = tid; e < a.k; e += kThreads) {
    const int j = e == tid ? j_first : a.index[r * a.ld_index + e];
    const bool there = j >= 0 && j < a.vocab;
    float t = e == tid ? t_first : read_float(a.teacher, r * a.ld_teacher + e, a.teacher_dtype);
    if (!there) t = -INFINITY;
    const int64_t v = there ? (int64_t(j) + lead) / E : -1;
    const bool mine = v >= c0 && v < c1;
    at[e] = mine ? j : -1;
    logit[e] = t;
    top_t = fmaxf(top_t, t);
    if (mine) {  // a slot of its index: whatever the order, the smallest entry stays
      const uint32_t mask = (1u << bits) - 1;
      uint32_t s = (static_cast<uint32_t>(j) * 2654435761u) >> (32 - bits);
      for (int old; (old = atomicCAS(&key[s], -1, j)) != -1 && old != j;) s = (s + 1) & mask;
      atomicMin(&first[s], e);
      owner[e] = static_cast<int>(s);
    }
  }
  auto fmax2 = [](float x, float y) { return fmaxf(x, y); };
  auto plus = [](auto x, auto y) { return x + y; };
  // Over the CTA, in the warps' order; `slot`: each reduction's own words.
  auto post = [&](int slot, float v) {
    if (lane == 0) red[slot][warp] = v;
  };
  auto fold = [&](int slot, auto&& f) {
    float v = red[slot][lane % kWarps];
#pragma unroll
    for (int d = kWarps / 2; d > 0; d >>= 1) v = f(v, __shfl_xor_sync(kFullMask, v, d));
    return v;
  };
  post(0, warp_fold(top_t, fmax2));
  __syncthreads();
  top_t = fold(0, fmax2);
  float z_t = 0.0f;
  for (int e = tid; e < a.k; e += kThreads) {
    const float p = weight_of(logit[e], top_t, rate);
    prob[e] = p;
    z_t += p;
    if (at[e] >= 0) owner[e] = first[owner[e]];
  }
  post(1, warp_fold(z_t, plus));

  // ------------------------------------------------------------ the student
  // Of a thread: the largest of its scores that are not listed, and the sum of
  // their weights below that.
  float top_rest = -INFINITY, top_in = -INFINITY;
  Pair z_rest;
  for (int p = 0; p < pieces; ++p) {
    const int v0 = c0 + p * piece_vecs, v1 = min(c1, v0 + piece_vecs);
    if (p > 0) {
      __syncthreads();  // the last piece has been read
      fetch(v0, v1);
    }
    arrived();
    if (!ok) break;
    // The listed scores are taken out.
    const int64_t j0 = int64_t(v0) * E - lead, j1 = int64_t(v1) * E - lead;
    for (int e = tid; e < a.k; e += kThreads) {
      const int j = at[e];
      if (j >= j0 && j < j1 && owner[e] == e) {
        const float s = Vec<T>::one(piece[j - j0]);
        reinterpret_cast<B*>(piece)[j - j0] = Bits<T>::kNone;
        score[e] = s;
      }
    }
    __syncthreads();
    const uint4* src = reinterpret_cast<const uint4*>(piece);
    // Of a thread's first scores the largest is found at once, then that of
    // four vectors at a time (a NaN loses: the sum finds it).
    float z_piece = 0.0f;  // of sixteen vectors at most
#pragma unroll 1
    for (int v = tid; v < v1 - v0; v += 4 * kThreads) {
      uint4 raw[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) raw[i] = v + i * kThreads < v1 - v0 ? src[v + i * kThreads] : vec_none<T>();
      float x[E];
      const float top = vec_top<T>(vec_max<T>(vec_max<T>(raw[0], raw[1]), vec_max<T>(raw[2], raw[3])));
      if (top > top_rest) {
        const float less = weight_of(top_rest, top, rate);
        z_rest = {z_rest.h * less, z_rest.l * less};
        z_piece *= less;
        top_rest = top;
      }
      const float base = top_rest == -INFINITY ? 0.0f : top_rest;
      const u64 nbase2 = pack2(-base, -base), rate2 = pack2(rate, rate);
      u64 sum[2] = {0, 0};  // two zeros each
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        Vec<T>::unpack(raw[i], x);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const u64 z = mul2(add2(pack2(x[e], x[e + 1]), nbase2), rate2);
          sum[e / 2 % 2] = add2(sum[e / 2 % 2], pack2(ex2(low2(z)), ex2(high2(z))));
        }
      }
      sum[0] = add2(sum[0], sum[1]);
      z_piece += low2(sum[0]) + high2(sum[0]);
    }
    z_rest = z_rest + Pair{z_piece, 0.0f};
  }

  // With what fp32 leaves out of rest * T.
  const float rest_low = fabsf(rest_t) < 1.0e30f ? __fmaf_rn(rest_raw, a.temperature, -rest_t) : 0.0f;
  const float rest_w = __fmaf_rn(weight_of(rest_t, top_t, rate), rest_low * rate * kLn2, weight_of(rest_t, top_t, rate));
  z_t = fold(1, plus);
  const float all_t = z_t + rest_w;
  const float inv_t = all_t == 0.0f ? 0.0f : 1.0f / all_t;
  const float p_in = z_t * inv_t, p_rest = rest_w * inv_t;
  {
    // The warp's, below its own largest.
    const float top = warp_fold(top_rest, fmax2);
    const float z = warp_fold((z_rest.h + z_rest.l) * weight_of(top_rest, top, rate), plus);  // of a thread's own -infinity: 0, or NaN
    if (lane == 0) {
      of_warp[0][warp] = top;
      of_warp[2][warp] = z;
    }
  }
  if (warp * 32 < a.k) {
    // The warp's listed scores: the sum, and the products, each below their
    // largest: beside scores at the type's lowest value a teacher's logit would vanish.
    for (int e = tid; e < a.k; e += kThreads)
      if (at[e] >= 0) top_in = fmaxf(top_in, score[owner[e]]);
    top_in = warp_fold(top_in, fmax2);
    float z_in = 0.0f, missed = 0.0f;
    Pair diff, mass;
    for (int e = tid; e < a.k; e += kThreads) {
      if (at[e] < 0) continue;
      const float s = score[owner[e]];
      if (owner[e] == e) z_in += weight_of(s, top_in, rate);
      if (prob[e] > 0.0f) {
        const float p = prob[e] * inv_t;
        if (s == -INFINITY)
          missed = 1.0f;
        else
          diff = diff + two_product(p, (logit[e] - top_t) * kPerUnit - (s * kPerUnit - top_in * kPerUnit));
        mass = mass + Pair{p, 0.0f};
      }
    }
    z_in = warp_fold(z_in, plus);
    missed = warp_fold(missed, fmax2);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      diff = diff + Pair{__shfl_xor_sync(kFullMask, diff.h, d), __shfl_xor_sync(kFullMask, diff.l, d)};
      mass = mass + Pair{__shfl_xor_sync(kFullMask, mass.h, d), __shfl_xor_sync(kFullMask, mass.l, d)};
    }
    if (lane == 0) {
      of_warp[1][warp] = top_in;
      of_warp[3][warp] = z_in;
      of_warp[4][warp] = mass.h;
      of_warp[8][warp] = mass.l;
      of_warp[5][warp] = missed;
      of_warp[6][warp] = diff.h;
      of_warp[7][warp] = diff.l;
    }
  }
  if (size > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  __syncthreads();
  if (warp == 0) {
    // The warps' below the CTA's largest, and their sums, a warp a lane.
    auto among = [&](float v, auto&& f) {
#pragma unroll
      for (int d = kWarps / 2; d > 0; d >>= 1) v = f(v, __shfl_xor_sync(kFullMask, v, d));
      return __shfl_sync(kFullMask, v, 0);
    };
    const float wr = of_warp[0][lane], wi = of_warp[1][lane], m = of_warp[4][lane];
    const float tr = among(wr, fmax2), ti = among(wi, fmax2);
    const float zr = among(wr == -INFINITY ? of_warp[2][lane] : of_warp[2][lane] * weight_of(wr, tr, rate), plus);
    const float zi = among(wi == -INFINITY ? of_warp[3][lane] : of_warp[3][lane] * weight_of(wi, ti, rate), plus);
    Pair d{of_warp[6][lane], of_warp[7][lane]};
    if (m > 0.0f && wi > -INFINITY) {
      const Pair apart = two_sum(ti * kPerUnit, -wi * kPerUnit), part = two_product(m, apart.h);
      d = d + Pair{part.h, __fmaf_rn(m, apart.l, part.l)};
    }
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) d = d + Pair{__shfl_xor_sync(kFullMask, d.h, o), __shfl_xor_sync(kFullMask, d.l, o)};
    d = {__shfl_sync(kFullMask, d.h, 0), __shfl_sync(kFullMask, d.l, 0)};
    if (among(of_warp[5][lane], fmax2) > 0.0f) d = {INFINITY, 0.0f};
    Pair mass{m, of_warp[8][lane]};
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) mass = mass + Pair{__shfl_xor_sync(kFullMask, mass.h, o), __shfl_xor_sync(kFullMask, mass.l, o)};
    mass = {__shfl_sync(kFullMask, mass.h, 0), __shfl_sync(kFullMask, mass.l, 0)};
    for (int i = lane; i < kWords * static_cast<int>(size); i += 32) {
      const int word = i % kWords;
      const float lo = word == 0 ? tr : word == 1 ? ti : word == 2 ? d.h : mass.h;
      const float hi = word == 0 ? zr : word == 1 ? zi : word == 2 ? d.l : mass.l;
      remote_store(remote(&said[rank][word], static_cast<uint32_t>(i / kWords)), static_cast<u64>(__float_as_uint(hi)) << 32 | __float_as_uint(lo));
    }
  }
  if (size > 1)
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  else
    __syncthreads();
  if (!ok) return;

  // Every thread joins what the CTAs have said, in their order (one warp's word to
  // the others would take a barrier more); a loss alone is for rank 0's first one.
  if (!a.grad && (rank != 0 || warp != 0)) return;
  auto low = [&](uint32_t c, int word) { return __uint_as_float(static_cast<uint32_t>(said[c][word])); };
  auto high = [&](uint32_t c, int word) { return __uint_as_float(static_cast<uint32_t>(said[c][word] >> 32)); };
  float tr = -INFINITY, ti = -INFINITY, zr = 0.0f, zi = 0.0f;
  for (uint32_t c = 0; c < size; ++c) {
    tr = fmaxf(tr, low(c, 0));
    ti = fmaxf(ti, low(c, 1));
  }
  for (uint32_t c = 0; c < size; ++c) {
    zr += low(c, 0) == -INFINITY ? high(c, 0) : high(c, 0) * weight_of(low(c, 0), tr, rate);  // 0, or a NaN that is alone
    zi += low(c, 1) == -INFINITY ? high(c, 1) : high(c, 1) * weight_of(low(c, 1), ti, rate);
  }
  // Both below one score: what is left of the other's weight is a factor.
  const float top_s = fmaxf(tr, ti);
  const float fr = weight_of(tr, top_s, rate), fi = weight_of(ti, top_s, rate);  // one of them 1
  const float zr_s = zr * fr, zi_s = zi * fi, z_s = zr_s + zi_s;
  const bool no_teacher = all_t == 0.0f, no_student = z_s == 0.0f;
  const bool live = !no_teacher && !no_student && w_row != 0.0f;
  const float inv_s = 1.0f / z_s;
  const float q_in = zi_s * inv_s, q_rest = zr_s * inv_s;

  if (a.loss && rank == 0 && tid == 0) {
    float loss = 0.0f;
    if (live) {
      // sum p_e (log p_e - log q_e) = sum p_e ((t_e - largest t) - (s_e - largest s)) / T - P log(Z_t / Z_s)
      // with P the sum of the very numbers p_e that stand in the first sum.
      Pair l, mass;
      bool missed = false;
      for (uint32_t c = 0; c < size; ++c) {
        const float m = low(c, 3);
        missed |= low(c, 2) == INFINITY;
        l = l + Pair{low(c, 2), high(c, 2)};
        mass = mass + Pair{m, high(c, 3)};
        if (m > 0.0f && low(c, 1) > -INFINITY) {
          const Pair apart = two_sum(top_s * kPerUnit, -low(c, 1) * kPerUnit), part = two_product(m, apart.h);
          l = l + Pair{part.h, __fmaf_rn(m, apart.l, part.l)};
        }
      }
      // Over the very T of the weights, log2(e) / rate: its 2^-25 would stand against logarithms of their sums.
      Pair of_t = two_product(rate, kLn2);
      of_t.l = __fmaf_rn(rate, kLn2Low, of_t.l);
      const Pair by_t = two_product(l.h, of_t.h);
      l = {by_t.h, by_t.l + __fmaf_rn(l.h, of_t.l, l.l * of_t.h)};
      if (p_in > 0.0f) {
        // The sums with what their last addition and the division leave out.
        const Pair zt = two_sum(z_t, rest_w), zs = two_sum(zr_s, zi_s);
        const float r = zt.h / zs.h;
        const float left = (__fmaf_rn(-r, zs.h, zt.h) + zt.l - r * zs.l) / zt.h;
        // log r = n log 2 + the logarithm of a number near 1, which keeps its last bits.
        const int bits_r = __float_as_int(r), n = (bits_r - 0x3F3504F3) >> 23;
        const float of_n = static_cast<float>(n);
        const Pair whole = two_product(of_n, kLn2), near = two_sum(whole.h, logf(__int_as_float(bits_r - (n << 23))));
        const Pair log_r{near.h, near.l + whole.l + of_n * kLn2Low + left};
        mass = {mass.h * kPerUnit, mass.l * kPerUnit};
        const Pair part = two_product(-mass.h, log_r.h);
        l = l + Pair{part.h, __fmaf_rn(-mass.h, log_r.l, __fmaf_rn(-mass.l, log_r.h, part.l))};
      }
      // p_r / q_r as (1 + listed / others) of both
      if (p_rest > 0.0f) {
        float ls;
        if (zr_s > 1.0e-30f) {
          ls = log1pf(zi_s / zr_s) * kPerUnit;
        } else if (zr > 0.0f) {
          ls = logf(zi / zr) * kPerUnit + (ti * kPerUnit - tr * kPerUnit) * rate * kLn2;
        } else {
          ls = INFINITY;
        }
        const float ratio_t = z_t / rest_w;
        const float lt = ratio_t < 1.0e30f ? log1pf(ratio_t) : logf(z_t) - logf(rest_w);
        l = ls == INFINITY ? Pair{INFINITY, 0.0f} : l + two_product(p_rest, ls - lt * kPerUnit);
      }
      loss = missed ? INFINITY : l.h + l.l;
      if (l.h == INFINITY) loss = INFINITY;
      if (p_in != p_in || z_s != z_s) loss = p_in + z_s;
      loss = loss * a.temperature * a.temperature;
      loss = fabsf(loss * kUnit) < INFINITY ? loss * kUnit * w_row : loss * w_row * kUnit;
    }
    a.loss[r] = loss;
  }
  if (!a.grad) return;

  // ----------------------------------------------------------- the gradient
  const float scale = live ? w_row * a.temperature : 0.0f;
  float factor = 0.0f;  // of a score that is not listed: softmax_rest times this
  if (live && zr != 0.0f)
    factor = scale * (p_rest == 0.0f ? q_rest : p_in < 0.5f ? p_in - q_in : q_rest - p_rest) / zr;
  else if (live)  // all of them at -infinity: 0, or a NaN of the list, the teacher or the weight
    factor = scale * (0.0f * (z_s + all_t));
  const float base = tr == -INFINITY ? 0.0f : tr;
  T* out = static_cast<T*>(a.grad) + r * a.ld_grad;
  const bool same = (reinterpret_cast<uintptr_t>(out) & 15) == (reinterpret_cast<uintptr_t>(row) & 15);
  for (int p = 0; p < pieces; ++p) {
    const int v0 = c0 + p * piece_vecs, v1 = min(c1, v0 + piece_vecs);
    const int64_t j0 = int64_t(v0) * E - lead, j1 = int64_t(v1) * E - lead;
    if (pieces > 1) {
      __syncthreads();
      fetch(v0, v1);
      arrived();
      if (!ok) return;
      for (int e = tid; e < a.k; e += kThreads)
        if (at[e] >= j0 && at[e] < j1) reinterpret_cast<B*>(piece)[at[e] - j0] = Bits<T>::kNone;
      __syncthreads();
    }
    const uint4* src = reinterpret_cast<const uint4*>(piece);
    const u64 nbase2 = pack2(-base, -base), rate2 = pack2(rate, rate), factor2 = pack2(factor, factor);
    auto grad_of = [&](float x) { return live ? ex2(__fmul_rn(__fsub_rn(x, base), rate)) * factor : 0.0f; };
    if (same) {
      // The vectors inside of the row, then the one or two that reach past it.
      const int f0 = max(v0, lead > 0 ? 1 : 0) - v0, f1 = min(v1, static_cast<int>((int64_t(a.vocab) + lead) / E)) - v0;
      uint4* to = reinterpret_cast<uint4*>(out + j0);
      if (live) {
#pragma unroll 2
        for (int v = f0 + tid; v < f1; v += kThreads) {
          float x[E], g[E];
          Vec<T>::unpack(src[v], x);
#pragma unroll
          for (int i = 0; i < E; i += 2) {
            const u64 z = mul2(add2(pack2(x[i], x[i + 1]), nbase2), rate2);
            const u64 w = mul2(pack2(ex2(low2(z)), ex2(high2(z))), factor2);
            g[i] = low2(w);
            g[i + 1] = high2(w);
          }
          __stcs(to + v, pack_vec<T>(g));
        }
      } else {
        for (int v = f0 + tid; v < f1; v += kThreads) __stcs(to + v, make_uint4(0u, 0u, 0u, 0u));
      }
      if (tid < 2 * E && v0 < v1) {
        const int v = tid < E ? 0 : v1 - v0 - 1;
        const int64_t j = j0 + int64_t(v) * E + tid % E;
        if ((v < f0 || v >= f1) && j >= 0 && j < a.vocab) out[j] = from_float<T>(grad_of(Vec<T>::one(piece[j - j0])));
      }
    } else {
      for (int64_t j = max(j0, int64_t(0)) + tid; j < min(j1, int64_t(a.vocab)); j += kThreads) out[j] = from_float<T>(grad_of(Vec<T>::one(piece[j - j0])));
    }
  }
  if (!live) return;
  // The listed ones: the first entry of an index adds up the probabilities of all that name it.
  __syncthreads();
  for (int e = tid; e < a.k; e += kThreads) {
    if (at[e] < 0 || owner[e] != e) continue;
    float p = prob[e];
    for (int o = e + 1; o < a.k; ++o)
      if (at[o] == at[e]) p += prob[o];
    const float q = weight_of(score[e], top_s, rate) * inv_s;  // at its first entry
    out[at[e]] = from_float<T>(scale * (q - p * inv_t));
  }
}

template <typename T, int kThreads>
cudaError_t launch_t(const DistillLaunch& a, int cluster_bits, int piece, int* err, uint64_t timeout_ns, cudaStream_t st) {
  const int cluster = 1 << cluster_bits;
  auto fn = distill_kernel<T, kThreads>;
  static PerDeviceOnce once;
  const cudaError_t ready = once.run([fn] {
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kPiece + list_bytes(kMaxTeacher));
    return e != cudaSuccess ? e : cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  });
  if (ready != cudaSuccess) return ready;
  // A grid has 2^31 - 1 CTAs: more rows go in parts.
  for (int64_t r = 0; r < a.rows; r += int64_t(1) << 26) {
    DistillLaunch p = a;
    p.rows = std::min<int64_t>(a.rows - r, int64_t(1) << 26);
    p.scores = static_cast<const T*>(a.scores) + r * a.ld_scores;
    p.index = a.index ? a.index + r * a.ld_index : nullptr;
    p.teacher = static_cast<const char*>(a.teacher) + r * a.ld_teacher * dtype_bytes(a.teacher_dtype);
    p.rest = a.rest ? a.rest + r : nullptr;
    p.weight = a.weight ? a.weight + r : nullptr;
    p.loss = a.loss ? a.loss + r : nullptr;
    p.grad = a.grad ? static_cast<T*>(a.grad) + r * a.ld_grad : nullptr;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.rows * cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(piece + list_bytes(a.k));
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1;  // a launch with clusters starts its CTAs more slowly
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, p, piece, cluster_bits, table_bits(a.k), kLog2e / a.temperature, err, timeout_ns);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename T>
cudaError_t launch_rows(const DistillLaunch& a, int* err, uint64_t timeout_ns, int num_sms, cudaStream_t st) {
  const int64_t bytes = (int64_t(a.vocab) * static_cast<int64_t>(sizeof(T)) / 16 + 2) * 16;
  int bits = 0;  // of the cluster's size
  while (1 << bits < kMaxCluster && (bytes >> bits) + 16 > kAim) ++bits;
  // Few rows: more CTAs a row, of 8 KB at least, until there are two an SM.
  while (1 << bits < kMaxCluster && a.rows << bits < 2 * num_sms && bytes >> bits > 8192) ++bits;
  const int piece = static_cast<int>(std::min<int64_t>(kPiece, ((bytes / 16 >> bits) + 1) * 16));
  if (piece <= kSmallCta) return launch_t<T, 64>(a, bits, piece, err, timeout_ns, st);
  return launch_t<T, kBigThreads>(a, bits, piece, err, timeout_ns, st);
}

}  // namespace

cudaError_t launch_distill(const DistillLaunch& a, int* err, uint64_t timeout_ns, int num_sms, cudaStream_t st) {
  if (a.dtype == kF32) return launch_rows<float>(a, err, timeout_ns, num_sms, st);
  if (a.dtype == kBF16) return launch_rows<__nv_bfloat16>(a, err, timeout_ns, num_sms, st);
  return launch_rows<__half>(a, err, timeout_ns, num_sms, st);
}

}  // namespace rbf
