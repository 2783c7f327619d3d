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
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "ops_internal.h"
#include "rbf_device.cuh"
#include "rbf_internal.h"
#include "score_rows.cuh"

namespace rbf {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kPiece = 64 * 1024;  // bytes of a row in a CTA's shared memory
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

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

// What a CTA says of its part to all of its cluster: the largest and the sum of
// the scores that are not listed, and of the listed ones (a float each, in a
// word), the sum of p_e ((t_e - largest t) - (s_e - largest of these)), and of p_e.
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

template <typename T>
__global__ void __launch_bounds__(kThreads) distill_kernel(const DistillLaunch a, int piece_bytes, int* err, uint64_t timeout_ns) {
  constexpr int E = Vec<T>::kLen;
  using B = typename Bits<T>::type;
  extern __shared__ __align__(16) uint8_t dyn[];
  T* piece = reinterpret_cast<T*>(dyn);                                   // piece_bytes
  int* at = reinterpret_cast<int*>(dyn + piece_bytes);                    // [k] index, -1: not in this CTA's part
  float* logit = reinterpret_cast<float*>(at + a.k);                      // [k] the teacher's, -infinity: no entry
  float* score = logit + a.k;                                             // [k] the student's
  float* prob = score + a.k;                                              // [k] p_e
  int* owner = reinterpret_cast<int*>(prob + a.k);                        // [k] the first entry with the same index
  __shared__ uint64_t full;
  __shared__ float red[2][kWarps];
  __shared__ u64 said[kMaxCluster][kWords];
  __shared__ double part_d[2];

  uint32_t rank, size;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(size));
  if (size > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t r = blockIdx.x / size;
  const T* row = static_cast<const T*>(a.scores) + r * a.ld_scores;
  const int lead = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
  const int vecs = static_cast<int>((int64_t(a.vocab) + lead + E - 1) / E);
  const int c0 = static_cast<int>(int64_t(vecs) * rank / size), c1 = static_cast<int>(int64_t(vecs) * (rank + 1) / size);
  const int piece_vecs = piece_bytes / 16;
  const int pieces = max(1, (c1 - c0 + piece_vecs - 1) / piece_vecs);
  if (tid == 0) {
    mbar_init(&full, 1);
    fence_mbar_init();
  }
  __syncthreads();

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
    if (!mbar_wait(&full, phase, timeout_ns)) {
      ok = false;
      mbar_wait(&full, phase, timeout_ns);  // no copy may be in flight when the CTA exits
    }
    phase ^= 1u;
    ok = __syncthreads_and(ok) != 0;
    if (!ok && tid == 0) atomicOr(err, kErrConsumerTimeout);
  };
  fetch(c0, min(c1, c0 + piece_vecs));

  // ------------------------------------------------------------ the teacher
  const float rate = kLog2e / a.temperature;
  const float w_row = a.weight ? a.weight[r] : 1.0f;
  float rest_t = a.rest ? a.rest[r] * a.temperature : -INFINITY;  // as a logit
  float top_t = rest_t;
  for (int e = tid; e < a.k; e += kThreads) {
    const int j = a.index[r * a.ld_index + e];
    const float t = j >= 0 && j < a.vocab ? read_float(a.teacher, r * a.ld_teacher + e, a.teacher_dtype) : -INFINITY;
    const int64_t v = j >= 0 && j < a.vocab ? (int64_t(j) + lead) / E : -1;
    at[e] = v >= c0 && v < c1 ? j : -1;
    logit[e] = t;
    top_t = fmaxf(top_t, t);
  }
  auto block_max = [&](float v) {
    v = warp_fold(v, [](float x, float y) { return fmaxf(x, y); });
    __syncthreads();
    if (lane == 0) red[0][warp] = v;
    __syncthreads();
    v = red[0][0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) v = fmaxf(v, red[0][w]);
    return v;
  };
  auto block_sum2 = [&](float& x, float& y) {
    x = warp_fold(x, [](float p, float q) { return p + q; });
    y = warp_fold(y, [](float p, float q) { return p + q; });
    __syncthreads();
    if (lane == 0) {
      red[0][warp] = x;
      red[1][warp] = y;
    }
    __syncthreads();
    x = y = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      x += red[0][w];
      y += red[1][w];
    }
  };
  top_t = block_max(top_t);
  float z_t = 0.0f, dummy = 0.0f;
  for (int e = tid; e < a.k; e += kThreads) {
    const float p = weight_of(logit[e], top_t, rate);
    prob[e] = p;
    z_t += p;
  }
  block_sum2(z_t, dummy);
  const float z_tr = weight_of(rest_t, top_t, rate);
  const float inv_t = z_t + z_tr > 0.0f || z_t != z_t || z_tr != z_tr ? 1.0f / (z_t + z_tr) : 0.0f;
  const float p_in = z_t * inv_t, p_rest = z_tr * inv_t;

  // ------------------------------------------------------------ the student
  float top_rest = -INFINITY, top_in = -INFINITY;
  float z_rest = 0.0f;  // this thread's
  double z_all = 0.0;   // and of the pieces before
  for (int p = 0; p < pieces; ++p) {
    const int v0 = c0 + p * piece_vecs, v1 = min(c1, v0 + piece_vecs);
    if (p > 0) {
      __syncthreads();  // the last piece has been read
      fetch(v0, v1);
    }
    arrived();
    if (!ok) break;
    // The listed scores are read, then the first entry of each index marks its
    // place with its number (the smallest stays, whatever the order of the
    // writes), and in the end the place becomes -infinity.
    const int64_t j0 = int64_t(v0) * E - lead, j1 = int64_t(v1) * E - lead;
    for (int e = tid; e < a.k; e += kThreads) {
      const int j = at[e];
      if (j >= j0 && j < j1) score[e] = Vec<T>::one(piece[j - j0]);
    }
    __syncthreads();
    B* mark = reinterpret_cast<B*>(piece);
    for (int e = tid; e < a.k; e += kThreads)
      if (at[e] >= j0 && at[e] < j1) mark[at[e] - j0] = static_cast<B>(e);
    bool again = true;
    while (again) {
      __syncthreads();
      bool lower = false;
      for (int e = tid; e < a.k; e += kThreads)
        lower |= at[e] >= j0 && at[e] < j1 && static_cast<B>(e) < *reinterpret_cast<volatile B*>(&mark[at[e] - j0]);
      again = __syncthreads_or(lower) != 0;
      if (lower)
        for (int e = tid; e < a.k; e += kThreads)
          if (at[e] >= j0 && at[e] < j1 && static_cast<B>(e) < *reinterpret_cast<volatile B*>(&mark[at[e] - j0]))
            *reinterpret_cast<volatile B*>(&mark[at[e] - j0]) = static_cast<B>(e);
    }
    for (int e = tid; e < a.k; e += kThreads)
      if (at[e] >= j0 && at[e] < j1) owner[e] = static_cast<int>(mark[at[e] - j0]);
    __syncthreads();
    for (int e = tid; e < a.k; e += kThreads)
      if (at[e] >= j0 && at[e] < j1) mark[at[e] - j0] = Bits<T>::kNone;
    __syncthreads();

    const uint4* src = reinterpret_cast<const uint4*>(piece);
    float top = -INFINITY;
    for (int v = tid; v < v1 - v0; v += kThreads) {
      float x[E];
      Vec<T>::unpack(src[v], x);
#pragma unroll
      for (int i = 0; i < E; ++i) top = fmaxf(top, x[i]);
    }
    top = fmaxf(block_max(top), top_rest);
    if (p > 0) z_all *= static_cast<double>(weight_of(top_rest, top, rate));
    top_rest = top;
    z_rest = 0.0f;
    const float base = top == -INFINITY ? 0.0f : top;
    for (int v = tid; v < v1 - v0; v += kThreads) {
      float x[E];
      Vec<T>::unpack(src[v], x);
      const u64 nb = pack2(-base, -base), r2 = pack2(rate, rate);
      u64 add = 0;
#pragma unroll
      for (int i = 0; i < E; i += 2) {
        const u64 z = mul2(add2(pack2(x[i], x[i + 1]), nb), r2);
        add = add2(add, pack2(ex2(low2(z)), ex2(high2(z))));
      }
      z_rest += low2(add) + high2(add);
    }
    if (pieces > 1) {
      z_all += static_cast<double>(z_rest);
      z_rest = 0.0f;
    }
  }
  if (pieces > 1) z_rest = static_cast<float>(z_all);

  // Of this CTA's listed scores: the largest, the sum, and the products.
  for (int e = tid; e < a.k; e += kThreads)
    if (at[e] >= 0) top_in = fmaxf(top_in, score[e]);
  top_in = block_max(top_in);
  float z_in = 0.0f;
  for (int e = tid; e < a.k; e += kThreads)
    if (at[e] >= 0 && owner[e] == e) z_in += weight_of(score[e], top_in, rate);
  block_sum2(z_rest, z_in);
  if (warp == 0) {
    // Each below its own largest: beside scores at the type's lowest value a teacher's logit would vanish.
    double d = 0.0;
    float m = 0.0f;
    for (int e = lane; e < a.k; e += 32) {
      if (at[e] < 0 || !(prob[e] > 0.0f)) continue;
      const float p = prob[e] * inv_t;
      d += score[e] == -INFINITY ? INFINITY : static_cast<double>(p) * static_cast<double>((logit[e] - top_t) - (score[e] - top_in));
      m += p;
    }
    d = warp_fold(d, [](double x, double y) { return x + y; });
    m = warp_fold(m, [](float x, float y) { return x + y; });
    if (lane == 0) {
      part_d[0] = d;
      part_d[1] = static_cast<double>(m);
    }
  }
  if (size > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  __syncthreads();
  if (tid < kWords * static_cast<int>(size)) {
    const int word = tid % kWords;
    const u64 v = word == 0   ? (static_cast<u64>(__float_as_uint(z_rest)) << 32 | __float_as_uint(top_rest))
                  : word == 1 ? (static_cast<u64>(__float_as_uint(z_in)) << 32 | __float_as_uint(top_in))
                              : static_cast<u64>(__double_as_longlong(part_d[word - 2]));
    remote_store(remote(&said[rank][word], static_cast<uint32_t>(tid / kWords)), v);
  }
  if (size > 1)
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  else
    __syncthreads();
  if (!ok) return;

  // Every thread joins what the CTAs have said, in their order.
  float tr = -INFINITY, ti = -INFINITY, zr = 0.0f, zi = 0.0f;
  for (uint32_t c = 0; c < size; ++c) {
    tr = fmaxf(tr, __uint_as_float(static_cast<uint32_t>(said[c][0])));
    ti = fmaxf(ti, __uint_as_float(static_cast<uint32_t>(said[c][1])));
  }
  for (uint32_t c = 0; c < size; ++c) {
    const float cr = __uint_as_float(static_cast<uint32_t>(said[c][0])), ci = __uint_as_float(static_cast<uint32_t>(said[c][1]));
    zr += __uint_as_float(static_cast<uint32_t>(said[c][0] >> 32)) * weight_of(cr, tr, rate);
    zi += __uint_as_float(static_cast<uint32_t>(said[c][1] >> 32)) * weight_of(ci, ti, rate);
  }
  // Both below one score: what is left of the other's weight is a factor.
  const float top_s = fmaxf(tr, ti);
  const float fr = weight_of(tr, top_s, rate), fi = weight_of(ti, top_s, rate);
  const float zr_s = zr * fr, zi_s = zi * fi, z_s = zr_s + zi_s;
  const bool no_teacher = z_t + z_tr == 0.0f, no_student = z_s == 0.0f;
  const bool live = !no_teacher && !no_student && w_row != 0.0f;
  const float inv_s = 1.0f / z_s;
  const float q_in = zi_s * inv_s, q_rest = zr_s * inv_s;

  if (a.loss && rank == 0 && tid == 0) {
    float loss = 0.0f;
    if (live) {
      double d = 0.0;
      // sum p_e (log p_e - log q_e) = sum p_e ((t_e - largest t) - (s_e - largest s)) / T - P log(Z_t / Z_s)
      for (uint32_t c = 0; c < size; ++c) {
        const double m = __longlong_as_double(static_cast<long long>(said[c][3]));
        d += __longlong_as_double(static_cast<long long>(said[c][2]));
        if (m > 0.0) d += m * (static_cast<double>(top_s) - static_cast<double>(__uint_as_float(static_cast<uint32_t>(said[c][1]))));
      }
      double l = d / static_cast<double>(a.temperature);
      if (p_in > 0.0f) l -= static_cast<double>(p_in) * static_cast<double>(logf((z_t + z_tr) * inv_s));
      // p_r / q_r as (1 + listed / others) of both
      if (p_rest > 0.0f) {
        const float others = zr > 0.0f ? zi / zr : INFINITY;
        const float gap = (ti == -INFINITY || zr == 0.0f) ? 0.0f : (ti - tr) * rate;
        const float ratio = ti == -INFINITY ? 0.0f : others * exp2f(gap);
        const float ls = ratio < 3.0e38f ? log1pf(ratio) : (zr > 0.0f ? logf(others) + gap * kLn2 : INFINITY);
        const float ratio_t = z_t / z_tr;
        const float lt = ratio_t < 1.0e30f ? log1pf(ratio_t) : logf(z_t) - logf(z_tr);
        l += static_cast<double>(p_rest) * (static_cast<double>(ls) - static_cast<double>(lt));
      }
      if (p_in != p_in || z_s != z_s) l = static_cast<double>(p_in + z_s);
      loss = static_cast<float>(l * static_cast<double>(a.temperature) * static_cast<double>(a.temperature) * static_cast<double>(w_row));
    }
    a.loss[r] = loss;
  }
  if (!a.grad) return;

  // ----------------------------------------------------------- the gradient
  const float scale = live ? w_row * a.temperature : 0.0f;
  float factor = 0.0f;  // of a score that is not listed: softmax_rest times this
  if (live && zr != 0.0f) factor = scale * (p_rest == 0.0f ? q_rest : p_in < 0.5f ? p_in - q_in : q_rest - p_rest) / zr;
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
    auto grad_of = [&](float x) { return live ? ex2(__fmul_rn(__fsub_rn(x, base), rate)) * factor : 0.0f; };
    if (same) {
      for (int v = tid; v < v1 - v0; v += kThreads) {
        float x[E];
        Vec<T>::unpack(src[v], x);
        float g[E];
#pragma unroll
        for (int i = 0; i < E; ++i) g[i] = grad_of(x[i]);
        const int64_t j = j0 + int64_t(v) * E;
        if (j >= 0 && j + E <= a.vocab) {
          __stcs(reinterpret_cast<uint4*>(out + j), pack_vec<T>(g));
        } else {
#pragma unroll
          for (int i = 0; i < E; ++i)
            if (j + i >= 0 && j + i < a.vocab) out[j + i] = from_float<T>(g[i]);
        }
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
    const float q = weight_of(score[e], top_s, rate) * inv_s;
    out[at[e]] = from_float<T>(scale * (q - p * inv_t));
  }
}

template <typename T>
cudaError_t launch_t(const DistillLaunch& a, int* err, uint64_t timeout_ns, int num_sms, cudaStream_t st) {
  auto fn = distill_kernel<T>;
  constexpr int kMost = kPiece + 5 * 4 * kMaxTeacher;
  static PerDeviceOnce once;
  const cudaError_t ready = once.run([fn] {
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    return e != cudaSuccess ? e : cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  });
  if (ready != cudaSuccess) return ready;
  const int64_t bytes = (int64_t(a.vocab) * static_cast<int64_t>(sizeof(T)) / 16 + 2) * 16;
  int cluster = 1;
  while (cluster < kMaxCluster && bytes / cluster + 16 > kPiece) cluster *= 2;
  while (cluster < kMaxCluster && a.rows * cluster < 2 * num_sms && bytes / cluster > 8192) cluster *= 2;
  const int64_t piece = std::min<int64_t>(kPiece, (bytes / 16 / cluster + 1) * 16);
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
    cfg.dynamicSmemBytes = static_cast<size_t>(piece) + 5 * 4 * static_cast<size_t>(a.k);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, p, static_cast<int>(piece), err, timeout_ns);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_distill(const DistillLaunch& a, int* err, uint64_t timeout_ns, int num_sms, cudaStream_t st) {
  if (a.dtype == kF32) return launch_t<float>(a, err, timeout_ns, num_sms, st);
  if (a.dtype == kBF16) return launch_t<__nv_bfloat16>(a, err, timeout_ns, num_sms, st);
  return launch_t<__half>(a, err, timeout_ns, num_sms, st);
}

}  // namespace rbf
