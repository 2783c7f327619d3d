// verify.cu -- drafted tokens checked against the target's scores
// (include/rbf_ops.h, verify_dev).
//
// With p_i and q_i the softmax of the target's and the draft's scores at place i
// (temperature T), drafted token x_i is accepted while u_i q_i(x_i) < p_i(x_i);
// the answer after the accepted ones is drawn from max(0, p_i - q_i) at the
// first place that is not, from p behind the last one.
//
// 1. verify_stats_kernel reads every row of a sequence's places once: the largest
//    score and the sum of 2^((x - max) log2(e) / T), in fp32, of a part of the row
//    a CTA. (Not above 0, T asks for the best index: then the first one at the
//    largest score, of the target's rows alone.)
// 2. verify_draw_kernel, a cluster of CTAs a sequence: every CTA joins the parts
//    and finds the number of accepted tokens from 2 count + 1 sums; the cluster
//    then draws from the one row (with no accepted count known ahead, every
//    place's sums are needed; which row is drawn from is only known here).
//
// The draw lies between running sums of up to 2^26 numbers, so its sums are of
// 64-bit integers, exact and in any order, and each number in them is right to
// 2^-30 of itself: weights in fp32 would put some draws in a thousand on another
// index than 64 bits do, where the tail is long. 2^z with z = (x - max) log2(e) / T
// - log2 Z as the sum of two fp32 numbers, split into whole 32nds (a table of 31-bit
// integers) and a rest of at most 2^-5 (a polynomial, as a 32-bit fraction).
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
constexpr int kMaxSplits = 64;
constexpr int kMaxHeld = 192 * 1024;  // of two rows in one CTA's shared memory
constexpr float kLog2e = 1.4426950408889634f;

// log2(e) / T as a finite number above 0 (sample_dev's); 0 where the best index is asked for.
__device__ __forceinline__ float rate_of(const VerifyLaunch& a, int64_t seq) {
  const float t = a.temperature ? a.temperature[seq] : 1.0f;
  return t > 0.0f ? fminf(fmaxf(__fdiv_rn(kLog2e, t), 1.4e-45f), 3.40282347e38f) : 0.0f;
}

__device__ __forceinline__ int count_of(const VerifyLaunch& a, int64_t seq) {
  return a.count ? min(max(a.count[seq], 0), a.drafts) : a.drafts;
}

template <typename T>
__device__ __forceinline__ const T* target_row(const VerifyLaunch& a, int64_t seq, int place) {
  return static_cast<const T*>(a.target) + seq * a.ld_target_seq + place * a.ld_target;
}
template <typename T>
__device__ __forceinline__ const T* draft_row(const VerifyLaunch& a, int64_t seq, int place) {
  return static_cast<const T*>(a.draft) + seq * a.ld_draft_seq + place * a.ld_draft;
}

// A largest score of +infinity leaves only the scores that equal it.
__device__ __forceinline__ float less_top(float x, float top) {
  return top == INFINITY ? (x == INFINITY ? 0.0f : -INFINITY) : __fsub_rn(x, top);
}

// ------------------------------------------------------------------- sums

// Parts of a row in fp32: the largest score and the sum of weights below it.
struct Sum {
  float top = -INFINITY, z = 0.0f;
  __device__ __forceinline__ void join(float t, float s, float rate) {
    const float best = fmaxf(top, t);
    if (best == -INFINITY) return;
    z = z * ex2(less_top(top, best) * rate) + s * ex2(less_top(t, best) * rate);
    top = best;
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) verify_stats_kernel(const VerifyLaunch a, VerifyPart* parts, int splits) {
  constexpr int E = Vec<T>::kLen;
  __shared__ VerifyPart part[kWarps];
  pdl_launch_dependents();
  const int places = a.drafts + 1;
  const int rows = places + (a.draft ? a.drafts : 0);  // of a sequence: the target's, then the draft's
  const int64_t row_id = blockIdx.x / splits;
  const int split = static_cast<int>(blockIdx.x % splits);
  const int64_t seq = row_id / rows;
  const int in = static_cast<int>(row_id % rows);
  const float rate = rate_of(a, seq);
  const int count = count_of(a, seq);
  const bool of_target = in < places;
  if (of_target ? in > count : (in - places >= count || rate == 0.0f)) return;
  const Row<T> row(of_target ? target_row<T>(a, seq, in) : draft_row<T>(a, seq, in - places), a.vocab);
  const int v0 = static_cast<int>(int64_t(row.vecs) * split / splits), v1 = static_cast<int>(int64_t(row.vecs) * (split + 1) / splits);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  Sum s;
  u64 first = 0;  // the key of the best index
  for (int v = v0 + static_cast<int>(threadIdx.x); v < v1; v += 4 * kThreads) {
    uint4 raw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) raw[i] = v + i * kThreads < v1 ? row.load(v + i * kThreads) : vec_none<T>();
    float x[4][E];
    uint4 best = vec_max<T>(vec_max<T>(raw[0], raw[1]), vec_max<T>(raw[2], raw[3]));
    Vec<T>::unpack(best, x[0]);
    float top = x[0][0];
#pragma unroll
    for (int i = 1; i < E; ++i) top = fmaxf(top, x[0][i]);
    if (rate == 0.0f) {
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        Vec<T>::unpack(raw[i], x[0]);
        for (int e = 0; e < E; ++e)
          if (x[0][e] > -INFINITY) first = umax64(first, make_key(x[0][e], static_cast<uint32_t>((v + i * kThreads) * E - row.lead + e)));
      }
      continue;
    }
    if (top == -INFINITY) continue;
    if (top > s.top) {
      s.z = s.top == -INFINITY ? 0.0f : s.z * ex2(less_top(s.top, top) * rate);
      s.top = top;
    }
    if (s.top == INFINITY) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        Vec<T>::unpack(raw[i], x[0]);
#pragma unroll
        for (int e = 0; e < E; ++e) s.z += x[0][e] == INFINITY ? 1.0f : 0.0f;
      }
      continue;
    }
    const u64 ntop2 = pack2(-s.top, -s.top), rate2 = pack2(rate, rate);
    float sum[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      Vec<T>::unpack(raw[i], x[i]);
      u64 add = 0;  // two zeros
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const u64 z = mul2(add2(pack2(x[i][e], x[i][e + 1]), ntop2), rate2);
        add = add2(add, pack2(ex2(low2(z)), ex2(high2(z))));
      }
      sum[i] = low2(add) + high2(add);
    }
    s.z += (sum[0] + sum[1]) + (sum[2] + sum[3]);
  }
  if (rate == 0.0f) {
    first = warp_max(first);
    if (lane == 0) part[warp].key = first;
  } else {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s.join(__shfl_xor_sync(kFullMask, s.top, d), __shfl_xor_sync(kFullMask, s.z, d), rate);
    if (lane == 0) part[warp] = VerifyPart{s.top, s.z, 0};
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    VerifyPart r = part[0];
    if (rate == 0.0f) {
      for (int w = 1; w < kWarps; ++w) r.key = umax64(r.key, part[w].key);
    } else {
      for (int w = 1; w < kWarps; ++w) s.join(part[w].top, part[w].z, rate);
      r = VerifyPart{s.top, s.z, 0};
    }
    parts[row_id * splits + split] = r;
  }
}

// -------------------------------------------------------------- exact draw

// 2^(i / 32) in units of 2^-30.
__constant__ uint32_t kRoots[32] = {
    1073741824u, 1097253708u, 1121280436u, 1145833280u, 1170923762u, 1196563654u, 1222764986u, 1249540052u,
    1276901417u, 1304861917u, 1333434672u, 1362633090u, 1392470869u, 1422962010u, 1454120821u, 1485961921u,
    1518500250u, 1551751076u, 1585730000u, 1620452965u, 1655936265u, 1692196547u, 1729250827u, 1767116489u,
    1805811301u, 1845353420u, 1885761398u, 1927054196u, 1969251188u, 2012372174u, 2056437387u, 2101467502u};

// 2^((x - top) rate - shift) for the scores of a row, in units of 2^-(62 - spare):
// `shift` is held as whole 32nds and a rest.
struct Weights {
  float top, rate_hi, rate_lo, rest;
  int whole, spare;
  const uint32_t* roots;  // in shared memory

  __device__ __forceinline__ void set(float t, double rate, double shift, int spare_bits, const uint32_t* table) {
    top = t;
    rate_hi = static_cast<float>(rate);
    rate_lo = rate_hi > 3.0e38f ? 0.0f : static_cast<float>(rate - rate_hi);
    const double n = rint(shift * 32.0);
    whole = static_cast<int>(n);
    rest = static_cast<float>(shift - n * (1.0 / 32.0));
    spare = spare_bits;
    roots = table;
  }
  __device__ __forceinline__ u64 of(float x) const {
    if (top == INFINITY) return x == INFINITY ? at(0.0f, 0.0f) : 0;
    // x - top as the sum of two numbers, and their product with the rate.
    const float d = __fsub_rn(x, top);
    const float back = __fsub_rn(d, x);  // -top, as far as d has it
    const float lost = __fsub_rn(__fsub_rn(x, __fsub_rn(d, back)), __fadd_rn(top, back));
    const float hi = __fmul_rn(d, rate_hi);
    if (!(hi > -64.0f)) return 0;
    const float lo = __fmaf_rn(lost, rate_hi, __fmaf_rn(d, rate_lo, __fmaf_rn(d, rate_hi, -hi)));
    return at(hi, lo);
  }

 private:
  __device__ __forceinline__ u64 at(float hi, float lo) const {
    const float n = rintf(hi * 32.0f);
    const float f = __fadd_rn(__fmaf_rn(n, -1.0f / 32.0f, hi), __fsub_rn(lo, rest));
    const int e = static_cast<int>(n) - whole;
    // 2^f - 1, |f| < 2^-4: the series of exp(f ln 2).
    float g = __fmaf_rn(f, 1.3333558e-3f, 9.6181291e-3f);
    g = __fmaf_rn(f, g, 5.5504109e-2f);
    g = __fmaf_rn(f, g, 2.4022651e-1f);
    g = __fmaf_rn(f, g, 6.9314718e-1f);
    const int frac = __float2int_rn(__fmul_rn(f, g) * 4294967296.0f);
    const u64 root = roots[e & 31];
    const u64 w = (root << 32) + static_cast<u64>(static_cast<long long>(root) * frac);
    const int down = spare - (e >> 5);
    return down < 64 ? (down > 0 ? w >> down : w) : 0;
  }
};

// Scores i0 .. i0 + kLen - 1 of a row of n that starts anywhere, -infinity where
// there are none: from the two aligned vectors that hold them.
template <typename T>
__device__ __forceinline__ uint4 load_shifted(const T* row, int i0, int n) {
  constexpr int E = Vec<T>::kLen;
  if (i0 < E || i0 + 2 * E > n) return load_edge(row, i0, n);
  const uintptr_t at = reinterpret_cast<uintptr_t>(row + i0);
  const uint4* src = reinterpret_cast<const uint4*>(at & ~uintptr_t(15));
  const uint4 a = src[0];
  if ((at & 15) == 0) return a;
  const uint4 b = src[1];
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (at & 8) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (at & 4) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  const int bits = static_cast<int>(at & 3) * 8;
  return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits), __funnelshift_r(w[2], w[3], bits),
                    __funnelshift_r(w[3], w[4], bits));
}

struct Place {  // what one place's parts say
  float top, z;
};

template <typename T, bool HELD>
__global__ void __launch_bounds__(kThreads) verify_draw_kernel(const VerifyLaunch a, const VerifyPart* parts, int splits, int held_vecs) {
  constexpr int E = Vec<T>::kLen;
  extern __shared__ __align__(16) uint8_t dyn[];
  uint4* held = reinterpret_cast<uint4*>(dyn);  // the target's part, then the draft's
  __shared__ uint32_t roots[32];
  __shared__ u64 slot[4][kMaxCluster];  // a word per CTA, written by all of them
  __shared__ u64 kept[kWarps];
  __shared__ int first_no;
  __shared__ Place row_p, row_q;

  uint32_t rank, size;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(size));
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t seq = blockIdx.x / size;
  const int places = a.drafts + 1, rows = places + (a.draft ? a.drafts : 0);
  // A CTA's shared memory may be written by others once it has started: all
  // arrive here and wait ahead of the first remote store.
  if (size > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const float rate = rate_of(a, seq);
  const int count = count_of(a, seq);
  if (threadIdx.x < 32) roots[threadIdx.x] = kRoots[threadIdx.x];
  if (threadIdx.x == 0) first_no = count;
  __syncthreads();
  pdl_wait();

  // The sums of a row, from its parts (every lane of a warp).
  auto join = [&](int row) {
    Sum s;
    const VerifyPart* from = parts + (seq * rows + row) * splits;
    for (int i = lane; i < splits; i += 32) s.join(__ldcg(&from[i].top), __ldcg(&from[i].z), rate);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s.join(__shfl_xor_sync(kFullMask, s.top, d), __shfl_xor_sync(kFullMask, s.z, d), rate);
    return Place{__shfl_sync(kFullMask, s.top, 0), __shfl_sync(kFullMask, s.z, 0)};
  };
  auto best_of = [&](int row) {  // its index, -1 where nothing is left
    u64 k = 0;
    const VerifyPart* from = parts + (seq * rows + row) * splits;
    for (int i = lane; i < splits; i += 32) k = umax64(k, __ldcg(&from[i].key));
    k = warp_max(k);
    return k ? static_cast<int>(key_index(k)) : -1;
  };
  // A token's score; a NaN counts as -infinity.
  auto score = [&](const T* row, int x) {
    const float v = Vec<T>::one(row[x]);
    return v == v ? v : -INFINITY;
  };
  auto log_p = [&](float x, const Place& p) { return __fsub_rn(less_top(x, p.top) * (rate * 0.69314718f), logf(p.z)); };

  int32_t* token = a.token + seq * places;
  float* logprob = a.logprob ? a.logprob + seq * places : nullptr;
  for (int i = warp; i < count; i += kWarps) {
    const int x = a.draft_token[seq * a.drafts + i];
    bool ok = x >= 0 && x < a.vocab;
    float lp = 0.0f;
    if (rate == 0.0f) {
      const int best = best_of(i);
      ok = ok && best == x;
    } else if (ok) {
      const Place p = join(i);
      const float xp = score(target_row<T>(a, seq, i), x);
      ok = xp > -INFINITY;
      lp = log_p(xp, p);
      if (ok) {
        // u q / p < 1, with the exponents' difference in 64 bits.
        double diff = -static_cast<double>(less_top(xp, p.top));
        float ratio = p.z;
        if (a.draft) {
          const Place q = join(places + i);
          const float xq = score(draft_row<T>(a, seq, i), x);
          diff += xq > -INFINITY ? static_cast<double>(less_top(xq, q.top)) : -INFINITY;
          ratio = xq > -INFINITY ? __fdiv_rn(p.z, q.z) : 0.0f;
        }
        const double e = diff * static_cast<double>(rate), n = rint(e);
        const float m = exp2f(static_cast<float>(e - n));
        ok = ratio == 0.0f ? a.u[seq * places + i] == a.u[seq * places + i]
                           : a.u[seq * places + i] * (ratio * m) * exp2f(static_cast<float>(fmin(fmax(n, -1000.0), 1000.0))) < 1.0f;
      }
    }
    if (lane == 0) {
      if (!ok) atomicMin(&first_no, i);
      if (rank == 0) {
        token[i] = x;
        if (logprob) logprob[i] = lp;
      }
    }
  }
  __syncthreads();
  const int accepted = first_no;
  const bool late = accepted < count;  // a token was refused
  if (rank == 0) {
    if (threadIdx.x == 0) a.accepted[seq] = accepted;
    for (int i = accepted + static_cast<int>(threadIdx.x); i < places; i += kThreads) {
      token[i] = -1;
      if (logprob) logprob[i] = -INFINITY;
    }
  }
  if (rate == 0.0f) {
    if (warp == 0) {
      const int best = best_of(accepted);
      if (rank == 0 && lane == 0 && best >= 0) {
        token[accepted] = best;
        if (logprob) logprob[accepted] = 0.0f;
      }
    }
    if (size > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    return;
  }
  if (warp == 0) {
    const Place p = join(accepted);
    if (lane == 0) row_p = p;
  } else if (warp == 1 && late && a.draft) {
    const Place q = join(places + accepted);
    if (lane == 0) row_q = q;
  }
  __syncthreads();
  if (size > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  const Place pp = row_p;
  if (pp.top == -INFINITY) return;  // nothing is left of the row: -1 stays
  const bool with_q = late && a.draft && row_q.top > -INFINITY;
  // Without draft scores the refused token is taken out of p.
  const int out = late && !a.draft ? a.draft_token[seq * a.drafts + accepted] : -1;

  const Row<T> rp(target_row<T>(a, seq, accepted), a.vocab);
  // The draft's row may lie otherwise on its 16-byte boundaries: it is taken by
  // the target's vectors.
  const T* dq = with_q ? draft_row<T>(a, seq, accepted) : nullptr;
  auto load_q = [&](int v) { return vec_max<T>(load_shifted(dq, v * E - rp.lead, a.vocab), vec_none<T>()); };
  const int c0 = static_cast<int>(int64_t(rp.vecs) * rank / size), c1 = static_cast<int>(int64_t(rp.vecs) * (rank + 1) / size);
  auto part_of = [](int lo, int hi, int w) { return lo + static_cast<int>(int64_t(hi - lo) * w / kWarps); };
  const int v0 = part_of(c0, c1, warp), v1 = part_of(c0, c1, warp + 1);
  auto get_p = [&](int v) -> uint4 { return HELD ? held[v - c0] : rp.load(v); };
  auto get_q = [&](int v) -> uint4 { return HELD ? held[held_vecs + v - c0] : load_q(v); };
  if (HELD) {
    for (int v = v0 + lane; v < v1; v += 32) {
      held[v - c0] = rp.load(v);
      if (with_q) held[held_vecs + v - c0] = load_q(v);
    }
    __syncwarp();
  }

  int turn = 0;
  // Sum over the cluster of every thread's v; slot[turn - 1] keeps the CTAs' own.
  auto total_of = [&](u64 v) {
    v = warp_sum(v);
    if (lane == 0) kept[warp] = v;
    __syncthreads();
    u64 r = lane < kWarps ? kept[lane] : 0ull;
    r = warp_sum(r);
    if (threadIdx.x < size) remote_store(remote(&slot[turn][rank], threadIdx.x), r);
    if (size > 1)
      asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    else
      __syncthreads();
    r = lane < static_cast<int>(size) ? slot[turn][lane] : 0ull;
    ++turn;
    return warp_sum(r);
  };

  // The two rows' sums, exactly; `spare` bits keep them within 62.
  const double rate64 = a.temperature ? fmin(fmax(1.4426950408889634 / static_cast<double>(a.temperature[seq]), 1.4e-45), 3.4e38)
                                      : 1.4426950408889634;
  const int spare = 33 - __clz(max(a.vocab, 1));
  Weights wp, wq;
  auto sum_of = [&](Weights& w, float top, auto&& get) {
    w.set(top, rate64, 0.0, spare, roots);
    u64 sum = 0;
#pragma unroll 1
    for (int v = v0 + lane; v < v1; v += 32) {
      float x[E];
      Vec<T>::unpack(get(v), x);
#pragma unroll
      for (int e = 0; e < E; ++e) sum += w.of(x[e]);
    }
    const u64 all = total_of(sum);
    w.set(top, rate64, log2(static_cast<double>(all)) + spare - 62, 0, roots);
  };
  sum_of(wp, pp.top, get_p);
  if (with_q) sum_of(wq, row_q.top, get_q);

  // What a vector's scores leave, from place 2^-62 of the whole on.
  bool left = with_q || out >= 0;
  auto weigh = [&](int v, u64 (&w)[E]) {
    float x[E];
    Vec<T>::unpack(get_p(v), x);
#pragma unroll
    for (int e = 0; e < E; ++e) w[e] = wp.of(x[e]);
    if (left && with_q) {
      Vec<T>::unpack(get_q(v), x);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const u64 q = wq.of(x[e]);
        w[e] = w[e] > q ? w[e] - q : 0;
      }
    } else if (left) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (v * E - rp.lead + e == out) w[e] = 0;
    }
  };
  auto sum_left = [&]() {
    u64 sum = 0;
#pragma unroll 1
    for (int v = v0 + lane; v < v1; v += 32) {
      u64 w[E];
      weigh(v, w);
#pragma unroll
      for (int e = 0; e < E; ++e) sum += w[e];
    }
    return total_of(sum);
  };
  u64 total = sum_left();
  if (left && total == 0) {  // p and q agree (or p is all on the refused token): what is left is rounding
    left = false;
    total = sum_left();
  }
  const float u = a.u[seq * places + a.drafts];
  const u64 part_u = min(static_cast<u64>(u > 0.0f ? fminf(floorf(u * 0x1p30f), 0x1p30f) : 0.0f), (u64(1) << 30) - 1);
  const u64 aim = share(total, part_u);
  u64 before = 0;
  for (uint32_t c = 0; c < rank; ++c) before += slot[turn - 1][c];
  // This CTA's warps, in order.
  for (int w = 0; w < warp; ++w) before += kept[w];
  if (aim < before || aim >= before + kept[warp]) return;
  for (int v = v0; v < v1; v += 32) {
    u64 w[E], sum = 0;
    if (v + lane < v1) {
      weigh(v + lane, w);
#pragma unroll
      for (int e = 0; e < E; ++e) sum += w[e];
    }
    const u64 upto = before + warp_scan(sum, lane);
    u64 run = upto - sum;
    if (sum > 0 && run <= aim && aim < upto) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (w[e] > 0 && run <= aim && aim < run + w[e]) {
          const int x = (v + lane) * E - rp.lead + e;
          token[accepted] = x;
          if (logprob) logprob[accepted] = log_p(score(rp.p, x), pp);
        }
        run += w[e];
      }
    }
    before = __shfl_sync(kFullMask, upto, 31);
    if (aim < before) break;
  }
}

template <typename T, bool HELD>
cudaError_t launch_draw_t(const VerifyLaunch& a, const VerifyPart* parts, int splits, int cluster, int held_vecs, cudaStream_t st) {
  auto fn = verify_draw_kernel<T, HELD>;
  static PerDeviceOnce once;
  const cudaError_t ready = once.run([fn] {
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxHeld);
    return e != cudaSuccess ? e : cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  });
  if (ready != cudaSuccess) return ready;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.seqs * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = HELD ? static_cast<size_t>(held_vecs) * 32 : 0;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, fn, a, parts, splits, held_vecs);
}

// CTAs a row: parts of some 32 KB, fewer bytes where that leaves SMs idle, as
// many as the workspace has room for.
int splits_of(const VerifyLaunch& a, int64_t max_parts, int num_sms) {
  const int64_t rows = a.seqs * (a.drafts + 1 + (a.draft ? a.drafts : 0));
  const int64_t bytes = a.vocab * static_cast<int64_t>(dtype_bytes(a.dtype));
  const int64_t fill = std::min((int64_t(num_sms) * 8 + rows - 1) / rows, bytes / 4096);
  const int64_t s = std::min<int64_t>(std::max((bytes + 32767) / 32768, fill), std::min<int64_t>(kMaxSplits, max_parts / rows));
  return static_cast<int>(std::max<int64_t>(1, s));
}

template <typename T>
cudaError_t launch_stats(const VerifyLaunch& a, VerifyPart* parts, int splits, cudaStream_t st) {
  const int64_t rows = a.seqs * (a.drafts + 1 + (a.draft ? a.drafts : 0));
  verify_stats_kernel<T><<<static_cast<unsigned>(rows * splits), kThreads, 0, st>>>(a, parts, splits);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_draw(const VerifyLaunch& a, const VerifyPart* parts, int splits, cudaStream_t st) {
  const int64_t vecs = a.vocab * static_cast<int64_t>(sizeof(T)) / 16 + 2;
  int cluster = 1;
  while (cluster < kMaxCluster && vecs / cluster > 512) cluster *= 2;
  const int64_t held = vecs / cluster + 2;
  return held * 32 <= kMaxHeld ? launch_draw_t<T, true>(a, parts, splits, cluster, static_cast<int>(held), st)
                               : launch_draw_t<T, false>(a, parts, splits, cluster, 0, st);
}

}  // namespace

int64_t verify_max_parts(int64_t max_rows, int num_sms) { return 4 * max_rows + 128 * int64_t(num_sms); }

cudaError_t launch_verify_stats(const VerifyLaunch& a, VerifyPart* parts, int64_t max_parts, int num_sms, cudaStream_t st) {
  const int splits = splits_of(a, max_parts, num_sms);
  if (a.dtype == kF32) return launch_stats<float>(a, parts, splits, st);
  if (a.dtype == kBF16) return launch_stats<__nv_bfloat16>(a, parts, splits, st);
  return launch_stats<__half>(a, parts, splits, st);
}

cudaError_t launch_verify_draw(const VerifyLaunch& a, const VerifyPart* parts, int64_t max_parts, int num_sms, cudaStream_t st) {
  const int splits = splits_of(a, max_parts, num_sms);
  if (a.dtype == kF32) return launch_draw<float>(a, parts, splits, st);
  if (a.dtype == kBF16) return launch_draw<__nv_bfloat16>(a, parts, splits, st);
  return launch_draw<__half>(a, parts, splits, st);
}

}  // namespace rbf
