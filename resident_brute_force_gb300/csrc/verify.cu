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
// 2. verify_draw_kernel, a cluster of CTAs a sequence: a warp a place joins its parts
//    and decides on its token, the first refusal of all is the answer's length, and the
//    cluster draws from that one row (every place's sums are needed ahead of it; which
//    row is drawn from is only known here).
//
// The draw lies between running sums of up to 2^26 numbers, so its sums are of 64-bit
// integers, exact and in any order, and each number in them is right to 2^-29 of itself
// and 2^-60 of the whole (what falls off their last place): weights in fp32 would put some
// draws in a thousand on another index than 64 bits do, where the tail is long. 2^z is
// taken by z's whole 32nds (a table of 31-bit integers) and a rest of at most 2^-6 (a
// polynomial, as a 32-bit fraction).
//
// What bounds it: of 64 sequences of 7 tokens over 128000 bf16 scores the rows' sums take
// 44 us (246 MB, 36 at the copy rate), the draws 46: some 5 for the accepted tokens,
// about 18 for either pass over the drawn rows (18 instructions a weight, 4 weights an index,
// and as much again around them), 3 for the index itself. Tried without gain: the rows
// kept in shared memory between the passes, or copied there ahead (cp.async), vectors
// fetched two rounds ahead, four scores at a time, the roots by shuffles.
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
constexpr int kGroupVecs = 4 * kThreads;  // vectors that a CTA of the rows' sums takes at a time
constexpr int kStatsCtas = 6;  // an SM, in the rows' sums: 40 registers a thread
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eLow = 1.4426950408889634 - static_cast<double>(kLog2e);  // what fp32 leaves out
// Of the draw, an SM: 512 threads, so that one has 128 registers for weights side by
// side. 64 x 7 x 128000 and 61 x 5 x 100003 in all: 90 and 65 us, with 640 threads 102 and 70, with 1024
// 107 and 69 (as CTAs of 256 99 and 72), with 256 104 and 75; CTAs of 256 and 512 threads 92 and 68, 89 and 67.
constexpr int kDrawThreads = 512;
constexpr int kDrawCta = 128;
constexpr float kLeastOctave = -1074.0f;  // a weight below 2^this is 0
constexpr unsigned long long kRounding = 1ull << 34;  // of shares of 2^62: 2^-28

// A sequence's temperature. From 2^100 on scores and T are taken 2^-64 times as large,
// exactly: there scores whose difference passes fp32's range have weight, and log2(e) / T
// falls out of the range in which it has all its bits. Below, such a difference is
// one of 2^28 octaves at least, and its weight 0.
struct Heat {
  float rate;   // log2(e) / T as a finite number above 0 (sample_dev's); 0 where the best index is asked for
  float t;      // T as the scores are taken
  float scale;  // of the scores, 1 or 2^-64
};
__device__ __forceinline__ Heat heat_of(const VerifyLaunch& a, int64_t seq) {
  Heat h;
  h.t = a.temperature ? a.temperature[seq] : 1.0f;
  h.scale = h.t >= 0x1p100f ? 0x1p-64f : 1.0f;
  h.t *= h.scale;
  h.rate = h.t > 0.0f ? fminf(fmaxf(__fdiv_rn(kLog2e, h.t), 1.4e-45f), 3.40282347e38f) : 0.0f;
  return h;
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

// What fp32 leaves out of x - top = d.
__device__ __forceinline__ float less_rest(float x, float top, float d) {
  if (top == INFINITY || !(d > -INFINITY)) return 0.0f;
  const float back = __fsub_rn(d, x);
  return __fsub_rn(__fsub_rn(x, __fsub_rn(d, back)), __fadd_rn(top, back));
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
__global__ void __launch_bounds__(kThreads, kStatsCtas) verify_stats_kernel(const VerifyLaunch a, VerifyPart* parts, int part_vecs) {
  constexpr int E = Vec<T>::kLen;
  __shared__ VerifyPart part[kWarps];
  pdl_launch_dependents();
  const int places = a.drafts + 1;
  const int rows = places + (a.draft ? a.drafts : 0);  // of a sequence: the target's, then the draft's
  // A sequence, its row, and the row's part.
  const int64_t seq = blockIdx.x;
  const int in = static_cast<int>(blockIdx.y), split = static_cast<int>(blockIdx.z), splits = static_cast<int>(gridDim.z);
  const int64_t row_id = seq * rows + in;
  const Heat heat = heat_of(a, seq);
  const float rate = heat.rate, scale = heat.scale;
  const int count = count_of(a, seq);
  const bool of_target = in < places;
  if (of_target ? in > count : (in - places >= count || rate == 0.0f)) return;
  const Row<T> row(of_target ? target_row<T>(a, seq, in) : draft_row<T>(a, seq, in - places), a.vocab);
  const int v0 = min(row.vecs, split * part_vecs), v1 = min(row.vecs, v0 + part_vecs);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  if (rate == 0.0f) {  // the key of the best index
    u64 first = 0;
    for (int v = v0 + static_cast<int>(threadIdx.x); v < v1; v += kThreads) {
      float x[E];
      Vec<T>::unpack(row.load(v), x);
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (x[e] > -INFINITY) first = umax64(first, make_key(x[e], static_cast<uint32_t>(v * E - row.lead + e)));
    }
    first = warp_max(first);
    if (lane == 0) part[warp].key = first;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kWarps; ++w) first = umax64(first, part[w].key);
      parts[row_id * splits + split] = VerifyPart{0.0f, 0.0f, first};
    }
    return;
  }

  Sum s;
  auto add = [&](auto n, uint4 (&raw)[4]) {  // the first n vectors
    constexpr int N = decltype(n)::value;
    float x[E];
    uint4 best = raw[0];
#pragma unroll
    for (int i = 1; i < N; ++i) best = vec_max<T>(best, raw[i]);
    const float top = vec_top<T>(best);
    if (top == -INFINITY) return;
    if (top > s.top) {
      s.z = s.top == -INFINITY ? 0.0f : s.z * ex2(less_top(s.top * scale, top * scale) * rate);
      s.top = top;
    }
    if (s.top == INFINITY || scale != 1.0f) {  // of the former only the scores that equal it count
#pragma unroll 1
      for (int i = 0; i < N; ++i) {
        Vec<T>::unpack(raw[0], x);
#pragma unroll
        for (int e = 0; e < E; ++e) s.z += ex2(less_top(x[e] * scale, s.top * scale) * rate);
#pragma unroll
        for (int o = 0; o < 3; ++o) raw[o] = raw[o + 1];
      }
      return;
    }
    const u64 ntop2 = pack2(-s.top, -s.top), rate2 = pack2(rate, rate);
    u64 sum[2] = {0, 0};  // two zeros each
#pragma unroll
    for (int i = 0; i < N; ++i) {
      Vec<T>::unpack(raw[i], x);
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const u64 z = mul2(add2(pack2(x[e], x[e + 1]), ntop2), rate2);
        sum[e / 2 % 2] = add2(sum[e / 2 % 2], pack2(ex2(low2(z)), ex2(high2(z))));
      }
    }
    sum[0] = add2(sum[0], sum[1]);
    s.z += low2(sum[0]) + high2(sum[0]);
  };
  {
    const int f0 = max(v0, row.lead > 0 ? 1 : 0), f1 = min(v1, (row.n + row.lead) / E);
    const uint4* src = reinterpret_cast<const uint4*>(row.p - row.lead);
    uint4 raw[4];
    int v = f0 + static_cast<int>(threadIdx.x);
#pragma unroll 1
    for (; v < f1; v += kGroupVecs) {
#pragma unroll
      for (int i = 0; i < 4; ++i) raw[i] = v + i * kThreads < f1 ? src[v + i * kThreads] : vec_none<T>();
#pragma unroll
      for (int i = 0; i < 4; ++i) raw[i] = vec_max<T>(raw[i], vec_none<T>());
      add(std::integral_constant<int, 4>{}, raw);
    }
    if (threadIdx.x < 2 && v0 < v1) {  // the one or two vectors that reach past the row
      const int e = threadIdx.x == 0 ? v0 : v1 - 1;
      if ((e < f0 || e >= f1) && !(threadIdx.x == 1 && e == v0)) {
        raw[0] = row.load(e);
        add(std::integral_constant<int, 1>{}, raw);
      }
    }
  }
  s.top *= scale;
  // Each below the largest of the warp, and then of the CTA.
  auto below = [&](Sum& v, int lanes) {
    float top = v.top;
    for (int d = lanes / 2; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, d));
    v.z = v.top == -INFINITY ? 0.0f : v.z * ex2(less_top(v.top, top) * rate);
    v.top = top;
    for (int d = lanes / 2; d > 0; d >>= 1) v.z += __shfl_xor_sync(kFullMask, v.z, d);
  };
  below(s, 32);
  if (lane == 0) part[warp] = VerifyPart{s.top, s.z, 0};
  __syncthreads();
  if (warp == 0) {
    s.top = part[lane % kWarps].top;
    s.z = part[lane % kWarps].z;
    below(s, kWarps);
    if (lane == 0) parts[row_id * splits + split] = VerifyPart{s.top, s.z, 0};
  }
}

// -------------------------------------------------------------- exact draw

struct Place {  // what one place's parts say
  float top, z;
};

// 2^(i / 32) in units of 2^-30.
__constant__ uint32_t kRoots[32] = {
    1073741824u, 1097253708u, 1121280436u, 1145833280u, 1170923762u, 1196563654u, 1222764986u, 1249540052u,
    1276901417u, 1304861917u, 1333434672u, 1362633090u, 1392470869u, 1422962010u, 1454120821u, 1485961921u,
    1518500250u, 1551751076u, 1585730000u, 1620452965u, 1655936265u, 1692196547u, 1729250827u, 1767116489u,
    1805811301u, 1845353420u, 1885761398u, 1927054196u, 1969251188u, 2012372174u, 2056437387u, 2101467502u};

// 2^((x - top) rate) for the scores of a row, each as a whole number of 31 bits and a
// shift, times a factor near 1 that all of them have. x rate, exact in a fused
// multiplication, is split into whole 32nds (1.5 * 2^18 rounds to them, and
// leaves their number in the low bits) and a rest of at most 2^-6: no difference
// x - top is formed, whose rounding would have to be followed. Where top * rate
// passes 2^16 it is, and exact: scores that have any weight are within 2^-8 of top then.
// A weight is right to 2^-29 of itself: 2^-31 each for the rest's two roundings,
// the polynomial's last one and the table's, 2^-30 for the product with it; and to
// what is shifted past its last place, 2^-60 of the whole: a probability of 2^-40 keeps
// 20 bits, one below 2^-60 may be none.
// At `one`, the weight 1 is 2^(30 + one): a sum of weights is set to stay below 2^64.
// The 32 roots are a warp's own in shared memory (as a register of each lane they
// would cost a shuffle, and a convergence check, a weight).
struct Weights {
  u64 nbase2, rate2, lo2, round2;
  uint32_t roots;  // in shared memory, on 128 bytes: in 2^-30
  int one;

  static constexpr float kRound = 393216.0f, kNone = kRound - 200.0f;  // no weight below that

  __device__ __forceinline__ void set(const Place& place, float rate_hi, float rate_lo, uint32_t* table, int lane) {
    const float top = place.top == INFINITY ? 0.0f : place.top;
    const float whole = fabsf(__fmul_rn(top, rate_hi)) < 65536.0f ? __fsub_rn(__fmaf_rn(top, rate_hi, kRound), kRound) : 0.0f;
    const float base = fabsf(__fmul_rn(top, rate_hi)) < 65536.0f ? 0.0f : top;
    nbase2 = pack2(-base, -base);
    rate2 = pack2(rate_hi, rate_hi);
    lo2 = pack2(rate_lo, rate_lo);
    round2 = pack2(kRound - whole, kRound - whole);
    __syncwarp();
    table[lane] = kRoots[lane];
    __syncwarp();
    roots = smem_addr(table);
    // An fp32 sum bounds the exact one: 2^31 times that, and a bit to spare, stays below 2^64.
    one = 31 - (static_cast<int>(__float_as_uint(place.z * 1.02f) >> 23) - 127);
  }
  // Every weight divided by `all`, a sum of them at the present `one`: shares of 2^62.
  __device__ __forceinline__ void divide(u64 all, uint32_t* table, int lane) {
    const uint32_t root = table[lane];
    const int up = __clzll(static_cast<long long>(all));
    const uint32_t head = static_cast<uint32_t>((all << up) >> 32);  // its first 32 bits
    // 2^63 / head = 2^(95 - up) / all, in 2^31 .. 2^32: by fp32's reciprocal, and
    // what that leaves of 2^63.
    const float inv = __frcp_rn(static_cast<float>(head));
    const u64 near = static_cast<u64>(inv * 0x1p63f);
    const long long rest = static_cast<long long>((u64(1) << 63) - near * head);
    const u64 f = near + static_cast<u64>(static_cast<long long>(rintf(static_cast<float>(rest) * inv)));
    const uint32_t factor = f > 0xFFFFFFFFull ? 0xFFFFFFFFu : static_cast<uint32_t>(f);
    one += up - 2;  // m f / 2^31 = m 2^(64 - up) / all; a share of 2^62 is m 2^(62 + one) / all
    // Of the factor, 1 .. 2 in 2^-31, whole 32nds of an octave go with the
    // scores' and what is left, below 2^(1/32), into the roots: those stay below 2^31.
    const int i0 = __popc(__ballot_sync(kFullMask, root <= factor >> 1)) - 1;
    const u64 less = static_cast<u64>(factor) * __shfl_sync(kFullMask, root, (32 - i0) & 31);
    const u64 scaled = (static_cast<u64>(root) * (less >> (i0 ? 31 : 30)) + (u64(1) << 30)) >> 31;
    __syncwarp();
    table[lane] = static_cast<uint32_t>(scaled < 0x7FFFFFFFull ? scaled : 0x7FFFFFFFull);
    __syncwarp();
    const float round = __fadd_rn(low2(round2), static_cast<float>(i0) * 0.03125f);
    round2 = pack2(round, round);
  }
  // Of two scores (with a largest score of +infinity: shifted): their weights, or their shares of the sum.
  __device__ __forceinline__ void of2(float x0, float x1, u64& w0, u64& w1) const {
    const u64 x = add2(pack2(x0, x1), nbase2);
    const u64 near = fma2(x, rate2, round2);
    const u64 n = pack2(fmaxf(low2(near), kNone), fmaxf(high2(near), kNone));  // -infinity among them
    const u64 f = fma2(x, lo2, fma2(x, rate2, fma2(n, pack2(-1.0f, -1.0f), round2)));  // any number where there is no weight
    // 2^32 (2^f - 1), |f| < 2^-5: the series of exp(f ln 2).
    constexpr float c1 = 0x1p32f * 6.9314718e-1f, c2 = 0x1p32f * 2.4022651e-1f, c3 = 0x1p32f * 5.5504109e-2f, c4 = 0x1p32f * 9.6181291e-3f;
    u64 g = fma2(f, pack2(c4, c4), pack2(c3, c3));
    g = fma2(f, g, pack2(c2, c2));
    g = fma2(f, g, pack2(c1, c1));
    g = mul2(f, g);
    w0 = place(low2(n), low2(g));
    w1 = place(high2(n), high2(g));
  }

 private:
  __device__ __forceinline__ u64 place(float n, float g) const {
    const uint32_t e = __float_as_uint(n);  // kRound's and the 32nds
    uint32_t r, m;  // e % 32's
    asm("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(roots | (e << 2 & 124u)) : "memory");
    asm("mad.hi.s32 %0, %1, %2, %1;" : "=r"(m) : "r"(r), "r"(__float2int_rn(g)));
    u64 w;  // m 2^(one + e / 32), nothing left of it past 64
    asm("shr.u64 %0, %1, %2;" : "=l"(w) : "l"(static_cast<u64>(m) << 32), "r"(32 + (0x48C00000 >> 5) - one - static_cast<int>(e >> 5)));
    return w;
  }
};

// Sixteen bytes from byte `at` on of two vectors.
__device__ __forceinline__ uint4 shifted(const uint4& a, const uint4& b, int at) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (at & 8) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (at & 4) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  const int bits = (at & 3) * 8;
  return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits), __funnelshift_r(w[2], w[3], bits),
                    __funnelshift_r(w[3], w[4], bits));
}

template <typename T>
__global__ void __launch_bounds__(kDrawCta, kDrawThreads / kDrawCta) verify_draw_kernel(const VerifyLaunch a, const VerifyPart* parts, int splits, int cluster_bits) {
  constexpr int kWarps = kDrawCta / 32;
  constexpr int E = Vec<T>::kLen;
  __shared__ u64 slot[4][kMaxCluster];  // a word per CTA, written by all of them
  __shared__ u64 kept[kWarps], kept_too[kWarps];
  __shared__ int first_no;
  __shared__ Place row_p, row_q;
  __shared__ __align__(128) uint32_t tables[kWarps][2][32];

  uint32_t rank;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const uint32_t size = 1u << cluster_bits;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t seq = blockIdx.x >> cluster_bits;
  const int places = a.drafts + 1, rows = places + (a.draft ? a.drafts : 0);
  auto cluster_meets = [&]() {
    if (size > 1)
      asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    else
      __syncthreads();
  };
  const Heat heat = heat_of(a, seq);
  const float rate = heat.rate;
  const int count = count_of(a, seq);
  if (threadIdx.x == 0) first_no = count;
  if (size > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  // What a place needs and no kernel before this one writes: on its way ahead of the
  // wait for the sums. A token's score: a NaN counts as -infinity.
  auto score = [&](const T* row, int x) {
    const float v = Vec<T>::one(row[x]);
    return v == v ? v * heat.scale : -INFINITY;
  };
  struct Drafted {
    int x = -1;
    float u = 0.0f, xp = -INFINITY, xq = -INFINITY;
  };
  auto look = [&](int i) {
    Drafted d;
    if (i >= count) return d;
    d.x = a.draft_token[seq * a.drafts + i];
    d.u = a.u[seq * places + i];
    if (d.x >= 0 && d.x < a.vocab) {
      d.xp = score(target_row<T>(a, seq, i), d.x);
      d.xq = a.draft ? score(draft_row<T>(a, seq, i), d.x) : 0.0f;
    }
    return d;
  };
  const int first_place = static_cast<int>(rank) * kWarps + warp;
  Drafted drafted = look(first_place);
  pdl_wait();
  if (size > 1)  // a CTA's shared memory may be written by others now
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  else
    __syncthreads();

  // The sums of a row, from its parts (every lane of a warp).
  auto join = [&](int row) {
    Sum s;
    const VerifyPart* from = parts + (seq * rows + row) * splits;
    for (int i = lane; i < splits; i += 32) s.join(__ldcg(&from[i].top), __ldcg(&from[i].z), rate);
#pragma unroll 1
    for (int d = 1; d < min(splits, 32); d <<= 1) s.join(__shfl_xor_sync(kFullMask, s.top, d), __shfl_xor_sync(kFullMask, s.z, d), rate);
    return Place{__shfl_sync(kFullMask, s.top, 0), __shfl_sync(kFullMask, s.z, 0)};
  };
  auto best_of = [&](int row) {  // its index, -1 where nothing is left
    u64 k = 0;
    const VerifyPart* from = parts + (seq * rows + row) * splits;
    for (int i = lane; i < splits; i += 32) k = umax64(k, __ldcg(&from[i].key));
    k = warp_max(k);
    return k ? static_cast<int>(key_index(k)) : -1;
  };
  auto log_p = [&](float x, const Place& p) { return __fsub_rn(less_top(x, p.top) * (rate * 0.69314718f), logf(p.z)); };

  int32_t* token = a.token + seq * places;
  float* logprob = a.logprob ? a.logprob + seq * places : nullptr;
  // A place a warp of the cluster.
  for (int i = first_place; i < count; i += kWarps << cluster_bits) {
    const int x = drafted.x;
    const float u = drafted.u, xp = drafted.xp, xq = drafted.xq;
    bool ok;
    float lp = 0.0f;
    if (rate == 0.0f) {
      ok = x >= 0 && best_of(i) == x;
    } else {
      const Place p = join(i), q = a.draft ? join(places + i) : Place{0.0f, 1.0f};
      lp = log_p(xp, p);
      // u q / p < 1, with the difference of the exponents as the sum of two numbers
      // (64-bit arithmetic runs at a 64th of fp32's rate).
      const float dp = less_top(xp, p.top), up = less_rest(xp, p.top, dp), dq = less_top(xq, q.top), uq = less_rest(xq, q.top, dq);
      // p(x) > 0, as in 64 bits: not for a finite score beside +infinity, nor for a mask of the type's lowest value.
      ok = dp * rate >= kLeastOctave;
      const float d = __fsub_rn(dq, dp), back = __fsub_rn(d, dq);
      const float lost = __fadd_rn(__fsub_rn(__fsub_rn(dq, __fsub_rn(d, back)), __fadd_rn(dp, back)), __fsub_rn(uq, up));
      const float e = __fmul_rn(d, rate), n = rintf(fminf(fmaxf(e, -1000.0f), 1000.0f));
      const float f = fabsf(e) < 1000.0f ? __fadd_rn(__fsub_rn(e, n), __fmaf_rn(lost, rate, __fmaf_rn(d, rate, -e))) : 0.0f;
      if (dq > -INFINITY)  // at u = 0 the powers may be infinite: 0 < p(x) is all that is asked
        ok = ok && (u <= 0.0f || u * (__fdiv_rn(p.z, q.z) * exp2f(f)) * exp2f(0.5f * n) * exp2f(0.5f * n) < 1.0f);
      else  // no mass of the draft's
        ok = ok && u == u;
    }
    if (!ok && lane < static_cast<int>(size))
      asm volatile("red.relaxed.cluster.shared::cluster.min.s32 [%0], %1;" ::"r"(remote(&first_no, lane)), "r"(i) : "memory");
    if (lane == 0) {
      token[i] = x;
      if (logprob) logprob[i] = lp;
    }
    drafted = look(i + (kWarps << cluster_bits));
  }
  cluster_meets();
  const int accepted = first_no;
  const bool late = accepted < count;  // a token was refused
  if (rank == 0) {
    if (threadIdx.x == 0) a.accepted[seq] = accepted;
    for (int i = accepted + static_cast<int>(threadIdx.x); i < places; i += kDrawCta) {
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
  const Place pp = row_p;
  if (pp.top == -INFINITY) return;  // nothing is left of the row: -1 stays
  const bool with_q = late && a.draft && row_q.top > -INFINITY;
  // Without draft scores the refused token is taken out of p.
  const int out = late && !a.draft ? a.draft_token[seq * a.drafts + accepted] : -1;

  const Row<T> rp(target_row<T>(a, seq, accepted), a.vocab);
  const int c0 = static_cast<int>(int64_t(rp.vecs) * rank >> cluster_bits), c1 = static_cast<int>(int64_t(rp.vecs) * (rank + 1) >> cluster_bits);
  auto part_of = [](int lo, int hi, int w) { return lo + static_cast<int>(int64_t(hi - lo) * w / kWarps); };
  const int v0 = part_of(c0, c1, warp), v1 = part_of(c0, c1, warp + 1);
  // The draft's row may lie otherwise on its 16-byte boundaries: a vector of the
  // target's scores has its draft's in vectors v - behind and the one after that.
  const Row<T> rq(with_q ? draft_row<T>(a, seq, accepted) : target_row<T>(a, seq, accepted), a.vocab);
  const int behind = rq.lead < rp.lead ? 1 : 0, shift = (rq.lead - rp.lead + behind * E) * static_cast<int>(sizeof(T));
  // A lane's vectors of a round as they are in memory: nothing waits for them before the round is due.
  const int fp0 = rp.lead > 0 ? 1 : 0, fp1 = (rp.n + rp.lead) / E, fq0 = rq.lead > 0 ? 1 : 0, fq1 = (rq.n + rq.lead) / E;
  const uint4* src_p = reinterpret_cast<const uint4*>(rp.p - rp.lead);
  const uint4* src_q = reinterpret_cast<const uint4*>(rq.p - rq.lead);
  struct Round {
    uint4 p, q, q_next;
  };
  auto load_q = [&](int w) { return w >= fq0 && w < fq1 ? src_q[w] : load_edge(rq.p, w * E - rq.lead, rq.n); };
  auto fetch = [&](int v, bool both, Round& r) {
    if (v >= v1) return;
    r.p = v >= fp0 && v < fp1 ? src_p[v] : load_edge(rp.p, v * E - rp.lead, rp.n);
    if (both) {
      r.q = load_q(v - behind);
      if (shift > 0) r.q_next = load_q(v - behind + 1);
    }
  };
  // What they hold, none past this warp's part; a NaN becomes -infinity.
  auto take = [&](int v, bool both, const Round& r, uint4& vp, uint4& vq) {
    vp = v < v1 ? vec_max<T>(r.p, vec_none<T>()) : vec_none<T>();
    vq = vec_none<T>();
    if (both && v < v1) vq = vec_max<T>(shift > 0 ? shifted(r.q, r.q_next, shift) : r.q, vec_none<T>());
  };
  int turn = 0;
  // Sum over the cluster of every thread's v (and w); slot[turn - 1] keeps the CTAs' own.
  auto total_of = [&](u64 v, u64* w) {
    v = warp_sum(v);
    if (w) *w = warp_sum(*w);
    if (lane == 0) {
      kept[warp] = v;
      if (w) kept_too[warp] = *w;
    }
    __syncthreads();
    if (warp == 0) {
      v = warp_sum(lane < kWarps ? kept[lane] : 0ull);
      if (lane < static_cast<int>(size)) remote_store(remote(&slot[turn][rank], lane), v);
      if (w) {
        *w = warp_sum(lane < kWarps ? kept_too[lane] : 0ull);
        if (lane < static_cast<int>(size)) remote_store(remote(&slot[turn + 1][rank], lane), *w);
      }
    }
    cluster_meets();
    if (w) *w = warp_sum(lane < static_cast<int>(size) ? slot[turn + 1][lane] : 0ull);
    v = warp_sum(lane < static_cast<int>(size) ? slot[turn][lane] : 0ull);
    turn += w ? 2 : 1;
    return v;
  };

  // log2(e) / T as the sum of two numbers (one, where it is at an end of the range).
  const float rest = __fadd_rn(__fmaf_rn(-rate, heat.t, kLog2e), kLog2eLow);
  const float rate_lo = rate > 1.4e-45f && rate < 3.4e38f ? __fdiv_rn(rest, heat.t) : 0.0f;
  // With a largest score of +infinity only those that equal it count.
  auto scores = [&](uint4 raw, float top, float (&x)[E]) {
    Vec<T>::unpack(raw, x);
    if (top == INFINITY || heat.scale != 1.0f) {
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = top == INFINITY ? (x[e] == INFINITY ? 0.0f : -INFINITY) : x[e] * heat.scale;
    }
  };
  const Place qq = row_q;
  Weights wp, wq;
  wp.set(pp, rate, rate_lo, tables[warp][0], lane);
  if (with_q) wq.set(qq, rate, rate_lo, tables[warp][1], lane);
  // body(v, p's vector, q's vector) for this warp's part, a vector a lane (none past
  // the end: the whole warp takes part).
  auto each = [&](bool both, auto&& body) {
    Round next{};
    fetch(v0 + lane, both, next);
#pragma unroll 1
    for (int v = v0 + lane; v - lane < v1; v += 32) {
      uint4 vp, vq;
      take(v, both, next, vp, vq);
      fetch(v + 32, both, next);
      body(v, vp, vq);
    }
  };
  // With a draft's row: both rows' sums, and then shares of 2^62, whose differences are what is left.
  if (with_q) {
    u64 sum_p = 0, sum_q = 0;
    each(true, [&](int, const uint4& vp, const uint4& vq) {
      float x[E], y[E];
      scores(vp, pp.top, x);
      scores(vq, qq.top, y);
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        u64 a0, a1;
        wp.of2(x[e], x[e + 1], a0, a1);
        sum_p += a0 + a1;
        wq.of2(y[e], y[e + 1], a0, a1);
        sum_q += a0 + a1;
      }
    });
    wp.divide(total_of(sum_p, &sum_q), tables[warp][0], lane);
    wq.divide(sum_q, tables[warp][1], lane);
  }
  bool left = with_q || out >= 0;
  auto weigh = [&](int v, const uint4& vp, const uint4& vq, u64 (&w)[E]) {
    float x[E];
    scores(vp, pp.top, x);
#pragma unroll
    for (int e = 0; e < E; e += 2) wp.of2(x[e], x[e + 1], w[e], w[e + 1]);
    if (left && with_q) {
      scores(vq, qq.top, x);
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        u64 q[2];
        wq.of2(x[e], x[e + 1], q[0], q[1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) w[e + i] = w[e + i] > q[i] ? w[e + i] - q[i] : 0;
      }
    } else if (left) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (v * E - rp.lead + e == out) w[e] = 0;
    }
  };
  // A warp's part as 32 stretches, of which each lane keeps one's sum: the draw goes through one of them again.
  const int stretch = max(1, (v1 - v0 + 1023) / 1024);  // rounds of 32 vectors
  u64 of_stretch = 0;
  auto sum_left = [&]() {
    u64 sum = 0;
    int rounds = 0, who = 0;
    of_stretch = 0;
    auto close = [&]() {
      const u64 all = warp_sum(sum);
      if (lane == who) of_stretch = all;
      ++who;
      sum = 0;
      rounds = 0;
    };
    each(left && with_q, [&](int v, const uint4& vp, const uint4& vq) {
      u64 w[E];
      weigh(v, vp, vq, w);
#pragma unroll
      for (int e = 0; e < E; ++e) sum += w[e];
      if (++rounds == stretch) close();
    });
    if (rounds > 0) close();
    return total_of(of_stretch, nullptr);
  };
  u64 total = sum_left();
  // p and q agree to the 2^-29 to which either's shares hold, so that what is left is
  // rounding; or p is all on the refused token, which is taken out exactly.
  if (left && total <= (with_q ? kRounding : 0)) {
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
  const u64 to_here = before + warp_scan(of_stretch, lane);
  const int which = __ffs(__ballot_sync(kFullMask, aim < to_here)) - 1;
  before = __shfl_sync(kFullMask, to_here - of_stretch, which);
#pragma unroll 1
  for (int v = v0 + which * stretch * 32; v < v1; v += 32) {
    Round here{};
    fetch(v + lane, left && with_q, here);
    uint4 vp, vq;
    take(v + lane, left && with_q, here, vp, vq);
    u64 w[E], sum = 0;
    weigh(v + lane, vp, vq, w);
#pragma unroll
    for (int e = 0; e < E; ++e) sum += w[e];
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

// A row's vectors, wherever it starts, and those of one of its parts: as many for each thread.
int vecs_of(const VerifyLaunch& a) { return static_cast<int>(a.vocab * static_cast<int64_t>(dtype_bytes(a.dtype)) / 16) + 2; }
int part_vecs_of(int vecs, int splits) {
  const int p = (vecs + splits - 1) / splits;
  return (p + kThreads - 1) / kThreads * kThreads;
}

template <typename T>
cudaError_t launch_draw(const VerifyLaunch& a, const VerifyPart* parts, int splits, int num_sms, cudaStream_t st) {
  auto fn = verify_draw_kernel<T>;
  static PerDeviceOnce once;
  const cudaError_t ready = once.run([fn] { return cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1); });
  if (ready != cudaSuccess) return ready;
  // As many CTAs a row as run at once, of a vector a thread at least.
  const int64_t vecs = vecs_of(a);
  int bits = 0;
  while (1 << bits < kMaxCluster && a.seqs << (bits + 1) <= int64_t(num_sms) * (kDrawThreads / kDrawCta) && vecs >> bits > kDrawCta) ++bits;
  const int cluster = 1 << bits;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.seqs * cluster));
  cfg.blockDim = dim3(kDrawCta);
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
  return cudaLaunchKernelEx(&cfg, fn, a, parts, splits, bits);
}

// CTAs a row, of 8 KB at least, as many as the workspace has room for: the number
// whose rounds of CTAs read the least, a CTA's own instructions counted as 16 KB.
// 960 rows of 128000 bf16 scores: 43 us as 4 parts each, which this chooses, 52 whole,
// 46 as 3, 44 as 8, 52 as 12, 66 as 24; 671 of 100003: 28 as 4, 54 whole, 26 as 6 to 16, 33 as 24.
int splits_of(const VerifyLaunch& a, int64_t max_parts, int num_sms) {
  const int64_t rows = a.seqs * (a.drafts + 1 + (a.draft ? a.drafts : 0)), places = int64_t(num_sms) * kStatsCtas;
  const int vecs = vecs_of(a);
  const int64_t most = std::min<int64_t>(std::min<int64_t>(kMaxSplits, max_parts / rows), vecs / 512);
  int64_t best = 1, least = INT64_MAX;
  for (int64_t s = 1; s <= std::max<int64_t>(most, 1); ++s) {
    const int64_t cost = (rows * s + places - 1) / places * (part_vecs_of(vecs, static_cast<int>(s)) * int64_t(16) + 16384);
    if (cost <= least) {
      least = cost;
      best = s;
    }
  }
  return static_cast<int>(best);
}

template <typename T>
cudaError_t launch_stats(const VerifyLaunch& a, VerifyPart* parts, int splits, cudaStream_t st) {
  const unsigned rows = static_cast<unsigned>(a.drafts + 1 + (a.draft ? a.drafts : 0));
  verify_stats_kernel<T><<<dim3(static_cast<unsigned>(a.seqs), rows, static_cast<unsigned>(splits)), kThreads, 0, st>>>(
      a, parts, part_vecs_of(vecs_of(a), splits));
  return cudaGetLastError();
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
  if (a.dtype == kF32) return launch_draw<float>(a, parts, splits, num_sms, st);
  if (a.dtype == kBF16) return launch_draw<__nv_bfloat16>(a, parts, splits, num_sms, st);
  return launch_draw<__half>(a, parts, splits, num_sms, st);
}

}  // namespace rbf
