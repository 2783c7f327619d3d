// pair_tiles.cuh -- what the tensor-core products of 8-bit matrices share: how
// CTA pairs divide tiles of the output, ring positions, and wrappers of the
// instructions that their warps use.
#pragma once

#include <algorithm>

#include "tcgen05.cuh"

namespace rbf {

// A pair's part of the work, one tile's stages [k0, k1) at a time: whole tiles,
// or an equal share of all stages (Params: tiles, stages, split).
struct Walk {
  int at, end, stages, step;
  bool split;

  template <typename Params>
  __device__ __forceinline__ Walk(const Params& p, int pair, int pairs) : stages(p.stages), step(pairs), split(p.split) {
    at = split ? share_start(p, pair, pairs) : pair;
    end = split ? share_start(p, pair + 1, pairs) : p.tiles;
  }
  template <typename Params>
  static __device__ __forceinline__ int share_start(const Params& p, int pair, int pairs) {
    return static_cast<int>(static_cast<int64_t>(p.tiles) * p.stages * pair / pairs);
  }
  __device__ __forceinline__ int total() const {
    return split ? end - at : (at < end ? (end - at + step - 1) / step * stages : 0);
  }
  __device__ __forceinline__ bool next(int& tile, int& k0, int& k1) {
    if (at >= end) return false;
    if (split) {
      tile = at / stages;
      k0 = at - tile * stages;
      k1 = min(stages, k0 + (end - at));
      at += k1 - k0;
    } else {
      tile = at;
      k0 = 0;
      k1 = stages;
      at += step;
    }
    return true;
  }
};

// A position in a ring of S slots; `phase` is the parity of its full barrier.
template <int S>
struct Slot {
  int i = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void advance(int by = 1) {
    i += by;
    if (i >= S) {
      i -= S;
      phase ^= 1u;
    }
  }
};

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_addr(dst)),
      "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar)), "l"(policy)
      : "memory");
}

// One lane of a converged warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
}
// 16 lanes x 8 (16) columns as 8 x 8 blocks: registers 0-1 lane / 4, 2-3 lane / 4 + 8, columns 2 (lane % 4) + {0, 1}.
__device__ __forceinline__ void tmem_ld_blocks1(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_ld_blocks2(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
// Wait for this thread's loads; the registers pass through, so that nothing
// that uses them can move ahead of the wait.
template <int N>
__device__ __forceinline__ void tmem_wait_ld(uint32_t* r) {
  if constexpr (N == 16)
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
  else
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                 :
                 : "memory");
}
inline bool make_map(CUtensorMap* map, CUtensorMapDataType type, const void* base, int64_t cols, int64_t rows, int64_t pitch_bytes,
              int box_cols, int box_rows, CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch_bytes)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace rbf
