// Device pieces shared by the attention kernels.
#pragma once

#include "attn_internal.cuh"
#include "f32x2.cuh"
#include "tc_ptx.cuh"

namespace sc {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi) {
  uint32_t r;
  if constexpr (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// One lane of the warp, the same one every time.
__device__ __forceinline__ bool elect_lane() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// A value that all lanes hold, as one of the warp: what is worked out from such
// values alone stays in the warp's own registers, which is where a product's
// operands are read from.
__device__ __forceinline__ uint32_t of_warp(uint32_t v) { return __reduce_or_sync(0xffffffffu, v); }
__device__ __forceinline__ int of_warp(int v) { return static_cast<int>(of_warp(static_cast<uint32_t>(v))); }

// Products of 128-row tiles.  The issuing warp runs as one and its elected lane
// issues: every operand is the warp's (of_warp), and the steps are unrolled with
// constant offsets, because a lane that works out a descriptor a step is slower
// than the tensor core (176 cycles a 128 x 128 x 16 step against 64).
//
// D = A B^T over the head's values: tiles of `ksteps` (at most DP / 16) steps
// of 16 values, 64-value panels of 16 KB.
template <int DP>
__device__ __forceinline__ void product_rows(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                             int ksteps) {
#pragma unroll
  for (int i = 0; i < DP / 16; ++i) {
    constexpr uint32_t kPanel = 16384 >> 4;
    const uint32_t off = (i >> 2) * kPanel + (i & 3) * 2;
    if (i < ksteps) tc_mma_lohi(d, a_lo + off, b_lo + off, hi, idesc, i > 0);
  }
}
// D (+)= A B over N steps of 16 rows of a tile from step I0 on.  A lies in TMEM,
// 8 columns a step; QUARTERS: two steps at the start of every 32 columns.
template <int I0, int N, bool QUARTERS = false>
__device__ __forceinline__ void product_cols(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                             bool add) {
#pragma unroll
  for (int i = I0; i < I0 + N; ++i)
    tc_mma_ts_lohi(d, a + i * 8 + (QUARTERS ? (i >> 1) * 16 : 0), b_lo + i * (2048 >> 4), b_hi, idesc, add || i > 0);
}

// A ring's place: stage and how often it came round.
template <int S>
struct RingPos {
  uint32_t st = 0, ph = 0;
  __device__ __forceinline__ void step() {
    if (++st == S) {
      st = 0;
      ph ^= 1;
    }
  }
  // `off` places on, off at most 2 S
  __device__ __forceinline__ RingPos at(uint32_t off) const {
    RingPos r = *this;
    r.st += off;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (r.st >= S) {
        r.st -= S;
        r.ph ^= 1;
      }
    return r;
  }
};

// Work units reach a block's warps through two slots: one warp takes the next
// unit from the list's counter, the others read it in turn.  Which block takes
// which unit changes no result.  A unit is taken when the loads ask for it, that
// is when those of the unit before have been issued, and not as soon as a slot
// is free: with two to four units a block, units taken two ahead are dealt out
// before anyone knows who is done first (some SMs were busy half the time of
// others, 29 % of a gradient's time over packed documents).
struct ItemSlots {
  uint64_t full[2], empty[2], ask;
  AttnItem item[2];
  int head[2];  // -1: no more work
  __device__ __forceinline__ void init(int readers) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), readers);
    }
    mbar_init(smem_u32(&ask), 1);
  }
};

__device__ __forceinline__ void hand_out(ItemSlots* sl, int* counter, const AttnItem* items, int units, int heads,
                                         volatile int* abort_flag) {
  for (uint32_t n = 0;; ++n) {
    const int slot = n & 1;
    const bool asked = mbar_wait_unit(smem_u32(&sl->ask), n & 1, abort_flag);
    const int u = atomicAdd(counter, 1);
    if (!asked || !mbar_wait_unit(smem_u32(&sl->empty[slot]), ((n >> 1) & 1) ^ 1, abort_flag)) {
      *abort_flag = 1;
      break;
    }
    if (u < units) {
      const uint4* src = reinterpret_cast<const uint4*>(items + u / heads);
      uint4* dst = reinterpret_cast<uint4*>(&sl->item[slot]);
      dst[0] = __ldcg(src);
      dst[1] = __ldcg(src + 1);
      dst[2] = __ldcg(src + 2);
    }
    sl->head[slot] = u < units ? u % heads : -1;
    mbar_arrive(smem_u32(&sl->full[slot]));
    if (u >= units) break;
  }
}

// A reader's side: one thread (the loads), or a warp as one.
struct ItemRing {
  ItemSlots* sl;
  uint32_t n = 0;
  __device__ __forceinline__ explicit ItemRing(ItemSlots* s) : sl(s) {}
  // The next item; false: no more (or the block gives up).
  __device__ __forceinline__ bool next(AttnItem* it, int* head, volatile int* abort_flag, bool warp) {
    const int slot = n & 1;
    if (!warp) mbar_arrive(smem_u32(&sl->ask));
    bool ok = mbar_wait_unit(smem_u32(&sl->full[slot]), (n >> 1) & 1, abort_flag);
    if (warp) ok = __all_sync(0xffffffffu, ok);
    if (!ok) {
      *abort_flag = 1;
      return false;
    }
    *it = sl->item[slot];
    *head = sl->head[slot];
    if (warp) __syncwarp();
    if (!warp || (threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&sl->empty[slot]));
    ++n;
    return *head >= 0;
  }
  // A warp's next item in place, for warps short of registers: null when there
  // is no more; it stays until release().
  __device__ __forceinline__ const AttnItem* peek(volatile int* abort_flag) {
    const int slot = n & 1;
    if (!__all_sync(0xffffffffu, mbar_wait_unit(smem_u32(&sl->full[slot]), (n >> 1) & 1, abort_flag))) {
      *abort_flag = 1;
      return nullptr;
    }
    return sl->head[slot] >= 0 ? &sl->item[slot] : nullptr;
  }
  __device__ __forceinline__ int head() const { return sl->head[n & 1]; }
  __device__ __forceinline__ void release() {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&sl->empty[n & 1]));
    ++n;
  }
};

}  // namespace
}  // namespace sc
