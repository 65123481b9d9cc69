// Device pieces shared by the attention kernels.
#pragma once

#include "attn_internal.cuh"
#include "tc_ptx.cuh"

namespace sc {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi) {
  uint32_t r;
  if constexpr (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}


__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Work units reach a block's warps through two slots: one warp takes the next
// unit from the list's counter, the others read it in turn.  Which block takes
// which unit changes no result.
struct ItemSlots {
  uint64_t full[2], empty[2];
  AttnItem item[2];
  int head[2];  // -1: no more work
  __device__ __forceinline__ void init(int readers) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), readers);
    }
  }
};

__device__ __forceinline__ void hand_out(ItemSlots* sl, int* counter, const AttnItem* items, int units, int heads,
                                         volatile int* abort_flag) {
  for (uint32_t n = 0;; ++n) {
    const int slot = n & 1;
    const int u = atomicAdd(counter, 1);
    if (!mbar_wait_inl(smem_u32(&sl->empty[slot]), ((n >> 1) & 1) ^ 1, abort_flag)) {
      *abort_flag = 1;
      break;
    }
    if (u < units) {
      const uint4* src = reinterpret_cast<const uint4*>(items + u / heads);
      uint4* dst = reinterpret_cast<uint4*>(&sl->item[slot]);
      dst[0] = src[0];
      dst[1] = src[1];
      dst[2] = src[2];
    }
    sl->head[slot] = u < units ? u % heads : -1;
    mbar_arrive(smem_u32(&sl->full[slot]));
    if (u >= units) break;
  }
}

// A reader's side: one thread, or a warp as one.
struct ItemRing {
  ItemSlots* sl;
  uint32_t n = 0;
  __device__ __forceinline__ explicit ItemRing(ItemSlots* s) : sl(s) {}
  // The next item; false: no more (or the block gives up).
  __device__ __forceinline__ bool next(AttnItem* it, int* head, volatile int* abort_flag, bool warp) {
    const int slot = n & 1;
    bool ok = mbar_wait_inl(smem_u32(&sl->full[slot]), (n >> 1) & 1, abort_flag);
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
};

}  // namespace
}  // namespace sc
