// Matrix products on few rows: what such a layer costs is reading its weights once, so they are
// spread over the whole card.
//
// The weights are A here: a block's tile is 128 output columns (the lanes of TMEM) by all the
// rows, padded to 16 (B, at most 128 of them).  The blocks of a cluster take runs of k of one
// tile, leave their fp32 sums in their own shared memory, and each adds a share of the rows over
// all of them, in the order of the runs, through the cluster's shared memory: one launch, no
// workspace, no order of arrival.  Two blocks an SM where their tiles are narrow, so that one
// streams while the other joins.
//
// Bound by latency, launch, first loads and the join: cold, 16 x 4,096 -> 4,096 takes 17 us in bf16, where
// its 34 MB would take 5, and 14.5 in 8 bits.  Outputs of few tiles leave SMs idle: 1 x 8,192 -> 1,024 (64
// blocks) takes 14.4 us where 2.5 would do.
#include <cmath>

#include "linear_internal.cuh"
#include "tc_ptx.cuh"
#include "tma_map.cuh"

namespace sc {
namespace {

constexpr int kEpiWarps = 4;
constexpr int kThreads = (kEpiWarps + 2) * 32;
constexpr int kMaxStages = 8;

struct FewParams {
  int64_t m, n;  // output columns, rows
  int kb, kb_per, bn, stages, tmem_cols, ways;
  uint32_t b_bytes, idesc;
  int* status;
  Epilogue ep;
};

__device__ __forceinline__ float ld_cluster(uint32_t at) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}

// This block's share of the rows (rank, rank + ways, ...), N at a time: the runs' sums in order.
template <bool BF16, int N>
__device__ __forceinline__ void join_rows(const FewParams& p, uint32_t base, int rank, int rows, int64_t col,
                                          float sw, float bias) {
#pragma unroll 1
  for (int t0 = rank; t0 < rows; t0 += N * p.ways) {
    float z[N] = {};
#pragma unroll 2
    for (int w = 0; w < p.ways; ++w) {
      const uint32_t at = map_to_rank(base + threadIdx.x * 4, static_cast<uint32_t>(w));
#pragma unroll
      for (int t = 0; t < N; ++t) z[t] += ld_cluster(at + min(t0 + t * p.ways, rows - 1) * 512);
    }
    finish_rows<BF16, N>(p.ep, t0, p.ways, min(N, (rows - t0 + p.ways - 1) / p.ways), col, z, sw, bias);
  }
}

template <bool E4M3, bool A_MN, bool BF16>
__global__ void __launch_bounds__(kThreads)
    k_gemm_few(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
               const __grid_constant__ FewParams p) {
  constexpr uint32_t kA = 128 * 128;
  constexpr int kBlock = E4M3 ? 128 : 64;
  constexpr uint32_t kPanel = 64 * 128;
  extern __shared__ uint8_t s_raw[];
  __shared__ uint64_t s_bar[2 * kMaxStages + 1];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort_word;
  volatile int* s_abort = &s_abort_word;
  const uint32_t base = (smem_u32(s_raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t stage = kA + p.b_bytes;
  const uint32_t full = smem_u32(s_bar), empty = full + 8 * kMaxStages, accf = empty + 8 * kMaxStages;
  const int rank = static_cast<int>(cluster_rank()), mt = blockIdx.x / p.ways;
  const int k0 = min(p.kb, rank * p.kb_per), k1 = min(p.kb, k0 + p.kb_per);  // may be none
  if (threadIdx.x == 0) {
    s_abort_word = 0;
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    mbar_init(accf, 1);
    fence_mbar_init();
  }
  if (warp == kEpiWarps && lane == 0) {
    prefetch_map(&ta);
    prefetch_map(&tb);
  }
  if (warp == kEpiWarps + 1) {
    tmem_alloc(smem_u32(&s_tmem), static_cast<uint32_t>(p.tmem_cols));
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  grid_release();
  grid_wait();

  if (warp == kEpiWarps) {
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 1;
      for (int kb = k0; kb < k1; ++kb) {
        if (!mbar_wait(empty + 8 * s, ph, s_abort)) {
          *s_abort = 1;
          break;
        }
        const uint32_t bar = full + 8 * s, da = base + s * stage;
        mbar_arrive_expect_tx(bar, stage);
        if (A_MN) {
          tma_load_2d(da, &ta, mt * 128, kb * kBlock, bar);
          tma_load_2d(da + kPanel, &ta, mt * 128 + 64, kb * kBlock, bar);
        } else {
          tma_load_2d(da, &ta, kb * kBlock, mt * 128, bar);
        }
        tma_load_2d(da + kA, &tb, kb * kBlock, 0, bar);
        if (++s == p.stages) s = 0, ph ^= 1;
      }
      // every copy landed before the block may end, also where the products gave up on one (a stage
      // that was never filled passes at once)
      for (int i = 0; i < p.stages; ++i) {
        if (!mbar_drain(full + 8 * s, ph)) *s_abort = 1;
        if (++s == p.stages) s = 0, ph ^= 1;
      }
    }
  } else if (warp == kEpiWarps + 1) {
    if (lane == 0) {
      const uint64_t a0 = A_MN ? smem_desc_mn(base, kPanel, 1024, 2) : smem_desc(base, 1024, 2);
      const uint64_t b0 = smem_desc(base + kA, 1024, 2);
      constexpr uint64_t kStepA = A_MN ? 16 * 128 / 16 : 2;
      int s = 0;
      uint32_t ph = 0;
      for (int kb = k0; kb < k1; ++kb) {
        if (!mbar_wait(full + 8 * s, ph, s_abort)) {
          *s_abort = 1;
          break;
        }
        tc_fence_after();
        const uint64_t at = static_cast<uint64_t>(s) * (stage >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tc_mma_any<false, E4M3>(tmem, a0 + at + k * kStepA, b0 + at + k * 2, p.idesc, kb > k0 || k > 0);
        tc_commit(empty + 8 * s);
        if (++s == p.stages) s = 0, ph ^= 1;
      }
      tc_commit(accf);
      if (!mbar_drain(accf, 0)) *s_abort = 1;
    }
  }
  // The products are done and shared memory is free for their sums.
  __syncthreads();
  tc_fence_after();
  const int rows = static_cast<int>(p.n);
  const int64_t col = static_cast<int64_t>(mt) * 128 + threadIdx.x;  // of the first four warps
  const bool mine = warp < kEpiWarps && col < p.m;
  const float bias = mine && p.ep.bias ? p.ep.bias[col] : 0.f, sw = mine && p.ep.sw ? p.ep.sw[col] : 1.f;
  if (warp < kEpiWarps && !*s_abort) {
    const uint32_t trow = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    for (int c = 0; c < rows; c += 16) {
      float v[16];
      if (k0 < k1) {
        __syncwarp();
        tmem_ld16(trow + static_cast<uint32_t>(c), v);
      } else {
#pragma unroll
        for (int t = 0; t < 16; ++t) v[t] = 0.f;
      }
      if (p.ways == 1) {
        if (mine) finish_rows<BF16, 16>(p.ep, c, 1, min(16, rows - c), col, v, sw, bias);
      } else {
#pragma unroll
        for (int t = 0; t < 16; ++t)
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(base + ((c + t) * 128 + threadIdx.x) * 4), "f"(v[t]) : "memory");
      }
    }
  }
  // TMEM goes back before the blocks of a cluster wait for each other: no block holds some
  // while it waits for one that may itself be waiting for some on an SM shared with others.
  tc_fence_before();
  __syncthreads();
  if (warp == kEpiWarps + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, static_cast<uint32_t>(p.tmem_cols));
  }
  __syncwarp();
  if (p.ways > 1) {
    cluster_sync_all();
    if (mine) {
      // up to eight rows at a time: their loads are in flight together
      const int per = (rows + p.ways - 1) / p.ways;
      if (per <= 1) join_rows<BF16, 1>(p, base, rank, rows, col, sw, bias);
      else if (per <= 2) join_rows<BF16, 2>(p, base, rank, rows, col, sw, bias);
      else join_rows<BF16, 8>(p, base, rank, rows, col, sw, bias);
    }
    __syncwarp();
    cluster_sync_all();
  }
  if (threadIdx.x == 0 && *s_abort) atomicOr(p.status, kDevErrTimeout);
}

template <bool BF16>
const void* kernel_of(const Product& p) {
  if (p.e4m3) return reinterpret_cast<const void*>(k_gemm_few<true, false, BF16>);
  return p.a.mn ? reinterpret_cast<const void*>(k_gemm_few<false, true, BF16>)
                : reinterpret_cast<const void*>(k_gemm_few<false, false, BF16>);
}

}  // namespace

sc_status product_few(const Product& p, cudaStream_t s) {
  const int block = p.e4m3 ? 128 : 64;
  FewParams g{};
  g.m = p.m;
  g.n = p.n;
  g.kb = static_cast<int>((p.k + block - 1) / block);
  g.bn = static_cast<int>((p.n + 15) / 16 * 16);
  g.b_bytes = static_cast<uint32_t>(g.bn) * 128;
  g.tmem_cols = 32;
  while (g.tmem_cols < g.bn) g.tmem_cols *= 2;
  g.idesc = p.e4m3 ? make_idesc_e4m3(128, g.bn) : make_idesc(p.ep.bf16, 128, g.bn) | (p.a.mn ? 1u << 15 : 0u);
  const int64_t tiles = (p.m + 127) / 128;
  // Runs of k until two blocks an SM have work, and no run below two k blocks.
  const int sms = device_sm_count();
  g.ways = 1;
  while (g.ways < 8 && tiles * g.ways * 2 <= 2 * sms && g.kb >= g.ways * 4) g.ways *= 2;
  g.kb_per = (g.kb + g.ways - 1) / g.ways;
  // As many stages as its run has, at most what leaves room for two blocks.
  const uint32_t stage = 128 * 128 + g.b_bytes;
  int stages = static_cast<int>((110u * 1024) / stage);
  if (stages > kMaxStages) stages = kMaxStages;
  g.stages = stages < g.kb_per ? stages : g.kb_per;
  size_t smem = static_cast<size_t>(g.stages) * stage;
  if (g.ways > 1 && smem < static_cast<size_t>(g.bn) * 512) smem = static_cast<size_t>(g.bn) * 512;
  smem += 1024;
  CUtensorMap ta, tb;
  sc_status st = product_map(&ta, p.a, p.m, p.k, p.e4m3, 128);
  if (!st) st = product_map(&tb, p.b, p.n, p.k, p.e4m3, g.bn);
  if (!st) st = rows_status_word(&g.status);
  if (st) return st;
  g.ep = p.ep;
  const void* kern = p.ep.bf16 ? kernel_of<true>(p) : kernel_of<false>(p);
  if ((st = kernel_setup(kern, smem, nullptr))) return st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = static_cast<unsigned>(g.ways);
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * g.ways));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  void* args[] = {&ta, &tb, &g};
  cudaError_t e;
  SC_LAUNCH("linear_few", s, e = cudaLaunchKernelExC(&cfg, kern, args));
  return e == cudaSuccess ? SC_OK : set_cuda_error(e, "matrix product launch");
}

}  // namespace sc
