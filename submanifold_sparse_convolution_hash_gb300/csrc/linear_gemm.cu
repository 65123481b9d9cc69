// The matrix products of the linear layers: persistent tcgen05 kernels.
//
// D tiles of 128 rows a block, or 256 a pair of blocks (cta_group::2: each block then
// stages half of B as well, so a tile costs half of B's reads), and bn columns.  One
// thread loads both operands by TMA into a ring of shared-memory stages of 128 bytes of
// k each, one issues the products, sixteen warps read the sums from TMEM and finish them;
// two accumulators let that overlap the next tile's products.
//
// What bounds it: long k, the tensor cores and the card's power (8,192 x 4,096 -> 16,384,
// bf16, gelu: 626 to 690 us by the card, 680 at the 1,597 MHz that its power limit left one; 1.59 to
// 1.76 PFLOP/s, where the library's plain product sustains 1.72; in 8 bits 8,192 x 4,096 -> 4,096 91 to 105
// us, 103 at 1,684 MHz, 2.6 to 3.0); short k, memory (480,000 x 256 -> 512, f16, silu, both outputs:
// 194 to 213 us, 5.8 to 6.3 TB/s); between them a k block's clocks: for the widest tiles what
// shared memory takes to be written and read once at 128 bytes a clock (640 of a pair's 665, 768 of 813), for
// smaller ones about 560 whatever the tile, where that explains 384 to 512.
// Four stages do what five or six do.  Two pairs that share B by TMA multicast were slower
// (715 against 658 us on the first of these): clusters of four leave 8 of 152 SMs out.
//
// Whatever its layout, an operand is staged as 128-byte rows with the 128-byte swizzle.
// K-major: a row holds 64 (8-bit: 128) values of k of one vector.  MN-major: a row holds
// 64 consecutive vectors' values at one k, 64 rows a panel.  TMA fills what lies past a
// tensor's end with zeros, so odd sizes need nothing else.
//
// Where there are too few tiles for the card, k is cut into runs; each writes fp32
// sums, which a second kernel adds in order and finishes.
#include <cmath>
#include <map>
#include <mutex>

#include "linear_internal.cuh"
#include "tc_ptx.cuh"
#include "tma_map.cuh"

namespace sc {
namespace {

__device__ int g_rows_status;
__global__ void k_rows_take_status(int* taken) { *taken = atomicExch(&g_rows_status, 0); }

constexpr int kEpiWarps = 16;
constexpr int kThreads = (kEpiWarps + 2) * 32;
constexpr int kMaxStages = 12;
constexpr int kSmemMost = 230400;                  // of 232,448, with the barriers and the alignment
constexpr uint32_t kTile = 32 * 64;               // 32 rows of 32 16-bit columns on their way out
constexpr uint32_t kStaging = kEpiWarps * 2 * kTile;
// Tile rows whose tiles are neighbours in time: they share B's columns in L2, and B is read once for each
// such group.  8,192 x 4,096 -> 16,384, 32 tile rows, one card under its power limit, us: 4 719, 8 690,
// 12 681, 16 673, 32 730.
constexpr int kGroup = 12;

struct GemmParams {
  int64_t m, n;
  int m_tiles, n_tiles, units, splits;
  int kb, kb_per;  // k blocks in all, and of a unit
  int bn, stages, tmem_cols;
  uint32_t b_bytes, idesc;
  float* part;  // splits > 1: the runs' sums [splits, m, n]
  Epilogue ep;
};

// Maps of what is written, and read beside the products: tiles of 32 rows and 32 columns.
struct OutMaps {
  CUtensorMap out, pre, res, part;
};

// 32 columns of a row from c on (of which `cols` exist): z from the sums.
__device__ __forceinline__ void scale32(const Epilogue& e, float sx, int64_t c, int cols, float (&z)[32]) {
  if (e.sw) {
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      if (4 * g >= cols) break;
      const float4 s = __ldg(reinterpret_cast<const float4*>(e.sw + c) + g);
      z[4 * g] *= sx * s.x, z[4 * g + 1] *= sx * s.y, z[4 * g + 2] *= sx * s.z, z[4 * g + 3] *= sx * s.w;
    }
  }
  if (e.bias) {
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      if (4 * g >= cols) break;
      const float4 s = __ldg(reinterpret_cast<const float4*>(e.bias + c) + g);
      z[4 * g] += s.x, z[4 * g + 1] += s.y, z[4 * g + 2] += s.z, z[4 * g + 3] += s.w;
    }
  }
}
template <int ACT>
__device__ __forceinline__ void each32(float (&z)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) z[i] = act_of(z[i], ACT);
}
__device__ __forceinline__ void act32(int act, float (&z)[32]) {
  if (act == SC_ACT_SILU) each32<SC_ACT_SILU>(z);
  else if (act == SC_ACT_GELU) each32<SC_ACT_GELU>(z);
  else if (act == SC_ACT_RELU) each32<SC_ACT_RELU>(z);
}
__device__ __forceinline__ void st_shared(uint32_t at, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 ld_shared(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at)
               : "memory");
  return v;
}

__device__ __forceinline__ void decode(const GemmParams& p, int u, int* mt, int* nt, int* k0, int* k1, int* split) {
  const int tiles = p.m_tiles * p.n_tiles;
  *split = u / tiles;
  const int t = u - *split * tiles;
  const int per = kGroup * p.n_tiles, g = t / per, r = t - g * per;
  const int rows = min(kGroup, p.m_tiles - g * kGroup);
  *nt = r / rows;
  *mt = g * kGroup + r - *nt * rows;
  *k0 = *split * p.kb_per;
  *k1 = min(p.kb, *k0 + p.kb_per);
}

template <int CTAS, bool E4M3, bool A_MN, bool B_MN, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    k_gemm(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
           const __grid_constant__ OutMaps om, const __grid_constant__ GemmParams p) {
  constexpr bool PAIR = CTAS == 2;
  constexpr uint32_t kA = 128 * 128;         // bytes of A a stage and block
  constexpr int kBlock = E4M3 ? 128 : 64;    // values of k a stage
  constexpr uint32_t kPanel = 64 * 128;      // MN-major: 64 values of k of 64 vectors
  extern __shared__ uint8_t s_raw[];
  __shared__ uint64_t s_bar[2 * kMaxStages + 5];
  __shared__ uint64_t s_res[kEpiWarps * 2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort_word;
  volatile int* s_abort = &s_abort_word;
  const uint32_t base = (smem_u32(s_raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_rank() : 0u;
  const uint32_t stage = kA + p.b_bytes;
  const uint32_t full = smem_u32(s_bar), empty = full + 8 * kMaxStages, accf = empty + 8 * kMaxStages,
                 acce = accf + 16, done = acce + 16;
  if (threadIdx.x == 0) {
    s_abort_word = 0;
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(accf + 8 * i, 1);
      mbar_init(acce + 8 * i, kEpiWarps * CTAS);
    }
    mbar_init(done, 1);
    for (int i = 0; i < kEpiWarps * 2; ++i) mbar_init(smem_u32(s_res + i), 1);
    fence_mbar_init();
  }
  if (warp == kEpiWarps && lane == 0) {
    prefetch_map(&ta);
    prefetch_map(&tb);
  }
  if (warp == kEpiWarps + 1) {
    if (PAIR) {
      tmem_alloc_pair(smem_u32(&s_tmem), static_cast<uint32_t>(p.tmem_cols));
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(&s_tmem), static_cast<uint32_t>(p.tmem_cols));
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if (PAIR) cluster_sync_all();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  grid_release();
  grid_wait();

  const int first = blockIdx.x / CTAS, stride = gridDim.x / CTAS;
  if (warp == kEpiWarps) {
    // ------------------------------------------------------------- loads
    if (lane == 0) {
      const uint32_t full_at = PAIR ? map_to_rank(full, 0) : full;
      int s = 0;
      uint32_t ph = 1;
      for (int u = first; u < p.units && !*s_abort; u += stride) {
        int mt, nt, k0, k1, split;
        decode(p, u, &mt, &nt, &k0, &k1, &split);
        const int am = (mt * CTAS + static_cast<int>(rank)) * 128;
        const int bw = p.bn / CTAS, bn0 = nt * p.bn + static_cast<int>(rank) * bw;
        for (int kb = k0; kb < k1; ++kb) {
          if (!mbar_wait(empty + 8 * s, ph, s_abort)) {
            *s_abort = 1;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(full + 8 * s, CTAS * stage);
          const uint32_t bar = full_at + 8 * s, da = base + s * stage, db = da + kA;
          const int k = kb * kBlock;
          auto load = [&](uint32_t dst, const CUtensorMap* t, int x, int y) {
            if (PAIR) tma_load_2d_pair(dst, t, x, y, bar);
            else tma_load_2d(dst, t, x, y, bar);
          };
          if (A_MN) {
            load(da, &ta, am, k);
            load(da + kPanel, &ta, am + 64, k);
          } else {
            load(da, &ta, k, am);
          }
          if (B_MN) {
            for (int c = 0; c < bw; c += 64) load(db + c * 128, &tb, bn0 + c, k);
          } else {
            load(db, &tb, k, bn0);
          }
          if (++s == p.stages) s = 0, ph ^= 1;
        }
      }
      // every stage read again before the block may end (after a timeout: its copies landed;
      // a stage that was never filled passes at once)
      for (int i = 0; i < p.stages; ++i) {
        if (!*s_abort && !mbar_wait(empty + 8 * s, ph, s_abort)) *s_abort = 1;
        if (*s_abort && rank == 0) mbar_drain(full + 8 * s, ph);
        if (++s == p.stages) s = 0, ph ^= 1;
      }
      if (rank != 0) mbar_drain(done, 0);  // nor while the pair's last arrival here is under way
    }
    __syncwarp();
  } else if (warp == kEpiWarps + 1) {
    // ---------------------------------------------------------- products
    if (lane == 0 && rank == 0) {
      const uint64_t a0 = A_MN ? smem_desc_mn(base, kPanel, 1024, 2) : smem_desc(base, 1024, 2);
      const uint64_t b0 = B_MN ? smem_desc_mn(base + kA, kPanel, 1024, 2) : smem_desc(base + kA, 1024, 2);
      // one step of 32 bytes of k: along the rows, or 16 rows down
      constexpr uint64_t kStepA = A_MN ? 16 * 128 / 16 : 2, kStepB = B_MN ? 16 * 128 / 16 : 2;
      int s = 0, j = 0;
      uint32_t ph = 0;
      for (int u = first; u < p.units && !*s_abort; u += stride, ++j) {
        int mt, nt, k0, k1, split;
        decode(p, u, &mt, &nt, &k0, &k1, &split);
        const int b = j & 1;
        if (!mbar_wait(acce + 8 * b, ((j >> 1) & 1) ^ 1, s_abort)) {
          *s_abort = 1;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(b * p.bn);
        for (int kb = k0; kb < k1; ++kb) {
          if (!mbar_wait(full + 8 * s, ph, s_abort)) {
            *s_abort = 1;
            break;
          }
          tc_fence_after();
          const uint64_t at = static_cast<uint64_t>(s) * (stage >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma_any<PAIR, E4M3>(d, a0 + at + k * kStepA, b0 + at + k * kStepB, p.idesc, kb > k0 || k > 0);
          if (PAIR) tc_commit_pair(empty + 8 * s);
          else tc_commit(empty + 8 * s);
          if (++s == p.stages) s = 0, ph ^= 1;
        }
        if (PAIR) tc_commit_pair(accf + 8 * b);
        else tc_commit(accf + 8 * b);
      }
      if (PAIR) tc_commit_pair(done);
      else tc_commit(done);
      if (!mbar_drain(done, 0)) *s_abort = 1;
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ results
    // Sixteen warps, four to each quarter of TMEM's lanes: the activation's instructions
    // are what few warps would be slow at.
    const int q = warp & 3, part = warp >> 2;
    const uint32_t acce_at = PAIR ? map_to_rank(acce, 0) : acce;
    int j = 0;
    // A warp's 32 rows leave 32 columns at a time through two tiles of
    // shared memory by TMA, one for `out` and one for `pre`, or by turns.  The residual
    // comes in the same way, into the tile that its sum leaves from, and where tiles take
    // turns ahead of its own.
    const uint32_t tiles = base + p.stages * stage + warp * 2 * kTile;
    const uint32_t res_bar = smem_u32(s_res + warp * 2);
    uint32_t res_ph = 0;  // a bit for each tile
    int turn = 0;
    bool ahead = false;
    const bool has_res = p.ep.res != nullptr, has_pre = p.ep.pre != nullptr;
    const uint32_t my_row = lane * 64, my_swz = (lane >> 1) & 3;
    auto load_res = [&](int mt, int nt, int c, int t) {
      mbar_arrive_expect_tx(res_bar + 8 * t, kTile);
      tma_load_2d(tiles + t * kTile, &om.res, nt * p.bn + c, (mt * CTAS + static_cast<int>(rank)) * 128 + q * 32,
                  res_bar + 8 * t);
    };
    for (int u = first; u < p.units; u += stride, ++j) {
      int mt, nt, k0, k1, split;
      decode(p, u, &mt, &nt, &k0, &k1, &split);
      const int b = j & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(accf + 8 * b, (j >> 1) & 1, s_abort))) {
        *s_abort = 1;
        break;
      }
      tc_fence_after();
      const int64_t i0 = static_cast<int64_t>(mt * CTAS + static_cast<int>(rank)) * 128 + q * 32, i = i0 + lane;
      const uint32_t trow = tmem + static_cast<uint32_t>(b * p.bn) + (static_cast<uint32_t>(q * 32) << 16);
      const int64_t n0 = static_cast<int64_t>(nt) * p.bn;
      if (p.splits > 1) {
        if (i0 < p.m) {
          for (int c = part * 32; c < p.bn && n0 + c < p.n; c += 128) {
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
            float v[32];
            tmem_ld32(trow + static_cast<uint32_t>(c), v);
#pragma unroll
            for (int g = 0; g < 8; ++g)
              st_shared(tiles + lane * 128 + ((g ^ (lane & 7)) << 4),
                        make_uint4(__float_as_uint(v[4 * g]), __float_as_uint(v[4 * g + 1]),
                                   __float_as_uint(v[4 * g + 2]), __float_as_uint(v[4 * g + 3])));
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_3d(&om.part, static_cast<int>(n0) + c, static_cast<int>(i0), split, tiles);
              bulk_commit();
            }
          }
        }
      } else if (i0 < p.m) {
        const float sx = p.ep.sw && i < p.m ? p.ep.sx[i] : 1.f;
        bool gone = false;
        for (int c = part * 32; c < p.bn && n0 + c < p.n; c += 128) {
          const int t = has_pre ? 0 : turn;
          const uint32_t tile = tiles + t * kTile;
          if (has_res && !ahead && lane == 0) {
            bulk_wait_read<0>();
            load_res(mt, nt, c, t);
          }
          float z[32];
          __syncwarp();
          tmem_ld32(trow + static_cast<uint32_t>(c), z);
          scale32(p.ep, sx, n0 + c, static_cast<int>(p.n - n0 - c), z);
          if (has_pre) {
            uint4 w[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) w[g] = pack8(z + 8 * g, BF16);
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
#pragma unroll
            for (int g = 0; g < 4; ++g) st_shared(tiles + kTile + my_row + ((g ^ my_swz) << 4), w[g]);
          }
          act32(p.ep.act, z);
          if (has_res) {
            if (!__all_sync(0xffffffffu, mbar_wait(res_bar + 8 * t, (res_ph >> t) & 1, s_abort))) {
              *s_abort = 1;
              gone = true;
              break;
            }
            res_ph ^= 1u << t;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              float r[8];
              unpack8(ld_shared(tile + my_row + ((g ^ my_swz) << 4)), BF16, r);
#pragma unroll
              for (int e = 0; e < 8; ++e) z[8 * g + e] += r[e];
            }
          } else if (!has_pre) {
            if (lane == 0) bulk_wait_read<1>();
            __syncwarp();
          }
#pragma unroll
          for (int g = 0; g < 4; ++g) st_shared(tile + my_row + ((g ^ my_swz) << 4), pack8(z + 8 * g, BF16));
          fence_proxy_async_smem();
          __syncwarp();
          turn ^= 1;
          if (lane == 0) {
            tma_store_2d(&om.out, static_cast<int>(n0) + c, static_cast<int>(i0), tile);
            if (has_pre) tma_store_2d(&om.pre, static_cast<int>(n0) + c, static_cast<int>(i0), tiles + kTile);
            bulk_commit();
          }
          // the residual of this warp's next tile: of this unit, else of its next one
          int u2 = u, c2 = c + 128;
          if (c2 >= p.bn || n0 + c2 >= p.n) u2 = u + stride, c2 = part * 32;
          ahead = has_res && !has_pre && u2 < p.units;
          if (ahead) {
            int mt2, nt2, x, y, z2;
            decode(p, u2, &mt2, &nt2, &x, &y, &z2);
            ahead = static_cast<int64_t>(nt2) * p.bn + c2 < p.n &&
                    static_cast<int64_t>(mt2 * CTAS + static_cast<int>(rank)) * 128 + q * 32 < p.m;
            if (ahead && lane == 0) {
              bulk_wait_read<1>();
              load_res(mt2, nt2, c2, turn);
            }
          }
        }
        if (gone) break;
      }
      __syncwarp();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (PAIR) mbar_arrive_cluster(acce_at + 8 * b);
        else mbar_arrive(acce + 8 * b);
      }
    }
    // after a timeout: a residual's tile on its way in lands before the block may end
    if (*s_abort && has_res && lane == 0) {
      mbar_drain(res_bar, res_ph & 1);
      mbar_drain(res_bar + 8, (res_ph >> 1) & 1);
    }
    __syncwarp();
  }

  if (warp < kEpiWarps && lane == 0) bulk_wait_all();
  __syncwarp();
  tc_fence_before();
  if (PAIR) cluster_sync_all();
  else __syncthreads();
  if (warp == kEpiWarps + 1) {
    tc_fence_after();
    if (PAIR) tmem_dealloc_pair(tmem, static_cast<uint32_t>(p.tmem_cols));
    else tmem_dealloc(tmem, static_cast<uint32_t>(p.tmem_cols));
  }
  if (threadIdx.x == 0 && *s_abort) atomicOr(&g_rows_status, kDevErrTimeout);
}

// Adds the runs' sums and finishes them, eight columns a thread.  Many runs: WAYS threads for
// them, each adding every WAYS-th run in order, and the first adds theirs.
template <int WAYS>
__global__ void __launch_bounds__(256) k_gemm_join(const float* __restrict__ part, int splits, int64_t rows,
                                                   int64_t cols, const Epilogue ep) {
  constexpr int kCols = 256 / WAYS;
  __shared__ float s_z[WAYS > 1 ? WAYS - 1 : 1][8][kCols + 1];
  grid_release();
  grid_wait();
  const int tx = threadIdx.x % kCols, ty = threadIdx.x / kCols;
  const int64_t per_row = cols >> 3, total = rows * per_row;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kCols;
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kCols; t0 < total; t0 += stride) {
    const int64_t t = t0 + tx, r = t / per_row, c = (t - r * per_row) * 8;
    float z[8] = {};
    if (t < total) {
#pragma unroll 4
      for (int s = ty; s < splits; s += WAYS) {
        const float4* src = reinterpret_cast<const float4*>(part + (s * rows + r) * cols + c);
        const float4 a = src[0], b = src[1];
        z[0] += a.x, z[1] += a.y, z[2] += a.z, z[3] += a.w;
        z[4] += b.x, z[5] += b.y, z[6] += b.z, z[7] += b.w;
      }
    }
    if constexpr (WAYS > 1) {
      if (ty > 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s_z[ty - 1][i][tx] = z[i];
      }
      __syncthreads();
      if (ty == 0) {
#pragma unroll
        for (int w = 0; w < WAYS - 1; ++w)
#pragma unroll
          for (int i = 0; i < 8; ++i) z[i] += s_z[w][i][tx];
      }
    }
    if (ty == 0 && t < total) finish8(ep, r, c, z);
    if constexpr (WAYS > 1) __syncthreads();
  }
}

// Tiles and cuts of a product.
struct Plan {
  int ctas, bn, splits, kb_per;
};

// Whether an operand's rows begin elsewhere than on lines of 128 bytes.
bool straddles(const Operand& o, bool e4m3) {
  return (reinterpret_cast<uintptr_t>(o.data) & 127) || (o.ld * (e4m3 ? 1 : 2)) % 128;
}

// The cheapest by an estimate in SM clocks.  A k block of a tile costs what shared memory takes to
// be written by TMA and read by the tensor cores, 128 bytes a clock (a pair's blocks read half
// of B from each other), and not below 560, a stage's own cost (measured: 570 to 590 for tiles of 64
// and 128 columns, 665 for a pair's 256, 813 for one block's 256); where an operand's rows straddle lines
// of 128 bytes, about 1.5 % of a clock more for each byte over 20 KB (9,973 x 1,992 x 1,048: 880 for
// a pair's 256 columns, 1,210 for one block's).  A unit costs that or what its
// sixteen warps take to finish it, whichever is longer (about 27 clocks a column for one
// block, 36 for a pair, whose halves wait for each other: 480,000 x 256 -> 512 with silu took
// 194 us with one block a tile, 250 with a pair).  Cut sums are written and read once more
// (about 16 bytes a clock and SM in each direction), by one more launch.
Plan plan_of(const Product& p, int kb) {
  const int sms = device_sm_count();
  const bool straddle = straddles(p.a, p.e4m3) || straddles(p.b, p.e4m3);
  Plan best{1, 64, 1, kb};
  double least = 1e300;
  for (int form = 0; form < 5; ++form) {
    const int ctas = form < 2 ? 2 : 1, bn = form == 0 || form == 2 ? 256 : form == 1 || form == 3 ? 128 : 64;
    const int64_t tiles = ((p.m + 128 * ctas - 1) / (128 * ctas)) * ((p.n + bn - 1) / bn);
    const int slots = sms / ctas;
    const double load = 128.0 * (128 + bn / ctas);  // bytes of a k block and block
    const double step = 1.04 * fmax(560.0, 256.0 + bn / ctas + bn) +
                        (straddle && load > 20480 ? 0.0145 * (load - 20480) : 0.0);
    const double finish = 700.0 + bn * (ctas == 2 ? 36.0 : 27.0);
    // whole k, and the cuts that fill one to four waves
    for (int wave = 0; wave <= 4; ++wave) {
      int64_t cuts = wave ? wave * slots / tiles : 1;
      if (wave && cuts > kb / 4) cuts = kb / 4;
      if (wave && cuts < 2) continue;
      const int per = static_cast<int>((kb + cuts - 1) / cuts), splits = (kb + per - 1) / per;
      const double waves = static_cast<double>((tiles * splits + slots - 1) / slots);
      double cost = waves * (fmax(per * step, finish) + 300.0) + 0.5 * finish;
      if (splits > 1) cost += 5000.0 + static_cast<double>(p.m) * p.n * 4.0 * splits * 2.0 / (16.0 * sms);
      if (cost < least) {
        least = cost;
        best = {ctas, bn, splits, per};
      }
    }
  }
  return best;
}

// A map of output rows in tiles of 32 rows and columns; `parts` of them one after the other.
sc_status make_out_map(CUtensorMap* map, const void* data, int64_t ld, int64_t rows, int64_t cols, int eb, int parts) {
  const EncodeTiledFn encode = tensor_map_encoder();
  if (!encode) return set_error(SC_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(parts)};
  const cuuint64_t row = static_cast<cuuint64_t>((rows > 1 ? ld : (cols + 7) / 8 * 8) * eb);
  const cuuint64_t strides[2] = {row, row * static_cast<cuuint64_t>(rows)};
  const cuuint32_t box[3] = {32, 32, 1};
  const cuuint32_t one[3] = {1, 1, 1};
  const CUresult r = encode(map, eb == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16,
                            parts ? 3 : 2, const_cast<void*>(data), dims, strides, box, one,
                            CU_TENSOR_MAP_INTERLEAVE_NONE,
                            eb == 4 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                            CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? SC_OK : set_error(SC_ERR_CUDA, "tensor map of an output");
}

template <bool BF16>
const void* kernel_of(const Product& p, int ctas) {
#define SC_K(...) reinterpret_cast<const void*>(k_gemm<__VA_ARGS__, BF16>)
#define SC_CTAS(...) (ctas == 2 ? SC_K(2, __VA_ARGS__) : SC_K(1, __VA_ARGS__))
  if (p.e4m3) return SC_CTAS(true, false, false);
  if (p.a.mn) return SC_CTAS(false, true, true);
  if (p.b.mn) return SC_CTAS(false, false, true);
  return SC_CTAS(false, false, false);
#undef SC_CTAS
#undef SC_K
}

}  // namespace

sc_status product_map(CUtensorMap* map, const Operand& o, int64_t vectors, int64_t k, bool e4m3, int box_vectors) {
  const EncodeTiledFn encode = tensor_map_encoder();
  if (!encode) return set_error(SC_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  const int eb = e4m3 ? 1 : 2;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(o.mn ? vectors : k), static_cast<cuuint64_t>(o.mn ? k : vectors)};
  // a single run's stride is never used; it has to be a legal one
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>((dims[1] > 1 ? o.ld : (dims[0] + 15) / 16 * 16) * eb)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / eb), static_cast<cuuint32_t>(o.mn ? 64 : box_vectors)};
  const cuuint32_t one[2] = {1, 1};
  const CUresult r =
      encode(map, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(o.data),
             dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? SC_OK : set_error(SC_ERR_CUDA, "tensor map of an operand");
}

sc_status rows_status_word(int** word) {
  static std::mutex mu;
  static std::map<int, int*> cache;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return set_cuda_error(e, "cudaGetDevice");
  std::lock_guard<std::mutex> lk(mu);
  int*& at = cache[dev];
  if (!at) {
    void* q = nullptr;
    e = cudaGetSymbolAddress(&q, g_rows_status);
    if (e != cudaSuccess) return set_cuda_error(e, "status word");
    at = static_cast<int*>(q);
  }
  *word = at;
  return SC_OK;
}

sc_status product_rows(const Product& p, cudaStream_t s) {
  const int block = p.e4m3 ? 128 : 64;
  const int kb = static_cast<int>((p.k + block - 1) / block);
  const Plan pl = plan_of(p, kb);
  GemmParams g{};
  g.m = p.m;
  g.n = p.n;
  const int64_t mt = (p.m + 128 * pl.ctas - 1) / (128 * pl.ctas), nt = (p.n + pl.bn - 1) / pl.bn;
  if (mt * nt * pl.splits > 0x7f000000) return set_error(SC_ERR_UNSUPPORTED, "a product of over 2^31 tiles");
  g.m_tiles = static_cast<int>(mt);
  g.n_tiles = static_cast<int>(nt);
  g.splits = pl.splits;
  g.units = static_cast<int>(mt * nt * pl.splits);
  g.kb = kb;
  g.kb_per = pl.kb_per;
  g.bn = pl.bn;
  g.b_bytes = static_cast<uint32_t>(pl.bn / pl.ctas) * 128;
  g.tmem_cols = 32;
  while (g.tmem_cols < 2 * pl.bn) g.tmem_cols *= 2;
  const uint32_t stage = 128 * 128 + g.b_bytes;
  g.stages = static_cast<int>((kSmemMost - 1024 - kStaging) / stage);
  if (g.stages > kMaxStages) g.stages = kMaxStages;
  const int M = 128 * pl.ctas;
  g.idesc = p.e4m3 ? make_idesc_e4m3(M, pl.bn)
                   : make_idesc(p.ep.bf16, M, pl.bn) | (p.a.mn ? 1u << 15 : 0u) | (p.b.mn ? 1u << 16 : 0u);
  g.ep = p.ep;
  CUtensorMap ta, tb;
  sc_status st = product_map(&ta, p.a, p.m, p.k, p.e4m3, 128);
  if (!st) st = product_map(&tb, p.b, p.n, p.k, p.e4m3, pl.bn / pl.ctas);
  if (st) return st;
  const void* kern = p.ep.bf16 ? kernel_of<true>(p, pl.ctas) : kernel_of<false>(p, pl.ctas);
  const size_t smem = 1024 + static_cast<size_t>(g.stages) * stage + kStaging;
  if ((st = kernel_setup(kern, smem, nullptr))) return st;
  if (pl.splits > 1) {
    st = dev_alloc(reinterpret_cast<void**>(&g.part), sizeof(float) * static_cast<size_t>(pl.splits) * p.m * p.n, s);
    if (st) return st;
  }
  OutMaps om{};
  if (pl.splits > 1) {
    st = make_out_map(&om.part, g.part, p.n, p.m, p.n, 4, pl.splits);
  } else {
    st = make_out_map(&om.out, p.ep.out, p.ep.ldo, p.m, p.n, 2, 0);
    if (!st && p.ep.pre) st = make_out_map(&om.pre, p.ep.pre, p.ep.ldp, p.m, p.n, 2, 0);
    if (!st && p.ep.res) st = make_out_map(&om.res, p.ep.res, p.ep.ldr, p.m, p.n, 2, 0);
  }
  if (st) {
    dev_free(g.part, s);
    return st;
  }
  const int slots = device_sm_count() / pl.ctas;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = static_cast<unsigned>(pl.ctas);
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((g.units < slots ? g.units : slots) * pl.ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  void* args[] = {&ta, &tb, &om, &g};
  cudaError_t e;
  SC_LAUNCH("linear_gemm", s, e = cudaLaunchKernelExC(&cfg, kern, args));
  if (e == cudaSuccess && pl.splits > 1) {
    int64_t rows = p.m, cols = p.n;
    const bool many = pl.splits > 8;
    const int per = many ? 32 : 256;
    int64_t blocks = (rows * (cols / 8) + per - 1) / per;
    if (blocks > device_sm_count() * 8) blocks = device_sm_count() * 8;
    int splits = pl.splits;
    Epilogue ep = p.ep;
    void* jargs[] = {&g.part, &splits, &rows, &cols, &ep};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    const void* join = many ? reinterpret_cast<const void*>(k_gemm_join<8>)
                            : reinterpret_cast<const void*>(k_gemm_join<1>);
    SC_LAUNCH("linear_join", s, e = cudaLaunchKernelExC(&cfg, join, jargs));
  }
  dev_free(g.part, s);
  return e == cudaSuccess ? SC_OK : set_cuda_error(e, "matrix product launch");
}

sc_status rows_take_status(cudaStream_t s, int* bits) {
  void* d = nullptr;
  sc_status st = dev_alloc(&d, sizeof(int), s);
  if (st) return st;
  SC_LAUNCH("rows_take_status", s, (k_rows_take_status<<<1, 1, 0, s>>>(static_cast<int*>(d))));
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = cudaMemcpyAsync(bits, d, sizeof(int), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  dev_free(d, s);
  return e == cudaSuccess ? SC_OK : set_cuda_error(e, "rows status");
}

}  // namespace sc
