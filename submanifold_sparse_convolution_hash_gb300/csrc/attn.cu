// Attention over packed sequences: the work list of its kernels, made on the
// device from the sequence offsets, and the latched status.
#include "attn_internal.cuh"

namespace sc {
namespace {

__device__ int g_attn_status;

// Reads and clears the word in one step: what other streams latch meanwhile is either
// in `taken` or stays for the next check.
__global__ void k_attn_take_status(int* taken) { *taken = atomicExch(&g_attn_status, 0); }

constexpr int kPlanThreads = 1024;
constexpr int kBuckets = 256;

// Exclusive prefix sum over the block's threads; returns this thread's and
// sets *total.
__device__ __forceinline__ int block_scan(int v, int* s_warp, int* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[w] = x;
  __syncthreads();
  if (w == 0) {
    int y = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    s_warp[lane] = y;
  }
  __syncthreads();
  const int base = w ? s_warp[w - 1] : 0;
  *total = s_warp[kPlanThreads / 32 - 1];
  __syncthreads();
  return base + x - v;
}

// One block lists the work, dearest first: a unit's cost is its number of
// 128-key (or 128-row) steps, and the kernels take units in the list's order
// as they get free, so the cheap ones fill the end.  Passes over the units
// (their largest cost, a histogram of costs, their places), each over runs of
// 1024 sequences whose offsets lie in shared memory.  Offsets are checked
// first; a list that breaks a rule gives no work and latches the error.
//
// The keys of a unit are cut where the card would otherwise wait for it: with
// fewer than two units an SM into about `over` parts an SM, else only units dearer
// than an SM's share.  A part costs its fp32 rows written and read once more (four
// scenes' 100 queries, 32 units, with a join slower than today's: four parts an SM
// 228 us in all, three 227, two 244).  One block, because the list is short and a second
// launch would cost more: 10 to 13 us between events around it, part of which the
// next kernel's start overlaps.
__global__ void __launch_bounds__(kPlanThreads) k_attn_plan(const PlanArgs pa, const PlanArgs pb) {
  const PlanArgs& p = blockIdx.x ? pb : pa;
  __shared__ int s_q[kPlanThreads + 1], s_k0[kPlanThreads], s_k1[kPlanThreads], s_pre[kPlanThreads + 1];
  __shared__ int s_hist[kBuckets], s_warp[32];
  __shared__ int s_bad, s_max, s_items, s_joins, s_parts, s_rows;
  __shared__ unsigned long long s_steps;
  const int tid = threadIdx.x;
  grid_release();
  if (tid == 0) {
    s_bad = 0;
    s_max = 1;
    s_items = 0;
    s_joins = 0;
    s_parts = 0;
    s_rows = 0;
    s_steps = 0;
  }
  if (tid < kBuckets) s_hist[tid] = 0;
  __syncthreads();
  int chunk = 0;     // key tiles of a part, 0: whole
  bool dual = false;  // single row tiles are worked on by both halves
  int my_max = 1, my_rows = 0;
  unsigned long long my_steps = 0;
  for (int pass = 0; pass < 3; ++pass) {
    for (int c0 = 0; c0 < p.n_seq; c0 += kPlanThreads) {
      const int cnt = min(kPlanThreads, p.n_seq - c0);
      int total = s_pre[cnt];  // one run: it stays from the first pass
      if (pass == 0 || p.n_seq > kPlanThreads) {
        __syncthreads();
        int q0 = 0, q1 = 0, k0 = 0, k1 = 0;
        if (tid < cnt) {
          const int s = c0 + tid;
          q0 = __ldg(p.q_off + s);
          q1 = __ldg(p.q_off + s + 1);
          k0 = __ldg(p.k_off + s);
          k1 = p.k_len ? k0 : __ldg(p.k_off + s + 1);
          bool bad = false;
          if (p.k_len) {
            const int len = __ldg(p.k_len + s);
            bad = len < 0 || k0 < 0 || k0 + static_cast<int64_t>(len) > p.t_k;
            if (!bad) k1 = k0 + len;
          }
          bad = bad || q0 < 0 || q1 < q0 || q1 > p.t_q || k0 < 0 || k1 < k0 || k1 > p.t_k;
          bad = bad || (s == 0 && q0 != 0) || (s == p.n_seq - 1 && q1 != p.t_q);
          if (p.packed_keys) bad = bad || (s == 0 && k0 != 0) || (s == p.n_seq - 1 && k1 != p.t_k);
          if (bad) s_bad = 1;
          s_q[tid] = q0;
          s_k0[tid] = k0;
          s_k1[tid] = k1;
          if (tid == cnt - 1) s_q[cnt] = q1;
        }
        __syncthreads();
        if (s_bad) break;
        int tiles = 0;
        if (tid < cnt)
          tiles = p.mode == kPlanRows ? (q1 - q0 + p.pos_per_item - 1) / p.pos_per_item
                                      : (k1 - k0 + kKeyTile - 1) / kKeyTile;
        s_pre[tid] = block_scan(tiles, s_warp, &total);
        if (tid == 0) {
          s_pre[cnt] = total;  // cnt == kPlanThreads: its own place
          if (pass == 0) s_items += total;
        }
        __syncthreads();
      }
      for (int u = tid; u < total; u += kPlanThreads) {
        int lo = 0, hi = cnt - 1;  // the sequence with s_pre[lo] <= u < s_pre[lo + 1]
        while (lo < hi) {
          const int m = (lo + hi + 1) >> 1;
          if (s_pre[m] <= u) lo = m;
          else hi = m - 1;
        }
        const int t = u - s_pre[lo];
        const int lq = s_q[lo + 1] - s_q[lo], lk = s_k1[lo] - s_k0[lo];
        AttnItem it;
        int cost;
        if (p.mode == kPlanRows) {
          const int i0 = t * p.pos_per_item;
          it.q_row = s_q[lo] + i0;
          it.n_pos = min(p.pos_per_item, lq - i0);
          it.lim0 = i0 + lk - lq;
          const int seen = p.causal ? max(0, min(lk, it.lim0 + it.n_pos)) : lk;
          it.kt0 = 0;
          it.kt1 = (seen + kKeyTile - 1) / kKeyTile;
          cost = it.kt1;
        } else {
          it.q_row = s_q[lo];
          it.n_pos = lq;
          it.lim0 = lk - lq;
          it.kt0 = t;
          it.kt1 = t + 1;
          const int first = p.causal ? max(0, t * kKeyTile - it.lim0) : 0;  // first query that sees the tile
          cost = (max(0, lq - first) + p.pos_per_item - 1) / p.pos_per_item;
        }
        it.k_row = s_k0[lo];
        it.lk = lk;
        it.seq = c0 + lo;
        it.dual = dual && 2 * it.n_pos <= p.pos_per_item && cost > 1;
        const int ns = chunk && cost > chunk ? (cost + chunk - 1) / chunk : 1;
        const int part = (cost + ns - 1) / ns;
        const int parts = ns * (it.dual ? 2 : 1);
        if (pass == 0) {
          my_max = max(my_max, cost);
          my_rows = max(my_rows, p.mode == kPlanRows ? it.n_pos * p.g : kKeyTile);
          my_steps += static_cast<unsigned long long>(cost);
        } else if (pass == 1) {
          const int b = static_cast<int>(static_cast<int64_t>(kBuckets - 1) * part / s_max);
          atomicAdd(&s_hist[kBuckets - 1 - b], ns);
          if (parts > 1) atomicAdd(&s_parts, parts);
        } else {
          const int b = static_cast<int>(static_cast<int64_t>(kBuckets - 1) * part / s_max);
          int at = atomicAdd(&s_hist[kBuckets - 1 - b], ns);
          it.nsplit = ns;
          it.split = 0;
          it.slot = -1;
          if (parts > 1) {
            it.slot = atomicAdd(&s_parts, parts);
            const int j = atomicAdd(&s_joins, 1);
            if (j < p.join_cap) p.joins[j] = it;
          }
          const int end = it.kt1;
          for (int i = 0; i < ns; ++i, ++at) {
            it.split = i;
            if (ns > 1 && p.mode == kPlanRows) {
              it.kt0 = min(end, i * part);
              it.kt1 = min(end, it.kt0 + part);
            }
            if (at < p.cap) p.items[at] = it;
          }
        }
      }
      __syncthreads();
    }
    if (s_bad) break;
    if (pass == 0) {
      my_max = __reduce_max_sync(0xffffffffu, my_max);
      my_rows = __reduce_max_sync(0xffffffffu, my_rows);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) my_steps += __shfl_xor_sync(0xffffffffu, my_steps, o);
      if ((tid & 31) == 0) {
        atomicMax(&s_max, my_max);
        atomicMax(&s_rows, my_rows);
        atomicAdd(&s_steps, my_steps);
      }
      __syncthreads();
      if (p.part_rows > 0) {
        const unsigned long long steps = s_steps * p.heads_kv;
        const bool few = static_cast<int64_t>(s_items) * p.heads_kv < 2 * p.sms;
        const unsigned long long over = static_cast<unsigned long long>(p.sms) * (few ? p.over : 1);
        const unsigned long long c = (steps + over - 1) / over;
        chunk = static_cast<int>(c < static_cast<unsigned long long>(p.min_tiles) ? p.min_tiles : c);
        dual = p.dual;
      }
    }
    if (pass == 1) {
      // partial results that do not fit: whole units after all
      if (s_parts * static_cast<int64_t>(p.heads_kv) * s_rows > p.part_rows) {
        __syncthreads();
        chunk = 0;
        dual = false;
        if (tid < kBuckets) s_hist[tid] = 0;
        if (tid == 0) s_parts = 0;
        pass = 0;  // the histogram again
        __syncthreads();
        continue;
      }
      int total;
      const int v = tid < kBuckets ? s_hist[tid] : 0;
      const int e = block_scan(v, s_warp, &total);
      if (tid < kBuckets) s_hist[tid] = e;
      if (tid == 0) {
        s_parts = 0;
        p.header[0] = min(total, p.cap);
      }
      __syncthreads();
    }
  }
  __syncthreads();
  if (tid == 0) {
    if (s_bad || p.n_seq == 0) p.header[0] = 0;
    if (s_bad) atomicOr(p.status, kDevErrRange);
    p.header[1] = 0;
    p.header[2] = s_bad ? 0 : min(s_joins, p.join_cap);
    p.header[3] = s_rows;
  }
  grid_wait();  // the kernel before this one is done when this one is
}

}  // namespace

int* attn_status_word() {
  void* p = nullptr;
  return cudaGetSymbolAddress(&p, g_attn_status) == cudaSuccess ? static_cast<int*>(p) : nullptr;
}

sc_status attn_plan(const PlanArgs& a, const PlanArgs* b, bool after, cudaStream_t s) {
  PlanArgs x = a, y = b ? *b : a;
  void* args[] = {&x, &y};
  const void* kern = reinterpret_cast<const void*>(k_attn_plan);
  const unsigned grid = b ? 2 : 1;
  cudaError_t e;
  SC_LAUNCH("attn_plan", s,
            (e = after ? launch_after(kern, grid, kPlanThreads, 0, s, args)
                       : cudaLaunchKernel(kern, dim3(grid), dim3(kPlanThreads), args, 0, s)));
  return e == cudaSuccess ? SC_OK : set_cuda_error(e, "attn_plan");
}

// The map of rows [tokens, heads, d] for boxes of 64 values x box_heads x
// box_tokens, rows of 128 bytes in shared memory with their 16-byte pieces
// swizzled as the matrix descriptors expect; past the ends it reads zeros.
sc_status attn_map(CUtensorMap* m, const void* data, sc_dtype dt, int d, int heads, int64_t tokens, int64_t ts,
                   int64_t hs, int box_heads, int box_tokens) {
  const EncodeTiledFn enc = tensor_map_encoder();
  if (!enc) return set_error(SC_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  // a dimension of one row needs a legal stride all the same
  const int64_t row = (static_cast<int64_t>(d) * 2 + 15) / 16 * 16;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(heads > 1 ? hs * 2 : row),
                                 static_cast<cuuint64_t>(tokens > 1 ? ts * 2 : row)};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_tokens)};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = enc(m, dt == SC_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                         const_cast<void*>(data), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return set_error(SC_ERR_UNSUPPORTED, "these strides make no tensor map");
  return SC_OK;
}

sc_status attn_take_status(cudaStream_t s, int* bits) {
  int* taken = nullptr;
  sc_status st = dev_alloc(reinterpret_cast<void**>(&taken), sizeof(int), s);
  if (st) return st;
  SC_LAUNCH("attn_take_status", s, (k_attn_take_status<<<1, 1, 0, s>>>(taken)));
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = cudaMemcpyAsync(bits, taken, sizeof(int), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  dev_free(taken, s);
  return e == cudaSuccess ? SC_OK : set_cuda_error(e, "attention status");
}

}  // namespace sc
