// Attention's gradients over packed sequences.
//
// With P = exp(scale Q K^T - lse), delta = gout . out per row,
//   dS = P * (gout V^T - delta),  gq = scale dS K,  gk = scale dS^T Q,  gv = P^T gout.
// Two kernels, each of whose blocks owns what it writes, so no sum depends on an order
// of arrival and the same inputs give the same bits:
//   gk, gv  a block owns 128 keys and walks the rows (all queries and heads of
//           the group): four products a step, S^T = K Q^T, dP^T = V gout^T,
//           gv += P^T gout, gk += dS^T Q
//   gq      a block owns 128 rows and walks the keys: three products a step,
//           S = Q K^T, dP = gout V^T, gq += dS K
// That is seven products where one pass with atomic adds to gq needs five; the
// two passes need no fp32 copy of gq and no order of arrival.
// P and dS go back to TMEM, rounded to 16 bits, as the first operand of the
// second products; sums stay in TMEM in fp32.  f16 has few bits below 2^-14 and
// a weight of a list of thousands lies there, so P is held times 2^8 (at most
// 256), and dS times a power of two of its sequence's own, from the largest |gout|
// and |v| (undone in fp32 as the sums are written).  delta is taken from `out` as the
// forward rounded it.  The roundings of dS and of `out` are what gq and gk are off by (1.5
// to 1.9 times the error of an fp32 computation rounded once, up to 2.5 where a few keys
// take most of the weight and dP - delta cancels).
//
// What bounds them.  A step is a chain: S, P, dP, dS, product, each part waiting
// for the one before; the tensor cores are busy 60 % (gk, gv) and 50 % (gq) of an
// SM's time at 128 values and 22 % and 18 % at 32, where the exponentials, the
// conversions and, for gk and gv, the row statistics read from shared memory by
// every key's lane (47 % of that path) take as long as the products.  Kernel
// times: five documents of 100 to 3500 tokens, causal, 16 query and 4 key heads of
// 128, bf16: 123 us and 97 us; 96 windows of 300 to 1000 voxels, 8 heads of 32,
// f16: 205 us and 190 us, and 27 us for the row statistics.  Measured and left out: tiles of 64 rows by two groups
// of warps (287 and 224 us for the windows); the next dP made as soon as this one
// has been read, with dS beside P (209 and 196 us).
#include "attn_device.cuh"

namespace sc {
namespace {

constexpr int kBwdThreads = 640;
constexpr int kBwdMaxStages = 12;
constexpr int kMinPartTiles = 8;  // least row tiles of a part
// gk, gv: registers a thread as launched; four warps drop, sixteen raise.
constexpr int kKvRegs = 96, kKvSideRegs = 64, kKvMainRegs = 104;
static_assert(128 * kKvSideRegs + 512 * kKvMainRegs <= kBwdThreads * kKvRegs, "no more than the block has");
// Ring tiles beside what stays: two pairs of K and V (one at 128 values) and
// pairs of Q and gout; or such pairs of Q and gout, and single K and V tiles.
constexpr int kv_pairs(int dp) { return dp == 64 ? 2 : 1; }
constexpr int kv_stages(int dp) { return dp == 64 ? 8 : 4; }
constexpr int q_pairs(int dp) { return dp == 64 ? 2 : 1; }
constexpr int q_stages(int dp) { return dp == 64 ? 8 : 5; }

// P is held times 2^kPShift.
template <bool BF16>
constexpr float kPShift = BF16 ? 0.f : 8.f;
template <bool BF16>
constexpr float kPDown = BF16 ? 1.f : 1.f / 256.f;

struct BwdParams {
  // [t_q, heads_q]: lse log2 e - kPShift (+inf: no key seen), delta 2^-kPShift
  const float2* stat;
  const int* header;
  int* counter;
  const AttnItem* items;
  uint8_t *o0, *o1;      // gq, or gk and gv
  int64_t o0_t, o0_h, o1_t, o1_h;  // bytes
  int heads_q, heads_kv, g, pos, d;
  float scale, scale_log2;
  int causal;
  int first;             // gq: no gk, gv kernel ran before it
  float* part;           // gk, gv of cut key tiles: [slot][head][2][128][d]
  const float* peak;     // f16: [sequence][largest value of |gout|, of |v|]; null: dS is held as it is
  int* status;
};

// f16 has few bits below 2^-14 and ends at 65504, and dS = P (dP - delta) may lie far
// to either side.  |dP - delta| is at most 2 d times the sequence's largest values of
// gout and of v, so dS is held times the power of two that takes this bound to between
// 2^14 and 2^15.
template <bool BF16>
__device__ __forceinline__ float ds_up(const BwdParams& p, const AttnItem& it) {
  if (BF16 || !p.peak) return 1.f;
  const float2 m = __ldcg(reinterpret_cast<const float2*>(p.peak) + it.seq);
  const float b = static_cast<float>(2 * p.d) * m.x * m.y;
  return b > 0.f ? __uint_as_float((127u + 14 + 127 - (__float_as_uint(b) >> 23)) << 23) : 1.f;
}
// 1 / up
__device__ __forceinline__ float ds_down(float up) { return __uint_as_float((254u << 23) - __float_as_uint(up)); }

// 8 values of a 16-bit row, times `f`.
template <bool BF16>
__device__ __forceinline__ void store8(uint8_t* dst, const uint32_t* v, float f) {
  *reinterpret_cast<uint4*>(dst) =
      make_uint4(pack_pair<BF16>(__uint_as_float(v[0]) * f, __uint_as_float(v[1]) * f),
                 pack_pair<BF16>(__uint_as_float(v[2]) * f, __uint_as_float(v[3]) * f),
                 pack_pair<BF16>(__uint_as_float(v[4]) * f, __uint_as_float(v[5]) * f),
                 pack_pair<BF16>(__uint_as_float(v[6]) * f, __uint_as_float(v[7]) * f));
}

// A TMEM accumulator row of d values to global memory (`have` false: zeros).
template <bool BF16>
__device__ __forceinline__ void store_acc(uint32_t t, uint8_t* dst, int d, float f, bool have, bool live) {
  for (int c = 0; c < d; c += 16) {
    uint32_t o[16];
    if (have) {
      tmem_ld16_raw(t + c, o);
    } else {
#pragma unroll
      for (int u = 0; u < 16; ++u) o[u] = 0u;
    }
    if (live) {
      store8<BF16>(dst + c * 2, o, f);
      if (c + 8 < d) store8<BF16>(dst + c * 2 + 16, o + 8, f);
    }
  }
}

// ------------------------------------------------------------ statistics --
struct StatParams {
  const uint8_t *gout, *out, *v;
  int64_t gt, gh, ot, oh, vt, vh;  // bytes
  const float* lse;
  float2* stat;
  int64_t rows, v_rows;  // t_q * heads_q; f16: t_k * heads_kv
  int heads_q, heads_kv, d;
  int runs;              // of 32 / LPR rows a warp, a multiple of kStatBatch
  unsigned blocks;       // of the rows; those of v come after them
  const int *q_off, *k_off;
  int n_seq;
  float* peak;           // f16: as in BwdParams
};

template <bool BF16>
__device__ __forceinline__ float dot2(uint32_t a, uint32_t b) {
  float2 x, y;
  if constexpr (BF16) {
    x = make_float2(__uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u));
    y = make_float2(__uint_as_float(b << 16), __uint_as_float(b & 0xFFFF0000u));
  } else {
    x = __half22float2(*reinterpret_cast<const __half2*>(&a));
    y = __half22float2(*reinterpret_cast<const __half2*>(&b));
  }
  return fmaf(x.x, y.x, x.y * y.y);
}

// The sequence that holds token t: the last one that begins at or before it.  A lane
// by itself, or a warp as one, which takes two steps to 1024 sequences.
__device__ __forceinline__ int seq_of(const int* off, int n_seq, int64_t t) {
  int lo = 0, hi = n_seq - 1;
  while (lo < hi) {
    const int m = (lo + hi + 1) >> 1;
    if (__ldg(off + m) <= t) lo = m;
    else hi = m - 1;
  }
  return lo;
}
__device__ __forceinline__ int seq_of_warp(const int* off, int n_seq, int64_t t) {
  int lo = 0, n = n_seq;  // among lo .. lo + n - 1
  while (n > 1) {
    const int step = (n + 31) / 32, at = (threadIdx.x & 31) * step;
    const bool past = at >= n || __ldg(off + lo + at) > t;
    const uint32_t b = __ballot_sync(0xffffffffu, past);
    const int k = max((b ? __ffs(b) - 1 : 32) - 1, 0);
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// The largest magnitude among the f16 values that a warp meets in consecutive rows,
// into their sequences' words.  The order of a maximum changes nothing; values that
// are not finite spoil their own rows and do not count; offsets that break the rules
// name some sequence or other.
struct Peak {
  float* peak;
  const int* off;
  int n_seq, heads, s;
  int64_t begin = 0, end = 0;  // rows of sequence s
  uint32_t m = 0;              // two f16 magnitudes
  __device__ __forceinline__ Peak(float* peak_, const int* off_, int n_seq_, int heads_)
      : peak(peak_), off(off_), n_seq(n_seq_), heads(heads_) {}
  __device__ __forceinline__ void start(int64_t row) {
    s = seq_of_warp(off, n_seq, row / heads);
    begin = static_cast<int64_t>(__ldg(off + s)) * heads;
    end = static_cast<int64_t>(__ldg(off + s + 1)) * heads;
  }
  static __device__ __forceinline__ uint32_t largest(uint32_t v) { return max(v & 0xFFFFu, v >> 16); }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  // f16 bits to a sequence's word, as fp32 bits (which order as the values do)
  __device__ __forceinline__ void put(int seq, uint32_t v) const {
    const float f = __half2float(__ushort_as_half(static_cast<unsigned short>(v)));
    atomicMax(reinterpret_cast<uint32_t*>(peak + 2 * static_cast<int64_t>(seq)), __float_as_uint(f));
  }
  __device__ __forceinline__ void flush() {
    const uint32_t v = __reduce_max_sync(0xffffffffu, largest(m));
    if ((threadIdx.x & 31) == 0 && v) put(s, v);
    m = 0;
  }
  // A lane's values of `row` (zeros past the end); `last`: the warp's last row.
  __device__ __forceinline__ void take(uint4 a, int64_t row, int64_t last) {
    constexpr uint32_t kAbs = 0x7FFF7FFFu, kInf = 0x7C00u;
    uint32_t v = max2(max2(a.x & kAbs, a.y & kAbs), max2(a.z & kAbs, a.w & kAbs));
    if (largest(v) >= kInf) [[unlikely]] {
      const uint32_t w[4] = {a.x & kAbs, a.y & kAbs, a.z & kAbs, a.w & kAbs};
      v = 0;
      for (int i = 0; i < 4; ++i) {
        if ((w[i] & 0xFFFFu) < kInf) v = max(v, w[i] & 0xFFFFu);
        if (w[i] >> 16 < kInf) v = max(v, w[i] >> 16);
      }
    }
    if (last < end) {
      m = max2(m, v);
      return;
    }
    // rows of this sequence, of the last row's, and of short ones between them
    const bool of_s = row < end;
    if (of_s) m = max2(m, v);
    flush();
    start(last);
    if (of_s) return;
    if (row >= begin) m = v;
    else if (v) put(seq_of(off, n_seq, row / heads), largest(v));
  }
};

// delta = gout . out and lse in powers of two, LPR lanes a row, a warp p.runs runs of
// consecutive rows; for f16 also the largest values of gout and v of each sequence.
// Memory bounds it (all are read once).
constexpr int kStatBatch = 3, kStatBlocks = 4;  // runs at a time; blocks an SM
template <bool BF16, int LPR>
__global__ void __launch_bounds__(256, kStatBlocks) k_attn_stat(const StatParams p) {
  constexpr int ROWS = 32 / LPR;
  grid_release();
  const int gl = threadIdx.x % LPR, lane = threadIdx.x & 31;
  const bool of_v = !BF16 && blockIdx.x >= p.blocks;
  const int64_t rows = of_v ? p.v_rows : p.rows;
  const int64_t block_first = (blockIdx.x - (of_v ? p.blocks : 0u)) * (8ll * ROWS * p.runs);
  const int64_t first = block_first + (threadIdx.x >> 5) * (static_cast<int64_t>(ROWS) * p.runs);
  const int heads = of_v ? p.heads_kv : p.heads_q;
  if (first >= rows) return;
  Peak peak(of_v ? p.peak + 1 : p.peak, of_v ? p.k_off : p.q_off, p.n_seq, heads);
  const int64_t xt = of_v ? p.vt : p.gt, xh = of_v ? p.vh : p.gh;
  // this lane's row, and its place in x and in out, a run further each time
  const int64_t t0 = (first + lane / LPR) / heads;
  int h = static_cast<int>(first + lane / LPR - t0 * heads);
  const int dt = ROWS / heads, dh = ROWS % heads;
  const uint8_t* x = (of_v ? p.v : p.gout) + t0 * xt + h * xh + gl * 16;
  const uint8_t* y = p.out + t0 * p.ot + h * p.oh + gl * 16;
  const int64_t x_run = dt * xt + dh * xh, x_wrap = xt - heads * xh;
  const int64_t y_run = dt * p.ot + dh * p.oh, y_wrap = p.ot - heads * p.oh;
#pragma unroll 1
  for (int i0 = 0; i0 < p.runs && first + i0 * ROWS < rows; i0 += kStatBatch) {
    uint4 a[kStatBatch], b[kStatBatch];
    float lse[kStatBatch];
#pragma unroll
    for (int i = 0; i < kStatBatch; ++i) {
      const int64_t r = first + (i0 + i) * ROWS + lane / LPR;
      a[i] = b[i] = make_uint4(0, 0, 0, 0);
      lse[i] = 0.f;
      if (r < rows && gl * 8 < p.d) {
        a[i] = __ldg(reinterpret_cast<const uint4*>(x));
        if (!of_v) {
          b[i] = __ldg(reinterpret_cast<const uint4*>(y));
          if (gl == 0) lse[i] = __ldg(p.lse + r);
        }
      }
      x += x_run;
      y += y_run;
      h += dh;
      if (h >= heads) {
        h -= heads;
        x += x_wrap;
        y += y_wrap;
      }
    }
    if (!BF16 && i0 == 0) peak.start(first);
#pragma unroll
    for (int i = 0; i < kStatBatch; ++i) {
      const int64_t r0 = first + (i0 + i) * ROWS, r = r0 + lane / LPR;
      if constexpr (!BF16) {
        if (r0 < rows) peak.take(a[i], r, min(r0 + ROWS, rows) - 1);
        if (of_v) continue;
      }
      float s = (dot2<BF16>(a[i].x, b[i].x) + dot2<BF16>(a[i].y, b[i].y)) +
                (dot2<BF16>(a[i].z, b[i].z) + dot2<BF16>(a[i].w, b[i].w));
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (gl == 0 && r < rows) {
        float l2 = lse[i] == -INFINITY ? INFINITY : fmaf(lse[i], kLog2e, -kPShift<BF16>);
        // The fp32 lse holds a weight's exponent to 2^-22 of |lse|.  Where that is more
        // than a fraction of a power of two a weight could come out as an infinity:
        // there the exponents are taken lower by as much, so that none is above 1.
        if (fabsf(l2) > 262144.f && l2 < INFINITY) l2 = fmaf(fabsf(l2), 0x1p-21f, l2);
        p.stat[r] = make_float2(l2, s * kPDown<BF16>);
      }
    }
  }
  if constexpr (!BF16) peak.flush();
}

// --------------------------------------------------------------- gk, gv --
constexpr int kRowSlots = 4;
struct KvSmem {
  uint64_t full[kBwdMaxStages], empty[kBwdMaxStages];
  uint64_t kv_full[2], kv_empty[2];
  uint64_t rows_ok[kRowSlots], rows_free[kRowSlots];  // row statistics (and the rows of a tile that ends inside)
  // p_ready: one for each S.  S of the next tile is there already, so a quick warp
  // may arrive for the next P before a slow one has for this; on one barrier the
  // two would count as one tile's.
  uint64_t s_full[2], p_ready[2], dp_full, ds_ready, acc_full;
  uint64_t drained;
  uint32_t tmem;
  int abort;
  ItemSlots slots;
  __align__(16) float nlse2[kRowSlots][128];  // negated, as the products take them
  __align__(16) float ndelta[kRowSlots][128];
  __align__(16) int lim[kRowSlots][128];  // causal: the last key that the row sees
};

// First row tile (of p.pos queries) of the item, of those that see its key tile,
// and their number.
__device__ __forceinline__ int row_tiles(const BwdParams& p, const AttnItem& it, int* first) {
  int i0 = 0;
  if (p.causal) i0 = max(0, it.kt0 * kKeyTile - it.lim0);
  *first = i0 / p.pos;
  if (i0 >= it.n_pos) return 0;
  int n = (it.n_pos + p.pos - 1) / p.pos - *first;
  if (it.nsplit > 1) {
    const int part = (n + it.nsplit - 1) / it.nsplit, skip = min(n, it.split * part);
    *first += skip;
    n = min(part, n - skip);
  }
  return n;
}

template <bool BF16, int DP>
__global__ void __launch_bounds__(kBwdThreads, 1)
    k_attn_bwd_kv(const BwdParams p, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap gmap,
                  const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  constexpr int PANELS = DP / 64, KVB = kv_pairs(DP);
  constexpr uint32_t PANEL = 128 * 128, TILE = PANELS * PANEL;
  constexpr uint32_t S = kv_stages(DP);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t skv = smem_u32(smem);                 // KVB pairs of K and V
  const uint32_t srow = skv + 2 * KVB * TILE;          // ring: Q, gout, Q, gout, ...
  KvSmem* sm = reinterpret_cast<KvSmem*>(smem + (2 * KVB + S) * TILE);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &sm->abort;
  const int used = p.pos * p.g;  // rows of a tile; the rest stays zero

  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < S; ++s) {
      mbar_init(smem_u32(&sm->full[s]), 1);
      mbar_init(smem_u32(&sm->empty[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&sm->kv_full[s]), 1);
      mbar_init(smem_u32(&sm->kv_empty[s]), 1);
      mbar_init(smem_u32(&sm->s_full[s]), 1);
      mbar_init(smem_u32(&sm->p_ready[s]), 16);
    }
    for (int s = 0; s < kRowSlots; ++s) {
      mbar_init(smem_u32(&sm->rows_ok[s]), 1);
      mbar_init(smem_u32(&sm->rows_free[s]), 16);
    }
    mbar_init(smem_u32(&sm->dp_full), 1);
    mbar_init(smem_u32(&sm->ds_ready), 16);
    mbar_init(smem_u32(&sm->acc_full), 1);
    mbar_init(smem_u32(&sm->drained), 1);
    sm->slots.init(19);  // 16 warps for the weights, loads, products, ends
    sm->abort = 0;
    fence_mbar_init();
  }
  if (warp == 17) {
    tmem_alloc(smem_u32(&sm->tmem), 512);
    tmem_relinquish();
  }
  // rows of the ring that no copy writes
  for (uint32_t s = 0; s < S * PANELS; ++s)
    for (int i = used * 8 + static_cast<int>(threadIdx.x); i < 128 * 8; i += kBwdThreads)
      *reinterpret_cast<uint4*>(smem + 2 * KVB * TILE + s * PANEL + i * 16) = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_wait();     // the plan and the statistics
  grid_release();  // gq's kernel needs no more than these either
  const uint32_t tmem = sm->tmem;
  // To 64 values there is room for a second S, so that the next tile's is made
  // ahead; else S waits for the product that reads P over it.
  constexpr int SB = DP == 64 ? 2 : 1;
  const uint32_t t_s = tmem, t_dp = tmem + SB * 128, t_dv = t_dp + 128, t_dk = t_dv + DP;
  const int units = __ldcg(p.header) * p.heads_kv;

  if (warp == 16) {
    // =========================================================== loads
    regs_drop<kKvSideRegs>();
    if (lane == 0) {
      ItemRing ring(&sm->slots);
      AttnItem it;
      int head;
      uint32_t k = 0, nkv = 0;
      RingPos<S> r;
      while (ring.next(&it, &head, abort_flag, false)) {
        int first;
        const int n = row_tiles(p, it, &first);
        if (n == 0) continue;
        const uint32_t b = nkv % KVB;
        if (!mbar_wait_inl(smem_u32(&sm->kv_empty[b]), ((nkv / KVB) & 1) ^ 1)) {
          sm->abort = 1;
          break;
        }
        ++nkv;
        mbar_arrive_expect_tx(smem_u32(&sm->kv_full[b]), 2 * TILE);
        for (int c = 0; c < PANELS; ++c) {
          tma_load_3d(skv + 2 * b * TILE + c * PANEL, &kmap, c * 64, head, it.k_row + it.kt0 * kKeyTile,
                      smem_u32(&sm->kv_full[b]));
          tma_load_3d(skv + (2 * b + 1) * TILE + c * PANEL, &vmap, c * 64, head, it.k_row + it.kt0 * kKeyTile,
                      smem_u32(&sm->kv_full[b]));
        }
        bool ok = true;
        for (int i = first; i < first + n && ok; ++i)
          for (int which = 0; which < 2; ++which, ++k, r.step()) {
            const uint32_t st = r.st;
            if (!mbar_wait_inl(smem_u32(&sm->empty[st]), r.ph ^ 1)) {
              sm->abort = 1;
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(smem_u32(&sm->full[st]), PANELS * used * 128);
            for (int c = 0; c < PANELS; ++c)
              tma_load_3d(srow + st * TILE + c * PANEL, which ? &gmap : &qmap, c * 64, head * p.g,
                          it.q_row + i * p.pos, smem_u32(&sm->full[st]));
          }
        if (!ok) break;
      }
      const uint32_t f0 = nkv > KVB ? nkv - KVB : 0;
      for (uint32_t i = f0; i < nkv; ++i)
        if (!mbar_wait_inl(smem_u32(&sm->kv_full[i % KVB]), (i / KVB) & 1)) sm->abort = 1;
      const uint32_t f1 = k > S ? k - S : 0;
      for (uint32_t i = f1; i < k; ++i)
        if (!mbar_wait_inl(smem_u32(&sm->full[i % S]), (i / S) & 1)) sm->abort = 1;
    }
    __syncwarp();
  } else if (warp == 17) {
    // ======================================================== products
    regs_drop<kKvSideRegs>();
    const int dn = (p.d + 15) & ~15;
    const int ksteps = dn / 16;
    const uint32_t id_s = make_idesc(BF16, 128, 128);
    const uint32_t id_a = make_idesc(BF16, 128, dn) | (1u << 16);
    const uint64_t dk = smem_desc(skv, 1024, 2), dt = smem_desc_mn(srow, PANEL, 1024, 2);
    const uint32_t kv_lo = static_cast<uint32_t>(dk), hi = static_cast<uint32_t>(dk >> 32);
    const uint32_t row_lo = static_cast<uint32_t>(smem_desc(srow, 1024, 2));
    const uint32_t rowt_lo = static_cast<uint32_t>(dt), rowt_hi = static_cast<uint32_t>(dt >> 32);
    constexpr uint32_t T16 = TILE >> 4;
    const uint32_t tb = of_warp(tmem);
    const uint32_t u_s = tb, u_dp = tb + SB * 128, u_dv = u_dp + 128, u_dk = u_dv + DP;
    ItemRing ring(&sm->slots);
    AttnItem it;
    int head;
    uint32_t nkv = 0, nr = 0, np = 0;
    RingPos<S> cur;  // the row tile's Q; its gout is the next stage
    while (ring.next(&it, &head, abort_flag, true)) {
      int first;
      const int n = of_warp(row_tiles(p, it, &first));
      if (n == 0) continue;
      const uint32_t b = nkv % KVB;
      bool ok = mbar_wait_inl(smem_u32(&sm->kv_full[b]), (nkv / KVB) & 1);
      ++nkv;
      const uint32_t k_at = kv_lo + 2 * b * T16, v_at = k_at + T16;
      // S of row tile nr, once its copies have landed and its rows are in order
      // (the statistics' warp has waited for the copies; they are looked at again,
      // because the products read them by another path)
      auto scores = [&](const RingPos<S>& at) {
        ok = ok && mbar_wait2_inl(smem_u32(&sm->rows_ok[nr % kRowSlots]), (nr / kRowSlots) & 1,
                                  smem_u32(&sm->full[at.st]), at.ph);
        tc_fence_after();
        if (elect_lane()) {
          product_rows<DP>(u_s + (SB == 2 ? (nr & 1) * 128 : 0), k_at, row_lo + at.st * T16, hi, id_s, ksteps);
          tc_commit(smem_u32(&sm->s_full[SB == 2 ? nr & 1 : 0]));
        }
        __syncwarp();
        ++nr;
      };
      auto dp = [&](const RingPos<S>& at) {
        ok = ok && mbar_wait_inl(smem_u32(&sm->full[at.st + 1]), at.ph);
        tc_fence_after();
        if (elect_lane()) {
          product_rows<DP>(u_dp, v_at, row_lo + (at.st + 1) * T16, hi, id_s, ksteps);
          tc_commit(smem_u32(&sm->dp_full));
        }
        __syncwarp();
      };
      scores(cur);
      dp(cur);
      if (SB == 2 && n > 1) scores(cur.at(2));
#pragma unroll 1
      for (int i = 0; i < n && ok; ++i, ++np) {
        const uint32_t sb = SB == 2 ? np & 1 : 0;
        ok = ok && mbar_wait_inl(smem_u32(&sm->p_ready[sb]), (SB == 2 ? np >> 1 : np) & 1);
        tc_fence_after();
        const uint32_t p_at = u_s + sb * 128;
        if (elect_lane()) product_cols<0, 8, true>(u_dv, p_at, rowt_lo + (cur.st + 1) * T16, rowt_hi, id_a, i > 0);
        __syncwarp();
        const RingPos<S> nxt = cur.at(2);
        if (SB == 1 && i + 1 < n) scores(nxt);
        ok = ok && mbar_wait_inl(smem_u32(&sm->ds_ready), np & 1);
        tc_fence_after();
        if (elect_lane()) {
          product_cols<0, 8, true>(u_dk, u_dp, rowt_lo + cur.st * T16, rowt_hi, id_a, i > 0);
          tc_commit(smem_u32(&sm->empty[cur.st]));
          tc_commit(smem_u32(&sm->empty[cur.st + 1]));
          if (i + 1 == n) {
            tc_commit(smem_u32(&sm->kv_empty[b]));
            tc_commit(smem_u32(&sm->acc_full));
          }
        }
        __syncwarp();
        if (i + 1 < n) dp(nxt);
        if (SB == 2 && i + 2 < n) scores(cur.at(4));
        cur = nxt;
        ok = __all_sync(0xffffffffu, ok);
      }
      if (!ok) {
        sm->abort = 1;
        break;
      }
    }
    if (elect_lane()) tc_commit(smem_u32(&sm->drained));
    __syncwarp();
    if (!mbar_wait_inl(smem_u32(&sm->drained), 0)) sm->abort = 1;
    __syncwarp();
  } else if (warp == 18) {
    regs_drop<kKvSideRegs>();
    if (lane == 0) hand_out(&sm->slots, p.counter, p.items, units, p.heads_kv, abort_flag);
    __syncwarp();
  } else if (warp == 19) {
    // ============================================== row statistics, ends
    regs_drop<kKvSideRegs>();
    // lse, delta and the causal limit of a tile's rows.  Rows past the
    // sequence's last query belong to someone else: their weight is 0 (lse =
    // +inf) and, the rows being summed over, so must be what they hold.
    // A tile's values are loaded while the one before it is written.
    ItemRing ring(&sm->slots);
    AttnItem it;
    int head;
    uint32_t nr = 0;
    RingPos<S> cur;
    int pos[4];       // this lane's rows lane + 32 u: query in the tile, place in stat
    int64_t off[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = lane + 32 * u;
      pos[u] = r / p.g;
      off[u] = static_cast<int64_t>(pos[u]) * p.heads_q + r % p.g;
    }
    while (ring.next(&it, &head, abort_flag, true)) {
      int first;
      const int n = row_tiles(p, it, &first);
      bool ok = true;
      const float up = ds_up<BF16>(p, it);
      const float2* src = p.stat + (static_cast<int64_t>(it.q_row) + first * p.pos) * p.heads_q + head * p.g;
      float2 st[4];
      auto load = [&](int i) {  // tile i's rows that belong to the sequence
        const int live = min(p.pos, it.n_pos - i * p.pos);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          st[u] = pos[u] < live ? __ldcg(src + off[u]) : make_float2(INFINITY, 0.f);
        src += static_cast<int64_t>(p.pos) * p.heads_q;
      };
      if (n > 0) load(first);
#pragma unroll 1
      for (int i = first; i < first + n && ok; ++i, ++nr, cur = cur.at(2)) {
        const uint32_t sl = nr % kRowSlots;
        ok = mbar_wait_inl(smem_u32(&sm->rows_free[sl]), ((nr / kRowSlots) & 1) ^ 1);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          sm->nlse2[sl][lane + 32 * u] = -st[u].x;
          sm->ndelta[sl][lane + 32 * u] = -st[u].y * up;
          sm->lim[sl][lane + 32 * u] = it.lim0 + i * p.pos + pos[u];
        }
        if (i + 1 < first + n) load(i + 1);
        ok = ok && mbar_wait2_inl(smem_u32(&sm->full[cur.st]), cur.ph, smem_u32(&sm->full[cur.st + 1]), cur.ph);
        ok = __all_sync(0xffffffffu, ok);
        const int live = min(p.pos, it.n_pos - i * p.pos) * p.g;
        if (live < used) [[unlikely]] {
          for (int w = 0; w < 2; ++w)
            for (int c = 0; c < PANELS; ++c) {
              uint8_t* tile = smem + (2 * KVB + cur.st + w) * TILE + c * PANEL;
              for (int j = live * 8 + lane; j < used * 8; j += 32)
                *reinterpret_cast<uint4*>(tile + j * 16) = make_uint4(0, 0, 0, 0);
            }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm->rows_ok[sl]));
      }
      if (!ok) {
        sm->abort = 1;
        break;
      }
    }
    __syncwarp();
  } else {
    // ================================================ weights and dS
    regs_raise<kKvMainRegs>();
    // A key a lane; four warps share 32 keys, 32 rows (columns) each.  Sixteen
    // warps and not eight, because the steps (reads, exponentials, conversions,
    // barriers) are chains of latencies.
    const int quarter = warp >> 2;
    const int key_lane = threadIdx.x & 127;
    const uint32_t lane_off = static_cast<uint32_t>(warp & 3) << 21;
    const uint32_t ts = t_s + lane_off + quarter * 32, tdp = t_dp + lane_off + quarter * 32;
    const uint64_t sl2 = pair2(p.scale_log2, p.scale_log2);
    ItemRing ring(&sm->slots);
    AttnItem it;
    int head;
    uint32_t np = 0, nr = 0, na = 0;
    while (ring.next(&it, &head, abort_flag, true)) {
      int first;
      const int n = row_tiles(p, it, &first);
      const int key = it.kt0 * kKeyTile + key_lane;
      const float up = ds_up<BF16>(p, it);
      const uint64_t down = pair2(kPDown<BF16> * up, kPDown<BF16> * up);
      bool ok = true;
#pragma unroll 1
      for (int i = first; i < first + n && ok; ++i, ++np, ++nr) {
        const uint32_t sl = nr % kRowSlots;
        const uint32_t sb = SB == 2 ? np & 1 : 0;
        ok = mbar_wait2_inl(smem_u32(&sm->rows_ok[sl]), (nr / kRowSlots) & 1, smem_u32(&sm->s_full[sb]),
                            (SB == 2 ? np >> 1 : np) & 1);
        tc_fence_after();
        uint32_t x[32], y[32], w[16];
        tmem_ld32_raw(ts + sb * 128, x);
        const ulonglong2* l4 = reinterpret_cast<const ulonglong2*>(sm->nlse2[sl] + quarter * 32);
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          const ulonglong2 l = l4[c / 4];
          float e[4];
          unpair2(fma2(pair2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), sl2, l.x), e[0], e[1]);
          unpair2(fma2(pair2(__uint_as_float(x[c + 2]), __uint_as_float(x[c + 3])), sl2, l.y), e[2], e[3]);
#pragma unroll
          for (int u = 0; u < 4; ++u) x[c + u] = __float_as_uint(ex2(e[u]));
        }
        if (p.causal && it.kt0 * kKeyTile + kKeyTile - 1 > it.lim0 + i * p.pos) [[unlikely]] {
          const int4* m4 = reinterpret_cast<const int4*>(sm->lim[sl] + quarter * 32);
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const int4 m = m4[c / 4];
            if (key > m.x) x[c] = 0u;
            if (key > m.y) x[c + 1] = 0u;
            if (key > m.z) x[c + 2] = 0u;
            if (key > m.w) x[c + 3] = 0u;
          }
        }
#pragma unroll
        for (int c = 0; c < 16; ++c)
          w[c] = pack_pair<BF16>(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1]));
        tmem_st16(ts + sb * 128, w);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm->p_ready[sb]));
        ok = ok && mbar_wait_inl(smem_u32(&sm->dp_full), np & 1);
        tc_fence_after();
        tmem_ld32_raw(tdp, y);
        const ulonglong2* d4 = reinterpret_cast<const ulonglong2*>(sm->ndelta[sl] + quarter * 32);
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          const ulonglong2 dl = d4[c / 4];
          float e[4];
          unpair2(mul2(pair2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])),
                       fma2(pair2(__uint_as_float(y[c]), __uint_as_float(y[c + 1])), down, dl.x)),
                  e[0], e[1]);
          unpair2(mul2(pair2(__uint_as_float(x[c + 2]), __uint_as_float(x[c + 3])),
                       fma2(pair2(__uint_as_float(y[c + 2]), __uint_as_float(y[c + 3])), down, dl.y)),
                  e[2], e[3]);
          w[c / 2] = pack_pair<BF16>(e[0], e[1]);
          w[c / 2 + 1] = pack_pair<BF16>(e[2], e[3]);
        }
        tmem_st16(tdp, w);
        tmem_wait_st();
        tc_fence_before();
        ok = __all_sync(0xffffffffu, ok);
        if (lane == 0) {
          mbar_arrive(smem_u32(&sm->ds_ready));
          mbar_arrive(smem_u32(&sm->rows_free[sl]));
        }
      }
      if (n > 0 && ok) {
        ok = __all_sync(0xffffffffu, mbar_wait_inl(smem_u32(&sm->acc_full), na & 1));
        ++na;
        tc_fence_after();
      }
      if (!ok) {
        sm->abort = 1;
        break;
      }
      // quarters 0 and 1 write the halves of gv's columns, 2 and 3 gk's
      const bool live = key < it.lk;
      const bool is_k = quarter >= 2;
      const uint32_t acc = (is_k ? t_dk : t_dv) + lane_off;
      const int split = (p.d / 2 + 15) & ~15;
      const int c0 = quarter & 1 ? split : 0, c1 = quarter & 1 ? p.d : min(split, p.d);
      if (it.slot < 0) {
        const int64_t row = static_cast<int64_t>(it.k_row) + key;
        uint8_t* dst = is_k ? p.o0 + row * p.o0_t + head * p.o0_h : p.o1 + row * p.o1_t + head * p.o1_h;
        if (c1 > c0)
          store_acc<BF16>(acc + c0, dst + c0 * 2, c1 - c0, is_k ? p.scale * ds_down(up) : kPDown<BF16>, n > 0, live);
      } else {
        float* dst = p.part + (((static_cast<int64_t>(it.slot + it.split) * p.heads_kv + head) * 2 + is_k) * 128 +
                               key_lane) * p.d;
#pragma unroll 1
        for (int c = c0; c < c1; c += 16) {
          uint32_t o[16] = {};
          if (n > 0) tmem_ld16_raw(acc + c, o);
          if (!BF16 && is_k)
#pragma unroll
            for (int u = 0; u < 16; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * ds_down(up));
#pragma unroll
          for (int u = 0; u < 16; u += 4)
            if (live && c + u < p.d) *reinterpret_cast<uint4*>(dst + c + u) = make_uint4(o[u], o[u + 1], o[u + 2], o[u + 3]);
        }
      }
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 17) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && *abort_flag) atomicOr(p.status, kDevErrTimeout);
}

// ------------------------------------------------------------------- gq --
struct QSmem {
  uint64_t full[kBwdMaxStages], empty[kBwdMaxStages];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], dp_full, ds_ready, acc_full;
  uint64_t fix_k, k_fixed;
  uint64_t drained;
  uint32_t tmem;
  int abort;
  int fix_at, fix_rows;  // ring stage of a K tile that ends inside, and its keys
  ItemSlots slots;
};

template <bool BF16, int DP>
__global__ void __launch_bounds__(kBwdThreads, 1)
    k_attn_bwd_q(const BwdParams p, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap gmap,
                 const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  constexpr int PANELS = DP / 64;
  constexpr uint32_t PANEL = 128 * 128, TILE = PANELS * PANEL;
  constexpr uint32_t S = q_stages(DP);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sq = smem_u32(smem);        // Q and gout
  constexpr int QB = q_pairs(DP);
  const uint32_t skv = sq + 2 * QB * TILE;   // ring: K, V, K, V, ...
  QSmem* sm = reinterpret_cast<QSmem*>(smem + (2 * QB + S) * TILE);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &sm->abort;

  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < S; ++s) {
      mbar_init(smem_u32(&sm->full[s]), 1);
      mbar_init(smem_u32(&sm->empty[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&sm->q_full[s]), 1);
      mbar_init(smem_u32(&sm->q_empty[s]), 1);
      mbar_init(smem_u32(&sm->s_full[s]), 1);
    }
    mbar_init(smem_u32(&sm->dp_full), 1);
    mbar_init(smem_u32(&sm->ds_ready), 16);
    mbar_init(smem_u32(&sm->acc_full), 1);
    mbar_init(smem_u32(&sm->fix_k), 1);
    mbar_init(smem_u32(&sm->k_fixed), 1);
    mbar_init(smem_u32(&sm->drained), 1);
    sm->slots.init(19);  // 16 warps for the weights, loads, products, ends
    sm->abort = 0;
    fence_mbar_init();
  }
  if (warp == 17) {
    tmem_alloc(smem_u32(&sm->tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (p.first) grid_wait();  // the plan and the statistics; else gk's kernel has waited for them
  const uint32_t tmem = sm->tmem;
  const uint32_t t_s = tmem, t_dp = tmem + 256, t_dq = tmem + 384;
  const int units = __ldcg(p.header) * p.heads_kv;

  if (warp == 16) {
    // =========================================================== loads
    if (lane == 0) {
      ItemRing ring(&sm->slots);
      AttnItem it;
      int head;
      uint32_t k = 0, nq = 0;
      RingPos<S> r;
      while (ring.next(&it, &head, abort_flag, false)) {
        if (it.kt1 == 0) continue;
        const uint32_t b = nq % QB;
        if (!mbar_wait_inl(smem_u32(&sm->q_empty[b]), ((nq / QB) & 1) ^ 1)) {
          sm->abort = 1;
          break;
        }
        ++nq;
        mbar_arrive_expect_tx(smem_u32(&sm->q_full[b]), 2 * PANELS * p.pos * p.g * 128);
        for (int c = 0; c < PANELS; ++c) {
          tma_load_3d(sq + 2 * b * TILE + c * PANEL, &qmap, c * 64, head * p.g, it.q_row, smem_u32(&sm->q_full[b]));
          tma_load_3d(sq + (2 * b + 1) * TILE + c * PANEL, &gmap, c * 64, head * p.g, it.q_row,
                      smem_u32(&sm->q_full[b]));
        }
        bool ok = true;
        for (int j = 0; j < it.kt1 && ok; ++j)
          for (int kv = 0; kv < 2; ++kv, ++k, r.step()) {
            const uint32_t st = r.st;
            if (!mbar_wait_inl(smem_u32(&sm->empty[st]), r.ph ^ 1)) {
              sm->abort = 1;
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(smem_u32(&sm->full[st]), TILE);
            for (int c = 0; c < PANELS; ++c)
              tma_load_3d(skv + st * TILE + c * PANEL, kv ? &vmap : &kmap, c * 64, head, it.k_row + j * kKeyTile,
                          smem_u32(&sm->full[st]));
          }
        if (!ok) break;
      }
      const uint32_t f0 = nq > QB ? nq - QB : 0;
      for (uint32_t i = f0; i < nq; ++i)
        if (!mbar_wait_inl(smem_u32(&sm->q_full[i % QB]), (i / QB) & 1)) sm->abort = 1;
      const uint32_t f1 = k > S ? k - S : 0;
      for (uint32_t i = f1; i < k; ++i)
        if (!mbar_wait_inl(smem_u32(&sm->full[i % S]), (i / S) & 1)) sm->abort = 1;
    }
    __syncwarp();
  } else if (warp == 17) {
    // ======================================================== products
    const int dn = (p.d + 15) & ~15;
    const int ksteps = dn / 16;
    const uint32_t id_s = make_idesc(BF16, 128, 128);
    const uint32_t id_a = make_idesc(BF16, 128, dn) | (1u << 16);
    const uint64_t dk = smem_desc(skv, 1024, 2), dt = smem_desc_mn(skv, PANEL, 1024, 2);
    const uint32_t kv_lo = static_cast<uint32_t>(dk), hi = static_cast<uint32_t>(dk >> 32);
    const uint32_t q_lo = static_cast<uint32_t>(smem_desc(sq, 1024, 2));
    const uint32_t kt_lo = static_cast<uint32_t>(dt), kt_hi = static_cast<uint32_t>(dt >> 32);
    constexpr uint32_t T16 = TILE >> 4;
    const uint32_t tb = of_warp(tmem);
    const uint32_t u_s = tb, u_dp = tb + 256, u_dq = tb + 384;
    ItemRing ring(&sm->slots);
    AttnItem it;
    int head;
    uint32_t nq = 0, nd = 0, nfix = 0, nbuf = 0;
    RingPos<S> rd;  // K of the tile in hand; its V is the next stage
    while (ring.next(&it, &head, abort_flag, true)) {
      const int n = of_warp(it.kt1), lk = of_warp(it.lk);
      if (n == 0) continue;
      const uint32_t qb = nq % QB, q_at = q_lo + 2 * qb * T16;
      bool ok = mbar_wait_inl(smem_u32(&sm->q_full[qb]), (nq / QB) & 1);
      ++nq;
      // S of key tile j into its buffer; the tile's rows past the keys are zeroed first
      auto scores = [&](int j, const RingPos<S>& at) {
        ok = ok && mbar_wait_inl(smem_u32(&sm->full[at.st]), at.ph);
        if (lk - j * kKeyTile < kKeyTile) {
          if (lane == 0) {
            sm->fix_at = static_cast<int>(at.st);
            sm->fix_rows = lk - j * kKeyTile;
            mbar_arrive(smem_u32(&sm->fix_k));
          }
          ok = ok && mbar_wait_inl(smem_u32(&sm->k_fixed), nfix & 1);
          ++nfix;
        }
        tc_fence_after();
        if (elect_lane()) {
          product_rows<DP>(u_s + (nbuf & 1) * 128, q_at, kv_lo + at.st * T16, hi, id_s, ksteps);
          tc_commit(smem_u32(&sm->s_full[nbuf & 1]));
        }
        __syncwarp();
        ++nbuf;
      };
      // dP of the tile whose V lies at `at`, which is then done with
      auto dp = [&](const RingPos<S>& at) {
        ok = ok && mbar_wait_inl(smem_u32(&sm->full[at.st]), at.ph);
        tc_fence_after();
        if (elect_lane()) {
          product_rows<DP>(u_dp, q_at + T16, kv_lo + at.st * T16, hi, id_s, ksteps);
          tc_commit(smem_u32(&sm->dp_full));
          tc_commit(smem_u32(&sm->empty[at.st]));
        }
        __syncwarp();
      };
      scores(0, rd);
      dp(rd.at(1));
      if (n > 1) scores(1, rd.at(2));
#pragma unroll 1
      for (int j = 0; j < n && ok; ++j, ++nd) {
        ok = ok && mbar_wait_inl(smem_u32(&sm->ds_ready), nd & 1);
        // dS lies over its S, so dP of the next tile comes first: it is waited for
        if (j + 1 < n) dp(rd.at(3));
        tc_fence_after();
        if (elect_lane()) {
          product_cols<0, 8, true>(u_dq, u_s + (nd & 1) * 128, kt_lo + rd.st * T16, kt_hi, id_a, j > 0);
          tc_commit(smem_u32(&sm->empty[rd.st]));
          if (j + 1 == n) {
            tc_commit(smem_u32(&sm->q_empty[qb]));
            tc_commit(smem_u32(&sm->acc_full));
          }
        }
        __syncwarp();
        if (j + 2 < n) scores(j + 2, rd.at(4));
        rd = rd.at(2);
        ok = __all_sync(0xffffffffu, ok);
      }
      if (!ok) {
        sm->abort = 1;
        break;
      }
    }
    if (elect_lane()) tc_commit(smem_u32(&sm->drained));
    __syncwarp();
    if (!mbar_wait_inl(smem_u32(&sm->drained), 0)) sm->abort = 1;
    __syncwarp();
  } else if (warp == 18) {
    if (lane == 0) hand_out(&sm->slots, p.counter, p.items, units, p.heads_kv, abort_flag);
    __syncwarp();
  } else if (warp == 19) {
    // ==================================================== tail of K
    ItemRing ring(&sm->slots);
    AttnItem it;
    int head;
    uint32_t n = 0;
    while (ring.next(&it, &head, abort_flag, true)) {
      if (it.kt1 == 0 || it.lk - (it.kt1 - 1) * kKeyTile >= kKeyTile) continue;
      if (!__all_sync(0xffffffffu, mbar_wait_unit(smem_u32(&sm->fix_k), n & 1, abort_flag))) {
        sm->abort = 1;
        break;
      }
      ++n;
      const int rows = sm->fix_rows;
      uint8_t* tile = smem + (2 * QB + sm->fix_at) * TILE;
      for (int c = 0; c < PANELS; ++c)
        for (int i = rows * 8 + lane; i < kKeyTile * 8; i += 32)
          *reinterpret_cast<uint4*>(tile + c * PANEL + i * 16) = make_uint4(0, 0, 0, 0);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm->k_fixed));
    }
    __syncwarp();
  } else {
    // ========================================================= dS
    // A row a lane; four warps share 32 rows, 32 keys (columns) of a tile each.
    const int quarter = warp >> 2;
    const int row = threadIdx.x & 127;
    const uint32_t lane_off = static_cast<uint32_t>(warp & 3) << 21;
    const uint32_t tdp = t_dp + lane_off + quarter * 32;
    const int pos = row / p.g, gh = row - pos * p.g;
    const uint64_t sl2 = pair2(p.scale_log2, p.scale_log2);
    ItemRing ring(&sm->slots);
    AttnItem it;
    int head;
    uint32_t nd = 0, na = 0;
    while (ring.next(&it, &head, abort_flag, true)) {
      const int n = it.kt1;
      const bool live = pos < p.pos && pos < it.n_pos;
      const int64_t tok = static_cast<int64_t>(it.q_row) + pos;
      const int h = head * p.g + gh;
      const int vis = p.causal ? min(it.lk, it.lim0 + pos + 1) : it.lk;
      float2 st = make_float2(INFINITY, 0.f);
      if (live) st = __ldcg(p.stat + tok * p.heads_q + h);
      const float up = ds_up<BF16>(p, it);
      const uint64_t nl = pair2(-st.x, -st.x), ndl = pair2(-st.y * up, -st.y * up);
      const uint64_t down = pair2(kPDown<BF16> * up, kPDown<BF16> * up);
      bool ok = true;
#pragma unroll 1
      for (int j = 0; j < n && ok; ++j, ++nd) {
        const uint32_t b = nd & 1;
        ok = mbar_wait_inl(smem_u32(&sm->s_full[b]), (nd >> 1) & 1);
        tc_fence_after();
        uint32_t x[32], y[32], w[16];
        tmem_ld32_raw(t_s + b * 128 + lane_off + quarter * 32, x);
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          float e0, e1;
          unpair2(fma2(pair2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), sl2, nl), e0, e1);
          x[c] = __float_as_uint(ex2(e0));
          x[c + 1] = __float_as_uint(ex2(e1));
        }
        ok = ok && mbar_wait_inl(smem_u32(&sm->dp_full), nd & 1);
        tc_fence_after();
        tmem_ld32_raw(tdp, y);
        const int seen = vis - j * kKeyTile - quarter * 32;
        if (__any_sync(0xffffffffu, seen < 32)) [[unlikely]] {  // both to zero: V may hold anything there
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (c >= seen) x[c] = y[c] = 0u;
        }
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          float e0, e1;
          unpair2(mul2(pair2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])),
                       fma2(pair2(__uint_as_float(y[c]), __uint_as_float(y[c + 1])), down, ndl)),
                  e0, e1);
          w[c / 2] = pack_pair<BF16>(e0, e1);
        }
        tmem_st16(t_s + b * 128 + lane_off + quarter * 32, w);
        tmem_wait_st();
        tc_fence_before();
        ok = __all_sync(0xffffffffu, ok);
        if (lane == 0) mbar_arrive(smem_u32(&sm->ds_ready));
      }
      if (n > 0 && ok) {
        ok = __all_sync(0xffffffffu, mbar_wait_inl(smem_u32(&sm->acc_full), na & 1));
        ++na;
        tc_fence_after();
      }
      if (!ok) {
        sm->abort = 1;
        break;
      }
      // each quarter writes its columns, 16 at a time
#pragma unroll 1
      for (int c = quarter * 16; c < p.d; c += 64)
        store_acc<BF16>(t_dq + lane_off + c, p.o0 + tok * p.o0_t + h * p.o0_h + c * 2, min(16, p.d - c),
                        p.scale * ds_down(up), n > 0, live);
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 17) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  grid_wait();  // done only when gk's kernel is
  if (threadIdx.x == 0 && *abort_flag) atomicOr(p.status, kDevErrTimeout);
}

// gk and gv of the key tiles whose rows were cut: the parts' sums in order, a
// row a warp, four values a lane.  Memory bounds it; 12 us for the five documents.
template <bool BF16>
__global__ void __launch_bounds__(256) k_attn_bwd_join(const BwdParams p, const AttnItem* joins) {
  grid_wait();
  const int n = __ldcg(p.header + 2) * p.heads_kv * 32;  // eight rows of one of the two a block
  const int c = (threadIdx.x & 31) * 4;
  const int64_t step = static_cast<int64_t>(p.heads_kv) * 256 * p.d;
  for (int u = blockIdx.x; u < n; u += gridDim.x) {
    const int jh = u >> 5, row = (u & 15) * 8 + (threadIdx.x >> 5), is_k = (u >> 4) & 1;
    const int j = jh / p.heads_kv, head = jh - j * p.heads_kv;
    const AttnItem* it = joins + j;
    const int key = it->kt0 * kKeyTile + row, parts = it->nsplit;
    if (key >= it->lk || c >= p.d) continue;
    const float* src = p.part + (((static_cast<int64_t>(it->slot) * p.heads_kv + head) * 2 + is_k) * 128 + row) * p.d + c;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int q = 0; q < parts; ++q) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(src + q * step));
      a.x += v.x;
      a.y += v.y;
      a.z += v.z;
      a.w += v.w;
    }
    const float f = is_k ? p.scale : kPDown<BF16>;
    const int64_t t = static_cast<int64_t>(it->k_row) + key;
    uint8_t* dst = is_k ? p.o0 + t * p.o0_t + head * p.o0_h : p.o1 + t * p.o1_t + head * p.o1_h;
    *reinterpret_cast<uint2*>(dst + c * 2) =
        make_uint2(pack_pair<BF16>(a.x * f, a.y * f), pack_pair<BF16>(a.z * f, a.w * f));
  }
}

template <bool BF16>
const void* kv_kernel(int dp) {
  return dp == 64 ? reinterpret_cast<const void*>(k_attn_bwd_kv<BF16, 64>)
                  : reinterpret_cast<const void*>(k_attn_bwd_kv<BF16, 128>);
}
template <bool BF16>
const void* q_kernel(int dp) {
  return dp == 64 ? reinterpret_cast<const void*>(k_attn_bwd_q<BF16, 64>)
                  : reinterpret_cast<const void*>(k_attn_bwd_q<BF16, 128>);
}

template <bool BF16>
void run_stat(StatParams p, cudaStream_t s) {
  const int lpr = p.d <= 16 ? 2 : p.d <= 32 ? 4 : p.d <= 64 ? 8 : 16;
  const int64_t rows = p.rows + p.v_rows, per_run = 8 * 32 / lpr;  // a block's
  const int64_t resident = static_cast<int64_t>(kStatBlocks) * device_sm_count();
  p.runs = static_cast<int>((rows + per_run * resident - 1) / (per_run * resident));
  p.runs = (p.runs + kStatBatch - 1) / kStatBatch * kStatBatch;
  const int64_t per_block = per_run * p.runs;
  p.blocks = static_cast<unsigned>((p.rows + per_block - 1) / per_block);
  const unsigned n = p.blocks + static_cast<unsigned>((p.v_rows + per_block - 1) / per_block);
  switch (lpr) {
    case 2: k_attn_stat<BF16, 2><<<n, 256, 0, s>>>(p); break;
    case 4: k_attn_stat<BF16, 4><<<n, 256, 0, s>>>(p); break;
    case 8: k_attn_stat<BF16, 8><<<n, 256, 0, s>>>(p); break;
    default: k_attn_stat<BF16, 16><<<n, 256, 0, s>>>(p); break;
  }
}

}  // namespace

sc_status attn_bwd(const AttnArgs& a) {
  const int g = a.heads_q / a.heads_kv, pos = 128 / g;
  const int sms = device_sm_count();
  const bool bf = a.dtype == SC_BF16;
  const int64_t q_items = a.t_q / pos + a.n_seq, k_items = a.t_k / kKeyTile + a.n_seq;
  if (q_items * a.heads_kv > 0x3fffffff || k_items * a.heads_kv > 0x3fffffff ||
      a.t_q * a.heads_q > (int64_t(1) << 34))
    return set_error(SC_ERR_UNSUPPORTED, "too many tiles");
  Arena ar;
  const size_t o_hq = ar.take(kPlanHeader * sizeof(int)), o_hk = ar.take(kPlanHeader * sizeof(int));
  const size_t o_iq = ar.take(static_cast<size_t>(q_items) * sizeof(AttnItem));
  // Partial gk and gv: room for two an SM where the key tiles are few (the plan
  // cuts those that are dearer than an SM's share) and a sequence may have more
  // rows than a part.
  const bool cut = k_items * a.heads_kv <= 8ll * sms && a.t_q > static_cast<int64_t>(kMinPartTiles) * pos;
  const int64_t slots = cut ? 2ll * sms / a.heads_kv + 2 : 0;
  const int64_t k_cap = k_items + slots;
  const size_t o_ik = ar.take(static_cast<size_t>(k_cap) * sizeof(AttnItem));
  const size_t o_st = ar.take(static_cast<size_t>(a.t_q) * a.heads_q * sizeof(float2));
  const size_t o_peak = ar.take(bf ? 0 : static_cast<size_t>(a.n_seq) * 2 * sizeof(float));
  const size_t o_joins = ar.take(cut ? static_cast<size_t>(k_items) * sizeof(AttnItem) : 0);
  const size_t o_part = ar.take(static_cast<size_t>(slots) * a.heads_kv * 256 * a.head_dim * sizeof(float));
  int* status = attn_status_word();
  if (!status) return set_error(SC_ERR_CUDA, "the attention status word is not available");
  const int dp = a.head_dim <= 64 ? 64 : 128;
  const size_t tile = static_cast<size_t>(dp) / 64 * 16384;
  const void* kk = bf ? kv_kernel<true>(dp) : kv_kernel<false>(dp);
  const void* kq = bf ? q_kernel<true>(dp) : q_kernel<false>(dp);
  const size_t kv_smem = (2 * kv_pairs(dp) + kv_stages(dp)) * tile + sizeof(KvSmem) + 1024;
  const size_t q_smem = (2 * q_pairs(dp) + q_stages(dp)) * tile + sizeof(QSmem) + 1024;
  int regs = 0;
  sc_status st = kernel_setup(kk, kv_smem, &regs);
  if (!st && regs != kKvRegs) st = set_error(SC_ERR_CUDA, "attention kernel: not the registers it was written for");
  if (!st) st = kernel_setup(kq, q_smem, nullptr);
  if (st) return st;
  const bool have_q = a.t_q > 0, have_k = a.t_k > 0;
  const void* any = have_q ? a.q.data : a.k.data;  // a side without rows: maps of legal sizes that nothing reads
  CUtensorMap qm, gm, km, vm;
  const int hq = have_q ? a.heads_q : 1, hk = have_k ? a.heads_kv : 1;
  const int64_t tq = have_q ? a.t_q : 1, tk = have_k ? a.t_k : 1;
  const auto map_of = [&](CUtensorMap* m, const sc_heads& v, bool have, int heads, int64_t tokens, int bh, int bt) {
    return attn_map(m, have ? v.data : any, a.dtype, a.head_dim, heads, tokens, v.token_stride, v.head_stride, bh, bt);
  };
  if ((st = map_of(&qm, a.q, have_q, hq, tq, g, pos)) || (st = map_of(&gm, a.gout, have_q, hq, tq, g, pos)) ||
      (st = map_of(&km, a.k, have_k, hk, tk, 1, kKeyTile)) || (st = map_of(&vm, a.v, have_k, hk, tk, 1, kKeyTile)))
    return st;
  void* ws = nullptr;
  if ((st = dev_alloc(&ws, ar.bytes, a.stream))) return st;
  uint8_t* base = static_cast<uint8_t*>(ws);
  PlanArgs pl{};
  pl.q_off = a.q_off;
  pl.k_off = a.k_off;
  pl.n_seq = static_cast<int>(a.n_seq);
  pl.t_q = a.t_q;
  pl.t_k = a.t_k;
  pl.pos_per_item = pos;
  pl.g = g;
  pl.sms = sms;
  pl.causal = a.causal;
  pl.packed_keys = 1;
  pl.heads_kv = a.heads_kv;
  pl.status = status;
  PlanArgs plq = pl, plk = pl;
  plq.mode = kPlanRows;
  plq.cap = static_cast<int>(q_items);
  plq.header = reinterpret_cast<int*>(base + o_hq);
  plq.items = reinterpret_cast<AttnItem*>(base + o_iq);
  plk.mode = kPlanKeys;
  plk.cap = static_cast<int>(k_cap);
  plk.part_rows = slots * a.heads_kv * kKeyTile;
  plk.over = 1;
  plk.min_tiles = kMinPartTiles;
  plk.join_cap = cut ? static_cast<int>(k_items) : 0;
  plk.joins = reinterpret_cast<AttnItem*>(base + o_joins);
  plk.header = reinterpret_cast<int*>(base + o_hk);
  plk.items = reinterpret_cast<AttnItem*>(base + o_ik);
  cudaError_t e = cudaSuccess;
  BwdParams p{};
  p.stat = reinterpret_cast<const float2*>(base + o_st);
  p.heads_q = a.heads_q;
  p.heads_kv = a.heads_kv;
  p.g = g;
  p.pos = pos;
  p.d = a.head_dim;
  p.scale = a.scale;
  p.scale_log2 = a.scale * kLog2e;
  p.causal = a.causal;
  p.status = status;
  if (!st && have_q) {
    StatParams sp{};
    sp.gout = static_cast<const uint8_t*>(a.gout.data);
    sp.out = static_cast<const uint8_t*>(a.out_in.data);
    sp.gt = a.gout.token_stride * 2;
    sp.gh = a.gout.head_stride * 2;
    sp.ot = a.out_in.token_stride * 2;
    sp.oh = a.out_in.head_stride * 2;
    sp.lse = a.lse;
    sp.stat = reinterpret_cast<float2*>(base + o_st);
    sp.rows = a.t_q * a.heads_q;
    sp.heads_q = a.heads_q;
    sp.heads_kv = a.heads_kv;
    sp.d = a.head_dim;
    if (!bf) {
      sp.v = static_cast<const uint8_t*>(a.v.data);
      sp.vt = a.v.token_stride * 2;
      sp.vh = a.v.head_stride * 2;
      sp.v_rows = a.t_k * a.heads_kv;
      sp.q_off = a.q_off;
      sp.k_off = a.k_off;
      sp.n_seq = static_cast<int>(a.n_seq);
      sp.peak = reinterpret_cast<float*>(base + o_peak);
      p.peak = sp.peak;
      e = cudaMemsetAsync(sp.peak, 0, static_cast<size_t>(a.n_seq) * 2 * sizeof(float), a.stream);
      if (e != cudaSuccess) st = set_cuda_error(e, "attention peaks");
    }
    if (!st) SC_LAUNCH("attn_stat", a.stream, (bf ? run_stat<true>(sp, a.stream) : run_stat<false>(sp, a.stream)));
    e = cudaGetLastError();
    if (e != cudaSuccess) st = set_cuda_error(e, "attn_stat");
  }
  if (!st) st = attn_plan(plk, &plq, have_q, a.stream);
  BwdParams joined = p;
  if (!st && have_k) {
    BwdParams pk = p;
    pk.header = plk.header;
    pk.counter = plk.header + 1;
    pk.items = plk.items;
    pk.o0 = static_cast<uint8_t*>(a.gk.data);
    pk.o0_t = a.gk.token_stride * 2;
    pk.o0_h = a.gk.head_stride * 2;
    pk.o1 = static_cast<uint8_t*>(a.gv.data);
    pk.o1_t = a.gv.token_stride * 2;
    pk.o1_h = a.gv.head_stride * 2;
    pk.part = reinterpret_cast<float*>(base + o_part);
    const int64_t most = k_cap * a.heads_kv;
    void* args[] = {&pk, &qm, &gm, &km, &vm};
    SC_LAUNCH("attn_bwd_kv", a.stream,
              (e = launch_after(kk, static_cast<unsigned>(most < sms ? most : sms), kBwdThreads, kv_smem, a.stream,
                                args)));
    if (e != cudaSuccess) st = set_cuda_error(e, "attn_bwd_kv");
    joined = pk;
  }
  if (!st && have_q) {
    BwdParams pq = p;
    pq.header = plq.header;
    pq.counter = plq.header + 1;
    pq.items = plq.items;
    pq.o0 = static_cast<uint8_t*>(a.gq.data);
    pq.o0_t = a.gq.token_stride * 2;
    pq.o0_h = a.gq.head_stride * 2;
    pq.first = !have_k;
    const int64_t most = q_items * a.heads_kv;
    void* args[] = {&pq, &qm, &gm, &km, &vm};
    SC_LAUNCH("attn_bwd_q", a.stream,
              (e = launch_after(kq, static_cast<unsigned>(most < sms ? most : sms), kBwdThreads, q_smem, a.stream,
                                args)));
    if (e != cudaSuccess) st = set_cuda_error(e, "attn_bwd_q");
  }
  if (!st && have_k && cut) {  // after gq's kernel, which outlasts gk's
    const AttnItem* joins = plk.joins;
    void* args[] = {&joined, &joins};
    const void* kj = bf ? reinterpret_cast<const void*>(k_attn_bwd_join<true>)
                        : reinterpret_cast<const void*>(k_attn_bwd_join<false>);
    SC_LAUNCH("attn_bwd_join", a.stream, (e = launch_after(kj, 4 * sms, 256, 0, a.stream, args)));
    if (e != cudaSuccess) st = set_cuda_error(e, "attn_bwd_join");
  }
  dev_free(ws, a.stream);
  return st;
}

}  // namespace sc
