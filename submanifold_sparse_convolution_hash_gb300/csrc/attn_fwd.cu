// Attention forward over packed sequences.
//
// A block takes one item (up to 2 P queries of a sequence, a key head, a run of
// 128-key tiles) at a time.  Its queries are two tiles of 128 packed rows.  Per
// key tile and row tile
//   S = Q K^T                        tensor cores, 128 x 128 in TMEM
//   m' = max(m, max S), P = exp2((S - m') scale log2 e), l = l 2^(..) + sum P
//   O = O 2^((m - m') ..) + P V      P back in TMEM as the first operand
// so the scores never leave the SM.  One warp loads by TMA; each row tile has a
// warp that issues its products and four for the exponentials, a row a thread;
// while one tile's exponentials run, the other tile's products do.  O is
// corrected only when a row's maximum grew by more than 2^8: until then P is up
// to 256 instead of 1, which costs no bits in floating point.  P is rounded to 16
// bits as the operand of the second product; S, O, m and l are fp32.  f16 has few
// bits below 2^-14 and none below 2^-24, where the weights of a long list under one
// dominant key lie: there P is held times 2^7 (at most 2^15), so that a weight is
// off by its rounding or by 2^-32 of the largest, whichever is more.
//
// What bounds it, with kernel times.  Long lists at 128 values: the tensor cores
// and the chain S, maximum, exponentials, P, O of the two row tiles that share
// them (16384 tokens, causal, 32 query and 8 key heads, bf16: 1299 us, 1.69
// PFLOP/s of the 1.97 that a library product reaches).  Heads of 32 or 64 values
// have the same exponentials for a half or a quarter of the products, and that
// chain bounds them (160 windows of 500 to 1000 voxels, 4 heads of 64, f16: 161
// us).  Few queries: memory (64 sequences, one query each, up to 16384 keys, 8 key
// heads of 128: 316 us, 6.9 TB/s).
//
// Measured and left out: sixteen warps for the exponentials, two a row with their
// maxima exchanged; two blocks an SM with 64-key tiles (191 us instead of 167 for
// the windows).
#include "attn_device.cuh"

namespace sc {
namespace {

constexpr int kFwdThreads = 384;
constexpr int kFwdMaxStages = 10;
constexpr int kMinPartTiles = 4;  // least key tiles of a part
constexpr float kLn2 = 0.6931471805599453f;
// K and V tiles in flight: 160 KB of them beside the two Q tiles.
constexpr int fwd_stages(int dp) { return dp == 64 ? 10 : 5; }
// Registers a thread: the block is launched with kFwdRegs for all, four warps
// drop to the lesser share and eight raise to the greater.
constexpr int kFwdRegs = 168, kFwdSideRegs = 72, kFwdMainRegs = 216;
static_assert(128 * kFwdSideRegs + 256 * kFwdMainRegs <= kFwdThreads * kFwdRegs, "no more than the block has");

struct FwdParams {
  uint8_t* out;
  int64_t out_t, out_h;  // bytes
  float* lse;            // [t_q, heads_q] or null
  const int* header;
  int* counter;          // next unit
  const AttnItem* items;
  float* part;           // partial results [slot][head][header[3] rows][d + 8]: O, m, l
  int heads_q, heads_kv, g, pos;  // pos: queries of a row tile
  int d;
  float scale_log2;
  int causal;
  int* status;
};

struct FwdSmem {
  uint64_t full[kFwdMaxStages], empty[kFwdMaxStages];
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_ready[2][2], o_full[2];
  uint64_t v_fixed;
  ItemSlots slots;
  uint64_t drained;
  uint32_t tmem;
  int abort;
};

// P is held times 2^kShift.
template <bool BF16>
constexpr float kShift = BF16 ? 0.f : 7.f;

// What a row's exponents are taken from: m scale - kShift as it rounds (0 before
// any key), and past 2^24, where rounding takes whole powers of two, what it left.
// The factor from one such base to the next.
constexpr float kFar = 16777216.f;
template <bool BF16>
__device__ __forceinline__ float base_of(float m, float scale_log2) {
  return m == -INFINITY ? 0.f : __fmaf_rn(m, scale_log2, -kShift<BF16>);
}
template <bool BF16>
__device__ __forceinline__ float rest_of(float m, float base, float scale_log2) {
  return fabsf(base) > kFar ? fmaf(m, scale_log2, -base) - kShift<BF16> : 0.f;
}
template <bool BF16>
__device__ __forceinline__ float step_down(float m, float mn, float base, float nb, float scale_log2) {
  return ex2((base - nb) + (rest_of<BF16>(m, base, scale_log2) - rest_of<BF16>(mn, nb, scale_log2)));
}

// Key tiles that row tile s of the item has to see: [kt0, end).  In a dual item
// both halves have the one row tile, half s every other key tile from kt0 + s.
__device__ __forceinline__ int tile_end(const FwdParams& p, const AttnItem& it, int s) {
  if (it.dual) s = 0;
  const int n = min(it.n_pos - s * p.pos, p.pos);  // queries of the tile
  if (n <= 0) return it.kt0;
  const int seen = p.causal ? min(it.lk, it.lim0 + s * p.pos + n) : it.lk;
  const int end = (max(seen, 0) + kKeyTile - 1) / kKeyTile;
  return max(it.kt0, min(end, it.kt1));
}

// Zeroes the rows of a tile from `rows` on, by a warp, for the products to come.
template <int PANELS>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int rows) {
#pragma unroll 1
  for (int i = rows * 8 + static_cast<int>(threadIdx.x & 31); i < kKeyTile * 8; i += 32)
#pragma unroll
    for (int c = 0; c < PANELS; ++c) *reinterpret_cast<uint4*>(tile + c * 16384 + i * 16) = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  __syncwarp();
}

template <bool BF16, int DP, bool ONE>
__global__ void __launch_bounds__(kFwdThreads, 1)
    k_attn_fwd(const FwdParams p, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
               const __grid_constant__ CUtensorMap vmap) {
  constexpr int PANELS = DP / 64;
  constexpr uint32_t PANEL = 128 * 128;          // bytes of 128 rows x 64 values
  constexpr uint32_t TILE = PANELS * PANEL;
  constexpr uint32_t S = fwd_stages(DP);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sq = smem_u32(smem);            // two Q tiles
  const uint32_t skv = sq + 2 * TILE;            // ring of K and V tiles
  FwdSmem* sm = reinterpret_cast<FwdSmem*>(smem + (2 + S) * TILE);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &sm->abort;

  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < S; ++s) {
      mbar_init(smem_u32(&sm->full[s]), 1);
      mbar_init(smem_u32(&sm->empty[s]), ONE ? 1 : 2);
    }
    mbar_init(smem_u32(&sm->q_full), 1);
    mbar_init(smem_u32(&sm->q_empty), ONE ? 1 : 2);
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&sm->s_full[s]), 1);
      for (int h = 0; h < 2; ++h) mbar_init(smem_u32(&sm->p_ready[s][h]), 4);
      mbar_init(smem_u32(&sm->o_full[s]), 1);
    }
    mbar_init(smem_u32(&sm->v_fixed), 1);
    mbar_init(smem_u32(&sm->drained), ONE ? 1 : 2);
    sm->slots.init(ONE ? 10 : 11);  // 8 softmax warps, loads, those for products
    sm->abort = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(&sm->tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_wait();  // the plan
  grid_release();
  const uint32_t tmem = sm->tmem;
  // TMEM: S of the two row tiles, 128 columns each, P over S, O of 128 columns.
  // One row tile of up to 64 values: P has 64 columns of its own behind S and O 64,
  // so that S of the next tile need not wait for the product that reads P (four
  // scenes' 100 queries of 8 heads of 64: 199 us, 209 with P over S; with two row
  // tiles P over S is the faster form, 161 us for 164 on 160 voxel windows,
  // because the product then begins with half of the keys).
  constexpr bool EARLY = DP == 64 && ONE;
  const uint32_t t_p = EARLY ? tmem + 256 : tmem, t_o = EARLY ? tmem + 384 : tmem + 256;
  constexpr uint32_t P_COLS = EARLY ? 64 : 128, O_COLS = EARLY ? 64 : 128;
  const int n_items = __ldcg(p.header);
  const int units = n_items * p.heads_kv;

  if (warp == 8) {
    // =========================================================== loads
    regs_drop<kFwdSideRegs>();
    if (lane == 0) {
      ItemRing ring(&sm->slots);
      AttnItem it;
      int head;
      uint32_t nq = 0, loads = 0;
      RingPos<S> r;
      const uint32_t q_bytes = static_cast<uint32_t>(p.pos * p.g) * 128;
      while (ring.next(&it, &head, abort_flag, false)) {
        const int e0 = tile_end(p, it, 0), e1 = tile_end(p, it, 1);
        const int end = max(e0, e1);
        if (end <= it.kt0) continue;
        if (!mbar_wait_inl(smem_u32(&sm->q_empty), (nq & 1) ^ 1)) {
          sm->abort = 1;
          break;
        }
        ++nq;
        const bool second = e1 > it.kt0 && !it.dual;
        mbar_arrive_expect_tx(smem_u32(&sm->q_full), ((e0 > it.kt0 ? 1 : 0) + (second ? 1 : 0)) * PANELS * q_bytes);
        for (int s = 0; s < 2; ++s) {
          if (s ? !second : e0 <= it.kt0) continue;
          for (int c = 0; c < PANELS; ++c)
            tma_load_3d(sq + s * TILE + c * PANEL, &qmap, c * 64, head * p.g, it.q_row + s * p.pos,
                        smem_u32(&sm->q_full));
        }
        bool ok = true;
        // K and V by turns; a dual item's in pairs: K K V V
        const int step = it.dual ? 2 : 1;
        for (int j = it.kt0; j < end && ok; j += step)
          for (int u = 0; u < 2 * step; ++u) {
            const int kv = u >= step, tile = j + u % step;
            if (tile >= end) continue;
            if (!mbar_wait_inl(smem_u32(&sm->empty[r.st]), r.ph ^ 1)) {
              sm->abort = 1;
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(smem_u32(&sm->full[r.st]), TILE);
            for (int c = 0; c < PANELS; ++c)
              tma_load_3d(skv + r.st * TILE + c * PANEL, kv ? &vmap : &kmap, c * 64, head, it.k_row + tile * kKeyTile,
                          smem_u32(&sm->full[r.st]));
            r.step();
            ++loads;
          }
        if (!ok) break;
      }
      // every copy has landed before the block may end
      if (nq > 0 && !mbar_wait_inl(smem_u32(&sm->q_full), (nq - 1) & 1)) sm->abort = 1;
      const uint32_t first = loads > S ? loads - S : 0;
      for (uint32_t i = first; i < loads; ++i)
        if (!mbar_wait_inl(smem_u32(&sm->full[i % S]), (i / S) & 1)) sm->abort = 1;
    }
    __syncwarp();
  } else if (warp == 9 || warp == 11) {
    // ======================================================== products
    // A warp for each half: its products wait for its softmax alone, and the two
    // keep the tensor cores busy by turns.  Every K and V tile is given back by
    // both, by a half that has no use for it as soon as it is there.  Where a row
    // tile is all an item has (ONE), one warp issues for both halves, which then
    // work on every other key tile: a tile is given back by its one reader.
    regs_drop<kFwdSideRegs>();
    const int s = warp == 11;
    const int dn = (p.d + 15) & ~15;
    const int ksteps = dn / 16;
    const uint32_t id_s = make_idesc(BF16, 128, 128);
    const uint32_t id_o = make_idesc(BF16, 128, dn) | (1u << 16);  // V: consecutive values of one key
    const uint64_t dk = smem_desc(skv, 1024, 2), dv = smem_desc_mn(skv, PANEL, 1024, 2);
    const uint32_t q_lo = static_cast<uint32_t>(smem_desc(sq, 1024, 2)), k_lo = static_cast<uint32_t>(dk),
                   v_lo = static_cast<uint32_t>(dv);
    const uint32_t k_hi = static_cast<uint32_t>(dk >> 32), v_hi = static_cast<uint32_t>(dv >> 32);
    const uint32_t tbase = of_warp(tmem);
    const uint32_t ts = tbase + s * 128, tp = tbase + (EARLY ? 256 : 0) + s * P_COLS,
                   to = tbase + (EARLY ? 384 : 256) + s * O_COLS;
    if constexpr (ONE) {
      ItemRing ring(&sm->slots);
      AttnItem it;
      int head;
      uint32_t nq = 0, np = 0;  // np: bit s, phase of p_ready[s]
      RingPos<S> kv;            // ring place of the tile's (a dual item's pair's) first K
      while (warp == 9 && ring.next(&it, &head, abort_flag, true)) {
        const int kt0 = of_warp(it.kt0), dual = of_warp(it.dual), lk = of_warp(it.lk);
        const int e0 = of_warp(tile_end(p, it, 0)) - kt0, e1 = of_warp(tile_end(p, it, 1)) - kt0;
        const int n = max(e0, e1);
        if (n <= 0) continue;
        bool ok = mbar_wait_inl(smem_u32(&sm->q_full), nq & 1), fixed = false;
        ++nq;
        // Step q is half q & 1's: P V of its tile t and S of its next one.
        const int steps = dual ? n + 2 : 2 * n + 2;
#pragma unroll 1
        for (int q = 0; q < steps && ok; ++q) {
          const int h = q & 1, t = dual ? q - 2 : (q >> 1) - 1, nt = t + 1 + dual;
          const int end = dual ? n : h ? e1 : e0;
          const bool cur = t >= 0 && t < end, more = nt < end;
          // ring places from the tile's first K: K V K V .., a dual item's pairs K K V V
          const RingPos<S> k = kv.at(t < 0 ? (dual ? h : 0) : dual ? 4 + h : 2);
          const RingPos<S> v = kv.at(dual ? h + ((t | 1) < n ? 2 : 1) : 1);
          const uint32_t sc = tbase + h * 128, pc = tbase + (EARLY ? 256 : 0) + h * P_COLS,
                         oc = tbase + (EARLY ? 384 : 256) + h * O_COLS;
          const uint32_t kk = k_lo + k.st * (TILE >> 4), vv = v_lo + v.st * (TILE >> 4);
          const uint32_t q_at = q_lo + (dual ? 0 : h * (TILE >> 4));
          if (cur) {
            ok = ok && mbar_wait_inl(smem_u32(&sm->full[v.st]), v.ph);
            const int rows = lk - (kt0 + t) * kKeyTile;
            if (rows < kKeyTile && !fixed) {  // the last tile ends inside, as below
              zero_rows<PANELS>(smem + (2 + v.st) * TILE, rows);
              fixed = true;
            }
            ok = ok && mbar_wait_inl(smem_u32(&sm->p_ready[h][0]), (np >> h) & 1);
            if constexpr (!EARLY) ok = ok && mbar_wait_inl(smem_u32(&sm->p_ready[h][1]), (np >> h) & 1);
            np ^= 1u << h;
            tc_fence_after();
            if (elect_lane()) {
              product_cols<0, 8>(oc, pc, vv, v_hi, id_o, t > (dual ? h : 0));
              if (EARLY || !more) tc_commit(smem_u32(&sm->o_full[h]));
              if (dual || h || t >= e1) tc_commit(smem_u32(&sm->empty[v.st]));  // its last reader
            }
            __syncwarp();
          }
          if (more) {  // waited for last: loads bound these calls, and V has been given back
            ok = ok && mbar_wait_inl(smem_u32(&sm->full[k.st]), k.ph);
            tc_fence_after();
            if (elect_lane()) {
              product_rows<DP>(sc, q_at, kk, k_hi, id_s, ksteps);
              tc_commit(smem_u32(&sm->s_full[h]));
              if (dual || h || nt >= e1) tc_commit(smem_u32(&sm->empty[k.st]));
              if (dual ? nt + 1 == n : nt + 1 == n && (h == (e1 == n))) tc_commit(smem_u32(&sm->q_empty));
            }
          }
          __syncwarp();
          ok = __all_sync(0xffffffffu, ok);
          if (t >= 0 && (dual ? h || t + 1 == n : h)) kv = kv.at(dual && h ? 4 : 2);
        }
        if (!__all_sync(0xffffffffu, ok)) {
          sm->abort = 1;
          break;
        }
      }
    } else {
      ItemRing ring(&sm->slots);
      AttnItem it;
      int head;
      uint32_t nq = 0, nfix = 0, np = 0;
      RingPos<S> kv;  // ring place of the tile's K
      while (ring.next(&it, &head, abort_flag, true)) {
        const int kt0 = of_warp(it.kt0), lk = of_warp(it.lk);
        const int e0 = of_warp(tile_end(p, it, 0)) - kt0, e1 = of_warp(tile_end(p, it, 1)) - kt0;
        const int n = max(e0, e1);
        if (n <= 0) continue;
        const int end = s ? e1 : e0;  // this half's tiles
        const uint32_t q_at = q_lo + s * (TILE >> 4);
        bool ok = __all_sync(0xffffffffu, mbar_wait_inl(smem_u32(&sm->q_full), nq & 1));
        ++nq;
        auto full = [&](const RingPos<S>& at) { ok = ok && mbar_wait_inl(smem_u32(&sm->full[at.st]), at.ph); };
        const bool tail = lk < (kt0 + n) * kKeyTile;  // the last tile ends inside
        const bool fixer = (e0 == n) == (s == 0);
        bool fixed = false;
        if (end <= 0 && lane == 0) mbar_arrive(smem_u32(&sm->q_empty));
        // Step t makes P V of this tile and S of the next one; the first makes S alone.
#pragma unroll 1
        for (int t = -1; t < end && ok; ++t) {
          const bool cur = t >= 0, more = t + 1 < end;
          const RingPos<S> k = cur ? kv.at(2) : kv, v = kv.at(1);
          const uint32_t kk = k_lo + k.st * (TILE >> 4), vv = v_lo + v.st * (TILE >> 4);
          if (more) full(k);
          if (cur) {
            full(v);
            if (tail && t + 1 == n) {
              // Rows of the last V tile past the sequence's keys belong to someone
              // else (or to nobody).  Their weights are zero, but zero times a NaN or
              // an infinity is not, so they are zeroed before the product.
              if (fixer) {
                zero_rows<PANELS>(smem + (2 + v.st) * TILE, lk - (kt0 + t) * kKeyTile);
                if (lane == 0) mbar_arrive(smem_u32(&sm->v_fixed));
              } else {
                ok = ok && mbar_wait_inl(smem_u32(&sm->v_fixed), nfix & 1);
              }
              fixed = true;
            }
            ok = ok && mbar_wait_inl(smem_u32(&sm->p_ready[s][0]), np & 1);
            tc_fence_after();  // the product begins with half of the keys
            if (elect_lane()) product_cols<0, 4>(to, tp, vv, v_hi, id_o, t > 0);
            __syncwarp();
            ok = ok && mbar_wait_inl(smem_u32(&sm->p_ready[s][1]), np & 1);
            ++np;
          }
          tc_fence_after();
          if (elect_lane()) {
            if (cur) {
              product_cols<4, 4>(to, tp, vv, v_hi, id_o, true);
              if (!more) tc_commit(smem_u32(&sm->o_full[s]));
              tc_commit(smem_u32(&sm->empty[v.st]));
            }
            if (more) {  // over this tile's P
              product_rows<DP>(ts, q_at, kk, k_hi, id_s, ksteps);
              tc_commit(smem_u32(&sm->s_full[s]));
              tc_commit(smem_u32(&sm->empty[k.st]));
              if (t + 2 >= end) tc_commit(smem_u32(&sm->q_empty));  // the last S
            }
          }
          __syncwarp();
          ok = __all_sync(0xffffffffu, ok);
          if (cur) kv = kv.at(2);
        }
#pragma unroll 1
        for (int u = 2 * max(end, 0); u < 2 * n; ++u, kv = kv.at(1)) {  // tiles that only the other half uses
          full(kv);
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sm->empty[kv.st]));
        }
        if (tail) {  // both keep the barrier's phase
          if (ok && !fixed) ok = mbar_wait_inl(smem_u32(&sm->v_fixed), nfix & 1);
          ++nfix;
        }
        if (!__all_sync(0xffffffffu, ok)) {
          sm->abort = 1;
          break;
        }
      }
    }
    if (!ONE || warp == 9) {
      if (elect_lane()) tc_commit(smem_u32(&sm->drained));  // every product is done before TMEM is freed
      __syncwarp();
      if (!mbar_wait_inl(smem_u32(&sm->drained), 0)) sm->abort = 1;
    }
    __syncwarp();
  } else if (warp == 10) {
    // ====================================================== work units
    regs_drop<kFwdSideRegs>();
    if (lane == 0) hand_out(&sm->slots, p.counter, p.items, units, p.heads_kv, abort_flag);
    __syncwarp();
  } else {
    // ======================================================== softmax
    regs_raise<kFwdMainRegs>();
    const int s = warp >> 2;                      // row tile
    const int row = threadIdx.x & 127;
    const uint32_t lane_off = static_cast<uint32_t>(warp & 3) << 21;
    const uint32_t ts = tmem + s * 128 + lane_off;
    const uint32_t tp = t_p + s * P_COLS + lane_off, to = t_o + s * O_COLS + lane_off;
    const int pos = row / p.g, gh = row - pos * p.g;
    const float sl = p.scale_log2;
    const float grow = 8.f / sl;                  // growth of the maximum that is let stand
    ItemRing ring(&sm->slots);
    uint32_t ns = 0, no = 0;
    while (const AttnItem* itp = ring.peek(abort_flag)) {
      const int dual = itp->dual;
      const int j0 = itp->kt0 + (dual ? s : 0), end = tile_end(p, *itp, s);
      const int i = (dual ? 0 : s * p.pos) + pos;  // this row's query in the item
      const int vis = p.causal ? min(itp->lk, itp->lim0 + i + 1) : itp->lk;  // keys it sees
      float m = -INFINITY, l = 0.f;
      float base = 0.f;  // P = exp2(S scale - base)
      bool ok = true;
      for (int j = j0; j < end; j += 1 + dual) {
        ok = __all_sync(0xffffffffu, mbar_wait_inl(smem_u32(&sm->s_full[s]), ns & 1));
        ++ns;
        if (!ok) break;
        tc_fence_after();
        uint32_t x[128];
        tmem_ld128_raw(ts, x);
        const int seen = vis - j * kKeyTile;
        if (__any_sync(0xffffffffu, seen < kKeyTile)) [[unlikely]] {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (!__any_sync(0xffffffffu, seen < 32 * q + 32)) continue;
#pragma unroll
            for (int c = 32 * q; c < 32 * q + 32; ++c)
              if (c >= seen) x[c] = 0xff800000u;
          }
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 128; c += 8)
#pragma unroll
          for (int u = 0; u < 4; ++u)
            mx[u] = max3(mx[u], __uint_as_float(x[c + 2 * u]), __uint_as_float(x[c + 2 * u + 1]));
        const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        if constexpr (EARLY) {  // the tile before: O is settled, P's columns are free
          if (j > j0) {
            ok = __all_sync(0xffffffffu, mbar_wait_inl(smem_u32(&sm->o_full[s]), no & 1));
            ++no;
            if (!ok) break;
            tc_fence_after();
          }
        }
        const bool raise = mt > m + grow || (m == -INFINITY && mt > m);
        if (__any_sync(0xffffffffu, raise)) [[unlikely]] {
          const float mn = raise ? mt : m;
          const float nb = base_of<BF16>(mn, sl);
          const float f = m == -INFINITY ? 0.f : step_down<BF16>(m, mn, base, nb, sl);  // 1 for rows that stay
          m = mn;
          base = nb;
          l *= f;
          if (j > j0) {
#pragma unroll 1
            for (int c = 0; c < p.d; c += 16) {
              uint32_t o[16];
              tmem_ld16_raw(to + c, o);
#pragma unroll
              for (int u = 0; u < 16; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * f);
              tmem_st16(to + c, o);
            }
          }
        }
        // P = exp2(S scale - base); base is m scale - kShift with its rounding, the same for
        // the whole row, which O, the sum and lse have too.  Where the rounding left
        // more than a fraction it is taken off as well; the vote only spares the other
        // warps that step, which changes no bit of a row whose rest is 0.
        const float rest = rest_of<BF16>(m, base, sl);
        const bool far = __any_sync(0xffffffffu, rest != 0.f);
        if (far) [[unlikely]] {
#pragma unroll
          for (int c = 0; c < 128; ++c) x[c] = __float_as_uint(fmaf(__uint_as_float(x[c]), sl, -base) - rest);
        }
        const uint64_t nm = far ? 0 : pair2(-base, -base), sl2 = far ? pair2(1.f, 1.f) : pair2(sl, sl);
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // 32 keys at a time, stored as they are done
          uint32_t w[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            float e0, e1;
            unpair2(fma2(pair2(__uint_as_float(x[q * 32 + 2 * c]), __uint_as_float(x[q * 32 + 2 * c + 1])), sl2, nm), e0,
                    e1);
            e0 = ex2(e0);
            e1 = ex2(e1);
            sum[c & 1] = add2(sum[c & 1], pair2(e0, e1));
            w[c] = pack_pair<BF16>(e0, e1);
          }
          tmem_st16(tp + q * 16, w);
          if (q == 3 || (q == 1 && !EARLY)) {  // half of the keys: their product can begin
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm->p_ready[s][EARLY ? 0 : q >> 1]));
          }
        }
        float s0, s1;
        unpair2(add2(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
      }
      if (!ok) {
        sm->abort = 1;
        break;
      }
      const bool have = end > j0;
      if (have) {
        if (!__all_sync(0xffffffffu, mbar_wait_inl(smem_u32(&sm->o_full[s]), no & 1))) {
          sm->abort = 1;
          break;
        }
        ++no;
        tc_fence_after();
      }
      const AttnItem it = *itp;
      const int head = ring.head();
      const bool live = pos < p.pos && i < it.n_pos;
      const int64_t tok = static_cast<int64_t>(it.q_row) + i;
      const int h = head * p.g + gh;
      if (it.slot < 0) {
        const float inv = vis > 0 ? 1.f / l : 0.f;  // a row that sees no key: 0
        uint8_t* dst = p.out + tok * p.out_t + h * p.out_h;
#pragma unroll 1
        for (int c = 0; c < p.d; c += 32) {  // O has whole 32s of columns
          uint32_t o[32], w[16];
          if (have) tmem_ld32_raw(to + c, o);
#pragma unroll
          for (int u = 0; u < 16; ++u)
            w[u] = have && vis > 0 ? pack_pair<BF16>(__uint_as_float(o[2 * u]) * inv, __uint_as_float(o[2 * u + 1]) * inv)
                                   : 0u;
#pragma unroll
          for (int u = 0; u < 16; u += 4)
            if (live && c + 2 * u < p.d)
              *reinterpret_cast<uint4*>(dst + c * 2 + u * 4) = make_uint4(w[u], w[u + 1], w[u + 2], w[u + 3]);
        }
        if (p.lse && live) p.lse[tok * p.heads_q + h] = vis > 0 ? base * kLn2 + logf(l) : -INFINITY;
      } else {
        // a part of the keys: O, m and l in fp32 for k_attn_join
        const int part = it.slot + (dual ? 2 * it.split + s : it.split);
        const int64_t first = (static_cast<int64_t>(part) * p.heads_kv + head) * __ldcg(p.header + 3);
        float* dst = p.part + (first + i * p.g + gh) * (p.d + 8);
        if (live) {
          dst[p.d] = have ? m : -INFINITY;
          dst[p.d + 1] = l;
        }
#pragma unroll 1
        for (int c = 0; c < p.d && have; c += 32) {
          uint32_t o[32];
          tmem_ld32_raw(to + c, o);
          if (live) {
#pragma unroll
            for (int u = 0; u < 32; u += 4)
              if (c + u < p.d) *reinterpret_cast<uint4*>(dst + c + u) = make_uint4(o[u], o[u + 1], o[u + 2], o[u + 3]);
          }
        }
      }
      ring.release();
      tc_fence_before();  // O has been read before the next item's products
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && *abort_flag) atomicOr(p.status, kDevErrTimeout);
}

// Joins the parts of the rows whose keys were cut, a warp a row, four values a
// lane (to 64 values two parts at a time): with m the largest of the parts'
// maxima, out = sum O_q f_q / sum l_q f_q, f_q = exp(scale (m_q - m)).  The parts
// are taken in order, whoever made them.  Memory bounds it: every part's fp32 rows
// are read once (four scenes' 100 queries in 38 parts each, 35 MB: 19 us, 29 with
// one part at a time).
template <bool BF16>
__global__ void __launch_bounds__(256) k_attn_join(const FwdParams p, const AttnItem* joins) {
  grid_wait();
  const int n = __ldcg(p.header + 2), stride = __ldcg(p.header + 3);
  const int lane = threadIdx.x & 31;
  const int64_t step = static_cast<int64_t>(p.heads_kv) * stride * (p.d + 8);  // one part to the next
  const int64_t total = static_cast<int64_t>(n) * p.heads_kv * stride;
  for (int64_t u = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 5; u < total;
       u += static_cast<int64_t>(gridDim.x) * 8) {
    const int r = static_cast<int>(u % stride);
    const int64_t jh = u / stride;
    const int head = static_cast<int>(jh % p.heads_kv);
    const AttnItem* it = joins + jh / p.heads_kv;
    if (r >= it->n_pos * p.g) continue;
    const int i = r / p.g, h = head * p.g + r - i * p.g;
    const int parts = it->nsplit * (it->dual ? 2 : 1);
    const float* src = p.part + ((static_cast<int64_t>(it->slot) * p.heads_kv + head) * stride + r) * (p.d + 8);
    float m = -INFINITY;
    for (int q = lane; q < parts; q += 32) m = fmaxf(m, __ldcg(src + q * step + p.d));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float base = base_of<BF16>(m, p.scale_log2);
    float l = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    const int per = p.d <= 64 ? 16 : 32;  // lanes of a part
    const int c = lane & (per - 1), first = lane / per, turn = 32 / per;
    const bool on = c * 4 < p.d;
    for (int q0 = 0; q0 < parts; q0 += 32) {
      // a part's factor a lane; 0 where it saw nothing (no O was written then)
      float f = 0.f, lq = 0.f;
      bool seen = false;
      if (q0 + lane < parts) {
        const float mq = __ldcg(src + (q0 + lane) * step + p.d);
        lq = __ldcg(src + (q0 + lane) * step + p.d + 1);
        seen = mq != -INFINITY;
        f = !seen ? 0.f : step_down<BF16>(mq, m, base_of<BF16>(mq, p.scale_log2), base, p.scale_log2);
      }
      const uint32_t have = __ballot_sync(0xffffffffu, seen);
      lq *= f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) lq += __shfl_xor_sync(0xffffffffu, lq, o);
      l += lq;
      const int cnt = min(32, parts - q0);
#pragma unroll 8
      for (int u = 0; u < cnt; u += turn) {
        const int q = u + first;  // past the last: its factor's lane holds 0
        const float fq = __shfl_sync(0xffffffffu, f, q);
        const float4 o = on && (have >> q & 1) ? __ldcg(reinterpret_cast<const float4*>(src + (q0 + q) * step) + c)
                                               : make_float4(0.f, 0.f, 0.f, 0.f);
        a.x = fmaf(o.x, fq, a.x);
        a.y = fmaf(o.y, fq, a.y);
        a.z = fmaf(o.z, fq, a.z);
        a.w = fmaf(o.w, fq, a.w);
      }
    }
    if (turn == 2) {
      a.x += __shfl_xor_sync(0xffffffffu, a.x, 16);
      a.y += __shfl_xor_sync(0xffffffffu, a.y, 16);
      a.z += __shfl_xor_sync(0xffffffffu, a.z, 16);
      a.w += __shfl_xor_sync(0xffffffffu, a.w, 16);
    }
    const int vis = p.causal ? min(it->lk, it->lim0 + i + 1) : it->lk;
    const float inv = vis > 0 ? 1.f / l : 0.f;
    const int64_t tok = static_cast<int64_t>(it->q_row) + i;
    if (on && first == 0)
      *reinterpret_cast<uint2*>(p.out + tok * p.out_t + h * p.out_h + c * 8) =
          vis > 0 ? make_uint2(pack_pair<BF16>(a.x * inv, a.y * inv), pack_pair<BF16>(a.z * inv, a.w * inv))
                  : make_uint2(0u, 0u);
    if (p.lse && lane == 0) p.lse[tok * p.heads_q + h] = vis > 0 ? base * kLn2 + logf(l) : -INFINITY;
  }
}

template <bool BF16, bool ONE>
const void* fwd_kernel(int dp) {
  return dp == 64 ? reinterpret_cast<const void*>(k_attn_fwd<BF16, 64, ONE>)
                  : reinterpret_cast<const void*>(k_attn_fwd<BF16, 128, ONE>);
}

}  // namespace

sc_status attn_fwd(const AttnArgs& a) {
  const int g = a.heads_q / a.heads_kv, pos = 128 / g;
  const int sms = device_sm_count();
  const int64_t items_ub = a.t_q / (2 * pos) + a.n_seq;
  if (items_ub * a.heads_kv > 0x3fffffff) return set_error(SC_ERR_UNSUPPORTED, "too many query tiles");
  // Partial results: room for about four parts an SM and two an item, where an
  // item has few rows (a guess from the average; the plan sees whether they
  // fit) or the items are few.
  const int64_t avg = a.n_seq ? (a.t_q * g + a.n_seq - 1) / a.n_seq : 0;
  const bool few = items_ub * a.heads_kv <= 8ll * sms;
  const int64_t rows_guess = few ? 2 * pos * g : 2 * avg;
  const int64_t slots = 8ll * sms / a.heads_kv + 2 + 2 * items_ub;
  // On average at most one row tile a sequence: the form whose halves share one.
  const bool one = avg <= 128;
  // no list of more keys than a part (a half) has: nothing to cut, and the join is not launched
  const bool cuts = a.t_k > (one ? 1 : kMinPartTiles) * kKeyTile && (few || avg <= 32);
  int64_t part_rows = cuts ? slots * a.heads_kv * (rows_guess < 2 * pos * g ? rows_guess : 2 * pos * g) : 0;
  const int64_t row_bytes = (a.head_dim + 8) * 4ll;
  if (part_rows * row_bytes > (int64_t(1) << 28)) part_rows = (int64_t(1) << 28) / row_bytes;
  const int64_t cap = items_ub + (part_rows ? slots : 0);
  Arena ar;
  const size_t o_head = ar.take(kPlanHeader * sizeof(int));
  const size_t o_items = ar.take(static_cast<size_t>(cap) * sizeof(AttnItem));
  const size_t o_joins = ar.take(part_rows ? static_cast<size_t>(items_ub) * sizeof(AttnItem) : 0);
  const size_t o_part = ar.take(static_cast<size_t>(part_rows * row_bytes));
  int* status = attn_status_word();
  if (!status) return set_error(SC_ERR_CUDA, "the attention status word is not available");
  const int dp = a.head_dim <= 64 ? 64 : 128;
  const size_t tile = static_cast<size_t>(dp) / 64 * 16384;
  FwdParams p{};
  const size_t smem = (2 + fwd_stages(dp)) * tile + sizeof(FwdSmem) + 1024;
  const void* kern = a.dtype == SC_BF16 ? (one ? fwd_kernel<true, true>(dp) : fwd_kernel<true, false>(dp))
                                        : (one ? fwd_kernel<false, true>(dp) : fwd_kernel<false, false>(dp));
  int regs = 0;
  sc_status st = kernel_setup(kern, smem, &regs);
  if (st) return st;
  if (regs != kFwdRegs) return set_error(SC_ERR_CUDA, "attention kernel: not the registers it was written for");
  CUtensorMap qm, km, vm;
  const void* any = a.q.data;  // no key rows: maps of legal sizes that nothing reads
  const bool keys = a.t_k > 0;
  if ((st = attn_map(&qm, a.q.data, a.dtype, a.head_dim, a.heads_q, a.t_q, a.q.token_stride, a.q.head_stride, g, pos)))
    return st;
  if ((st = attn_map(&km, keys ? a.k.data : any, a.dtype, a.head_dim, keys ? a.heads_kv : 1, keys ? a.t_k : 1,
                     a.k.token_stride, a.k.head_stride, 1, kKeyTile)))
    return st;
  if ((st = attn_map(&vm, keys ? a.v.data : any, a.dtype, a.head_dim, keys ? a.heads_kv : 1, keys ? a.t_k : 1,
                     a.v.token_stride, a.v.head_stride, 1, kKeyTile)))
    return st;
  void* ws = nullptr;
  if ((st = dev_alloc(&ws, ar.bytes, a.stream))) return st;
  uint8_t* base = static_cast<uint8_t*>(ws);
  PlanArgs pl{};
  pl.q_off = a.q_off;
  pl.k_off = a.k_off;
  pl.k_len = a.k_len;
  pl.n_seq = static_cast<int>(a.n_seq);
  pl.t_q = a.t_q;
  pl.t_k = a.t_k;
  pl.pos_per_item = 2 * pos;
  pl.causal = a.causal;
  pl.heads_kv = a.heads_kv;
  pl.mode = kPlanRows;
  pl.g = g;
  pl.sms = sms;
  pl.over = 4;
  pl.part_rows = part_rows;
  pl.min_tiles = kMinPartTiles;
  pl.dual = one;
  pl.cap = static_cast<int>(cap);
  pl.join_cap = part_rows ? static_cast<int>(items_ub) : 0;
  pl.header = reinterpret_cast<int*>(base + o_head);
  pl.items = reinterpret_cast<AttnItem*>(base + o_items);
  pl.joins = reinterpret_cast<AttnItem*>(base + o_joins);
  pl.status = status;
  st = attn_plan(pl, nullptr, false, a.stream);
  if (!st) {
    p.out = static_cast<uint8_t*>(a.out.data);
    p.out_t = a.out.token_stride * 2;
    p.out_h = a.out.head_stride * 2;
    p.lse = a.lse;
    p.header = pl.header;
    p.counter = pl.header + 1;
    p.items = pl.items;
    p.part = reinterpret_cast<float*>(base + o_part);
    p.heads_q = a.heads_q;
    p.heads_kv = a.heads_kv;
    p.g = g;
    p.pos = pos;
    p.d = a.head_dim;
    p.scale_log2 = a.scale * kLog2e;
    p.causal = a.causal;
    p.status = status;
    const int64_t most = cap * a.heads_kv;
    const int grid = static_cast<int>(most < sms ? most : sms);
    void* args[] = {&p, &qm, &km, &vm};
    cudaError_t e;
    SC_LAUNCH("attn_fwd", a.stream,
              (e = launch_after(kern, grid, kFwdThreads, smem, a.stream, args)));
    if (e != cudaSuccess) st = set_cuda_error(e, "attn_fwd");
    if (!st && part_rows) {
      const int64_t warps = a.t_q * a.heads_q;
      const unsigned nb = static_cast<unsigned>(warps < 32ll * sms ? (warps + 7) / 8 : 4 * sms);
      const AttnItem* joins = pl.joins;
      void* jargs[] = {&p, &joins};
      const void* jk = a.dtype == SC_BF16 ? reinterpret_cast<const void*>(k_attn_join<true>)
                                          : reinterpret_cast<const void*>(k_attn_join<false>);
      SC_LAUNCH("attn_join", a.stream, (e = launch_after(jk, nb, 256, 0, a.stream, jargs)));
      if (e != cudaSuccess) st = set_cuda_error(e, "attn_join");
    }
  }
  dev_free(ws, a.stream);
  return st;
}

}  // namespace sc
