// The norm of each head of queries and keys with the position rotation in the
// same pass, and its gradients.
//
// One row is one head of one token, D values x.  With a norm weight w
//   z = w x r,  r = 1 / sqrt(mean(x^2) + eps)      (without one: z = x)
// and the first R values turn in pairs i in [0, R/2) by phi_i = pos[axis(i)] f_i:
//   y_a = amp (z_a cos phi - z_b sin phi),  y_b = amp (z_b cos phi + z_a sin phi).
// The gradient turns gy back (the transpose of a rotation) and goes through the
// norm: g = R^T gy, h = g w, gx = r (h - x r mean(h x r)), gw = sum g x r.
//
// Every value is read once and written once and takes about ten operations, so
// memory should bound it; what comes near is the instructions a value takes.  A
// row lies in a group of LPR lanes, eight consecutive values (one 16-byte load of
// 16-bit types) a lane, so the norm is a sum over the group by shuffles; the
// partner of a pair comes from the lane that holds it.  A group takes one token's
// heads, or some of them, one after the other: a lane's angles are the same for
// all heads of a token, so it works them out once and keeps them, with the weights
// folded in, in registers (read from a table for every row they made the kernel
// three times slower).  The forward has four rows' loads in flight and four blocks
// an SM; the gradient, which needs twice the registers, has two blocks an SM and
// its rows copied to shared memory two steps ahead (the forward was slower that
// way: 241 us instead of 207 for the voxels below).
//
// Kernel times: 32768 tokens, 32 + 8 heads of 128, bf16: 126 us, 5.3 TB/s; 480000
// tokens, 4 + 4 heads of 64 turned by three axes, f16: forward 196 us (5.0 TB/s; issue
// slots 60 % busy, DRAM 61 %, no one unit), gradient 269 us (5.5 TB/s, bound by the
// instructions it issues: issue slots 70 % busy; 368 us with the angles worked out for
// each side and one value an instruction); 240000 of them, f32: 205 us (4.8 TB/s) and
// 364 us (4.1 TB/s).  Four blocks an SM leave the forward 64 registers: its 16-bit forms
// spill 28 to 128 bytes.
#include "f32x2.cuh"
#include "sc_internal.cuh"
#include "tc_ptx.cuh"

namespace sc {
namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------ 8 values --
// As four pairs (v[2i], v[2i + 1]), which one instruction takes at once: the
// kernels are bound by the instructions they issue before memory is.
template <typename T>
struct Vec8;
template <>
struct Vec8<__half> {
  static constexpr int kWords = 4;
  static __device__ __forceinline__ void unpack(const uint32_t (&w)[4], uint64_t (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[i] = pair2(f.x, f.y);
    }
  }
  static __device__ __forceinline__ void pack(const uint64_t (&x)[4], uint32_t (&w)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      unpair2(x[i], lo, hi);
      const __half2 h = __floats2half2_rn(lo, hi);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
};
template <>
struct Vec8<__nv_bfloat16> {
  static constexpr int kWords = 4;
  static __device__ __forceinline__ void unpack(const uint32_t (&w)[4], uint64_t (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = pair2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  }
  static __device__ __forceinline__ void pack(const uint64_t (&x)[4], uint32_t (&w)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      unpair2(x[i], lo, hi);
      const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
};
template <>
struct Vec8<float> {
  static constexpr int kWords = 8;
  static __device__ __forceinline__ void unpack(const uint32_t (&w)[8], uint64_t (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = pair2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  }
  static __device__ __forceinline__ void pack(const uint64_t (&x)[4], uint32_t (&w)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      unpair2(x[i], lo, hi);
      w[2 * i] = __float_as_uint(lo);
      w[2 * i + 1] = __float_as_uint(hi);
    }
  }
};

template <int NW>
__device__ __forceinline__ void load_words(const void* p, uint32_t (&w)[NW]) {
#pragma unroll
  for (int i = 0; i < NW / 4; ++i) {
    const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p) + i);
    w[4 * i] = v.x;
    w[4 * i + 1] = v.y;
    w[4 * i + 2] = v.z;
    w[4 * i + 3] = v.w;
  }
}
template <int NW>
__device__ __forceinline__ void store_words(void* p, const uint32_t (&w)[NW]) {
#pragma unroll
  for (int i = 0; i < NW / 4; ++i)
    __stcs(reinterpret_cast<uint4*>(p) + i, make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]));
}

// The sum of a lane's four pairs.
__device__ __forceinline__ float sum8(const uint64_t (&v)[4]) {
  float lo, hi;
  unpair2(add2(add2(v[0], v[1]), add2(v[2], v[3])), lo, hi);
  return lo + hi;
}

template <int LPR>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// cos and sin of pos * f, times amp.  The product can be thousands of turns, and
// 32 bits of it would leave few for the fraction (1e-3 radians at position 32768,
// f = 1).  Positions are whole numbers, so whole turns a position change nothing:
// f / 2 pi is kept as a fixed-point fraction of a turn, c of 2^64, and pos * c
// modulo 2^64 is the product's fraction, off by 2^-33 of a turn at any position.
// The rows are f32 (EXACT: a few units in the last place) or 16-bit, for which its
// upper half and the fast sine's 2^-20 are far below the output's rounding.
typedef uint64_t Turn;
// |f| = m 2^e times 1 / 2 pi, of which 128 bits after the point are enough for
// e <= 40 (|f| < 2^64); `finite`: f is.
__device__ __forceinline__ Turn turn_of(float f, bool* finite) {
  constexpr uint64_t kHi = 0x28be60db9391054aull, kLo = 0x7f09d5f47d4d3770ull;  // 1 / 2 pi
  const uint32_t bits = __float_as_uint(f);
  const int ex = bits >> 23 & 255;
  *finite = ex != 255;
  const uint64_t m = ex ? (bits & 0x7fffff) | 0x800000 : bits & 0x7fffff;
  const int shift = 64 - ((ex ? ex : 1) - 150);  // the product's places below 2^-64
  const uint64_t w0 = m * kLo, w1 = m * kHi + __umul64hi(m, kLo);
  const uint64_t w2 = __umul64hi(m, kHi) + (w1 < __umul64hi(m, kLo));
  uint64_t c;
  if (shift >= 128) c = shift < 192 ? w2 >> (shift - 128) : 0;
  else if (shift >= 64) c = shift > 64 ? w1 >> (shift - 64) | w2 << (128 - shift) : w1;
  else if (shift >= 0) c = shift > 0 ? w0 >> shift | w1 << (64 - shift) : w0;
  else c = w0 << -shift;
  return bits >> 31 ? 0 - c : c;
}
template <bool EXACT>
__device__ __forceinline__ float2 angle(int pos, Turn c, float amp) {
  float s, co;
  if constexpr (EXACT) {
    const uint64_t t = static_cast<uint64_t>(static_cast<int64_t>(pos)) * c;
    sincospif(__ll2float_rn(static_cast<int64_t>(t)) * 0x1p-63f, &s, &co);
  } else {
    const uint32_t lo = static_cast<uint32_t>(c), hi = static_cast<uint32_t>(c >> 32), x = static_cast<uint32_t>(pos);
    const uint32_t t = x * hi + __umulhi(x, lo) - (pos < 0 ? lo : 0u);  // the product's upper half
    __sincosf(static_cast<float>(static_cast<int>(t)) * (6.283185307179586f * 0x1p-32f), &s, &co);
  }
  return make_float2(co * amp, s * amp);
}

struct RopeParams {
  const uint8_t* x[2];       // q and k (backward: the forward's inputs)
  const uint8_t* gy[2];      // backward: gradients of the outputs
  uint8_t* y[2];             // outputs (backward: gradients of the inputs)
  int64_t xt[2], xh[2];      // strides in bytes: token, head
  int64_t gt[2], gh[2];
  int64_t yt[2], yh[2];
  int heads[2];
  const float* w[2];
  float* gw_part;            // backward with a norm: [blocks][side][D]
  const int* pos;
  int64_t pos_stride;        // elements between tokens
  const float* freq;
  int64_t tokens;
  int d, half, per;          // half = R / 2 pairs, per = pairs of one axis
  int chunks;                // groups that share a token's heads
  int per_chunk[2];          // heads of each
  float eps, amp;
};

// How the partners of a lane's eight values, pairs (i, i + half), are fetched.
enum Pairing {
  kInterleaved,  // pairs (2i, 2i + 1): in the lane itself
  kHalf8,        // half a multiple of 8: a whole lane's values, by shuffles
  kHalf2,        // even: two values at a time from the warp's rows in shared memory
  kHalf1,        // odd: one at a time
};

template <typename T, int LPR, int PAIRING>
__device__ __forceinline__ void partners(const uint32_t (&w)[Vec8<T>::kWords], uint64_t (&p)[4], int gl, int half,
                                         T* stage) {
  constexpr int NW = Vec8<T>::kWords;
  if constexpr (PAIRING == kInterleaved) {
    uint32_t o[NW];  // the neighbours of values that do not turn are no partners
#pragma unroll
    for (int i = 0; i < NW; ++i) o[i] = i * (8 / NW) < 2 * half - gl * 8 ? w[i] : 0u;
    uint64_t x[4];
    Vec8<T>::unpack(o, x);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float lo, hi;
      unpair2(x[j], lo, hi);
      p[j] = pair2(hi, lo);
    }
  } else if constexpr (PAIRING == kHalf8) {
    const int step = half >> 3;
    const int from = gl < step ? gl + step : (gl < 2 * step ? gl - step : gl);
    uint32_t o[NW];
#pragma unroll
    for (int i = 0; i < NW; ++i) o[i] = __shfl_sync(0xffffffffu, w[i], from, LPR);
    Vec8<T>::unpack(o, p);
  } else {
    // word k of the warp's lane l at [k][l]: neither side has bank conflicts
    uint32_t* words = reinterpret_cast<uint32_t*>(stage);
    const int row = (threadIdx.x & 31) / LPR * LPR;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < NW; ++i) words[i * 32 + row + gl] = w[i];
    __syncwarp();
    if constexpr (PAIRING == kHalf2 && sizeof(T) == 2) {
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = gl * 8 + 2 * j;
        const int from = (e < half ? e + half : (e < 2 * half ? e - half : e)) >> 1;
        o[j] = words[(from & 3) * 32 + row + (from >> 2)];
      }
      Vec8<T>::unpack(o, p);
    } else {
      constexpr int PER = 8 / NW;  // values of a word
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float v[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int e = gl * 8 + 2 * j + k;
          const int from = e < half ? e + half : (e < 2 * half ? e - half : e);
          v[k] = static_cast<float>(stage[((from / PER % NW) * 32 + row + (from >> 3)) * PER + from % PER]);
        }
        p[j] = pair2(v[0], v[1]);
      }
    }
  }
}

// Value e's pair (-1: past the rotated ones) and its partner.
template <int PAIRING>
__device__ __forceinline__ int pair_of(int e, int half) {
  if (e >= 2 * half) return -1;
  if constexpr (PAIRING == kInterleaved) return e >> 1;
  return e < half ? e : e - half;
}
template <int PAIRING>
__device__ __forceinline__ int partner_of(int e, int half) {
  if (e >= 2 * half) return e;
  if constexpr (PAIRING == kInterleaved) return e ^ 1;
  return e < half ? e + half : e - half;
}

// y_e = z_e ca_e + z_partner(e) sb_e turns by a token's angles: the partner's
// sine has the sign of the second member's formula, and `back` turns back.  A
// value that does not turn is its own partner (with neighbours for pairs it has
// none, a zero), with the factors 1 and 2^-60: the sum rounds to the value, an
// infinity stays one (times 0 it would be NaN), and no other value has a part in it.
// The group's lanes work out the token's pairs between them, four each, and put
// each under both its values in `table`, value e of the warp's group g in row e % 8
// at g * LPR + e / 8, each row turned by some places from the one before: then
// neither the lanes that write consecutive pairs nor those that read their eight
// values meet in a bank.
template <int LPR, int PAIRING>
struct Angles {
  Turn f[4];
  int axis;         // of the lane's four pairs, a byte each; 128: the frequency is not finite
  uint32_t to[4];   // a pair's two places in the table (bytes, 16 bits each)
  float2* table;
  static __device__ __forceinline__ int place(int col, int e) {  // value e of the group whose lane 0 is `col`
    const int j = e & 7;
    return j * 32 + ((col + (e >> 3) + j * (LPR >= 16 ? 2 : 1)) & 31);
  }
  __device__ __forceinline__ Angles(const RopeParams& p, int gl, float2* table_) : axis(0), table(table_) {
    const int col = (threadIdx.x & 31) / LPR * LPR;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int pair = gl + i * LPR;
      bool finite;
      f[i] = turn_of(pair < p.half ? __ldg(p.freq + pair) : 0.f, &finite);
      axis |= ((pair >= p.per) + (pair >= 2 * p.per) + (pair >= 3 * p.per) + (finite ? 0 : 128)) << (8 * i);
      const int e0 = PAIRING == kInterleaved ? 2 * pair : pair, e1 = PAIRING == kInterleaved ? e0 + 1 : pair + p.half;
      to[i] = static_cast<uint32_t>(place(col, e0)) * 8 | static_cast<uint32_t>(place(col, e1)) * 8 << 16;
    }
    for (int j = 0; j < 8; ++j) table[place(col, gl * 8 + j)] = make_float2(1.f, 0x1p-60f);  // values that do not turn
    __syncwarp();
  }
  // Token t's positions, ahead of its angles.
  __device__ __forceinline__ void positions(const RopeParams& p, int64_t t, int gl, int (&pos)[4]) const {
    const int* at = p.pos + t * p.pos_stride;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (gl + i * LPR < p.half) pos[i] = __ldg(at + (axis >> (8 * i) & 3));
  }
  template <typename T>
  __device__ __forceinline__ void fill(const RopeParams& p, const int (&pos)[4], int gl, bool back) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (gl + i * LPR < p.half) {
        float2 cs = angle<sizeof(T) == 4>(pos[i], f[i], p.amp);
        if (back) cs.y = -cs.y;
        uint8_t* at = reinterpret_cast<uint8_t*>(table);
        *reinterpret_cast<float2*>(at + (to[i] & 0xFFFF)) = make_float2(cs.x, -cs.y);
        *reinterpret_cast<float2*>(at + (to[i] >> 16)) = cs;
      }
    }
    if (axis & 0x80808080) [[unlikely]] {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (axis >> (8 * i) & 128)
          *reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(table) + (to[i] & 0xFFFF)) =
              *reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(table) + (to[i] >> 16)) = make_float2(NAN, NAN);
    }
    __syncwarp();
  }
  // The lane's eight values' factors.
  __device__ __forceinline__ void read(int gl, uint64_t (&a)[4], uint64_t (&b)[4]) const {
    const int col = (threadIdx.x & 31) / LPR * LPR;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 u = table[place(col, gl * 8 + 2 * j)], v = table[place(col, gl * 8 + 2 * j + 1)];
      a[j] = pair2(u.x, v.x);
      b[j] = pair2(u.y, v.y);
    }
  }
};

// A group's token and part of its heads; whole warps run the loops, for the
// shuffles, and groups without a token do nothing in them.
struct Unit {
  int64_t token;
  int chunk;
  bool on;
};
template <int LPR>
__device__ __forceinline__ Unit unit_of(const RopeParams& p, int64_t block) {
  const int64_t u = block * (kThreads / LPR) + threadIdx.x / LPR;
  Unit r;
  r.token = u;
  r.chunk = 0;
  if (p.chunks > 1) {  // few tokens: the units fit 32 bits
    r.token = static_cast<uint32_t>(u) / static_cast<uint32_t>(p.chunks);
    r.chunk = static_cast<int>(static_cast<uint32_t>(u) % static_cast<uint32_t>(p.chunks));
  }
  r.on = r.token < p.tokens;
  if (!r.on) r.token = 0;
  return r;
}

// Rows on their way: each lane copies its own 16 or 32 bytes of a row to its
// own places in shared memory, ST steps of U rows ahead of the one it works on
// (of the unit's next heads, its other side, or the next unit), so no barrier is
// needed and the copies cost no registers.
template <int N>
__device__ __forceinline__ void copies_left() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <typename T, int LPR, int NSRC>
struct Rows {
  static constexpr int NW = Vec8<T>::kWords, Q = NW / 4, U = sizeof(T) == 4 ? 1 : 2, ST = 4;
  static constexpr int bytes() { return ST * U * NSRC * Q * 16 * kThreads; }
  uint32_t mine, put = 0, got = 0;  // stages
  int64_t blk, blocks, count;
  int side, last, i, n, left;       // side: the next rows'; last: of a unit
  const uint8_t* src[NSRC];
  __device__ __forceinline__ Rows(const RopeParams& p, void* smem, int64_t first, int64_t count_, int64_t blocks_,
                                  int side0, int side1)
      : mine(smem_u32(smem) + threadIdx.x * 16), blk(first), blocks(blocks_), count(count_), side(side0), last(side1) {
    place(p);
#pragma unroll
    for (int k = 0; k < ST - 1; ++k) fetch(p, side0);
  }
  __device__ __forceinline__ const uint8_t* base(const RopeParams& p, int which) const {
    return which == 0 ? p.gy[side] : p.x[side];
  }
  __device__ __forceinline__ int64_t head_stride(const RopeParams& p, int which) const {
    return which == 0 ? p.gh[side] : p.xh[side];
  }
  __device__ __forceinline__ void place(const RopeParams& p) {
    i = 0;
    n = p.per_chunk[side];
    left = 0;
    if (blk >= blocks) return;
    const Unit u = unit_of<LPR>(p, blk);
    const int e0 = threadIdx.x % LPR * 8, h0 = u.chunk * n;
    if (u.on && e0 < p.d) left = min(n, p.heads[side] - h0);
#pragma unroll
    for (int k = 0; k < NSRC; ++k)
      src[k] = base(p, k) + u.token * (k == 0 ? p.gt[side] : p.xt[side]) + e0 * sizeof(T) +
               h0 * head_stride(p, k);
  }
  __device__ __forceinline__ void fetch(const RopeParams& p, int side0) {
    if (blk < blocks) {
#pragma unroll
      for (int q = 0; q < U; ++q)
        if (i + q < left)
#pragma unroll
          for (int k = 0; k < NSRC; ++k)
#pragma unroll
            for (int h = 0; h < Q; ++h)
              cp_async_16(mine + (((put * U + q) * NSRC + k) * Q + h) * (16 * kThreads),
                          src[k] + q * head_stride(p, k) + h * 16, 16);
      i += U;
#pragma unroll
      for (int k = 0; k < NSRC; ++k) src[k] += U * head_stride(p, k);
      if (i >= n) {
        if (side == last) {
          side = side0;
          blk += count;
        } else {
          side = last;
        }
        place(p);
      }
      put = put + 1 == ST ? 0 : put + 1;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // The oldest step's rows have landed.
  __device__ __forceinline__ void land() { copies_left<ST - 2>(); }
  __device__ __forceinline__ void read(int q, int k, bool on, uint32_t (&w)[NW]) const {
#pragma unroll
    for (int h = 0; h < Q; ++h) {
      uint32_t a = 0, b = 0, c = 0, d = 0;
      if (on)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
                     : "r"(mine + (((got * U + q) * NSRC + k) * Q + h) * (16 * kThreads))
                     : "memory");
      w[4 * h] = a;
      w[4 * h + 1] = b;
      w[4 * h + 2] = c;
      w[4 * h + 3] = d;
    }
  }
  __device__ __forceinline__ void next() { got = got + 1 == ST ? 0 : got + 1; }
};

template <typename T, int LPR, int PAIRING, bool NORM>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 3 : 4) k_rope_fwd(const RopeParams p) {
  constexpr int NW = Vec8<T>::kWords, GROUPS = kThreads / LPR, U = sizeof(T) == 4 ? 2 : 4;
  __shared__ __align__(16) T s_stage[PAIRING >= kHalf2 ? kThreads * 8 : 8];
  __shared__ float2 s_table[kThreads * 8];
  // [side][a value's, its partner's][values 0-3, 4-7 of a lane][lane]
  __shared__ float4 s_w[NORM ? 2 : 1][2][2][NORM ? LPR : 1];
  T* stage = s_stage + (PAIRING >= kHalf2 ? (threadIdx.x >> 5) * 256 : 0);
  const int gl = threadIdx.x % LPR;
  const int e0 = gl * 8;
  const float inv_d = 1.f / static_cast<float>(p.d);
  if constexpr (NORM) {
    for (int i = threadIdx.x; i < 4 * LPR * 8; i += kThreads) {
      const int side = i / (2 * LPR * 8), which = i / (LPR * 8) & 1, e = i % (LPR * 8);
      const int o = which ? partner_of<PAIRING>(e, p.half) : e;
      reinterpret_cast<float*>(&s_w[side][which][e >> 2 & 1][e >> 3])[e & 3] =
          p.heads[side] && o < p.d ? __ldg(p.w[side] + o) : 0.f;
    }
    __syncthreads();
  }
  Angles<LPR, PAIRING> angles(p, gl, s_table + (threadIdx.x >> 5) * 256);
  const int64_t blocks = (p.tokens * p.chunks + GROUPS - 1) / GROUPS;
  int pos[4] = {};
  if (blockIdx.x < blocks) angles.positions(p, unit_of<LPR>(p, blockIdx.x).token, gl, pos);
#pragma unroll 1
  for (int64_t blk = blockIdx.x; blk < blocks; blk += gridDim.x) {
    const Unit u = unit_of<LPR>(p, blk);
    const bool act = u.on && e0 < p.d;
    angles.template fill<T>(p, pos, gl, false);
    if (blk + gridDim.x < blocks) angles.positions(p, unit_of<LPR>(p, blk + gridDim.x).token, gl, pos);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const int n = p.per_chunk[side];
      uint64_t a[4], b[4];
      angles.read(gl, a, b);
      if constexpr (NORM) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 wa = s_w[side][0][h][gl], wb = s_w[side][1][h][gl];
          a[2 * h] = mul2(a[2 * h], pair2(wa.x, wa.y)), a[2 * h + 1] = mul2(a[2 * h + 1], pair2(wa.z, wa.w));
          b[2 * h] = mul2(b[2 * h], pair2(wb.x, wb.y)), b[2 * h + 1] = mul2(b[2 * h + 1], pair2(wb.z, wb.w));
        }
      }
      const int h0 = u.chunk * n;
      const int left = act ? min(n, p.heads[side] - h0) : 0;
      const int64_t xh = p.xh[side], yh = p.yh[side];
      const uint8_t* x = p.x[side] + u.token * p.xt[side] + e0 * sizeof(T) + h0 * xh;
      uint8_t* y = p.y[side] + u.token * p.yt[side] + e0 * sizeof(T) + h0 * yh;
#pragma unroll 1
      for (int i = 0; i < n; i += U, x += U * xh, y += U * yh) {
        uint32_t w[U][NW];
#pragma unroll
        for (int q = 0; q < U; ++q) {
#pragma unroll
          for (int k = 0; k < NW; ++k) w[q][k] = 0u;
          if (i + q < left) load_words<NW>(x + q * xh, w[q]);
        }
#pragma unroll
        for (int q = 0; q < U; ++q) {
          uint64_t v[4], vp[4];
          Vec8<T>::unpack(w[q], v);
          partners<T, LPR, PAIRING>(w[q], vp, gl, p.half, stage);
          uint64_t rn = 0;
          if constexpr (NORM) {
            uint64_t ss[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) ss[j] = mul2(v[j], v[j]);
            const float r = rsqrtf(group_sum<LPR>(sum8(ss)) * inv_d + p.eps);
            rn = pair2(r, r);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[j] = fma2(v[j], a[j], mul2(vp[j], b[j]));
            if constexpr (NORM) v[j] = mul2(v[j], rn);
          }
          if (i + q < left) {
            Vec8<T>::pack(v, w[q]);
            store_words<NW>(y + q * yh, w[q]);
          }
        }
      }
    }
  }
}

// The gradient.  A block walks q's and k's heads of its tokens, keeps its sums of
// both weights' gradients in registers and writes them once, [block][side][D] in
// gw_part; k_rope_gw adds the blocks in order (the same result every time).
template <typename T, int LPR, int PAIRING, bool NORM>
__global__ void __launch_bounds__(kThreads, NORM ? 2 : 3) k_rope_bwd(const RopeParams p) {
  using R = Rows<T, LPR, NORM ? 2 : 1>;
  constexpr int NW = R::NW, U = R::U, GROUPS = kThreads / LPR;
  extern __shared__ __align__(16) uint8_t s_rows[];
  __shared__ __align__(16) T s_stage[PAIRING >= kHalf2 ? kThreads * 8 : 8];
  __shared__ float2 s_table[kThreads * 8];
  __shared__ ulonglong2 s_w[NORM ? 2 : 1][2][NORM ? LPR : 1];  // [side][values 0-3, 4-7 of a lane][lane]
  T* stage = s_stage + (PAIRING >= kHalf2 ? (threadIdx.x >> 5) * 256 : 0);
  const int gl = threadIdx.x % LPR, grp = threadIdx.x / LPR;
  const int e0 = gl * 8;
  const float inv_d = 1.f / static_cast<float>(p.d);
  const int64_t blocks = (p.tokens * p.chunks + GROUPS - 1) / GROUPS;
  const int side0 = p.heads[0] ? 0 : 1, side1 = p.heads[1] ? 1 : 0;
  R rows(p, s_rows, blockIdx.x, gridDim.x, blocks, side0, side1);
  if constexpr (NORM) {
    for (int i = threadIdx.x; i < 2 * LPR * 8; i += kThreads) {
      const int side = i / (LPR * 8), e = i % (LPR * 8);
      reinterpret_cast<float*>(&s_w[side][e >> 2 & 1][e >> 3])[e & 3] =
          p.heads[side] && e < p.d ? __ldg(p.w[side] + e) : 0.f;
    }
    __syncthreads();
  }
  uint64_t gw[2][4] = {};
  Angles<LPR, PAIRING> angles(p, gl, s_table + (threadIdx.x >> 5) * 256);
  int pos[4] = {};
  if (blockIdx.x < blocks) angles.positions(p, unit_of<LPR>(p, blockIdx.x).token, gl, pos);
#pragma unroll 1
  for (int64_t blk = blockIdx.x; blk < blocks; blk += gridDim.x) {
    const Unit u = unit_of<LPR>(p, blk);
    const bool act = u.on && e0 < p.d;
    angles.template fill<T>(p, pos, gl, true);
    if (blk + gridDim.x < blocks) angles.positions(p, unit_of<LPR>(p, blk + gridDim.x).token, gl, pos);
    uint64_t c[4], s[4];
    angles.read(gl, c, s);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const int n = p.per_chunk[side];
      const int h0 = u.chunk * n, left = act ? min(n, p.heads[side] - h0) : 0;
      const int64_t yh = p.yh[side];
      uint8_t* y = p.y[side] + u.token * p.yt[side] + e0 * sizeof(T) + h0 * yh;
      uint64_t wt[4] = {};
      if constexpr (NORM) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const ulonglong2 w2 = s_w[side][h][gl];
          wt[2 * h] = w2.x, wt[2 * h + 1] = w2.y;
        }
      }
#pragma unroll 1
      for (int i = 0; i < n; i += U, y += U * yh) {
        rows.land();
        uint32_t wg[U][NW], wx[U][NW];
#pragma unroll
        for (int q = 0; q < U; ++q) {
          rows.read(q, 0, i + q < left, wg[q]);
          if constexpr (NORM) rows.read(q, 1, i + q < left, wx[q]);
        }
        rows.fetch(p, side0);
        rows.next();
#pragma unroll
        for (int q = 0; q < U; ++q) {
          const bool on = i + q < left;
          uint64_t g[4], gp[4];
          Vec8<T>::unpack(wg[q], g);
          partners<T, LPR, PAIRING>(wg[q], gp, gl, p.half, stage);
#pragma unroll
          for (int j = 0; j < 4; ++j) g[j] = fma2(g[j], c[j], mul2(gp[j], s[j]));
          if constexpr (NORM) {
            uint64_t v[4], h[4], t[4];
            Vec8<T>::unpack(wx[q], v);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              t[j] = mul2(v[j], v[j]);
              h[j] = mul2(g[j], wt[j]);
            }
            const float rs = rsqrtf(group_sum<LPR>(sum8(t)) * inv_d + p.eps), r = on ? rs : 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) t[j] = mul2(h[j], v[j]);
            const float m = -group_sum<LPR>(sum8(t)) * r * inv_d;  // -mean(h x r)
            const uint64_t rn = pair2(r, r), mm = pair2(m, m);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              v[j] = mul2(v[j], rn);  // 0 in a row that is not there
              gw[side][j] = fma2(g[j], v[j], gw[side][j]);
              g[j] = mul2(rn, fma2(v[j], mm, h[j]));
            }
          }
          if (on) {
            Vec8<T>::pack(g, wg[q]);
            store_words<NW>(y + q * yh, wg[q]);
          }
        }
      }
    }
  }
  if constexpr (NORM) {
    // the groups' sums in order, in the table's place
    uint64_t* s_gw = reinterpret_cast<uint64_t*>(s_table);  // [GROUPS][LPR * 4] pairs
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 4; ++j) s_gw[grp * (LPR * 4) + gl * 4 + j] = gw[side][j];
      __syncthreads();
      for (int col = threadIdx.x; col < p.d; col += kThreads) {
        float v = 0.f;
        for (int g = 0; g < GROUPS; ++g) v += reinterpret_cast<const float*>(s_gw)[g * (LPR * 8) + col];
        p.gw_part[(static_cast<int64_t>(blockIdx.x) * 2 + side) * p.d + col] = v;
      }
    }
  }
}

// gw[c] = sum over the blocks of part[block][side][c], each column by one warp:
// lanes take blocks in strides, then a fixed tree.
__global__ void __launch_bounds__(kThreads) k_rope_gw(const float* __restrict__ part, int blocks, int d, float* gwq,
                                                      float* gwk) {
  const int col = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (col >= 2 * d) return;
  float v = 0.f;
  for (int b = lane; b < blocks; b += 32) v += __ldcg(part + static_cast<int64_t>(b) * 2 * d + col);
  v = group_sum<32>(v);
  float* dst = col >= d ? gwk : gwq;
  if (lane == 0 && dst) dst[col >= d ? col - d : col] = v;
}

using Kern = void (*)(RopeParams);

template <typename T>
size_t ring_bytes(bool norm) {
  return norm ? Rows<T, 8, 2>::bytes() : Rows<T, 8, 1>::bytes();
}

template <typename T, int LPR, int PAIRING>
Kern pick_norm(bool bwd, bool norm) {
  if (bwd) return norm ? k_rope_bwd<T, LPR, PAIRING, true> : k_rope_bwd<T, LPR, PAIRING, false>;
  return norm ? k_rope_fwd<T, LPR, PAIRING, true> : k_rope_fwd<T, LPR, PAIRING, false>;
}
template <typename T, int LPR>
Kern pick_pairing(bool bwd, bool norm, int pairing) {
  switch (pairing) {
    case kInterleaved: return pick_norm<T, LPR, kInterleaved>(bwd, norm);
    case kHalf8: return pick_norm<T, LPR, kHalf8>(bwd, norm);
    case kHalf2:
      if constexpr (sizeof(T) == 2) return pick_norm<T, LPR, kHalf2>(bwd, norm);  // f32: one at a time
    default: return pick_norm<T, LPR, kHalf1>(bwd, norm);
  }
}
template <typename T>
Kern pick(int lpr, bool bwd, bool norm, int pairing) {
  switch (lpr) {
    case 4: return pick_pairing<T, 4>(bwd, norm, pairing);
    case 8: return pick_pairing<T, 8>(bwd, norm, pairing);
    case 16: return pick_pairing<T, 16>(bwd, norm, pairing);
    default: return pick_pairing<T, 32>(bwd, norm, pairing);
  }
}

int lanes_per_row(int d) {
  int l = 4;
  while (l * 8 < d) l *= 2;
  return l;
}

}  // namespace

sc_status rope_run(const RopeArgs& a) {
  const int64_t heads = a.heads_q + a.heads_k;
  const bool bwd = a.backward;
  const bool norm = a.w[0] || a.w[1];
  if (a.tokens == 0 || heads == 0) {
    if (bwd && norm) {
      for (int s = 0; s < 2; ++s)
        if (a.gw[s]) {
          const cudaError_t e = cudaMemsetAsync(a.gw[s], 0, sizeof(float) * a.head_dim, a.stream);
          if (e != cudaSuccess) return set_cuda_error(e, "rope gradient memset");
        }
    }
    return SC_OK;
  }
  const int64_t eb = a.dtype == SC_F32 ? 4 : 2;
  RopeParams p{};
  for (int s = 0; s < 2; ++s) {
    p.x[s] = static_cast<const uint8_t*>(a.x[s].data);
    p.xt[s] = a.x[s].token_stride * eb;
    p.xh[s] = a.x[s].head_stride * eb;
    p.gy[s] = static_cast<const uint8_t*>(a.gy[s].data);
    p.gt[s] = a.gy[s].token_stride * eb;
    p.gh[s] = a.gy[s].head_stride * eb;
    p.y[s] = static_cast<uint8_t*>(a.y[s].data);
    p.yt[s] = a.y[s].token_stride * eb;
    p.yh[s] = a.y[s].head_stride * eb;
    p.w[s] = a.w[s];
  }
  p.heads[0] = a.heads_q;
  p.heads[1] = a.heads_k;
  p.pos = a.pos;
  p.pos_stride = a.pos_stride;
  p.freq = a.freq;
  p.tokens = a.tokens;
  p.d = a.head_dim;
  p.half = a.rot_dim / 2;
  p.per = a.axes ? p.half / a.axes : 1;
  if (p.per < 1) p.per = 1;
  p.eps = a.eps;
  p.amp = a.amp;
  const int lpr = lanes_per_row(p.d), groups = kThreads / lpr;
  const int sms = device_sm_count();
  // A token's heads go to as many groups as fill the card (2048 threads an SM).
  const int most = a.heads_q > a.heads_k ? a.heads_q : a.heads_k;
  int64_t chunks = 2048ll * sms / (a.tokens * lpr);
  p.chunks = static_cast<int>(chunks < 1 ? 1 : chunks > most ? most : chunks);
  p.per_chunk[0] = (a.heads_q + p.chunks - 1) / p.chunks;
  p.per_chunk[1] = (a.heads_k + p.chunks - 1) / p.chunks;
  const int64_t steps = (a.tokens * p.chunks + groups - 1) / groups;
  const int pairing = a.interleaved ? kInterleaved : p.half % 8 == 0 ? kHalf8 : p.half % 2 == 0 ? kHalf2 : kHalf1;
  Kern k = a.dtype == SC_F32   ? pick<float>(lpr, bwd, norm, pairing)
           : a.dtype == SC_F16 ? pick<__half>(lpr, bwd, norm, pairing)
                               : pick<__nv_bfloat16>(lpr, bwd, norm, pairing);
  if (steps > 0x7fffffff) return set_error(SC_ERR_UNSUPPORTED, "too many tokens");
  if (!bwd) {
    const int64_t most_blocks = 4ll * sms;  // as many as are resident (f32 rows: three an SM)
    const unsigned grid = static_cast<unsigned>(steps < most_blocks ? steps : most_blocks);
    SC_LAUNCH("qk_norm_rope_fwd", a.stream, (k<<<grid, kThreads, 0, a.stream>>>(p)));
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SC_OK : set_cuda_error(e, "qk_norm_rope_fwd");
  }
  const size_t ring = a.dtype == SC_F32 ? ring_bytes<float>(norm) : ring_bytes<__half>(norm);
  // the ring lies beside up to 24 KB of static shared memory
  const sc_status set = kernel_setup(reinterpret_cast<const void*>(k), 96 * 1024, nullptr);
  if (set) return set;
  const int64_t resident = (norm ? 2ll : 3ll) * sms;
  const int blocks = static_cast<int>(steps < resident ? steps : resident);
  void* part = nullptr;
  if (norm) {
    const sc_status st = dev_alloc(&part, sizeof(float) * 2 * p.d * static_cast<size_t>(blocks), a.stream);
    if (st) return st;
    p.gw_part = static_cast<float*>(part);
  }
  SC_LAUNCH("qk_norm_rope_bwd", a.stream, (k<<<blocks, kThreads, ring, a.stream>>>(p)));
  cudaError_t e = cudaGetLastError();
  if (norm && e == cudaSuccess) {
    const int grid = (2 * p.d * 32 + kThreads - 1) / kThreads;
    SC_LAUNCH("qk_norm_rope_gw", a.stream,
              (k_rope_gw<<<grid, kThreads, 0, a.stream>>>(p.gw_part, blocks, p.d, a.gw[0], a.gw[1])));
    e = cudaGetLastError();
  }
  dev_free(part, a.stream);
  return e == cudaSuccess ? SC_OK : set_cuda_error(e, "qk_norm_rope_bwd");
}

}  // namespace sc
