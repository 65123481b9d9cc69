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
// memory bounds it.  A row lies in a group of LPR lanes, eight consecutive
// values (one 16-byte load of 16-bit types) a lane, so the norm is a sum over
// the group by shuffles; the partner of a pair comes from the lane that holds
// it.  A group takes one token's heads, or some of them, one after the other,
// four rows' loads in flight: a lane's angles are the same for all heads of a
// token, so it works them out once and keeps them, with the weights folded in,
// in registers (a table in shared memory, read for every row, made the kernel
// three times slower).
#include "sc_internal.cuh"

namespace sc {
namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------ 8 values --
template <typename T>
struct Vec8;
template <>
struct Vec8<__half> {
  static constexpr int kWords = 4;
  static __device__ __forceinline__ void unpack(const uint32_t (&w)[4], float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ void pack(const float (&x)[8], uint32_t (&w)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
};
template <>
struct Vec8<__nv_bfloat16> {
  static constexpr int kWords = 4;
  static __device__ __forceinline__ void unpack(const uint32_t (&w)[4], float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ void pack(const float (&x)[8], uint32_t (&w)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
};
template <>
struct Vec8<float> {
  static constexpr int kWords = 8;
  static __device__ __forceinline__ void unpack(const uint32_t (&w)[8], float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
  }
  static __device__ __forceinline__ void pack(const float (&x)[8], uint32_t (&w)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(x[i]);
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

template <int LPR>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// cos and sin of pos * f, times amp.  The product can be thousands of turns,
// and 32 bits of it would leave few for the fraction (1e-3 radians at position
// 32768, f = 1).  So it is formed in turns, c = f / 2 pi as a sum of two floats,
// and the product's rounding error is taken along by fma; a position that a
// float does not hold goes in two parts, a multiple of 4096 and a rest.  The
// rows are then f32 (EXACT: a few units in the last place) or 16-bit, for which
// the fast sine's 2^-20 is far below the output's rounding.
struct Turn {
  float c, ce;  // f / 2 pi, as a sum
};
__device__ __forceinline__ Turn turn_of(float f) {
  const float kInv2PiHi = 0x1.45f306p-3f;   // 1 / 2 pi to 24 bits
  const float kInv2PiLo = 0x1.b9391p-28f;   // the rest of it
  Turn r;
  r.c = f * kInv2PiHi;
  r.ce = fmaf(f, kInv2PiHi, -r.c) + f * kInv2PiLo;
  return r;
}
template <bool EXACT>
__device__ __forceinline__ float2 angle(int pos, Turn f, float amp) {
  const bool small = pos > -(1 << 24) && pos < (1 << 24);
  const int lo = small ? 0 : pos & 4095;
  const float xh = static_cast<float>(pos - lo);
  float t = xh * f.c;
  float e = fmaf(xh, f.c, -t) + xh * f.ce;
  t -= rintf(t);
  if (!small) [[unlikely]] {
    const float xl = static_cast<float>(lo), tl = xl * f.c;
    e += fmaf(xl, f.c, -tl) + xl * f.ce;
    t += tl - rintf(tl);
  }
  t += e;
  t -= rintf(t);
  float s, co;
  if constexpr (EXACT) sincospif(2.f * t, &s, &co);
  else __sincosf(6.283185307179586f * t, &s, &co);
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
  float* gw_part;            // backward with a norm: [blocks][D]
  const int* pos;
  int64_t pos_stride;        // elements between tokens
  const float* freq;
  int64_t tokens;
  int d, half, per;          // half = R / 2 pairs, per = pairs of one axis
  int chunks;                // groups that share a token's heads
  int per_chunk[2];          // heads of each
  int blocks_q;              // backward: blocks that take q, the others take k
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
__device__ __forceinline__ void partners(const uint32_t (&w)[Vec8<T>::kWords], float (&p)[8], int gl, int half,
                                         T* stage) {
  constexpr int NW = Vec8<T>::kWords;
  if constexpr (PAIRING == kInterleaved) {
    float x[8];
    Vec8<T>::unpack(w, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = x[j ^ 1];
  } else if constexpr (PAIRING == kHalf8) {
    const int step = half >> 3;
    const int from = gl < step ? gl + step : (gl < 2 * step ? gl - step : gl);
    uint32_t o[NW];
#pragma unroll
    for (int i = 0; i < NW; ++i) o[i] = __shfl_sync(0xffffffffu, w[i], from, LPR);
    Vec8<T>::unpack(o, p);
  } else {
    T* row = stage + ((threadIdx.x & 31) / LPR) * (LPR * 8);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < NW / 4; ++i)
      reinterpret_cast<uint4*>(row + gl * 8)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    __syncwarp();
    if constexpr (PAIRING == kHalf2 && sizeof(T) == 2) {
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = gl * 8 + 2 * j;
        o[j] = *reinterpret_cast<const uint32_t*>(row + (e < half ? e + half : (e < 2 * half ? e - half : e)));
      }
      Vec8<T>::unpack(o, p);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = gl * 8 + j;
        p[j] = static_cast<float>(row[e < half ? e + half : (e < 2 * half ? e - half : e)]);
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
// sine has the sign of the second member's formula, and `back` turns back.  The
// group's lanes work out the token's pairs between them, four each, and put each
// under both its values in `table`, value e of the warp's group g at
// [e % 8][g * LPR + e / 8]: a lane then reads its eight without conflicts.
template <int LPR, int PAIRING>
struct Angles {
  Turn f[4];
  int axis[4];
  float2* mine;
  __device__ __forceinline__ Angles(const RopeParams& p, int gl, float2* table) {
    mine = table + ((threadIdx.x & 31) / LPR) * LPR;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int pair = gl + i * LPR;
      f[i] = turn_of(pair < p.half ? __ldg(p.freq + pair) : 0.f);
      axis[i] = (pair >= p.per) + (pair >= 2 * p.per) + (pair >= 3 * p.per);
    }
    for (int j = 0; j < 8; ++j) mine[j * 32 + gl] = make_float2(1.f, 0.f);  // values that do not turn
    __syncwarp();
  }
  template <typename T>
  __device__ __forceinline__ void fill(const RopeParams& p, int64_t t, int gl, bool back) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int pair = gl + i * LPR;
      if (pair < p.half) {
        float2 cs = angle<sizeof(T) == 4>(__ldg(p.pos + t * p.pos_stride + axis[i]), f[i], p.amp);
        if (back) cs.y = -cs.y;
        const int e0 = PAIRING == kInterleaved ? 2 * pair : pair, e1 = PAIRING == kInterleaved ? e0 + 1 : pair + p.half;
        mine[(e0 & 7) * 32 + (e0 >> 3)] = make_float2(cs.x, -cs.y);
        mine[(e1 & 7) * 32 + (e1 >> 3)] = cs;
      }
    }
    __syncwarp();
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

constexpr int kRows = 4;  // rows in flight

template <typename T, int LPR, int PAIRING, bool NORM>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 3 : 4) k_rope_fwd(const RopeParams p) {
  constexpr int NW = Vec8<T>::kWords, GROUPS = kThreads / LPR, U = sizeof(T) == 4 ? kRows / 2 : kRows;
  __shared__ __align__(16) T s_stage[PAIRING >= kHalf2 ? kThreads * 8 : 8];
  __shared__ float2 s_table[kThreads * 8];
  __shared__ __align__(16) float s_w[NORM ? 2 : 1][2][NORM ? LPR * 8 : 4];  // [side][a value's, its partner's][value]
  T* stage = s_stage + (PAIRING >= kHalf2 ? (threadIdx.x >> 5) * 256 : 0);
  const int gl = threadIdx.x % LPR;
  const int e0 = gl * 8;
  const float inv_d = 1.f / static_cast<float>(p.d);
  if constexpr (NORM) {
    for (int i = threadIdx.x; i < 4 * LPR * 8; i += kThreads) {
      const int side = i / (2 * LPR * 8), which = i / (LPR * 8) & 1, e = i % (LPR * 8);
      const int o = which ? partner_of<PAIRING>(e, p.half) : e;
      s_w[side][which][e] = p.heads[side] && o < p.d ? __ldg(p.w[side] + o) : 0.f;
    }
    __syncthreads();
  }
  Angles<LPR, PAIRING> angles(p, gl, s_table + (threadIdx.x >> 5) * 256);
  const int64_t blocks = (p.tokens * p.chunks + GROUPS - 1) / GROUPS;
#pragma unroll 1
  for (int64_t blk = blockIdx.x; blk < blocks; blk += gridDim.x) {
    const Unit u = unit_of<LPR>(p, blk);
    const bool act = u.on && e0 < p.d;
    angles.template fill<T>(p, u.token, gl, false);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const int n = p.per_chunk[side];
      float a[8], b[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 cs = angles.mine[j * 32 + gl];
        a[j] = cs.x;
        b[j] = cs.y;
        if constexpr (NORM) {
          a[j] *= s_w[side][0][e0 + j];
          b[j] *= s_w[side][1][e0 + j];
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
          float v[8], vp[8];
          Vec8<T>::unpack(w[q], v);
          partners<T, LPR, PAIRING>(w[q], vp, gl, p.half, stage);
          float rn = 1.f;
          if constexpr (NORM) {
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
            rn = rsqrtf(group_sum<LPR>(ss) * inv_d + p.eps);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            v[j] = fmaf(v[j], a[j], vp[j] * b[j]);
            if constexpr (NORM) v[j] *= rn;
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

// The gradient.  The first blocks_q blocks walk q's units, the others k's, so
// that each keeps its sum of one weight's gradient in registers and writes it
// once: [block][D] in gw_part, summed in order by k_rope_gw (the same result
// every time).
template <typename T, int LPR, int PAIRING, bool NORM>
__global__ void __launch_bounds__(kThreads, 3) k_rope_bwd(const RopeParams p) {
  constexpr int NW = Vec8<T>::kWords, GROUPS = kThreads / LPR, U = sizeof(T) == 4 || NORM ? kRows / 2 : kRows;
  __shared__ __align__(16) T s_stage[PAIRING >= kHalf2 ? kThreads * 8 : 8];
  __shared__ float2 s_table[kThreads * 8];
  T* stage = s_stage + (PAIRING >= kHalf2 ? (threadIdx.x >> 5) * 256 : 0);
  const int gl = threadIdx.x % LPR, grp = threadIdx.x / LPR;
  const int e0 = gl * 8;
  const int side = static_cast<int>(blockIdx.x) >= p.blocks_q;
  const int first = side ? p.blocks_q : 0, count = side ? gridDim.x - p.blocks_q : p.blocks_q;
  const int n = side ? p.per_chunk[1] : p.per_chunk[0], heads = side ? p.heads[1] : p.heads[0];
  const int64_t gh = side ? p.gh[1] : p.gh[0], xh = side ? p.xh[1] : p.xh[0], yh = side ? p.yh[1] : p.yh[0];
  float gw[8] = {}, wt[8] = {};
  if constexpr (NORM) {
#pragma unroll
    for (int j = 0; j < 8; ++j) wt[j] = e0 + j < p.d ? __ldg((side ? p.w[1] : p.w[0]) + e0 + j) : 0.f;
  }
  const float inv_d = 1.f / static_cast<float>(p.d);
  Angles<LPR, PAIRING> angles(p, gl, s_table + (threadIdx.x >> 5) * 256);
  const int64_t blocks = (p.tokens * p.chunks + GROUPS - 1) / GROUPS;
#pragma unroll 1
  for (int64_t blk = static_cast<int64_t>(blockIdx.x) - first; blk < blocks; blk += count) {
    const Unit u = unit_of<LPR>(p, blk);
    const bool act = u.on && e0 < p.d;
    angles.template fill<T>(p, u.token, gl, true);
    float c[8], s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 cs = angles.mine[j * 32 + gl];
      c[j] = cs.x;
      s[j] = cs.y;
    }
    const int h0 = u.chunk * n, left = act ? min(n, heads - h0) : 0;
    const uint8_t* gy = (side ? p.gy[1] : p.gy[0]) + u.token * (side ? p.gt[1] : p.gt[0]) + e0 * sizeof(T) + h0 * gh;
    const uint8_t* x = (side ? p.x[1] : p.x[0]) + u.token * (side ? p.xt[1] : p.xt[0]) + e0 * sizeof(T) + h0 * xh;
    uint8_t* y = (side ? p.y[1] : p.y[0]) + u.token * (side ? p.yt[1] : p.yt[0]) + e0 * sizeof(T) + h0 * yh;
    for (int i = 0; i < n; i += U, gy += U * gh, x += U * xh, y += U * yh) {
      uint32_t wg[U][NW], wx[U][NW];
#pragma unroll
      for (int q = 0; q < U; ++q) {
#pragma unroll
        for (int k = 0; k < NW; ++k) wg[q][k] = wx[q][k] = 0u;
        if (i + q < left) {
          load_words<NW>(gy + q * gh, wg[q]);
          if constexpr (NORM) load_words<NW>(x + q * xh, wx[q]);
        }
      }
#pragma unroll
      for (int q = 0; q < U; ++q) {
        const bool on = i + q < left;
        float g[8], gp[8];
        Vec8<T>::unpack(wg[q], g);
        partners<T, LPR, PAIRING>(wg[q], gp, gl, p.half, stage);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = fmaf(g[j], c[j], gp[j] * s[j]);
        if constexpr (NORM) {
          float v[8], ss = 0.f, hx = 0.f;
          Vec8<T>::unpack(wx[q], v);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            ss = fmaf(v[j], v[j], ss);
            hx = fmaf(g[j] * wt[j], v[j], hx);
          }
          const float rn = rsqrtf(group_sum<LPR>(ss) * inv_d + p.eps);
          const float m = group_sum<LPR>(hx) * rn * inv_d;  // mean(h x r)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float xn = v[j] * rn;
            if (on) gw[j] = fmaf(g[j], xn, gw[j]);
            g[j] = rn * (g[j] * wt[j] - xn * m);
          }
        }
        if (on) {
          Vec8<T>::pack(g, wg[q]);
          store_words<NW>(y + q * yh, wg[q]);
        }
      }
    }
  }
  if constexpr (NORM) {
    // the groups' sums in order, in the table's place
    float* s_gw = reinterpret_cast<float*>(s_table);  // [GROUPS][LPR * 8]
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) s_gw[grp * (LPR * 8) + e0 + j] = gw[j];
    __syncthreads();
    for (int col = threadIdx.x; col < p.d; col += kThreads) {
      float v = 0.f;
      for (int g = 0; g < GROUPS; ++g) v += s_gw[g * (LPR * 8) + col];
      p.gw_part[static_cast<int64_t>(blockIdx.x) * p.d + col] = v;
    }
  }
}

// gw[c] = sum over its side's blocks of part[block][c], each column by one warp:
// lanes take blocks in strides, then a fixed tree.
__global__ void __launch_bounds__(kThreads) k_rope_gw(const float* __restrict__ part, int blocks_q, int blocks, int d,
                                                      float* gwq, float* gwk) {
  const int col = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (col >= 2 * d) return;
  const bool k = col >= d;
  const int c = k ? col - d : col;
  float v = 0.f;
  for (int b = (k ? blocks_q : 0) + lane; b < (k ? blocks : blocks_q); b += 32)
    v += __ldg(part + static_cast<int64_t>(b) * d + c);
  v = group_sum<32>(v);
  float* dst = k ? gwk : gwq;
  if (lane == 0 && dst) dst[c] = v;
}

using Kern = void (*)(RopeParams);

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
    const int64_t most_blocks = 4ll * sms;  // as many as are resident
    SC_LAUNCH("qk_norm_rope_fwd", a.stream, (k<<<static_cast<unsigned>(steps < most_blocks ? steps : most_blocks), kThreads, 0, a.stream>>>(p)));
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SC_OK : set_cuda_error(e, "qk_norm_rope_fwd");
  }
  // blocks by the sides' heads, one at least for each that has some
  const int64_t cap = 3ll * sms;
  int64_t nb[2] = {0, 0};
  for (int s = 0; s < 2; ++s)
    if (p.heads[s]) {
      nb[s] = (cap * p.heads[s] + heads / 2) / heads;
      nb[s] = nb[s] < 1 ? 1 : nb[s] > steps ? steps : nb[s];
    }
  p.blocks_q = static_cast<int>(nb[0]);
  const int blocks = static_cast<int>(nb[0] + nb[1]);
  void* part = nullptr;
  if (norm) {
    const sc_status st = dev_alloc(&part, sizeof(float) * p.d * static_cast<size_t>(blocks), a.stream);
    if (st) return st;
    p.gw_part = static_cast<float*>(part);
  }
  SC_LAUNCH("qk_norm_rope_bwd", a.stream, (k<<<blocks, kThreads, 0, a.stream>>>(p)));
  cudaError_t e = cudaGetLastError();
  if (norm && e == cudaSuccess) {
    const int grid = (2 * p.d * 32 + kThreads - 1) / kThreads;
    SC_LAUNCH("qk_norm_rope_gw", a.stream,
              (k_rope_gw<<<grid, kThreads, 0, a.stream>>>(p.gw_part, p.blocks_q, blocks, p.d, a.gw[0], a.gw[1])));
    e = cudaGetLastError();
  }
  dev_free(part, a.stream);
  return e == cudaSuccess ? SC_OK : set_cuda_error(e, "qk_norm_rope_bwd");
}

}  // namespace sc
