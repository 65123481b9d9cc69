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
// it.  The angles of a token serve all its heads: a block computes them once
// for its tokens and keeps them in shared memory.
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
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
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
    reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}

template <int LPR>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// cos and sin of pos * f, times amp.  The product can be thousands of turns,
// and 32 bits of it would leave few for the fraction (1e-3 radians at position
// 32768, f = 1).  So it is formed in turns and in parts whose whole turns drop
// out exactly: c = f / 2 pi as a sum of two floats, the position as a multiple
// of 4096 and a rest, and the rounding error of each product by fma.
__device__ __forceinline__ float2 angle(int pos, float f, float amp) {
  const float kInv2PiHi = 0x1.45f306p-3f;   // 1 / 2 pi to 24 bits
  const float kInv2PiLo = 0x1.b9391p-28f;   // the rest of it
  const float c = f * kInv2PiHi;
  const float ce = fmaf(f, kInv2PiHi, -c) + f * kInv2PiLo;
  const int lo = pos & 4095;
  const float xh = static_cast<float>(pos - lo), xl = static_cast<float>(lo);
  const float th = xh * c, tl = xl * c;
  const float eh = fmaf(xh, c, -th) + xh * ce, el = fmaf(xl, c, -tl) + xl * ce;
  float t = (th - rintf(th)) + (tl - rintf(tl));
  t += eh + el;
  t -= rintf(t);
  float s, co;
  sincospif(2.f * t, &s, &co);
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
  float* gw_part;            // backward with a norm: [blocks][2][D]
  const int* pos;
  int64_t pos_stride;        // elements between tokens
  const float* freq;
  int64_t tokens;
  int d, half, per;          // half = R / 2 pairs, per = pairs of one axis
  int nt;                    // tokens of a block's step
  float eps, amp;
};

// Partner values (the other member of the pair) of this lane's eight, pairs
// (i, i + half): by shuffles where half is a multiple of 8 (a whole lane's
// values move), else through `stage`, the warp's rows in shared memory.
template <typename T, int LPR, bool ALIGNED>
__device__ __forceinline__ void partner_half(const uint32_t (&w)[Vec8<T>::kWords], float (&p)[8], int gl, int half,
                                             T* stage) {
  constexpr int NW = Vec8<T>::kWords;
  if constexpr (ALIGNED) {
    const int step = half >> 3;
    const int from = gl < step ? gl + step : (gl < 2 * step ? gl - step : gl);
    uint32_t o[NW];
#pragma unroll
    for (int i = 0; i < NW; ++i) o[i] = __shfl_sync(0xffffffffu, w[i], from, LPR);
    Vec8<T>::unpack(o, p);
  } else {
    const int lane = threadIdx.x & 31;
    T* row = stage + (lane / LPR) * (LPR * 8);
    __syncwarp();
    store_words<NW>(row + gl * 8, w);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = gl * 8 + j;
      const int o = e < half ? e + half : (e < 2 * half ? e - half : e);
      p[j] = static_cast<float>(row[o]);
    }
  }
}

// The angles of a step's tokens into shared memory: [nt][half].
__device__ __forceinline__ void fill_angles(const RopeParams& p, int64_t t0, float2* s_cs) {
  const int n = static_cast<int>(min(static_cast<int64_t>(p.nt), p.tokens - t0)) * p.half;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int t = i / p.half, pair = i - t * p.half;
    const int pos = __ldg(p.pos + (t0 + t) * p.pos_stride + pair / p.per);
    s_cs[i] = angle(pos, __ldg(p.freq + pair), p.amp);
  }
}

// Turns z (this lane's values e0 .. e0 + 7) by its angles, `sign` -1 for the
// transpose.  zp: the partners of z.
template <bool ILV>
__device__ __forceinline__ void turn(float (&y)[8], const float (&z)[8], const float (&zp)[8], const float2* cs,
                                     int e0, int half, float sign) {
  if constexpr (ILV) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const int pair = (e0 + j) >> 1;
      const float2 c = pair < half ? cs[pair] : make_float2(1.f, 0.f);
      y[j] = z[j] * c.x - sign * z[j + 1] * c.y;
      y[j + 1] = z[j + 1] * c.x + sign * z[j] * c.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = e0 + j;
      const bool first = e < half;
      const int pair = first ? e : e - half;
      const float2 c = pair < half ? cs[pair] : make_float2(1.f, 0.f);
      y[j] = z[j] * c.x + (first ? -sign : sign) * zp[j] * c.y;
    }
  }
}

// One block's step covers nt tokens: rows of q, then rows of k.
template <typename T, int LPR, bool ILV, bool ALIGNED, bool NORM>
__global__ void __launch_bounds__(kThreads) k_rope_fwd(const RopeParams p) {
  constexpr int NW = Vec8<T>::kWords, GROUPS = kThreads / LPR;
  extern __shared__ float2 s_cs[];
  T* stage = reinterpret_cast<T*>(s_cs + ((p.nt * p.half + 1) & ~1)) + (threadIdx.x >> 5) * 256;
  const int gl = threadIdx.x % LPR, grp = threadIdx.x / LPR;
  const int e0 = gl * 8;
  const bool act = e0 < p.d;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.nt;
  const int nt = static_cast<int>(min(static_cast<int64_t>(p.nt), p.tokens - t0));
  fill_angles(p, t0, s_cs);
  __syncthreads();
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const int heads = p.heads[side];
    if (heads == 0) continue;
    const int rows = nt * heads;
    float w[8], wp[8];
    if constexpr (NORM) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = e0 + j;
        const int o = e < p.half ? e + p.half : (e < 2 * p.half ? e - p.half : e);
        w[j] = e < p.d ? __ldg(p.w[side] + e) : 0.f;
        wp[j] = o < p.d ? __ldg(p.w[side] + o) : 0.f;
      }
    }
    // whole warps stay in the loop: the shuffles below are warp-wide
    for (int r0 = 0; r0 < rows; r0 += GROUPS) {
      const int r = r0 + grp;
      const bool on = r < rows && act;
      const int t = on ? r / heads : 0, h = on ? r - t * heads : 0;
      uint32_t a[NW] = {};
      if (on) load_words<NW>(p.x[side] + (t0 + t) * p.xt[side] + h * p.xh[side] + e0 * sizeof(T), a);
      float x[8], xp[8] = {}, y[8];
      Vec8<T>::unpack(a, x);
      if constexpr (!ILV) partner_half<T, LPR, ALIGNED>(a, xp, gl, p.half, stage);
      if constexpr (NORM) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
        const float rn = 1.f / sqrtf(group_sum<LPR>(ss) / static_cast<float>(p.d) + p.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[j] *= rn * w[j];
          if constexpr (!ILV) xp[j] *= rn * wp[j];
        }
      }
      turn<ILV>(y, x, xp, s_cs + t * p.half, e0, p.half, 1.f);
      if (on) {
        Vec8<T>::pack(y, a);
        store_words<NW>(p.y[side] + (t0 + t) * p.yt[side] + h * p.yh[side] + e0 * sizeof(T), a);
      }
    }
  }
}

// The gradient.  Blocks walk the steps grid-wide, so that each keeps its sum of
// the weights' gradient in registers and writes it once: [block][2][D] in
// gw_part, summed in order by k_rope_gw (the same result every time).
template <typename T, int LPR, bool ILV, bool ALIGNED, bool NORM>
__global__ void __launch_bounds__(kThreads) k_rope_bwd(const RopeParams p) {
  constexpr int NW = Vec8<T>::kWords, GROUPS = kThreads / LPR;
  extern __shared__ float2 s_cs[];
  T* stage = reinterpret_cast<T*>(s_cs + ((p.nt * p.half + 1) & ~1)) + (threadIdx.x >> 5) * 256;
  const int gl = threadIdx.x % LPR, grp = threadIdx.x / LPR;
  const int e0 = gl * 8;
  const bool act = e0 < p.d;
  float gw[2][8] = {};
  float w[2][8];
  if constexpr (NORM) {
#pragma unroll
    for (int side = 0; side < 2; ++side)
#pragma unroll
      for (int j = 0; j < 8; ++j) w[side][j] = p.heads[side] && e0 + j < p.d ? __ldg(p.w[side] + e0 + j) : 0.f;
  }
  const int64_t steps = (p.tokens + p.nt - 1) / p.nt;
  for (int64_t s = blockIdx.x; s < steps; s += gridDim.x) {
    const int64_t t0 = s * p.nt;
    const int nt = static_cast<int>(min(static_cast<int64_t>(p.nt), p.tokens - t0));
    __syncthreads();  // the previous step's angles have been read
    fill_angles(p, t0, s_cs);
    __syncthreads();
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const int heads = p.heads[side];
      if (heads == 0) continue;
      const int rows = nt * heads;
      for (int r0 = 0; r0 < rows; r0 += GROUPS) {
        const int r = r0 + grp;
        const bool on = r < rows && act;
        const int t = on ? r / heads : 0, h = on ? r - t * heads : 0;
        uint32_t a[NW] = {}, b[NW] = {};
        if (on) {
          load_words<NW>(p.gy[side] + (t0 + t) * p.gt[side] + h * p.gh[side] + e0 * sizeof(T), a);
          if constexpr (NORM) load_words<NW>(p.x[side] + (t0 + t) * p.xt[side] + h * p.xh[side] + e0 * sizeof(T), b);
        }
        float gy[8], gp[8] = {}, g[8];
        Vec8<T>::unpack(a, gy);
        if constexpr (!ILV) partner_half<T, LPR, ALIGNED>(a, gp, gl, p.half, stage);
        turn<ILV>(g, gy, gp, s_cs + t * p.half, e0, p.half, -1.f);
        if constexpr (NORM) {
          float x[8];
          Vec8<T>::unpack(b, x);
          float ss = 0.f, hx = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            ss = fmaf(x[j], x[j], ss);
            hx = fmaf(g[j] * w[side][j], x[j], hx);
          }
          const float inv_d = 1.f / static_cast<float>(p.d);
          const float rn = 1.f / sqrtf(group_sum<LPR>(ss) * inv_d + p.eps);
          const float m = group_sum<LPR>(hx) * rn * inv_d;  // mean(h x r)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float xn = x[j] * rn;
            // rows past the end hold zeros, and the masked add keeps NaN weights of idle lanes out
            if (on) gw[side][j] = fmaf(g[j], xn, gw[side][j]);
            g[j] = rn * (g[j] * w[side][j] - xn * m);
          }
        }
        if (on) {
          Vec8<T>::pack(g, a);
          store_words<NW>(p.y[side] + (t0 + t) * p.yt[side] + h * p.yh[side] + e0 * sizeof(T), a);
        }
      }
    }
  }
  if constexpr (NORM) {
    // groups' sums in order, one side at a time
    float* s_gw = reinterpret_cast<float*>(s_cs);  // [GROUPS][LPR * 8], sized by the launch
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) s_gw[grp * (LPR * 8) + e0 + j] = gw[side][j];
      __syncthreads();
      for (int c = threadIdx.x; c < p.d; c += kThreads) {
        float v = 0.f;
        for (int g = 0; g < GROUPS; ++g) v += s_gw[g * (LPR * 8) + c];
        p.gw_part[(static_cast<int64_t>(blockIdx.x) * 2 + side) * p.d + c] = v;
      }
    }
  }
}

// gw[side][c] = sum over blocks of part[block][side][c], each column by one
// warp: lanes take blocks in strides, then a fixed tree.
__global__ void __launch_bounds__(kThreads) k_rope_gw(const float* __restrict__ part, int blocks, int d, float* gwq,
                                                      float* gwk) {
  const int col = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (col >= 2 * d) return;
  float v = 0.f;
  for (int b = lane; b < blocks; b += 32) v += __ldg(part + static_cast<int64_t>(b) * 2 * d + col);
  v = group_sum<32>(v);
  float* dst = col < d ? gwq : gwk;
  if (lane == 0 && dst) dst[col < d ? col : col - d] = v;
}

using Kern = void (*)(RopeParams);

template <typename T, int LPR, bool ILV, bool ALIGNED>
Kern pick_norm(bool bwd, bool norm) {
  if (bwd) return norm ? k_rope_bwd<T, LPR, ILV, ALIGNED, true> : k_rope_bwd<T, LPR, ILV, ALIGNED, false>;
  return norm ? k_rope_fwd<T, LPR, ILV, ALIGNED, true> : k_rope_fwd<T, LPR, ILV, ALIGNED, false>;
}
template <typename T, int LPR>
Kern pick_layout(bool bwd, bool norm, bool ilv, bool aligned) {
  if (ilv) return pick_norm<T, LPR, true, true>(bwd, norm);
  return aligned ? pick_norm<T, LPR, false, true>(bwd, norm) : pick_norm<T, LPR, false, false>(bwd, norm);
}
template <typename T>
Kern pick(int lpr, bool bwd, bool norm, bool ilv, bool aligned) {
  switch (lpr) {
    case 2: return pick_layout<T, 2>(bwd, norm, ilv, aligned);
    case 4: return pick_layout<T, 4>(bwd, norm, ilv, aligned);
    case 8: return pick_layout<T, 8>(bwd, norm, ilv, aligned);
    case 16: return pick_layout<T, 16>(bwd, norm, ilv, aligned);
    default: return pick_layout<T, 32>(bwd, norm, ilv, aligned);
  }
}

int lanes_per_row(int d) {
  int l = 2;
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
  // tokens of a step: enough rows for four passes of the block's groups, but
  // first enough blocks for the card (a few tokens: one block each)
  int64_t nt = (4 * groups + heads - 1) / heads;
  const int64_t most = a.tokens / (4 * sms);
  if (nt > most) nt = most;
  if (nt < 1) nt = 1;
  while (nt > 1 && nt * p.half * 8 > 16384) --nt;
  p.nt = static_cast<int>(nt);
  const bool aligned = p.half % 8 == 0;
  size_t smem = static_cast<size_t>(p.nt) * p.half * sizeof(float2);
  smem = (smem + 15) & ~size_t(15);
  if (!a.interleaved && !aligned) smem += kThreads / 32 * 256 * static_cast<size_t>(eb);
  if (bwd && norm && smem < static_cast<size_t>(groups) * lpr * 8 * 4) smem = static_cast<size_t>(groups) * lpr * 8 * 4;
  const int64_t steps = (a.tokens + nt - 1) / nt;
  Kern k = a.dtype == SC_F32   ? pick<float>(lpr, bwd, norm, a.interleaved, aligned)
           : a.dtype == SC_F16 ? pick<__half>(lpr, bwd, norm, a.interleaved, aligned)
                               : pick<__nv_bfloat16>(lpr, bwd, norm, a.interleaved, aligned);
  if (steps > 0x7fffffff) return set_error(SC_ERR_UNSUPPORTED, "too many tokens");
  if (!bwd) {
    SC_LAUNCH("qk_norm_rope_fwd", a.stream, (k<<<static_cast<unsigned>(steps), kThreads, smem, a.stream>>>(p)));
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SC_OK : set_cuda_error(e, "qk_norm_rope_fwd");
  }
  const int64_t cap = 6ll * sms;
  const int blocks = static_cast<int>(steps < cap ? steps : cap);
  void* part = nullptr;
  if (norm) {
    const sc_status st = dev_alloc(&part, sizeof(float) * 2 * p.d * static_cast<size_t>(blocks), a.stream);
    if (st) return st;
    p.gw_part = static_cast<float*>(part);
  }
  SC_LAUNCH("qk_norm_rope_bwd", a.stream, (k<<<blocks, kThreads, smem, a.stream>>>(p)));
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
