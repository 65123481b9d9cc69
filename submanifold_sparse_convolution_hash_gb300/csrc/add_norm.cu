// The residual's addition and the norm of rows, with 16-bit or 8-bit output, and
// the gradients.
//
// One pass over memory: a row's values stay in the registers of the lanes (up to
// 1024 channels: at most a warp a row) or of the block that hold it, its sums cross
// them once, and the next rows' loads are issued before this row's sums.  y is a
// positive factor r = 1 / sqrt(mean h^2 + eps) times w h, so the largest |y| of the
// 8-bit form is r max |w h| and rides along with the sum of squares.
//
// Bound by memory: 32,768 rows of 4,096, bf16, residual, to 8 bits 140 us (6.69 TB/s of the 6.78 that a
// copy reaches), gradients of 480,000 rows of 256, f16, 162 (6.07).  f32, cold, floors beside: 480,000 rows
// of 256 forward 326 us (290), to 8 bits 247 (236), gradients 300 (290); 32,768 of 4,096 350 (317),
// 287 (257), 325 (317).
#include <cmath>
#include <type_traits>

#include "sc_internal.cuh"
#include "tc_ptx.cuh"

namespace sc {
namespace {

constexpr float kE4m3Max = 448.f;
// Rows ahead of a wide form's, each with its two or three tensors.
constexpr int kRing = 3;
constexpr size_t kRingMost = 200 * 1024;  // a gradient's row of 16,384 f32 channels takes 192 KB: one slot

template <typename T>
struct Vec8 {
  uint4 raw[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Vec8<T> ld_vec(const T* p) {
  Vec8<T> v;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) v.raw[i] = *(reinterpret_cast<const uint4*>(p) + i);
  return v;
}
template <typename T>
__device__ __forceinline__ Vec8<T> zero_vec() {
  Vec8<T> v;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) v.raw[i] = make_uint4(0, 0, 0, 0);
  return v;
}
template <typename T>
__device__ __forceinline__ void unpack(const Vec8<T>& v, float (&f)[8]) {
  if constexpr (std::is_same_v<T, float>) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f[4 * i] = __uint_as_float(v.raw[i].x);
      f[4 * i + 1] = __uint_as_float(v.raw[i].y);
      f[4 * i + 2] = __uint_as_float(v.raw[i].z);
      f[4 * i + 3] = __uint_as_float(v.raw[i].w);
    }
  } else {
    const uint32_t w[4] = {v.raw[0].x, v.raw[0].y, v.raw[0].z, v.raw[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 t;
      if constexpr (std::is_same_v<T, __half>) t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      else t = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
}
template <typename T>
__device__ __forceinline__ void st_vec(T* p, const float (&f)[8]) {
  if constexpr (std::is_same_v<T, float>) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same_v<T, __half>) {
        const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
// Two values as e4m3, the first in the low byte; beyond 448 they become 448.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The sum of a and, with MAX, the largest of b over a row's lanes: a subgroup of G lanes, or
// (G = 0) the block.  A block's values cross in shared memory; `turn` alternates two
// places, so that one barrier a row is enough.
template <int G, bool MAX>
__device__ __forceinline__ void row_reduce(float& a, float& b, float2 (*s_red)[32], int turn) {
  constexpr int W = G == 0 ? 32 : G;
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    const float t = __shfl_xor_sync(0xffffffffu, b, o);
    b = MAX ? fmaxf(b, t) : b + t;
  }
  if constexpr (G == 0) {
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) s_red[turn][threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    float2 v = lane < warps ? s_red[turn][lane] : make_float2(0.f, 0.f);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
      const float t = __shfl_xor_sync(0xffffffffu, v.y, o);
      v.y = MAX ? fmaxf(v.y, t) : v.y + t;
    }
    a = v.x;
    b = v.y;
  }
}

// Eight weights of the vector `at`: kept in registers over the rows up to two vectors a
// lane, else read again for each row (they stay in L1).  The narrow gradients read them again
// too: their registers are worth more (524,288 rows of 256, bf16: 172 us, kept 215).
__device__ __forceinline__ void ld_w(const float* w, int at, float (&f)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(w + at * 8), b = *reinterpret_cast<const float4*>(w + at * 8 + 4);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
  f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
template <int NV, bool kKept = (NV <= 2)>
struct Weights {
  float f[kKept ? NV : 1][8];
  const float* w;
  int lane, lanes, nvec;
  __device__ __forceinline__ Weights(const float* w_, int lane_, int lanes_, int nvec_)
      : w(w_), lane(lane_), lanes(lanes_), nvec(nvec_) {
    if constexpr (kKept) {
#pragma unroll
      for (int v = 0; v < NV; ++v) read(v, f[v]);
    }
  }
  __device__ __forceinline__ void read(int v, float (&t)[8]) const {
    const int at = lane + v * lanes;
    if (w && at < nvec) {
      ld_w(w, at, t);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = 1.f;
    }
  }
  __device__ __forceinline__ void get(int v, float (&t)[8]) const {
    if constexpr (kKept) {
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = f[v][i];
    } else {
      read(v, t);
    }
  }
};

// Whether the next row's loads are issued before this row's sums: where a lane has one or
// two 16-byte loads a tensor of its own row in flight.
template <typename T, int NV>
constexpr bool loads_ahead() {
  return NV * sizeof(T) <= 4;
}

struct NormParams {
  const void *x, *res, *gout;
  void *sum, *out;
  int64_t ldx, ldres, ldgout, ldsum, ldout;
  float* scale;
  const float* w;
  float* part;  // backward: [blocks, channels], or null
  int64_t rows;
  int channels;
  float eps;
  int ring;     // wide gradients: rows ahead
  int* status;
};

// The rest of a row once its sums are there: the sum, and y in the output's type.
template <typename T, int NV, bool E4M3>
__device__ __forceinline__ void store_row(const NormParams& p, const Weights<NV>& w, const float (&h)[NV][8], float ss,
                                          float top, int64_t row, int lane, int lanes, int nvec) {
  if (p.sum) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int at = lane + v * lanes;
      if (at < nvec) st_vec(static_cast<T*>(p.sum) + row * p.ldsum + at * 8, h[v]);
    }
  }
  const float r = p.w ? rsqrtf(ss / static_cast<float>(p.channels) + p.eps) : 1.f;
  if constexpr (E4M3) {
    float s = top * r / kE4m3Max;
    if (s < 0x1p-126f) s = 0.f;
    // squares past fp32 (r = 0, and top r 0 or NaN): no value, and a scale that says so; a NaN stays one
    if (p.w && !(ss < INFINITY)) s = ss;
    const float f = s > 0.f ? 1.f / s : 0.f;
    if (lane == 0) p.scale[row] = s;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int at = lane + v * lanes;
      if (at >= nvec) continue;
      float y[8];
      w.get(v, y);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] *= h[v][i] * r * f;
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + row * p.ldout + at * 8) =
          make_uint2(e4m3x2(y[0], y[1]) | (e4m3x2(y[2], y[3]) << 16), e4m3x2(y[4], y[5]) | (e4m3x2(y[6], y[7]) << 16));
    }
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int at = lane + v * lanes;
      if (at >= nvec) continue;
      float y[8];
      w.get(v, y);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] *= h[v][i] * r;
      st_vec(static_cast<T*>(p.out) + row * p.ldout + at * 8, y);
    }
  }
}

constexpr int kBlock = 256;  // of the forms in which lanes hold a row

// A row is held by G lanes, or by the block (G = 0, at most 256 threads), vectors of 8 values lane,
// lane + G, ...  Three blocks an SM: 32,768 rows of 4,096 to 8 bits took 140 us so, 157 when three
// more registers made it two, and 146 to 164 with rows ahead in shared memory.
template <typename T, int NV, int G, bool E4M3>
__global__ void __launch_bounds__(kBlock, NV * sizeof(T) <= 4 ? 3 : 1) k_add_norm(const NormParams p) {
  __shared__ float2 s_red[2][32];
  const int lanes = G ? G : blockDim.x;
  const int lane = threadIdx.x % lanes;
  constexpr int groups = G ? kBlock / (G ? G : 1) : 1;
  const int nvec = p.channels >> 3;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  const T* x = static_cast<const T*>(p.x);
  const T* res = static_cast<const T*>(p.res);
  grid_release();
  grid_wait();
  const Weights<NV> w(p.w, lane, lanes, nvec);
  Vec8<T> nx[NV], nr[NV];
  auto load = [&](int64_t r) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int at = lane + v * lanes;
      const bool in = r < p.rows && at < nvec;
      nx[v] = in ? ld_vec(x + r * p.ldx + at * 8) : zero_vec<T>();
      nr[v] = in && res ? ld_vec(res + r * p.ldres + at * 8) : zero_vec<T>();
    }
  };
  int64_t row = static_cast<int64_t>(blockIdx.x) * groups + threadIdx.x / lanes;
  constexpr bool kAhead = loads_ahead<T, NV>();
  if (kAhead) load(row);
  int turn = 0;
  // the warp's subgroups stay together (their shuffles name the whole warp)
  for (int64_t base = row - (G ? (threadIdx.x & 31) / lanes : 0); base < p.rows; base += step, row += step) {
    if (!kAhead) load(row);
    float h[NV][8];
    float ss = 0.f, top = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float t[8];
      unpack(nx[v], h[v]);
      unpack(nr[v], t);
      if (res) {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[v][i] += t[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(h[v][i], h[v][i], ss);
      if constexpr (E4M3) {
        w.get(v, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(h[v][i] * t[i]));
      }
    }
    if (kAhead) load(row + step);
    row_reduce<G, true>(ss, top, s_red, turn);
    turn ^= 1;
    if (row < p.rows) store_row<T, NV, E4M3>(p, w, h, ss, top, row, lane, lanes, nvec);
  }
}

// The gradients.  With z = w gout and r as in the forward, one crossing of the lanes
// gives sum h^2 and sum z h, and gin = r z - h r^3 (sum z h) / channels + gsum.  The
// weights' gradient gathers in registers over the rows that a lane's block walks and
// goes out once a block.
//
// At four vectors a lane (520 to 1,024 channels) 128 registers do not hold a row's three tensors and
// the sums: 112 to 216 bytes spill (131,072 rows of 1,024, bf16, cold: 209 us, floor 158; 65,536 of 2,048, which
// the wide form takes, 184).
template <typename T, int NV, int G>
__global__ void __launch_bounds__(kBlock, NV * sizeof(T) <= 2 ? 3 : 2)
    k_add_norm_bwd(const NormParams p) {
  __shared__ float s_gw[G * NV * 8];
  constexpr int lanes = G;
  const int lane = threadIdx.x % lanes;
  constexpr int groups = kBlock / G;
  const int nvec = p.channels >> 3;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  const T* x = static_cast<const T*>(p.x);
  const T* gs = static_cast<const T*>(p.res);
  const T* go = static_cast<const T*>(p.gout);
  grid_release();
  grid_wait();
  const Weights<NV, false> w(p.w, lane, lanes, nvec);
  float gw[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) gw[v][i] = 0.f;
  Vec8<T> nx[NV], ng[NV], ns[NV];
  auto load = [&](int64_t r) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int at = lane + v * lanes;
      const bool in = r < p.rows && at < nvec;
      nx[v] = in ? ld_vec(x + r * p.ldx + at * 8) : zero_vec<T>();
      ng[v] = in ? ld_vec(go + r * p.ldgout + at * 8) : zero_vec<T>();
      ns[v] = in && gs ? ld_vec(gs + r * p.ldres + at * 8) : zero_vec<T>();
    }
  };
  int64_t row = static_cast<int64_t>(blockIdx.x) * groups + threadIdx.x / lanes;
  constexpr bool kAhead = loads_ahead<T, NV>();
  if (kAhead) load(row);
  for (int64_t base = row - (threadIdx.x & 31) / lanes; base < p.rows; base += step, row += step) {
    if (!kAhead) load(row);
    Vec8<T> cx[NV], cg[NV], cs[NV];
    float ss = 0.f, zh = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      cx[v] = nx[v];
      cg[v] = ng[v];
      cs[v] = ns[v];
      float h[8], g[8], wv[8];
      unpack(cx[v], h);
      unpack(cg[v], g);
      w.get(v, wv);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss = fmaf(h[i], h[i], ss);
        zh = fmaf(g[i] * wv[i], h[i], zh);
      }
    }
    if (kAhead) load(row + step);
    row_reduce<G, false>(ss, zh, nullptr, 0);
    const float n = static_cast<float>(p.channels);
    const float r = rsqrtf(ss / n + p.eps);
    const float c = zh / n * r * r;
    if (row >= p.rows) continue;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int at = lane + v * lanes;
      if (at >= nvec) continue;
      float h[8], g[8], s[8], wv[8];
      unpack(cx[v], h);
      unpack(cg[v], g);
      unpack(cs[v], s);
      w.get(v, wv);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        gw[v][i] = fmaf(g[i], h[i] * r, gw[v][i]);
        s[i] = fmaf(r, g[i] * wv[i] - c * h[i], s[i]);
      }
      st_vec(static_cast<T*>(p.out) + row * p.ldout + at * 8, s);
    }
  }
  if (!p.part) return;
  float* part = p.part + static_cast<int64_t>(blockIdx.x) * p.channels;
  // one group after the other, so that the order is fixed
  const int group = threadIdx.x / lanes;
  for (int g = 0; g < groups; ++g) {
    if (g == group) {
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float* s = s_gw + (v * G + lane) * 8 + i;
          *s = g == 0 ? gw[v][i] : *s + gw[v][i];
        }
    }
    __syncthreads();
  }
  for (int c = threadIdx.x; c < p.channels; c += kBlock) part[c] = s_gw[c];
}

// The gradients of wide rows, a block a row.  Rows come ahead of their turn into a ring of
// shared memory by bulk copies, so that what is in flight does not wait for the block's
// barriers: with loads into registers, one row ahead, 9,973 rows of 2,056 took 51 us (36 so; floor 24).
// Above 8,192 channels a lane holds four vectors and spills 40 to 172 bytes, and one block an SM works on
// one row at a time (11,000 rows of 12,000, bf16, cold: 229 us, floor 156).
template <typename T, int NV>
__global__ void __launch_bounds__(512, NV == 1 && sizeof(T) == 2 ? 2 : 1) k_add_norm_bwd_wide(const NormParams p) {
  extern __shared__ __align__(16) uint8_t s_rows[];
  __shared__ float2 s_red[2][32];
  __shared__ __align__(8) uint64_t s_full[kRing];
  __shared__ int s_late[2];
  const int lanes = blockDim.x, lane = threadIdx.x;
  const int nvec = p.channels >> 3;
  const uint32_t row_bytes = static_cast<uint32_t>(p.channels) * sizeof(T), slot_bytes = 3 * row_bytes;
  const uint32_t base = smem_u32(s_rows), full = smem_u32(s_full);
  const int64_t step = gridDim.x;
  if (lane == 0) {
    for (int i = 0; i < kRing; ++i) mbar_init(full + 8 * i, 1);
    fence_mbar_init();
    s_late[0] = s_late[1] = 0;
  }
  __syncthreads();
  grid_release();
  grid_wait();
  auto load = [&](int64_t r, int slot) {
    const uint32_t dst = base + slot * slot_bytes, bar = full + 8 * slot;
    mbar_arrive_expect_tx(bar, p.res ? slot_bytes : 2 * row_bytes);
    bulk_g2s(dst, static_cast<const T*>(p.x) + r * p.ldx, row_bytes, bar);
    bulk_g2s(dst + row_bytes, static_cast<const T*>(p.gout) + r * p.ldgout, row_bytes, bar);
    if (p.res) bulk_g2s(dst + 2 * row_bytes, static_cast<const T*>(p.res) + r * p.ldres, row_bytes, bar);
  };
  if (lane == 0) {
    for (int i = 0; i < p.ring; ++i)
      if (blockIdx.x + i * step < p.rows) load(blockIdx.x + i * step, i);
  }
  const Weights<NV> w(p.w, lane, lanes, nvec);
  float gw[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) gw[v][i] = 0.f;
  int slot = 0, turn = 0;
  uint32_t ph = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += step) {
    if (!mbar_wait_inl(full + 8 * slot, ph)) s_late[turn] = 1;
    const uint8_t* src = s_rows + slot * slot_bytes;
    Vec8<T> cx[NV], cg[NV], cs[NV];
    float ss = 0.f, zh = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int at = lane + v * lanes;
      const bool in = at < nvec;
      cx[v] = in ? ld_vec(reinterpret_cast<const T*>(src) + at * 8) : zero_vec<T>();
      cg[v] = in ? ld_vec(reinterpret_cast<const T*>(src + row_bytes) + at * 8) : zero_vec<T>();
      cs[v] = in && p.res ? ld_vec(reinterpret_cast<const T*>(src + 2 * row_bytes) + at * 8) : zero_vec<T>();
      float h[8], g[8], wv[8];
      unpack(cx[v], h);
      unpack(cg[v], g);
      w.get(v, wv);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss = fmaf(h[i], h[i], ss);
        zh = fmaf(g[i] * wv[i], h[i], zh);
      }
    }
    row_reduce<0, false>(ss, zh, s_red, turn);  // with a barrier: the slot has been read
    if (s_late[turn]) {  // a copy did not land within seconds: the block gives up as one
      if (lane == 0) {
        atomicOr(p.status, kDevErrTimeout);
        for (int i = 0; i < p.ring; ++i) mbar_drain(full + 8 * i, i < slot ? ph ^ 1 : ph);
      }
      break;
    }
    turn ^= 1;
    if (lane == 0 && row + p.ring * step < p.rows) {
      fence_proxy_async_smem();
      load(row + p.ring * step, slot);
    }
    if (++slot == p.ring) slot = 0, ph ^= 1;
    const float n = static_cast<float>(p.channels);
    const float r = rsqrtf(ss / n + p.eps);
    const float c = zh / n * r * r;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int at = lane + v * lanes;
      if (at >= nvec) continue;
      float h[8], g[8], s[8], wv[8];
      unpack(cx[v], h);
      unpack(cg[v], g);
      unpack(cs[v], s);
      w.get(v, wv);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        gw[v][i] = fmaf(g[i], h[i] * r, gw[v][i]);
        s[i] = fmaf(r, g[i] * wv[i] - c * h[i], s[i]);
      }
      st_vec(static_cast<T*>(p.out) + row * p.ldout + at * 8, s);
    }
  }
  if (!p.part) return;
  float* part = p.part + static_cast<int64_t>(blockIdx.x) * p.channels;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int at = lane + v * lanes;
    if (at >= nvec) continue;
#pragma unroll
    for (int i = 0; i < 8; ++i) part[at * 8 + i] = gw[v][i];
  }
}

// The forward of rows that no 256 threads can hold, and of few rows, a block a row, with the same ring.
template <typename T, int NV, bool E4M3>
__global__ void __launch_bounds__(512, NV == 1 ? 2 : 1) k_add_norm_wide(const NormParams p) {
  extern __shared__ __align__(16) uint8_t s_rows[];
  __shared__ float2 s_red[2][32];
  __shared__ __align__(8) uint64_t s_full[kRing];
  __shared__ int s_late[2];
  const int lanes = blockDim.x, lane = threadIdx.x;
  const int nvec = p.channels >> 3;
  const uint32_t row_bytes = static_cast<uint32_t>(p.channels) * sizeof(T), slot_bytes = 2 * row_bytes;
  const uint32_t base = smem_u32(s_rows), full = smem_u32(s_full);
  const int64_t step = gridDim.x;
  if (lane == 0) {
    for (int i = 0; i < kRing; ++i) mbar_init(full + 8 * i, 1);
    fence_mbar_init();
    s_late[0] = s_late[1] = 0;
  }
  __syncthreads();
  grid_release();
  grid_wait();
  auto load = [&](int64_t r, int slot) {
    const uint32_t dst = base + slot * slot_bytes, bar = full + 8 * slot;
    mbar_arrive_expect_tx(bar, p.res ? slot_bytes : row_bytes);
    bulk_g2s(dst, static_cast<const T*>(p.x) + r * p.ldx, row_bytes, bar);
    if (p.res) bulk_g2s(dst + row_bytes, static_cast<const T*>(p.res) + r * p.ldres, row_bytes, bar);
  };
  if (lane == 0) {
    for (int i = 0; i < p.ring; ++i)
      if (blockIdx.x + i * step < p.rows) load(blockIdx.x + i * step, i);
  }
  const Weights<NV> w(p.w, lane, lanes, nvec);
  int slot = 0, turn = 0;
  uint32_t ph = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += step) {
    if (!mbar_wait_inl(full + 8 * slot, ph)) s_late[turn] = 1;
    const uint8_t* src = s_rows + slot * slot_bytes;
    float h[NV][8];
    float ss = 0.f, top = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int at = lane + v * lanes;
      unpack(at < nvec ? ld_vec(reinterpret_cast<const T*>(src) + at * 8) : zero_vec<T>(), h[v]);
      float t[8];
      if (p.res) {
        unpack(at < nvec ? ld_vec(reinterpret_cast<const T*>(src + row_bytes) + at * 8) : zero_vec<T>(), t);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[v][i] += t[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(h[v][i], h[v][i], ss);
      if constexpr (E4M3) {
        w.get(v, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(h[v][i] * t[i]));
      }
    }
    row_reduce<0, true>(ss, top, s_red, turn);  // with a barrier: the slot has been read
    if (s_late[turn]) {  // a copy did not land within seconds: the block gives up as one
      if (lane == 0) {
        atomicOr(p.status, kDevErrTimeout);
        for (int i = 0; i < p.ring; ++i) mbar_drain(full + 8 * i, i < slot ? ph ^ 1 : ph);
      }
      break;
    }
    turn ^= 1;
    if (lane == 0 && row + p.ring * step < p.rows) {
      fence_proxy_async_smem();
      load(row + p.ring * step, slot);
    }
    if (++slot == p.ring) slot = 0, ph ^= 1;
    store_row<T, NV, E4M3>(p, w, h, ss, top, row, lane, lanes, nvec);
  }
}

// The blocks' partial sums, 32 columns and 32 runs of blocks a thread block.
__global__ void __launch_bounds__(1024) k_column_join(const float* __restrict__ part, int blocks, int channels,
                                                      float* __restrict__ out) {
  __shared__ float s[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  grid_release();
  grid_wait();
  float a = 0.f;
  if (c < channels) {
    // loads in flight together, added in order
    int b = threadIdx.y;
    for (; b + 7 * 32 < blocks; b += 8 * 32) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = part[static_cast<int64_t>(b + k * 32) * channels + c];
#pragma unroll
      for (int k = 0; k < 8; ++k) a += v[k];
    }
#pragma unroll 7
    for (; b < blocks; b += 32) a += part[static_cast<int64_t>(b) * channels + c];
  }
  s[threadIdx.y][threadIdx.x] = a;
  __syncthreads();
  a = s[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  const int cc = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && cc < channels) out[cc] = a;
}

cudaError_t launch(const char* name, const void* kern, unsigned grid, unsigned block, size_t smem, NormParams& p,
                   cudaStream_t s) {
  void* args[] = {&p};
  cudaError_t e;
  SC_LAUNCH(name, s, e = launch_after(kern, grid, block, smem, s, args));
  return e;
}

// Which form holds a row of nvec vectors: how many a lane, the lanes (0: a block), the block's
// threads, and whether its rows come through the ring.
struct Form {
  int nv, g, threads;
  bool wide;
};
Form form_of(int nvec, int64_t rows, bool bwd) {
  if (nvec <= 4) return {1, 4, kBlock, false};
  if (nvec <= 8) return {1, 8, kBlock, false};
  if (nvec <= 16) return {1, 16, kBlock, false};
  if (nvec <= 32) return {1, 32, kBlock, false};
  const bool many = rows > 2048;
  if (many && nvec <= 64) return {2, 32, kBlock, false};
  if (many && nvec <= 128) return {4, 32, kBlock, false};
  const bool regs = !bwd && many && nvec <= 512;
  const int nv = regs ? (nvec <= 256 ? 1 : 2) : nvec <= 512 ? 1 : nvec <= 1024 ? 2 : 4;
  return {nv, 0, ((nvec + nv - 1) / nv + 31) / 32 * 32, !regs};
}

template <typename T, bool E4M3>
const void* fwd_kernel(const Form& f) {
  switch (f.g * 8 + f.nv) {
    case 4 * 8 + 1: return reinterpret_cast<const void*>(k_add_norm<T, 1, 4, E4M3>);
    case 8 * 8 + 1: return reinterpret_cast<const void*>(k_add_norm<T, 1, 8, E4M3>);
    case 16 * 8 + 1: return reinterpret_cast<const void*>(k_add_norm<T, 1, 16, E4M3>);
    case 32 * 8 + 1: return reinterpret_cast<const void*>(k_add_norm<T, 1, 32, E4M3>);
    case 32 * 8 + 2: return reinterpret_cast<const void*>(k_add_norm<T, 2, 32, E4M3>);
    case 32 * 8 + 4: return reinterpret_cast<const void*>(k_add_norm<T, 4, 32, E4M3>);
    case 1: return reinterpret_cast<const void*>(f.wide ? k_add_norm_wide<T, 1, E4M3> : k_add_norm<T, 1, 0, E4M3>);
    case 2: return reinterpret_cast<const void*>(f.wide ? k_add_norm_wide<T, 2, E4M3> : k_add_norm<T, 2, 0, E4M3>);
    default: return reinterpret_cast<const void*>(k_add_norm_wide<T, 4, E4M3>);
  }
}
template <typename T>
const void* bwd_kernel(const Form& f) {
  switch (f.g * 8 + f.nv) {
    case 4 * 8 + 1: return reinterpret_cast<const void*>(k_add_norm_bwd<T, 1, 4>);
    case 8 * 8 + 1: return reinterpret_cast<const void*>(k_add_norm_bwd<T, 1, 8>);
    case 16 * 8 + 1: return reinterpret_cast<const void*>(k_add_norm_bwd<T, 1, 16>);
    case 32 * 8 + 1: return reinterpret_cast<const void*>(k_add_norm_bwd<T, 1, 32>);
    case 32 * 8 + 2: return reinterpret_cast<const void*>(k_add_norm_bwd<T, 2, 32>);
    case 32 * 8 + 4: return reinterpret_cast<const void*>(k_add_norm_bwd<T, 4, 32>);
    case 1: return reinterpret_cast<const void*>(k_add_norm_bwd_wide<T, 1>);
    case 2: return reinterpret_cast<const void*>(k_add_norm_bwd_wide<T, 2>);
    default: return reinterpret_cast<const void*>(k_add_norm_bwd_wide<T, 4>);
  }
}

// The ring of a wide form whose rows have so many tensors: its depth and shared memory.
sc_status ring_setup(const Form& f, const void* kern, int tensors, const NormArgs& a, NormParams* p, size_t* smem) {
  if (!f.wide) return SC_OK;
  const size_t slot = static_cast<size_t>(tensors) * a.channels * (a.dtype == SC_F32 ? 4 : 2);
  p->ring = slot * kRing <= kRingMost ? kRing : static_cast<int>(kRingMost / slot);
  *smem = p->ring * slot;
  const sc_status st = rows_status_word(&p->status);
  return st ? st : kernel_setup(kern, *smem, nullptr);
}

unsigned grid_of(const Form& f, int64_t rows, int per_sm) {
  const int64_t groups = f.g ? f.threads / f.g : 1;
  const int64_t need = (rows + groups - 1) / groups, most = static_cast<int64_t>(device_sm_count()) * per_sm;
  return static_cast<unsigned>(need < most ? need : most);
}

}  // namespace

sc_status column_join(const float* part, int blocks, int channels, float* out, cudaStream_t s) {
  void* args[] = {&part, &blocks, &channels, &out};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((channels + 31) / 32);
  cfg.blockDim = dim3(32, 32);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaError_t e;
  SC_LAUNCH("column_join", s, e = cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(k_column_join), args));
  return e == cudaSuccess ? SC_OK : set_cuda_error(e, "column sums launch");
}

sc_status add_norm_fwd(const NormArgs& a) {
  if (a.rows == 0) return SC_OK;
  NormParams p{};
  p.x = a.x.data, p.ldx = a.x.stride;
  p.res = a.res.data, p.ldres = a.res.stride;
  p.sum = a.sum.data, p.ldsum = a.sum.stride;
  p.out = a.out.data, p.ldout = a.out.stride;
  p.scale = a.scale;
  p.w = a.w;
  p.rows = a.rows;
  p.channels = a.channels;
  p.eps = a.eps;
  const Form f = form_of(a.channels / 8, a.rows, false);
  const void* k;
  if (a.dtype == SC_F32) k = a.e4m3 ? fwd_kernel<float, true>(f) : fwd_kernel<float, false>(f);
  else if (a.dtype == SC_F16) k = a.e4m3 ? fwd_kernel<__half, true>(f) : fwd_kernel<__half, false>(f);
  else k = a.e4m3 ? fwd_kernel<__nv_bfloat16, true>(f) : fwd_kernel<__nv_bfloat16, false>(f);
  size_t smem = 0;
  const sc_status st = ring_setup(f, k, 2, a, &p, &smem);
  if (st) return st;
  const cudaError_t e = launch("add_norm_fwd", k, grid_of(f, a.rows, kernel_residency(k, f.threads, smem)), f.threads,
                               smem, p, a.stream);
  return e == cudaSuccess ? SC_OK : set_cuda_error(e, "norm launch");
}

sc_status add_norm_bwd(const NormArgs& a) {
  if (a.rows == 0) {
    if (!a.gw) return SC_OK;
    const cudaError_t e = cudaMemsetAsync(a.gw, 0, sizeof(float) * a.channels, a.stream);
    return e == cudaSuccess ? SC_OK : set_cuda_error(e, "norm weight gradient clear");
  }
  NormParams p{};
  p.x = a.x.data, p.ldx = a.x.stride;
  p.res = a.res.data, p.ldres = a.res.stride;
  p.gout = a.gout.data, p.ldgout = a.gout.stride;
  p.out = a.out.data, p.ldout = a.out.stride;
  p.w = a.w;
  p.rows = a.rows;
  p.channels = a.channels;
  p.eps = a.eps;
  const Form f = form_of(a.channels / 8, a.rows, true);
  const void* k = a.dtype == SC_F32 ? bwd_kernel<float>(f)
                                    : a.dtype == SC_F16 ? bwd_kernel<__half>(f) : bwd_kernel<__nv_bfloat16>(f);
  size_t smem = 0;
  sc_status st = ring_setup(f, k, 3, a, &p, &smem);
  if (st) return st;
  const unsigned grid = grid_of(f, a.rows, kernel_residency(k, f.threads, smem));
  if (a.gw) {
    st = dev_alloc(reinterpret_cast<void**>(&p.part), sizeof(float) * grid * a.channels, a.stream);
    if (st) return st;
  }
  const cudaError_t e = launch("add_norm_bwd", k, grid, f.threads, smem, p, a.stream);
  st = e == cudaSuccess ? SC_OK : set_cuda_error(e, "norm gradient launch");
  if (!st && a.gw) st = column_join(p.part, static_cast<int>(grid), a.channels, a.gw, a.stream);
  dev_free(p.part, a.stream);
  return st;
}

}  // namespace sc
