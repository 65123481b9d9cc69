// What the matrix products on rows share: the operands' and the epilogue's
// parameters, activations and their slopes.
#pragma once

#include <cuda.h>

#include "sc_internal.cuh"

namespace sc {

// z = acc * sx[r] * sw[c] + bias[c]; pre = z; out = act(z) + res.
struct Epilogue {
  void *out, *pre;
  const void* res;
  int64_t ldo, ldp, ldr;
  const float *bias, *sx, *sw;
  int act;
  bool bf16;
};

namespace {

// 2^x and 1 / x to two units in the last place; results below the normal range are 0.
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float recip_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// 1 / (1 + exp(-z)): 1 + infinity has the reciprocal 0.
__device__ __forceinline__ float logistic(float z) { return recip_fast(1.f + exp2_fast(z * -1.44269504f)); }
// The normal distribution's integral up to z, and e = exp(-z^2 / 2).  With a = |z| and t = 1 / (1 + 0.3 a),
// as Hastings' formulas for the error function go, the integral up to -a is e times a
// polynomial in t.  Its coefficients are this project's own: weighted least squares for the
// smallest largest relative error on a in [0, 14], 6e-8 (evaluated in fp32: 4e-7, and with e
// 1.4e-6 up to a = 5; the integral itself is off by at most 1.7e-7).  erff took twice the
// instructions, and these are what the wide layers' epilogues wait for.
__device__ __forceinline__ float normal_cdf(float z, float* e) {
  const float a = fabsf(z);
  const float t = recip_fast(fmaf(0.3f, a, 1.f));
  *e = exp2_fast(a * a * -0.72134752f);
  float q = 0.03837805241346359f;
  q = fmaf(q, t, -0.16916505992412567f);
  q = fmaf(q, t, 0.22865813970565796f);
  q = fmaf(q, t, -0.07650448381900787f);
  q = fmaf(q, t, 0.1425343006849289f);
  q = fmaf(q, t, 0.09468398243188858f);
  q = fmaf(q, t, 0.12192023545503616f);
  q = fmaf(q, t, 0.1194877028465271f);
  q = fmaf(q, t, 7.168207048380282e-06f) * *e;
  return z > 0.f ? 1.f - q : q;
}

__device__ __forceinline__ float act_of(float z, int act) {
  switch (act) {
    case SC_ACT_RELU: return z > 0.f ? z : (z != z ? z : 0.f);
    case SC_ACT_GELU: {
      float e;
      return z * normal_cdf(z, &e);
    }
    case SC_ACT_SILU: return z * logistic(z);
    default: return z;
  }
}
__device__ __forceinline__ float slope_of(float z, int act) {
  switch (act) {
    case SC_ACT_RELU: return z > 0.f ? 1.f : 0.f;
    case SC_ACT_GELU: {
      float e;
      const float p = normal_cdf(z, &e);
      return fmaf(z * 0.39894228f, e, p);
    }
    case SC_ACT_SILU: {
      const float p = logistic(z);
      return p * fmaf(z, 1.f - p, 1.f);
    }
    default: return 1.f;
  }
}

__device__ __forceinline__ uint32_t pack16(float lo, float hi, bool bf16) {
  if (bf16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack16(uint32_t w, bool bf16) {
  if (bf16) return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ void unpack8(const uint4& u, bool bf16, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = unpack16(w[i], bf16);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}
__device__ __forceinline__ uint4 pack8(const float* f, bool bf16) {
  return make_uint4(pack16(f[0], f[1], bf16), pack16(f[2], f[3], bf16), pack16(f[4], f[5], bf16),
                    pack16(f[6], f[7], bf16));
}
__device__ __forceinline__ float load16(const void* p, int64_t at, bool bf16) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[at])
              : __half2float(static_cast<const __half*>(p)[at]);
}
__device__ __forceinline__ void store16(void* p, int64_t at, float v, bool bf16) {
  if (bf16) static_cast<__nv_bfloat16*>(p)[at] = __float2bfloat16_rn(v);
  else static_cast<__half*>(p)[at] = __float2half_rn(v);
}

// Eight columns of row r from c on: z from the sums, then the outputs.
__device__ __forceinline__ void finish8(const Epilogue& e, int64_t r, int64_t c, float (&z)[8]) {
  if (e.sw) {
    const float a = e.sx[r];
    const float4 s0 = *reinterpret_cast<const float4*>(e.sw + c), s1 = *reinterpret_cast<const float4*>(e.sw + c + 4);
    z[0] *= a * s0.x, z[1] *= a * s0.y, z[2] *= a * s0.z, z[3] *= a * s0.w;
    z[4] *= a * s1.x, z[5] *= a * s1.y, z[6] *= a * s1.z, z[7] *= a * s1.w;
  }
  if (e.bias) {
    const float4 s0 = *reinterpret_cast<const float4*>(e.bias + c),
                 s1 = *reinterpret_cast<const float4*>(e.bias + c + 4);
    z[0] += s0.x, z[1] += s0.y, z[2] += s0.z, z[3] += s0.w;
    z[4] += s1.x, z[5] += s1.y, z[6] += s1.z, z[7] += s1.w;
  }
  if (e.pre) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(e.pre) + r * e.ldp + c) = pack8(z, e.bf16);
  if (e.act) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = act_of(z[i], e.act);
  }
  if (e.res) {
    float t[8];
    unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(e.res) + r * e.ldr + c), e.bf16, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] += t[i];
  }
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(e.out) + r * e.ldo + c) = pack8(z, e.bf16);
}
// N rows r, r + step, ... of one column, of which `count` exist: for the form whose lanes hold columns.
template <bool BF16, int N>
__device__ __forceinline__ void finish_rows(const Epilogue& e, int64_t r, int step, int count, int64_t c,
                                            float (&z)[N], float sw, float bias) {
  if (e.sw) {
#pragma unroll
    for (int t = 0; t < N; ++t) z[t] *= e.sx[r + min(t, count - 1) * step] * sw;
  }
#pragma unroll
  for (int t = 0; t < N; ++t) z[t] += bias;
  if (e.pre) {
#pragma unroll
    for (int t = 0; t < N; ++t)
      if (t < count) store16(e.pre, (r + t * step) * e.ldp + c, z[t], BF16);
  }
  if (e.act) {
#pragma unroll
    for (int t = 0; t < N; ++t) z[t] = act_of(z[t], e.act);
  }
  if (e.res) {
    float v[N];
#pragma unroll
    for (int t = 0; t < N; ++t) v[t] = load16(e.res, (r + min(t, count - 1) * step) * e.ldr + c, BF16);
#pragma unroll
    for (int t = 0; t < N; ++t) z[t] += v[t];
  }
#pragma unroll
  for (int t = 0; t < N; ++t)
    if (t < count) store16(e.out, (r + t * step) * e.ldo + c, z[t], BF16);
}

}  // namespace

// D [m, n] = A B on the tensor cores, A's row i and B's column j vectors of k
// values.  An operand is K-major (its vectors lie along k, `ld` apart) or MN-major
// (memory holds for each k a run over i or j, runs `ld` apart).
struct Operand {
  const void* data;
  int64_t ld;  // elements
  bool mn;
};
struct Product {
  Operand a, b;
  int64_t m, n, k;
  bool e4m3;  // both operands, K-major (else 16 bits: bf16 as in the epilogue)
  Epilogue ep;
};
// D's rows are the output's (linear_gemm.cu).
sc_status product_rows(const Product& p, cudaStream_t s);
// D's rows are the output's columns: A holds the weights, B, K-major, few rows (linear_few.cu).
sc_status product_few(const Product& p, cudaStream_t s);
// A tensor map of an operand in boxes of 128 bytes by `box_vectors` (K-major) or 64 values of k.
sc_status product_map(CUtensorMap* map, const Operand& o, int64_t vectors, int64_t k, bool e4m3, int box_vectors);
}  // namespace sc
