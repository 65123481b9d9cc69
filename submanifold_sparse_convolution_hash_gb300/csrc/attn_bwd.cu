// Attention's gradients: the plain forms of their kernels, one warp a row, fp32
// throughout.
//   S = scale q k^T, lse = log sum exp S, out = softmax(S) v, and the gradients.
#include "attn_internal.cuh"

namespace sc {
namespace {


struct View {
  const uint8_t* p;
  int64_t ts, hs;
};
struct SimpleParams {
  View q, k, v, out, gout, gq, gk, gv;
  float* lse;
  float* delta;
  const int *q_off, *k_off, *k_len;
  int n_seq;
  int64_t t_q, t_k;
  int hq, hk, g, d;
  float scale;
  int causal;
  int* bad;
  int* status;
};

template <typename T>
__device__ __forceinline__ void load_row(const View& v, int64_t t, int h, int d, float (&x)[4]) {
  const T* p = reinterpret_cast<const T*>(v.p) + t * v.ts + h * v.hs;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = lane + 32 * i < d ? static_cast<float>(p[lane + 32 * i]) : 0.f;
}
template <typename T>
__device__ __forceinline__ void store_row(const View& v, int64_t t, int h, int d, const float (&x)[4]) {
  T* p = reinterpret_cast<T*>(const_cast<uint8_t*>(v.p)) + t * v.ts + h * v.hs;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (lane + 32 * i < d) p[lane + 32 * i] = T(x[i]);
}
__device__ __forceinline__ float dot(const float (&a)[4], const float (&b)[4]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) s = fmaf(a[i], b[i], s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}
// the sequence s with off[s] <= t < off[s + 1]
__device__ __forceinline__ int find(const int* off, int n, int t) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int m = (lo + hi + 1) >> 1;
    if (__ldg(off + m) <= t) lo = m;
    else hi = m - 1;
  }
  return lo;
}
struct Range {
  int64_t q0, q1, k0, k1;
};
__device__ __forceinline__ Range range_of(const SimpleParams& p, int s) {
  Range r;
  r.q0 = p.q_off[s];
  r.q1 = p.q_off[s + 1];
  r.k0 = p.k_off[s];
  r.k1 = p.k_len ? r.k0 + p.k_len[s] : p.k_off[s + 1];
  return r;
}

// Checks the offsets; *bad stays 0 when every rule holds.
__global__ void k_check(const SimpleParams p, int packed_keys) {
  for (int s = threadIdx.x; s < p.n_seq; s += blockDim.x) {
    const Range r = range_of(p, s);
    bool bad = r.q0 < 0 || r.q1 > p.t_q || r.k0 < 0 || r.k1 > p.t_k || r.q1 < r.q0 || r.k1 < r.k0;
    bad = bad || (s == 0 && r.q0 != 0) || (s == p.n_seq - 1 && r.q1 != p.t_q);
    if (packed_keys) bad = bad || (s == 0 && r.k0 != 0) || (s == p.n_seq - 1 && r.k1 != p.t_k);
    if (bad) {
      *p.bad = 1;
      atomicOr(p.status, kDevErrRange);
    }
  }
}

template <typename T>
__global__ void k_simple_gq(const SimpleParams p) {
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  if (w >= p.t_q * p.hq || *p.bad) return;
  const int64_t t = w / p.hq;
  const int h = static_cast<int>(w % p.hq);
  const Range r = range_of(p, find(p.q_off, p.n_seq, static_cast<int>(t)));
  const int64_t end = p.causal ? min(r.k1, r.k1 - (r.q1 - t) + 1) : r.k1;
  float q[4], k[4], v[4], g[4], o[4], acc[4] = {};
  load_row<T>(p.q, t, h, p.d, q);
  load_row<T>(p.gout, t, h, p.d, g);
  load_row<T>(p.out, t, h, p.d, o);
  const float delta = dot(g, o), lse = p.lse[t * p.hq + h];
  if ((threadIdx.x & 31) == 0) p.delta[t * p.hq + h] = delta;
  for (int64_t j = r.k0; j < end; ++j) {
    load_row<T>(p.k, j, h / p.g, p.d, k);
    load_row<T>(p.v, j, h / p.g, p.d, v);
    const float ds = expf(dot(q, k) * p.scale - lse) * (dot(g, v) - delta) * p.scale;
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = fmaf(ds, k[i], acc[i]);
  }
  store_row<T>(p.gq, t, h, p.d, acc);
}

template <typename T>
__global__ void k_simple_gkv(const SimpleParams p) {
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  if (w >= p.t_k * p.hk || *p.bad) return;
  const int64_t t = w / p.hk;
  const int h = static_cast<int>(w % p.hk);
  const Range r = range_of(p, find(p.k_off, p.n_seq, static_cast<int>(t)));
  float q[4], k[4], v[4], g[4], ak[4] = {}, av[4] = {};
  load_row<T>(p.k, t, h, p.d, k);
  load_row<T>(p.v, t, h, p.d, v);
  int64_t first = r.q0;
  if (p.causal) first = max(first, r.q1 - (r.k1 - t));
  for (int64_t i = first; i < r.q1; ++i)
    for (int gh = h * p.g; gh < (h + 1) * p.g; ++gh) {
      load_row<T>(p.q, i, gh, p.d, q);
      load_row<T>(p.gout, i, gh, p.d, g);
      const float pr = expf(dot(q, k) * p.scale - p.lse[i * p.hq + gh]);
      const float ds = pr * (dot(g, v) - p.delta[i * p.hq + gh]) * p.scale;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        ak[c] = fmaf(ds, q[c], ak[c]);
        av[c] = fmaf(pr, g[c], av[c]);
      }
    }
  store_row<T>(p.gk, t, h, p.d, ak);
  store_row<T>(p.gv, t, h, p.d, av);
}

View view(const sc_heads& v) { return {static_cast<const uint8_t*>(v.data), v.token_stride, v.head_stride}; }
View view(const sc_heads_out& v) { return {static_cast<const uint8_t*>(v.data), v.token_stride, v.head_stride}; }

SimpleParams params(const AttnArgs& a) {
  SimpleParams p{};
  p.q = view(a.q);
  p.k = view(a.k);
  p.v = view(a.v);
  p.lse = a.lse;
  p.q_off = a.q_off;
  p.k_off = a.k_off;
  p.k_len = a.k_len;
  p.n_seq = static_cast<int>(a.n_seq);
  p.t_q = a.t_q;
  p.t_k = a.t_k;
  p.hq = a.heads_q;
  p.hk = a.heads_kv;
  p.g = a.heads_q / a.heads_kv;
  p.d = a.head_dim;
  p.scale = a.scale;
  p.causal = a.causal;
  return p;
}
sc_status check_offsets(SimpleParams& p, const AttnArgs& a, bool packed_keys) {
  void* bad = nullptr;
  const sc_status st = dev_alloc(&bad, sizeof(int), a.stream);
  if (st) return st;
  p.bad = static_cast<int*>(bad);
  p.status = attn_status_word();
  cudaMemsetAsync(bad, 0, sizeof(int), a.stream);
  SC_LAUNCH("attn_check", a.stream, (k_check<<<1, 256, 0, a.stream>>>(p, packed_keys)));
  return SC_OK;
}
unsigned blocks(int64_t warps) { return static_cast<unsigned>((warps + 7) / 8); }

}  // namespace

sc_status attn_bwd(const AttnArgs& a) {
  SimpleParams p = params(a);
  p.out = view(a.out_in);
  p.gout = view(a.gout);
  p.gq = view(a.gq);
  p.gk = view(a.gk);
  p.gv = view(a.gv);
  void* delta = nullptr;
  sc_status st = dev_alloc(&delta, sizeof(float) * a.t_q * a.heads_q, a.stream);
  if (st) return st;
  p.delta = static_cast<float*>(delta);
  if ((st = check_offsets(p, a, true))) {
    dev_free(delta, a.stream);
    return st;
  }
  if (a.t_q > 0) {
    const unsigned n = blocks(a.t_q * a.heads_q);
    SC_LAUNCH("attn_bwd_q", a.stream,
              (a.dtype == SC_F16 ? k_simple_gq<__half><<<n, 256, 0, a.stream>>>(p)
                                 : k_simple_gq<__nv_bfloat16><<<n, 256, 0, a.stream>>>(p)));
  }
  if (a.t_k > 0) {
    const unsigned n = blocks(a.t_k * a.heads_kv);
    SC_LAUNCH("attn_bwd_kv", a.stream,
              (a.dtype == SC_F16 ? k_simple_gkv<__half><<<n, 256, 0, a.stream>>>(p)
                                 : k_simple_gkv<__nv_bfloat16><<<n, 256, 0, a.stream>>>(p)));
  }
  dev_free(delta, a.stream);
  dev_free(p.bad, a.stream);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SC_OK : set_cuda_error(e, "attn_bwd");
}

}  // namespace sc
