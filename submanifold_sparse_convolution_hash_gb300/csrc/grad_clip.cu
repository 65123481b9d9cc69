// The norm of many gradients together, and their scaling to a largest norm.
//
// Two passes over memory are what the mathematics asks for (every output depends on
// every value); in the second each block walks its run of chunks backwards, so that it begins
// with what the first left in L2.  The gradients' addresses travel in the launch's parameters (up to
// 32 KB), so there is no table to upload and a captured graph holds its own copy.
//
// Bound by memory: 400M values in 300 gradients, bf16 and f32, to another place 484 to 490 us, 3 GB in both passes
// (6.1 TB/s); few small gradients are two launches, about 8 us.
#include <cmath>
#include <type_traits>

#include "sc_internal.cuh"

namespace sc {
namespace {

constexpr int kThreads = 256;
constexpr int kChunkBytes = 32768;  // what a block takes at a time, of one gradient
constexpr int kVecs = kChunkBytes / 16 / kThreads;  // 16-byte loads a thread of it

struct Entry {
  const void* data;
  void* out;
  int64_t n;
  uint32_t chunk0;  // chunks of the launch before this gradient's
  uint32_t dtype;
};
struct Head {
  double* part;      // a sum of squares for each block of each of the first pass's launches
  float* norm;
  int count;         // gradients of this launch
  uint32_t chunks;   // and their chunks
  int slot;          // first pass: where this launch's sums go; second: how many sums there are
  float max_norm;
};
// Up to MAX gradients a launch; few gradients take the short table, whose launch
// carries 2 KB of parameters and not 31.
template <int MAX>
struct Table {
  Head h;
  Entry e[MAX];
};
constexpr int kSmall = 62, kLarge = 960;
static_assert(sizeof(Table<kLarge>) <= 32764, "launch parameters");

// The gradient that chunk c belongs to.
template <int MAX>
__device__ __forceinline__ int entry_of(const Table<MAX>& t, uint32_t c) {
  int lo = 0, hi = t.h.count - 1;
  while (lo < hi) {
    const int m = (lo + hi + 1) >> 1;
    if (t.e[m].chunk0 <= c) lo = m;
    else hi = m - 1;
  }
  return lo;
}

__host__ __device__ __forceinline__ int chunk_values(uint32_t dtype) {
  return dtype == SC_F32 ? kChunkBytes / 4 : kChunkBytes / 2;
}
// How far a gradient's first value lies behind the 128-byte line that it is on, in values.
// Chunks are cut from that line on, so that all but the first and the last are whole lines:
// cut from the values themselves, 500M 16-bit ones a value off a line took 15 % longer.
__host__ __device__ __forceinline__ int line_shift(const void* p, uint32_t dtype) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(p) & 127) / (dtype == SC_F32 ? 4 : 2));
}
// Chunk c of its gradient: the value its line begins at (of the first chunk it may lie before
// the gradient), and the values [*lo, *hi) from there that it has.
__device__ __forceinline__ int64_t chunk_at(const Entry& e, uint32_t c, int* lo, int* hi) {
  const int size = chunk_values(e.dtype), shift = line_shift(e.data, e.dtype);
  const int64_t at = static_cast<int64_t>(c - e.chunk0) * size - shift;
  *lo = at < 0 ? shift : 0;
  *hi = static_cast<int>(e.n - at < size ? e.n - at : size);
  return at;
}
// Where block b's run of chunks begins.  Runs, not every so many-th chunk: the search in the table costs
// a block about as much as a third of a chunk's way from memory.
__device__ __forceinline__ uint32_t chunk_of(uint32_t chunks, uint32_t b) {
  return static_cast<uint32_t>(static_cast<uint64_t>(chunks) * b / gridDim.x);
}

template <typename T>
__device__ __forceinline__ float to_f(T v) {
  if constexpr (std::is_same_v<T, float>) return v;
  else if constexpr (std::is_same_v<T, __half>) return __half2float(v);
  else return __bfloat162float(v);
}
// And back, rounded.
template <typename T>
__device__ __forceinline__ uint4 pack16(const float (&f)[16 / sizeof(T)]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same_v<T, float>) {
      w[i] = __float_as_uint(f[i]);
    } else if constexpr (std::is_same_v<T, __half>) {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename T>
__device__ __forceinline__ T from_f(float v) {
  if constexpr (std::is_same_v<T, float>) return v;
  else if constexpr (std::is_same_v<T, __half>) return __float2half_rn(v);
  else return __float2bfloat16_rn(v);
}
// The 16 bytes of a vector as floats.
template <typename T>
__device__ __forceinline__ void unpack16(const uint4& u, float (&f)[16 / sizeof(T)]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same_v<T, float>) {
      f[i] = __uint_as_float(w[i]);
    } else {
      float2 t;
      if constexpr (std::is_same_v<T, __half>) t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      else t = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
}

// A chunk's whole 16-byte vectors [v0, v1), and the values before and after them.
template <typename T>
struct Span16 {
  int v0, v1, head, tail;  // head values from lo on, tail values from v1's place on
  __device__ __forceinline__ Span16(int lo, int hi) {
    constexpr int V = 16 / sizeof(T);
    v0 = (lo + V - 1) / V;
    v1 = hi / V;
    if (v0 > v1) {  // within one vector
      v0 = v1;
      head = hi - lo;
      tail = 0;
    } else {
      head = v0 * V - lo;
      tail = hi - v1 * V;
    }
  }
};

// This thread's share of a chunk's sum of squares.  In fp32 over its 65 values or fewer;
// where that leaves fp32's range at either end, again in 64 bits.
template <typename T>
__device__ __forceinline__ double squares(const T* p, int lo, int hi) {
  constexpr int V = 16 / sizeof(T);
  constexpr int L = kVecs;
  const Span16<T> sp(lo, hi);
  const uint4* body = reinterpret_cast<const uint4*>(p);
  float s[2] = {0.f, 0.f};
  uint32_t any = 0;
  uint4 u[L];
#pragma unroll
  for (int l = 0; l < L; ++l) {
    const int v = threadIdx.x + l * kThreads;
    u[l] = v >= sp.v0 && v < sp.v1 ? __ldg(body + v) : make_uint4(0, 0, 0, 0);
  }
  float edge = 0.f;
  if (static_cast<int>(threadIdx.x) < sp.head) edge = to_f(p[lo + threadIdx.x]);
  else if (threadIdx.x >= 32 && static_cast<int>(threadIdx.x) - 32 < sp.tail)
    edge = to_f(p[sp.v1 * V + threadIdx.x - 32]);
#pragma unroll
  for (int l = 0; l < L; ++l) {
    any |= u[l].x | u[l].y | u[l].z | u[l].w;
    float f[V];
    unpack16<T>(u[l], f);
#pragma unroll
    for (int i = 0; i < V; ++i) s[i & 1] = fmaf(f[i], f[i], s[i & 1]);
  }
  s[0] = fmaf(edge, edge, s[0]);
  const float sum = s[0] + s[1];
  if (sum >= 0x1p-90f && sum <= 0x1p126f) return sum;
  if (!any && edge == 0.f) return 0.0;
  double d = static_cast<double>(edge) * edge;
#pragma unroll 1
  for (int l = 0; l < L; ++l) {
    const int v = threadIdx.x + l * kThreads;
    if (v < sp.v0 || v >= sp.v1) continue;
    float f[V];
    unpack16<T>(__ldg(body + v), f);
#pragma unroll
    for (int i = 0; i < V; ++i) d += static_cast<double>(f[i]) * f[i];
  }
  return d;
}

__device__ __forceinline__ double block_sum(double v, double* s_warp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) v += s_warp[w];
  return v;
}

template <int MAX>
__global__ void __launch_bounds__(kThreads, 4) k_grad_squares(const __grid_constant__ Table<MAX> t) {
  __shared__ double s_warp[kThreads / 32];
  grid_release();
  grid_wait();
  double sum = 0.0;
  const uint32_t c0 = chunk_of(t.h.chunks, blockIdx.x), c1 = chunk_of(t.h.chunks, blockIdx.x + 1);
  int i = entry_of(t, c0);
  for (uint32_t c = c0; c < c1; ++c) {
    while (i + 1 < t.h.count && t.e[i + 1].chunk0 <= c) ++i;
    const Entry& e = t.e[i];
    int lo, hi;
    const int64_t at = chunk_at(e, c, &lo, &hi);
    if (e.dtype == SC_F32) sum += squares(static_cast<const float*>(e.data) + at, lo, hi);
    else if (e.dtype == SC_F16) sum += squares(static_cast<const __half*>(e.data) + at, lo, hi);
    else sum += squares(static_cast<const __nv_bfloat16*>(e.data) + at, lo, hi);
  }
  sum = block_sum(sum, s_warp);
  if (threadIdx.x == 0) t.h.part[t.h.slot + blockIdx.x] = sum;
}

// What the values are multiplied by.  Below fp32's normal range a factor has lost bits that the
// product needs (values near 2^127 to a norm of 1): there `by` is 2^126 times it, at most 1, and
// `down` 2^-126, else 1.  Factors are above 2^-277, so `by` is off by 2^-150 at most and a product by 2^-148.
struct Factor {
  float by, down;
  __device__ __forceinline__ explicit Factor(double f)
      : by(static_cast<float>(f < 0x1p-126 ? f * 0x1p126 : f)), down(f < 0x1p-126 ? 0x1p-126f : 1.f) {}
  __device__ __forceinline__ float operator()(float v) const { return v * by * down; }
};

template <typename T>
__device__ __forceinline__ void scale_chunk(const T* p, T* o, int lo, int hi, const Factor& by) {
  constexpr int V = 16 / sizeof(T);
  // no common boundary: value by value (200M bf16 values to an output one value off: 186 us, else 131)
  if ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(o)) & 15) {
    for (int i0 = lo + threadIdx.x; i0 < hi; i0 += 8 * kThreads) {
      float f[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = i0 + k * kThreads < hi ? to_f(p[i0 + k * kThreads]) : 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (i0 + k * kThreads < hi) o[i0 + k * kThreads] = from_f<T>(by(f[k]));
    }
    return;
  }
  const Span16<T> sp(lo, hi);
  const uint4* body = reinterpret_cast<const uint4*>(p);
  uint4* dst = reinterpret_cast<uint4*>(o);
  if (static_cast<int>(threadIdx.x) < sp.head) {
    o[lo + threadIdx.x] = from_f<T>(by(to_f(p[lo + threadIdx.x])));
  } else if (threadIdx.x >= 32 && static_cast<int>(threadIdx.x) - 32 < sp.tail) {
    const int i = sp.v1 * V + threadIdx.x - 32;
    o[i] = from_f<T>(by(to_f(p[i])));
  }
  // four loads in flight a thread (eight, or more blocks an SM, measured the same)
#pragma unroll 1
  for (int l0 = sp.v0 + threadIdx.x; l0 < sp.v1; l0 += 4 * kThreads) {
    uint4 u[4];
#pragma unroll
    for (int l = 0; l < 4; ++l) u[l] = body[min(l0 + l * kThreads, sp.v1 - 1)];
#pragma unroll
    for (int l = 0; l < 4; ++l) {
      if (l0 + l * kThreads >= sp.v1) continue;
      float f[V];
      unpack16<T>(u[l], f);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = by(f[i]);
      dst[l0 + l * kThreads] = pack16<T>(f);
    }
  }
}

template <int MAX>
__global__ void __launch_bounds__(kThreads, 4) k_grad_scale(const __grid_constant__ Table<MAX> t) {
  __shared__ double s_warp[kThreads / 32];
  grid_release();
  grid_wait();
  double sum = 0.0;
  for (int i = threadIdx.x; i < t.h.slot; i += kThreads) sum += t.h.part[i];
  const double norm = sqrt(block_sum(sum, s_warp));
  const float said = static_cast<float>(norm);
  if (blockIdx.x == 0 && threadIdx.x == 0) *t.h.norm = said;
  // a norm past fp32's range is said to be infinite, so it scales nothing either
  const bool cut = isfinite(said) && norm > static_cast<double>(t.h.max_norm);
  const Factor by(cut ? static_cast<double>(t.h.max_norm) / norm : 1.0);
  const uint32_t c0 = chunk_of(t.h.chunks, blockIdx.x), c1 = chunk_of(t.h.chunks, blockIdx.x + 1);
  if (c0 == c1) return;
  int i = entry_of(t, c1 - 1);
  for (uint32_t c = c1; c-- > c0;) {
    while (t.e[i].chunk0 > c) --i;
    const Entry& e = t.e[i];
    if (!cut && e.out == e.data) continue;
    int lo, hi;
    const int64_t at = chunk_at(e, c, &lo, &hi);
    if (e.dtype == SC_F32)
      scale_chunk(static_cast<const float*>(e.data) + at, static_cast<float*>(e.out) + at, lo, hi, by);
    else if (e.dtype == SC_F16)
      scale_chunk(static_cast<const __half*>(e.data) + at, static_cast<__half*>(e.out) + at, lo, hi, by);
    else
      scale_chunk(static_cast<const __nv_bfloat16*>(e.data) + at, static_cast<__nv_bfloat16*>(e.out) + at, lo, hi, by);
  }
}

unsigned grid_of(const void* kern, uint32_t chunks) {
  const uint32_t most = static_cast<uint32_t>(device_sm_count() * kernel_residency(kern, kThreads));
  const uint32_t g = chunks < most ? chunks : most;
  return g ? g : 1;
}

// Fills a table with gradients from *at on; those without values are left out.
template <int MAX>
void fill(Table<MAX>& t, const sc_grad* grads, int64_t count, int64_t* at) {
  t.h.count = 0;
  uint64_t chunks = 0;
  for (; *at < count && t.h.count < MAX; ++*at) {
    const sc_grad& g = grads[*at];
    if (g.n == 0) continue;
    const uint64_t more = static_cast<uint64_t>((g.n - 1 + line_shift(g.data, g.dtype)) / chunk_values(g.dtype) + 1);
    if (chunks + more > 0x7fffffffull) break;
    Entry& e = t.e[t.h.count++];
    e.data = g.data;
    e.out = g.out;
    e.n = g.n;
    e.chunk0 = static_cast<uint32_t>(chunks);
    e.dtype = static_cast<uint32_t>(g.dtype);
    chunks += more;
  }
  t.h.chunks = static_cast<uint32_t>(chunks);
}

template <int MAX>
sc_status run(const sc_grad* grads, int64_t count, float max_norm, float* d_norm, cudaStream_t s) {
  const void* sq = reinterpret_cast<const void*>(k_grad_squares<MAX>);
  const void* sc = reinterpret_cast<const void*>(k_grad_scale<MAX>);
  Table<MAX> t{};
  int slots = 0;
  for (int64_t at = 0; at < count;) {
    fill(t, grads, count, &at);
    if (t.h.count) slots += static_cast<int>(grid_of(sq, t.h.chunks));
  }
  t.h.norm = d_norm;
  t.h.max_norm = max_norm;
  sc_status st = dev_alloc(reinterpret_cast<void**>(&t.h.part), sizeof(double) * static_cast<size_t>(slots), s);
  if (st) return st;
  cudaError_t e = cudaSuccess;
  void* args[] = {&t};
  int slot = 0;
  for (int64_t at = 0; at < count && e == cudaSuccess;) {
    fill(t, grads, count, &at);
    if (!t.h.count) continue;
    t.h.slot = slot;
    const unsigned g = grid_of(sq, t.h.chunks);
    SC_LAUNCH("grad_squares", s, e = launch_after(sq, g, kThreads, 0, s, args));
    slot += static_cast<int>(g);
  }
  t.h.slot = slots;
  bool first = true;
  for (int64_t at = 0; (at < count || first) && e == cudaSuccess; first = false) {
    fill(t, grads, count, &at);
    if (!t.h.count && !first) continue;
    SC_LAUNCH("grad_scale", s, e = launch_after(sc, grid_of(sc, t.h.chunks), kThreads, 0, s, args));
  }
  dev_free(t.h.part, s);
  return e == cudaSuccess ? SC_OK : set_cuda_error(e, "gradient clipping launch");
}

}  // namespace

sc_status grad_clip(const sc_grad* grads, int64_t count, float max_norm, float* d_norm, cudaStream_t s) {
  return count <= kSmall ? run<kSmall>(grads, count, max_norm, d_norm, s)
                         : run<kLarge>(grads, count, max_norm, d_norm, s);
}

}  // namespace sc
