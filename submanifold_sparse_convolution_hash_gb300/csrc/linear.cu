// Matrix products on rows: the layer, its gradients, and the pass that makes the
// gradient before the activation and sums the bias's.
//
// The gradients are that pass and two products.  120,000 rows, 256 -> 512, f16, silu: 155 us, the pass 56
// (bound by memory: 6.5 TB/s), the products 40 and 39.  Rounding gz to the rows' type is what the
// tensor cores' operands ask for; a product of it is off by that rounding once more.
#include "linear_internal.cuh"

namespace sc {
namespace {

constexpr int kThreads = 256;
// Up to here the form for few rows, whose tiles have the rows for columns; above it tiles of 128 rows or more.
// Kernels, cold, us, in this form and in tiles (with their join), at 16, at 64 and at 128 rows:
//   4,096 -> 4,096   17.3 22.4   20.7 23.0   24.7 23.8
//   8,192 -> 1,024   14.7 18.8   18.5 19.5   22.9 21.4
//   1,024 -> 1,024   10.4 16.3   12.5 16.6   16.4 16.6
//   4,096 -> 256     12.3 16.3   14.4 16.6   18.5 16.8
//   256 -> 4,096     10.2 10.5   14.1 10.3   18.5 10.5
// A rule on the rows alone: where k is short, so that tiles need no cuts, they are faster from 20 rows or so on.
constexpr int64_t kFewRows = 128;

// gz = gout * act'(pre), in 16 bits, and the columns' sums of the unrounded values.  A block
// holds blockDim.x vectors of eight columns of blockDim.y rows, which it takes in turn, and writes
// its sums once.  The widths are cut evenly into runs of at most 64 vectors: cut into 32 lanes
// wherever that ends, a fifth of the blocks had 3 of 131 vectors (9,973 x 1,048, gelu).
template <int ACT, bool BF16>
__global__ void __launch_bounds__(kThreads, 3)
    k_act_grad(const uint16_t* __restrict__ gout, int64_t ldg, const uint16_t* __restrict__ pre, int64_t ldp,
               uint16_t* __restrict__ gz, float* __restrict__ part, int64_t rows, int channels) {
  __shared__ float s_sum[kThreads * 8];
  grid_release();
  grid_wait();
  const int c = (blockIdx.x * blockDim.x + threadIdx.x) * 8;
  const bool in = c < channels;
  float sum[8] = {};
  constexpr int kRows = 4;  // rows in flight
  const int64_t step = static_cast<int64_t>(gridDim.y) * blockDim.y;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.y) * blockDim.y + threadIdx.y; r0 < rows && in; r0 += kRows * step) {
    uint4 g[kRows], z[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int64_t r = r0 + k * step;
      if (r >= rows) continue;
      g[k] = *reinterpret_cast<const uint4*>(gout + r * ldg + c);
      if (ACT) z[k] = *reinterpret_cast<const uint4*>(pre + r * ldp + c);
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int64_t r = r0 + k * step;
      if (r >= rows) continue;
      float f[8];
      unpack8(g[k], BF16, f);
      if (ACT) {
        float t[8];
        unpack8(z[k], BF16, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= slope_of(t[i], ACT);
        *reinterpret_cast<uint4*>(gz + r * channels + c) = pack8(f, BF16);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += f[i];
    }
  }
  if (!part) return;
  const int width = blockDim.x * 8;
#pragma unroll
  for (int i = 0; i < 8; ++i) s_sum[threadIdx.y * width + threadIdx.x * 8 + i] = sum[i];
  __syncthreads();
  for (int t = threadIdx.y * blockDim.x + threadIdx.x; t < width; t += blockDim.x * blockDim.y) {
    const int cc = blockIdx.x * width + t;
    if (cc >= channels) break;
    float a = 0.f;
    for (int y = 0; y < static_cast<int>(blockDim.y); ++y) a += s_sum[y * width + t];
    part[static_cast<int64_t>(blockIdx.y) * channels + cc] = a;
  }
}

template <bool BF16>
const void* act_grad_kernel(int act) {
  switch (act) {
    case SC_ACT_RELU: return reinterpret_cast<const void*>(k_act_grad<SC_ACT_RELU, BF16>);
    case SC_ACT_GELU: return reinterpret_cast<const void*>(k_act_grad<SC_ACT_GELU, BF16>);
    case SC_ACT_SILU: return reinterpret_cast<const void*>(k_act_grad<SC_ACT_SILU, BF16>);
    default: return reinterpret_cast<const void*>(k_act_grad<SC_ACT_NONE, BF16>);
  }
}

// rows x columns, by the form that fits the number of rows.
sc_status run(Product& p, const Operand& rows_op, const Operand& cols_op, int64_t rows, int64_t cols, cudaStream_t s) {
  const bool few = rows <= kFewRows;
  p.a = few ? cols_op : rows_op;
  p.b = few ? rows_op : cols_op;
  p.m = few ? cols : rows;
  p.n = few ? rows : cols;
  return few ? product_few(p, s) : product_rows(p, s);
}

}  // namespace

sc_status linear_fwd(const LinearArgs& a) {
  if (a.rows == 0) return SC_OK;
  Product p{};
  p.e4m3 = a.in == SC_E4M3;
  p.k = a.c_in;
  const Operand x{a.x.data, a.x.stride, false};
  const Operand w{a.W, p.e4m3 ? a.c_in : a.c_out, !p.e4m3};
  p.ep = {a.out.data, a.pre.data, a.res.data, a.out.stride, a.pre.stride, a.res.stride, a.bias,
          a.scale_x,  a.scale_w,  a.act,      a.dtype == SC_BF16};
  return run(p, x, w, a.rows, a.c_out, a.stream);
}

sc_status linear_bwd(const LinearBwdArgs& a) {
  const bool bf16 = a.dtype == SC_BF16;
  cudaStream_t s = a.stream;
  if (a.rows == 0) {
    cudaError_t e = cudaSuccess;
    if (a.gW) e = cudaMemsetAsync(a.gW, 0, static_cast<size_t>(a.c_in) * a.c_out * 2, s);
    if (e == cudaSuccess && a.gbias) e = cudaMemsetAsync(a.gbias, 0, sizeof(float) * a.c_out, s);
    return e == cudaSuccess ? SC_OK : set_cuda_error(e, "weight gradient clear");
  }
  const bool act = a.act != SC_ACT_NONE;
  sc_rows gz{a.gout.data, a.gout.stride};
  void* buf = nullptr;
  float* part = nullptr;
  sc_status st = SC_OK;
  if (act || a.gbias) {
    const int nvec = a.c_out / 8, cols = (nvec + 63) / 64, lanes = (nvec + cols - 1) / cols, streams = kThreads / lanes;
    // six blocks an SM, and at least eight rows a thread
    int64_t runs = (static_cast<int64_t>(device_sm_count()) * 6 + cols - 1) / cols;
    const int64_t most = (a.rows + streams * 8 - 1) / (streams * 8);
    if (runs > most) runs = most;
    if (act) {
      st = dev_alloc(&buf, static_cast<size_t>(a.rows) * a.c_out * 2, s);
      gz = {buf, a.c_out};
    }
    if (!st && a.gbias)
      st = dev_alloc(reinterpret_cast<void**>(&part), sizeof(float) * static_cast<size_t>(runs) * a.c_out, s);
    if (!st) {
      const uint16_t* g = static_cast<const uint16_t*>(a.gout.data);
      const uint16_t* pre = static_cast<const uint16_t*>(a.pre.data);
      uint16_t* out = static_cast<uint16_t*>(buf);
      int64_t ldg = a.gout.stride, ldp = a.pre.stride, rows = a.rows;
      int channels = a.c_out;
      void* args[] = {&g, &ldg, &pre, &ldp, &out, &part, &rows, &channels};
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      at[0].val.programmaticStreamSerializationAllowed = 1;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(cols, static_cast<unsigned>(runs));
      cfg.blockDim = dim3(lanes, streams);
      cfg.stream = s;
      cfg.attrs = at;
      cfg.numAttrs = 1;
      const void* k = bf16 ? act_grad_kernel<true>(a.act) : act_grad_kernel<false>(a.act);
      cudaError_t e;
      SC_LAUNCH("act_grad", s, e = cudaLaunchKernelExC(&cfg, k, args));
      if (e != cudaSuccess) st = set_cuda_error(e, "activation gradient launch");
      if (!st && a.gbias) st = column_join(part, static_cast<int>(runs), a.c_out, a.gbias, s);
    }
  }
  if (!st && a.gin.data) {  // rows x c_in, summed over c_out
    Product p{};
    p.k = a.c_out;
    p.ep.out = a.gin.data, p.ep.ldo = a.gin.stride, p.ep.bf16 = bf16;
    st = run(p, {gz.data, gz.stride, false}, {a.W, a.c_out, false}, a.rows, a.c_in, s);
  }
  if (!st && a.gW) {  // c_in x c_out, summed over rows
    Product p{};
    p.a = {a.x.data, a.x.stride, true};
    p.b = {gz.data, gz.stride, true};
    p.m = a.c_in, p.n = a.c_out, p.k = a.rows;
    p.ep.out = a.gW, p.ep.ldo = a.c_out, p.ep.bf16 = bf16;
    st = product_rows(p, s);
  }
  dev_free(part, s);
  dev_free(buf, s);
  return st;
}

}  // namespace sc
