// C ABI of the operators on rows (declared in include/sc.h): argument checks, then
// the kernels of add_norm.cu, linear*.cu and grad_clip.cu.
#include <cuda.h>

#include <cmath>
#include <string>
#include <utility>

#include "linear_internal.cuh"
#include "views.cuh"

using namespace sc;

namespace {

// A view of rows as one head a row: its checks and the memory it spans.
sc_status take(const char* what, const void* data, int64_t stride, int64_t rows, int channels, int eb, bool apart,
               Span* span) {
  return check_heads(what, data, stride, 0, rows, 1, channels, eb, apart, span);
}
sc_status take_in(const char* what, const sc_rows* v, int64_t rows, int channels, int eb, bool apart, sc_rows* dst,
                  Span* span) {
  if (!v) return invalid(std::string(what) + " is NULL");
  *dst = *v;
  return take(what, v->data, v->stride, rows, channels, eb, apart, span);
}
sc_status take_out(const char* what, const sc_rows_out* v, int64_t rows, int channels, int eb, sc_rows_out* dst,
                   Span* span) {
  if (!v) return invalid(std::string(what) + " is NULL");
  *dst = *v;
  return take(what, v->data, v->stride, rows, channels, eb, true, span);
}
// A dense run of bytes.
Span dense(const void* p, int64_t bytes) {
  Span s;
  if (!p || bytes <= 0) return s;
  s.lo = reinterpret_cast<uintptr_t>(p);
  s.hi = s.lo + static_cast<uintptr_t>(bytes);
  s.width = bytes;
  s.n[0] = s.n[1] = 1;
  return s;
}
// Whether an output may stand where an input is: it overlaps it in no byte, or is that very view.
bool clear_of(const Span& out, const sc_rows_out& o, const Span& in, const sc_rows& i, bool may_be) {
  if (!overlap(out, in)) return true;
  return may_be && o.data == i.data && o.stride == i.stride;
}

// Checks many addresses: those in an allocation that the call has met already need no
// further asking (48 gradients and their outputs took 10 of a call's 17 us).
class Allocations {
 public:
  sc_status check(const void* p, size_t align, const char* what) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    for (const auto& r : last_)
      if (at >= r.first && at < r.second && at % align == 0) return SC_OK;
    const sc_status st = check_dev_ptr(p, align, what);
    if (st) return st;
    static const AddressRangeFn range = address_range();
    CUdeviceptr base = 0;
    size_t bytes = 0;
    if (range && range(&base, &bytes, static_cast<CUdeviceptr>(at)) == CUDA_SUCCESS)
      last_[next_++ % 4] = {static_cast<uintptr_t>(base), static_cast<uintptr_t>(base) + bytes};
    return SC_OK;
  }

 private:
  typedef CUresult (*AddressRangeFn)(CUdeviceptr*, size_t*, CUdeviceptr);
  static AddressRangeFn address_range() {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuMemGetAddressRange", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    return reinterpret_cast<AddressRangeFn>(f);
  }
  std::pair<uintptr_t, uintptr_t> last_[4] = {};
  unsigned next_ = 0;
};

sc_status norm_sizes(int64_t rows, int channels, float eps, sc_dtype dtype) {
  if (dtype != SC_F32 && dtype != SC_F16 && dtype != SC_BF16) return invalid("rows must be f32, f16 or bf16");
  if (rows < 0 || rows > 0x7fffff00) return invalid("rows must be in [0, 2^31 - 256]");
  if (channels < 8 || channels > 16384 || channels % 8)
    return set_error(SC_ERR_UNSUPPORTED, "channels must be a multiple of 8 in [8, 16384]");
  if (!std::isfinite(eps) || eps < 0.f) return invalid("eps must be finite and not negative");
  return SC_OK;
}

sc_status linear_sizes(int64_t rows, int c_in, int c_out, int unit_in, int act) {
  if (rows < 0 || rows > 0x7fffff00) return invalid("rows must be in [0, 2^31 - 256]");
  if (c_in < unit_in || c_in > 65536 || c_in % unit_in || c_out < 8 || c_out > 65536 || c_out % 8)
    return set_error(SC_ERR_UNSUPPORTED, unit_in == 8 ? "c_in and c_out must be multiples of 8 up to 65536"
                                                      : "c_in must be a multiple of 16 and c_out of 8, up to 65536");
  if (act < SC_ACT_NONE || act > SC_ACT_SILU) return invalid("unknown activation");
  return SC_OK;
}

}  // namespace

extern "C" {

sc_status sc_add_norm_fwd(const sc_rows* x, const sc_rows* res, const sc_rows_out* sum, const sc_rows_out* out,
                          float* d_scale, const float* d_w, int64_t rows, int channels, float eps, sc_dtype dtype,
                          sc_dtype out_dtype, sc_stream stream) {
  sc_status st = norm_sizes(rows, channels, eps, dtype);
  if (st) return st;
  const bool e4m3 = out_dtype == SC_E4M3;
  if (!e4m3 && out_dtype != dtype) return invalid("out_dtype must be dtype or SC_E4M3");
  if (!e4m3 && !d_w) return invalid("norm weights may be NULL for 8-bit output only");
  if (!e4m3 && d_scale) return invalid("d_scale is for 8-bit output only");
  if (rows == 0) return SC_OK;
  NormArgs a{};
  a.rows = rows;
  a.channels = channels;
  a.eps = eps;
  a.dtype = dtype;
  a.e4m3 = e4m3;
  a.w = d_w;
  a.scale = d_scale;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  const int eb = dtype == SC_F32 ? 4 : 2;
  Span sx, sr, ss, so;
  if ((st = take_in("x", x, rows, channels, eb, false, &a.x, &sx))) return st;
  if (res && (st = take_in("res", res, rows, channels, eb, false, &a.res, &sr))) return st;
  if (sum && (st = take_out("sum", sum, rows, channels, eb, &a.sum, &ss))) return st;
  if (e4m3) {
    // stored eight values at a time, so that rows of 8, 24, ... channels may be dense
    if (!out) return invalid("out is NULL");
    a.out = *out;
    if ((st = check_heads("out", out->data, out->stride, 0, rows, 1, channels, 1, true, &so, 8))) return st;
    if ((st = check_dev_ptr(d_scale, 4, "scales"))) return st;
  } else if ((st = take_out("out", out, rows, channels, eb, &a.out, &so))) {
    return st;
  }
  if (d_w && (st = check_dev_ptr(d_w, 16, "norm weights"))) return st;
  const Span sw = dense(d_w, 4ll * channels), sc = dense(e4m3 ? d_scale : nullptr, 4 * rows);
  if (!clear_of(so, a.out, sx, a.x, !e4m3) || (res && !clear_of(so, a.out, sr, a.res, !e4m3)))
    return invalid("out overlaps an input");
  if (sum && (!clear_of(ss, a.sum, sx, a.x, true) || (res && !clear_of(ss, a.sum, sr, a.res, true))))
    return invalid("sum overlaps an input");
  if (sum && overlap(ss, so)) return invalid("the outputs overlap");
  if (overlap(so, sw) || overlap(so, sc) || overlap(sc, sx) || overlap(sc, sw) || (res && overlap(sc, sr)) ||
      (sum && (overlap(ss, sw) || overlap(ss, sc))))
    return invalid("an output overlaps the weights, the scales or an input");
  return add_norm_fwd(a);
}

sc_status sc_add_norm_bwd(const sc_rows* gout, const sc_rows* h, const sc_rows* gsum, const sc_rows_out* gin,
                          float* d_gw, const float* d_w, int64_t rows, int channels, float eps, sc_dtype dtype,
                          sc_stream stream) {
  sc_status st = norm_sizes(rows, channels, eps, dtype);
  if (st) return st;
  NormArgs a{};
  a.rows = rows;
  a.channels = channels;
  a.eps = eps;
  a.dtype = dtype;
  a.w = d_w;
  a.gw = d_gw;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  if (d_gw && (st = check_dev_ptr(d_gw, 4, "weight gradients"))) return st;
  if (rows > 0) {
    const int eb = dtype == SC_F32 ? 4 : 2;
    Span sg, sh, ss, so;
    if ((st = take_in("gout", gout, rows, channels, eb, false, &a.gout, &sg))) return st;
    if ((st = take_in("h", h, rows, channels, eb, false, &a.x, &sh))) return st;
    if (gsum && (st = take_in("gsum", gsum, rows, channels, eb, false, &a.res, &ss))) return st;
    if ((st = take_out("gin", gin, rows, channels, eb, &a.out, &so))) return st;
    if ((st = check_dev_ptr(d_w, 16, "norm weights"))) return st;
    if (!clear_of(so, a.out, sg, a.gout, true) || !clear_of(so, a.out, sh, a.x, true) ||
        (gsum && !clear_of(so, a.out, ss, a.res, true)))
      return invalid("gin overlaps an input");
    const Span sw = dense(d_w, 4ll * channels), sgw = dense(d_gw, 4ll * channels);
    if (overlap(so, sw) || overlap(so, sgw) || overlap(sgw, sw) || overlap(sgw, sg) || overlap(sgw, sh) ||
        (gsum && overlap(sgw, ss)))
      return invalid("a gradient overlaps an input or another gradient");
  }
  return add_norm_bwd(a);
}

sc_status sc_linear_fwd(const sc_rows* x, const void* d_W, const float* d_scale_x, const float* d_scale_w,
                        const float* d_bias, const sc_rows* res, const sc_rows_out* out, const sc_rows_out* pre,
                        int64_t rows, int c_in, int c_out, sc_act act, sc_dtype in_dtype, sc_dtype dtype,
                        sc_stream stream) {
  const bool e4m3 = in_dtype == SC_E4M3;
  if (dtype == SC_F32 || in_dtype == SC_F32) return set_error(SC_ERR_UNSUPPORTED, "linear layers take f16 or bf16");
  if (dtype != SC_F16 && dtype != SC_BF16) return invalid("the outputs' dtype must be f16 or bf16");
  if (!e4m3 && in_dtype != dtype) return invalid("in_dtype must be dtype or SC_E4M3");
  sc_status st = linear_sizes(rows, c_in, c_out, e4m3 ? 16 : 8, act);
  if (st) return st;
  if (!e4m3 && (d_scale_x || d_scale_w)) return invalid("scales are for 8-bit rows and weights only");
  if (rows == 0) return SC_OK;
  LinearArgs a{};
  a.W = d_W;
  a.scale_x = d_scale_x;
  a.scale_w = d_scale_w;
  a.bias = d_bias;
  a.rows = rows;
  a.c_in = c_in;
  a.c_out = c_out;
  a.in = in_dtype;
  a.dtype = dtype;
  a.act = act;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  const int ei = e4m3 ? 1 : 2;
  Span sx, sr, so, sp;
  if ((st = take_in("x", x, rows, c_in, ei, true, &a.x, &sx))) return st;
  if (res && (st = take_in("res", res, rows, c_out, 2, true, &a.res, &sr))) return st;
  if ((st = take_out("out", out, rows, c_out, 2, &a.out, &so))) return st;
  if (pre && (st = take_out("pre", pre, rows, c_out, 2, &a.pre, &sp))) return st;
  if ((st = check_dev_ptr(d_W, 16, "W"))) return st;
  if (e4m3 && ((st = check_dev_ptr(d_scale_x, 4, "scales of x")) || (st = check_dev_ptr(d_scale_w, 16, "scales of W"))))
    return st;
  if (d_bias && (st = check_dev_ptr(d_bias, 16, "bias"))) return st;
  const Span in[5] = {sx, dense(d_W, static_cast<int64_t>(c_in) * c_out * ei), dense(d_scale_x, 4 * rows),
                      dense(d_scale_w, 4ll * c_out), dense(d_bias, 4ll * c_out)};
  for (const Span& s : in)
    if (overlap(so, s) || (pre && overlap(sp, s))) return invalid("an output overlaps an input");
  if (res && (!clear_of(so, a.out, sr, a.res, true) || (pre && overlap(sp, sr))))
    return invalid("an output overlaps res");
  if (pre && overlap(sp, so)) return invalid("the outputs overlap");
  return linear_fwd(a);
}

sc_status sc_linear_bwd(const sc_rows* gout, const sc_rows* x, const sc_rows* pre, const void* d_W,
                        const sc_rows_out* gin, void* d_gW, float* d_gbias, int64_t rows, int c_in, int c_out,
                        sc_act act, sc_dtype dtype, sc_stream stream) {
  if (dtype == SC_F32) return set_error(SC_ERR_UNSUPPORTED, "linear layers take f16 or bf16");
  if (dtype != SC_F16 && dtype != SC_BF16) return invalid("dtype must be f16 or bf16");
  sc_status st = linear_sizes(rows, c_in, c_out, 8, act);
  if (st) return st;
  LinearBwdArgs a{};
  a.W = d_W;
  a.gW = d_gW;
  a.gbias = d_gbias;
  a.rows = rows;
  a.c_in = c_in;
  a.c_out = c_out;
  a.dtype = dtype;
  a.act = act;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  const int64_t wb = static_cast<int64_t>(c_in) * c_out * 2;
  if (d_gW && (st = check_dev_ptr(d_gW, 16, "weight gradients"))) return st;
  if (d_gbias && (st = check_dev_ptr(d_gbias, 4, "bias gradients"))) return st;
  Span sg, sx, sp, so;
  Span sw, sgw = dense(d_gW, wb), sgb = dense(d_gbias, 4ll * c_out);
  if (overlap(sgw, sgb)) return invalid("the gradients overlap");
  if (rows > 0 && (gin || d_gW || d_gbias)) {
    if ((st = take_in("gout", gout, rows, c_out, 2, true, &a.gout, &sg))) return st;
    if (act != SC_ACT_NONE && (st = take_in("pre", pre, rows, c_out, 2, false, &a.pre, &sp))) return st;
    if (d_gW && (st = take_in("x", x, rows, c_in, 2, true, &a.x, &sx))) return st;
    if (gin) {
      if ((st = take_out("gin", gin, rows, c_in, 2, &a.gin, &so))) return st;
      if ((st = check_dev_ptr(d_W, 16, "W"))) return st;
      sw = dense(d_W, wb);
    }
    const Span in[4] = {sg, sx, sp, sw};
    for (const Span& s : in)
      if (overlap(so, s) || overlap(sgw, s) || overlap(sgb, s)) return invalid("a gradient overlaps an input");
    if (overlap(so, sgw) || overlap(so, sgb)) return invalid("the gradients overlap");
  } else if (rows > 0) {
    return SC_OK;
  }
  return linear_bwd(a);
}

sc_status sc_rows_check(sc_stream stream) {
  int bits = 0;
  const sc_status st = rows_take_status(reinterpret_cast<cudaStream_t>(stream), &bits);
  return st ? st : status_from_bits(bits);
}

sc_status sc_grad_clip(const sc_grad* grads, int64_t count, float max_norm, float* d_norm, sc_stream stream) {
  if (count < 0 || count > (1 << 24)) return invalid("the number of gradients must be in [0, 2^24]");
  if (count > 0 && !grads) return invalid("grads is NULL");
  if (!(max_norm >= 0.f)) return invalid("max_norm must not be negative or NaN");
  sc_status st = check_dev_ptr(d_norm, 4, "norm");
  if (st) return st;
  Allocations seen;
  for (int64_t i = 0; i < count; ++i) {
    const sc_grad& g = grads[i];
    if (g.dtype != SC_F32 && g.dtype != SC_F16 && g.dtype != SC_BF16)
      return invalid("gradient " + std::to_string(i) + ": must be f32, f16 or bf16");
    if (g.n < 0 || g.n > (int64_t(1) << 40)) return invalid("gradient " + std::to_string(i) + ": bad size");
    if (g.n == 0) continue;
    const uintptr_t size = g.dtype == SC_F32 ? 4 : 2;
    if (!g.data || !g.out || reinterpret_cast<uintptr_t>(g.data) % size || reinterpret_cast<uintptr_t>(g.out) % size)
      return invalid("gradient " + std::to_string(i) + ": NULL or not aligned to its type");
    // a shift of a few values would be read after it was written
    const uintptr_t d = reinterpret_cast<uintptr_t>(g.data), o = reinterpret_cast<uintptr_t>(g.out);
    const uintptr_t bytes = static_cast<uintptr_t>(g.n) * size;
    if (d != o && d < o + bytes && o < d + bytes)
      return invalid("gradient " + std::to_string(i) + ": out overlaps data without being it");
    // a block writes the norm while others still scale
    const uintptr_t at = reinterpret_cast<uintptr_t>(d_norm);
    if ((at < d + bytes && d < at + 4) || (at < o + bytes && o < at + 4))
      return invalid("gradient " + std::to_string(i) + ": the norm lies among its values");
    if ((st = seen.check(g.data, size, "a gradient"))) return st;
    if (g.out != g.data && (st = seen.check(g.out, size, "a gradient's output"))) return st;
  }
  return grad_clip(grads, count, max_norm, d_norm, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
