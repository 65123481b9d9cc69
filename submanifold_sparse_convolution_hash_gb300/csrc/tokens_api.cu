// C ABI of the operators on token rows (declared in include/sc.h): argument
// checks, then the kernels of rope.cu and attn*.cu.
#include <cmath>
#include <string>

#include "sc_internal.cuh"

using namespace sc;

namespace {

sc_status invalid(const std::string& msg) { return set_error(SC_ERR_INVALID_ARG, msg.c_str()); }

// The bytes of a view of rows: [lo, hi) from its first to past its last value, and
// how they repeat: `n[0]` pieces of `width` bytes `step[0]` apart, n[1] of those
// step[1] apart, the larger step last.
struct Span {
  uintptr_t lo = 0, hi = 0;
  int64_t width = 0, step[2] = {0, 0}, n[2] = {0, 0};
};

// A view of `tokens` rows of `heads` heads of `d` values of `eb` bytes.
// `apart`: a view that is written, whose rows must not share memory.
sc_status check_heads(const char* what, const void* data, int64_t ts, int64_t hs, int64_t tokens, int heads, int d,
                      int eb, bool apart, Span* span) {
  const sc_status st = check_dev_ptr(data, 16, what);
  if (st) return st;
  const int64_t unit = 16 / eb;
  if (ts < 0 || hs < 0 || (tokens > 1 && ts % unit) || (heads > 1 && hs % unit))
    return invalid(std::string(what) + ": strides must be multiples of 16 bytes and not negative");
  if (ts > (int64_t(1) << 36) || hs > (int64_t(1) << 36)) return invalid(std::string(what) + ": stride too large");
  if (tokens <= 1) ts = 0;
  if (heads <= 1) hs = 0;
  // below 2^48 bytes, so that no offset passes 64 bits here or in the kernels
  if ((static_cast<double>(tokens - 1) * ts + static_cast<double>(heads - 1) * hs) * eb > 0x1p48)
    return invalid(std::string(what) + ": rows past the address space");
  if (apart) {
    const bool heads_ok = heads <= 1 || hs >= d;
    const bool tokens_inner = tokens > 1 && heads > 1 && hs >= (tokens - 1) * ts + d && ts >= d;
    const bool tokens_outer = tokens <= 1 || ts >= (heads - 1) * hs + d;
    if (!heads_ok || !(tokens_outer || tokens_inner)) return invalid(std::string(what) + ": rows overlap");
  }
  const bool by_token = ts >= hs;  // heads within a token, or tokens within a head
  span->width = static_cast<int64_t>(d) * eb;
  span->step[0] = (by_token ? hs : ts) * eb;
  span->step[1] = (by_token ? ts : hs) * eb;
  span->n[0] = by_token ? heads : tokens;
  span->n[1] = by_token ? tokens : heads;
  span->lo = reinterpret_cast<uintptr_t>(data);
  span->hi = span->lo + static_cast<uintptr_t>((tokens - 1) * ts * eb + (heads - 1) * hs * eb + span->width);
  return SC_OK;
}

// Whether pieces of `wa` bytes at `at` mod `pitch` and of `wb` at 0 can meet.
bool meet(int64_t at, int64_t wa, int64_t wb, int64_t pitch) {
  at = (at % pitch + pitch) % pitch;
  return at < wb || at + wa > pitch;
}

// Whether two views may share a byte.  Of views that repeat with the same outer step,
// as parts of one buffer do, the places within a step are compared: as whole runs,
// and where those meet (heads of one between heads of the other) piece by piece, up
// to 4096 of them.
bool overlap(const Span& a, const Span& b) {
  if (a.lo == a.hi || b.lo == b.hi || a.hi <= b.lo || b.hi <= a.lo) return false;
  const int64_t pitch = a.step[1];
  if (pitch == 0 || pitch != b.step[1]) return true;
  const int64_t at = static_cast<int64_t>(a.lo - b.lo);
  const int64_t ra = (a.n[0] - 1) * a.step[0] + a.width, rb = (b.n[0] - 1) * b.step[0] + b.width;
  if (ra <= pitch && rb <= pitch && !meet(at, ra, rb, pitch)) return false;
  if (a.step[0] == b.step[0]) {
    // only the difference of two places counts
    if (a.n[0] + b.n[0] > 4096) return true;
    for (int64_t i = 1 - b.n[0]; i < a.n[0]; ++i)
      if (meet(at + i * a.step[0], a.width, b.width, pitch)) return true;
    return false;
  }
  if (a.n[0] * b.n[0] > 4096) return true;
  for (int64_t i = 0; i < a.n[0]; ++i)
    for (int64_t j = 0; j < b.n[0]; ++j)
      if (meet(at + i * a.step[0] - j * b.step[0], a.width, b.width, pitch)) return true;
  return false;
}

sc_status check_ints(const void* p, const char* what) { return check_dev_ptr(p, 4, what); }

sc_status rope_call(const sc_heads* gout[2], const sc_heads* x[2], const sc_heads_out* y[2], float* gw[2],
                    const float* w[2], const int32_t* pos, int64_t pos_stride, int axes, const float* freq,
                    int64_t tokens, int heads_q, int heads_k, int head_dim, int rot_dim, float eps, float amp,
                    sc_dtype dtype, unsigned flags, sc_stream stream, bool bwd) {
  if (flags & ~SC_ROPE_INTERLEAVED) return invalid("unknown rotation flag");
  if (dtype != SC_F32 && dtype != SC_F16 && dtype != SC_BF16) return invalid("unknown dtype");
  if (tokens < 0 || tokens > 0x7fffffff || heads_q < 0 || heads_k < 0 || heads_q > 4096 || heads_k > 4096)
    return invalid("tokens must be in [0, 2^31) and the head counts in [0, 4096]");
  if (head_dim < 16 || head_dim > 256 || head_dim % 8)
    return set_error(SC_ERR_UNSUPPORTED, "head_dim must be a multiple of 8 in [16, 256]");
  if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 2) return invalid("rot_dim must be even and in [0, head_dim]");
  if (!std::isfinite(amp) || !std::isfinite(eps) || eps < 0.f) return invalid("amp and eps must be finite, eps >= 0");
  const int heads[2] = {heads_q, heads_k};
  const bool norm = w[0] || w[1];
  if (norm) {  // both are written, that of a side without rows with zeros
    for (int s = 0; s < 2; ++s) {
      const sc_status st = gw[s] ? check_dev_ptr(gw[s], 4, "weight gradients") : SC_OK;
      if (st) return st;
    }
  }
  RopeArgs a{};
  if (tokens > 0 && heads_q + heads_k > 0) {
    sc_status st;
    if (rot_dim > 0) {
      if (axes < 1 || axes > 4 || (rot_dim / 2) % axes)
        return invalid("axes must be in [1, 4] and divide rot_dim / 2");
      if (pos_stride < 0 || (tokens > 1 && pos_stride > (int64_t(1) << 32))) return invalid("bad position stride");
      if ((st = check_ints(pos, "positions"))) return st;
      if ((st = check_dev_ptr(freq, 4, "frequencies"))) return st;
    }
    const int eb = dtype == SC_F32 ? 4 : 2;
    Span in[4], out[2];
    const char* names[2][3] = {{"q", "the gradient of q's output", "q's output"},
                               {"k", "the gradient of k's output", "k's output"}};
    for (int s = 0; s < 2; ++s) {
      if (!heads[s]) continue;
      if (norm && !w[s]) return invalid("norm weights: both sides that have heads need one, or neither");
      if (norm && (st = check_dev_ptr(w[s], 4, "norm weights"))) return st;
      if (!y[s] || (bwd && !gout[s])) return invalid(std::string(names[s][2]) + " is NULL");
      if (!bwd || norm) {
        if (!x[s]) return invalid(std::string(names[s][0]) + " is NULL");
        if ((st = check_heads(names[s][0], x[s]->data, x[s]->token_stride, x[s]->head_stride, tokens, heads[s],
                              head_dim, eb, false, &in[s])))
          return st;
        a.x[s] = *x[s];
      }
      if (bwd) {
        if ((st = check_heads(names[s][1], gout[s]->data, gout[s]->token_stride, gout[s]->head_stride, tokens,
                              heads[s], head_dim, eb, false, &in[2 + s])))
          return st;
        a.gy[s] = *gout[s];
      }
      if ((st = check_heads(names[s][2], y[s]->data, y[s]->token_stride, y[s]->head_stride, tokens, heads[s],
                            head_dim, eb, true, &out[s])))
        return st;
      a.y[s] = *y[s];
    }
    // a row may be overwritten in place (the forward's input, the backward's gout), nothing else
    for (int s = 0; s < 2; ++s) {
      if (!heads[s]) continue;
      for (int i = 0; i < 4; ++i) {
        if (!overlap(out[s], in[i])) continue;
        const sc_heads& v = i < 2 ? a.x[i] : a.gy[i - 2];
        const bool same = v.data == a.y[s].data && v.token_stride == a.y[s].token_stride &&
                          v.head_stride == a.y[s].head_stride && i == (bwd ? 2 + s : s);
        if (!same) return invalid(std::string(names[s][2]) + " overlaps an input");
      }
    }
    if (overlap(out[0], out[1])) return invalid("the outputs overlap");
  }
  for (int s = 0; s < 2; ++s) {
    a.w[s] = w[s];
    a.gw[s] = gw[s];
  }
  a.pos = pos;
  a.pos_stride = pos_stride;
  a.axes = axes;
  a.freq = freq;
  a.tokens = tokens;
  a.heads_q = heads_q;
  a.heads_k = heads_k;
  a.head_dim = head_dim;
  a.rot_dim = rot_dim;
  a.eps = eps;
  a.amp = amp;
  a.dtype = dtype;
  a.interleaved = (flags & SC_ROPE_INTERLEAVED) != 0;
  a.backward = bwd;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  return rope_run(a);
}

sc_status attn_sizes(const AttnArgs& a, unsigned flags) {
  if (flags & ~SC_ATTN_CAUSAL) return invalid("unknown attention flag");
  if (a.dtype != SC_F32 && a.dtype != SC_F16 && a.dtype != SC_BF16) return invalid("unknown dtype");
  if (a.dtype == SC_F32) return set_error(SC_ERR_UNSUPPORTED, "attention takes f16 or bf16");
  if (a.n_seq < 0 || a.n_seq >= (1 << 20) || a.t_q < 0 || a.t_k < 0 || a.t_q > 0x7fffff00 || a.t_k > 0x7fffff00)
    return invalid("n_seq must be in [0, 2^20), token counts in [0, 2^31 - 256]");
  if (a.heads_q < 1 || a.heads_kv < 1 || a.heads_q % a.heads_kv)
    return invalid("heads_q must be a positive multiple of heads_kv");
  if (a.heads_q > 65535 || a.heads_q / a.heads_kv > 128)
    return set_error(SC_ERR_UNSUPPORTED, "at most 128 query heads a key head, 65535 in all");
  if (a.head_dim < 16 || a.head_dim > 128 || a.head_dim % 8)
    return set_error(SC_ERR_UNSUPPORTED, "head_dim must be a multiple of 8 in [16, 128]");
  if (!(a.scale > 0.f) || !std::isfinite(a.scale * 1.4426950408889634f))
    return invalid("scale must be positive and, times log2 e, finite");
  if (a.n_seq == 0 && a.t_q > 0) return invalid("query rows, but no sequence");
  sc_status st = SC_OK;
  if (a.n_seq > 0) {
    if ((st = check_ints(a.q_off, "query offsets"))) return st;
    if ((st = check_ints(a.k_off, "key offsets"))) return st;
    if (a.k_len && (st = check_ints(a.k_len, "key lengths"))) return st;
  }
  return st;
}

// One input view into *dst and its span; a view without rows is not looked at.
sc_status take_in(const char* what, const sc_heads* v, int64_t tokens, int heads, int d, sc_heads* dst, Span* span) {
  if (tokens == 0) return SC_OK;
  if (!v) return invalid(std::string(what) + " is NULL");
  const sc_status st = check_heads(what, v->data, v->token_stride, v->head_stride, tokens, heads, d, 2, false, span);
  *dst = *v;
  return st;
}
sc_status take_out(const char* what, const sc_heads_out* v, int64_t tokens, int heads, int d, sc_heads_out* dst,
                   Span* span) {
  if (tokens == 0) return SC_OK;
  if (!v) return invalid(std::string(what) + " is NULL");
  const sc_status st = check_heads(what, v->data, v->token_stride, v->head_stride, tokens, heads, d, 2, true, span);
  *dst = *v;
  return st;
}

}  // namespace

extern "C" {

sc_status sc_qk_norm_rope_fwd(const sc_heads* q, const sc_heads* k, const sc_heads_out* out_q,
                              const sc_heads_out* out_k, const float* d_w_q, const float* d_w_k,
                              const int32_t* d_pos, int64_t pos_stride, int axes, const float* d_freq,
                              int64_t tokens, int heads_q, int heads_k, int head_dim, int rot_dim, float eps,
                              float amp, sc_dtype dtype, unsigned flags, sc_stream stream) {
  const sc_heads *g[2] = {nullptr, nullptr}, *x[2] = {q, k};
  const sc_heads_out* y[2] = {out_q, out_k};
  float* gw[2] = {nullptr, nullptr};
  const float* w[2] = {d_w_q, d_w_k};
  return rope_call(g, x, y, gw, w, d_pos, pos_stride, axes, d_freq, tokens, heads_q, heads_k, head_dim, rot_dim, eps,
                   amp, dtype, flags, stream, false);
}

sc_status sc_qk_norm_rope_bwd(const sc_heads* gout_q, const sc_heads* gout_k, const sc_heads* q, const sc_heads* k,
                              const sc_heads_out* gin_q, const sc_heads_out* gin_k, float* d_gw_q, float* d_gw_k,
                              const float* d_w_q, const float* d_w_k, const int32_t* d_pos, int64_t pos_stride,
                              int axes, const float* d_freq, int64_t tokens, int heads_q, int heads_k, int head_dim,
                              int rot_dim, float eps, float amp, sc_dtype dtype, unsigned flags, sc_stream stream) {
  const sc_heads *g[2] = {gout_q, gout_k}, *x[2] = {q, k};
  const sc_heads_out* y[2] = {gin_q, gin_k};
  float* gw[2] = {d_gw_q, d_gw_k};
  const float* w[2] = {d_w_q, d_w_k};
  return rope_call(g, x, y, gw, w, d_pos, pos_stride, axes, d_freq, tokens, heads_q, heads_k, head_dim, rot_dim, eps,
                   amp, dtype, flags, stream, true);
}

sc_status sc_attn_fwd(const sc_heads* q, const sc_heads* k, const sc_heads* v, const sc_heads_out* out,
                      float* d_lse, const int32_t* d_q_off, const int32_t* d_k_off, const int32_t* d_k_len,
                      int64_t n_seq, int64_t t_q, int64_t t_k, int heads_q, int heads_kv, int head_dim, float scale,
                      sc_dtype dtype, unsigned flags, sc_stream stream) {
  AttnArgs a{};
  a.q_off = d_q_off;
  a.k_off = d_k_off;
  a.k_len = d_k_len;
  a.n_seq = n_seq;
  a.t_q = t_q;
  a.t_k = t_k;
  a.heads_q = heads_q;
  a.heads_kv = heads_kv;
  a.head_dim = head_dim;
  a.scale = scale;
  a.dtype = dtype;
  a.causal = (flags & SC_ATTN_CAUSAL) != 0;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  a.lse = d_lse;
  sc_status st = attn_sizes(a, flags);
  if (st) return st;
  Span s[4];
  if ((st = take_in("q", q, t_q, heads_q, head_dim, &a.q, &s[0]))) return st;
  if ((st = take_in("k", k, t_k, heads_kv, head_dim, &a.k, &s[1]))) return st;
  if ((st = take_in("v", v, t_k, heads_kv, head_dim, &a.v, &s[2]))) return st;
  if ((st = take_out("out", out, t_q, heads_q, head_dim, &a.out, &s[3]))) return st;
  if (t_q == 0) return SC_OK;
  if (d_lse && (st = check_dev_ptr(d_lse, 4, "lse"))) return st;
  for (int i = 0; i < 3; ++i)
    if (overlap(s[i], s[3])) return invalid("out overlaps q, k or v");
  return attn_fwd(a);
}

sc_status sc_attn_bwd(const sc_heads* gout, const sc_heads* q, const sc_heads* k, const sc_heads* v,
                      const sc_heads* out, const float* d_lse, const sc_heads_out* gq, const sc_heads_out* gk,
                      const sc_heads_out* gv, const int32_t* d_q_off, const int32_t* d_k_off, int64_t n_seq,
                      int64_t t_q, int64_t t_k, int heads_q, int heads_kv, int head_dim, float scale,
                      sc_dtype dtype, unsigned flags, sc_stream stream) {
  AttnArgs a{};
  a.q_off = d_q_off;
  a.k_off = d_k_off;
  a.n_seq = n_seq;
  a.t_q = t_q;
  a.t_k = t_k;
  a.heads_q = heads_q;
  a.heads_kv = heads_kv;
  a.head_dim = head_dim;
  a.scale = scale;
  a.dtype = dtype;
  a.causal = (flags & SC_ATTN_CAUSAL) != 0;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  a.lse = const_cast<float*>(d_lse);
  sc_status st = attn_sizes(a, flags);
  if (st) return st;
  if (n_seq == 0 && t_k > 0) return invalid("key rows, but no sequence");
  Span s[8];
  if ((st = take_in("gout", gout, t_q, heads_q, head_dim, &a.gout, &s[0]))) return st;
  if ((st = take_in("q", q, t_q, heads_q, head_dim, &a.q, &s[1]))) return st;
  if ((st = take_in("k", k, t_k, heads_kv, head_dim, &a.k, &s[2]))) return st;
  if ((st = take_in("v", v, t_k, heads_kv, head_dim, &a.v, &s[3]))) return st;
  if ((st = take_in("out", out, t_q, heads_q, head_dim, &a.out_in, &s[4]))) return st;
  if ((st = take_out("gq", gq, t_q, heads_q, head_dim, &a.gq, &s[5]))) return st;
  if ((st = take_out("gk", gk, t_k, heads_kv, head_dim, &a.gk, &s[6]))) return st;
  if ((st = take_out("gv", gv, t_k, heads_kv, head_dim, &a.gv, &s[7]))) return st;
  if (t_q > 0 && (st = check_dev_ptr(d_lse, 4, "lse"))) return st;
  for (int o = 5; o < 8; ++o)
    for (int i = 0; i < o; ++i)
      if (overlap(s[i], s[o])) return invalid("a gradient overlaps an input or another gradient");
  if (t_q == 0 && t_k == 0) return SC_OK;
  return attn_bwd(a);
}

sc_status sc_attn_check(sc_stream stream) {
  int bits = 0;
  const sc_status st = attn_take_status(reinterpret_cast<cudaStream_t>(stream), &bits);
  if (st) return st;
  if (bits & kDevErrRange) return set_error(SC_ERR_OUT_OF_RANGE, "sequence offsets decrease or leave the rows");
  return status_from_bits(bits);
}

}  // extern "C"
