// Checks of the strided views that the entry points take: their addresses and
// strides, and whether two of them share memory.
#pragma once

#include <string>

#include "sc_internal.cuh"

namespace sc {
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
// `align`: bytes that the address and the strides are multiples of.
sc_status check_heads(const char* what, const void* data, int64_t ts, int64_t hs, int64_t tokens, int heads, int d,
                      int eb, bool apart, Span* span, int align = 16) {
  const sc_status st = check_dev_ptr(data, align, what);
  if (st) return st;
  const int64_t unit = align / eb;
  if (ts < 0 || hs < 0 || (tokens > 1 && ts % unit) || (heads > 1 && hs % unit))
    return invalid(std::string(what) + ": strides must be multiples of " + std::to_string(align) +
                   " bytes and not negative");
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

}  // namespace
}  // namespace sc
