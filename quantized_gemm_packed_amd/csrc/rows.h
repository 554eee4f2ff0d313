// Which bytes strided tensors share (host code): the checks of calls whose
// outputs may not overlap what other workgroups still read.
#pragma once

#include <cstdint>

namespace hum {

typedef __int128 wide_t;  // (strides are the caller's: no product of them overflows)

// The rows of a [tokens][heads][row] tensor, in bytes.
struct Rows {
  int64_t at;  // address of the first row
  int64_t tokens, heads;
  wide_t ts, hs;  // from token to token, from head to head; any sign
  int64_t row;    // bytes of a row
};
inline Rows bytes_at(const void* p, int64_t bytes) { return Rows{(int64_t)(intptr_t)p, 1, 1, 0, 0, bytes}; }

enum class Overlap { kNo, kYes, kUnknown };

namespace rows_detail {

typedef wide_t wide;

inline wide floor_div(wide a, wide b) {  // b > 0
  return a >= 0 ? a / b : -((-a + b - 1) / b);
}
inline wide ceil_div(wide a, wide b) { return -floor_div(-a, b); }

// One tensor with strides >= 0, 0 where it has one token or head.
struct Norm {
  wide at, ts, hs, row;
  int64_t tokens, heads;
  explicit Norm(const Rows& r) : at(r.at), ts(r.tokens > 1 ? r.ts : 0), hs(r.heads > 1 ? r.hs : 0), row(r.row), tokens(r.tokens), heads(r.heads) {
    if (ts < 0) {
      at += (tokens - 1) * ts;
      ts = -ts;
    }
    if (hs < 0) {
      at += (heads - 1) * hs;
      hs = -hs;
    }
  }
  bool empty() const { return tokens < 1 || heads < 1 || row < 1; }
  wide end() const { return at + (tokens - 1) * ts + (heads - 1) * hs + row; }
};

// Whether -la < base + i * so + j * si < lb for an i in [i0, i1] and a j in
// [j0, j1], (0, 0) left out where `self`.  so >= si >= 0.
inline bool hits(wide base, wide so, wide i0, wide i1, wide si, wide j0, wide j1, wide la, wide lb, bool self) {
  if (so > 0) {  // only the i from which some j reaches the interval
    const wide lo = ceil_div(1 - la - base - j1 * si, so), hi = floor_div(lb - 1 - base - j0 * si, so);
    if (lo > i0) i0 = lo;
    if (hi < i1) i1 = hi;
  } else if (!self) {
    i0 = i1 = 0;  // (0 lies in every such range)
  }
  for (wide i = i0; i <= i1; ++i) {
    const wide b = base + i * so;
    wide lo = j0, hi = j1;
    if (si > 0) {
      const wide l = ceil_div(1 - la - b, si), h = floor_div(lb - 1 - b, si);
      if (l > lo) lo = l;
      if (h < hi) hi = h;
    } else if (!(b > -la && b < lb)) {
      continue;
    }
    if (lo > hi) continue;
    if (self && i == 0 && lo == 0 && hi == 0) continue;
    return true;
  }
  return false;
}

// Whether rows of a and b meet, which have the strides ts and hs where they
// have any: their rows' distances are then base + i ts + j hs.
inline bool meet(const Norm& a, const Norm& b, wide ts, wide hs) {
  const wide base = a.at - b.at, t0 = 1 - b.tokens, t1 = a.tokens - 1, h0 = 1 - b.heads, h1 = a.heads - 1;
  return ts >= hs ? hits(base, ts, t0, t1, hs, h0, h1, a.row, b.row, false)
                  : hits(base, hs, h0, h1, ts, t0, t1, a.row, b.row, false);
}

}  // namespace rows_detail

// Whether two rows of r share a byte.
inline bool overlaps_itself(const Rows& r) {
  using namespace rows_detail;
  const Norm a(r);
  if (a.empty()) return false;
  const bool by_token = a.ts >= a.hs;
  const wide so = by_token ? a.ts : a.hs, si = by_token ? a.hs : a.ts;
  const wide no = by_token ? a.tokens : a.heads, ni = by_token ? a.heads : a.tokens;
  if ((ni == 1 || si >= a.row) && (no == 1 || so >= (ni - 1) * si + a.row)) return false;
  return hits(0, so, 1 - no, no - 1, si, 1 - ni, ni - 1, a.row, a.row, true);
}

// Whether a row of x and a row of y share a byte.  kUnknown only for tensors
// that lie in one another, with different strides and more than 2^20 rows
// each.
inline Overlap overlap(const Rows& x, const Rows& y) {
  using namespace rows_detail;
  const Norm a(x), b(y);
  if (a.empty() || b.empty() || a.end() <= b.at || b.end() <= a.at) return Overlap::kNo;
  auto yes = [](bool v) { return v ? Overlap::kYes : Overlap::kNo; };
  const bool ts = a.tokens == 1 || b.tokens == 1 || a.ts == b.ts, hs = a.heads == 1 || b.heads == 1 || a.hs == b.hs;
  if (ts && hs) return yes(meet(a, b, a.tokens > 1 ? a.ts : b.ts, a.heads > 1 ? a.hs : b.hs));
  // one row of the smaller at a time: any strides are its own
  const bool swap = (wide)a.tokens * a.heads > (wide)b.tokens * b.heads;
  const Norm &few = swap ? b : a, &many = swap ? a : b;
  if ((wide)few.tokens * few.heads > 1 << 20) return Overlap::kUnknown;
  Norm one = few;
  one.tokens = one.heads = 1;
  for (int64_t t = 0; t < few.tokens; ++t)
    for (int64_t h = 0; h < few.heads; ++h) {
      one.at = few.at + t * few.ts + h * few.hs;
      if (meet(one, many, many.ts, many.hs)) return Overlap::kYes;
    }
  return Overlap::kNo;
}

}  // namespace hum
