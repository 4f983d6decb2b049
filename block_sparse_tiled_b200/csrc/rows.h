// Where the rows of a call's operands lie, for the checks that refuse outputs over memory that the call still reads or
// also writes.
#pragma once
#include <cstdint>

namespace vsa {

// n tokens of `heads` rows each, all in bytes: a row of `row` bytes, `hd` between heads, `ld` between tokens.
struct Rows {
  const void* base;
  int64_t n, ld, heads, hd, row;
};

using Wide = __int128;  // strides times counts may pass 64 bits in a call that is refused

inline Wide rows_begin(const Rows& a) { return static_cast<Wide>(reinterpret_cast<uintptr_t>(a.base)); }
inline Wide rows_end(const Rows& a) {
  return rows_begin(a) + static_cast<Wide>(a.n - 1) * a.ld + static_cast<Wide>(a.heads - 1) * a.hd + a.row;
}

// The same rows in the same places: an output that replaces an input.
inline bool same_rows(const Rows& a, const Rows& b) {
  return a.base == b.base && a.n == b.n && (a.n == 1 || a.ld == b.ld) && a.heads == b.heads &&
         (a.heads == 1 || a.hd == b.hd) && a.row == b.row;
}

// Whether no two rows of `a` share a byte: each token's heads inside its stride, or each head's tokens inside its own.
inline bool rows_disjoint(const Rows& a) {
  const bool token_major =
      (a.heads == 1 || a.hd >= a.row) && (a.n == 1 || a.ld >= static_cast<Wide>(a.heads - 1) * a.hd + a.row);
  const bool head_major =
      (a.n == 1 || a.ld >= a.row) && (a.heads == 1 || a.hd >= static_cast<Wide>(a.n - 1) * a.ld + a.row);
  return token_major || head_major;
}

// Whether combs of one period are apart: teeth of `a` bytes at 0, `period`, .., and of `b` bytes at d, d + period, ..
inline bool combs_apart(Wide d, Wide a, Wide b, Wide period) {
  if (period <= 0) return false;
  d = (d % period + period) % period;
  return d >= a && d + b <= period;
}

// Whether some row of `a` and some row of `b` share a byte.  Operands whose address ranges are apart do not, nor do
// slices of one projection: rows of equal strides that lie beside one another inside a token (or a head).  Every other
// layout in one address range counts as meeting.
inline bool rows_meet(const Rows& a, const Rows& b) {
  if (rows_end(a) <= rows_begin(b) || rows_end(b) <= rows_begin(a)) return false;
  const Wide d = rows_begin(b) - rows_begin(a);
  const bool same_ld = a.n == 1 || b.n == 1 || a.ld == b.ld, same_hd = a.heads == 1 || b.heads == 1 || a.hd == b.hd;
  const int64_t ld = a.n == 1 ? b.ld : a.ld, hd = a.heads == 1 ? b.hd : a.hd;
  const bool tokens = a.n > 1 || b.n > 1, heads = a.heads > 1 || b.heads > 1;
  const auto span = [](const Rows& r, bool of_tokens) {  // what a head's tokens cover, or a token's heads
    return static_cast<Wide>(of_tokens ? r.n - 1 : r.heads - 1) * (of_tokens ? r.ld : r.hd) + r.row;
  };
  if (tokens && same_ld && combs_apart(d, span(a, false), span(b, false), ld)) return false;
  if (heads && same_hd && combs_apart(d, span(a, true), span(b, true), hd)) return false;
  // rows beside one another inside a period that both strides keep
  if (tokens && same_ld && (!heads || (same_hd && hd > 0 && ld % hd == 0)) && combs_apart(d, a.row, b.row, heads ? hd : ld)) return false;
  if (heads && same_hd && (!tokens || (same_ld && ld > 0 && hd % ld == 0)) && combs_apart(d, a.row, b.row, tokens ? ld : hd)) return false;
  return true;
}

}  // namespace vsa
