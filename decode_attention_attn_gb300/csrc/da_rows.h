// da_rows.h -- host-side rules of the row operators' launches (host code only; no CUDA types):
// where strided row tensors lie, so that results over inputs are refused, and how many blocks share
// a row.
#pragma once

#include <cstdint>
#include <utility>

namespace da {

// Rows of a [rows, heads, d] tensor: runs of `run` bytes at address + r row + h head (bytes).
struct RowRuns {
  uint64_t address;
  int64_t rows, row, heads, head, run;
};

// Strides may be any 64-bit numbers; what is formed of them needs more.
typedef __int128 wide;

namespace rows_detail {

struct Span {   // [lo, hi)
  wide lo, hi;
};
// What `count` steps of `stride` from `address` reach, each `run` long.
inline Span reach(wide address, int64_t count, int64_t stride, wide run) {
  const wide far = (wide)(count - 1) * stride;
  return {address + (far < 0 ? far : 0), address + (far > 0 ? far : 0) + run};
}
inline uint64_t gcd(uint64_t a, uint64_t b) {
  while (b) {
    const uint64_t t = a % b;
    a = b;
    b = t;
  }
  return a;
}
inline uint64_t magnitude(int64_t x) { return x < 0 ? 0 - (uint64_t)x : (uint64_t)x; }

// Whether spans lie apart modulo m.
inline bool apart_modulo(const Span& a, const Span& b, wide m) {
  if (m <= 0) return false;
  wide d = (b.lo - a.lo) % m;
  if (d < 0) d += m;
  return d >= a.hi - a.lo && d + (b.hi - b.lo) <= m;
}

}  // namespace rows_detail

// Whether a result's rows lie apart from one another.
inline bool lie_apart(const RowRuns& t) {
  int64_t n = t.rows, s = t.row, n2 = t.heads, s2 = t.head;   // the smaller stride in s2
  if (n > 1 && (n2 == 1 || s < s2)) {
    std::swap(n, n2);
    std::swap(s, s2);
  }
  if (n2 > 1 && s2 < t.run) return false;
  return n <= 1 || (wide)s >= (wide)(n2 - 1) * s2 + t.run;
}

// Whether two tensors' rows may share memory. "No" is certain; tensors whose ranges overlap count as apart
// where they do so modulo what all their strides divide by, or modulo a stride that both have (parts
// of one tensor's rows, or of its heads).
inline bool may_share(const RowRuns& a, const RowRuns& b) {
  using namespace rows_detail;
  const Span ah = reach(a.address, a.heads, a.head, a.run), bh = reach(b.address, b.heads, b.head, b.run);
  const Span al = reach(ah.lo, a.rows, a.row, ah.hi - ah.lo), bl = reach(bh.lo, b.rows, b.row, bh.hi - bh.lo);
  if (al.hi <= bl.lo || bl.hi <= al.lo) return false;
  uint64_t g = 0;
  for (const RowRuns* t : {&a, &b}) {
    if (t->rows > 1) g = gcd(g, magnitude(t->row));
    if (t->heads > 1) g = gcd(g, magnitude(t->head));
  }
  const Span a0 = {(wide)a.address, (wide)a.address + a.run}, b0 = {(wide)b.address, (wide)b.address + b.run};
  if (apart_modulo(a0, b0, g)) return false;
  if ((a.rows == 1 || b.rows == 1 || a.row == b.row) &&
      apart_modulo(ah, bh, a.rows > 1 ? a.row : b.row))
    return false;
  if ((a.heads == 1 || b.heads == 1 || a.head == b.head) &&
      apart_modulo(reach(a.address, a.rows, a.row, a.run), reach(b.address, b.rows, b.row, b.run),
                   a.heads > 1 ? a.head : b.head))
    return false;
  return true;
}

// Whether a result may be written over or beside an input: apart from it, or the input itself.
inline bool result_ok(const RowRuns& in, const RowRuns& out) {
  if (in.address == out.address) return in.row == out.row && in.head == out.head;
  return !may_share(in, out);
}

// Blocks that a row's `passes` (of as many heads as a block takes at once) are spread over: where rows are few,
// as many as two blocks an SM allow.
inline int row_slices(int64_t rows, int passes, int sms) {
  const int64_t blocks = 2 * (int64_t)sms;
  const int64_t n = rows >= blocks ? 1 : (blocks + rows - 1) / rows;
  return n < passes ? (int)n : passes;
}

}  // namespace da
