// na_packed.cuh -- what the packed-attention kernels share: where a sequence
// lies, which keys a row sees, and which sequence a block works on.
//
// Rows.  A row of the kernels is one (position, head) pair of a group of
// G = heads_q / heads_k query heads that read the same key head: row r of a
// sequence is position r / G, head r % G of the group.  The heads of a group
// so share each staged key tile, and the gradient of a shared head is a plain
// sum over rows.
//
// The lengths are device data, which the host cannot check.  They are read
// through clamps: whatever they hold, every index made from them lies inside
// the tensors.
#pragma once

#include "na2d_common.cuh"
#include "na2d_internal.h"

namespace na2d {
namespace packed {

struct Span {
  int q0, nq, k0, nk;  // first row and row count, first key and key count
};

NA_DEVICE int clamped(const int* cu, int s, int total) { return min(max(__ldg(cu + s), 0), total); }

NA_DEVICE Span span_of(const PackedArgs& p, int s) {
  Span r;
  r.q0 = clamped(p.cu_q, s, p.total_q);
  r.nq = max(clamped(p.cu_q, s + 1, p.total_q) - r.q0, 0);
  r.k0 = clamped(p.cu_k, s, p.total_k);
  r.nk = max(clamped(p.cu_k, s + 1, p.total_k) - r.k0, 0);
  if (p.len_k) r.nk = min(r.nk, max(__ldg(p.len_k + s), 0));
  return r;
}

// Keys [lo, hi) of a sequence with nq rows and nk keys that its row i sees.
NA_DEVICE void visible(const PackedArgs& p, const Span& s, int i, int* lo, int* hi) {
  *lo = 0;
  *hi = s.nk;
  if (p.causal) {
    const int at = i + (s.nk - s.nq);  // the row's position among the keys
    *hi = min(max(at + 1, 0), s.nk);
    if (p.window > 0 && at >= p.window) *lo = at - p.window + 1;
    *lo = min(*lo, *hi);
  }
}

// Rows [lo, hi) of the sequence that see its key j: the inverse of visible().
NA_DEVICE void seen_by(const PackedArgs& p, const Span& s, int j, int* lo, int* hi) {
  *lo = 0;
  *hi = s.nq;
  if (p.causal) {
    const int first = j - (s.nk - s.nq);  // the row at the key's position
    *lo = min(max(first, 0), s.nq);
    if (p.window > 0) *hi = (int)min((long long)s.nq, max((long long)first + p.window, 0ll));
    *hi = max(*hi, *lo);
  }
}

// Parts of `per` consecutive units of the sequences' entries, `mul` units an
// entry, are numbered without counting them: sequence s owns the numbers from
// cu[s] mul / per + s on, which are enough for its ceil(n mul / per) parts, as
// floor((a + n) / per) - floor(a / per) + 1 >= ceil(n / per).  That makes
// total mul / per + nseq numbers; those past a sequence's last part stay
// without work (idx past the last part, or negative).
__host__ __device__ __forceinline__ long long part_numbers(int nseq, long long total, int mul, int per) {
  return total * mul / per + nseq;
}
NA_DEVICE long long first_number(const int* cu, int s, int total, int mul, int per) {
  return (long long)clamped(cu, s, total) * mul / per + s;
}
NA_DEVICE void find_part(const int* cu, int nseq, int total, int mul, int per, long long number, int* s,
                         long long* idx) {
  int a = 0, b = nseq - 1;  // the last s whose first number is <= number
  while (a < b) {
    const int m = (a + b + 1) >> 1;
    if (first_number(cu, m, total, mul, per) <= number)
      a = m;
    else
      b = m - 1;
  }
  *s = a;
  *idx = number - first_number(cu, a, total, mul, per);
}

}  // namespace packed
}  // namespace na2d
