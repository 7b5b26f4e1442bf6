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

// Rows of the `per` positions from `pos` on that are a sequence's of nq positions,
// and where position `at` stands among them.  Positions are cut to the tile
// before they are multiplied: a sequence's rows may be more than 2^31.
__host__ __device__ __forceinline__ int rows_of_tile(int nq, int pos, int per, int group) {
  return (nq - pos < per ? nq - pos : per) * group;
}
__host__ __device__ __forceinline__ int row_in_tile(int at, int pos, int per, int group) {
  return (at < pos ? 0 : at - pos < per ? at - pos : per) * group;
}

// Keys of a piece of a sequence whose keys are cut: fixed, or its share when
// every sequence is cut into the same number of pieces.
NA_DEVICE int piece_length(const PackedArgs& p, const Span& s) {
  if (p.piece_keys > 0) return p.piece_keys;
  return max((s.nk + p.max_pieces * 128 - 1) / (p.max_pieces * 128), 1) * 128;
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

// find_part by a whole warp: 32 probes at once, so that one round of loads
// finds the sequence among 32 and two among 1024.
NA_DEVICE void find_part_warp(const int* cu, int nseq, int total, int mul, int per, long long number, int* s,
                              long long* idx) {
  const int lane = threadIdx.x & 31;
  int a = 0, n = nseq;  // the answer is one of a .. a + n - 1
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = a + lane * step;
    const bool below = lane * step < n && first_number(cu, at, total, mul, per) <= number;
    const unsigned votes = __ballot_sync(0xffffffffu, below) | 1u;
    const int last = 31 - __clz(votes);
    const int end = a + n;
    a += last * step;
    n = min(step, end - a);
  }
  *s = a;
  *idx = number - first_number(cu, a, total, mul, per);
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// What brings an fp16 gradient row of squared norm n2 to a norm of 16 to 32, a
// power of two.  Rows of zeros and such as are not finite, for which any will do,
// get the largest there is, that of one entry of 2^-24.
constexpr float kMostLift = 268435456.f;  // 2^28
NA_DEVICE float lift_of(float n2) {
  if (!(n2 > 0.f && n2 < INFINITY)) return kMostLift;
  const int e = (int)(__float_as_uint(n2) >> 23) - 127;  // 2^e <= n2 < 2^(e + 1)
  return __uint_as_float((uint32_t)(127 + 4 - (e >> 1)) << 23);
}

template <typename T> NA_DEVICE float to_f(T x);
template <> NA_DEVICE float to_f<float>(float x) { return x; }
template <> NA_DEVICE float to_f<__half>(__half x) { return __half2float(x); }
template <> NA_DEVICE float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> NA_DEVICE T from_f(float x);
template <> NA_DEVICE float from_f<float>(float x) { return x; }
template <> NA_DEVICE __half from_f<__half>(float x) { return __float2half_rn(x); }
template <> NA_DEVICE __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// two values rounded and packed, a in the low half
template <typename T> NA_DEVICE uint32_t pack2(float a, float b) {
  static_assert(sizeof(T) == 2);
  uint32_t r;
  if constexpr (__is_same(T, __half))
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

NA_DEVICE float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
NA_DEVICE float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// a . b of D elements
template <typename T, int D> NA_DEVICE float dot_row(const T* a, const T* b) {
  constexpr int VEC = 16 / sizeof(T);
  float s = 0.f;
  for (int i = 0; i < D; i += VEC) {
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(a + i)), y = __ldg(reinterpret_cast<const uint4*>(b + i));
    const T *u = reinterpret_cast<const T*>(&x), *v = reinterpret_cast<const T*>(&y);
#pragma unroll
    for (int e = 0; e < VEC; ++e) s = fmaf(to_f<T>(u[e]), to_f<T>(v[e]), s);
  }
  return s;
}

// One row over its keys [lo, hi) by a whole warp, from global memory: every
// key outside is left out of the sums, not multiplied by zero.  Matrix
// instructions cannot leave out single entries, so a row whose result is not
// finite is taken again by this.  acc holds the result's columns lane + 32 e,
// zeros with an lse of -inf for a row without weights: one that sees no key comes
// here too, when a value that its neighbours see is not finite.
template <typename T, int D>
NA_DEVICE void exact_row(const PackedArgs& p, const T* q, const T* k, const T* v, long long stride, int lo, int hi,
                         float (&acc)[(D + 31) / 32], float* lse) {
  const int lane = threadIdx.x & 31;
  const float sl2 = p.scale * kLog2e;
  float m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < (D + 31) / 32; ++e) acc[e] = 0.f;
  for (int j0 = lo; j0 < hi; j0 += 32) {
    const bool live = j0 + lane < hi;
    const float s = live ? dot_row<T, D>(q, k + (j0 + lane) * stride) * sl2 : -INFINITY;
    const float mx = fmaxf(m, warp_max(s));
    const float ref = mx == -INFINITY ? 0.f : mx;
    const float f = exp2f(m - ref);
    const float e = live ? exp2f(s - ref) : 0.f;
    l = fmaf(l, f, warp_sum(e));
    m = mx;
#pragma unroll
    for (int c = 0; c < (D + 31) / 32; ++c) acc[c] *= f;
    for (int t = 0; t < min(32, hi - j0); ++t) {
      const float w = __shfl_sync(0xffffffffu, e, t);
#pragma unroll
      for (int c = 0; c < (D + 31) / 32; ++c)
        if (lane + 32 * c < D) acc[c] = fmaf(w, to_f<T>(v[(j0 + t) * stride + lane + 32 * c]), acc[c]);
    }
  }
#pragma unroll
  for (int c = 0; c < (D + 31) / 32; ++c) acc[c] = l == 0.f ? 0.f : acc[c] / l;
  *lse = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace packed
}  // namespace na2d
