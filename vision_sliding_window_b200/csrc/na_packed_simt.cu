// na_packed_simt.cu -- attention over packed sequences on the CUDA cores, its
// gradients, and the join of partial results; for float32, and for the shapes
// that the tensor-core kernels do not take.
//
// Forward.  A block owns 32 rows (16 with single tokens) of one key head and
// walks the keys they see in tiles of 64 with a running maximum and sum.  S and
// the output stay in registers, each thread a 2 x 8 patch of S and 2 rows x d/8
// columns of the output, fed from float32 tiles in shared memory by 16-byte
// loads.  float32 tiles are copied asynchronously: the next keys come while the
// softmax and the second product run, the next values while S is made.  Shared
// memory's 128 bytes a clock bound it: 10 loads of 4 clocks for 64 FMAs.  Rows
// of 32 rather than 64, in 128 threads, leave more blocks to an SM: 700 + 33 +
// 512 + 257 rows of 8 heads, d = 64, window 200, take 39 us, against 54 in
// blocks of 64 rows and 256 threads.
//
// Backward.  P and dS are recomputed from the rows' log-sum-exp, once with a
// block owning 64 keys (dk, dv) and once with a block owning 64 rows (dq): two
// more products than one kernel that adds dq with atomics, but each gradient
// is one block's sum in a fixed order.  256 threads a block, as its shared
// memory leaves room for two an SM where d <= 64 and one where d = 128; the
// walk over a key tile's rows is cut where key tiles are few (3453 rows, 8 heads
// on 2, d = 64: 490 us, 870 uncut in 128 threads).
//
// A product never touches a masked entry: weights of masked places are
// skipped, not multiplied by zero, so that what they hold (NaN, infinities)
// cannot reach a result.
#include <type_traits>

#include "na2d_sm100.cuh"
#include "na_packed.cuh"

namespace na2d {
namespace {

using namespace packed;

constexpr int kKeys = 64;  // keys of a tile
constexpr int kLdW = kKeys + 4;  // floats a row of staged weights: read by 16-byte loads

// Brings 16 bytes of a row, as float32, into shared memory; zeros where not
// live.  float32 goes by itself (wait_copies), other types through registers.
template <typename T> NA_DEVICE void load_vec(const T* g, float* s, int v, bool live) {
  if constexpr (sizeof(T) == 4) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sm100::smem_addr(s + v * 4)), "l"(g + v * 4),
                 "r"(live ? 16 : 0)
                 : "memory");
  } else {
    constexpr int VEC = 16 / sizeof(T);
    float f[VEC];
    const uint4 u = live ? __ldg(reinterpret_cast<const uint4*>(g) + v) : make_uint4(0, 0, 0, 0);
    const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = to_f<T>(e[i]);
#pragma unroll
    for (int i = 0; i < VEC; i += 4)
      *reinterpret_cast<float4*>(s + v * VEC + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
  }
}
// A thread's copies since the last call are a group; wait_copies<N> leaves the
// N newest groups in flight.
NA_DEVICE void end_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> NA_DEVICE void wait_copies() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <int D> struct Tile {
  static constexpr int LD = D + 4;  // floats a staged row: 16-byte loads of 8 rows fall on distinct banks
  static constexpr int CPT = D / 8;  // output columns a thread
  static constexpr int CV = CPT >= 4 ? 4 : CPT;  // of which this many are consecutive
};

// Rows [r0, r0 + n) of one key head's rows of a sequence (position r / G, head
// r % G) from a tensor [total_q][hq][D].
template <typename T, int D, int ROWS, int THREADS>
NA_DEVICE void load_rows(const PackedArgs& p, const Span& sp, const T* g, int kh, long long r0, int n, float* s) {
  constexpr int VPR = D * sizeof(T) / 16;
#pragma unroll 4
  for (int e = threadIdx.x; e < ROWS * VPR; e += THREADS) {
    const int r = e / VPR, v = e % VPR;
    const bool live = r < n;
    const long long rr = live ? r0 + r : r0;
    const long long at = ((long long)sp.q0 + rr / p.group) * p.hq + kh * p.group + rr % p.group;
    load_vec<T>(g + at * D, s + r * Tile<D>::LD, v, live);
  }
}
template <typename T, int D, int THREADS>
NA_DEVICE void load_keys(const PackedArgs& p, const Span& sp, const T* g, int kh, int k0, int n, float* s) {
  constexpr int VPR = D * sizeof(T) / 16;
#pragma unroll 4
  for (int e = threadIdx.x; e < kKeys * VPR; e += THREADS) {
    const int j = e / VPR, v = e % VPR;
    const bool live = j < n;
    const long long at = ((long long)sp.k0 + (live ? k0 + j : k0)) * p.hk + kh;
    load_vec<T>(g + at * D, s + j * Tile<D>::LD, v, live);
  }
}

// c[r][j] = a row (ty R + r) . b row (tx + 8 j) of two staged tiles.  Even and
// odd columns are summed apart, two of them an instruction.
template <int D, int R>
NA_DEVICE void dot_patch(const float* a, const float* b, int ty, int tx, float (&c)[R][8]) {
  constexpr int LD = Tile<D>::LD;
  float even[R][8], odd[R][8];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int j = 0; j < 8; ++j) even[r][j] = odd[r][j] = 0.f;
#pragma unroll 2
  for (int d = 0; d < D; d += 4) {
    float4 x[R];
#pragma unroll
    for (int r = 0; r < R; ++r) x[r] = *reinterpret_cast<const float4*>(a + (ty * R + r) * LD + d);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float4 y = *reinterpret_cast<const float4*>(b + (tx + 8 * j) * LD + d);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        sm100::fma2(even[r][j], odd[r][j], x[r].x, x[r].y, y.x, y.y, even[r][j], odd[r][j]);
        sm100::fma2(even[r][j], odd[r][j], x[r].z, x[r].w, y.z, y.w, even[r][j], odd[r][j]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int j = 0; j < 8; ++j) c[r][j] = even[r][j] + odd[r][j];
}

// acc[r][.] += w[ty R + r][j] * b[j][this thread's columns] for j inside row
// r's [lo, hi), which lie in [0, kKeys).  A thread's rows are neighbours and
// their ranges all but alike, so the keys go by fours, and only fours that some
// row sees in part are asked key by key.
template <int D, int R>
NA_DEVICE void weighted_sum(const float* w, const float* b, int ty, int tx, const int (&lo)[R], const int (&hi)[R],
                            float (&acc)[R][Tile<D>::CPT]) {
  constexpr int LD = Tile<D>::LD, CPT = Tile<D>::CPT, CV = Tile<D>::CV;
  auto columns = [&](int j, float (&v)[CPT]) {
#pragma unroll
    for (int c = 0; c < CPT / CV; ++c) {
      const float* from = b + j * LD + c * 8 * CV + tx * CV;
      if constexpr (CV == 4) {
        const float4 f = *reinterpret_cast<const float4*>(from);
        v[4 * c] = f.x, v[4 * c + 1] = f.y, v[4 * c + 2] = f.z, v[4 * c + 3] = f.w;
      } else {
        const float2 f = *reinterpret_cast<const float2*>(from);
        v[0] = f.x, v[1] = f.y;
      }
    }
  };
  auto add = [&](int r, float x, const float (&v)[CPT]) {
#pragma unroll
    for (int c = 0; c < CPT; c += 2)
      sm100::fma2(acc[r][c], acc[r][c + 1], x, x, v[c], v[c + 1], acc[r][c], acc[r][c + 1]);
  };
  int first = kKeys, last = 0, all_lo = 0, all_hi = kKeys;  // seen by some row; seen by all
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (lo[r] < hi[r]) {
      first = min(first, lo[r]);
      last = max(last, hi[r]);
    }
    all_lo = max(all_lo, lo[r]);
    all_hi = min(all_hi, hi[r]);
  }
  for (int j = first & ~3; j < last; j += 4) {
    float4 x[R];
#pragma unroll
    for (int r = 0; r < R; ++r) x[r] = *reinterpret_cast<const float4*>(w + (ty * R + r) * kLdW + j);
    float v[CPT];
    if (j >= all_lo && j + 4 <= all_hi) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        columns(j + i, v);
#pragma unroll
        for (int r = 0; r < R; ++r) add(r, (&x[r].x)[i], v);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        columns(j + i, v);
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (j + i >= lo[r] && j + i < hi[r]) add(r, (&x[r].x)[i], v);
      }
    }
  }
}

// acc times f; zeros where f is 0, whatever acc holds
template <typename T, int D, int R>
NA_DEVICE void store_cols(T* g, int tx, const float (&acc)[Tile<D>::CPT], float f) {
  constexpr int CPT = Tile<D>::CPT, CV = Tile<D>::CV;
#pragma unroll
  for (int c = 0; c < CPT; ++c) g[(c / CV) * 8 * CV + tx * CV + c % CV] = from_f<T>(f == 0.f ? 0.f : acc[c] * f);
}

template <int D, int ROWS> constexpr int fwd_smem() {
  return (ROWS * Tile<D>::LD + 2 * kKeys * Tile<D>::LD + ROWS * kLdW) * (int)sizeof(float);
}

// ----------------------------------------------------------------- forward
template <typename T, int D, int R, int THREADS>
__global__ void __launch_bounds__(THREADS) packed_forward_simt_kernel(PackedArgs p) {
  constexpr int ROWS = THREADS / 8 * R, LD = Tile<D>::LD, CPT = Tile<D>::CPT;
  extern __shared__ __align__(16) float sm[];
  float* Qs = sm;
  float* Ks = Qs + ROWS * LD;
  float* Vs = Ks + kKeys * LD;
  float* Ps = Vs + kKeys * LD;
  const int ty = threadIdx.x / 8, tx = threadIdx.x % 8;
  const int kh = blockIdx.y;
  const float sl2 = p.scale * kLog2e;
  int s;
  long long idx;
  // keys in pieces of one length, or a share of every sequence's a plane
  const bool split = p.max_pieces > 1, by_keys = p.piece_keys > 0;
  if (by_keys)
    find_part(p.cu_k, p.nseq, p.total_k, 1, p.piece_keys, blockIdx.x, &s, &idx);
  else
    find_part(p.cu_q, p.nseq, p.total_q, p.group, ROWS, blockIdx.x, &s, &idx);
  if (idx < 0) return;
  const Span sp = span_of(p, s);
  const long long all_rows = (long long)sp.nq * p.group;
  int piece0 = 0, piece1 = sp.nk;
  long long t0 = idx, t1 = idx + 1;
  int piece = 0;
  if (split) {
    const int len = piece_length(p, sp);
    if (by_keys && (idx >= p.max_pieces || idx * len >= sp.nk)) return;
    piece = by_keys ? (int)idx : (int)blockIdx.z;
    piece0 = (int)min((long long)piece * len, (long long)sp.nk);
    piece1 = min(piece0 + len, sp.nk);
  }
  if (by_keys) {
    t0 = 0;
    t1 = (all_rows + ROWS - 1) / ROWS;
  }
  for (long long t = t0; t < t1; ++t) {
    const long long r0 = t * ROWS;
    if (r0 >= all_rows) return;
    const int n = (int)min((long long)ROWS, all_rows - r0);
    int lo[R], hi[R], kb, ke, unused;
    visible(p, sp, (int)(r0 / p.group), &kb, &unused);
    visible(p, sp, (int)((r0 + n - 1) / p.group), &unused, &ke);
    kb = max(kb, piece0);
    ke = min(ke, piece1);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int row = ty * R + r;
      visible(p, sp, (int)((r0 + min(row, n - 1)) / p.group), &lo[r], &hi[r]);
      if (row >= n) hi[r] = lo[r];
    }
    __syncthreads();
    load_rows<T, D, ROWS, THREADS>(p, sp, (const T*)p.q, kh, r0, n, Qs);
    auto ask = [&](const void* g, int k0, float* to) {
      if (k0 < ke) load_keys<T, D, THREADS>(p, sp, (const T*)g, kh, k0, min(kKeys, ke - k0), to);
      end_copies();
    };
    ask(p.k, kb, Ks);
    ask(p.v, kb, Vs);
    float m[R], l[R], acc[R][CPT];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int c = 0; c < CPT; ++c) acc[r][c] = 0.f;
    }
    for (int k0 = kb; k0 < ke; k0 += kKeys) {
      const int nk = min(kKeys, ke - k0);
      wait_copies<1>();  // K is here, V may be on its way
      __syncthreads();
      float sc[R][8];
      dot_patch<D, R>(Qs, Ks, ty, tx, sc);
      __syncthreads();
      ask(p.k, k0 + kKeys, Ks);
      int tlo[R], thi[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        tlo[r] = max(lo[r] - k0, 0);
        thi[r] = min(hi[r] - k0, nk);
        float mx = m[r];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int key = tx + 8 * j;
          if (!(key >= tlo[r] && key < thi[r])) sc[r][j] = -INFINITY;
          mx = fmaxf(mx, sc[r][j]);
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float ref = mx == -INFINITY ? 0.f : mx * sl2;
        const float f = exp2f(fmaf(m[r], sl2, -ref));
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float e = exp2f(fmaf(sc[r][j], sl2, -ref));
          sum += e;
          Ps[(ty * R + r) * kLdW + tx + 8 * j] = e;
        }
        l[r] = fmaf(l[r], f, sum);
        m[r] = mx;
#pragma unroll
        for (int c = 0; c < CPT; ++c) acc[r][c] *= f;
      }
      wait_copies<1>();
      __syncthreads();
      weighted_sum<D, R>(Ps, Vs, ty, tx, tlo, thi, acc);
      __syncthreads();
      ask(p.v, k0 + kKeys, Vs);
    }
    wait_copies<0>();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float sum = l[r];
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const int row = ty * R + r;
      if (row >= n) continue;
      const long long rr = r0 + row;
      const long long i = (long long)sp.q0 + rr / p.group;
      const int head = kh * p.group + (int)(rr % p.group);
      // a row that saw no key: zeros and -inf
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const float lse = sum == 0.f ? -INFINITY : fmaf(m[r], p.scale, log2f(sum) * kLn2);
      if (split) {
        const long long at = ((long long)piece * p.total_q + i) * p.hq + head;
        store_cols<float, D, R>(p.part_o + at * D, tx, acc[r], inv);
        if (tx == 0) p.part_lse[at] = lse;
      } else {
        store_cols<T, D, R>((T*)p.out + (i * p.hq + head) * D, tx, acc[r], inv);
        if (tx == 0 && p.lse) p.lse[(long long)head * p.total_q + i] = lse;
      }
    }
  }
}

// Joins the pieces of every row: out = sum_c e^(lse_c - lse) o_c.  One warp a
// row; rows behind the last sequence belong to none and are left alone.
template <typename T>
__global__ void __launch_bounds__(256) packed_join_kernel(PackedArgs p) {
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= (long long)p.total_q * p.hq) return;
  const int i = (int)(row / p.hq), head = (int)(row % p.hq);
  int a = 0, b = p.nseq - 1;  // the last sequence that starts at or before i
  while (a < b) {
    const int mid = (a + b + 1) >> 1;
    if (clamped(p.cu_q, mid, p.total_q) <= i)
      a = mid;
    else
      b = mid - 1;
  }
  const Span sp = span_of(p, a);
  if (i < sp.q0 || i >= sp.q0 + sp.nq) return;
  int lo, hi;
  visible(p, sp, i - sp.q0, &lo, &hi);
  const int len = piece_length(p, sp);
  const int c0 = lo / len, c1 = lo < hi ? min((hi - 1) / len + 1, p.max_pieces) : c0;
  const long long step = (long long)p.total_q * p.hq;
  float mx = -INFINITY;
  for (int c = c0 + lane; c < c1; c += 32) mx = fmaxf(mx, p.part_lse[c * step + row]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float ref = mx == -INFINITY ? 0.f : mx;
  float acc[4] = {0.f, 0.f, 0.f, 0.f}, sum = 0.f;
  for (int c = c0; c < c1; ++c) {
    const float lse = p.part_lse[c * step + row], w = expf(lse - ref);
    sum += w;
    if (lse == -INFINITY) continue;  // a piece of which the row saw nothing
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (lane + 32 * e < p.d) acc[e] = fmaf(w, p.part_o[(c * step + row) * p.d + lane + 32 * e], acc[e]);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (lane + 32 * e < p.d) ((T*)p.out)[row * p.d + lane + 32 * e] = from_f<T>(acc[e] * inv);
  if (lane == 0 && p.lse) p.lse[(long long)head * p.total_q + i] = sum == 0.f ? -INFINITY : ref + logf(sum);
}

// ---------------------------------------------------------------- backward
// Every row's log-sum-exp in units of log2 and delta = out . dout, and where
// asked for its lift.
template <typename T, int D> __global__ void __launch_bounds__(256) packed_terms_kernel(PackedArgs p) {
  constexpr int VEC = 16 / sizeof(T), LPR = D / VEC;  // lanes a row
  const long long row = ((long long)blockIdx.x * 256 + threadIdx.x) / LPR;
  const int v = threadIdx.x % LPR;
  const bool live = row < (long long)p.total_q * p.hq;
  float s = 0.f, n2 = 0.f;
  if (live) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p.o) + row * LPR + v);
    const uint4 b = __ldg(reinterpret_cast<const uint4*>(p.dout) + row * LPR + v);
    const T *x = reinterpret_cast<const T*>(&a), *y = reinterpret_cast<const T*>(&b);
#pragma unroll
    for (int i = 0; i < VEC; ++i) s = fmaf(to_f<T>(x[i]), to_f<T>(y[i]), s);
    if (p.row_lifts)
#pragma unroll
      for (int i = 0; i < VEC; ++i) n2 = fmaf(to_f<T>(y[i]), to_f<T>(y[i]), n2);
  }
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (p.row_lifts) {
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) n2 += __shfl_xor_sync(0xffffffffu, n2, o);
    if (live && v == 0) p.row_lifts[row] = lift_of(n2);
  }
  if (live && v == 0) {
    const float lse = p.lse_in[row % p.hq * p.total_q + row / p.hq];
    // a row that sees no key has no weights, whatever its gradient holds
    p.terms[row] = lse == -INFINITY ? make_float2(INFINITY, 0.f) : make_float2(lse * kLog2e, s);
  }
}

// The lift of a sequence's rows of one key head: that of its largest row.  A
// thread keeps to one head of the group (there are 128 at most here), so that
// nothing is divided between the loads, which are what this waits for.
constexpr int kLiftThreads = 512;
__global__ void __launch_bounds__(kLiftThreads) packed_lifts_kernel(PackedArgs p) {
  __shared__ float least[kLiftThreads / 32];
  const int per = kLiftThreads / p.group, at = threadIdx.x / p.group, g = threadIdx.x % p.group;
  for (long long u = blockIdx.x; u < (long long)p.nseq * p.hk; u += gridDim.x) {
    const Span sp = span_of(p, (int)(u / p.hk));
    const int kh = (int)(u % p.hk);
    float f = kMostLift;
    const float* from = p.row_lifts + (long long)sp.q0 * p.hq + kh * p.group + g;
    if (at < per)
#pragma unroll 8
      for (int i = at; i < sp.nq; i += per) f = fminf(f, from[(long long)i * p.hq]);
    f = -warp_max(-f);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) least[threadIdx.x >> 5] = f;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
      for (int w = 1; w < kLiftThreads / 32; ++w) f = fminf(f, least[w]);
      p.lifts[u] = f;
    }
  }
}

template <int D> constexpr int bwd_smem() {
  return (4 * kKeys * Tile<D>::LD + 2 * kKeys * kLdW + 2 * kKeys) * (int)sizeof(float);
}

// lse (in units of log2) and delta of the staged rows
NA_DEVICE void load_row_terms(const PackedArgs& p, const Span& sp, int kh, long long r0, int n, float* lse,
                              float* delta) {
  if (threadIdx.x < kKeys) {
    const int r = threadIdx.x;
    const long long rr = r0 + (r < n ? r : 0);
    const long long i = (long long)sp.q0 + rr / p.group;
    const int head = kh * p.group + (int)(rr % p.group);
    const float2 t = p.terms[i * p.hq + head];
    lse[r] = t.x;
    delta[r] = t.y;
  }
}

constexpr int kBwdThreads = 256;

template <typename T, int D>
__global__ void __launch_bounds__(kBwdThreads, D == 128 ? 1 : 2) packed_dkdv_simt_kernel(PackedArgs p) {
  constexpr int R = 2, LD = Tile<D>::LD, CPT = Tile<D>::CPT;
  extern __shared__ __align__(16) float sm[];
  float* Ks = sm;
  float* Vs = Ks + kKeys * LD;
  float* Qs = Vs + kKeys * LD;
  float* Os = Qs + kKeys * LD;
  float* Ps = Os + kKeys * LD;
  float* Ss = Ps + kKeys * kLdW;
  float* lse = Ss + kKeys * kLdW;
  float* delta = lse + kKeys;
  const int ty = threadIdx.x / 8, tx = threadIdx.x % 8;
  const int kh = blockIdx.y;
  const float sl2 = p.scale * kLog2e;
  int s;
  long long idx;
  find_part(p.cu_k, p.nseq, p.total_k, 1, kKeys, blockIdx.x, &s, &idx);
  if (idx < 0) return;
  const Span sp = span_of(p, s);
  if (idx * kKeys >= sp.nk) return;
  const int j0 = (int)idx * kKeys, nk = min(kKeys, sp.nk - j0);
  load_keys<T, D, kBwdThreads>(p, sp, (const T*)p.k, kh, j0, nk, Ks);
  load_keys<T, D, kBwdThreads>(p, sp, (const T*)p.v, kh, j0, nk, Vs);
  long long lo[R], hi[R];  // rows that see this thread's keys
  int a, b;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int j = ty * R + r;
    seen_by(p, sp, j0 + min(j, nk - 1), &a, &b);
    lo[r] = (long long)a * p.group;
    hi[r] = j < nk ? (long long)b * p.group : lo[r];
  }
  float dk[R][CPT], dv[R][CPT];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < CPT; ++c) dk[r][c] = dv[r][c] = 0.f;
  int unused, first, last;
  seen_by(p, sp, j0, &first, &unused);
  seen_by(p, sp, j0 + nk - 1, &unused, &last);
  // this block's piece of the rows that see its keys
  const long long begin = (long long)first * p.group, tiles = ((long long)last * p.group - begin + kKeys - 1) / kKeys;
  const long long per = (tiles + gridDim.z - 1) / gridDim.z * kKeys;
  const long long from = begin + blockIdx.z * per, to = min(from + per, (long long)last * p.group);
  for (long long r0 = from; r0 < to; r0 += kKeys) {
    const int n = (int)min((long long)kKeys, to - r0);
    __syncthreads();
    load_rows<T, D, kKeys, kBwdThreads>(p, sp, (const T*)p.q, kh, r0, n, Qs);
    load_rows<T, D, kKeys, kBwdThreads>(p, sp, (const T*)p.dout, kh, r0, n, Os);
    end_copies();
    load_row_terms(p, sp, kh, r0, n, lse, delta);
    wait_copies<0>();
    __syncthreads();
    float sc[R][8], dp[R][8];
    dot_patch<D, R>(Ks, Qs, ty, tx, sc);
    dot_patch<D, R>(Vs, Os, ty, tx, dp);
    int tlo[R], thi[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      tlo[r] = (int)max(lo[r] - r0, 0ll);
      thi[r] = (int)min(max(hi[r] - r0, 0ll), (long long)n);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int row = tx + 8 * j;
        const float e = exp2f(fmaf(sc[r][j], sl2, -lse[row]));
        Ps[(ty * R + r) * kLdW + row] = e;
        Ss[(ty * R + r) * kLdW + row] = e * (dp[r][j] - delta[row]);
      }
    }
    __syncwarp();
    weighted_sum<D, R>(Ps, Os, ty, tx, tlo, thi, dv);
    weighted_sum<D, R>(Ss, Qs, ty, tx, tlo, thi, dk);
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int j = ty * R + r;
    if (j >= nk) continue;
    const long long at = ((long long)(sp.k0 + j0 + j) * p.hk + kh) * D;
    if (gridDim.z > 1) {
      const long long all = (long long)p.total_k * p.hk * D;
      float* part = p.part_o + blockIdx.z * 2 * all + at;
      store_cols<float, D, R>(part, tx, dv[r], 1.f);
      store_cols<float, D, R>(part + all, tx, dk[r], p.scale);
    } else {
      store_cols<T, D, R>((T*)p.dk + at, tx, dk[r], p.scale);
      store_cols<T, D, R>((T*)p.dv + at, tx, dv[r], 1.f);
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kBwdThreads, D == 128 ? 1 : 2) packed_dq_simt_kernel(PackedArgs p) {
  constexpr int R = 2, LD = Tile<D>::LD, CPT = Tile<D>::CPT, ROWS = 64;
  extern __shared__ __align__(16) float sm[];
  float* Ks = sm;
  float* Vs = Ks + kKeys * LD;
  float* Qs = Vs + kKeys * LD;
  float* Os = Qs + kKeys * LD;
  float* Ss = Os + kKeys * LD;
  float* lse = Ss + 2 * kKeys * kLdW;
  float* delta = lse + kKeys;
  const int ty = threadIdx.x / 8, tx = threadIdx.x % 8;
  const int kh = blockIdx.y;
  const float sl2 = p.scale * kLog2e;
  int s;
  long long idx;
  find_part(p.cu_q, p.nseq, p.total_q, p.group, ROWS, blockIdx.x, &s, &idx);
  if (idx < 0) return;
  const Span sp = span_of(p, s);
  const long long all_rows = (long long)sp.nq * p.group, r0 = idx * ROWS;
  if (r0 >= all_rows) return;
  const int n = (int)min((long long)ROWS, all_rows - r0);
  load_rows<T, D, ROWS, kBwdThreads>(p, sp, (const T*)p.q, kh, r0, n, Qs);
  load_rows<T, D, ROWS, kBwdThreads>(p, sp, (const T*)p.dout, kh, r0, n, Os);
  load_row_terms(p, sp, kh, r0, n, lse, delta);
  int lo[R], hi[R], kb, ke, unused;
  visible(p, sp, (int)(r0 / p.group), &kb, &unused);
  visible(p, sp, (int)((r0 + n - 1) / p.group), &unused, &ke);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = ty * R + r;
    visible(p, sp, (int)((r0 + min(row, n - 1)) / p.group), &lo[r], &hi[r]);
    if (row >= n) hi[r] = lo[r];
  }
  float dq[R][CPT];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < CPT; ++c) dq[r][c] = 0.f;
  for (int k0 = kb; k0 < ke; k0 += kKeys) {
    const int nk = min(kKeys, ke - k0);
    __syncthreads();
    load_keys<T, D, kBwdThreads>(p, sp, (const T*)p.k, kh, k0, nk, Ks);
    load_keys<T, D, kBwdThreads>(p, sp, (const T*)p.v, kh, k0, nk, Vs);
    end_copies();
    wait_copies<0>();
    __syncthreads();
    float sc[R][8], dp[R][8];
    dot_patch<D, R>(Qs, Ks, ty, tx, sc);
    dot_patch<D, R>(Os, Vs, ty, tx, dp);
    int tlo[R], thi[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      tlo[r] = max(lo[r] - k0, 0);
      thi[r] = min(hi[r] - k0, nk);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        Ss[(ty * R + r) * kLdW + tx + 8 * j] =
            exp2f(fmaf(sc[r][j], sl2, -lse[ty * R + r])) * (dp[r][j] - delta[ty * R + r]);
    }
    __syncwarp();
    weighted_sum<D, R>(Ss, Ks, ty, tx, tlo, thi, dq);
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = ty * R + r;
    if (row >= n) continue;
    const long long rr = r0 + row;
    const long long at = ((long long)sp.q0 + rr / p.group) * p.hq + kh * p.group + rr % p.group;
    store_cols<T, D, R>((T*)p.dq + at * D, tx, dq[r], p.scale);
  }
}

// ---------------------------------------------------------------- launches
template <typename K> cudaError_t with_smem(K kern, int bytes) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

bool few_rows(const PackedArgs& p) { return (long long)p.total_q * p.group <= 16ll * p.nseq; }

template <typename T, int D, int R, int THREADS> cudaError_t forward_r(const PackedArgs& p, cudaStream_t st) {
  constexpr int ROWS = THREADS / 8 * R;
  const long long blocks = p.piece_keys > 0 ? part_numbers(p.nseq, p.total_k, 1, p.piece_keys)
                                            : part_numbers(p.nseq, p.total_q, p.group, ROWS);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  auto kern = packed_forward_simt_kernel<T, D, R, THREADS>;
  cudaError_t e = with_smem(kern, fwd_smem<D, ROWS>());
  if (e != cudaSuccess) return e;
  const unsigned planes = p.piece_keys > 0 ? 1u : (unsigned)p.max_pieces;
  kern<<<dim3((unsigned)blocks, (unsigned)p.hk, planes), THREADS, fwd_smem<D, ROWS>(), st>>>(p);
  return cudaGetLastError();
}
template <typename T, int D> cudaError_t forward_d(const PackedArgs& p, cudaStream_t st) {
  return few_rows(p) ? forward_r<T, D, 1, 128>(p, st) : forward_r<T, D, 2, 128>(p, st);
}
template <typename T> cudaError_t forward_t(const PackedArgs& p, cudaStream_t st) {
  switch (p.d) {
    case 16: return forward_d<T, 16>(p, st);
    case 32: return forward_d<T, 32>(p, st);
    case 64: return forward_d<T, 64>(p, st);
    case 128: return forward_d<T, 128>(p, st);
  }
  return cudaErrorInvalidValue;
}
template <typename T> constexpr na_dtype dt_of() {
  return sizeof(T) == 4 ? NA_F32 : std::is_same_v<T, __half> ? NA_F16 : NA_BF16;
}
template <typename T, int D> cudaError_t backward_d(const PackedArgs& p, cudaStream_t st) {
  const long long kb = part_numbers(p.nseq, p.total_k, 1, kKeys), qb = part_numbers(p.nseq, p.total_q, p.group, 64);
  if (kb > 0x7fffffffLL || qb > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaError_t e = with_smem(packed_dkdv_simt_kernel<T, D>, bwd_smem<D>());
  if (e == cudaSuccess) e = with_smem(packed_dq_simt_kernel<T, D>, bwd_smem<D>());
  if (e != cudaSuccess) return e;
  packed_dkdv_simt_kernel<T, D><<<dim3((unsigned)kb, (unsigned)p.hk, (unsigned)p.max_pieces), kBwdThreads, bwd_smem<D>(), st>>>(p);
  packed_dq_simt_kernel<T, D><<<dim3((unsigned)qb, (unsigned)p.hk), kBwdThreads, bwd_smem<D>(), st>>>(p);
  cudaError_t launched = cudaGetLastError();
  if (launched == cudaSuccess && p.max_pieces > 1) launched = launch_packed_dkdv_join(p, dt_of<T>(), st);
  return launched;
}
template <typename T> cudaError_t backward_t(const PackedArgs& p, cudaStream_t st) {
  switch (p.d) {
    case 16: return backward_d<T, 16>(p, st);
    case 32: return backward_d<T, 32>(p, st);
    case 64: return backward_d<T, 64>(p, st);
    case 128: return backward_d<T, 128>(p, st);
  }
  return cudaErrorInvalidValue;
}
template <typename T, int D> cudaError_t terms_d(const PackedArgs& p, cudaStream_t st) {
  constexpr int kRows = 256 * 16 / ((int)sizeof(T) * D);
  const long long rows = (long long)p.total_q * p.hq, blocks = (rows + kRows - 1) / kRows;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  packed_terms_kernel<T, D><<<(unsigned)blocks, 256, 0, st>>>(p);
  return cudaGetLastError();
}
template <typename T> cudaError_t terms_t(const PackedArgs& p, cudaStream_t st) {
  switch (p.d) {
    case 16: return terms_d<T, 16>(p, st);
    case 32: return terms_d<T, 32>(p, st);
    case 64: return terms_d<T, 64>(p, st);
    case 128: return terms_d<T, 128>(p, st);
  }
  return cudaErrorInvalidValue;
}

template <typename T> cudaError_t join_t(const PackedArgs& p, cudaStream_t st) {
  const long long blocks = ((long long)p.total_q * p.hq + 7) / 8;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  packed_join_kernel<T><<<(unsigned)blocks, 256, 0, st>>>(p);
  return cudaGetLastError();
}

// One call of a template for each element type.
template <typename F> cudaError_t by_type(na_dtype dt, F f) {
  if (dt == NA_F32) return f(float{});
  if (dt == NA_F16) return f(__half{});
  return f(__nv_bfloat16{});
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

// Which kernel runs a forward call, and how it cuts the keys, from sizes and
// type alone.
//
// Few rows a sequence (16 on average: single tokens of up to 16 heads a group)
// run the kernel for few rows; float32, groups wider than a row tile and calls
// without keys run on the CUDA cores; the rest on the tensor cores.
//
// A cut of the keys pays where the rows alone leave SMs idle.  The kernel for
// few rows shares a sequence's keys among 8 blocks by itself and cuts only
// where sequences times heads are fewer than 19, which leaves SMs without a
// block, and sequences are longer than 4096 keys on average, of which a block's
// share takes longer than a second launch.  It and the CUDA-core kernel for few
// rows cut every sequence into pieces of one length, as long as leaves about
// `want` blocks but not under 256 keys (each piece's rows pay for writing and
// joining a float32 output), so that long sequences make more pieces than short
// ones.  The kernels for many rows cut every sequence into the same number of
// pieces of 512 keys at least, as their grids count row tiles.
void packed_plan(PackedArgs* p, na_dtype dt) {
  constexpr long long kSms = 148, kMost = 256ll << 20;
  p->piece_keys = 0;
  p->max_pieces = 1;
  const bool few = (long long)p->total_q * p->group <= 16ll * p->nseq;
  p->path = dt == NA_F32 || p->group > 128 || p->total_k == 0 ? kPathSimt : few ? kPathRows : kPathTc;
  const long long row_bytes = (long long)p->total_q * p->hq * (p->d + 1) * 4;
  if (p->path == kPathTc || !few) {
    const bool tc = p->path == kPathTc;
    const long long tiles = p->hk * (tc ? part_numbers(p->nseq, p->total_q, 1, packed_row_tiles(p->d) * (128 / p->group))
                                        : part_numbers(p->nseq, p->total_q, p->group, 32));
    long long pieces = (tc ? kSms : 2 * kSms) / tiles;
    if (pieces > p->total_k / p->nseq / 512) pieces = p->total_k / p->nseq / 512;
    while (pieces > 1 && pieces * row_bytes > kMost) --pieces;
    if (pieces > 1) p->max_pieces = (int)pieces;
    return;
  }
  if (p->path == kPathRows && ((long long)p->nseq * p->hk * 8 >= kSms || p->total_k / p->nseq <= 4096)) return;
  const long long want = (p->path == kPathRows ? 4 : 8) * kSms, least = 256;
  const long long per_seq = ((long long)p->total_q * p->group / p->nseq + 16) / 16;  // row tiles, about
  if (per_seq * p->nseq * p->hk >= 4 * kSms) return;
  long long keys = (long long)p->total_k * p->hk * per_seq / want;
  if (keys < least) keys = least;
  keys = (keys + 127) / 128 * 128;
  while (keys < p->total_k && (p->total_k + keys - 1) / keys * row_bytes > kMost) keys *= 2;
  if (p->total_k == 0 || keys >= p->total_k / p->nseq) return;  // a sequence of average length makes one
  p->piece_keys = (int)keys;
  p->max_pieces = (int)((p->total_k + keys - 1) / keys);
}

size_t packed_workspace_bytes(const PackedArgs& p, na_dtype dt) {
  PackedArgs c = p;
  packed_plan(&c, dt);
  if (c.max_pieces < 2) return 0;
  const size_t rows = (size_t)c.max_pieces * c.total_q * c.hq;
  return up256(rows * c.d * 4) + up256(rows * 4);
}

// The backward's kernels, chosen as the forward's.  The key tiles' walks over
// rows are cut into pieces, whose sums are added afterwards, where the key
// tiles alone are fewer than about 5 blocks for 2 SMs: causal walks have
// unequal lengths and the longest would run alone.
void packed_backward_plan(PackedArgs* p, na_dtype dt) {
  constexpr long long kSms = 148, kMost = 512ll << 20;
  p->piece_keys = 0;
  p->max_pieces = 1;
  const bool tc = !(dt == NA_F32 || p->group > 128 || p->total_k == 0 || p->total_q == 0);
  p->path = tc ? kPathTc : kPathSimt;
  if (p->total_k == 0 || p->total_q == 0) return;
  const long long tiles = part_numbers(p->nseq, p->total_k, 1, tc ? 128 : kKeys) * p->hk;
  // row tiles of a key tile, about
  const long long walk = tc ? (long long)p->total_q / p->nseq / (128 / p->group)
                            : (long long)p->total_q * p->group / p->nseq / 64;
  long long pieces = (5 * kSms / 2 + tiles - 1) / tiles;
  if (pieces > walk / (tc ? 8 : 4)) pieces = walk / (tc ? 8 : 4);
  if (pieces > 8) pieces = 8;
  while (pieces > 1 && pieces * p->total_k * p->hk * p->d * 8 > kMost) --pieces;
  if (pieces > 1) p->max_pieces = (int)pieces;
}

// Where the parts of the backward's workspace lie, and its size.
struct BackwardParts {
  size_t sums, row_lifts, lifts, size;
};
static BackwardParts backward_parts(const PackedArgs& p, na_dtype dt) {  // p as planned
  BackwardParts w;
  const bool lifted = p.path == kPathTc && dt == NA_F16;
  w.sums = up256((size_t)p.total_q * p.hq * 8);
  w.row_lifts = w.sums + (p.max_pieces > 1 ? up256((size_t)p.max_pieces * p.total_k * p.hk * p.d * 8) : 0);
  w.lifts = w.row_lifts + (lifted ? up256((size_t)p.total_q * p.hq * 4) : 0);
  w.size = w.lifts + (lifted ? up256((size_t)p.nseq * p.hk * 4) : 0);
  return w;
}
size_t packed_backward_workspace_bytes(const PackedArgs& p, na_dtype dt) {
  PackedArgs c = p;
  packed_backward_plan(&c, dt);
  return backward_parts(c, dt).size;
}

cudaError_t launch_packed_forward(PackedArgs p, void* workspace, na_dtype dt, cudaStream_t st) {
  packed_plan(&p, dt);
  if (p.max_pieces > 1) {
    p.part_o = (float*)workspace;
    p.part_lse = (float*)((char*)workspace + up256((size_t)p.max_pieces * p.total_q * p.hq * p.d * 4));
  }
  cudaError_t e = p.path == kPathTc     ? launch_packed_forward_tc(p, dt, st)
                  : p.path == kPathRows ? launch_packed_forward_rows(p, dt, st)
                                        : by_type(dt, [&](auto t) { return forward_t<decltype(t)>(p, st); });
  if (e == cudaSuccess && p.max_pieces > 1) e = by_type(dt, [&](auto t) { return join_t<decltype(t)>(p, st); });
  return e;
}

cudaError_t launch_packed_backward(PackedArgs p, void* workspace, na_dtype dt, cudaStream_t st) {
  packed_backward_plan(&p, dt);
  const BackwardParts w = backward_parts(p, dt);
  p.terms = (float2*)workspace;
  p.part_o = (float*)((char*)workspace + w.sums);
  const bool lifted = p.path == kPathTc && dt == NA_F16;
  if (lifted) {
    p.row_lifts = (float*)((char*)workspace + w.row_lifts);
    p.lifts = (float*)((char*)workspace + w.lifts);
  }
  if (p.total_q > 0) {
    cudaError_t e = by_type(dt, [&](auto t) { return terms_t<decltype(t)>(p, st); });
    if (e != cudaSuccess) return e;
  }
  if (lifted) {
    const long long blocks = (long long)p.nseq * p.hk, most = 148 * 8;
    packed_lifts_kernel<<<(unsigned)(blocks < most ? blocks : most), kLiftThreads, 0, st>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (p.path == kPathTc) return launch_packed_backward_tc(p, dt, st);
  return by_type(dt, [&](auto t) { return backward_t<decltype(t)>(p, st); });
}

}  // namespace na2d
