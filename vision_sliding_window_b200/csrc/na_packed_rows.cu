// na_packed_rows.cu -- the packed attention of few rows over many keys, fp16
// and bf16: single tokens (and a few more) over a cache.
//
// Every key and value is read once for the rows of its group, 2 d FLOPs a
// row and key: HBM bounds it, and what matters is how many bytes a block has
// in flight.  A block takes a piece of a sequence's keys of one key head; its
// four warps take 16 keys in turn, each with a running maximum and sum of its
// own, joined at the end through shared memory.  Keys and values go straight
// from global memory into the operand registers of m16n8k16 products, with no
// shared memory and no barrier in the loop: a product's contraction index and
// its output columns may be numbered in any order, so a thread takes 16
// consecutive bytes and calls them its own indices.  The next keys are asked
// for as soon as the logits are done, the next values after their product.
// The rows of a group fill a 16-row operand only in part; the idle rows cost
// tensor time that nothing waits for (tcgen05's 128-row tiles would need
// the keys staged for a tile that is 1/32 full).
#include "na_packed.cuh"

namespace na2d {
namespace {

using namespace packed;

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr float kSlack = 8.f;  // log2 of how far a maximum may pass its reference

template <typename T>
NA_DEVICE void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (__is_same(T, __half))
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// N 32-bit words of consecutive elements, zeros if not live
template <int N> NA_DEVICE void load_words(uint32_t (&r)[N], const void* from, bool live) {
  if constexpr (N == 4) {
    const uint4 u = live ? __ldg((const uint4*)from) : make_uint4(0, 0, 0, 0);
    r[0] = u.x, r[1] = u.y, r[2] = u.z, r[3] = u.w;
  } else if constexpr (N == 2) {
    const uint2 u = live ? __ldg((const uint2*)from) : make_uint2(0, 0);
    r[0] = u.x, r[1] = u.y;
  } else {
    r[0] = live ? __ldg((const uint32_t*)from) : 0u;
  }
}

template <int D> struct Rows {
  static constexpr int KE = D >= 32 ? 8 : 4;   // consecutive columns of a key a thread takes
  static constexpr int KC = D / (4 * KE);      // of which it takes this many runs
  static constexpr int VE = D >= 64 ? 8 : D / 8;  // the same for values
  static constexpr int VC = D / (8 * VE);
  static constexpr int LD = D + 4;
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) packed_rows_kernel(PackedArgs p) {
  using R = Rows<D>;
  __shared__ float so[kWarps][16][R::LD];
  __shared__ float sm[kWarps][16], sl[kWarps][16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int kh = blockIdx.y;
  const float sl2 = p.scale * kLog2e;
  const bool split = p.piece_keys > 0;
  int s;
  long long idx;
  if (split)
    find_part_warp(p.cu_k, p.nseq, p.total_k, 1, p.piece_keys, blockIdx.x, &s, &idx);
  else
    find_part_warp(p.cu_q, p.nseq, p.total_q, p.group, 16, blockIdx.x, &s, &idx);
  if (idx < 0) return;
  const Span sp = span_of(p, s);
  const long long all_rows = (long long)sp.nq * p.group;
  int piece0 = 0, piece1 = sp.nk;
  long long t0 = idx, t1 = idx + 1;
  if (split) {
    if (idx >= p.max_pieces || idx * p.piece_keys >= sp.nk) return;
    piece0 = (int)idx * p.piece_keys;
    piece1 = (int)min((long long)piece0 + p.piece_keys, (long long)sp.nk);
    t0 = 0;
    t1 = (all_rows + 15) / 16;
  }
  const long long stride = (long long)p.hk * D;
  const T* kbase = (const T*)p.k + ((long long)sp.k0 * p.hk + kh) * D;
  const T* vbase = (const T*)p.v + ((long long)sp.k0 * p.hk + kh) * D;
  for (long long t = t0; t < t1; ++t) {
    const long long r0 = t * 16;
    if (r0 >= all_rows) return;
    const int n = (int)min(16ll, all_rows - r0);
    // this thread's rows g and g + 8: where they lie and what they see
    int lo[2], hi[2], kb, ke, unused;
    const T* qrow[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const long long r = r0 + min(g + 8 * h, n - 1);
      const int pos = (int)(r / p.group);
      visible(p, sp, pos, &lo[h], &hi[h]);
      if (g + 8 * h >= n) hi[h] = lo[h];
      qrow[h] = (const T*)p.q + (((long long)sp.q0 + pos) * p.hq + kh * p.group + (int)(r - (long long)pos * p.group)) * D;
    }
    visible(p, sp, (int)(r0 / p.group), &kb, &unused);
    visible(p, sp, (int)((r0 + n - 1) / p.group), &unused, &ke);
    kb = max(kb, piece0);
    ke = min(ke, piece1);

    uint32_t kr[2][R::KC][R::KE / 2], vr[4][R::VC][R::VE / 2];
    auto load_k = [&](int j0) {
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const int key = j0 + nt * 8 + g;
        const T* from = kbase + key * stride + q * R::KE;
#pragma unroll
        for (int c = 0; c < R::KC; ++c) load_words(kr[nt][c], from + c * 4 * R::KE, key < ke);
      }
    };
    auto load_v = [&](int j0) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int key = j0 + (e >> 1) * 8 + 2 * q + (e & 1);
        const T* from = vbase + key * stride + g * R::VE;
#pragma unroll
        for (int c = 0; c < R::VC; ++c) load_words(vr[e][c], from + c * 8 * R::VE, key < ke);
      }
    };
    int j0 = kb + warp * 16;
    if (j0 < ke) {
      load_k(j0);
      load_v(j0);
    }
    // the rows' operand, columns numbered as the keys' are; idle rows are zero
    uint32_t qa[R::KC][R::KE / 4][4];
#pragma unroll
    for (int c = 0; c < R::KC; ++c)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t w[R::KE / 2];
        load_words(w, qrow[h] + c * 4 * R::KE + q * R::KE, g + 8 * h < n);
#pragma unroll
        for (int x = 0; x < R::KE / 4; ++x) qa[c][x][h] = w[2 * x], qa[c][x][2 + h] = w[2 * x + 1];
      }
    float o[R::VC][R::VE][4], ref[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < R::VC; ++c)
#pragma unroll
      for (int i = 0; i < R::VE; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[c][i][x] = 0.f;

    for (; j0 < ke; j0 += 16 * kWarps) {
      float sc[2][4] = {};
#pragma unroll
      for (int c = 0; c < R::KC; ++c)
#pragma unroll
        for (int x = 0; x < R::KE / 4; ++x)
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
            mma16816<T>(sc[nt], qa[c][x][0], qa[c][x][1], qa[c][x][2], qa[c][x][3], kr[nt][c][2 * x], kr[nt][c][2 * x + 1]);
      const int next = j0 + 16 * kWarps;
      if (next < ke) load_k(next);
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int key = j0 + nt * 8 + 2 * q + (x & 1), h = x >> 1;
          if (!(key >= lo[h] && key < hi[h] && key < ke)) sc[nt][x] = -INFINITY;
          top[h] = fmaxf(top[h], sc[nt][x]);
        }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
        top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
      }
      // -inf - -inf is NaN and compares false: nothing seen yet stays so
      if (__any_sync(0xffffffffu, (top[0] - ref[0]) * sl2 > kSlack || (top[1] - ref[1]) * sl2 > kSlack)) {
        float f[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float to = fmaxf(ref[h], top[h]);
          f[h] = ref[h] == to ? 1.f : exp2f((ref[h] - to) * sl2);
          ref[h] = to;
          sum[h] *= f[h];
        }
#pragma unroll
        for (int c = 0; c < R::VC; ++c)
#pragma unroll
          for (int i = 0; i < R::VE; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[c][i][x] = f[x >> 1] == 0.f ? 0.f : o[c][i][x] * f[x >> 1];
      }
      uint32_t pa[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float shift = ref[h] == -INFINITY ? 0.f : -ref[h] * sl2;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const float a = exp2f(fmaf(sc[nt][2 * h], sl2, shift)), b = exp2f(fmaf(sc[nt][2 * h + 1], sl2, shift));
          sum[h] += a + b;
          pa[2 * nt + h] = pack2<T>(a, b);
        }
      }
#pragma unroll
      for (int c = 0; c < R::VC; ++c)
#pragma unroll
        for (int i = 0; i < R::VE; ++i) {
          // column i of this thread's run, of keys (2q, 2q+1) and (2q+8, 2q+9)
          const uint32_t pick = (i & 1) ? 0x7632u : 0x5410u;
          const uint32_t b0 = __byte_perm(vr[0][c][i / 2], vr[1][c][i / 2], pick);
          const uint32_t b1 = __byte_perm(vr[2][c][i / 2], vr[3][c][i / 2], pick);
          mma16816<T>(o[c][i], pa[0], pa[1], pa[2], pa[3], b0, b1);
        }
      if (next < ke) load_v(next);
    }
    // ------------------------------------------------- join the four warps
    __syncthreads();  // a row tile before this one may still be read
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 1);
      sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 2);
      if (q == 0) sm[warp][g + 8 * h] = ref[h], sl[warp][g + 8 * h] = sum[h];
    }
#pragma unroll
    for (int c = 0; c < R::VC; ++c)
#pragma unroll
      for (int i = 0; i < R::VE; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          so[warp][g + 8 * (x >> 1)][c * 8 * R::VE + (2 * q + (x & 1)) * R::VE + i] = o[c][i][x];
    __syncthreads();
    for (int r = warp; r < n; r += kWarps) {
      float m = -INFINITY, f[kWarps], l = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm[w][r]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        f[w] = sm[w][r] == m ? 1.f : exp2f((sm[w][r] - m) * sl2);
        l += sl[w][r] * f[w];
      }
      float acc[(D + 31) / 32];
      bool finite = fabsf(l) < INFINITY;
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
      for (int e = 0; e < (D + 31) / 32; ++e) {
        acc[e] = 0.f;
        if (lane + 32 * e < D)
#pragma unroll
          for (int w = 0; w < kWarps; ++w)
            if (f[w] != 0.f) acc[e] = fmaf(so[w][r][lane + 32 * e], f[w], acc[e]);
        acc[e] *= inv;
        finite = finite && fabsf(acc[e]) < INFINITY;
      }
      const long long rr = r0 + r;
      const int pos = (int)(rr / p.group), head = kh * p.group + (int)(rr - (long long)pos * p.group);
      const long long i = (long long)sp.q0 + pos, row = i * p.hq + head;
      float lse = l == 0.f ? -INFINITY : fmaf(m, p.scale, log2f(l) * kLn2);
      if (__any_sync(0xffffffffu, !finite)) {
        int a, b;
        visible(p, sp, pos, &a, &b);
        exact_row<T, D>(p, (const T*)p.q + row * D, kbase, vbase, stride, max(a, piece0), min(b, piece1), acc, &l, &m);
#pragma unroll
        for (int e = 0; e < (D + 31) / 32; ++e) acc[e] /= l;
        lse = (m + log2f(l)) * kLn2;
      }
      const long long at = split ? (idx * p.total_q + i) * p.hq + head : row;
#pragma unroll
      for (int e = 0; e < (D + 31) / 32; ++e)
        if (lane + 32 * e < D) {
          if (split)
            p.part_o[at * D + lane + 32 * e] = acc[e];
          else
            ((T*)p.out)[at * D + lane + 32 * e] = from_f<T>(acc[e]);
        }
      if (lane == 0) {
        if (split)
          p.part_lse[at] = lse;
        else if (p.lse)
          p.lse[(long long)head * p.total_q + i] = lse;
      }
    }
  }
}

template <typename T, int D> cudaError_t launch(const PackedArgs& p, cudaStream_t st) {
  const long long blocks = p.piece_keys > 0 ? part_numbers(p.nseq, p.total_k, 1, p.piece_keys)
                                            : part_numbers(p.nseq, p.total_q, p.group, 16);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  packed_rows_kernel<T, D><<<dim3((unsigned)blocks, (unsigned)p.hk), kThreads, 0, st>>>(p);
  return cudaGetLastError();
}
template <typename T> cudaError_t launch_d(const PackedArgs& p, cudaStream_t st) {
  switch (p.d) {
    case 16: return launch<T, 16>(p, st);
    case 32: return launch<T, 32>(p, st);
    case 64: return launch<T, 64>(p, st);
    case 128: return launch<T, 128>(p, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_packed_forward_rows(const PackedArgs& p, na_dtype dt, cudaStream_t st) {
  return dt == NA_F16 ? launch_d<__half>(p, st) : launch_d<__nv_bfloat16>(p, st);
}

}  // namespace na2d
