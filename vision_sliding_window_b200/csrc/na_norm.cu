// na_norm.cu -- the norms around a block, fused with its gate and residual:
//
//   y = x + scale * gate . P(o),   h = N(y) w + b,
//
// N a LayerNorm or RMS norm over the C channels of a row, P such a norm of
// the block's output o with its own weight and bias, or the identity; and
// the gradients of both.
//
// A row lives in registers between its one read and its one write, so the
// forward pass moves x, o, y and h once each and the backward pass y, o, dy,
// dh, dx and do once each: HBM bounds both.  Rows of up to 32 lanes' worth of
// channels are held by a part of a warp, wider ones by a whole block.
//
// Statistics are float32.  A LayerNorm's mean and variance come from each
// lane's own mean and centred sum of squares, which are exact to rounding
// whatever the mean, joined pairwise by
//   M = Ma + Mb + (mb - ma)^2 na nb / (na + nb):
// one reduction instead of the two of "mean first, then deviations", and
// none of the cancellation of "sum of squares minus squared sum".
#include <type_traits>

#include "na2d_common.cuh"
#include "na2d_internal.h"

namespace na2d {
namespace {

constexpr int kMaxThreads = 1024;

// ------------------------------------------------------------- elements
template <typename T> NA_DEVICE float to_f(T x);
template <> NA_DEVICE float to_f<float>(float x) { return x; }
template <> NA_DEVICE float to_f<__half>(__half x) { return __half2float(x); }
template <> NA_DEVICE float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> NA_DEVICE T from_f(float x);
template <> NA_DEVICE float from_f<float>(float x) { return x; }
template <> NA_DEVICE __half from_f<__half>(float x) { return __float2half_rn(x); }
template <> NA_DEVICE __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// VEC consecutive elements, moved as one access (16 bytes, or one element
// where the channel count does not keep rows 16-byte aligned).
template <typename T, int VEC> struct alignas(sizeof(T) * VEC) Pack { T e[VEC]; };

template <typename T, int VEC> NA_DEVICE Pack<T, VEC> load_pack(const T* p) {
  Pack<T, VEC> r;
  if constexpr (sizeof(T) * VEC == 16) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    r = *reinterpret_cast<const Pack<T, VEC>*>(&u);
  } else {
    r = *reinterpret_cast<const Pack<T, VEC>*>(p);
  }
  return r;
}
// rows that are read once: kept out of the way of the weights in L1.  Plain
// (coherent) loads, as x may be the buffer that y is written to.
template <typename T, int VEC> NA_DEVICE Pack<T, VEC> load_row(const T* p) {
  Pack<T, VEC> r;
  if constexpr (sizeof(T) * VEC == 16) {
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
    r = *reinterpret_cast<const Pack<T, VEC>*>(&u);
  } else {
    r = *reinterpret_cast<const Pack<T, VEC>*>(p);
  }
  return r;
}
template <typename T, int VEC> NA_DEVICE void store_pack(T* p, const float (&v)[VEC]) {
  Pack<T, VEC> r;
#pragma unroll
  for (int i = 0; i < VEC; ++i) r.e[i] = from_f<T>(v[i]);
  *reinterpret_cast<Pack<T, VEC>*>(p) = r;
}

// ----------------------------------------------------------- reductions
// A row is held by `lanes` consecutive threads: a power of two <= 32, or
// (BLOCK) all threads of the block.  `slot` alternates between two rows of
// shared memory, so that one barrier a reduction is enough.
struct Moments {
  float n, mean, m2;
};
NA_DEVICE Moments join(const Moments& a, const Moments& b) {
  const float n = a.n + b.n;
  const float d = b.mean - a.mean, f = n > 0.f ? b.n / n : 0.f;
  return Moments{n, a.mean + d * f, a.m2 + b.m2 + d * d * a.n * f};
}

struct Reducer {
  float (*scratch)[3][32];  // [2][3][32]
  int lanes, slot;

  template <bool BLOCK, int K> NA_DEVICE void sum(float (&v)[K]) {
    const int width = BLOCK ? 32 : lanes;
    for (int o = width >> 1; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if constexpr (BLOCK) {
      const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
      if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) scratch[slot][k][warp] = v[k];
      __syncthreads();
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] = (threadIdx.x & 31) < nw ? scratch[slot][k][threadIdx.x & 31] : 0.f;
      for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
      slot ^= 1;
    }
  }
  template <bool BLOCK> NA_DEVICE Moments moments(Moments m) {
    const int width = BLOCK ? 32 : lanes;
    auto across = [&](int o) {
      const Moments b{__shfl_xor_sync(0xffffffffu, m.n, o), __shfl_xor_sync(0xffffffffu, m.mean, o),
                      __shfl_xor_sync(0xffffffffu, m.m2, o)};
      // both partners join in the same order, so that they hold the same result
      m = (threadIdx.x & o) ? join(b, m) : join(m, b);
    };
    for (int o = 1; o < width; o <<= 1) across(o);
    if constexpr (BLOCK) {
      const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5, lane = threadIdx.x & 31;
      if (lane == 0) {
        scratch[slot][0][warp] = m.n;
        scratch[slot][1][warp] = m.mean;
        scratch[slot][2][warp] = m.m2;
      }
      __syncthreads();
      m = lane < nw ? Moments{scratch[slot][0][lane], scratch[slot][1][lane], scratch[slot][2][lane]}
                    : Moments{0.f, 0.f, 0.f};
      for (int o = 1; o < 32; o <<= 1) across(o);
      slot ^= 1;
    }
    return m;
  }
};

// Mean (0 for an RMS norm) and reciprocal deviation of a row's values v.
template <bool BLOCK, int NV, int VEC>
NA_DEVICE void row_stats(const float (&v)[NV][VEC], const bool (&in)[NV], int C, bool rms, float eps, Reducer& red,
                         float* mean, float* rstd) {
  const float inv = 1.f / (float)C;
  if (rms) {
    float s[1] = {0.f};
#pragma unroll
    for (int a = 0; a < NV; ++a)
#pragma unroll
      for (int i = 0; i < VEC; ++i) s[0] += in[a] ? v[a][i] * v[a][i] : 0.f;
    red.sum<BLOCK>(s);
    *mean = 0.f;
    *rstd = rsqrtf(s[0] * inv + eps);
    return;
  }
  int n = 0;
  float s = 0.f;
#pragma unroll
  for (int a = 0; a < NV; ++a) {
    n += in[a] ? VEC : 0;
#pragma unroll
    for (int i = 0; i < VEC; ++i) s += in[a] ? v[a][i] : 0.f;
  }
  Moments m{(float)n, n ? s / (float)n : 0.f, 0.f};
#pragma unroll
  for (int a = 0; a < NV; ++a)
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const float d = v[a][i] - m.mean;
      m.m2 += in[a] ? d * d : 0.f;
    }
  m = red.moments<BLOCK>(m);
  *mean = m.mean;
  *rstd = rsqrtf(m.m2 * inv + eps);
}

// ----------------------------------------------------------------- forward
template <typename T, int VEC, int NV, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? kMaxThreads : 256) norm_forward_kernel(NormArgs p) {
  __shared__ float scratch[2][3][32];
  Reducer red{scratch, BLOCK ? (int)blockDim.x : p.lanes, 0};
  const int lane = BLOCK ? threadIdx.x : threadIdx.x & (p.lanes - 1);
  const int per_block = BLOCK ? 1 : blockDim.x / p.lanes;
  const int sub = BLOCK ? 0 : threadIdx.x / p.lanes;
  const int lanes = red.lanes;
  const T *x = (const T*)p.x, *o = (const T*)p.o, *w = (const T*)p.w, *b = (const T*)p.b, *pw = (const T*)p.pw,
          *pb = (const T*)p.pb, *gate = (const T*)p.gate;
  T *yo = (T*)p.y, *h = (T*)p.h;
  bool in[NV];
  int col[NV];
#pragma unroll
  for (int a = 0; a < NV; ++a) {
    col[a] = (lane + a * lanes) * VEC;
    in[a] = col[a] < p.C;
  }
  // all lanes of a warp keep the same trip count: shuffles need them all
  for (long long base = (long long)blockIdx.x * per_block; base < p.rows; base += (long long)gridDim.x * per_block) {
    const long long row = base + sub;
    const bool live = row < p.rows;
    const long long at = (live ? row : p.rows - 1) * p.C;
    Pack<T, VEC> px[NV], po[NV];
#pragma unroll
    for (int a = 0; a < NV; ++a)
      if (in[a]) px[a] = load_row<T, VEC>(x + at + col[a]);
    if (o)
#pragma unroll
      for (int a = 0; a < NV; ++a)
        if (in[a]) po[a] = load_row<T, VEC>(o + at + col[a]);
    float y[NV][VEC];
    if (o) {
      float v[NV][VEC];
#pragma unroll
      for (int a = 0; a < NV; ++a)
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[a][i] = in[a] ? to_f<T>(po[a].e[i]) : 0.f;
      if (p.post) {
        float mean, rstd;
        row_stats<BLOCK>(v, in, p.C, p.rms, p.eps, red, &mean, &rstd);
#pragma unroll
        for (int a = 0; a < NV; ++a) {
          if (!in[a]) continue;
          Pack<T, VEC> k;
          if (pw) k = load_pack<T, VEC>(pw + col[a]);
#pragma unroll
          for (int i = 0; i < VEC; ++i) v[a][i] = (v[a][i] - mean) * rstd * (pw ? to_f<T>(k.e[i]) : 1.f);
          if (pb) {
            k = load_pack<T, VEC>(pb + col[a]);
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[a][i] += to_f<T>(k.e[i]);
          }
        }
      }
      const T* g = gate ? gate + (live ? row / p.gate_rows : 0) * p.C : nullptr;
#pragma unroll
      for (int a = 0; a < NV; ++a) {
        Pack<T, VEC> k;
        if (g && in[a]) k = load_pack<T, VEC>(g + col[a]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float f = g ? p.scale * (in[a] ? to_f<T>(k.e[i]) : 0.f) : p.scale;
          y[a][i] = in[a] ? fmaf(f, v[a][i], to_f<T>(px[a].e[i])) : 0.f;
        }
        if (in[a] && live) store_pack<T, VEC>(yo + at + col[a], y[a]);
      }
    } else {
#pragma unroll
      for (int a = 0; a < NV; ++a)
#pragma unroll
        for (int i = 0; i < VEC; ++i) y[a][i] = in[a] ? to_f<T>(px[a].e[i]) : 0.f;
    }
    if (h) {
      // h is the norm of y before y's rounding to T: one rounding, not two
      float mean, rstd;
      row_stats<BLOCK>(y, in, p.C, p.rms, p.eps, red, &mean, &rstd);
#pragma unroll
      for (int a = 0; a < NV; ++a) {
        if (!in[a]) continue;
        Pack<T, VEC> k;
        if (w) k = load_pack<T, VEC>(w + col[a]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) y[a][i] = (y[a][i] - mean) * rstd * (w ? to_f<T>(k.e[i]) : 1.f);
        if (b) {
          k = load_pack<T, VEC>(b + col[a]);
#pragma unroll
          for (int i = 0; i < VEC; ++i) y[a][i] += to_f<T>(k.e[i]);
        }
        if (live) store_pack<T, VEC>(h + at + col[a], y[a]);
      }
    }
  }
}

// ---------------------------------------------------------------- backward
// dx = dy + N'(dh);  dP = scale gate . dx;  do = P'(dP);
// dw = sum dh n, db = sum dh, dpw = sum dP m, dpb = sum dP,
// dgate = sum scale dx . P(o) over the rows of a gate row,
// with n, m the normalised rows and, for t = dn . w (or dP . pw),
//   N'(t) = rstd (t - mean(t) - n mean(t n))    (no mean(t) for an RMS norm).
//
// Rows are cut into chunks, one a block, none of which crosses a gate row
// unless it holds whole ones.  The sums over rows stay in registers, one set
// of columns a thread; a block's sums go to the workspace and a second kernel
// adds the blocks' in a fixed order, so results do not vary from run to run.
enum { kSumW, kSumB, kSumPW, kSumPB, kSumG, kSums };

// Adds the sums of the block's rows in `part` [sub][lanes][VEC*NV] order and
// writes them to `to`: with BLOCK every thread owns its columns alone.
template <int VEC, int NV, bool BLOCK>
NA_DEVICE void flush(float (&acc)[NV][VEC], float* to, const int (&col)[NV], const bool (&in)[NV], int lanes, int C,
                     float* buf) {
  if constexpr (!BLOCK) {
    const int nsub = blockDim.x / lanes;
    const int lane = threadIdx.x & (lanes - 1), sub = threadIdx.x / lanes;
    const int padded = lanes * NV * VEC;
    __syncthreads();
#pragma unroll
    for (int a = 0; a < NV; ++a)
#pragma unroll
      for (int i = 0; i < VEC; ++i) buf[sub * padded + (lane + a * lanes) * VEC + i] = acc[a][i];
    __syncthreads();
    for (int c = threadIdx.x; c < C; c += blockDim.x) {
      float s = 0.f;
      for (int u = 0; u < nsub; ++u) s += buf[u * padded + c];
      to[c] = s;
    }
  } else {
#pragma unroll
    for (int a = 0; a < NV; ++a)
      if (in[a])
#pragma unroll
        for (int i = 0; i < VEC; ++i) to[col[a] + i] = acc[a][i];
  }
#pragma unroll
  for (int a = 0; a < NV; ++a)
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[a][i] = 0.f;
}

template <typename T, int VEC, int NV, bool BLOCK, bool POST>
__global__ void __launch_bounds__(BLOCK ? (VEC == 1 ? kMaxThreads : 512) : 256) norm_backward_kernel(NormArgs p) {
  __shared__ float scratch[2][3][32];
  extern __shared__ float buf[];
  Reducer red{scratch, BLOCK ? (int)blockDim.x : p.lanes, 0};
  const int lane = BLOCK ? threadIdx.x : threadIdx.x & (p.lanes - 1);
  const int per_block = BLOCK ? 1 : blockDim.x / p.lanes;
  const int sub = BLOCK ? 0 : threadIdx.x / p.lanes;
  const int lanes = red.lanes;
  const T *yi = (const T*)p.x, *o = (const T*)p.o, *w = (const T*)p.w, *pw = (const T*)p.pw, *pb = (const T*)p.pb,
          *gate = (const T*)p.gate, *dy = (const T*)p.dy, *dh = (const T*)p.dh;
  T *dxo = (T*)p.dx, *doo = (T*)p.dout;
  const float inv = 1.f / (float)p.C;
  bool in[NV];
  int col[NV];
#pragma unroll
  for (int a = 0; a < NV; ++a) {
    col[a] = (lane + a * lanes) * VEC;
    in[a] = col[a] < p.C;
  }
  float aw[NV][VEC] = {}, ab[NV][VEC] = {}, apw[NV][VEC] = {}, apb[NV][VEC] = {}, ag[NV][VEC] = {};

  const long long chunk = blockIdx.x;
  long long r0, r1;
  if (p.pieces > 0) {  // a chunk is one of `pieces` parts of a gate row's rows
    const long long g = chunk / p.pieces, piece = chunk % p.pieces;
    r0 = g * p.gate_rows + piece * p.chunk_rows;
    r1 = min(r0 + p.chunk_rows, (g + 1) * p.gate_rows);
  } else {  // a chunk holds whole gate rows
    r0 = chunk * p.chunk_rows;
    r1 = min(r0 + p.chunk_rows, p.rows);
  }
  // rows run gate row by gate row, so that a gate row's sum can be written
  // out when its last row is done
  for (long long seg = r0; seg < r1;) {
    const long long seg_end = p.pieces > 0 ? r1 : min(r1, seg + p.gate_rows);
    for (long long base = seg; base < seg_end; base += per_block) {
      const long long row = base + sub;
      const bool live = row < seg_end;
      const long long at = (live ? row : seg) * p.C;
      Pack<T, VEC> py[NV], po[NV], pdy[NV], pdh[NV];
#pragma unroll
      for (int a = 0; a < NV; ++a)
        if (in[a]) {
          if (dh) py[a] = load_row<T, VEC>(yi + at + col[a]);
          if (dh) pdh[a] = load_row<T, VEC>(dh + at + col[a]);
          if (dy) pdy[a] = load_row<T, VEC>(dy + at + col[a]);
          if (o) po[a] = load_row<T, VEC>(o + at + col[a]);
        }
      float dx[NV][VEC];
#pragma unroll
      for (int a = 0; a < NV; ++a)
#pragma unroll
        for (int i = 0; i < VEC; ++i) dx[a][i] = (dy && in[a]) ? to_f<T>(pdy[a].e[i]) : 0.f;
      if (dh) {
        float n[NV][VEC], mean, rstd;
#pragma unroll
        for (int a = 0; a < NV; ++a)
#pragma unroll
          for (int i = 0; i < VEC; ++i) n[a][i] = in[a] ? to_f<T>(py[a].e[i]) : 0.f;
        row_stats<BLOCK>(n, in, p.C, p.rms, p.eps, red, &mean, &rstd);
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int a = 0; a < NV; ++a) {
          Pack<T, VEC> k;
          if (w && in[a]) k = load_pack<T, VEC>(w + col[a]);
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            if (!in[a]) continue;
            n[a][i] = (n[a][i] - mean) * rstd;
            const float g = to_f<T>(pdh[a].e[i]);
            const float t = w ? g * to_f<T>(k.e[i]) : g;
            s[0] += t;
            s[1] = fmaf(t, n[a][i], s[1]);
            if (live) {
              aw[a][i] = fmaf(g, n[a][i], aw[a][i]);
              ab[a][i] += g;
            }
          }
        }
        red.sum<BLOCK>(s);
        const float m0 = p.rms ? 0.f : s[0] * inv, m1 = s[1] * inv;
#pragma unroll
        for (int a = 0; a < NV; ++a) {
          Pack<T, VEC> k;
          if (w && in[a]) k = load_pack<T, VEC>(w + col[a]);
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            if (!in[a]) continue;
            const float g = to_f<T>(pdh[a].e[i]);
            const float t = w ? g * to_f<T>(k.e[i]) : g;
            dx[a][i] += rstd * (t - m0 - n[a][i] * m1);
          }
        }
      }
      if (live)
#pragma unroll
        for (int a = 0; a < NV; ++a)
          if (in[a]) store_pack<T, VEC>(dxo + at + col[a], dx[a]);
      if (o) {
        const T* g = gate ? gate + (live ? row : seg) / p.gate_rows * p.C : nullptr;
        float m[NV][VEC], mean = 0.f, rstd = 1.f;
#pragma unroll
        for (int a = 0; a < NV; ++a)
#pragma unroll
          for (int i = 0; i < VEC; ++i) m[a][i] = in[a] ? to_f<T>(po[a].e[i]) : 0.f;
        if constexpr (POST) row_stats<BLOCK>(m, in, p.C, p.rms, p.eps, red, &mean, &rstd);
        float s[2] = {0.f, 0.f};
        // dx becomes dP . pw, the gradient of the post norm's normalised row
#pragma unroll
        for (int a = 0; a < NV; ++a) {
          Pack<T, VEC> kg, kw, kb;
          if (in[a]) {
            if (g) kg = load_pack<T, VEC>(g + col[a]);
            if constexpr (POST) {
              if (pw) kw = load_pack<T, VEC>(pw + col[a]);
              if (pb) kb = load_pack<T, VEC>(pb + col[a]);
            }
          }
          float gp[VEC];
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            if (!in[a]) continue;
            const float wv = POST && pw ? to_f<T>(kw.e[i]) : 1.f;
            if constexpr (POST) m[a][i] = (m[a][i] - mean) * rstd;
            const float d = p.scale * dx[a][i];
            const float pv = POST ? fmaf(m[a][i], wv, pb ? to_f<T>(kb.e[i]) : 0.f) : m[a][i];
            gp[i] = d * pv;
            if (live) ag[a][i] += gp[i];
            const float dp = g ? d * to_f<T>(kg.e[i]) : d;
            if constexpr (POST) {
              if (live) {
                apw[a][i] = fmaf(dp, m[a][i], apw[a][i]);
                apb[a][i] += dp;
              }
              dx[a][i] = dp * wv;
              s[0] += dx[a][i];
              s[1] = fmaf(dx[a][i], m[a][i], s[1]);
            } else {
              dx[a][i] = dp;
            }
          }
          if (p.gate_rows == 1 && p.dgate && live && in[a])
#pragma unroll
            for (int i = 0; i < VEC; ++i) p.dgate[at + col[a] + i] = gp[i];
        }
        if constexpr (POST) {
          red.sum<BLOCK>(s);
          const float m0 = p.rms ? 0.f : s[0] * inv, m1 = s[1] * inv;
#pragma unroll
          for (int a = 0; a < NV; ++a)
#pragma unroll
            for (int i = 0; i < VEC; ++i)
              if (in[a]) dx[a][i] = rstd * (dx[a][i] - m0 - m[a][i] * m1);
        }
        if (live)
#pragma unroll
          for (int a = 0; a < NV; ++a)
            if (in[a]) store_pack<T, VEC>(doo + at + col[a], dx[a]);
      }
    }
    if (p.pieces == 0 && p.dgate && p.gate_rows > 1)
      flush<VEC, NV, BLOCK>(ag, p.dgate + seg / p.gate_rows * p.C, col, in, lanes, p.C, buf);
    seg = seg_end;
  }
  float* part = p.partial + chunk * p.C;
  const long long step = p.chunks * (long long)p.C;
  if (p.dw) flush<VEC, NV, BLOCK>(aw, part + kSumW * step, col, in, lanes, p.C, buf);
  if (p.db) flush<VEC, NV, BLOCK>(ab, part + kSumB * step, col, in, lanes, p.C, buf);
  if constexpr (POST) {
    if (p.dpw) flush<VEC, NV, BLOCK>(apw, part + kSumPW * step, col, in, lanes, p.C, buf);
    if (p.dpb) flush<VEC, NV, BLOCK>(apb, part + kSumPB * step, col, in, lanes, p.C, buf);
  }
  if (p.pieces > 0 && p.dgate) flush<VEC, NV, BLOCK>(ag, part + kSumG * step, col, in, lanes, p.C, buf);
}

// Adds the chunks' sums: 32 columns x 8 chunk lanes a block, each lane its
// chunks in order, then the lanes in order.
__global__ void __launch_bounds__(256) norm_reduce_kernel(NormArgs p) {
  __shared__ float buf[8][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
  const int which = blockIdx.y < 4 ? (int)blockIdx.y : (int)kSumG;
  float* to = which == kSumW ? p.dw : which == kSumB ? p.db : which == kSumPW ? p.dpw : which == kSumPB ? p.dpb : p.dgate;
  if (!to || (which == kSumG && p.pieces == 0)) return;
  long long k0 = 0, k1 = p.chunks;
  if (which == kSumG) {
    const long long g = blockIdx.y - 4;
    k0 = g * p.pieces;
    k1 = k0 + p.pieces;
    to += g * p.C;
  }
  const float* from = p.partial + which * p.chunks * (long long)p.C;
  float s = 0.f;
  if (c < p.C)
    for (long long k = k0 + part; k < k1; k += 8) s += from[k * p.C + c];
  buf[part][threadIdx.x & 31] = s;
  __syncthreads();
  if (part == 0 && c < p.C) {
#pragma unroll
    for (int u = 1; u < 8; ++u) s += buf[u][threadIdx.x];
    to[c] = s;
  }
}

// ---------------------------------------------------------------- launches
int sms() {
  static int counts[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  if (!counts[dev]) cudaDeviceGetAttribute(&counts[dev], cudaDevAttrMultiProcessorCount, dev);
  return counts[dev] > 0 ? counts[dev] : 148;
}

int pow2_at_least(int n) {
  int p = 1;
  while (p < n) p *= 2;
  return p;
}

// How a row is held: lanes <= 32 of a warp (block = 0), or a block of that
// many threads, nv vectors a thread.
struct Plan {
  int lanes, block, nv;
};
Plan plan_for(int C, int vec, int max_warp_nv, int block_nv) {
  const int n = (C + vec - 1) / vec;
  if (n <= 32) return {pow2_at_least(n), 0, 1};
  for (int nv = 2; nv <= max_warp_nv; nv *= 2)
    if (n <= 32 * nv) return {32, 0, nv};
  int nv = block_nv;
  const int threads = ((n + nv - 1) / nv + 31) / 32 * 32;
  return {0, threads, nv};
}

template <typename T, int VEC, int NV, bool BLOCK>
cudaError_t forward_one(const NormArgs& p, const Plan& pl, cudaStream_t st) {
  const int threads = BLOCK ? pl.block : 256;
  const long long per_block = BLOCK ? 1 : 256 / pl.lanes;
  const long long need = (p.rows + per_block - 1) / per_block;
  const long long most = (long long)sms() * 64;
  norm_forward_kernel<T, VEC, NV, BLOCK><<<(unsigned)(need < most ? need : most), threads, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T, int VEC> cudaError_t forward_vec(NormArgs p, cudaStream_t st) {
  constexpr int kBlockNV = VEC == 1 ? 8 : 4;
  const Plan pl = plan_for(p.C, VEC, 4, kBlockNV);
  p.lanes = pl.lanes;
  if (pl.block) return forward_one<T, VEC, kBlockNV, true>(p, pl, st);
  if (pl.nv == 1) return forward_one<T, VEC, 1, false>(p, pl, st);
  if (pl.nv == 2) return forward_one<T, VEC, 2, false>(p, pl, st);
  return forward_one<T, VEC, 4, false>(p, pl, st);
}

template <typename T> cudaError_t forward_t(const NormArgs& p, cudaStream_t st) {
  constexpr int kVec = 16 / sizeof(T);
  return p.C % kVec == 0 ? forward_vec<T, kVec>(p, st) : forward_vec<T, 1>(p, st);
}

// Chunks: about two blocks an SM, but not under 8 rows a block.
struct Chunks {
  long long count, rows;
  int pieces;
};
Chunks chunks_for(long long rows, long long gate_rows) {
  const long long blocks = 2ll * 148;  // also on a device with other SM counts: the sums' order is fixed by it
  long long r = (rows + blocks - 1) / blocks;
  if (r < 8) r = 8;
  if (gate_rows >= r) {
    const long long pieces = (gate_rows + r - 1) / r;
    const long long per = (gate_rows + pieces - 1) / pieces;
    return {rows / gate_rows * pieces, per, (int)pieces};
  }
  const long long per = r / gate_rows * gate_rows;
  return {(rows + per - 1) / per, per, 0};
}

template <typename T, int VEC, int NV, bool BLOCK, bool POST>
cudaError_t backward_one(const NormArgs& p, const Plan& pl, cudaStream_t st) {
  const int threads = BLOCK ? pl.block : 256;
  const size_t smem = BLOCK ? 0 : sizeof(float) * 256 * NV * VEC;
  norm_backward_kernel<T, VEC, NV, BLOCK, POST><<<(unsigned)p.chunks, threads, smem, st>>>(p);
  return cudaGetLastError();
}
template <typename T, int VEC, int NV, bool BLOCK>
cudaError_t backward_post(const NormArgs& p, const Plan& pl, cudaStream_t st) {
  return p.post ? backward_one<T, VEC, NV, BLOCK, true>(p, pl, st) : backward_one<T, VEC, NV, BLOCK, false>(p, pl, st);
}
template <typename T, int VEC> cudaError_t backward_vec(NormArgs p, cudaStream_t st) {
  constexpr int kBlockNV = VEC == 1 ? 8 : 16 / VEC;  // 16 columns a thread (8 where they are moved one by one)
  const Plan pl = plan_for(p.C, VEC, 2, kBlockNV);
  p.lanes = pl.lanes;
  if (pl.block) return backward_post<T, VEC, kBlockNV, true>(p, pl, st);
  if (pl.nv == 1) return backward_post<T, VEC, 1, false>(p, pl, st);
  return backward_post<T, VEC, 2, false>(p, pl, st);
}
template <typename T> cudaError_t backward_t(const NormArgs& p, cudaStream_t st) {
  constexpr int kVec = 16 / sizeof(T);
  return p.C % kVec == 0 ? backward_vec<T, kVec>(p, st) : backward_vec<T, 1>(p, st);
}

}  // namespace

size_t norm_workspace_bytes(long long rows, int C, long long gate_rows) {
  return (size_t)chunks_for(rows, gate_rows).count * (size_t)C * kSums * sizeof(float);
}

cudaError_t launch_norm_forward(const NormArgs& p, na_dtype dt, cudaStream_t st) {
  if (dt == NA_F32) return forward_t<float>(p, st);
  if (dt == NA_F16) return forward_t<__half>(p, st);
  return forward_t<__nv_bfloat16>(p, st);
}

cudaError_t launch_norm_backward(NormArgs p, na_dtype dt, cudaStream_t st) {
  const Chunks c = chunks_for(p.rows, p.gate_rows);
  p.chunks = c.count;
  p.chunk_rows = c.rows;
  p.pieces = c.pieces;
  cudaError_t e = dt == NA_F32 ? backward_t<float>(p, st)
                  : dt == NA_F16 ? backward_t<__half>(p, st)
                                 : backward_t<__nv_bfloat16>(p, st);
  if (e != cudaSuccess) return e;
  const long long gates = p.dgate && p.pieces > 0 ? p.rows / p.gate_rows : 0;
  if (!p.dw && !p.db && !p.dpw && !p.dpb && gates == 0) return cudaSuccess;
  norm_reduce_kernel<<<dim3((unsigned)((p.C + 31) / 32), (unsigned)(4 + gates)), 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace na2d
