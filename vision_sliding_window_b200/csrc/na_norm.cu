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
// Statistics are float32: the mean first, then the mean square of the
// deviations from it, which is exact to rounding whatever the mean is, as "sum
// of squares minus squared sum" is not.  Rows are in registers, so the second
// pass costs one more reduction and no memory.
#include <type_traits>

#include "na2d_common.cuh"
#include "na2d_internal.h"
#include "na2d_sm100.cuh"

namespace na2d {
namespace {

// ------------------------------------------------------------- elements
template <typename T> NA_DEVICE float to_f(T x);
template <> NA_DEVICE float to_f<float>(float x) { return x; }
template <> NA_DEVICE float to_f<__half>(__half x) { return __half2float(x); }
template <> NA_DEVICE float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> NA_DEVICE T from_f(float x);
template <> NA_DEVICE float from_f<float>(float x) { return x; }
template <> NA_DEVICE __half from_f<__half>(float x) { return __float2half_rn(x); }
template <> NA_DEVICE __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Which gate row a row has.  A 64-bit division costs more than a row's other
// arithmetic, so it is kept for counts that need it.
NA_DEVICE long long gate_of(const NormArgs& p, long long row) {
  if (p.gate_rows >= p.rows) return 0;
  if (p.rows <= 0xffffffffll) return (uint32_t)row / (uint32_t)p.gate_rows;
  return row / p.gate_rows;
}

// VEC consecutive elements, moved as one access: 16 bytes where the channel
// count keeps rows so aligned, else four elements or one.
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
struct Reducer {
  float (*scratch)[2][32];  // [2][2][32]
  int lanes, slot;

  template <bool BLOCK, int K> NA_DEVICE void sum(float (&v)[K]) {
    if constexpr (!BLOCK) {
      for (int o = lanes >> 1; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    } else {
      const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
      if (lane == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) scratch[slot][k][warp] = v[k];
      __syncthreads();
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] = lane < nw ? scratch[slot][k][lane] : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
      slot ^= 1;
    }
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
      for (int i = 0; i < VEC; ++i) s[0] = fmaf(v[a][i], v[a][i], s[0]);  // 0 where not in
    red.sum<BLOCK>(s);
    *mean = 0.f;
    *rstd = rsqrtf(s[0] * inv + eps);
    return;
  }
  float s[1] = {0.f}, m2[1] = {0.f};
#pragma unroll
  for (int a = 0; a < NV; ++a)
#pragma unroll
    for (int i = 0; i < VEC; ++i) s[0] += v[a][i];  // 0 where not in
  red.sum<BLOCK>(s);
  *mean = s[0] * inv;
#pragma unroll
  for (int a = 0; a < NV; ++a)
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const float d = v[a][i] - *mean;
      m2[0] += in[a] ? d * d : 0.f;
    }
  red.sum<BLOCK>(m2);
  *rstd = rsqrtf(m2[0] * inv + eps);
}

// ----------------------------------------------------------------- forward
// Rows are asked for one ahead: while a row goes through its reductions, the
// loads of the next are in flight.
template <typename T, int VEC, int NV, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 1024 : 256, 1)
norm_forward_kernel(NormArgs p) {
  __shared__ float scratch[2][2][32];
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
  Pack<T, VEC> px[NV], po[NV];
  auto ask = [&](long long base) {
    const long long at = min(base + sub, p.rows - 1) * p.C;
#pragma unroll
    for (int a = 0; a < NV; ++a)
      if (in[a]) px[a] = load_row<T, VEC>(x + at + col[a]);
    if (o)
#pragma unroll
      for (int a = 0; a < NV; ++a)
        if (in[a]) po[a] = load_row<T, VEC>(o + at + col[a]);
  };
  const long long step = (long long)gridDim.x * per_block;
  long long base = (long long)blockIdx.x * per_block;
  if (base < p.rows) ask(base);
  // all lanes of a warp keep the same trip count: shuffles need them all
  for (; base < p.rows; base += step) {
    const long long row = base + sub;
    const bool live = row < p.rows;
    const long long at = (live ? row : p.rows - 1) * p.C;
    float y[NV][VEC], v[NV][VEC];
#pragma unroll
    for (int a = 0; a < NV; ++a)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        y[a][i] = in[a] ? to_f<T>(px[a].e[i]) : 0.f;
        v[a][i] = o && in[a] ? to_f<T>(po[a].e[i]) : 0.f;
      }
    if (base + step < p.rows) ask(base + step);
    if (o) {
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
      const T* g = gate ? gate + gate_of(p, live ? row : 0) * p.C : nullptr;
#pragma unroll
      for (int a = 0; a < NV; ++a) {
        if (!in[a]) continue;
        Pack<T, VEC> k;
        if (g) k = load_pack<T, VEC>(g + col[a]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) y[a][i] = fmaf(g ? p.scale * to_f<T>(k.e[i]) : p.scale, v[a][i], y[a][i]);
        if (live) store_pack<T, VEC>(yo + at + col[a], y[a]);
      }
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

// As in the forward pass, a row's loads are in flight while the one before it
// is worked on: a block of a wide row is alone on its SM, as its sums (up to
// five a column) fill the registers.
template <typename T, int VEC, int NV, bool BLOCK, bool POST>
__global__ void __launch_bounds__(BLOCK ? 512 : 256, BLOCK ? 1 : 2) norm_backward_kernel(NormArgs p) {
  __shared__ float scratch[2][2][32];
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
  Pack<T, VEC> py[NV], po[NV], pdy[NV], pdh[NV];
  auto ask = [&](long long row) {
    const long long at = row * p.C;
#pragma unroll
    for (int a = 0; a < NV; ++a)
      if (in[a]) {
        if (dh) py[a] = load_row<T, VEC>(yi + at + col[a]);
        if (dh) pdh[a] = load_row<T, VEC>(dh + at + col[a]);
        if (dy) pdy[a] = load_row<T, VEC>(dy + at + col[a]);
        if (o) po[a] = load_row<T, VEC>(o + at + col[a]);
      }
  };
  auto end_of = [&](long long seg) { return p.pieces > 0 ? r1 : min(r1, seg + p.gate_rows); };
  // rows past the segment are read as its first, whose values go nowhere
  if (r0 < r1) ask(r0 + sub < end_of(r0) ? r0 + sub : r0);
  for (long long seg = r0; seg < r1;) {
    const long long seg_end = end_of(seg), gate_row = gate_of(p, seg);
    for (long long base = seg; base < seg_end; base += per_block) {
      const long long row = base + sub;
      const bool live = row < seg_end;
      const long long at = (live ? row : seg) * p.C;
      Pack<T, VEC> cy[NV], co[NV], cdy[NV], cdh[NV];
#pragma unroll
      for (int a = 0; a < NV; ++a) cy[a] = py[a], co[a] = po[a], cdy[a] = pdy[a], cdh[a] = pdh[a];
      {
        const bool same = base + per_block < seg_end;
        const long long next = same ? base + per_block : seg_end, first = same ? seg : seg_end;
        if (next < r1) ask(next + sub < end_of(first) ? next + sub : first);
      }
      float dx[NV][VEC];
#pragma unroll
      for (int a = 0; a < NV; ++a)
#pragma unroll
        for (int i = 0; i < VEC; ++i) dx[a][i] = (dy && in[a]) ? to_f<T>(cdy[a].e[i]) : 0.f;
      if (dh) {
        float n[NV][VEC], mean, rstd;
#pragma unroll
        for (int a = 0; a < NV; ++a)
#pragma unroll
          for (int i = 0; i < VEC; ++i) n[a][i] = in[a] ? to_f<T>(cy[a].e[i]) : 0.f;
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
            const float g = to_f<T>(cdh[a].e[i]);
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
            const float g = to_f<T>(cdh[a].e[i]);
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
        const T* g = gate ? gate + gate_row * p.C : nullptr;
        float m[NV][VEC], mean = 0.f, rstd = 1.f;
#pragma unroll
        for (int a = 0; a < NV; ++a)
#pragma unroll
          for (int i = 0; i < VEC; ++i) m[a][i] = in[a] ? to_f<T>(co[a].e[i]) : 0.f;
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
      flush<VEC, NV, BLOCK>(ag, p.dgate + gate_row * p.C, col, in, lanes, p.C, buf);
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

// -------------------------------------------------------------- wide rows
// A block holds a row of more channels than a warp takes, whose bytes are a
// multiple of 16.  Rows come through a
// ring of bulk copies in shared memory, so that what is in flight does not
// hang on registers or on how many blocks an SM holds; the copy of a later row
// starts as soon as a reduction's barrier has shown that all threads have
// read the row.  Arithmetic is in pairs (two float32 an instruction), as
// instruction issue came next.
constexpr int kMaxStages = 8;

struct Ring {
  uint32_t data, bars, stage_bytes, row_bytes;
  int stages;
  NA_DEVICE uint32_t at(long long it) const { return data + (uint32_t)(it % stages) * stage_bytes; }
  NA_DEVICE uint32_t bar(long long it) const { return bars + (uint32_t)(it % stages) * 8; }
};

template <typename T, int VEC> NA_DEVICE void lds_floats(uint32_t at, float (&v)[VEC]) {
  Pack<T, VEC> r;
  if constexpr (sizeof(r) == 16) {
    uint4 u;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(at));
    r = *reinterpret_cast<const Pack<T, VEC>*>(&u);
  } else {
    uint2 u;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(u.x), "=r"(u.y) : "r"(at));
    r = *reinterpret_cast<const Pack<T, VEC>*>(&u);
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i) v[i] = to_f<T>(r.e[i]);
}
template <typename T, int VEC> NA_DEVICE void ldg_floats(const T* p, float (&v)[VEC]) {
  const Pack<T, VEC> r = load_pack<T, VEC>(p);
#pragma unroll
  for (int i = 0; i < VEC; ++i) v[i] = to_f<T>(r.e[i]);
}

#define NA_PAIRS(i) _Pragma("unroll") for (int i = 0; i < VEC; i += 2)
#define NA_RUNS(a) _Pragma("unroll") for (int a = 0; a < NV; ++a)

// Sums of the K rows v[0 .. K) and of the squares of their deviations from the
// mean (from 0 for an RMS norm), all K in each reduction.  Values are 0 where
// a thread's columns are past the row, and masked where that matters.
template <int K, int NV, int VEC>
NA_DEVICE void wide_stats(float (&v)[K][NV][VEC], const bool (&in)[NV], float inv, bool rms, float eps, Reducer& red,
                          float (&mean)[K], float (&rstd)[K]) {
  float s[K];
  if (!rms) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float a0 = 0.f, a1 = 0.f;
      NA_RUNS(a) NA_PAIRS(i) sm100::add2(a0, a1, a0, a1, v[k][a][i], v[k][a][i + 1]);
      s[k] = a0 + a1;
    }
    red.sum<true>(s);
#pragma unroll
    for (int k = 0; k < K; ++k) mean[k] = s[k] * inv;
#pragma unroll
    for (int k = 0; k < K; ++k) NA_RUNS(a) if (in[a]) {
        NA_PAIRS(i) sm100::add2(v[k][a][i], v[k][a][i + 1], v[k][a][i], v[k][a][i + 1], -mean[k], -mean[k]);
      }
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float a0 = 0.f, a1 = 0.f;
    NA_RUNS(a) NA_PAIRS(i) sm100::fma2(a0, a1, v[k][a][i], v[k][a][i + 1], v[k][a][i], v[k][a][i + 1], a0, a1);
    s[k] = a0 + a1;
  }
  red.sum<true>(s);
#pragma unroll
  for (int k = 0; k < K; ++k) rstd[k] = rsqrtf(s[k] * inv + eps);
}

template <typename T, int VEC, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? 3 : 1) norm_forward_wide_kernel(NormArgs p, int stages) {
  using namespace sm100;
  extern __shared__ __align__(128) uint8_t ring_data[];
  __shared__ float scratch[2][2][32];
  __shared__ uint64_t ring_bars[kMaxStages];
  __shared__ volatile int abort_flag;
  Reducer red{scratch, (int)blockDim.x, 0};
  const T *w = (const T*)p.w, *b = (const T*)p.b, *pw = (const T*)p.pw, *pb = (const T*)p.pb, *gate = (const T*)p.gate;
  const bool two = p.o != nullptr;
  const uint32_t row_bytes = (uint32_t)p.C * sizeof(T);
  const Ring ring{smem_addr(ring_data), smem_addr(ring_bars), row_bytes * (two ? 2 : 1), row_bytes, stages};
  auto ask = [&](long long it) {  // by thread 0
    const long long row = blockIdx.x + it * gridDim.x;
    if (row >= p.rows) return;
    mbar_expect_tx(ring.bar(it), ring.stage_bytes);
    bulk_load(ring.at(it), (const T*)p.x + row * p.C, row_bytes, ring.bar(it));
    if (two) bulk_load(ring.at(it) + row_bytes, (const T*)p.o + row * p.C, row_bytes, ring.bar(it));
  };
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < stages; ++i) mbar_init(ring.bars + i * 8, 1);
    mbar_init_fence();
  }
  __syncthreads();
  if (threadIdx.x == 0)
    for (int i = 0; i < stages; ++i) ask(i);
  bool in[NV];
  int col[NV];
  NA_RUNS(a) {
    col[a] = (threadIdx.x + a * blockDim.x) * VEC;
    in[a] = col[a] < p.C;
  }
  const float inv = 1.f / (float)p.C;
  long long it = 0;
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x, ++it) {
    if (!mbar_wait(ring.bar(it), (uint32_t)(it / stages) & 1, &abort_flag, p.status)) return;
    float y[1][NV][VEC], v[1][NV][VEC], mean[1], rstd[1];
    NA_RUNS(a) {
      NA_PAIRS(i) y[0][a][i] = y[0][a][i + 1] = v[0][a][i] = v[0][a][i + 1] = 0.f;
      if (!in[a]) continue;
      lds_floats<T, VEC>(ring.at(it) + col[a] * sizeof(T), y[0][a]);
      if (two) lds_floats<T, VEC>(ring.at(it) + row_bytes + col[a] * sizeof(T), v[0][a]);
    }
    bool read = false;  // a barrier has shown that the row is in registers
    auto next = [&] {
      if (!read && threadIdx.x == 0) ask(it + stages);
      read = true;
    };
    if (two) {
      float f[NV][VEC];  // what the branch is multiplied by
      NA_RUNS(a) NA_PAIRS(i) f[a][i] = f[a][i + 1] = p.scale;
      if (gate) {
        const T* g = gate + gate_of(p, row) * p.C;
        NA_RUNS(a) if (in[a]) {
          float k[VEC];
          ldg_floats<T, VEC>(g + col[a], k);
          NA_PAIRS(i) mul2(f[a][i], f[a][i + 1], f[a][i], f[a][i + 1], k[i], k[i + 1]);
        }
      }
      if (p.post) {
        wide_stats<1, NV, VEC>(v, in, inv, p.rms, p.eps, red, mean, rstd);
        next();
        NA_RUNS(a) if (in[a]) {
          float k[VEC];
          NA_PAIRS(i) k[i] = k[i + 1] = 1.f;
          if (pw) ldg_floats<T, VEC>(pw + col[a], k);
          NA_PAIRS(i) mul2(k[i], k[i + 1], k[i], k[i + 1], rstd[0], rstd[0]);
          if (pb) {
            float c[VEC];
            ldg_floats<T, VEC>(pb + col[a], c);
            NA_PAIRS(i) fma2(v[0][a][i], v[0][a][i + 1], v[0][a][i], v[0][a][i + 1], k[i], k[i + 1], c[i], c[i + 1]);
          } else {
            NA_PAIRS(i) mul2(v[0][a][i], v[0][a][i + 1], v[0][a][i], v[0][a][i + 1], k[i], k[i + 1]);
          }
        }
      }
      NA_RUNS(a) if (in[a]) {
        NA_PAIRS(i)
        fma2(y[0][a][i], y[0][a][i + 1], f[a][i], f[a][i + 1], v[0][a][i], v[0][a][i + 1], y[0][a][i], y[0][a][i + 1]);
        store_pack<T, VEC>((T*)p.y + row * p.C + col[a], y[0][a]);
      }
    }
    if (p.h) {
      // h is the norm of y before y's rounding to T: one rounding, not two
      wide_stats<1, NV, VEC>(y, in, inv, p.rms, p.eps, red, mean, rstd);
      next();
      NA_RUNS(a) if (in[a]) {
        float k[VEC];
        NA_PAIRS(i) k[i] = k[i + 1] = 1.f;
        if (w) ldg_floats<T, VEC>(w + col[a], k);
        NA_PAIRS(i) mul2(k[i], k[i + 1], k[i], k[i + 1], rstd[0], rstd[0]);
        if (b) {
          float c[VEC];
          ldg_floats<T, VEC>(b + col[a], c);
          NA_PAIRS(i) fma2(y[0][a][i], y[0][a][i + 1], y[0][a][i], y[0][a][i + 1], k[i], k[i + 1], c[i], c[i + 1]);
        } else {
          NA_PAIRS(i) mul2(y[0][a][i], y[0][a][i + 1], y[0][a][i], y[0][a][i + 1], k[i], k[i + 1]);
        }
        store_pack<T, VEC>((T*)p.h + row * p.C + col[a], y[0][a]);
      }
    }
    if (!read) {
      __syncthreads();
      next();
    }
  }
}

// The chunks, the sums and their order are those of norm_backward_kernel.  Both
// norms' statistics share their reductions.
template <typename T, int VEC, int NV, bool POST>
__global__ void __launch_bounds__(512, 1) norm_backward_wide_kernel(NormArgs p, int stages) {
  using namespace sm100;
  extern __shared__ __align__(128) uint8_t ring_data[];
  __shared__ float scratch[2][2][32];
  __shared__ uint64_t ring_bars[kMaxStages];
  __shared__ volatile int abort_flag;
  Reducer red{scratch, (int)blockDim.x, 0};
  const T *w = (const T*)p.w, *pw = (const T*)p.pw, *pb = (const T*)p.pb, *gate = (const T*)p.gate;
  const bool has_h = p.dh != nullptr, has_y = p.dy != nullptr, has_o = p.o != nullptr;
  const uint32_t row_bytes = (uint32_t)p.C * sizeof(T);
  // a stage: y, dh (both with dh), dy, o
  const uint32_t dy_off = has_h ? 2 * row_bytes : 0, o_off = dy_off + (has_y ? row_bytes : 0);
  const Ring ring{smem_addr(ring_data), smem_addr(ring_bars), o_off + (has_o ? row_bytes : 0), row_bytes, stages};
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
  auto ask = [&](long long it) {  // by thread 0
    const long long row = r0 + it;
    if (row >= r1) return;
    const uint32_t at = ring.at(it), bar = ring.bar(it);
    mbar_expect_tx(bar, ring.stage_bytes);
    if (has_h) {
      bulk_load(at, (const T*)p.x + row * p.C, row_bytes, bar);
      bulk_load(at + row_bytes, (const T*)p.dh + row * p.C, row_bytes, bar);
    }
    if (has_y) bulk_load(at + dy_off, (const T*)p.dy + row * p.C, row_bytes, bar);
    if (has_o) bulk_load(at + o_off, (const T*)p.o + row * p.C, row_bytes, bar);
  };
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < stages; ++i) mbar_init(ring.bars + i * 8, 1);
    mbar_init_fence();
  }
  __syncthreads();
  if (threadIdx.x == 0)
    for (int i = 0; i < stages; ++i) ask(i);
  bool in[NV];
  int col[NV];
  NA_RUNS(a) {
    col[a] = (threadIdx.x + a * blockDim.x) * VEC;
    in[a] = col[a] < p.C;
  }
  const float inv = 1.f / (float)p.C;
  float aw[NV][VEC] = {}, ab[NV][VEC] = {}, apw[NV][VEC] = {}, apb[NV][VEC] = {}, ag[NV][VEC] = {};
  long long gate_row = r0 < r1 ? gate_of(p, r0) : 0, gate_end = (gate_row + 1) * p.gate_rows;
  long long it = 0;
  for (long long row = r0; row < r1; ++row, ++it) {
    if (!mbar_wait(ring.bar(it), (uint32_t)(it / stages) & 1, &abort_flag, p.status)) return;
    const uint32_t from = ring.at(it);
    const long long at = row * p.C;
    float n[2][NV][VEC], dx[NV][VEC], t[NV][VEC], mean[2], rstd[2];  // n: of y, and of o
    NA_RUNS(a) {
      NA_PAIRS(i) {
        n[0][a][i] = n[0][a][i + 1] = n[1][a][i] = n[1][a][i + 1] = 0.f;
        dx[a][i] = dx[a][i + 1] = t[a][i] = t[a][i + 1] = 0.f;
      }
      if (!in[a]) continue;
      const uint32_t c = from + col[a] * sizeof(T);
      if (has_h) {
        lds_floats<T, VEC>(c, n[0][a]);
        lds_floats<T, VEC>(c + row_bytes, t[a]);
      }
      if (has_y) lds_floats<T, VEC>(c + dy_off, dx[a]);
      if (has_o) lds_floats<T, VEC>(c + o_off, n[1][a]);
    }
    if (!POST && !has_h) __syncthreads();
    if constexpr (POST) {
      wide_stats<2, NV, VEC>(n, in, inv, p.rms, p.eps, red, mean, rstd);
    } else if (has_h) {
      float one[1][NV][VEC], m1[1], r1v[1];
      NA_RUNS(a) NA_PAIRS(i) one[0][a][i] = n[0][a][i], one[0][a][i + 1] = n[0][a][i + 1];
      wide_stats<1, NV, VEC>(one, in, inv, p.rms, p.eps, red, m1, r1v);
      NA_RUNS(a) NA_PAIRS(i) n[0][a][i] = one[0][a][i], n[0][a][i + 1] = one[0][a][i + 1];
      rstd[0] = r1v[0];
    }
    if (threadIdx.x == 0) ask(it + stages);  // all threads have read this row
    if (has_h) {
      float s[2], s0 = 0.f, s1 = 0.f, q0 = 0.f, q1 = 0.f;
      NA_RUNS(a) if (in[a]) {
        float k[VEC];
        NA_PAIRS(i) k[i] = k[i + 1] = 1.f;
        if (w) ldg_floats<T, VEC>(w + col[a], k);
        NA_PAIRS(i) {
          float &x0 = n[0][a][i], &x1 = n[0][a][i + 1], &g0 = t[a][i], &g1 = t[a][i + 1];
          mul2(x0, x1, x0, x1, rstd[0], rstd[0]);
          fma2(aw[a][i], aw[a][i + 1], g0, g1, x0, x1, aw[a][i], aw[a][i + 1]);
          add2(ab[a][i], ab[a][i + 1], ab[a][i], ab[a][i + 1], g0, g1);
          mul2(g0, g1, g0, g1, k[i], k[i + 1]);
          add2(s0, s1, s0, s1, g0, g1);
          fma2(q0, q1, g0, g1, x0, x1, q0, q1);
        }
      }
      s[0] = s0 + s1;
      s[1] = q0 + q1;
      red.sum<true>(s);
      const float m0 = p.rms ? 0.f : -s[0] * inv, m1 = -s[1] * inv;
      NA_RUNS(a) if (in[a]) NA_PAIRS(i) {
        float u0, u1;
        fma2(u0, u1, n[0][a][i], n[0][a][i + 1], m1, m1, m0, m0);
        add2(u0, u1, t[a][i], t[a][i + 1], u0, u1);
        fma2(dx[a][i], dx[a][i + 1], u0, u1, rstd[0], rstd[0], dx[a][i], dx[a][i + 1]);
      }
    }
    NA_RUNS(a) if (in[a]) store_pack<T, VEC>((T*)p.dx + at + col[a], dx[a]);
    if (has_o) {
      float s0 = 0.f, s1 = 0.f, q0 = 0.f, q1 = 0.f;
      // dx becomes dP . pw, the gradient of the post norm's normalised row
      NA_RUNS(a) if (in[a]) {
        float kg[VEC], kw[VEC], kb[VEC];
        NA_PAIRS(i) kg[i] = kg[i + 1] = kw[i] = kw[i + 1] = 1.f, kb[i] = kb[i + 1] = 0.f;
        if (gate) ldg_floats<T, VEC>(gate + gate_row * p.C + col[a], kg);
        if (POST && pw) ldg_floats<T, VEC>(pw + col[a], kw);
        if (POST && pb) ldg_floats<T, VEC>(pb + col[a], kb);
        float gp[VEC];
        NA_PAIRS(i) {
          float &m0 = n[1][a][i], &m1 = n[1][a][i + 1], &d0 = dx[a][i], &d1 = dx[a][i + 1], v0 = m0, v1 = m1;
          if constexpr (POST) {
            mul2(m0, m1, m0, m1, rstd[1], rstd[1]);
            fma2(v0, v1, m0, m1, kw[i], kw[i + 1], kb[i], kb[i + 1]);
          }
          mul2(d0, d1, d0, d1, p.scale, p.scale);
          mul2(gp[i], gp[i + 1], d0, d1, v0, v1);
          add2(ag[a][i], ag[a][i + 1], ag[a][i], ag[a][i + 1], gp[i], gp[i + 1]);
          mul2(d0, d1, d0, d1, kg[i], kg[i + 1]);
          if constexpr (POST) {
            fma2(apw[a][i], apw[a][i + 1], d0, d1, m0, m1, apw[a][i], apw[a][i + 1]);
            add2(apb[a][i], apb[a][i + 1], apb[a][i], apb[a][i + 1], d0, d1);
            mul2(d0, d1, d0, d1, kw[i], kw[i + 1]);
            add2(s0, s1, s0, s1, d0, d1);
            fma2(q0, q1, d0, d1, m0, m1, q0, q1);
          }
        }
        if (p.gate_rows == 1 && p.dgate)
#pragma unroll
          for (int i = 0; i < VEC; ++i) p.dgate[at + col[a] + i] = gp[i];
      }
      if constexpr (POST) {
        float s[2] = {s0 + s1, q0 + q1};
        red.sum<true>(s);
        const float m0 = p.rms ? 0.f : -s[0] * inv, m1 = -s[1] * inv;
        NA_RUNS(a) if (in[a]) NA_PAIRS(i) {
          float u0, u1;
          fma2(u0, u1, n[1][a][i], n[1][a][i + 1], m1, m1, m0, m0);
          add2(u0, u1, dx[a][i], dx[a][i + 1], u0, u1);
          mul2(dx[a][i], dx[a][i + 1], u0, u1, rstd[1], rstd[1]);
        }
      }
      NA_RUNS(a) if (in[a]) store_pack<T, VEC>((T*)p.dout + at + col[a], dx[a]);
    }
    if (row + 1 == gate_end || row + 1 == r1) {
      if (p.pieces == 0 && p.dgate && p.gate_rows > 1)
        flush<VEC, NV, true>(ag, p.dgate + gate_row * p.C, col, in, 0, p.C, nullptr);
      ++gate_row;
      gate_end += p.gate_rows;
    }
  }
  float* part = p.partial + chunk * p.C;
  const long long step = p.chunks * (long long)p.C;
  if (p.dw) flush<VEC, NV, true>(aw, part + kSumW * step, col, in, 0, p.C, nullptr);
  if (p.db) flush<VEC, NV, true>(ab, part + kSumB * step, col, in, 0, p.C, nullptr);
  if constexpr (POST) {
    if (p.dpw) flush<VEC, NV, true>(apw, part + kSumPW * step, col, in, 0, p.C, nullptr);
    if (p.dpb) flush<VEC, NV, true>(apb, part + kSumPB * step, col, in, 0, p.C, nullptr);
  }
  if (p.pieces > 0 && p.dgate) flush<VEC, NV, true>(ag, part + kSumG * step, col, in, 0, p.C, nullptr);
}
#undef NA_PAIRS
#undef NA_RUNS

// Stages of a ring: what is left of the SM's shared memory for each of its
// blocks, kMaxStages at most and 1 at least.
int ring_stages(size_t stage_bytes, int blocks_per_sm) {
  const size_t budget = (size_t)(216 / blocks_per_sm) * 1024;
  size_t n = budget / stage_bytes;
  return n > kMaxStages ? kMaxStages : n < 1 ? 1 : (int)n;
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

// How a row is held: lanes <= 32 of a warp with nv vectors each (block = 0), or
// a block, `block` vectors in all.
struct Plan {
  int lanes, block, nv;
};
Plan plan_for(int C, int vec, int max_warp_nv) {
  const int n = (C + vec - 1) / vec;
  if (n <= 32) return {pow2_at_least(n), 0, 1};
  for (int nv = 2; nv <= max_warp_nv; nv *= 2)
    if (n <= 32 * nv) return {32, 0, nv};
  return {0, n, 0};
}
int block_of(int vectors, int nv) { return ((vectors + nv - 1) / nv + 31) / 32 * 32; }

template <typename T, int VEC, int NV, bool BLOCK>
cudaError_t forward_one(const NormArgs& p, int lanes, int block, cudaStream_t st) {
  const int threads = BLOCK ? block : 256;
  const long long per_block = BLOCK ? 1 : 256 / lanes;
  const long long need = (p.rows + per_block - 1) / per_block;
  int resident = 1;
  cudaError_t e =
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident, norm_forward_kernel<T, VEC, NV, BLOCK>, threads, 0);
  if (e != cudaSuccess) return e;
  const long long most = (long long)sms() * (resident > 0 ? resident : 1);
  norm_forward_kernel<T, VEC, NV, BLOCK><<<(unsigned)(need < most ? need : most), threads, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T, int VEC, int NV, int THREADS>
cudaError_t forward_wide(const NormArgs& p, int block, cudaStream_t st) {
  auto kern = norm_forward_wide_kernel<T, VEC, NV, THREADS>;
  const int per_sm = THREADS == 256 ? (block <= 128 ? 6 : 3) : 1;  // as many as registers leave room for
  const size_t stage = (size_t)p.C * sizeof(T) * (p.o ? 2 : 1);
  const int stages = ring_stages(stage, per_sm);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 216 * 1024);
  if (e != cudaSuccess) return e;
  const long long most = (long long)sms() * per_sm;
  kern<<<(unsigned)(p.rows < most ? p.rows : most), block, stage * stages, st>>>(p, stages);
  return cudaGetLastError();
}

template <typename T, int VEC> cudaError_t forward_vec(NormArgs p, cudaStream_t st) {
  const Plan pl = plan_for(p.C, VEC, 4);
  p.lanes = pl.lanes;
  if (pl.block) {
    // 16 columns a thread: each warp's share of reductions and addresses is
    // most of its instructions with 8, and registers spill with 32
    if constexpr (VEC * sizeof(T) == 16)  // rows that bulk copies can take
    {
      const int block = block_of(pl.block, 16 / VEC);
      return block <= 256 ? forward_wide<T, VEC, 16 / VEC, 256>(p, block, st)
                          : forward_wide<T, VEC, 16 / VEC, 512>(p, block, st);
    }
    else
      return forward_one<T, VEC, 8 / VEC, true>(p, 0, block_of(pl.block, 8 / VEC), st);
  }
  if (pl.nv == 1) return forward_one<T, VEC, 1, false>(p, pl.lanes, 0, st);
  if (pl.nv == 2) return forward_one<T, VEC, 2, false>(p, pl.lanes, 0, st);
  return forward_one<T, VEC, 4, false>(p, pl.lanes, 0, st);
}

template <typename T> cudaError_t forward_t(const NormArgs& p, cudaStream_t st) {
  constexpr int kVec = 16 / sizeof(T);
  if (p.C % kVec == 0) return forward_vec<T, kVec>(p, st);
  return p.C % 4 == 0 ? forward_vec<T, 4>(p, st) : forward_vec<T, 1>(p, st);
}

// The backward pass's chunks: as many as blocks run at once, but not under 8
// rows.  Registers leave room for 512 threads an SM; a block has 256, or what a
// wide row takes.  148 SMs, also on a device with other counts: the sums' order
// is fixed by it.
struct Chunks {
  long long count, rows;
  int pieces;
};
int vec_for(int C, na_dtype dt) {
  if (dt != NA_F32 && C % 8 == 0) return 8;
  return C % 4 == 0 ? 4 : 1;
}
Chunks chunks_for(long long rows, long long gate_rows, int C, na_dtype dt) {
  const int vec = vec_for(C, dt), vectors = (C + vec - 1) / vec;
  const int threads = vectors <= (vec == 8 ? 32 : 64) ? 256 : vec == 1 ? vectors / 8 : vectors;
  const long long blocks = 148ll * (threads > 256 ? 1 : threads > 128 ? 2 : 4), gates = rows / gate_rows;
  long long r = (rows + blocks - 1) / blocks;
  if (r < 8) r = 8;
  if (gate_rows >= r) {
    long long pieces = blocks / gates;  // not one block more than run at once
    if (pieces > (gate_rows + 7) / 8) pieces = (gate_rows + 7) / 8;
    if (pieces < 1) pieces = 1;
    const long long per = (gate_rows + pieces - 1) / pieces;
    pieces = (gate_rows + per - 1) / per;
    return {gates * pieces, per, (int)pieces};
  }
  const long long per = r / gate_rows * gate_rows;
  return {(rows + per - 1) / per, per, 0};
}

template <typename T, int VEC, int NV, bool BLOCK, bool POST>
cudaError_t backward_one(const NormArgs& p, int block, cudaStream_t st) {
  const size_t smem = BLOCK ? 0 : sizeof(float) * 256 * NV * VEC;
  norm_backward_kernel<T, VEC, NV, BLOCK, POST><<<(unsigned)p.chunks, BLOCK ? block : 256, smem, st>>>(p);
  return cudaGetLastError();
}
template <typename T, int VEC, int NV, bool BLOCK>
cudaError_t backward_post(const NormArgs& p, int block, cudaStream_t st) {
  return p.post ? backward_one<T, VEC, NV, BLOCK, true>(p, block, st)
                : backward_one<T, VEC, NV, BLOCK, false>(p, block, st);
}
template <typename T, int VEC, int NV, bool POST>
cudaError_t backward_wide(const NormArgs& p, int block, cudaStream_t st) {
  auto kern = norm_backward_wide_kernel<T, VEC, NV, POST>;
  const size_t stage = (size_t)p.C * sizeof(T) * ((p.dh ? 2 : 0) + (p.dy ? 1 : 0) + (p.o ? 1 : 0));
  const int stages = ring_stages(stage, block > 256 ? 1 : block > 128 ? 2 : 4);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 216 * 1024);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)p.chunks, block, stage * stages, st>>>(p, stages);
  return cudaGetLastError();
}

template <typename T, int VEC> cudaError_t backward_vec(NormArgs p, cudaStream_t st) {
  constexpr int kWarpNV = VEC == 8 ? 1 : 2;
  const Plan pl = plan_for(p.C, VEC, kWarpNV);
  p.lanes = pl.lanes;
  if (pl.block) {  // as few vectors a thread as blocks of 512 allow
    constexpr int kOne = VEC == 1 ? 8 : 1;
    const int one = block_of(pl.block, kOne), two = block_of(pl.block, 2 * kOne), four = block_of(pl.block, 4);
    if constexpr (VEC * sizeof(T) == 16) {  // rows that bulk copies can take
      if (one <= 512)
        return p.post ? backward_wide<T, VEC, 1, true>(p, one, st) : backward_wide<T, VEC, 1, false>(p, one, st);
      if (VEC == 8 || two <= 512)
        return p.post ? backward_wide<T, VEC, 2, true>(p, two, st) : backward_wide<T, VEC, 2, false>(p, two, st);
      if constexpr (VEC == 4)
        return p.post ? backward_wide<T, VEC, 4, true>(p, four, st) : backward_wide<T, VEC, 4, false>(p, four, st);
    } else {
      if (one <= 512) return backward_post<T, VEC, kOne, true>(p, one, st);
      if (VEC == 1 || two <= 512) return backward_post<T, VEC, 2 * kOne, true>(p, two, st);
      if constexpr (VEC == 4) return backward_post<T, VEC, 4, true>(p, four, st);
    }
  }
  if (pl.nv == 1) return backward_post<T, VEC, 1, false>(p, 0, st);
  if constexpr (kWarpNV == 2) return backward_post<T, VEC, 2, false>(p, 0, st);
  return cudaErrorInvalidValue;
}
template <typename T> cudaError_t backward_t(const NormArgs& p, cudaStream_t st) {
  constexpr int kVec = 16 / sizeof(T);
  if (p.C % kVec == 0) return backward_vec<T, kVec>(p, st);
  return p.C % 4 == 0 ? backward_vec<T, 4>(p, st) : backward_vec<T, 1>(p, st);
}

}  // namespace

size_t norm_workspace_bytes(long long rows, int C, long long gate_rows, na_dtype dt) {
  return (size_t)chunks_for(rows, gate_rows, C, dt).count * (size_t)C * kSums * sizeof(float);
}

cudaError_t launch_norm_forward(const NormArgs& p, na_dtype dt, cudaStream_t st) {
  if (dt == NA_F32) return forward_t<float>(p, st);
  if (dt == NA_F16) return forward_t<__half>(p, st);
  return forward_t<__nv_bfloat16>(p, st);
}

cudaError_t launch_norm_backward(NormArgs p, na_dtype dt, cudaStream_t st) {
  const Chunks c = chunks_for(p.rows, p.gate_rows, p.C, dt);
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
