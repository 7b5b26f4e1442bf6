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
// dh, dx and do once each.  HBM would bound both (82 us and 61 us at 16387 and
// 8168 rows of 4096, bf16, both norms and a gate); what they take, 104 and 151
// us, goes to instruction issue and to the waits of the reductions between a
// row's steps.  So arithmetic is in pairs (two float32 an instruction), weights
// stay in registers, rows that fill their threads have kernels without a
// question about columns, and reductions are few.  Rows of up to 32 lanes'
// worth of channels are held by a part of a warp, wider ones by a whole block.
//
// Statistics are float32.  Forward: the mean first, then the mean square of the
// deviations from it, which is exact to rounding whatever the mean is, as "sum
// of squares minus squared sum" is not.  Backward: sums over differences from a
// few of the row's own values, see backward_row.
#include <atomic>
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
// ----------------------------------------------------------- reductions
// Sums over the lanes of a row: a power of two of them within a warp, or
// (BLOCK) all threads of a block of 512 at most.  In a block the values of a
// warp are summed by halves - each step a lane keeps the half of the values
// that its bit names - which for 8 values takes 9 shuffles where a butterfly
// takes 40; then one 16-byte load a lane reads all warps' sums.  `slot`
// alternates between two areas of shared memory, so that one barrier a
// reduction is enough.
//
// All lanes of a warp, or all threads of a block, call sum() together, also for
// rows that are not theirs to write: several rows share a warp, and a sum that
// only some rows take would shuffle with lanes that are not there.
constexpr int kMaxWarps = 16, kMaxSums = 8;

struct Reducer {
  float (*scratch)[kMaxSums * kMaxWarps];  // [2]; those of absent warps stay 0
  int lanes, slot;

  // zeroes the areas; the caller's next barrier is before their first use
  NA_DEVICE void init() {
    for (int i = threadIdx.x; i < 2 * kMaxSums * kMaxWarps; i += blockDim.x) (&scratch[0][0])[i] = 0.f;
  }
  template <bool BLOCK, int K> NA_DEVICE void sum(float (&v)[K]) {
    if constexpr (!BLOCK) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1)
        if (o < lanes)
#pragma unroll
          for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    } else {
      constexpr int P = K > 4 ? 8 : K > 2 ? 4 : K;  // a power of two
      const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
      float part[P];
#pragma unroll
      for (int k = 0; k < P; ++k) part[k] = k < K ? v[k] : 0.f;
      int held = 0;  // which of the P sums this lane ends up with
#pragma unroll
      for (int n = P / 2, o = 16; o > 0; o >>= 1, n /= 2) {
        if (n > 0) {
          const bool upper = lane & o;
#pragma unroll
          for (int k = 0; k < n; ++k) {
            const float keep = upper ? part[k + n] : part[k], send = upper ? part[k] : part[k + n];
            part[k] = keep + __shfl_xor_sync(0xffffffffu, send, o);
          }
          held = held * 2 + upper;
        } else {
          part[0] += __shfl_xor_sync(0xffffffffu, part[0], o);
        }
      }
      if ((lane & (32 / P - 1)) == 0) scratch[slot][held * kMaxWarps + warp] = part[0];
      __syncthreads();
      const float4 four = *reinterpret_cast<const float4*>(scratch[slot] + lane * 4);
      float s = (four.x + four.y) + (four.z + four.w);
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] = __shfl_sync(0xffffffffu, s, 4 * k);
      slot ^= 1;
    }
  }
};

// ---------------------------------------------------------- runs of VEC values
// Elementwise on VEC values, two an instruction where there are two: these lie
// in 64-bit registers throughout, as packing pairs for each instruction took as
// many moves as there is arithmetic.  A scalar operand is given as one float.
NA_DEVICE uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
NA_DEVICE float2 halves(uint64_t p) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
  return r;
}
template <int VEC> struct Run {
  uint64_t v[VEC / 2];
  NA_DEVICE float operator[](int i) const { return i & 1 ? halves(v[i / 2]).y : halves(v[i / 2]).x; }
};
template <> struct Run<1> {
  float v;
  NA_DEVICE float operator[](int) const { return v; }
};
template <int VEC> constexpr bool kScalar = VEC == 1;
NA_DEVICE float one_of(float s, int) { return s; }
NA_DEVICE float one_of(const Run<1>& r, int) { return r.v; }
NA_DEVICE uint64_t two_of(float s, int) { return pair(s, s); }
template <int VEC> NA_DEVICE uint64_t two_of(const Run<VEC>& r, int i) { return r.v[i]; }

template <int VEC, typename A, typename B> NA_DEVICE void add(Run<VEC>& d, const A& a, const B& b) {
  if constexpr (kScalar<VEC>)
    d.v = one_of(a, 0) + one_of(b, 0);
  else
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i)
      asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v[i]) : "l"(two_of(a, i)), "l"(two_of(b, i)));
}
template <int VEC, typename A, typename B> NA_DEVICE void mul(Run<VEC>& d, const A& a, const B& b) {
  if constexpr (kScalar<VEC>)
    d.v = one_of(a, 0) * one_of(b, 0);
  else
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i)
      asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v[i]) : "l"(two_of(a, i)), "l"(two_of(b, i)));
}
template <int VEC, typename A, typename B, typename C>
NA_DEVICE void fma(Run<VEC>& d, const A& a, const B& b, const C& c) {
  if constexpr (kScalar<VEC>)
    d.v = fmaf(one_of(a, 0), one_of(b, 0), one_of(c, 0));
  else
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i)
      asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v[i]) : "l"(two_of(a, i)), "l"(two_of(b, i)), "l"(two_of(c, i)));
}
template <int VEC> NA_DEVICE void set(Run<VEC>& d, float s) {
  if constexpr (kScalar<VEC>)
    d.v = s;
  else
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) d.v[i] = pair(s, s);
}
template <int VEC> NA_DEVICE float total(const Run<VEC>& r) {
  if constexpr (kScalar<VEC>) {
    return r.v;
  } else {
    uint64_t s = r.v[0];
#pragma unroll
    for (int i = 1; i < VEC / 2; ++i) asm("add.rn.f32x2 %0, %1, %2;" : "=l"(s) : "l"(s), "l"(r.v[i]));
    const float2 h = halves(s);
    return h.x + h.y;
  }
}
template <typename T, int VEC> NA_DEVICE void unpack(Run<VEC>& d, const Pack<T, VEC>& p) {
  if constexpr (kScalar<VEC>) {
    d.v = to_f<T>(p.e[0]);
  } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(&p);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) d.v[i] = pair(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
  } else {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) d.v[i] = pair(to_f<T>(p.e[2 * i]), to_f<T>(p.e[2 * i + 1]));
  }
}
template <typename T, int VEC> NA_DEVICE void read(Run<VEC>& d, const T* p) { unpack<T, VEC>(d, load_pack<T, VEC>(p)); }
template <typename T, int VEC> NA_DEVICE void write(T* p, const Run<VEC>& r) {
  Pack<T, VEC> out;
  if constexpr (kScalar<VEC>) {
    out.e[0] = from_f<T>(r.v);
  } else {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      const float2 h = halves(r.v[i]);
      if constexpr (std::is_same_v<T, float>)
        out.e[2 * i] = h.x, out.e[2 * i + 1] = h.y;
      else if constexpr (std::is_same_v<T, __half>)
        reinterpret_cast<__half2*>(&out)[i] = __floats2half2_rn(h.x, h.y);
      else
        reinterpret_cast<__nv_bfloat162*>(&out)[i] = __floats2bfloat162_rn(h.x, h.y);
    }
  }
  *reinterpret_cast<Pack<T, VEC>*>(p) = out;
}

// What a thread holds of a row: NV runs, at the columns col, those past the
// row's end not `in`.  Their values are kept at 0 by factors and shifts of 0
// (own), and their columns are the row's last, so that only a row's loads and
// stores ask; a branch around each run's arithmetic cost a fifth to a third of
// the time.  FULL: there are none.
template <int NV> struct Place {
  int col[NV];
  bool in[NV];
  float inv;  // 1 / channels
  NA_DEVICE float own(int a, float s) const { return in[a] ? s : 0.f; }
};
template <int VEC, int NV, bool FULL> NA_DEVICE Place<NV> place_of(int lane, int lanes, int C) {
  Place<NV> r;
#pragma unroll
  for (int a = 0; a < NV; ++a) {
    r.col[a] = (lane + a * lanes) * VEC;
    r.in[a] = FULL || r.col[a] < C;
    if (!r.in[a]) r.col[a] = C - VEC;
  }
  r.inv = 1.f / (float)C;
  return r;
}

#define NA_RUNS(a) _Pragma("unroll") for (int a = 0; a < NV; ++a)

// A vector over the channels (a weight, a bias, a gate's row) at a thread's
// columns.  HELD keeps them in registers, as read, from row to row: read again
// for every row they are three to five more loads from L2, one after the other
// between the reductions, which cost wide rows a third of their time.
template <typename T, int VEC, int NV, bool HELD> struct Channels {
  const T* g;
  Pack<T, VEC> held[HELD ? NV : 1];

  NA_DEVICE void point(const T* from, const Place<NV>& at) {
    g = from;
    if constexpr (HELD)
      if (g) NA_RUNS(a) held[a] = load_pack<T, VEC>(g + at.col[a]);
  }
  NA_DEVICE bool given() const { return g != nullptr; }
  NA_DEVICE void get(Run<VEC>& d, int a, const Place<NV>& at) const {
    if constexpr (HELD)
      unpack<T>(d, held[a]);
    else
      read<T>(d, g + at.col[a]);
  }
};
// 16 bits: 4 registers for 8 channels.  float32 would take as many as the rows.
template <typename T, int VEC, int NV, int MOST> constexpr bool hold() { return sizeof(T) == 2 && VEC * NV <= MOST; }

// Takes its mean off the row v (not for an RMS norm) and finds its reciprocal
// deviation.  Values past the row's end are 0 and stay so.
template <bool BLOCK, int NV, int VEC>
NA_DEVICE float centre(Run<VEC> (&v)[NV], const Place<NV>& at, bool rms, float eps, Reducer& red) {
  float s[1];
  Run<VEC> sum;
  if (!rms) {
    sum = v[0];
#pragma unroll
    for (int a = 1; a < NV; ++a) add(sum, sum, v[a]);
    s[0] = total(sum);
    red.sum<BLOCK>(s);
    NA_RUNS(a) add(v[a], v[a], at.own(a, -s[0] * at.inv));
  }
  mul(sum, v[0], v[0]);
#pragma unroll
  for (int a = 1; a < NV; ++a) fma(sum, v[a], v[a], sum);
  s[0] = total(sum);
  red.sum<BLOCK>(s);
  return rsqrtf(s[0] * at.inv + eps);
}

// ----------------------------------------------------------------- forward
template <typename T, int VEC, int NV, bool kHeld> struct ForwardVectors {
  Channels<T, VEC, NV, kHeld> w, b, pw, pb, gate;
  long long gate_row = -1;

  NA_DEVICE ForwardVectors(const NormArgs& p, const Place<NV>& at) {
    w.point((const T*)p.w, at);
    b.point((const T*)p.b, at);
    pw.point((const T*)p.pw, at);
    pb.point((const T*)p.pb, at);
    gate.point(nullptr, at);
  }
  NA_DEVICE void at_row(const NormArgs& p, const Place<NV>& at, long long row) {
    if (!p.gate) return;
    const long long r = gate_of(p, row);
    if (r == gate_row) return;
    gate_row = r;
    gate.point((const T*)p.gate + r * p.C, at);
  }
};

// One row: y holds x, v holds o.  `taken` is called after the first barrier of a
// block that follows the row's reading (by then all its threads have read it).
template <typename T, bool BLOCK, int VEC, int NV, bool HELD, typename F>
NA_DEVICE void forward_row(const NormArgs& p, Run<VEC> (&y)[NV], Run<VEC> (&v)[NV], long long row, bool live,
                           const Place<NV>& at, ForwardVectors<T, VEC, NV, HELD>& c, Reducer& red, F taken) {
  const long long off = row * p.C;
  bool met = false;
  // v - its mean, times rstd w, + b
  auto scaled = [&](Run<VEC>& d, int a, float rstd, const auto& w, const auto& b) {
    Run<VEC> k;
    if (w.given()) {
      w.get(k, a, at);
      mul(k, k, rstd);
    } else {
      set(k, rstd);
    }
    if (b.given()) {
      Run<VEC> plus;
      b.get(plus, a, at);
      fma(d, d, k, plus);
    } else {
      mul(d, d, k);
    }
  };
  if (p.o) {
    c.at_row(p, at, row);
    if (p.post) {
      const float rstd = centre<BLOCK>(v, at, p.rms, p.eps, red);
      taken();
      met = true;
      NA_RUNS(a) scaled(v[a], a, rstd, c.pw, c.pb);
    }
    NA_RUNS(a) {
      if (c.gate.given()) {
        Run<VEC> k;
        c.gate.get(k, a, at);
        mul(v[a], v[a], k);
      }
      fma(y[a], v[a], at.own(a, p.scale), y[a]);
      if (live && at.in[a]) write<T>((T*)p.y + off + at.col[a], y[a]);
    }
  }
  if (p.h) {
    // h is the norm of y before y's rounding to T: one rounding, not two
    const float rstd = centre<BLOCK>(y, at, p.rms, p.eps, red);
    if (!met) taken();
    met = true;
    NA_RUNS(a) {
      scaled(y[a], a, rstd, c.w, c.b);
      if (live && at.in[a]) write<T>((T*)p.h + off + at.col[a], y[a]);
    }
  }
  if (!met) {
    if constexpr (BLOCK) __syncthreads();
    taken();
  }
}

// Rows straight from memory, asked for one ahead: while a row goes through its
// reductions, the loads of the next are in flight.
template <typename T, int VEC, int NV, bool BLOCK, bool FULL>
__global__ void __launch_bounds__(BLOCK ? 512 : 256, 1) norm_forward_kernel(NormArgs p) {
  __shared__ __align__(16) float scratch[2][kMaxSums * kMaxWarps];
  Reducer red{scratch, BLOCK ? (int)blockDim.x : p.lanes, 0};
  if constexpr (BLOCK) {
    red.init();
    __syncthreads();
  }
  const int lane = BLOCK ? threadIdx.x : threadIdx.x & (p.lanes - 1);
  const int per_block = BLOCK ? 1 : blockDim.x / p.lanes;
  const int sub = BLOCK ? 0 : threadIdx.x / p.lanes;
  const T *x = (const T*)p.x, *o = (const T*)p.o;
  const Place<NV> at = place_of<VEC, NV, FULL>(lane, red.lanes, p.C);
  ForwardVectors<T, VEC, NV, hold<T, VEC, NV, 8>()> c(p, at);
  Pack<T, VEC> px[NV], po[NV];
  auto ask = [&](long long base) {
    const long long off = min(base + sub, p.rows - 1) * p.C;
    NA_RUNS(a) if (at.in[a]) px[a] = load_row<T, VEC>(x + off + at.col[a]);
    if (o) NA_RUNS(a) if (at.in[a]) po[a] = load_row<T, VEC>(o + off + at.col[a]);
  };
  const long long step = (long long)gridDim.x * per_block;
  long long base = (long long)blockIdx.x * per_block;
  if (base < p.rows) ask(base);
  // all lanes of a warp keep the same trip count: shuffles need them all
  for (; base < p.rows; base += step) {
    const bool live = base + sub < p.rows;
    Run<VEC> y[NV], v[NV];
    NA_RUNS(a) {
      set(y[a], 0.f);
      set(v[a], 0.f);
      if (at.in[a]) unpack<T>(y[a], px[a]);
      if (at.in[a] && o) unpack<T>(v[a], po[a]);
    }
    if (base + step < p.rows) ask(base + step);
    forward_row<T, BLOCK>(p, y, v, live ? base + sub : p.rows - 1, live, at, c, red, [] {});
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
NA_DEVICE void flush(Run<VEC> (&acc)[NV], float* to, const Place<NV>& at, int lanes, int C, float* buf) {
  if constexpr (!BLOCK) {
    const int nsub = blockDim.x / lanes;
    const int lane = threadIdx.x & (lanes - 1), sub = threadIdx.x / lanes;
    const int padded = lanes * NV * VEC;
    __syncthreads();
    NA_RUNS(a)
#pragma unroll
    for (int i = 0; i < VEC; ++i) buf[sub * padded + (lane + a * lanes) * VEC + i] = acc[a][i];
    __syncthreads();
    for (int c = threadIdx.x; c < C; c += blockDim.x) {
      float s = 0.f;
      for (int u = 0; u < nsub; ++u) s += buf[u * padded + c];
      to[c] = s;
    }
  } else {
    NA_RUNS(a) if (at.in[a])
#pragma unroll
    for (int i = 0; i < VEC; ++i) to[at.col[a] + i] = acc[a][i];
  }
  NA_RUNS(a) set(acc[a], 0.f);
}

template <int NV, int VEC> struct Sums {
  Run<VEC> w[NV], b[NV], pw[NV], pb[NV], g[NV];
  NA_DEVICE Sums() {
    NA_RUNS(a) {
      set(w[a], 0.f);
      set(b[a], 0.f);
      set(pw[a], 0.f);
      set(pb[a], 0.f);
      set(g[a], 0.f);
    }
  }
};

template <typename T, int VEC, int NV, bool ONE, bool kHeld> struct BackwardVectors {
  Channels<T, VEC, NV, kHeld> w, pw, gate;
  Channels<T, VEC, NV, kHeld && !ONE> pb;  // ONE: read by flush_chunk alone

  NA_DEVICE BackwardVectors(const NormArgs& p, const Place<NV>& at) {
    w.point((const T*)p.w, at);
    pw.point((const T*)p.pw, at);
    pb.point((const T*)p.pb, at);
    gate.point(nullptr, at);
  }
  NA_DEVICE void at_gate(const NormArgs& p, const Place<NV>& at, long long gate_row) {
    if (p.gate) gate.point((const T*)p.gate + gate_row * p.C, at);
  }
};

// One row: n holds y and o, t holds dh, dx holds dy; first holds a value each
// near y's and o's means.  Rows that are not live take part in the reductions
// and leave nothing.
//
// All statistics of both norms are sums over differences from `first`, taken in
// one reduction: variance = mean square - squared mean of them.  With `first`
// the mean of m of the row's own C values this loses at most a factor 1 + C / m
// to cancellation, as those m values alone make the variance m / C times their
// mean's squared distance; mostly it loses nothing.  In wide 16-bit rows m is
// 64, so that C = 8192 loses 7 bits of float32 at worst; other rows take the
// mean itself.
//
// ONE (one gate row in all of the block's rows): the gate is a factor of whole
// sums, so that sums.pw and sums.pb gather dx . m and dx (dx . o in sums.pw
// without a post norm), of which flush_chunk makes dpw, dpb and dgate.
template <typename T, bool BLOCK, bool POST, bool ONE, int VEC, int NV, bool HELD, typename F>
NA_DEVICE void backward_row(const NormArgs& p, Run<VEC> (&n)[2][NV], Run<VEC> (&t)[NV], Run<VEC> (&dx)[NV],
                            const float (&first)[2], long long row, bool live, const Place<NV>& at,
                            const BackwardVectors<T, VEC, NV, ONE, HELD>& c, Reducer& red, Sums<NV, VEC>& sums, F taken) {
  const long long off = row * p.C;
  constexpr int K = POST ? 6 : 4;
  Run<VEC> r[6];
#pragma unroll
  for (int k = 0; k < 6; ++k) set(r[k], 0.f);
  if (p.dh) NA_RUNS(a) {
    Run<VEC> u = t[a];
    if (c.w.given()) {
      Run<VEC> k;
      c.w.get(k, a, at);
      mul(u, u, k);
    }
    add(n[0][a], n[0][a], at.own(a, -first[0]));
    add(r[0], r[0], n[0][a]);
    fma(r[1], n[0][a], n[0][a], r[1]);
    add(r[2], r[2], u);
    fma(r[3], u, n[0][a], r[3]);
  }
  if constexpr (POST) NA_RUNS(a) {
    add(n[1][a], n[1][a], at.own(a, -first[1]));
    add(r[4], r[4], n[1][a]);
    fma(r[5], n[1][a], n[1][a], r[5]);
  }
  float s[K];
#pragma unroll
  for (int k = 0; k < K; ++k) s[k] = total(r[k]) * at.inv;
  red.sum<BLOCK>(s);
  taken();
  auto deviation = [&](float mean, float square) {
    const float var = square - mean * mean;
    return rsqrtf((var < 0.f ? 0.f : var) + p.eps);  // NaN stays
  };
  if (p.dh) {
    const float mean = p.rms ? 0.f : s[0], rstd = deviation(mean, s[1]);
    const float m0 = p.rms ? 0.f : s[2], m1 = rstd * (s[3] - mean * s[2]);
    // dx += rstd (u - m0 - n m1), n = (y - mean) rstd
    NA_RUNS(a) {
      fma(n[0][a], n[0][a], rstd, -mean * rstd);
      if (live) {
        fma(sums.w[a], t[a], n[0][a], sums.w[a]);
        add(sums.b[a], sums.b[a], t[a]);
      }
      if (c.w.given()) {
        Run<VEC> k;
        c.w.get(k, a, at);
        mul(t[a], t[a], k);
      }
      fma(n[0][a], n[0][a], -m1, -m0);
      add(n[0][a], t[a], n[0][a]);
      fma(dx[a], n[0][a], at.own(a, rstd), dx[a]);
    }
  }
  if (live) NA_RUNS(a) if (at.in[a]) write<T>((T*)p.dx + off + at.col[a], dx[a]);
  if (!p.o) return;
  float mean = 0.f, rstd = 1.f;
  if constexpr (POST) {
    mean = p.rms ? 0.f : s[4];
    rstd = deviation(mean, s[5]);
  }
  Run<VEC> s0, s1;
  set(s0, 0.f);
  set(s1, 0.f);
  // dx becomes dP . pw, the gradient of the post norm's normalised row
  NA_RUNS(a) {
    Run<VEC> k;
    if constexpr (POST) fma(n[1][a], n[1][a], rstd, -mean * rstd);
    if constexpr (ONE) {
      if (live && (POST || c.gate.given())) {
        fma(sums.pw[a], dx[a], n[1][a], sums.pw[a]);
        if constexpr (POST) add(sums.pb[a], sums.pb[a], dx[a]);
      }
      mul(dx[a], dx[a], p.scale);
      if (c.gate.given()) {
        c.gate.get(k, a, at);
        mul(dx[a], dx[a], k);
      }
    } else {
      Run<VEC> v = n[1][a];
      if constexpr (POST) {
        if (c.pw.given()) {
          c.pw.get(k, a, at);
          mul(v, v, k);
        }
        if (c.pb.given()) {
          c.pb.get(k, a, at);
          add(v, v, k);
        }
      }
      mul(dx[a], dx[a], p.scale);
      mul(v, dx[a], v);
      if (live) {
        add(sums.g[a], sums.g[a], v);
        if (p.gate_rows == 1 && p.dgate && at.in[a])
#pragma unroll
          for (int i = 0; i < VEC; ++i) p.dgate[off + at.col[a] + i] = v[i];
      }
      c.gate.get(k, a, at);
      mul(dx[a], dx[a], k);
      if (POST && live) {
        fma(sums.pw[a], dx[a], n[1][a], sums.pw[a]);
        add(sums.pb[a], sums.pb[a], dx[a]);
      }
    }
    if constexpr (POST) {
      if (c.pw.given()) {
        c.pw.get(k, a, at);
        mul(dx[a], dx[a], k);
      }
      add(s0, s0, dx[a]);
      fma(s1, dx[a], n[1][a], s1);
    }
  }
  if constexpr (POST) {
    float m[2] = {total(s0) * at.inv, total(s1) * at.inv};
    red.sum<BLOCK>(m);
    const float m0 = p.rms ? 0.f : -m[0], m1 = -m[1];
    NA_RUNS(a) {
      fma(n[1][a], n[1][a], m1, m0);
      add(n[1][a], dx[a], n[1][a]);
      mul(dx[a], n[1][a], rstd);
    }
  }
  if (live) NA_RUNS(a) if (at.in[a]) write<T>((T*)p.dout + off + at.col[a], dx[a]);
}

// The rows [r0, r1) of a chunk.
NA_DEVICE void chunk_rows_of(const NormArgs& p, long long chunk, long long* r0, long long* r1) {
  if (p.pieces > 0) {  // a chunk is one of `pieces` parts of a gate row's rows
    const long long g = chunk / p.pieces, piece = chunk % p.pieces;
    *r0 = g * p.gate_rows + piece * p.chunk_rows;
    *r1 = min(*r0 + p.chunk_rows, (g + 1) * p.gate_rows);
  } else {  // a chunk holds whole gate rows
    *r0 = chunk * p.chunk_rows;
    *r1 = min(*r0 + p.chunk_rows, p.rows);
  }
}
template <typename T, bool BLOCK, bool POST, bool ONE, int VEC, int NV, bool HELD>
NA_DEVICE void flush_chunk(const NormArgs& p, Sums<NV, VEC>& s, const Place<NV>& at,
                           const BackwardVectors<T, VEC, NV, ONE, HELD>& c, int lanes, float* buf) {
  float* part = p.partial + (long long)blockIdx.x * p.C;
  const long long step = p.chunks * (long long)p.C;
  if constexpr (ONE) {
    if (p.o) NA_RUNS(a) {
      Run<VEC> k, g;
      Run<VEC>&dm = s.pw[a], &d = s.pb[a];
      mul(dm, dm, p.scale);
      mul(d, d, p.scale);
      g = dm;
      if constexpr (POST) {
        if (c.pw.given()) {
          c.pw.get(k, a, at);
          mul(g, g, k);
        }
        if (c.pb.given()) {
          c.pb.get(k, a, at);
          fma(g, d, k, g);
        }
        if (c.gate.given()) {
          c.gate.get(k, a, at);
          mul(dm, dm, k);
          mul(d, d, k);
        }
      }
      s.g[a] = g;
    }
  }
  if (p.dw) flush<VEC, NV, BLOCK>(s.w, part + kSumW * step, at, lanes, p.C, buf);
  if (p.db) flush<VEC, NV, BLOCK>(s.b, part + kSumB * step, at, lanes, p.C, buf);
  if constexpr (POST) {
    if (p.dpw) flush<VEC, NV, BLOCK>(s.pw, part + kSumPW * step, at, lanes, p.C, buf);
    if (p.dpb) flush<VEC, NV, BLOCK>(s.pb, part + kSumPB * step, at, lanes, p.C, buf);
  }
  if (ONE && p.dgate) flush<VEC, NV, BLOCK>(s.g, part + kSumG * step, at, lanes, p.C, buf);
}

// As in the forward pass, a row's loads are in flight while the one before it
// is worked on.
template <typename T, int VEC, int NV, bool BLOCK, bool POST, bool ONE, bool FULL>
__global__ void __launch_bounds__(BLOCK ? 512 : 256, BLOCK ? 1 : 2) norm_backward_kernel(NormArgs p) {
  __shared__ __align__(16) float scratch[2][kMaxSums * kMaxWarps];
  extern __shared__ float buf[];
  Reducer red{scratch, BLOCK ? (int)blockDim.x : p.lanes, 0};
  if constexpr (BLOCK) {
    red.init();
    __syncthreads();
  }
  const int lane = BLOCK ? threadIdx.x : threadIdx.x & (p.lanes - 1);
  const int per_block = BLOCK ? 1 : blockDim.x / p.lanes;
  const int sub = BLOCK ? 0 : threadIdx.x / p.lanes;
  const T *y = (const T*)p.x, *o = (const T*)p.o, *dy = (const T*)p.dy, *dh = (const T*)p.dh;
  const Place<NV> at = place_of<VEC, NV, FULL>(lane, red.lanes, p.C);
  // with a post norm the next row's loads take the registers
  BackwardVectors<T, VEC, NV, ONE, !POST && hold<T, VEC, NV, 8>()> c(p, at);
  Sums<NV, VEC> sums;
  long long r0, r1;
  chunk_rows_of(p, blockIdx.x, &r0, &r1);
  Pack<T, VEC> py[NV], po[NV], pdy[NV], pdh[NV];
  auto ask = [&](long long row) {
    const long long off = row * p.C;
    NA_RUNS(a) if (at.in[a]) {
      if (dh) py[a] = load_row<T, VEC>(y + off + at.col[a]);
      if (dh) pdh[a] = load_row<T, VEC>(dh + off + at.col[a]);
      if (dy) pdy[a] = load_row<T, VEC>(dy + off + at.col[a]);
      if (o) po[a] = load_row<T, VEC>(o + off + at.col[a]);
    }
  };
  // rows run gate row by gate row, so that a gate row's sum can be written
  // out when its last row is done
  auto end_of = [&](long long seg) { return ONE ? r1 : min(r1, seg + p.gate_rows); };
  // rows past the segment are read as its first, whose values go nowhere
  if (r0 < r1) ask(r0 + sub < end_of(r0) ? r0 + sub : r0);
  for (long long seg = r0; seg < r1;) {
    const long long seg_end = end_of(seg), gate_row = gate_of(p, seg);
    c.at_gate(p, at, gate_row);
    for (long long base = seg; base < seg_end; base += per_block) {
      const bool live = base + sub < seg_end;
      Run<VEC> n[2][NV], t[NV], dx[NV];
      NA_RUNS(a) {
        set(n[0][a], 0.f);
        set(n[1][a], 0.f);
        set(t[a], 0.f);
        set(dx[a], 0.f);
        if (!at.in[a]) continue;
        if (dh) unpack<T>(n[0][a], py[a]);
        if (dh) unpack<T>(t[a], pdh[a]);
        if (dy) unpack<T>(dx[a], pdy[a]);
        if (o) unpack<T>(n[1][a], po[a]);
      }
      const bool same = base + per_block < seg_end;
      const long long next = same ? base + per_block : seg_end, first_row = same ? seg : seg_end;
      if (next < r1) ask(next + sub < end_of(first_row) ? next + sub : first_row);
      float first[2] = {0.f, 0.f};
      if (!p.rms) {
        Run<VEC> a0 = n[0][0], a1 = n[1][0];
#pragma unroll
        for (int a = 1; a < NV; ++a) {
          add(a0, a0, n[0][a]);
          add(a1, a1, n[1][a]);
        }
        first[0] = total(a0) * at.inv;
        first[1] = total(a1) * at.inv;
        red.sum<BLOCK>(first);
      }
      backward_row<T, BLOCK, POST, ONE>(p, n, t, dx, first, live ? base + sub : seg, live, at, c, red, sums, [] {});
    }
    if (!ONE && p.dgate && p.gate_rows > 1)
      flush<VEC, NV, BLOCK>(sums.g, p.dgate + gate_row * p.C, at, red.lanes, p.C, buf);
    seg = seg_end;
  }
  flush_chunk<T, BLOCK, POST, ONE>(p, sums, at, c, red.lanes, buf);
}

// Adds the chunks' sums: 32 columns x 32 chunk lanes a block, each lane its
// chunks in order, then the lanes in order.
__global__ void __launch_bounds__(1024) norm_reduce_kernel(NormArgs p) {
  __shared__ float buf[32][33];
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
#pragma unroll 4
    for (long long k = k0 + part; k < k1; k += 32) s += from[k * p.C + c];
  buf[part][threadIdx.x & 31] = s;
  __syncthreads();
  if (part == 0 && c < p.C) {
#pragma unroll
    for (int u = 1; u < 32; ++u) s += buf[u][threadIdx.x];
    to[c] = s;
  }
}

// -------------------------------------------------------------- wide rows
// A block holds a row of more channels than a warp takes, whose bytes are a
// multiple of 16.  Rows come through a
// ring of bulk copies in shared memory, so that what is in flight does not
// hang on registers or on how many blocks an SM holds; the copy of a later row
// starts as soon as a reduction's barrier has shown that all threads have
// read the row.
constexpr int kMaxStages = 8;

struct Ring {
  uint32_t data, bars, stage_bytes, row_bytes;
  int stages;
  NA_DEVICE uint32_t at(int it) const { return data + (uint32_t)(it % stages) * stage_bytes; }
  NA_DEVICE uint32_t bar(int it) const { return bars + (uint32_t)(it % stages) * 8; }
};

template <typename T, int VEC> NA_DEVICE void read_shared(Run<VEC>& d, uint32_t at) {
  uint4 u;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(at));
  unpack<T>(d, *reinterpret_cast<const Pack<T, VEC>*>(&u));
}
// The mean of the first 8 VEC values of a row in shared memory, which wide rows
// have, by each warp for itself: no barrier.  Of 32 VEC, 3% slower.
template <typename T, int VEC> NA_DEVICE float first_of(uint32_t at) {
  Run<VEC> r;
  read_shared<T>(r, at + (threadIdx.x & 7) * VEC * (uint32_t)sizeof(T));
  float s = total(r);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s * (1.f / (8 * VEC));
}
NA_DEVICE void ring_init(const Ring& ring, volatile int* abort_flag) {
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < ring.stages; ++i) sm100::mbar_init(ring.bars + i * 8, 1);
    sm100::mbar_init_fence();
  }
  __syncthreads();
}

// Warps that give up waiting for row `it` leave, each as a whole, so that the
// barriers of the others keep whole warps.  The one that asks for the rows first
// lets those land that may be on their way: a copy that came later would write
// another block's memory.  The limit is for all of them, as those past the
// block's last row were not asked for.  Kept out of the loop over rows: as part
// of it, it cost registers that the loop needs (139 us where this takes 104, at
// 16387 rows of 4096).  Rows are counted in 32 bits: 64 cost 5 us there, in
// divisions by the number of stages.
__device__ __noinline__ void ring_settle(uint32_t bars, int it, int stages) {
  const unsigned long long t0 = globaltimer_ns();
  for (int u = it; u < it + stages; ++u)
    while (!sm100::mbar_try_wait(bars + (uint32_t)(u % stages) * 8, (uint32_t)(u / stages) & 1))
      if (globaltimer_ns() - t0 > kWaitLimitNs) return;
}

// Blocks of 256 threads an SM: with weights held (16 bits) registers leave room
// for two; a third spills, and costs 112 us where two take 104 (16387 rows of
// 4096).  float32 reads its weights again and has three, 80 us where two take 98
// (8000 rows of 2500).
template <typename T> constexpr int kWideBlocks = sizeof(T) == 2 ? 2 : 3;

template <typename T, int VEC, int NV, int THREADS, bool FULL>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? kWideBlocks<T> : 1)
     norm_forward_wide_kernel(NormArgs p, int stages) {
  using namespace sm100;
  extern __shared__ __align__(128) uint8_t ring_data[];
  __shared__ __align__(16) float scratch[2][kMaxSums * kMaxWarps];
  __shared__ uint64_t ring_bars[kMaxStages];
  __shared__ volatile int abort_flag;
  Reducer red{scratch, (int)blockDim.x, 0};
  red.init();
  const bool two = p.o != nullptr;
  const uint32_t row_bytes = (uint32_t)p.C * sizeof(T);
  const Ring ring{smem_addr(ring_data), smem_addr(ring_bars), row_bytes * (two ? 2 : 1), row_bytes, stages};
  auto ask = [&](int it) {  // by thread 0
    const long long row = blockIdx.x + (long long)it * gridDim.x;
    if (row >= p.rows) return;
    mbar_expect_tx(ring.bar(it), ring.stage_bytes);
    bulk_load(ring.at(it), (const T*)p.x + row * p.C, row_bytes, ring.bar(it));
    if (two) bulk_load(ring.at(it) + row_bytes, (const T*)p.o + row * p.C, row_bytes, ring.bar(it));
  };
  ring_init(ring, &abort_flag);
  if (threadIdx.x == 0)
    for (int i = 0; i < stages; ++i) ask(i);
  const Place<NV> at = place_of<VEC, NV, FULL>(threadIdx.x, blockDim.x, p.C);
  ForwardVectors<T, VEC, NV, hold<T, VEC, NV, 16>()> c(p, at);
  int it = 0;
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x, ++it) {
    if (!__all_sync(0xffffffffu, mbar_wait(ring.bar(it), (uint32_t)(it / stages) & 1, &abort_flag, p.status))) {
      if (threadIdx.x < 32) ring_settle(ring.bars, it, stages);
      return;
    }
    Run<VEC> y[NV], v[NV];
    NA_RUNS(a) {
      set(y[a], 0.f);
      set(v[a], 0.f);
      if (!at.in[a]) continue;
      read_shared<T>(y[a], ring.at(it) + at.col[a] * (uint32_t)sizeof(T));
      if (two) read_shared<T>(v[a], ring.at(it) + row_bytes + at.col[a] * (uint32_t)sizeof(T));
    }
    forward_row<T, true>(p, y, v, row, true, at, c, red, [&] {
      if (threadIdx.x == 0) ask(it + stages);
    });
  }
}

// The chunks, the sums and their order are those of norm_backward_kernel.
template <typename T, int VEC, int NV, bool POST, bool ONE, bool FULL>
__global__ void __launch_bounds__(512, 1) norm_backward_wide_kernel(NormArgs p, int stages) {
  using namespace sm100;
  extern __shared__ __align__(128) uint8_t ring_data[];
  __shared__ __align__(16) float scratch[2][kMaxSums * kMaxWarps];
  __shared__ uint64_t ring_bars[kMaxStages];
  __shared__ volatile int abort_flag;
  Reducer red{scratch, (int)blockDim.x, 0};
  red.init();
  const bool has_h = p.dh != nullptr, has_y = p.dy != nullptr, has_o = p.o != nullptr;
  const uint32_t row_bytes = (uint32_t)p.C * sizeof(T);
  // a stage: y, dh (both with dh), dy, o
  const uint32_t dy_off = has_h ? 2 * row_bytes : 0, o_off = dy_off + (has_y ? row_bytes : 0);
  const Ring ring{smem_addr(ring_data), smem_addr(ring_bars), o_off + (has_o ? row_bytes : 0), row_bytes, stages};
  long long r0, r1;
  chunk_rows_of(p, blockIdx.x, &r0, &r1);
  auto ask = [&](int it) {  // by thread 0
    const long long row = r0 + it;
    if (row >= r1) return;
    const uint32_t to = ring.at(it), bar = ring.bar(it);
    mbar_expect_tx(bar, ring.stage_bytes);
    if (has_h) {
      bulk_load(to, (const T*)p.x + row * p.C, row_bytes, bar);
      bulk_load(to + row_bytes, (const T*)p.dh + row * p.C, row_bytes, bar);
    }
    if (has_y) bulk_load(to + dy_off, (const T*)p.dy + row * p.C, row_bytes, bar);
    if (has_o) bulk_load(to + o_off, (const T*)p.o + row * p.C, row_bytes, bar);
  };
  ring_init(ring, &abort_flag);
  if (threadIdx.x == 0)
    for (int i = 0; i < stages; ++i) ask(i);
  const Place<NV> at = place_of<VEC, NV, FULL>(threadIdx.x, blockDim.x, p.C);
  BackwardVectors<T, VEC, NV, ONE, hold<T, VEC, NV, 8>()> c(p, at);
  Sums<NV, VEC> sums;
  long long gate_row = r0 < r1 ? gate_of(p, r0) : 0, gate_end = (gate_row + 1) * p.gate_rows;
  c.at_gate(p, at, gate_row);
  int it = 0;
  for (long long row = r0; row < r1; ++row, ++it) {
    if (!__all_sync(0xffffffffu, mbar_wait(ring.bar(it), (uint32_t)(it / stages) & 1, &abort_flag, p.status))) {
      if (threadIdx.x < 32) ring_settle(ring.bars, it, stages);
      return;
    }
    Run<VEC> n[2][NV], t[NV], dx[NV];
    NA_RUNS(a) {
      set(n[0][a], 0.f);
      set(n[1][a], 0.f);
      set(t[a], 0.f);
      set(dx[a], 0.f);
      if (!at.in[a]) continue;
      const uint32_t from = ring.at(it) + at.col[a] * (uint32_t)sizeof(T);
      if (has_h) {
        read_shared<T>(n[0][a], from);
        read_shared<T>(t[a], from + row_bytes);
      }
      if (has_y) read_shared<T>(dx[a], from + dy_off);
      if (has_o) read_shared<T>(n[1][a], from + o_off);
    }
    float first[2] = {0.f, 0.f};
    if (!p.rms) {
      if constexpr (sizeof(T) == 4) {  // the means themselves
        NA_RUNS(a) {
          first[0] += total(n[0][a]) * at.inv;
          first[1] += total(n[1][a]) * at.inv;
        }
        red.sum<true>(first);
      } else {
        if (has_h) first[0] = first_of<T, VEC>(ring.at(it));
        if (POST) first[1] = first_of<T, VEC>(ring.at(it) + o_off);
      }
    }
    backward_row<T, true, POST, ONE>(p, n, t, dx, first, row, true, at, c, red, sums, [&] {
      if (threadIdx.x == 0) ask(it + stages);
    });
    if constexpr (!ONE)
      if (row + 1 == gate_end || row + 1 == r1) {
        if (p.dgate && p.gate_rows > 1)
          flush<VEC, NV, true>(sums.g, p.dgate + gate_row * p.C, at, 0, p.C, nullptr);
        ++gate_row;
        gate_end += p.gate_rows;
        if (row + 1 < r1) c.at_gate(p, at, gate_row);
      }
  }
  flush_chunk<T, true, POST, ONE>(p, sums, at, c, 0, nullptr);
}
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
  static std::atomic<int> counts[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  int n = counts[dev];
  if (n == 0 && cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess) counts[dev] = n;
  return n > 0 ? n : 148;
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
  for (int nv = 2; nv <= max_warp_nv; ++nv)
    if (n <= 32 * nv) return {32, 0, nv};
  return {0, n, 0};
}
int block_of(int vectors, int nv) { return ((vectors + nv - 1) / nv + 31) / 32 * 32; }

// Whether `lanes` threads of NV runs end where a row does.  8, 16 and 32 lanes
// and blocks of 8 or 16 channels a thread mostly do (C = 64 ... 8192).
bool is_full(const NormArgs& p, int lanes, int nv, int vec) { return (long long)lanes * nv * vec == p.C; }

template <typename T, int VEC, int NV, bool BLOCK>
cudaError_t forward_one(const NormArgs& p, int lanes, int block, cudaStream_t st) {
  const int threads = BLOCK ? block : 256;
  const long long per_block = BLOCK ? 1 : 256 / lanes;
  const long long need = (p.rows + per_block - 1) / per_block;
  const long long most = (long long)sms() * (2048 / threads);
  const unsigned grid = (unsigned)(need < most ? need : most);
  if (!BLOCK && VEC > 1 && is_full(p, lanes, NV, VEC))
    norm_forward_kernel<T, VEC, NV, BLOCK, (!BLOCK && VEC > 1)><<<grid, threads, 0, st>>>(p);
  else
    norm_forward_kernel<T, VEC, NV, BLOCK, false><<<grid, threads, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T, int VEC, int NV, int THREADS>
cudaError_t forward_wide(const NormArgs& p, int block, cudaStream_t st) {
  auto kern = is_full(p, block, NV, VEC) ? norm_forward_wide_kernel<T, VEC, NV, THREADS, true>
                                         : norm_forward_wide_kernel<T, VEC, NV, THREADS, false>;
  const int per_sm = THREADS == 256 ? (block <= 128 ? 2 : 1) * kWideBlocks<T> : 1;
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
    if constexpr (VEC * sizeof(T) == 16) {  // rows that bulk copies can take
      const int block = block_of(pl.block, 16 / VEC);
      return block <= 256 ? forward_wide<T, VEC, 16 / VEC, 256>(p, block, st)
                          : forward_wide<T, VEC, 16 / VEC, 512>(p, block, st);
    } else if (VEC == 1 && p.C <= 4096)  // with 16 a row of few hundred leaves a third of its warp's places empty
      return forward_one<T, VEC, 8, true>(p, 0, block_of(pl.block, 8), st);
    else
      return forward_one<T, VEC, 16 / VEC, true>(p, 0, block_of(pl.block, 16 / VEC), st);
  }
  if (pl.nv == 1) return forward_one<T, VEC, 1, false>(p, pl.lanes, 0, st);
  if (pl.nv == 2) return forward_one<T, VEC, 2, false>(p, pl.lanes, 0, st);
  if (pl.nv == 3) return forward_one<T, VEC, 3, false>(p, pl.lanes, 0, st);
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
  if (gate_rows >= r || gates == 1) {
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

template <typename T, int VEC, int NV, bool BLOCK, bool POST, bool ONE>
cudaError_t backward_one(const NormArgs& p, int block, cudaStream_t st) {
  const size_t smem = BLOCK ? 0 : sizeof(float) * 256 * NV * VEC;
  if (!BLOCK && VEC > 1 && is_full(p, p.lanes, NV, VEC))
    norm_backward_kernel<T, VEC, NV, BLOCK, POST, ONE, (!BLOCK && VEC > 1)>
        <<<(unsigned)p.chunks, BLOCK ? block : 256, smem, st>>>(p);
  else
    norm_backward_kernel<T, VEC, NV, BLOCK, POST, ONE, false><<<(unsigned)p.chunks, BLOCK ? block : 256, smem, st>>>(p);
  return cudaGetLastError();
}
template <typename T, int VEC, int NV, bool BLOCK>
cudaError_t backward_post(const NormArgs& p, int block, cudaStream_t st) {
  if (p.pieces > 0)
    return p.post ? backward_one<T, VEC, NV, BLOCK, true, true>(p, block, st)
                  : backward_one<T, VEC, NV, BLOCK, false, true>(p, block, st);
  return p.post ? backward_one<T, VEC, NV, BLOCK, true, false>(p, block, st)
                : backward_one<T, VEC, NV, BLOCK, false, false>(p, block, st);
}
template <typename T, int VEC, int NV, bool POST, bool ONE>
cudaError_t backward_wide_one(const NormArgs& p, int block, cudaStream_t st) {
  auto kern = is_full(p, block, NV, VEC) ? norm_backward_wide_kernel<T, VEC, NV, POST, ONE, true>
                                         : norm_backward_wide_kernel<T, VEC, NV, POST, ONE, false>;
  const size_t stage = (size_t)p.C * sizeof(T) * ((p.dh ? 2 : 0) + (p.dy ? 1 : 0) + (p.o ? 1 : 0));
  const int stages = ring_stages(stage, block > 256 ? 1 : block > 128 ? 2 : 4);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 216 * 1024);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)p.chunks, block, stage * stages, st>>>(p, stages);
  return cudaGetLastError();
}
template <typename T, int VEC, int NV> cudaError_t backward_wide(const NormArgs& p, int block, cudaStream_t st) {
  if (p.pieces > 0)
    return p.post ? backward_wide_one<T, VEC, NV, true, true>(p, block, st)
                  : backward_wide_one<T, VEC, NV, false, true>(p, block, st);
  return p.post ? backward_wide_one<T, VEC, NV, true, false>(p, block, st)
                : backward_wide_one<T, VEC, NV, false, false>(p, block, st);
}

template <typename T, int VEC> cudaError_t backward_vec(NormArgs p, cudaStream_t st) {
  constexpr int kWarpNV = VEC == 8 ? 1 : 2;
  const Plan pl = plan_for(p.C, VEC, kWarpNV);
  p.lanes = pl.lanes;
  if (pl.block) {  // as few vectors a thread as blocks of 512 allow
    constexpr int kOne = VEC == 1 ? 8 : 1;
    const int one = block_of(pl.block, kOne), two = block_of(pl.block, 2 * kOne), four = block_of(pl.block, 4);
    if constexpr (VEC * sizeof(T) == 16) {  // rows that bulk copies can take
      if (one <= 512) return backward_wide<T, VEC, 1>(p, one, st);
      if (VEC == 8 || two <= 512) return backward_wide<T, VEC, 2>(p, two, st);
      if constexpr (VEC == 4) return backward_wide<T, VEC, 4>(p, four, st);
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
  norm_reduce_kernel<<<dim3((unsigned)((p.C + 31) / 32), (unsigned)(4 + gates)), 1024, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace na2d
