// na_packed_tc.cu -- forward of the packed attention on the tensor cores, fp16
// and bf16.
//
// A block owns two row tiles (A and B) of one key head and walks the keys they
// see in tiles of 128:
//
//   S_t = Q_t K_j^T  ->  P_t = 2^(S_t scale log2e - ref), 16 bits over S_t's
//   columns  ->  O_t += P_t V_j        (S, P and O in tensor memory)
//
// with one softmax warpgroup a tile, a thread a row.  While one tile's
// softmax runs, the tensor pipe works for the other, so both the special
// functions and the tensor cores stay busy; with one row tile a block they
// would wait for each other.  O is rescaled only when a row's maximum has
// grown by 2^8 over its reference: P then stays below 2^8, far inside the
// 16-bit types, and most tiles rescale nothing; the softmax warps do it
// themselves, as S_t's arrival implies that the last P V of t is done.
//
// P is rounded to the input type for its product with V; its sum is taken
// before that, in float32.
//
// Roles: warp 0 loads (TMA), warp 1 issues the MMAs, warpgroups 1 and 2 are
// the softmax and the epilogue of tiles A and B.
#include "na_packed_tc.cuh"

namespace na2d {
namespace {

using namespace packed;

template <int D> struct Fwd {
  using G = Geo<D>;
  static constexpr int SLOTS = D == 128 ? 4 : 8;  // ring of K and V tiles, in the order they are used
  static constexpr int Q_OFF = 0;
  static constexpr int RING_OFF = 2 * G::TILE_BYTES;
  static constexpr int BAR_OFF = RING_OFF + SLOTS * G::TILE_BYTES;
  static constexpr int SMEM = BAR_OFF + 256 + 1024;
  // one block an SM, as it holds all of tensor memory
  static constexpr int SMEM_ASKED = SMEM > 116 * 1024 ? SMEM : 116 * 1024;
  static_assert(SMEM <= kMaxSmem, "fits");
  static constexpr int THREADS = 384;
  static constexpr int REGS_CTRL = 72, REGS_SOFTMAX = 216;
  static constexpr int O_COL = 256;  // S_A at 0, S_B at 128, O_t at 256 + t D
};

constexpr float kSlack = 8.f;  // log2 of how far a maximum may pass its reference

template <typename T, int D>
__global__ void __launch_bounds__(Fwd<D>::THREADS, 1)
packed_forward_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                         const __grid_constant__ CUtensorMap mv, const PackedArgs p) {
  using C = Fwd<D>;
  using G = Geo<D>;
  constexpr bool BF16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int SLOTS = C::SLOTS;
  extern __shared__ uint8_t raw[];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ------------------------------------------------------------ what to do
  const int P = kTile / p.group;  // positions of a row tile
  const int kh = blockIdx.y;
  int s;
  long long idx;
  find_part_warp(p.cu_q, p.nseq, p.total_q, 1, 2 * P, blockIdx.x, &s, &idx);
  const Span sp = span_of(p, s);
  // the last rows, which see the most keys, first: the short blocks fill the
  // gaps at the end
  const long long part = (sp.nq + 2 * P - 1) / (2 * P) - 1 - idx;
  if (idx < 0 || part < 0) return;
  const int pos0 = (int)part * 2 * P;
  int piece0 = 0, piece1 = sp.nk;
  if (p.max_pieces > 1) {
    const int len = piece_length(p, sp);
    piece0 = (int)min((long long)blockIdx.z * len, (long long)sp.nk);
    piece1 = (int)min((long long)piece0 + len, (long long)sp.nk);
    if (blockIdx.z > 0 && piece0 >= piece1) return;
  }
  // tile t: positions [pos0 + t P, ...), key tiles 0 .. steps[t] from kb on
  int kb = 0, steps[2], ends[2];
  {
    int lo, hi, unused;
    visible(p, sp, pos0, &lo, &unused);
    kb = max(lo, piece0);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int last = min(pos0 + (t + 1) * P, sp.nq) - 1;
      if (last < pos0 + t * P) {
        ends[t] = kb;
      } else {
        visible(p, sp, last, &unused, &hi);
        ends[t] = max(min(hi, piece1), kb);
      }
      steps[t] = (ends[t] - kb + kTile - 1) / kTile;
    }
  }
  const int n = max(steps[0], steps[1]);

  // --------------------------------------------------------------- set up
  const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
  auto q_tile = [&](int t) { return base + C::Q_OFF + t * G::TILE_BYTES; };
  auto slot = [&](int i) { return base + C::RING_OFF + (i % SLOTS) * G::TILE_BYTES; };
  const uint32_t bars = base + C::BAR_OFF;
  auto bar_q = [&]() { return bars; };
  auto bar_full = [&](int i) { return bars + 8 + (i % SLOTS) * 8; };
  auto bar_empty = [&](int i) { return bars + 8 + (SLOTS + i % SLOTS) * 8; };
  auto bar_s = [&](int t) { return bars + 8 + (2 * SLOTS + t) * 8; };
  auto bar_p = [&](int t) { return bars + 8 + (2 * SLOTS + 2 + t) * 8; };
  auto bar_o = [&](int t) { return bars + 8 + (2 * SLOTS + 4 + t) * 8; };
  const uint32_t bar_tail = bars + 8 + (2 * SLOTS + 6) * 8, bar_done = bar_tail + 8;
  if (threadIdx.x == 0) {
    abort_flag = 0;
    mbar_init(bar_q(), 1);
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(bar_full(i), 1);
      mbar_init(bar_empty(i), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar_s(t), 1);
      mbar_init(bar_p(t), 4);
      mbar_init(bar_o(t), 1);
    }
    mbar_init(bar_tail, 1);
    mbar_init(bar_done, 1);
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc(smem_addr(&tmem_slot), 512);
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&mq);
    tma_prefetch_desc(&mk);
    tma_prefetch_desc(&mv);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  volatile int* ab = &abort_flag;

  if (warp < 4) {
    regs_dec<C::REGS_CTRL>();
    if (warp == 0 && n > 0) {
      // ------------------------------------------------------------- loads
      // The ring holds K_0, V_0, K_1, V_1, ...
      if (lane == 0) {
        mbar_expect_tx(bar_q(), (uint32_t)(2 * P * p.group * D * 2));
        for (int t = 0; t < 2; ++t) load_row_tile<D>(q_tile(t), &mq, bar_q(), kh, sp.q0 + pos0 + t * P);
      }
      bool tail_used = false;
      int i = 0;
      for (; i < 2 * n; ++i) {
        if (i >= SLOTS && !mbar_wait(bar_empty(i), ((i / SLOTS) - 1) & 1, ab, p.status)) break;
        const int k0 = kb + (i / 2) * kTile;
        const CUtensorMap* m = (i & 1) ? &mv : &mk;
        // values past the sequence's keys are zeroed, as their zero weights
        // would not stop a NaN
        const bool tail = (i & 1) && k0 + kTile > sp.nk;
        const uint32_t bar = tail ? bar_tail : bar_full(i);
        if (lane == 0) {
          mbar_expect_tx(bar, G::TILE_BYTES);
          load_key_tile<D>(slot(i), m, bar, kh, sp.k0 + k0);
        }
        __syncwarp();
        if (tail) {
          tail_used = true;
          if (!mbar_wait(bar_tail, 0, ab, p.status)) break;
          zero_rows<D>(slot(i), sp.nk - k0);
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_full(i));
        }
      }
      if (*ab) {  // leave no copy in flight
        mbar_wait_settle(bar_q(), 0);
        if (tail_used) mbar_wait_settle(bar_tail, 0);
        for (int u = max(0, i - SLOTS); u < i; ++u) mbar_wait_settle(bar_full(u), (u / SLOTS) & 1);
      }
    } else if (warp == 1 && n > 0) {
      // -------------------------------------------------------------- MMAs
      if (lane == 0) {
        auto s_mma = [&](int t, int j) {
          mma_rows_by_rows<D, BF16>(tmem + t * kTile, q_tile(t), slot(2 * j));
          mma_commit(bar_s(t));
        };
        bool ok = mbar_wait(bar_q(), 0, ab, p.status) && mbar_wait(bar_full(0), 0, ab, p.status);
        if (ok) {
          tc_fence_after();
          for (int t = 0; t < 2; ++t)
            if (steps[t] > 0) s_mma(t, 0);
          mma_commit(bar_empty(0));
          for (int j = 0; j < n && ok; ++j) {
            if (!(ok = mbar_wait(bar_full(2 * j + 1), ((2 * j + 1) / SLOTS) & 1, ab, p.status))) break;
            if (j + 1 < n && !(ok = mbar_wait(bar_full(2 * j + 2), ((2 * j + 2) / SLOTS) & 1, ab, p.status))) break;
            for (int t = 0; t < 2; ++t) {
              if (j >= steps[t]) continue;
              if (!(ok = mbar_wait(bar_p(t), j & 1, ab, p.status))) break;
              tc_fence_after();
              mma_weights_by_tile<D, BF16>(tmem + C::O_COL + t * D, tmem + t * kTile, slot(2 * j + 1), j > 0);
              if (j + 1 < steps[t])
                s_mma(t, j + 1);
              else
                mma_commit(bar_o(t));
            }
            mma_commit(bar_empty(2 * j + 1));
            if (j + 1 < n) mma_commit(bar_empty(2 * j + 2));
          }
        }
        // every MMA has finished before tensor memory is freed
        mma_commit(bar_done);
        mbar_wait_settle(bar_done, 0);
      }
      __syncwarp();
    }
  } else {
    regs_inc<C::REGS_SOFTMAX>();
    // ---------------------------------------------------- softmax, epilogue
    const int t = (warp >> 2) - 1, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + t * kTile, o_at = tmem + lanes + C::O_COL + t * D;
    const int at = row / p.group;  // position in the tile
    const int pos = pos0 + t * P + at;
    const bool live = at < P && pos < sp.nq;
    int lo, hi;
    visible(p, sp, live ? pos : min(max(sp.nq - 1, 0), pos0 + t * P), &lo, &hi);
    lo = max(lo, piece0);
    hi = min(hi, piece1);
    // keys that all rows of the warp see
    const int all_lo = __reduce_max_sync(0xffffffffu, lo), all_hi = __reduce_min_sync(0xffffffffu, hi);
    const float sl2 = p.scale * kLog2e;
    const int my_steps = t ? steps[1] : steps[0];
    float ref = -INFINITY, sum = 0.f;  // ref in units of raw logits
    bool ok = true;
    for (int j = 0; j < my_steps; ++j) {
      if (!(ok = mbar_wait(bar_s(t), j & 1, ab, p.status))) break;
      tc_fence_after();
      uint32_t x[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(s_at + 32 * c, x[c]);
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_wait_ld_regs(x[c]);
      const int k0 = kb + j * kTile;
      if (k0 < all_lo || k0 + kTile > all_hi) {
        const int a = lo - k0, b = hi - k0;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (32 * c + i < a || 32 * c + i >= b) x[c][i] = 0xff800000u;
      }
      float m4[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        m4[c] = __uint_as_float(x[c][0]);
#pragma unroll
        for (int i = 1; i < 31; i += 2) m4[c] = max3(m4[c], __uint_as_float(x[c][i]), __uint_as_float(x[c][i + 1]));
        m4[c] = fmaxf(m4[c], __uint_as_float(x[c][31]));
      }
      const float top = fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]);
      if (j == 0) {
        ref = top;
      } else if (__any_sync(0xffffffffu, (top - ref) * sl2 > kSlack)) {
        // -inf - -inf is NaN and compares false: nothing seen yet stays so
        const float next = fmaxf(ref, top);
        const float f = ref == next ? 1.f : exp2f((ref - next) * sl2);
        ref = next;
        sum *= f;
        constexpr int W = D < 32 ? D : 32;
#pragma unroll
        for (int c = 0; c < D / W; ++c) {
          uint32_t o[W];
          if constexpr (W == 32) tmem_ld32(o_at + W * c, o); else tmem_ld16(o_at, o);
          tmem_wait_ld_regs(o);
#pragma unroll
          for (int i = 0; i < W; ++i) o[i] = f == 0.f ? 0u : __float_as_uint(__uint_as_float(o[i]) * f);
          if constexpr (W == 32) tmem_st32(o_at + W * c, o); else tmem_st16(o_at, o);
        }
      }
      const float shift = ref == -INFINITY ? 0.f : -ref * sl2;
      float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          float a0 = __uint_as_float(x[c][i]), a1 = __uint_as_float(x[c][i + 1]);
          float b0 = __uint_as_float(x[c][i + 2]), b1 = __uint_as_float(x[c][i + 3]);
          fma2(a0, a1, a0, a1, sl2, sl2, shift, shift);
          fma2(b0, b1, b0, b1, sl2, sl2, shift, shift);
          a0 = ex2(a0);
          a1 = ex2(a1);
          b0 = ex2(b0);
          b1 = ex2(b1);
          add2(s0, s1, s0, s1, a0, a1);
          add2(s2, s3, s2, s3, b0, b1);
          w[i / 2] = pack2<T>(a0, a1);
          w[i / 2 + 1] = pack2<T>(b0, b1);
        }
        tmem_st16(s_at + 16 * c, w);
      }
      sum += (s0 + s1) + (s2 + s3);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_p(t));
    }
    if (ok && my_steps > 0) ok = mbar_wait(bar_o(t), 0, ab, p.status);
    if (ok) {
      tc_fence_after();
      const bool split = p.max_pieces > 1;
      const long long i = (long long)sp.q0 + pos;
      const int head = kh * p.group + row % p.group;
      const long long out_row = i * p.hq + head;
      const long long part_row = ((long long)blockIdx.z * p.total_q + i) * p.hq + head;
      // a row that saw no key: zeros and -inf
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const float lse = sum == 0.f ? -INFINITY : fmaf(ref, p.scale, log2f(sum) * kLn2);
      bool finite = fabsf(sum) < INFINITY;
      constexpr int W = D < 32 ? D : 32;
#pragma unroll
      for (int c = 0; c < D / W; ++c) {
        uint32_t o[W];
        if (my_steps > 0) {
          if constexpr (W == 32) tmem_ld32(o_at + W * c, o); else tmem_ld16(o_at, o);
          tmem_wait_ld_regs(o);
        } else {
#pragma unroll
          for (int e = 0; e < W; ++e) o[e] = 0u;
        }
        float f[W];
#pragma unroll
        for (int e = 0; e < W; ++e) {
          f[e] = __uint_as_float(o[e]) * inv;
          finite = finite && fabsf(f[e]) < INFINITY;
        }
        if (live) {
          if (split) {
#pragma unroll
            for (int e = 0; e < W; e += 4)
              *reinterpret_cast<float4*>(p.part_o + part_row * D + W * c + e) =
                  make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
          } else {
            T* to = (T*)p.out + out_row * D + W * c;
#pragma unroll
            for (int e = 0; e < W; e += 8)
              *reinterpret_cast<uint4*>(to + e) = make_uint4(pack2<T>(f[e], f[e + 1]), pack2<T>(f[e + 2], f[e + 3]),
                                                             pack2<T>(f[e + 4], f[e + 5]), pack2<T>(f[e + 6], f[e + 7]));
          }
        }
      }
      if (live) {
        if (split)
          p.part_lse[part_row] = lse;
        else if (p.lse)
          p.lse[(long long)head * p.total_q + i] = lse;
      }
      // rows with a result that is not finite are taken again, key by key
      unsigned again = __ballot_sync(0xffffffffu, live && !finite);
      while (again) {
        const int src = __ffs(again) - 1;
        again &= again - 1;
        const long long to = __shfl_sync(0xffffffffu, out_row, src), pto = __shfl_sync(0xffffffffu, part_row, src);
        const int l0 = __shfl_sync(0xffffffffu, lo, src), h0 = __shfl_sync(0xffffffffu, hi, src);
        const long long stride = (long long)p.hk * D, first = ((long long)sp.k0 * p.hk + kh) * D;
        float acc[(D + 31) / 32], l, m;
        exact_row<T, D>(p, (const T*)p.q + to * D, (const T*)p.k + first, (const T*)p.v + first, stride, l0, h0, acc,
                        &l, &m);
#pragma unroll
        for (int e = 0; e < (D + 31) / 32; ++e) {
          if (lane + 32 * e >= D) continue;
          const float r = acc[e] / l;
          if (split)
            p.part_o[pto * D + lane + 32 * e] = r;
          else
            ((T*)p.out)[to * D + lane + 32 * e] = from_f<T>(r);
        }
        if (lane == 0) {
          const float again_lse = (m + log2f(l)) * kLn2;
          if (split)
            p.part_lse[pto] = again_lse;
          else if (p.lse)
            p.lse[(to % p.hq) * p.total_q + to / p.hq] = again_lse;
        }
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <typename T, int D> cudaError_t launch(const PackedArgs& p, cudaStream_t st) {
  using C = Fwd<D>;
  constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  const long long blocks = part_numbers(p.nseq, p.total_q, 1, 2 * (kTile / p.group));
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaError_t e = prepare_kernel<packed_forward_tc_kernel<T, D>>(
      C::SMEM_ASKED, C::THREADS, 128 * C::REGS_CTRL + 256 * C::REGS_SOFTMAX);
  if (e != cudaSuccess) return e;
  CUtensorMap mq, mk, mv;
  if (!row_map(&mq, p.q, p, bf16) || !key_map(&mk, p.k, p, bf16) || !key_map(&mv, p.v, p, bf16))
    return cudaErrorInvalidValue;
  packed_forward_tc_kernel<T, D>
      <<<dim3((unsigned)blocks, (unsigned)p.hk, (unsigned)(p.max_pieces > 1 ? p.max_pieces : 1)), C::THREADS,
         C::SMEM_ASKED, st>>>(mq, mk, mv, p);
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

cudaError_t launch_packed_forward_tc(const PackedArgs& p, na_dtype dt, cudaStream_t st) {
  return dt == NA_F16 ? launch_d<__half>(p, st) : launch_d<__nv_bfloat16>(p, st);
}

}  // namespace na2d
