// na_packed_tc.cu -- forward of the packed attention on the tensor cores, fp16
// and bf16.
//
// A block owns two row tiles (A and B; one where d <= 64, with two blocks an
// SM) of one key head and walks the keys they see in tiles of 128:
//
//   S_t = Q_t K_j^T  ->  P_t = 2^(S_t scale log2e - ref) in 16 bits
//   ->  O_t += P_t V_j                        (S, P and O in tensor memory)
//
// with one softmax warpgroup a tile, a thread a row.  A softmax takes S into
// registers at once, and the next S is made while it works, so that a tile's
// chain is its softmax alone and the products hide behind it.  That needs P in
// columns of its own; tensor memory then has room for one S, which two tiles
// use in turn (each holds it for its product and the load).  With P over S, softmax and products of a tile took
// turns: 3.3 thousand cycles a step where the tensor pipe needs 2.0.
//
// O is rescaled only when a row's maximum has grown by 2^8 over its reference:
// P then stays below 2^8, far inside the 16-bit types, and most tiles rescale
// nothing; the softmax warps do it themselves.
//
// P is rounded to the input type for its product with V; its sum is taken
// before that, in float32.
//
// Roles: warp 0 loads (TMA), warp 1 issues S, warp 2 issues P V, warpgroups 1
// and 2 are the softmax and the epilogue of tiles A and B.
#include "na_packed_tc.cuh"

namespace na2d {
namespace {

using namespace packed;

template <int D> struct Fwd {
  using G = Geo<D>;
  static constexpr int TILES = packed_row_tiles(D);
  static constexpr int SLOTS = 4;  // ring of K and V tiles, in the order they are used
  static constexpr int Q_OFF = 0;
  static constexpr int RING_OFF = TILES * G::TILE_BYTES;
  static constexpr int BAR_OFF = RING_OFF + SLOTS * G::TILE_BYTES;
  static constexpr int SMEM = BAR_OFF + 256 + 1024;
  // As many blocks an SM as share tensor memory: one of two tiles, or two of
  // one tile, whose starts and ends then overlap the other's work.
  static constexpr int BLOCKS = TILES == 2 ? 1 : 2;
  static constexpr int SMEM_LEAST = BLOCKS == 1 ? 116 * 1024 : 78 * 1024;
  static constexpr int SMEM_ASKED = SMEM > SMEM_LEAST ? SMEM : SMEM_LEAST;
  static_assert(SMEM_ASKED * BLOCKS <= kMaxSmem, "fits");
  static constexpr int THREADS = 128 + 128 * TILES;
  static constexpr int REGS_CTRL = TILES == 2 ? 72 : 40, REGS_SOFTMAX = TILES == 2 ? 216 : 208;
  // tensor memory: S of 128 columns, P_t of 64, O_t of d
  static constexpr int P_COL = kTile, O_COL = P_COL + TILES * 64;
  static constexpr int TMEM = 512 / BLOCKS;
  static_assert(O_COL + TILES * D <= TMEM, "fits");
};

constexpr float kSlack = 8.f;  // log2 of how far a maximum may pass its reference

template <typename T, int D>
__global__ void __launch_bounds__(Fwd<D>::THREADS, Fwd<D>::BLOCKS)
packed_forward_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                         const __grid_constant__ CUtensorMap mv, const PackedArgs p) {
  using C = Fwd<D>;
  using G = Geo<D>;
  constexpr bool BF16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int SLOTS = C::SLOTS, TILES = C::TILES;
  extern __shared__ uint8_t raw[];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ------------------------------------------------------------ what to do
  const int P = kTile / p.group;  // positions of a row tile
  const int kh = blockIdx.x % p.hk;  // the heavy tiles of all heads start first
  int s;
  long long idx;
  find_part_warp(p.cu_q, p.nseq, p.total_q, 1, TILES * P, blockIdx.x / p.hk, &s, &idx);
  const Span sp = span_of(p, s);
  // the last rows, which see the most keys, first: the short blocks fill the
  // gaps at the end
  const long long part = (sp.nq + TILES * P - 1) / (TILES * P) - 1 - idx;
  if (idx < 0 || part < 0) return;
  const int pos0 = (int)part * TILES * P;
  int piece0 = 0, piece1 = sp.nk;
  if (p.max_pieces > 1) {
    const int len = piece_length(p, sp);
    piece0 = (int)min((long long)blockIdx.y * len, (long long)sp.nk);
    piece1 = (int)min((long long)piece0 + len, (long long)sp.nk);
    if (blockIdx.y > 0 && piece0 >= piece1) return;
  }
  // tile t: positions [pos0 + t P, ...), key tiles 0 .. steps[t] from kb on
  int kb = 0, steps[2] = {0, 0};
  {
    int lo, hi, unused;
    visible(p, sp, pos0, &lo, &unused);
    kb = max(lo, piece0);
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      const int last = min(pos0 + (t + 1) * P, sp.nq) - 1;
      if (last < pos0 + t * P) continue;
      visible(p, sp, last, &unused, &hi);
      steps[t] = (max(min(hi, piece1), kb) - kb + kTile - 1) / kTile;
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
  auto bar_s = [&](int t) { return bars + 8 + (2 * SLOTS + t) * 8; };       // S_t is made
  auto bar_pv = [&](int t) { return bars + 8 + (2 * SLOTS + 2 + t) * 8; };  // O_t has P_t V
  auto bar_p = [&](int t, int half) { return bars + 8 + (2 * SLOTS + 4 + 2 * t + half) * 8; };
  const uint32_t bar_free = bars + 8 + (2 * SLOTS + 8) * 8;  // S is in registers
  const uint32_t bar_tail = bars + 8 + (2 * SLOTS + 10) * 8, bar_done0 = bar_tail + 8;
  auto bar_done = [&](int w) { return bar_done0 + w * 8; };
  if (threadIdx.x == 0) {
    abort_flag = 0;
    mbar_init(bar_q(), 1);
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(bar_full(i), 1);
      mbar_init(bar_empty(i), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar_s(t), 1);
      mbar_init(bar_p(t, 0), 4);
      mbar_init(bar_p(t, 1), 4);
      mbar_init(bar_pv(t), 1);

    }
    mbar_init(bar_free, 4);
    mbar_init(bar_tail, 1);
    mbar_init(bar_done(0), 1);
    mbar_init(bar_done(1), 1);
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc(smem_addr(&tmem_slot), C::TMEM);
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
  // fp16 weights are lifted by 2^7, which the sum takes out again: with the
  // slack they stay below 2^15, and small ones keep their bits
  constexpr float kLift = BF16 ? 0.f : 7.f;

  if (warp < 4) {
    regs_dec<C::REGS_CTRL>();
    if (warp == 0 && n > 0) {
      // ------------------------------------------------------------- loads
      // The ring holds K_0, V_0, K_1, V_1, ...
      if (lane == 0) {
        mbar_expect_tx(bar_q(), (uint32_t)(TILES * P * p.group * D * 2));
        for (int t = 0; t < TILES; ++t) load_row_tile<D>(q_tile(t), &mq, bar_q(), kh, sp.q0 + pos0 + t * P);
      }
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
          if (!mbar_wait(bar_tail, 0, ab, p.status)) {
            mbar_wait_settle(bar_tail, 0);
            break;
          }
          zero_rows<D>(slot(i), sp.nk - k0);
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_full(i));
        }
      }
      mbar_wait_settle(bar_q(), 0);
      settle_ring(0, i, SLOTS, bar_full);
    } else if (warp == 1 && n > 0) {
      // ----------------------------------------------------------- S = Q K^T
      // The whole warp walks the steps, which keeps what the operands are made
      // of in uniform registers, and one lane issues.
      bool ok = mbar_wait(bar_q(), 0, ab, p.status);
      int made = 0;
      for (int j = 0; j < n; ++j) {
        ok = ok && mbar_wait(bar_full(2 * j), (2 * j / SLOTS) & 1, ab, p.status);
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
          if (j >= steps[t]) continue;
          if (made > 0) ok = ok && mbar_wait(bar_free, (made - 1) & 1, ab, p.status);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          ++made;
          tc_fence_after();
          if (elect_one()) {
            mma_rows_by_rows<D, BF16>(tmem, q_tile(t), slot(2 * j));
            mma_commit(bar_s(t));
          }
        }
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        if (elect_one()) mma_commit(bar_empty(2 * j));
      }
      // every MMA has finished before tensor memory is freed
      if (elect_one()) mma_commit(bar_done(0));
      mbar_wait_settle(bar_done(0), 0);
      __syncwarp();
    } else if (warp == 2 && n > 0) {
      // ---------------------------------------------------------- O += P V
      bool ok = true;
      for (int j = 0; j < n && ok; ++j) {
        ok = mbar_wait(bar_full(2 * j + 1), ((2 * j + 1) / SLOTS) & 1, ab, p.status);
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
          if (j >= steps[t]) continue;
          const uint32_t o = tmem + C::O_COL + t * D, w = tmem + C::P_COL + t * 64;
          ok = ok && mbar_wait(bar_p(t, 0), j & 1, ab, p.status);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          tc_fence_after();
          if (elect_one()) mma_weights_by_tile<D, BF16, 32, 0, 4>(o, w, slot(2 * j + 1), j > 0);
          ok = mbar_wait(bar_p(t, 1), j & 1, ab, p.status);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          tc_fence_after();
          if (elect_one()) {
            mma_weights_by_tile<D, BF16, 32, 4, 8>(o, w, slot(2 * j + 1), true);
            mma_commit(bar_pv(t));
          }
        }
        if (ok && elect_one()) mma_commit(bar_empty(2 * j + 1));
      }
      if (elect_one()) mma_commit(bar_done(1));
      mbar_wait_settle(bar_done(1), 0);
      __syncwarp();
    }
  } else {
    regs_inc<C::REGS_SOFTMAX>();
    // ---------------------------------------------------- softmax, epilogue
    const int t = (warp >> 2) - 1, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes, w_at = tmem + lanes + C::P_COL + t * 64;
    const uint32_t o_at = tmem + lanes + C::O_COL + t * D;
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
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_free);
      const int k0 = kb + j * kTile;
      const bool masked = k0 < all_lo || k0 + kTile > all_hi;
      if (masked) {
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
        for (int i = 1; i < 31; i += 2)
          m4[c] = max3_nan(m4[c], __uint_as_float(x[c][i]), __uint_as_float(x[c][i + 1]));
        m4[c] = max_nan(m4[c], __uint_as_float(x[c][31]));
      }
      const float top = max_nan(max3_nan(m4[0], m4[1], m4[2]), m4[3]);
      // the last product has read P, and O can be changed
      if (j > 0 && !(ok = mbar_wait(bar_pv(t), (j - 1) & 1, ab, p.status))) break;
      tc_fence_after();
      if (j == 0) {
        ref = top;
      } else if (__any_sync(0xffffffffu, live && !((top - ref) * sl2 <= kSlack))) {
        // Rows that are not the sequence's have no say, or its bits would depend
        // on them.  Also where nothing was seen yet (-inf - -inf) and for NaN, which
        // makes the row's whole result NaN
        const float next = max_nan(ref, top);
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
          for (int i = 0; i < W; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);  // NaN stays, also under 0
          if constexpr (W == 32) tmem_st32(o_at + W * c, o); else tmem_st16(o_at, o);
        }
      }
      // an infinite reference makes the whole row NaN, as inf - inf does
      const float shift = ref == -INFINITY ? 0.f : fmaf(-ref, sl2, ref - ref) + kLift;
      float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
      auto weights = [&](auto poly) {
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
            if (decltype(poly)::value && i % 8 == 4) {
              exp2_poly2(b0, b1);
            } else {
              b0 = ex2(b0);
              b1 = ex2(b1);
            }
            add2(s0, s1, s0, s1, a0, a1);
            add2(s2, s3, s2, s3, b0, b1);
            w[i / 2] = pack2<T>(a0, a1);
            w[i / 2 + 1] = pack2<T>(b0, b1);
          }
          tmem_st16(w_at + 16 * c, w);
          if (c & 1) {  // half of the weights: their product can start
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_p(t, c >> 1));
          }
        }
      };
      // A quarter of the exponentials by polynomial, but not where masked places
      // must give exactly 0.
      if (masked)
        weights(std::false_type{});
      else
        weights(std::true_type{});
      sum += (s0 + s1) + (s2 + s3);
    }
    if (ok && my_steps > 0) ok = mbar_wait(bar_pv(t), (my_steps - 1) & 1, ab, p.status);
    if (ok) {
      tc_fence_after();
      const bool split = p.max_pieces > 1;
      const long long i = (long long)sp.q0 + pos;
      const int head = kh * p.group + row % p.group;
      const long long out_row = i * p.hq + head;
      const long long part_row = ((long long)blockIdx.y * p.total_q + i) * p.hq + head;
      // every logit was -inf: no weights, where the polynomial made some of 2^-126
      if (ref == -INFINITY) sum = 0.f;
      // a row that saw no key: zeros and -inf
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const float lse = sum == 0.f ? -INFINITY : fmaf(ref, p.scale, (log2f(sum) - kLift) * kLn2);
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
        float acc[(D + 31) / 32], again_lse;
        exact_row<T, D>(p, (const T*)p.q + to * D, (const T*)p.k + first, (const T*)p.v + first, stride, l0, h0, acc,
                        &again_lse);
#pragma unroll
        for (int e = 0; e < (D + 31) / 32; ++e) {
          if (lane + 32 * e >= D) continue;
          if (split)
            p.part_o[pto * D + lane + 32 * e] = acc[e];
          else
            ((T*)p.out)[to * D + lane + 32 * e] = from_f<T>(acc[e]);
        }
        if (lane == 0) {
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
    tmem_dealloc(tmem, C::TMEM);
  }
}

template <typename T, int D> cudaError_t launch(const PackedArgs& p, cudaStream_t st) {
  using C = Fwd<D>;
  constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  const long long blocks = part_numbers(p.nseq, p.total_q, 1, C::TILES * (kTile / p.group));
  if (blocks * p.hk > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaError_t e = prepare_kernel<packed_forward_tc_kernel<T, D>>(
      C::SMEM_ASKED, C::THREADS, 128 * C::REGS_CTRL + 128 * C::TILES * C::REGS_SOFTMAX);
  if (e != cudaSuccess) return e;
  CUtensorMap mq, mk, mv;
  if (!row_map(&mq, p.q, p, bf16) || !key_map(&mk, p.k, p, bf16) || !key_map(&mv, p.v, p, bf16))
    return cudaErrorInvalidValue;
  packed_forward_tc_kernel<T, D>
      <<<dim3((unsigned)(blocks * p.hk), (unsigned)p.max_pieces), C::THREADS,
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
