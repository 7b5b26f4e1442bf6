// na_packed_tc_bwd.cu -- gradients of the packed attention on the tensor cores,
// fp16 and bf16.
//
// Two kernels, both of which recompute the weights from the rows' log-sum-exp:
//
//   dk, dv   a block owns 128 keys and walks the row tiles that see them:
//            S^T = K Q^T, dP^T = V dO^T, P^T = 2^(S^T scale log2e - lse),
//            dS^T = P^T (dP^T - delta), dV += P^T dO, dK += dS^T Q;
//   dq       a block owns a row tile and walks the keys it sees:
//            S = Q K^T, dP = dO V^T, dS likewise, dQ += dS K.
//
// That is seven products where one kernel that owned keys and added dq to
// memory with atomics would need five; in exchange each gradient is one
// block's sum in a fixed order and no float32 copy of dq goes through memory.
// The heads of a group are rows like any others, so a shared head's gradient
// needs no further sum.
//
// P^T and dS^T are written over S^T and dP^T (16 bits) and read as operands
// from tensor memory; the next S^T and dP^T are written over those by the thread
// that issued their products before, as one thread's products run in order.  The
// products are issued so that the tensor pipe always
// has one while a half of the element-wise work runs: dV and the next S^T
// beside dS^T, dK and the next dP^T beside P^T.  Two warpgroups share a tile,
// each 64 of its columns, a thread a lane.  The tiles that are walked come
// through two rings, as Q and dO (K and V) are done with at different times:
// with both in one ring of two stages at d = 128, a step waited 1.5 of 3.5
// thousand cycles for its loads.
//
// P and dS are rounded to the input type for their products.  fp16 weights are
// lifted by 2^15, which leaves them below 2^16 and keeps the bits of small ones.
// fp16 dS = P (dP - delta) would vanish for gradients of 1e-3 over some thousand
// keys.  It is lifted by the power of two that brings the norm of dO's row (for
// dk, whose products sum over rows, of the largest row of the sequence and key
// head) to 16 to 32, and stays below 2^16 where values' norms are below 2^10,
// as |dS| <= 2 |dO| |V|; above that the row or key is taken again in float32.
//
// delta = dout . out comes from an out that was rounded.  Where all of a row's
// keys are in one tile (the first rows of a causal sequence, whose out is
// largest) the dq kernel takes it from P and dP instead, for itself and for the
// kernel of dk and dv, which runs after it.
#include "na_packed_tc.cuh"

namespace na2d {
namespace {

using namespace packed;

template <int D> struct Bwd {
  using G = Geo<D>;
  // slots of the rings: A for Q (K), which are needed first and kept longest, B
  // for dO (V)
  static constexpr int SA = D == 128 ? 3 : 4, SB = D == 128 ? 2 : 4, ST = 2;
  static constexpr int A_OFF = 2 * G::TILE_BYTES;  // the two tiles that stay come first
  static constexpr int B_OFF = A_OFF + SA * G::TILE_BYTES;
  static constexpr int TERMS_OFF = B_OFF + SB * G::TILE_BYTES;
  static constexpr int BAR_OFF = TERMS_OFF + ST * 2 * kTile * 4;
  static constexpr int kBars = 15 + 2 * SA + 2 * SB + 2 * ST;
  static constexpr int TMEM_SLOT = kBars * 8, ABORT = TMEM_SLOT + 4;
  static constexpr int SMEM = BAR_OFF + (ABORT + 4 + 15) / 16 * 16;
  static constexpr int SMEM_ASKED = SMEM > 116 * 1024 ? SMEM : 116 * 1024;  // one block an SM: it holds all of tensor memory
  static_assert(SMEM <= kMaxSmem, "fits");
  static constexpr int THREADS = 384;
  static constexpr int REGS_CTRL = 72, REGS_WORK = 216;
};

// The barriers, and the two words behind them: tensor memory's address and the
// block's abort flag.
//
// What is done once a step has two barriers, used in turn: step i waits for
// phase i / 2 of the (i & 1)-th.  With one, a warp held back for a step would
// find two phases complete, which its parity cannot tell from none, and wait
// for good: the dq kernel's S is made a step ahead, and a `turn` is announced
// before the last one needs to have been looked at.  Step i + 2 of each is only
// begun after all that wait for step i have passed it.
template <int D> struct Bars {
  using C = Bwd<D>;
  uint32_t base;
  NA_DEVICE uint32_t kept() const { return base; }
  NA_DEVICE uint32_t done() const { return base + 8; }
  NA_DEVICE uint32_t tail() const { return base + 16; }  // of both rings' last tile
  NA_DEVICE uint32_t s(int i) const { return base + 24 + (i & 1) * 8; }
  NA_DEVICE uint32_t dp(int i) const { return base + 40 + (i & 1) * 8; }
  NA_DEVICE uint32_t p_half(int i) const { return base + 56 + (i & 1) * 8; }
  NA_DEVICE uint32_t p_ready(int i) const { return base + 72 + (i & 1) * 8; }
  NA_DEVICE uint32_t ds_ready(int i) const { return base + 88 + (i & 1) * 8; }
  NA_DEVICE uint32_t turn(int i) const { return base + 104 + (i & 1) * 8; }  // of the other MMA warp
  NA_DEVICE uint32_t full_a(int i) const { return base + 120 + (i % C::SA) * 8; }
  NA_DEVICE uint32_t empty_a(int i) const { return base + 120 + (C::SA + i % C::SA) * 8; }
  NA_DEVICE uint32_t full_b(int i) const { return base + 120 + (2 * C::SA + i % C::SB) * 8; }
  NA_DEVICE uint32_t empty_b(int i) const { return base + 120 + (2 * C::SA + C::SB + i % C::SB) * 8; }
  NA_DEVICE uint32_t full_t(int i) const { return base + 120 + (2 * C::SA + 2 * C::SB + i % C::ST) * 8; }
  NA_DEVICE uint32_t empty_t(int i) const { return base + 120 + (2 * C::SA + 2 * C::SB + C::ST + i % C::ST) * 8; }
  NA_DEVICE uint32_t tmem_slot() const { return base + C::TMEM_SLOT; }
  NA_DEVICE void init(int empty_b_count) const {
    mbar_init(kept(), 1);
    mbar_init(done(), 2);  // both MMA warps'
    mbar_init(tail(), 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(s(i), 1);
      mbar_init(dp(i), 1);
      mbar_init(p_half(i), 8);
      mbar_init(p_ready(i), 8);
      mbar_init(ds_ready(i), 8);
      mbar_init(turn(i), 1);
    }
    for (int i = 0; i < C::SA; ++i) mbar_init(full_a(i), 1), mbar_init(empty_a(i), 1);
    for (int i = 0; i < C::SB; ++i) mbar_init(full_b(i), 1), mbar_init(empty_b(i), empty_b_count);
    for (int i = 0; i < C::ST; ++i) mbar_init(full_t(i), 1), mbar_init(empty_t(i), 8);
    mbar_init_fence();
  }
};
// Shared memory is asked for without room to align it: tiles need 1024 bytes.
NA_DEVICE bool aligned_or_report(uint32_t base, unsigned* status) {
  if ((base & 1023u) == 0) return true;
  if (threadIdx.x == 0) atomicOr(status, kStatusTimeout);
  return false;
}

template <int W> NA_DEVICE void tmem_ld_n(uint32_t at, uint32_t (&r)[W]) {
  if constexpr (W == 32)
    tmem_ld32(at, r);
  else if constexpr (W == 16)
    tmem_ld16(at, r);
  else
    tmem_ld8(at, r);
  tmem_wait_ld_regs(r);
}

// Columns outside [a, b) become `to`.
NA_DEVICE void mask_outside(uint32_t (&x)[2][32], int a, int b, uint32_t to) {
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (32 * c + e < a || 32 * c + e >= b) x[c][e] = to;
}

// A store of W consecutive results, in dt or in float32.
template <typename T, int W> NA_DEVICE void store_run(T* to, const float (&f)[W]) {
#pragma unroll
  for (int e = 0; e < W; e += 8)
    *reinterpret_cast<uint4*>(to + e) = make_uint4(pack2<T>(f[e], f[e + 1]), pack2<T>(f[e + 2], f[e + 3]),
                                                   pack2<T>(f[e + 4], f[e + 5]), pack2<T>(f[e + 6], f[e + 7]));
}
template <int W> NA_DEVICE void store_run(float* to, const float (&f)[W]) {
#pragma unroll
  for (int e = 0; e < W; e += 4) *reinterpret_cast<float4*>(to + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
}

// The weight and its gradient of one row and key, from global memory; term holds
// the row's log-sum-exp and delta, which the dq kernel writes while it runs.
template <typename T, int D>
NA_DEVICE void exact_pair(const PackedArgs& p, float2 term, long long row, long long key, float* w, float* ds) {
  const float s = dot_row<T, D>((const T*)p.q + row * D, (const T*)p.k + key * D);
  const float dp = dot_row<T, D>((const T*)p.dout + row * D, (const T*)p.v + key * D);
  *w = exp2f(fmaf(s, p.scale * kLog2e, -term.x));
  *ds = *w * (dp - term.y);
}

// ------------------------------------------------------------------ dk, dv
template <typename T, int D>
__global__ void __launch_bounds__(Bwd<D>::THREADS, 1)
packed_dkdv_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mo,
                      const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                      const PackedArgs p) {
  using C = Bwd<D>;
  using G = Geo<D>;
  constexpr bool BF16 = std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ __align__(1024) uint8_t raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // heads and pieces first, then tiles: the heavy tiles of all heads start first
  const int P = kTile / p.group, Z = p.max_pieces, lanes_of_tile = p.hk * Z;
  const int kh = blockIdx.x % lanes_of_tile / Z, z = blockIdx.x % Z;
  int s;
  long long idx;
  find_part_warp(p.cu_k, p.nseq, p.total_k, 1, kTile, blockIdx.x / lanes_of_tile, &s, &idx);
  if (idx < 0) return;
  const Span sp = span_of(p, s);
  if (idx * kTile >= sp.nk) return;
  const int j0 = (int)idx * kTile, nk = min(kTile, sp.nk - j0);
  // row tiles: positions first + (z + i Z) P, i = 0 .. n - 1
  int first, last, unused;
  seen_by(p, sp, j0, &first, &unused);
  seen_by(p, sp, j0 + nk - 1, &unused, &last);
  const int tiles = last > first ? (last - first + P - 1) / P : 0;
  const int n = tiles > z ? (tiles - z + Z - 1) / Z : 0;
  auto tile_pos = [&](int i) { return first + (z + i * Z) * P; };

  const uint32_t base = smem_addr(raw);
  if (!aligned_or_report(base, p.status)) return;
  const uint32_t k_tile = base, v_tile = base + G::TILE_BYTES;
  auto q_tile = [&](int i) { return base + C::A_OFF + (i % C::SA) * G::TILE_BYTES; };
  auto o_tile = [&](int i) { return base + C::B_OFF + (i % C::SB) * G::TILE_BYTES; };
  auto lse_of = [&](int i) { return reinterpret_cast<float*>(raw + C::TERMS_OFF) + (i % C::ST) * 2 * kTile; };
  const Bars<D> bar{base + C::BAR_OFF};
  volatile int* ab = reinterpret_cast<volatile int*>(raw + C::BAR_OFF + C::ABORT);
  if (threadIdx.x == 0) {
    *ab = 0;
    bar.init(2);  // dO goes into dP and dV
  }
  if (warp == 1) tmem_alloc(bar.tmem_slot(), 512);
  if (P * p.group < kTile && warp >= 4)  // rows of a tile that no copy fills
    for (int i = warp - 4; i < C::SA + C::SB; i += 8) zero_rows<D>(base + C::A_OFF + i * G::TILE_BYTES, P * p.group);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(raw + C::BAR_OFF + C::TMEM_SLOT);
  const uint32_t s_at = tmem, dp_at = tmem + 128, dv_at = tmem + 256, dk_at = tmem + 256 + D;
  // log2 of the weights' lift, and what turns dP - delta into the factor that,
  // times them, is the lifted dS
  constexpr float kLift = BF16 ? 0.f : 15.f, kUnlift = BF16 ? 1.f : 1.f / 32768.f;
  const float lift = BF16 ? 1.f : p.lifts[(long long)s * p.hk + kh], to_ds = kUnlift * lift;

  if (warp < 4) {
    regs_dec<C::REGS_CTRL>();
    if ((warp == 0 || warp == 2) && n > 0) {
      // ------------------ loads: K, V and the row tiles' Q by one warp, their
      // log-sum-exp, delta and dO by another
      const bool first_warp = warp == 0;
      if (first_warp && lane == 0) {
        mbar_expect_tx(bar.kept(), 2 * G::TILE_BYTES);
        load_key_tile<D>(k_tile, &mk, bar.kept(), kh, sp.k0 + j0);
        load_key_tile<D>(v_tile, &mv, bar.kept(), kh, sp.k0 + j0);
      }
      const uint32_t bytes = (uint32_t)(P * p.group * D * 2);
      int i = 0;
      for (; i < n; ++i) {
        const int pos = tile_pos(i);
        if (!first_warp) {
          if (i >= C::ST && !mbar_wait(bar.empty_t(i), ((i / C::ST) - 1) & 1, ab, p.status)) break;
          float* lse = lse_of(i);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = lane + 32 * e, at = r / p.group;
            float2 t = make_float2(INFINITY, 0.f);  // a row that is not there: weights 0
            if (at < P && pos + at < sp.nq)
              t = p.terms[((long long)sp.q0 + pos + at) * p.hq + kh * p.group + (r - at * p.group)];
            lse[r] = t.x - kLift;
            lse[kTile + r] = t.y * to_ds;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar.full_t(i));
        }
        const uint32_t empty = first_warp ? bar.empty_a(i) : bar.empty_b(i);
        const int slots = first_warp ? C::SA : C::SB;
        if (i >= slots && !mbar_wait(empty, ((i / slots) - 1) & 1, ab, p.status)) break;
        if (!load_ring_tile<D>(first_warp ? q_tile(i) : o_tile(i), first_warp ? bar.full_a(i) : bar.full_b(i), bar.tail(),
                          rows_of_tile(sp.nq, pos, P, p.group), P * p.group, bytes, ab, p.status, [&](uint32_t dst, uint32_t b) {
                            load_row_tile<D>(dst, first_warp ? &mq : &mo, b, kh, sp.q0 + pos);
                          }))
          break;
      }
      if (first_warp) mbar_wait_settle(bar.kept(), 0);
      settle_ring(0, i, first_warp ? C::SA : C::SB, [&](int u) { return first_warp ? bar.full_a(u) : bar.full_b(u); });
    } else if ((warp == 1 || warp == 3) && n > 0) {
      // -------------------------------------------------------------- MMAs
      // One warp for S^T and dV, one for dP^T and dK: each runs its two in
      // turn, and while one looks at its barriers the tensor pipe has the
      // other's.  dK waits until the next S^T is issued, which the threads need
      // first: all at once, S^T came 0.9 thousand cycles of a step later.  The whole warp walks the steps, which keeps what the operands
      // are made of in uniform registers, and one lane issues.
      const bool first_warp = warp == 1;
      const uint32_t at = first_warp ? s_at : dp_at, to = first_warp ? dv_at : dk_at;
      const uint32_t kept = first_warp ? k_tile : v_tile;
      auto made = [&](int i) { return first_warp ? bar.s(i) : bar.dp(i); };
      // S^T is made of a row tile's Q and dV summed with its dO; dP^T and dK the other way round
      auto with = [&](int i) { return first_warp ? q_tile(i) : o_tile(i); };
      auto sums = [&](int i) { return first_warp ? o_tile(i) : q_tile(i); };
      auto wait_a = [&](int i) { return mbar_wait(bar.full_a(i), (i / C::SA) & 1, ab, p.status); };
      auto wait_b = [&](int i) { return mbar_wait(bar.full_b(i), (i / C::SB) & 1, ab, p.status); };
      bool ok = mbar_wait(bar.kept(), 0, ab, p.status) && (first_warp ? wait_a(0) : wait_b(0));
      if (__all_sync(0xffffffffu, ok)) {
        tc_fence_after();
        if (elect_one()) {
          mma_rows_by_rows<D, BF16>(at, kept, with(0));
          mma_commit(made(0));
          if (!first_warp) mma_commit(bar.empty_b(0));
        }
        for (int i = 0; i < n; ++i) {
          // the next tile is there long before it is needed; asking for it here
          // keeps the question out of the way between two products
          ok = first_warp ? wait_b(i) : wait_a(i);
          if (i + 1 < n) ok = ok && (first_warp ? wait_a(i + 1) : wait_b(i + 1));
          if (first_warp) {
            // P^T comes in halves: 32 of each warpgroup's 64 columns
            ok = ok && mbar_wait(bar.p_half(i), (i >> 1) & 1, ab, p.status);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            if (elect_one()) {
              mma_weights_by_tile<D, BF16, 64, 0, 2>(to, at, sums(i), i > 0);  // the halves lie 64 columns apart
              mma_weights_by_tile<D, BF16, 64, 4, 6>(to, at, sums(i), true);
            }
          }
          ok = ok && mbar_wait(first_warp ? bar.p_ready(i) : bar.ds_ready(i), (i >> 1) & 1, ab, p.status);
          if (!first_warp) ok = ok && mbar_wait(bar.turn(i), (i >> 1) & 1, ab, p.status);
          if (!__all_sync(0xffffffffu, ok)) break;
          tc_fence_after();
          if (elect_one()) {
            if (first_warp) {
              mma_weights_by_tile<D, BF16, 64, 2, 4>(to, at, sums(i), true);
              mma_weights_by_tile<D, BF16, 64, 6, 8>(to, at, sums(i), true);
            } else {
              mma_weights_by_tile<D, BF16, 64>(to, at, sums(i), i > 0);
            }
            mma_commit(first_warp ? bar.empty_b(i) : bar.empty_a(i));
            if (i + 1 < n) {
              mma_rows_by_rows<D, BF16>(at, kept, with(i + 1));
              mma_commit(made(i + 1));
              if (!first_warp) mma_commit(bar.empty_b(i + 1));
            }
            if (first_warp) mbar_arrive(bar.turn(i));
          }
        }
      }
      if (elect_one()) mma_commit(bar.done());
      mbar_wait_settle(bar.done(), 0);
      __syncwarp();
    }
  } else {
    regs_inc<C::REGS_WORK>();
    // ------------------------------------------------- P^T, dS^T, epilogue
    const int half = (warp >> 2) - 1, key = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t my_s = s_at + lanes + half * 64, my_dp = dp_at + lanes + half * 64;
    const bool live = key < nk;
    int lo, hi;  // positions that see this key
    seen_by(p, sp, j0 + min(key, nk - 1), &lo, &hi);
    // positions that see all keys of the warp, and those of any
    const int all_lo = __reduce_max_sync(0xffffffffu, lo), all_hi = __reduce_min_sync(0xffffffffu, hi);
    const float sl2 = p.scale * kLog2e;
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      if (!(ok = mbar_wait(bar.full_t(i), (i / C::ST) & 1, ab, p.status))) break;
      if (!(ok = mbar_wait(bar.s(i), (i >> 1) & 1, ab, p.status))) break;
      tc_fence_after();
      const int pos = tile_pos(i);
      const bool masked = pos < all_lo || pos + P > all_hi;
      const int a = row_in_tile(lo, pos, P, p.group) - half * 64, b = row_in_tile(hi, pos, P, p.group) - half * 64;
      const float4* lse = reinterpret_cast<const float4*>(lse_of(i) + half * 64);
      const float4* delta = lse + kTile / 4;
      uint32_t x[2][32];
      tmem_ld32(my_s, x[0]);
      tmem_ld32(my_s + 32, x[1]);
      tmem_wait_ld_regs(x[0]);
      tmem_wait_ld_regs(x[1]);
      if (masked) mask_outside(x, a, b, 0xff800000u);
      // a quarter by polynomial, but not where masked places must give exactly 0
      auto weights = [&](auto poly) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 l = lse[8 * c + e / 4];
          float f[4] = {__uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1]), __uint_as_float(x[c][e + 2]),
                        __uint_as_float(x[c][e + 3])};
          fma2(f[0], f[1], f[0], f[1], sl2, sl2, -l.x, -l.y);
          fma2(f[2], f[3], f[2], f[3], sl2, sl2, -l.z, -l.w);
          f[0] = ex2(f[0]);
          f[1] = ex2(f[1]);
          if (decltype(poly)::value && e % 8 == 4) {
            exp2_poly2(f[2], f[3]);
          } else {
            f[2] = ex2(f[2]);
            f[3] = ex2(f[3]);
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) x[c][e + u] = __float_as_uint(f[u]);
          w[e / 2] = pack2<T>(f[0], f[1]);
          w[e / 2 + 1] = pack2<T>(f[2], f[3]);
        }
        tmem_st16(my_s + 16 * c, w);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(c == 0 ? bar.p_half(i) : bar.p_ready(i));
      }
      };
      if (masked)
        weights(std::false_type{});
      else
        weights(std::true_type{});
      if (!(ok = mbar_wait(bar.dp(i), (i >> 1) & 1, ab, p.status))) break;
      tc_fence_after();
      uint32_t y[2][32];
      tmem_ld32(my_dp, y[0]);
      tmem_ld32(my_dp + 32, y[1]);
      tmem_wait_ld_regs(y[0]);
      tmem_wait_ld_regs(y[1]);
      // a zero weight does not stop a NaN
      if (masked) mask_outside(y, a, b, 0u);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 l = delta[8 * c + e / 4];
          float f[4] = {__uint_as_float(y[c][e]), __uint_as_float(y[c][e + 1]), __uint_as_float(y[c][e + 2]),
                        __uint_as_float(y[c][e + 3])};
          fma2(f[0], f[1], f[0], f[1], to_ds, to_ds, -l.x, -l.y);
          fma2(f[2], f[3], f[2], f[3], to_ds, to_ds, -l.z, -l.w);
#pragma unroll
          for (int u = 0; u < 4; ++u) f[u] *= __uint_as_float(x[c][e + u]);
          w[e / 2] = pack2<T>(f[0], f[1]);
          w[e / 2 + 1] = pack2<T>(f[2], f[3]);
        }
        tmem_st16(my_dp + 16 * c, w);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar.ds_ready(i));
        mbar_arrive(bar.empty_t(i));
      }
    }
    if (ok && n > 0) ok = mbar_wait(bar.done(), 0, ab, p.status);
    if (ok) {
      tc_fence_after();
      // the first warpgroup writes dv, the second dk
      const float f0 = half ? p.scale : 1.f, taken = half ? p.scale / lift : kUnlift;
      const uint32_t from = (half ? dk_at : dv_at) + lanes;
      const long long at = ((long long)(sp.k0 + j0 + key) * p.hk + kh) * D;
      T* to = (T*)(half ? p.dk : p.dv) + at;
      float* part = p.part_o + ((long long)z * 2 + half) * p.total_k * p.hk * D + at;
      bool finite = true;
      constexpr int W = D < 32 ? D : 32;
#pragma unroll
      for (int c = 0; c < D / W; ++c) {
        uint32_t o[W] = {};
        if (n > 0) tmem_ld_n<W>(from + W * c, o);
        float f[W];
#pragma unroll
        for (int e = 0; e < W; ++e) {
          f[e] = __uint_as_float(o[e]) * taken;
          finite = finite && fabsf(f[e]) < INFINITY;
        }
        if (live) {
          if (Z > 1)
            store_run<W>(part + W * c, f);
          else
            store_run<T, W>(to + W * c, f);
        }
      }
      // keys with a result that is not finite are taken again, row by row
      unsigned again = __ballot_sync(0xffffffffu, live && !finite);
      while (again) {
        const int src = __ffs(again) - 1;
        again &= again - 1;
        const int l0 = __shfl_sync(0xffffffffu, lo, src), h0 = __shfl_sync(0xffffffffu, hi, src);
        const long long kat = __shfl_sync(0xffffffffu, at, src);
        float acc[(D + 31) / 32] = {};
        for (int i = 0; i < n; ++i) {
          const long long r0 = (long long)max(tile_pos(i), l0) * p.group,
                          r1 = (long long)min(tile_pos(i) + P, h0) * p.group;
          for (long long r = r0; r < r1; r += 32) {
            float wgt = 0.f, ds = 0.f;
            const long long mine = min(r + lane, r1 - 1);
            const long long row = ((long long)sp.q0 + mine / p.group) * p.hq + kh * p.group + mine % p.group;
            if (r + lane < r1) exact_pair<T, D>(p, p.terms[row], row, kat / D, &wgt, &ds);
            for (int t = 0; t < (int)min(32ll, r1 - r); ++t) {
              const float u = __shfl_sync(0xffffffffu, half ? ds : wgt, t);
              const long long rt = __shfl_sync(0xffffffffu, row, t);
              const T* src_row = (const T*)(half ? p.q : p.dout) + rt * D;
#pragma unroll
              for (int e = 0; e < (D + 31) / 32; ++e)
                if (lane + 32 * e < D) acc[e] = fmaf(u, to_f<T>(src_row[lane + 32 * e]), acc[e]);
            }
          }
        }
#pragma unroll
        for (int e = 0; e < (D + 31) / 32; ++e) {
          if (lane + 32 * e >= D) continue;
          if (Z > 1)
            p.part_o[((long long)z * 2 + half) * p.total_k * p.hk * D + kat + lane + 32 * e] = acc[e] * f0;
          else
            ((T*)(half ? p.dk : p.dv))[kat + lane + 32 * e] = from_f<T>(acc[e] * f0);
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

// Adds the pieces' dk and dv in order; slots of no sequence are left alone.
template <typename T> __global__ void __launch_bounds__(256) packed_dkdv_join_kernel(PackedArgs p) {
  const int vecs = p.d / 8;
  const long long e = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long per = (long long)p.total_k * p.hk * vecs;
  if (e >= per) return;
  const int key = (int)(e / ((long long)p.hk * vecs));
  int a = 0, b = p.nseq - 1;  // the last sequence that starts at or before the key
  while (a < b) {
    const int m = (a + b + 1) >> 1;
    if (clamped(p.cu_k, m, p.total_k) <= key)
      a = m;
    else
      b = m - 1;
  }
  const Span sp = span_of(p, a);
  if (key < sp.k0 || key >= sp.k0 + sp.nk) return;
  const int which = blockIdx.y;
  const float* from = p.part_o + which * per * 8 + e * 8;
  float f[8] = {};
  for (int z = 0; z < p.max_pieces; ++z) {
    const float4 u = *reinterpret_cast<const float4*>(from + (long long)z * 2 * per * 8);
    const float4 v = *reinterpret_cast<const float4*>(from + (long long)z * 2 * per * 8 + 4);
    f[0] += u.x, f[1] += u.y, f[2] += u.z, f[3] += u.w, f[4] += v.x, f[5] += v.y, f[6] += v.z, f[7] += v.w;
  }
  T* to = (T*)(which ? p.dk : p.dv) + e * 8;
  if constexpr (sizeof(T) == 4)
    store_run<8>(to, f);
  else
    store_run<T, 8>(to, f);
}

// ---------------------------------------------------------------------- dq
template <typename T, int D>
__global__ void __launch_bounds__(Bwd<D>::THREADS, 1)
packed_dq_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mo,
                    const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                    const PackedArgs p) {
  using C = Bwd<D>;
  using G = Geo<D>;
  constexpr bool BF16 = std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ __align__(1024) uint8_t raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const int P = kTile / p.group, kh = blockIdx.x % p.hk;
  int s;
  long long idx;
  find_part_warp(p.cu_q, p.nseq, p.total_q, 1, P, blockIdx.x / p.hk, &s, &idx);
  const Span sp = span_of(p, s);
  const long long part = (sp.nq + P - 1) / P - 1 - idx;  // the rows that see most keys first
  if (idx < 0 || part < 0) return;
  const int pos0 = (int)part * P;
  int kb, ke, unused;
  visible(p, sp, pos0, &kb, &unused);
  visible(p, sp, min(pos0 + P, sp.nq) - 1, &unused, &ke);
  const int n = ke > kb ? (ke - kb + kTile - 1) / kTile : 0;

  const uint32_t base = smem_addr(raw);
  if (!aligned_or_report(base, p.status)) return;
  const uint32_t q_tile = base, o_tile = base + G::TILE_BYTES;
  auto k_tile = [&](int i) { return base + C::A_OFF + (i % C::SA) * G::TILE_BYTES; };
  auto v_tile = [&](int i) { return base + C::B_OFF + (i % C::SB) * G::TILE_BYTES; };
  const Bars<D> bar{base + C::BAR_OFF};
  volatile int* ab = reinterpret_cast<volatile int*>(raw + C::BAR_OFF + C::ABORT);
  if (threadIdx.x == 0) {
    *ab = 0;
    bar.init(1);
  }
  if (warp == 1) tmem_alloc(bar.tmem_slot(), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(raw + C::BAR_OFF + C::TMEM_SLOT);
  const uint32_t dp_at = tmem + 256, dq_at = tmem + 384;  // S in two slots of 128 columns

  if (warp < 4) {
    regs_dec<C::REGS_CTRL>();
    if ((warp == 0 || warp == 3) && n > 0) {
      // ------------- loads: Q, dO and the keys by one warp, values by another
      const bool first_warp = warp == 0;
      if (first_warp && lane == 0) {
        mbar_expect_tx(bar.kept(), (uint32_t)(2 * P * p.group * D * 2));
        load_row_tile<D>(q_tile, &mq, bar.kept(), kh, sp.q0 + pos0);
        load_row_tile<D>(o_tile, &mo, bar.kept(), kh, sp.q0 + pos0);
      }
      int i = 0;
      for (; i < n; ++i) {
        const int k0 = kb + i * kTile, slots = first_warp ? C::SA : C::SB;
        const uint32_t empty = first_warp ? bar.empty_a(i) : bar.empty_b(i);
        if (i >= slots && !mbar_wait(empty, ((i / slots) - 1) & 1, ab, p.status)) break;
        if (!load_ring_tile<D>(first_warp ? k_tile(i) : v_tile(i), first_warp ? bar.full_a(i) : bar.full_b(i), bar.tail(),
                          sp.nk - k0, kTile, G::TILE_BYTES, ab, p.status, [&](uint32_t dst, uint32_t b) {
                            load_key_tile<D>(dst, first_warp ? &mk : &mv, b, kh, sp.k0 + k0);
                          }))
          break;
      }
      if (first_warp) mbar_wait_settle(bar.kept(), 0);
      settle_ring(0, i, first_warp ? C::SA : C::SB, [&](int u) { return first_warp ? bar.full_a(u) : bar.full_b(u); });
    } else if ((warp == 1 || warp == 2) && n > 0) {
      // -------------------------------------------------------------- MMAs
      // One warp for S and dQ, one for dP, for the same reason as above; dQ waits
      // until the next dP is issued.
      auto wait_a = [&](int i) { return mbar_wait(bar.full_a(i), (i / C::SA) & 1, ab, p.status); };
      auto wait_b = [&](int i) { return mbar_wait(bar.full_b(i), (i / C::SB) & 1, ab, p.status); };
      bool ok = mbar_wait(bar.kept(), 0, ab, p.status) && (warp == 1 ? wait_a(0) : wait_b(0));
      if (__all_sync(0xffffffffu, ok)) {
        tc_fence_after();
        if (elect_one()) {
          if (warp == 1) {
            mma_rows_by_rows<D, BF16>(tmem, q_tile, k_tile(0));
            mma_commit(bar.s(0));
          } else {
            mma_rows_by_rows<D, BF16>(dp_at, o_tile, v_tile(0));
            mma_commit(bar.dp(0));
            mma_commit(bar.empty_b(0));
          }
        }
        for (int i = 0; i < n; ++i) {
          if (warp == 1 && i + 1 < n) {
            if (!__all_sync(0xffffffffu, wait_a(i + 1))) break;
            tc_fence_after();
            if (elect_one()) {
              mma_rows_by_rows<D, BF16>(tmem + ((i + 1) & 1) * kTile, q_tile, k_tile(i + 1));
              mma_commit(bar.s(i + 1));
            }
          }
          ok = mbar_wait(bar.ds_ready(i), (i >> 1) & 1, ab, p.status);
          if (warp == 1) ok = ok && mbar_wait(bar.turn(i), (i >> 1) & 1, ab, p.status);
          if (warp == 2 && i + 1 < n) ok = ok && wait_b(i + 1);
          if (!__all_sync(0xffffffffu, ok)) break;
          tc_fence_after();
          if (elect_one()) {
            if (warp == 1) {
              mma_weights_by_tile<D, BF16, 64>(dq_at, tmem + (i & 1) * kTile, k_tile(i), i > 0);
              mma_commit(bar.empty_a(i));
            } else {
              if (i + 1 < n) {
                mma_rows_by_rows<D, BF16>(dp_at, o_tile, v_tile(i + 1));
                mma_commit(bar.dp(i + 1));
                mma_commit(bar.empty_b(i + 1));
              }
              mbar_arrive(bar.turn(i));
            }
          }
        }
      }
      if (elect_one()) mma_commit(bar.done());
      mbar_wait_settle(bar.done(), 0);
      __syncwarp();
    }
  } else {
    regs_inc<C::REGS_WORK>();
    // ------------------------------------------------------- dS, epilogue
    const int half = (warp >> 2) - 1, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const int at = row / p.group, pos = pos0 + at;
    const bool live = at < P && pos < sp.nq;
    const long long out_row = ((long long)sp.q0 + (live ? pos : pos0)) * p.hq + kh * p.group + (live ? row - at * p.group : 0);
    int lo, hi;
    visible(p, sp, live ? pos : pos0, &lo, &hi);
    const int all_lo = __reduce_max_sync(0xffffffffu, lo), all_hi = __reduce_min_sync(0xffffffffu, hi);
    float2 term = p.terms[out_row];
    const float lift = BF16 ? 1.f : p.row_lifts[out_row];
    const float sl2 = p.scale * kLog2e;
    bool ok = true;
    // both warpgroups meet once where n is 1, also when one has given up
    auto meet = [] { asm volatile("bar.sync 1, 256;" ::: "memory"); };
    for (int i = 0; i < n; ++i) {
      const uint32_t my_s = tmem + lanes + (i & 1) * kTile + half * 64, my_dp = dp_at + lanes + half * 64;
      if (!(ok = mbar_wait(bar.s(i), (i >> 1) & 1, ab, p.status))) {
        if (n == 1) meet();
        break;
      }
      tc_fence_after();
      const int k0 = kb + i * kTile;
      const bool masked = k0 < all_lo || k0 + kTile > all_hi;
      const int a = lo - k0 - half * 64, b = hi - k0 - half * 64;
      uint32_t x[2][32];
      tmem_ld32(my_s, x[0]);
      tmem_ld32(my_s + 32, x[1]);
      tmem_wait_ld_regs(x[0]);
      tmem_wait_ld_regs(x[1]);
      if (masked) mask_outside(x, a, b, 0xff800000u);
      auto weights = [&](auto poly) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float f0 = __uint_as_float(x[c][e]), f1 = __uint_as_float(x[c][e + 1]);
            fma2(f0, f1, f0, f1, sl2, sl2, -term.x, -term.x);
            if (decltype(poly)::value && e % 8 == 6) {
              exp2_poly2(f0, f1);
            } else {
              f0 = ex2(f0);
              f1 = ex2(f1);
            }
            x[c][e] = __float_as_uint(f0);
            x[c][e + 1] = __float_as_uint(f1);
          }
      };
      if (masked)
        weights(std::false_type{});
      else
        weights(std::true_type{});
      if (!(ok = mbar_wait(bar.dp(i), (i >> 1) & 1, ab, p.status))) {
        if (n == 1) meet();
        break;
      }
      tc_fence_after();
      uint32_t y[2][32];
      tmem_ld32(my_dp, y[0]);
      tmem_ld32(my_dp + 32, y[1]);
      tmem_wait_ld_regs(y[0]);
      tmem_wait_ld_regs(y[1]);
      if (masked) mask_outside(y, a, b, 0u);
      if (n == 1) {
        // all of the row's weights are here: delta from them
        float d0 = 0.f, d1 = 0.f;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            fma2(d0, d1, __uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1]), __uint_as_float(y[c][e]),
                 __uint_as_float(y[c][e + 1]), d0, d1);
        float* sums = reinterpret_cast<float*>(raw + C::TERMS_OFF);
        sums[half * kTile + row] = d0 + d1;
        meet();
        term.y = sums[row] + sums[kTile + row];
        if (live && half == 0) p.terms[out_row].y = term.y;
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float f0 = __uint_as_float(y[c][e]), f1 = __uint_as_float(y[c][e + 1]);
          if constexpr (BF16)
            add2(f0, f1, f0, f1, -term.y, -term.y);
          else
            fma2(f0, f1, f0, f1, lift, lift, -term.y * lift, -term.y * lift);
          f0 *= __uint_as_float(x[c][e]);
          f1 *= __uint_as_float(x[c][e + 1]);
          w[e / 2] = pack2<T>(f0, f1);
        }
        tmem_st16(my_s + 16 * c, w);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar.ds_ready(i));
    }
    if (ok && n > 0) ok = mbar_wait(bar.done(), 0, ab, p.status);
    if (ok) {
      tc_fence_after();
      // each warpgroup writes half of the columns
      constexpr int H = D / 2, W = H < 32 ? H : 32;
      const float taken = p.scale / lift;
      T* to = (T*)p.dq + out_row * D + half * H;
      bool finite = true;
#pragma unroll
      for (int c = 0; c < H / W; ++c) {
        uint32_t o[W] = {};
        if (n > 0) tmem_ld_n<W>(dq_at + lanes + half * H + W * c, o);
        float f[W];
#pragma unroll
        for (int e = 0; e < W; ++e) {
          f[e] = __uint_as_float(o[e]) * taken;
          finite = finite && fabsf(f[e]) < INFINITY;
        }
        if (live) store_run<T, W>(to + W * c, f);
      }
      // rows with a result that is not finite are taken again, key by key
      unsigned again = __ballot_sync(0xffffffffu, live && !finite);
      while (again) {
        const int src = __ffs(again) - 1;
        again &= again - 1;
        const int l0 = __shfl_sync(0xffffffffu, lo, src), h0 = __shfl_sync(0xffffffffu, hi, src);
        const long long r = __shfl_sync(0xffffffffu, out_row, src);
        const float2 t0 = make_float2(__shfl_sync(0xffffffffu, term.x, src), __shfl_sync(0xffffffffu, term.y, src));
        float acc[(D + 31) / 32] = {};
        for (int j = l0; j < h0; j += 32) {
          float wgt, ds = 0.f;
          if (j + lane < h0) exact_pair<T, D>(p, t0, r, (long long)(sp.k0 + j + lane) * p.hk + kh, &wgt, &ds);
          for (int t = 0; t < min(32, h0 - j); ++t) {
            const float u = __shfl_sync(0xffffffffu, ds, t);
            const T* key = (const T*)p.k + ((long long)(sp.k0 + j + t) * p.hk + kh) * D;
#pragma unroll
            for (int e = 0; e < (D + 31) / 32; ++e)
              if (lane + 32 * e < D) acc[e] = fmaf(u, to_f<T>(key[lane + 32 * e]), acc[e]);
          }
        }
#pragma unroll
        for (int e = 0; e < (D + 31) / 32; ++e) {
          const int c = lane + 32 * e;
          if (c >= half * H && c < half * H + H) ((T*)p.dq)[r * D + c] = from_f<T>(acc[e] * p.scale);
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
  using C = Bwd<D>;
  constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int kRegs = 128 * C::REGS_CTRL + 256 * C::REGS_WORK;
  const long long kb = part_numbers(p.nseq, p.total_k, 1, kTile);
  const long long qb = part_numbers(p.nseq, p.total_q, 1, kTile / p.group);
  if (kb * p.hk * p.max_pieces > 0x7fffffffLL || qb * p.hk > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaError_t e = prepare_kernel<packed_dkdv_tc_kernel<T, D>>(C::SMEM_ASKED, C::THREADS, kRegs);
  if (e == cudaSuccess) e = prepare_kernel<packed_dq_tc_kernel<T, D>>(C::SMEM_ASKED, C::THREADS, kRegs);
  if (e != cudaSuccess) return e;
  CUtensorMap mq, mo, mk, mv;
  if (!row_map(&mq, p.q, p, bf16) || !row_map(&mo, p.dout, p, bf16) || !key_map(&mk, p.k, p, bf16) ||
      !key_map(&mv, p.v, p, bf16))
    return cudaErrorInvalidValue;
  // dq first: it improves rows' delta on its way
  packed_dq_tc_kernel<T, D><<<(unsigned)(qb * p.hk), C::THREADS, C::SMEM_ASKED, st>>>(mq, mo, mk, mv, p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  packed_dkdv_tc_kernel<T, D>
      <<<(unsigned)(kb * p.hk * p.max_pieces), C::THREADS, C::SMEM_ASKED, st>>>(mq, mo, mk, mv, p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return p.max_pieces > 1 ? launch_packed_dkdv_join(p, bf16 ? NA_BF16 : NA_F16, st) : cudaSuccess;
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

cudaError_t launch_packed_dkdv_join(const PackedArgs& p, na_dtype dt, cudaStream_t st) {
  const long long blocks = ((long long)p.total_k * p.hk * (p.d / 8) + 255) / 256;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)blocks, 2);
  if (dt == NA_F32)
    packed_dkdv_join_kernel<float><<<grid, 256, 0, st>>>(p);
  else if (dt == NA_F16)
    packed_dkdv_join_kernel<__half><<<grid, 256, 0, st>>>(p);
  else
    packed_dkdv_join_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_packed_backward_tc(const PackedArgs& p, na_dtype dt, cudaStream_t st) {
  return dt == NA_F16 ? launch_d<__half>(p, st) : launch_d<__nv_bfloat16>(p, st);
}

}  // namespace na2d
