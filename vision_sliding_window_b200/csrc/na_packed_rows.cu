// na_packed_rows.cu -- the packed attention of few rows over many keys, fp16
// and bf16: single tokens (and a few more) over a cache.
//
// Every key and value is read once for the rows of its group, 2 d FLOPs a
// row and key: HBM bounds it, and what matters is how many bytes an SM has in
// flight.  Keys and values come through a ring of TMA tiles of 64 keys, filled
// by a warp of its own, about 100 KB ahead a block and two blocks an SM (loads
// into registers, as deep as those allow, reached 4.1 of 6.5 TB/s).  Four warps
// take 16 keys of a tile each, with a running maximum and sum of their own, for
// m16n8k16 products.  A product's contraction index and its output columns may
// be numbered in any order, so a thread takes 16-byte pieces of the swizzled
// rows, chosen to fall on distinct banks, and calls them its own indices.  The
// rows of a group fill a 16-row operand only in part; the idle rows cost tensor
// time that nothing waits for (tcgen05's 128-row tiles would be 1/32 full).
//
// The keys of a sequence are shared by a cluster of 8 blocks, which join their
// parts through each other's shared memory: no second kernel and no workspace.
// Where sequences times heads are too few for that to fill the SMs, keys are
// cut into pieces, one a block, which a second kernel joins.
#include "na_packed_tc.cuh"

namespace na2d {
namespace {

using namespace packed;

constexpr int kWarps = 4, kThreads = 32 * kWarps + 32;  // and the loading warp
constexpr int kTileKeys = 64, kCluster = 8;
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

// N 32-bit words of consecutive elements
template <int N> NA_DEVICE void words_of_row(uint32_t (&r)[N], const void* from, bool live) {
  if constexpr (N == 4) {
    const uint4 u = live ? __ldg((const uint4*)from) : make_uint4(0, 0, 0, 0);
    r[0] = u.x, r[1] = u.y, r[2] = u.z, r[3] = u.w;
  } else {
    const uint2 u = live ? __ldg((const uint2*)from) : make_uint2(0, 0);
    r[0] = u.x, r[1] = u.y;
  }
}
template <int N> NA_DEVICE void words_of_tile(uint32_t (&r)[N], uint32_t at) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(at));
  else
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r[0]) : "r"(at));
}

NA_DEVICE uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Every block of a cluster comes to each of these, also when it gave up a wait.
NA_DEVICE void cluster_meet() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
NA_DEVICE float ld_cluster(const float* mine, uint32_t rank) {
  uint32_t at;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(mine)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at));
  return v;
}

// Geometry of a tile of 64 keys: column blocks of 64 rows of ROWB bytes, whose
// 16-byte pieces TMA swizzles by the row.
template <int D> struct Rows {
  static constexpr int BLOCKS = Geo<D>::BLOCKS, COLS = Geo<D>::COLS, ROWB = Geo<D>::ROWB;
  static constexpr int TILE_BYTES = kTileKeys * D * 2;
  static constexpr int STAGES = 100 * 1024 / (2 * TILE_BYTES) > 8 ? 8 : 100 * 1024 / (2 * TILE_BYTES);
  static constexpr int KE = D >= 32 ? 8 : 4;   // consecutive columns of a key a thread takes
  static constexpr int KC = D / (4 * KE);      // of which it takes this many runs
  static constexpr int VE = D >= 64 ? 8 : D / 8;  // the same for values
  static constexpr int VC = D / (8 * VE);
  static constexpr int LD = D + 4;
  // the join's sums take the ring's place
  static constexpr int SUM_BYTES = kWarps * 16 * LD * 4;
  static constexpr int RING_BYTES = STAGES * 2 * TILE_BYTES;
  static constexpr int SMEM = (RING_BYTES > SUM_BYTES ? RING_BYTES : SUM_BYTES) + 1024;

  // Byte `byte` of row `row` of a tile, moved as the swizzle moves its piece:
  // the piece's number XOR the row's number in its group of 8 (4, 2) rows.
  NA_DEVICE static uint32_t at(uint32_t tile, int row, int col) {
    const int block = BLOCKS > 1 ? col / COLS : 0;
    const uint32_t byte = (uint32_t)(col - block * COLS) * 2, piece = byte >> 4;
    const uint32_t turn = ROWB == 128 ? row & 7 : ROWB == 64 ? (row >> 1) & 3 : (row >> 2) & 1;
    return tile + block * kTileKeys * ROWB + row * ROWB + ((piece ^ turn) << 4) + (byte & 15);
  }
  // First column of run c of the q-th thread of a row.  At 64 columns a block
  // the four threads take every other piece, and neighbouring rows' turns differ
  // in the lowest bit: eight threads of two rows read eight distinct pieces.
  NA_DEVICE static int key_col(int c, int q) {
    return ROWB == 128 ? (c / 2) * COLS + (2 * q + (c & 1)) * KE : c * 4 * KE + q * KE;
  }
  NA_DEVICE static int value_col(int c, int g) { return c * 8 * VE + g * VE; }
};

template <typename T, int D, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, 2)
packed_rows_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const PackedArgs p) {
  using R = Rows<D>;
  extern __shared__ uint8_t raw[];
  __shared__ uint64_t bars[16];
  __shared__ float sm[kWarps][16], sl[kWarps][16], jm[16], jl[16];
  __shared__ volatile int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const float sl2 = p.scale * kLog2e;
  const uint32_t rank = CLUSTER ? cluster_rank() : 0;
  int s, kh;
  long long idx = 0;
  if constexpr (CLUSTER) {
    const int unit = blockIdx.x / kCluster;
    s = unit / p.hk;
    kh = unit - s * p.hk;
  } else {
    kh = blockIdx.x % p.hk;
    find_part_warp(p.cu_k, p.nseq, p.total_k, 1, p.piece_keys, blockIdx.x / p.hk, &s, &idx);
    if (idx < 0) return;
  }
  const Span sp = span_of(p, s);
  const long long all_rows = (long long)sp.nq * p.group;
  if (all_rows == 0) return;  // the whole cluster
  int piece0 = 0, piece1 = sp.nk;
  if (!CLUSTER) {
    if (idx >= p.max_pieces || idx * p.piece_keys >= sp.nk) return;
    piece0 = (int)idx * p.piece_keys;
    piece1 = (int)min((long long)piece0 + p.piece_keys, (long long)sp.nk);
  }
  const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
  float* so = reinterpret_cast<float*>(raw + (base - smem_addr(raw)));  // [kWarps][16][LD]
  const uint32_t bar0 = smem_addr(bars);
  auto full = [&](int i) { return bar0 + (i % R::STAGES) * 8; };
  auto empty = [&](int i) { return bar0 + (R::STAGES + i % R::STAGES) * 8; };
  auto k_tile = [&](int i) { return base + (i % R::STAGES) * 2 * R::TILE_BYTES; };
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < R::STAGES; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), kWarps);
    }
    mbar_init_fence();
  }
  __syncthreads();
  const long long stride = (long long)p.hk * D;
  const T* kbase = (const T*)p.k + ((long long)sp.k0 * p.hk + kh) * D;
  const T* vbase = (const T*)p.v + ((long long)sp.k0 * p.hk + kh) * D;
  int done = 0;  // tiles of earlier row tiles, which went through the ring too
  for (long long r0 = 0; r0 < all_rows; r0 += 16) {
    // After a wait was given up the ring's barriers mean nothing.  The block
    // still walks the rows, without tiles: its cluster meets at every one.
    const bool gave_up = abort_flag;
    const int n = (int)min(16ll, all_rows - r0);
    int kb, ke, unused;
    visible(p, sp, (int)(r0 / p.group), &kb, &unused);
    visible(p, sp, (int)((r0 + n - 1) / p.group), &unused, &ke);
    kb = max(kb, piece0);
    ke = min(ke, piece1);
    if constexpr (CLUSTER) {  // this block's share, in whole tiles
      const int tiles = ke > kb ? (ke - kb + kTileKeys - 1) / kTileKeys : 0;
      const int from = kb + (int)((long long)tiles * rank / kCluster) * kTileKeys;
      ke = min(ke, kb + (int)((long long)tiles * (rank + 1) / kCluster) * kTileKeys);
      kb = from;
    }
    const int tiles = ke > kb && !gave_up ? (ke - kb + kTileKeys - 1) / kTileKeys : 0;
    if (warp == kWarps) {
      // --------------------------------------------------------------- loads
      int i = 0;
      for (; i < tiles; ++i) {
        const int u = done + i;
        if (u >= R::STAGES && !mbar_wait(empty(u), ((u / R::STAGES) - 1) & 1, &abort_flag, p.status)) break;
        if (lane == 0) {
          mbar_expect_tx(full(u), 2 * R::TILE_BYTES);
#pragma unroll
          for (int b = 0; b < R::BLOCKS; ++b) {
            const uint32_t to = k_tile(u) + b * kTileKeys * R::ROWB;
            tma_load_3d(to, &mk, full(u), b * R::COLS, kh, sp.k0 + kb + i * kTileKeys);
            tma_load_3d(to + R::TILE_BYTES, &mv, full(u), b * R::COLS, kh, sp.k0 + kb + i * kTileKeys);
          }
        }
        __syncwarp();
      }
      settle_ring(done, i, R::STAGES, full);
    } else {
      // this thread's rows g and g + 8: where they lie and what they see
      int lo[2], hi[2];
      uint32_t qa[R::KC][R::KE / 4][4];  // their operand, columns numbered as the keys' are; idle rows are zero
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const long long r = r0 + min(g + 8 * h, n - 1);
        const int pos = (int)(r / p.group);
        visible(p, sp, pos, &lo[h], &hi[h]);
        if (g + 8 * h >= n) hi[h] = lo[h];
        const T* row =
            (const T*)p.q + (((long long)sp.q0 + pos) * p.hq + kh * p.group + (int)(r - (long long)pos * p.group)) * D;
#pragma unroll
        for (int c = 0; c < R::KC; ++c) {
          uint32_t w[R::KE / 2];
          words_of_row(w, row + R::key_col(c, q), g + 8 * h < n);
#pragma unroll
          for (int x = 0; x < R::KE / 4; ++x) qa[c][x][h] = w[2 * x], qa[c][x][2 + h] = w[2 * x + 1];
        }
      }
      float o[R::VC][R::VE][4], ref[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
#pragma unroll
      for (int c = 0; c < R::VC; ++c)
#pragma unroll
        for (int i = 0; i < R::VE; ++i)
#pragma unroll
          for (int x = 0; x < 4; ++x) o[c][i][x] = 0.f;
      for (int it = 0; it < tiles; ++it) {
        const int u = done + it, j0 = kb + it * kTileKeys + warp * 16;
        if (!mbar_wait(full(u), (u / R::STAGES) & 1, &abort_flag, p.status)) break;
        const uint32_t ks = k_tile(u), vs = ks + R::TILE_BYTES;
        float sc[2][4] = {};
#pragma unroll
        for (int c = 0; c < R::KC; ++c)
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            uint32_t kr[R::KE / 2];
            words_of_tile(kr, R::at(ks, warp * 16 + nt * 8 + g, R::key_col(c, q)));
#pragma unroll
            for (int x = 0; x < R::KE / 4; ++x)
              mma16816<T>(sc[nt], qa[c][x][0], qa[c][x][1], qa[c][x][2], qa[c][x][3], kr[2 * x], kr[2 * x + 1]);
          }
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
              for (int x = 0; x < 4; ++x) o[c][i][x] *= f[x >> 1];  // NaN stays, also under 0
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
        const bool cut = j0 + 16 > ke;  // values past the keys are not numbers to be trusted
#pragma unroll
        for (int c = 0; c < R::VC; ++c) {
          uint32_t vr[4][(R::VE + 1) / 2];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = (e >> 1) * 8 + 2 * q + (e & 1);
            words_of_tile(vr[e], R::at(vs, warp * 16 + key, R::value_col(c, g)));
            if (cut && j0 + key >= ke)
#pragma unroll
              for (int i = 0; i < (R::VE + 1) / 2; ++i) vr[e][i] = 0u;
          }
#pragma unroll
          for (int i = 0; i < R::VE; ++i) {
            // column i of this thread's run, of keys (2q, 2q+1) and (2q+8, 2q+9)
            const uint32_t pick = (i & 1) ? 0x7632u : 0x5410u;
            mma16816<T>(o[c][i], pa[0], pa[1], pa[2], pa[3], __byte_perm(vr[0][i / 2], vr[1][i / 2], pick),
                        __byte_perm(vr[2][i / 2], vr[3][i / 2], pick));
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty(u));
      }
      // ----------------------------------------------- this warp's part
      __syncwarp();
      asm volatile("bar.sync 1, 128;" ::: "memory");  // all four warps have read the ring
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
            so[(warp * 16 + g + 8 * (x >> 1)) * R::LD + R::value_col(c, 2 * q + (x & 1)) + i] = o[c][i][x];
    }
    done += tiles;
    __syncthreads();
    // the block's sums over its warps, in the first warp's place
    if (warp < kWarps)
      for (int r = warp; r < n; r += kWarps) {
        float m = -INFINITY, f[kWarps], l = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm[w][r]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          f[w] = sm[w][r] == m ? 1.f : exp2f((sm[w][r] - m) * sl2);
          l += sl[w][r] * f[w];
        }
#pragma unroll
        for (int e = 0; e < (D + 31) / 32; ++e) {
          if (lane + 32 * e >= D) continue;
          float acc = 0.f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w)
            acc = fmaf(so[(w * 16 + r) * R::LD + lane + 32 * e], f[w], acc);
          so[r * R::LD + lane + 32 * e] = acc;
        }
        if (lane == 0) jm[r] = m, jl[r] = l;
      }
    if constexpr (CLUSTER)
      cluster_meet();
    else
      __syncthreads();
    // a warp a row: over the cluster's blocks, which take the rows in turn
    const int workers = CLUSTER ? kCluster * kWarps : kWarps;
    if (warp < kWarps)
      for (int r = (int)rank * kWarps + warp; r < n; r += workers) {
        constexpr int B = CLUSTER ? kCluster : 1;
        float m = -INFINITY, f[B], l = 0.f, bm[B];
#pragma unroll
        for (int b = 0; b < B; ++b) {
          bm[b] = CLUSTER ? ld_cluster(&jm[r], b) : jm[r];
          m = fmaxf(m, bm[b]);
        }
#pragma unroll
        for (int b = 0; b < B; ++b) {
          f[b] = bm[b] == m ? 1.f : exp2f((bm[b] - m) * sl2);
          l += (CLUSTER ? ld_cluster(&jl[r], b) : jl[r]) * f[b];
        }
        float acc[(D + 31) / 32];
        bool finite = fabsf(l) < INFINITY;
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int e = 0; e < (D + 31) / 32; ++e) {
          acc[e] = 0.f;
          if (lane + 32 * e < D)
#pragma unroll
            for (int b = 0; b < B; ++b) {
              const float* at = so + r * R::LD + lane + 32 * e;
              const float v = CLUSTER ? ld_cluster(at, b) : *at;
              acc[e] = fmaf(v, f[b], acc[e]);
            }
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
          exact_row<T, D>(p, (const T*)p.q + row * D, kbase, vbase, stride, max(a, piece0), min(b, piece1), acc, &lse);
        }
        const long long at = CLUSTER ? row : (idx * p.total_q + i) * p.hq + head;
#pragma unroll
        for (int e = 0; e < (D + 31) / 32; ++e)
          if (lane + 32 * e < D) {
            if (CLUSTER)
              ((T*)p.out)[at * D + lane + 32 * e] = from_f<T>(acc[e]);
            else
              p.part_o[at * D + lane + 32 * e] = acc[e];
          }
        if (lane == 0) {
          if (!CLUSTER)
            p.part_lse[at] = lse;
          else if (p.lse)
            p.lse[(long long)head * p.total_q + i] = lse;
        }
      }
    // the sums are read before the ring is filled again, or the block ends
    fence_async_smem();
    if constexpr (CLUSTER)
      cluster_meet();
    else
      __syncthreads();
  }
}

template <typename T, int D, bool CLUSTER>
cudaError_t launch_one(const PackedArgs& p, long long blocks, cudaStream_t st) {
  constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int smem = Rows<D>::SMEM;
  static_assert(2 * (smem + 2048) <= kMaxSmem, "two blocks an SM");
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaError_t e = prepare_kernel<packed_rows_kernel<T, D, CLUSTER>>(smem, kThreads, 0);
  if (e != cudaSuccess) return e;
  CUtensorMap mk, mv;
  if (!key_map(&mk, p.k, p, bf16, kTileKeys) || !key_map(&mv, p.v, p, bf16, kTileKeys)) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = kCluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = CLUSTER ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, packed_rows_kernel<T, D, CLUSTER>, mk, mv, p);
}
template <typename T, int D> cudaError_t launch(const PackedArgs& p, cudaStream_t st) {
  if (p.piece_keys > 0)
    return launch_one<T, D, false>(p, part_numbers(p.nseq, p.total_k, 1, p.piece_keys) * p.hk, st);
  return launch_one<T, D, true>(p, (long long)p.nseq * p.hk * kCluster, st);
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
