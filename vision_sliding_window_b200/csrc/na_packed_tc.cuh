// na_packed_tc.cuh -- what the tensor-core kernels of the packed attention
// share: tile geometry, tensor maps, descriptors and shared-memory tiles.
//
// A tile is 128 rows of D 16-bit elements, in D / 64 (at least 1) column
// blocks of 128 swizzled rows, as TMA writes it and tcgen05 reads it.  Key
// tiles are 128 keys of one key head.  Row tiles are P = 128 / G positions
// times the G query heads of a key head, row = position * G + head, which in
// q [total_q][hk][G][d] is one box of P x 1 x G x d; rows past P * G of a tile
// hold nothing and nothing is read from them.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>
#include <type_traits>

#include "na2d_sm100.cuh"
#include "na_packed.cuh"

namespace na2d {
namespace packed {

using namespace sm100;

constexpr int kTile = 128;
constexpr int kMaxSmem = 227 * 1024;

template <int D> struct Geo {
  static constexpr int BLOCKS = D > 64 ? D / 64 : 1;
  static constexpr int COLS = D / BLOCKS;        // columns of a block
  static constexpr int ROWB = COLS * 2;          // bytes of a row of a block
  static constexpr int BLOCK_BYTES = kTile * ROWB;
  static constexpr int TILE_BYTES = BLOCKS * BLOCK_BYTES;
  static constexpr uint32_t LAYOUT = ROWB == 128 ? kLayoutSW128 : ROWB == 64 ? kLayoutSW64 : kLayoutSW32;
};

// Operand descriptors, split in halves: the low word holds the address and the
// leading offset, so that a step inside a tile is one 32-bit addition; the
// high word is a constant.  One thread issues all MMAs of a block, and what it
// computes between two of them is time that the tensor pipe may wait.
template <int D> struct KMajor {  // rows x D, 16 columns a step
  using G = Geo<D>;
  static constexpr uint32_t HI = (8 * G::ROWB >> 4) | 1u << 14 | G::LAYOUT << 29;
  static constexpr int PER = G::COLS / 16;
  NA_DEVICE static uint32_t lo(uint32_t tile) { return (tile >> 4) | 1u << 16; }
  static constexpr uint32_t step(int kk) { return ((kk / PER) * G::BLOCK_BYTES + (kk % PER) * 32) >> 4; }
};
template <int D> struct MnMajor {  // D x rows, 16 rows a step
  using G = Geo<D>;
  static constexpr uint32_t HI = KMajor<D>::HI;
  NA_DEVICE static uint32_t lo(uint32_t tile) { return (tile >> 4) | (uint32_t)(G::BLOCK_BYTES >> 4) << 16; }
  static constexpr uint32_t step(int kk) { return (kk * 16 * G::ROWB) >> 4; }
};
NA_DEVICE void mma_ss_lo(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.b32 p, %5, 0;\n mov.b64 x, {%1, %3};\n mov.b64 y, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
NA_DEVICE void mma_ts_lo(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 y;\n setp.ne.b32 p, %5, 0;\n mov.b64 y, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}

// D[128 x 128] = A B^T over D columns, both tiles K-major.
template <int D, bool BF16> NA_DEVICE void mma_rows_by_rows(uint32_t d, uint32_t a, uint32_t b) {
  constexpr uint32_t idesc = idesc_f16(BF16, kTile, kTile, false);
  const uint32_t x = KMajor<D>::lo(a), y = KMajor<D>::lo(b);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk)
    mma_ss_lo(d, x + KMajor<D>::step(kk), y + KMajor<D>::step(kk), KMajor<D>::HI, idesc, kk > 0);
}
// D[128 x D] (+)= A B, A 128 x 128 of 16 bits in tensor memory, B a tile; the
// second half of A's columns begins GAP columns after the first; steps FROM to
// TO of 16 rows of B.
template <int D, bool BF16, int GAP = 32, int FROM = 0, int TO = 8>
NA_DEVICE void mma_weights_by_tile(uint32_t d, uint32_t a, uint32_t b, bool add) {
  constexpr uint32_t idesc = idesc_f16(BF16, kTile, D, true);
  const uint32_t y = MnMajor<D>::lo(b);
#pragma unroll
  for (int kk = FROM; kk < TO; ++kk)
    mma_ts_lo(d, a + (kk / 4) * GAP + (kk % 4) * 8, y + MnMajor<D>::step(kk), MnMajor<D>::HI, idesc, add || kk > 0);
}

// All column blocks of 128 keys from key `row` on of head kh.
template <int D> NA_DEVICE void load_key_tile(uint32_t dst, const CUtensorMap* m, uint32_t bar, int kh, int row) {
  using G = Geo<D>;
#pragma unroll
  for (int b = 0; b < G::BLOCKS; ++b) tma_load_3d(dst + b * G::BLOCK_BYTES, m, bar, b * G::COLS, kh, row);
}
// All column blocks of the row tile of key head kh whose first position is `pos`.
template <int D> NA_DEVICE void load_row_tile(uint32_t dst, const CUtensorMap* m, uint32_t bar, int kh, int pos) {
  using G = Geo<D>;
#pragma unroll
  for (int b = 0; b < G::BLOCKS; ++b) tma_load_4d(dst + b * G::BLOCK_BYTES, m, bar, b * G::COLS, 0, kh, pos);
}
// Zeros the rows [from, 128) of a tile, by a warp; rows are whole under the
// swizzle, which moves 16-byte pieces inside a row.
template <int D> NA_DEVICE void zero_rows(uint32_t tile, int from) {
  using G = Geo<D>;
  constexpr int PER = G::ROWB / 16;
  const int lane = threadIdx.x & 31;
  for (int e = from * PER + lane; e < kTile * PER; e += 32)
#pragma unroll
    for (int b = 0; b < G::BLOCKS; ++b)
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tile + b * G::BLOCK_BYTES + e * 16), "r"(0u)
                   : "memory");
  fence_async_smem();
}

// One tile of a ring, by a warp: `load` starts the copies of `bytes` to the slot
// on a barrier.  Of a sequence's last tile, rows `left` to `rows`, which are not
// the sequence's, are zeroed before the slot counts as full: neither a zero
// weight nor a zero gradient stops a NaN.  `tail` is a barrier for that copy
// (two of them, one for each of two rings: it completes when both have landed).
template <int D, typename F>
NA_DEVICE bool load_ring_tile(uint32_t slot, uint32_t full, uint32_t tail, int left, int rows, uint32_t bytes,
                              volatile int* ab, unsigned* status, F load) {
  const int lane = threadIdx.x & 31;
  const bool cut = left < rows;
  if (lane == 0) {
    mbar_expect_tx(cut ? tail : full, bytes);
    load(slot, cut ? tail : full);
  }
  __syncwarp();
  if (!cut) return true;
  if (!mbar_wait(tail, 0, ab, status)) {
    mbar_wait_settle(tail, 0);
    return false;
  }
  zero_rows<D>(slot, left);
  __syncwarp();
  if (lane == 0) mbar_arrive(full);
  return true;
}

// The last thing a loading warp does: of the tiles that it asked for, `count`
// from the `first` on, the last `slots` may still be on their way, also where a
// wait was given up.  A copy that landed after its block has ended would write
// another block's memory.
template <typename F> NA_DEVICE void settle_ring(int first, int count, int slots, F full) {
  for (int u = first + max(0, count - slots); u < first + count; ++u) mbar_wait_settle(full(u), (u / slots) & 1);
}

// 2^x without the special-function unit, which bounds a softmax fed by the
// tensor cores: x = n + f with n the nearest integer, 2^f by the polynomial of
// degree 4 that meets it at the five Chebyshev points of [-1/2, 1/2] (off by at
// most 4e-6, a hundredth of the rounding of a 16-bit weight), n added to the
// exponent.  For x < 127; below -126 (-inf too) it gives about 2^-126, and for
// NaN a number too large for 16 bits.
NA_DEVICE void exp2_poly2(float& a, float& b) {
  constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer
  constexpr float c0 = 1.f, c1 = 0.693121016f, c2 = 0.240223497f, c3 = 0.0559219755f, c4 = 0.00966636837f;
  const float xa = max_nan(a, -126.f), xb = max_nan(b, -126.f);
  float ta, tb, fa, fb, pa, pb;
  add2(ta, tb, xa, xb, kMagic, kMagic);
  add2(fa, fb, ta, tb, -kMagic, -kMagic);
  fma2(fa, fb, fa, fb, -1.f, -1.f, xa, xb);
  fma2(pa, pb, fa, fb, c4, c4, c3, c3);
  fma2(pa, pb, pa, pb, fa, fb, c2, c2);
  fma2(pa, pb, pa, pb, fa, fb, c1, c1);
  fma2(pa, pb, pa, pb, fa, fb, c0, c0);
  a = __uint_as_float(__float_as_uint(pa) + (__float_as_uint(ta) << 23));
  b = __uint_as_float(__float_as_uint(pb) + (__float_as_uint(tb) << 23));
}

// ------------------------------------------------------------------ host
inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    cudaDriverEntryPointQueryResult q;
    void* f = nullptr;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}
inline CUtensorMapSwizzle swizzle_of(int row_bytes) {
  return row_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                          : row_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B;
}
// [total_k][hk][d] with a box of `keys` keys of one head.
inline bool key_map(CUtensorMap* m, const void* base, const PackedArgs& p, bool bf16, int keys = kTile) {
  auto enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)p.d, (cuuint64_t)p.hk, (cuuint64_t)p.total_k};
  const cuuint64_t strides[2] = {(cuuint64_t)p.d * 2, (cuuint64_t)p.hk * p.d * 2};
  const cuuint32_t box[3] = {(cuuint32_t)(p.d > 64 ? 64 : p.d), 1, (cuuint32_t)keys};
  const cuuint32_t one[3] = {1, 1, 1};
  return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
             const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             swizzle_of(2 * (int)box[0]), CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// [total_q][hk][G][d] with a box of P positions of one key head's G heads.
inline bool row_map(CUtensorMap* m, const void* base, const PackedArgs& p, bool bf16) {
  auto enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)p.d, (cuuint64_t)p.group, (cuuint64_t)p.hk, (cuuint64_t)p.total_q};
  const cuuint64_t strides[3] = {(cuuint64_t)p.d * 2, (cuuint64_t)p.group * p.d * 2, (cuuint64_t)p.hq * p.d * 2};
  const cuuint32_t box[4] = {(cuuint32_t)(p.d > 64 ? 64 : p.d), (cuuint32_t)p.group, 1,
                             (cuuint32_t)(kTile / p.group)};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
             const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             swizzle_of(2 * (int)box[0]), CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Sets a kernel's shared memory once on a device, and checks that the
// registers that setmaxnreg hands out are those of the launch: a sum above
// them would wait forever.
template <auto KERNEL> cudaError_t prepare_kernel(int smem, int threads, int regs_handed_out) {
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(mu);
  if (done[dev]) return cudaSuccess;
  cudaFuncAttributes fa;
  cudaError_t e = cudaFuncGetAttributes(&fa, KERNEL);
  if (e != cudaSuccess) return e;
  if (regs_handed_out > fa.numRegs * threads) return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) done[dev] = true;
  return e;
}

}  // namespace packed
}  // namespace na2d
