// Pieces of the kernels whose CTA pairs multiply 256 x 256 tiles with
// tcgen05.mma.cta_group::2: the tile's constants, descriptors, copies, and the
// tensor maps of operands and results.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstdint>
#include <mutex>

#include "fct_common.cuh"
#include "fct_internal.h"

namespace fct {
namespace pair {

constexpr int kCtaRows = 128;  // rows of A and of B each CTA of a pair stages
constexpr int kBM = 256, kBN = 256, kBK = 64;  // the pair's tile
constexpr int kGStages = 6;
constexpr uint32_t kHalfBytes = kCtaRows * kBK * 2;  // 16 KB: one operand's rows of a CTA
constexpr uint32_t kGStageBytes = 2 * kHalfBytes;     // A and B rows of a CTA
constexpr uint32_t kBoxBytes = 64 * kBK * 2;          // one 64 x 64 box of an MN-major operand
constexpr uint32_t kTmemCols = 2 * kBN;               // two fp32 accumulators of 256 columns
// A staging buffer for a result: 32 rows x 128 bytes, written in the 128-byte
// swizzle of its tensor map and sent out by TMA.
constexpr uint32_t kOutBufBytes = 32 * 128;

// Instruction descriptor of tcgen05.mma kind::f16: fp32 accumulator (bits
// 4-5 = 1), A and B bf16 (bits 7-9 and 10-12 = 1), A and B major-ness
// (bits 15 and 16: 0 K-major, 1 MN-major), N / 8 at bits 17-22, M / 16 at
// bits 24-28.
template <bool kAmn, bool kBmn>
__host__ __device__ constexpr uint32_t idesc() {
  return (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(kAmn) << 15) | (uint32_t(kBmn) << 16) |
         (uint32_t(kBN >> 3) << 17) | (uint32_t(kBM >> 4) << 24);
}

// Shared-memory matrix descriptor of a tile written by TMA with 128-byte
// swizzle (8-row atoms of 128-byte rows, 1024 bytes): start address, leading
// and stride byte offsets in 16-byte units, version 1 (bits 46-47), swizzle
// mode 2 = 128-byte (bits 61-63).
//   K-major: rows are the M (N) index, 64 K elements per row; atoms of 8
//   rows are 1024 bytes apart (stride offset); the leading offset is unused.
//   A K step of 16 advances the start by 32 bytes inside the atom.
//   MN-major: rows are the K index, 64 M (N) elements per row; atoms of 8 K
//   rows are 1024 bytes apart (stride offset), the next 64 M (N) elements
//   start one 64 x 64 box later (leading offset 8192 bytes).  A K step of 16
//   advances the start by 16 rows = 2048 bytes.
template <bool kMn>
__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr) {
  uint64_t d = uint64_t((saddr & 0x3FFFFu) >> 4);
  d |= uint64_t(kMn ? (kBoxBytes >> 4) : 1u) << 16;
  d |= uint64_t(1024 >> 4) << 32;
  d |= uint64_t(1) << 46;
  d |= uint64_t(2) << 61;
  return d;
}
template <bool kMn>
__host__ __device__ constexpr uint64_t desc_k_step() {  // one K step of 16 elements, in 16-byte units
  return kMn ? (16 * 128) >> 4 : (16 * 2) >> 4;
}

// A 2-D TMA load into this CTA's shared memory whose completion is counted
// on the mbarrier at cluster address `bar` (the pair's rank-0 CTA's).
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

// A CTA's rows of an operand for k block kb: rows r0 .. r0 + 127 of the M (N)
// index.  K-major: one box {64 K, 128}.  MN-major: two boxes {64 M (N),
// 64 K}, 8 KB apart.
template <bool kMn>
__device__ __forceinline__ void load_rows(uint32_t dst, const CUtensorMap* map, int r0, int kb,
                                          uint32_t bar) {
  if constexpr (kMn) {
#pragma unroll
    for (int j = 0; j < kCtaRows / 64; ++j)
      tma_load_2d(dst + j * kBoxBytes, map, r0 + 64 * j, kb * kBK, bar);
  } else {
    tma_load_2d(dst, map, kb * kBK, r0, bar);
  }
}

__device__ __forceinline__ uint32_t cluster_ctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The cluster address of this CTA's shared variable at `saddr` in CTA `rank`.
__device__ __forceinline__ uint32_t map_to_rank(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
               "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <uint32_t kIdesc>
__device__ __forceinline__ void umma_bf16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(kIdesc), "r"(accumulate)
      : "memory");
}

// Arrives once on the mbarrier at `bar`'s offset in both CTAs of the pair
// when every tcgen05 operation this thread issued before has completed.
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(smem_addr(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// 32 lanes x 32 consecutive 32-bit columns of tensor memory: thread i of the
// warp receives lane (lane base + i), columns [col, col + 32).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// TMA from this CTA's shared memory to C: a plain store, or an fp32 add
// performed at L2 (the read-modify-write of an accumulated C never reaches
// the SM).  Completion is tracked per thread in bulk groups.
template <bool kAdd>
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int x, int y, uint32_t src) {
  if constexpr (kAdd)
    asm volatile(
        "cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group"
        " [%0, {%1, %2}], [%3];" ::"l"(reinterpret_cast<uint64_t>(map)),
        "r"(x), "r"(y), "r"(src)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
            reinterpret_cast<uint64_t>(map)),
        "r"(x), "r"(y), "r"(src)
        : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// Waits until at most one (none) of this thread's bulk groups still reads
// shared memory.
__device__ __forceinline__ void bulk_wait_read_1() {
  asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait_read_0() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait_all() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// One thread's 128-byte row of a staging buffer, 16-byte chunk j at chunk
// position j ^ (row % 8): the 128-byte swizzle of the C tensor map, which
// also spreads a warp's chunk stores over all banks.
__device__ __forceinline__ void stage_row(uint32_t buf, int row, const uint32_t (&w)[32]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t a = buf + uint32_t(row) * 128u + uint32_t((j ^ (row & 7)) * 16);
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(w[4 * j]),
                 "r"(w[4 * j + 1]), "r"(w[4 * j + 2]), "r"(w[4 * j + 3])
                 : "memory");
  }
}

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    else
      cudaGetLastError();
  });
  return fn;
}

// Tensor map of a bf16 operand: `inner` contiguous elements per line, `outer`
// lines ld elements apart; boxes of 64 x box_outer, 128-byte swizzle, zero
// fill outside the matrix.
inline bool make_map(CUtensorMap* map, const void* base, int64_t inner, int64_t outer, int64_t ld,
              uint32_t box_outer) {
  auto encode = encode_fn();
  if (encode == nullptr) return false;
  const cuuint64_t dims[2] = {cuuint64_t(inner), cuuint64_t(outer)};
  const cuuint64_t strides[1] = {cuuint64_t(ld) * 2};
  const cuuint32_t box[2] = {64u, box_outer};
  const cuuint32_t elem[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides,
                box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// C's map for the epilogue's stores: M rows of N elements, ldc apart, boxes
// of 32 rows x 128 bytes (32 fp32 or 64 bf16), 128-byte swizzle.
inline bool make_c_map(CUtensorMap* map, void* C, int64_t M, int64_t N, int64_t ldc, bool bf16) {
  auto encode = encode_fn();
  if (encode == nullptr) return false;
  const size_t es = bf16 ? 2 : 4;
  const cuuint64_t dims[2] = {cuuint64_t(N), cuuint64_t(M)};
  const cuuint64_t strides[1] = {cuuint64_t(ldc) * es};
  const cuuint32_t box[2] = {cuuint32_t(128 / es), 32u};
  const cuuint32_t elem[2] = {1, 1};
  return encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2,
                C, dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The operand's map: K-major rows x K with boxes {64 K, tile rows};
// MN-major K lines of `rows` elements with boxes {64, 64}.
inline bool operand_map(CUtensorMap* map, const GemmOperand& x, int64_t rows, int64_t K,
                 uint32_t tile_rows) {
  return x.mn_major ? make_map(map, x.ptr, rows, K, x.ld, 64)
                    : make_map(map, x.ptr, K, rows, x.ld, tile_rows);
}

}  // namespace pair
}  // namespace fct
