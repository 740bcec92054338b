// Head-indexed tensor maps and TMEM load helpers of the tcgen05 attention
// kernels.
//
// A row of q|k|v (or of O, dO, dq|dk|dv) is a sequence of heads of hd
// bf16 values; the maps below describe it as [rows][heads][hd], so a tile is
// addressed as (0, head, row) and its box is always 64 values wide with
// 128-byte swizzle, the layout the kernels' UMMA descriptors expect.  For
// hd = 64 the box is exactly one head.  For hd = 32 the box reaches past the
// head's 32 values, which lie outside the tensor's innermost extent: a load
// fills them with zeros (so Q K^T, P V, dO V^T and the row sums dO . O are
// the head-32 values, and the products' columns 32..63 are zero) and a store
// skips them (only the head's own 32 columns are written).  The
// packed kernels take any multiple of 8 so (past 64, forward, as two boxes).
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstdint>

#include "packed.cuh"
#include "tcgen05.cuh"

namespace llm {
namespace attn_maps {

// What a kernel over packed sequences gets besides the tensor maps: the work
// plan, the row count (stride of the heads in lse and D) and the output rows
// for tiles that a sequence's end cuts.
struct PkView {
  int *n_tiles;  // [0] tiles of the plan, [2] counter of the queue
  const PkTile *tiles;
  int64_t n_rows;
  __nv_bfloat16 *out;
  int64_t out_ld;
  // without a plan (tiles null): the offsets, one item a block
  const int32_t *cu;
  int n_seq;
  // backward: L beside D, and the stride of their heads (PkPlan)
  float *L;
  int64_t stat;
};
// One work item: 128-row block (query or key), head, sequence.
struct Item {
  int blk, h, b, row0, T, seq;
};
// (tile: what pk_find gave, for a block's only item)
LLM_DEV Item pk_item(const PkView &pk, const int4 &tile, int item, int heads, bool keys) {
  const int4 t = pk.tiles ? ld_int4(pk.tiles + item / heads) : tile;
  const int n = (t.y + PK_BLOCK - 1) / PK_BLOCK;
  // (the plan's tiles carry the sequence, pk_find's the sequence + 1)
  return Item{keys ? n - 1 - t.z : t.z, item % heads, 0, t.x, t.y, pk.tiles ? t.w : t.w - 1};
}
// Rows [first, 32) of the 32-row group at `rows` (128-byte rows) to zero, by
// the 128 threads of the group's four warps (t = 0 .. 127): the rows of a
// tile past its sequence's end belong to another sequence or to none, and
// 0 * NaN is NaN in a product.
LLM_DEV void zero_rows(uint8_t *rows, int first, int t) {
  if ((t >> 2) >= first) {
    uint4 *p = reinterpret_cast<uint4 *>(rows + (t >> 2) * 128 + (t & 3) * 32);
    p[0] = p[1] = make_uint4(0, 0, 0, 0);
  }
  tc::fence_proxy_async();
}
// The staged rows [r0, r0 + 8) of a 128-byte-swizzled tile that lie before
// `end`, head columns [0, hd), to out (row r0 of the tile; row stride ld).
LLM_DEV void store_cut(const uint8_t *tile, int r0, int end, __nv_bfloat16 *out, int64_t ld, int hd,
                       int lane) {
  const int r = r0 + (lane >> 2);
  if (r >= end) return;
#pragma unroll
  for (int k = 0; k < 2; k++) {
    const int c = (lane & 3) + 4 * k;
    if (c * 8 < hd)
      *reinterpret_cast<uint4 *>(out + (int64_t)(lane >> 2) * ld + c * 8) =
          *reinterpret_cast<const uint4 *>(tile + r * 128 + ((c ^ (r & 7)) << 4));
  }
}

LLM_DEV void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"((uint64_t)map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// Bulk tensor store of a staged box (the caller commits the group).
LLM_DEV void tma_store_4d(const CUtensorMap *map, uint32_t src, int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(
          (uint64_t)map),
      "r"(x), "r"(y), "r"(z), "r"(w), "r"(src)
      : "memory");
}

// TMEM loads without their own wait (32x32b shape: lane = row, N columns
// of 32 bits), so several can be in flight; tmem_wait_regs waits for all of
// them and re-defines each loaded register after the wait, so no use of one
// can be scheduled before it.
template <int N>
LLM_DEV void tmem_ld_raw(uint32_t taddr, uint32_t (&r)[N]) {
  static_assert(N == 8 || N == 16 || N == 32, "8, 16 or 32 columns");
  if constexpr (N == 8) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
  } else if constexpr (N == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
  }
}
// A pair of equal loads (two TMEM regions of this thread's lane) under one wait.
template <int N>
LLM_DEV void tmem_ld_pair(uint32_t a, uint32_t b, float (&va)[N], float (&vb)[N]) {
  uint32_t ra[N], rb[N];
  tmem_ld_raw<N>(a, ra);
  tmem_ld_raw<N>(b, rb);
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; i++) {
    asm volatile("" : "+r"(ra[i]), "+r"(rb[i]));
    va[i] = __uint_as_float(ra[i]);
    vb[i] = __uint_as_float(rb[i]);
  }
}
LLM_DEV void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
template <int N>
LLM_DEV void tmem_after_wait(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; i++) asm volatile("" : "+r"(r[i]));
}

inline PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    cudaDriverEntryPointQueryResult q;
    void *fn = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return (PFN_cuTensorMapEncodeTiled_v12000) nullptr;
    return (PFN_cuTensorMapEncodeTiled_v12000)fn;
  }();
  return encode;
}

// Loads: [rows][heads][hd] over a row-major [rows][ld] bf16 array (ld a
// multiple of 8, at least heads * hd), box 64 x 1 head x box_rows rows.
inline bool head_map_load(CUtensorMap *map, const void *base, int hd, int64_t heads, int64_t rows,
                          int64_t ld, int box_rows) {
  auto encode = encoder();
  if (!encode || ((uintptr_t)base & 15) || hd < 8 || hd > 128 || hd % 8 || ld < heads * hd || ld % 8)
    return false;
  cuuint64_t dims[3] = {(cuuint64_t)hd, (cuuint64_t)heads, (cuuint64_t)rows};
  cuuint64_t strides[2] = {(cuuint64_t)hd * 2, (cuuint64_t)ld * 2};
  cuuint32_t box[3] = {64, 1, (cuuint32_t)box_rows};
  cuuint32_t es[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides,
                box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Stores: [batches][T][heads][hd] over a row-major [batches * T][ld] bf16
// array (ld as above), box 64 x 1 head x box_rows rows x 1 batch (rows past T, and a
// head-32 box's upper 32 values, are not written).
inline bool head_map_store(CUtensorMap *map, void *base, int hd, int64_t heads, int64_t T,
                           int64_t batches, int64_t ld, int box_rows) {
  auto encode = encoder();
  if (!encode || ((uintptr_t)base & 15) || hd < 8 || hd > 128 || hd % 8 || ld < heads * hd || ld % 8)
    return false;
  cuuint64_t dims[4] = {(cuuint64_t)hd, (cuuint64_t)heads, (cuuint64_t)T, (cuuint64_t)batches};
  cuuint64_t strides[3] = {(cuuint64_t)hd * 2, (cuuint64_t)ld * 2, (cuuint64_t)(ld * T * 2)};
  cuuint32_t box[4] = {64, 1, (cuuint32_t)box_rows, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, box, es,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace attn_maps
}  // namespace llm
