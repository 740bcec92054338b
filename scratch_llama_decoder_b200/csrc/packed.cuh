// Packed sequences: rows of several sequences end to end in one array, rows
// [cu[s], cu[s+1]) belonging to sequence s.  Shared by the packed attention
// kernels (work plan in the caller's workspace) and the paged cache.
#pragma once
#include "common.cuh"

namespace llm {

constexpr int PK_BLOCK = 128;             // rows of a work tile
constexpr int64_t PK_MAX_ROWS = 1 << 20;  // packed rows of one call
constexpr int PK_MAX_SEQ = 65536;         // sequences of one call
// bits OR-ed into the caller's flag word (FLAG_TIMEOUT is bit 4)
enum : int { PK_BAD_OFFSETS = 1, PK_BAD_PAGE = 2 };

// One 128-row tile of a sequence: first packed row and length of the sequence,
// block index within it, the sequence.  As a key tile the same entry stands for
// block n - 1 - blk (n blocks), whose query blocks are as many.
struct PkTile {
  int row0, len, blk, seq;
};
// The workspace: tile count, a flag word for callers without one, the counter
// of a queue of items (cleared by the plan); then the tiles (most work first), then scratch
// of the plan (clamped offsets, ranks), then D of the backward.
struct PkPlan {
  int *n_tiles;
  PkTile *tiles;
  int *off, *rank;
  // the backward's statistics: [H][n_rows] D, or [2: D, L][H][stat] with every
  // sequence's first row on 16 bytes (row r of sequence s at (row0 + 3 s) / 4 * 4
  // + r), for bulk copies of 128 rows
  float *D;
  int64_t stat;
  int64_t cap, bytes;
};
inline PkPlan pk_plan(void *ws, int64_t n_rows, int n_seq, int H, bool backward) {
  PkPlan p;
  uint8_t *b = (uint8_t *)ws;
  const int64_t nonempty = n_seq < n_rows ? n_seq : n_rows;
  p.cap = n_rows / PK_BLOCK + nonempty;
  int64_t at = 0;
  auto take = [&](int64_t n) {
    uint8_t *q = b + at;
    at = (at + n + 255) / 256 * 256;
    return q;
  };
  p.n_tiles = (int *)take(12);
  p.tiles = (PkTile *)take(p.cap * (int64_t)sizeof(PkTile));
  p.off = (int *)take(4 * ((int64_t)n_seq + 1));
  p.rank = (int *)take(4 * (int64_t)n_seq);
  p.stat = (n_rows + 3 * (int64_t)n_seq + 256 + 3) / 4 * 4;
  p.D = (float *)take(backward ? 2 * 4 * p.stat * H : 0);
  p.bytes = at;
  return p;
}

// Without a plan, where every block gets one item at most: tile k (in the
// sequences' order) of `block` rows, found by a whole warp from the offsets
// themselves, clamped as the plan clamps them.  {first row, length, block,
// sequence + 1 or 0 for no such tile}.
LLM_DEV int4 pk_find(const int32_t *cu, int n_seq, int n_rows, int block, int k, int *flag) {
  const int lane = threadIdx.x & 31;
  if (k == 0 && flag) {  // the first tile's block looks at all, the others to their tile
    bool bad = false;
#pragma unroll 4
    for (int s = 32 + lane; s < n_seq; s += 32) {
      const int a = cu[s], b = cu[s + 1];
      bad |= a < 0 || a > b || b > n_rows;
    }
    if (bad) atomicOr(flag, PK_BAD_OFFSETS);
  }
  int top = 0;  // the largest offset so far
  for (int s0 = 0; s0 < n_seq; s0 += 32) {
    const int s = min(s0 + lane, n_seq - 1);
    const int a = cu[s], b = cu[s + 1];
    if (flag && (a < 0 || a > b || b > n_rows)) atomicOr(flag, PK_BAD_OFFSETS);
    int lo = max(min(max(a, 0), n_rows), top), hi = min(max(b, 0), n_rows);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {  // lo = running maximum of the starts
      const int t = __shfl_up_sync(0xffffffffu, lo, o);
      if (lane >= o) lo = max(lo, t);
    }
    hi = max(hi, lo);
    int n = s0 + lane < n_seq ? (hi - lo + block - 1) / block : 0;
    const int own = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, n, o);
      if (lane >= o) n += t;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, k < n);
    if (hit) {
      const int src = __ffs(hit) - 1;
      return make_int4(__shfl_sync(0xffffffffu, lo, src), __shfl_sync(0xffffffffu, hi - lo, src),
                       __shfl_sync(0xffffffffu, k - (n - own), src), s0 + src + 1);
    }
    k -= __shfl_sync(0xffffffffu, n, 31);
    top = __shfl_sync(0xffffffffu, hi, 31);
  }
  return make_int4(0, 0, 0, 0);
}
constexpr int PK_FIND_SEQ = 256;  // sequences that a block looks through

struct PkArgs {
  const void *qkv;
  int64_t ld;
  DType dt;
  const int32_t *cu;
  int n_seq;
  int64_t n_rows;
  int H, Hkv, hd;
  int *flag;  // device word, may be null
  cudaStream_t s;
};
// Where the kernels of 64-row blocks find their tiles: a plan, or (tiles null) the offsets.
struct PkTiles {
  const int *n_tiles;
  const PkTile *tiles;
  const int32_t *cu;
  int n_seq, n_rows;
  int *flag;
};
// Work item of a block: (tile, head, half of the tile's 128 rows).
LLM_DEV bool pk_item64(const PkTiles &w, int heads, PkTile &t, int &h, int &half) {
  const int i = blockIdx.x >> 1, k = i / heads;
  h = i % heads;
  half = blockIdx.x & 1;
  pk_release();
  pk_wait();  // the plan, and D for dK/dV, come from the kernels before
  int4 u;
  if (w.tiles) {
    if (k >= ld_int(w.n_tiles)) return false;
    u = ld_int4(w.tiles + k);
  } else {  // every warp for itself
    u = pk_find(w.cu, w.n_seq, w.n_rows, PK_BLOCK, k, w.flag);
    if (!u.w) return false;
  }
  t = PkTile{u.x, u.y, u.z, 0};
  return true;
}

// No plan where all blocks run at once anyway.
inline bool pk_planned(const PkArgs &a, const PkPlan &p) {
  return 2 * p.cap * a.H > 2 * device_sms() || a.n_seq > PK_FIND_SEQ;
}
inline PkTiles pk_tiles(const PkArgs &a, const PkPlan &p) {
  return PkTiles{p.n_tiles, pk_planned(a, p) ? p.tiles : nullptr, a.cu, a.n_seq, (int)a.n_rows, a.flag};
}
// Enqueues the plan.
void packed_plan(const PkArgs &a, const PkPlan &p);
// tcgen05 kernels (with their plan): bfloat16, head sizes that are multiples of
// 8 (to 128 forward, to 64 backward), rows that start on 16 bytes; false
// (nothing launched) otherwise.  flag:
// non-null device word.
bool packed_fwd_tc(const PkArgs &a, const PkPlan &p, void *o, float *lse, int *flag);
bool packed_bwd_tc(const PkArgs &a, const PkPlan &p, const void *o, const float *lse,
                   const void *dout, void *dqkv, int64_t dld, int *flag);
// mma.sync kernels (with their plan): bfloat16, head sizes that are multiples
// of 8 to 128, input rows that start on 16 bytes; false otherwise, and (fwd;
// bwd where `shorts`) where the sequences are too long for them to win.
bool packed_fwd_mma(const PkArgs &a, const PkPlan &p, void *o, float *lse);
bool packed_bwd_mma(const PkArgs &a, const PkPlan &p, const void *o, const float *lse,
                    const void *dout, void *dqkv, int64_t dld, bool shorts);
// CUDA-core kernels (with their plan): float32 arithmetic, either type, head sizes to 128.
bool packed_fwd_tile(const PkArgs &a, const PkPlan &p, void *o, float *lse);
bool packed_bwd_tile(const PkArgs &a, const PkPlan &p, const void *o, const float *lse,
                     const void *dout, void *dqkv, int64_t dld);

}  // namespace llm
