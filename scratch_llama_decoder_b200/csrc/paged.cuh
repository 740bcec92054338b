// Paged key/value cache: pages [n_pages][2: k, v][Hkv][page_size][hd] of one
// element format, and for the 8-bit formats one float32 scale per row,
// [n_pages][2][Hkv][page_size].  Position p of sequence s lives in row
// p % page_size of page table[s * table_ld + p / page_size].
#pragma once
#include "packed.cuh"

namespace llm {

enum KvFormat { KV_F32 = 0, KV_BF16 = 1, KV_E4M3 = 2, KV_INT8 = 3 };

struct KvView {
  uint8_t *pages;
  float *scales;
  const int32_t *table;
  int64_t table_ld, n_pages;
  int table_pages, fmt, Hkv, hd, ps;
  int *flag;  // device word, may be null
};
inline int kv_bytes(int fmt) { return fmt == KV_F32 ? 4 : fmt == KV_BF16 ? 2 : 1; }

// Row index (of hd elements, and of a scale) of position pos of sequence s,
// kv head 0's keys; -1 when the table does not hold the position or names a
// page that does not exist.
LLM_DEV int64_t kv_row(const KvView &kv, int s, int64_t pos) {
  // table_pages * ps is at most 2^30: 32-bit division from here on
  if (pos < 0 || pos >= (int64_t)kv.table_pages * kv.ps) return -1;
  const uint32_t pg = (uint32_t)pos / (uint32_t)kv.ps;
  const int64_t page = kv.table[(int64_t)s * kv.table_ld + pg];
  if (page < 0 || page >= kv.n_pages) return -1;
  return page * (2 * (int64_t)kv.Hkv * kv.ps) + ((uint32_t)pos - pg * (uint32_t)kv.ps);
}

void kv_write(const KvView &kv, const void *qkv, int64_t ld, DType dt, const int32_t *cu,
              const int32_t *start, int n_seq, int64_t n_rows, int H, cudaStream_t s);
void kv_read(const KvView &kv, const int32_t *cu, const int32_t *start, int n_seq, int64_t n_rows,
             void *k, void *v, DType dt, cudaStream_t s);

// Attention of one query per sequence over its first lens[s] positions.
constexpr int PG_MAX_SEQ = 8192;  // sequences of one call
constexpr int PG_UNIT = 64;       // positions of a unit of work
constexpr int PG_SETUP = 3;       // units that stand for what a (sequence, kv head) costs besides
struct PagedArgs {
  KvView kv;
  const void *q;
  int64_t q_ld;
  DType dt;
  const int32_t *lens;
  int n_seq, H;
  void *o;
  float *lse;  // may be null
  void *ws;
  cudaStream_t s;
};
int64_t paged_ws_bytes(const KvView &kv, int n_seq, int H);
bool paged_attention(const PagedArgs &a);

}  // namespace llm
