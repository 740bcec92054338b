// C entries of the packed attention and the paged cache: argument checks on
// the host, then the launches.
#include "../../include/llm.h"
#include "../../include/llm_kernels.h"
#include "overlap.h"
#include "paged.cuh"

using namespace llm;

static_assert(LLM_PACKED_BAD_CU == PK_BAD_OFFSETS && LLM_KV_BAD_PAGE == PK_BAD_PAGE &&
                  LLM_PACKED_TIMEOUT == FLAG_TIMEOUT,
              "flag bits");
static_assert(LLM_KV_F32 == KV_F32 && LLM_KV_BF16 == KV_BF16 && LLM_KV_E4M3 == KV_E4M3 &&
                  LLM_KV_INT8 == KV_INT8,
              "cache formats");
static_assert(LLM_FP32 == DT_F32 && LLM_BF16 == DT_BF16, "element types");

namespace {

bool aligned(const void *p, int64_t n) { return p && !((uintptr_t)p & (uintptr_t)(n - 1)); }
int elem(int dtype) { return dtype == LLM_BF16 ? 2 : 4; }
bool heads_ok(int H, int Hkv, int hd) {
  return H >= 1 && H <= 1024 && Hkv >= 1 && H % Hkv == 0 && hd >= 2 && hd <= 128 && hd % 2 == 0;
}
bool rows_ok(int n_seq, int64_t n_rows) {
  return n_seq >= 0 && n_seq <= PK_MAX_SEQ && n_rows >= 0 && n_rows <= PK_MAX_ROWS;
}
bool dtype_ok(int dtype) { return dtype == LLM_FP32 || dtype == LLM_BF16; }

// Arguments of the packed attention calls; false for LLM_ERR_ARG.
bool packed_args(PkArgs *a, const void *qkv, int64_t ld, int dtype, const int32_t *cu, int n_seq,
                 int64_t n_rows, int H, int Hkv, int hd, int32_t *flag, void *stream) {
  if (!dtype_ok(dtype) || !rows_ok(n_seq, n_rows) || !heads_ok(H, Hkv, hd) ||
      ld < (int64_t)(H + 2 * Hkv) * hd)
    return false;
  *a = PkArgs{qkv, ld, (DType)dtype, cu, n_seq, n_rows, H, Hkv, hd, flag, (cudaStream_t)stream};
  if (n_rows == 0 || n_seq == 0) return true;
  return aligned(qkv, elem(dtype)) && aligned(cu, 4) && (!flag || aligned(flag, 4));
}

// The kernels' view of a cache; false for LLM_ERR_ARG.
bool kv_view(const llm_kv *kv, KvView *v) {
  if (!kv || kv->format < LLM_KV_F32 || kv->format > LLM_KV_INT8 || kv->n_kv_head < 1 ||
      kv->n_kv_head > 1024 || kv->head_dim < 2 || kv->head_dim > 128 || kv->head_dim % 2 ||
      kv->page_size < 1 || kv->page_size > 65536 || kv->n_pages < 1 || kv->table_pages < 0 ||
      kv->table_ld < kv->table_pages ||
      (int64_t)kv->table_pages * kv->page_size > ((int64_t)1 << 30))
    return false;
  // the row index of every element fits 2^62 whatever the head size
  if (kv->n_pages > ((int64_t)1 << 40) / ((int64_t)kv->n_kv_head * kv->page_size)) return false;
  if (!aligned(kv->d_pages, kv_bytes(kv->format)) ||
      (kv->format >= LLM_KV_E4M3 && !aligned(kv->d_scales, 4)) ||
      (kv->table_pages > 0 && !aligned(kv->d_table, 4)) || (kv->d_flag && !aligned(kv->d_flag, 4)))
    return false;
  *v = KvView{(uint8_t *)kv->d_pages, kv->d_scales, kv->d_table, kv->table_ld, kv->n_pages,
              kv->table_pages, kv->format, kv->n_kv_head, kv->head_dim, kv->page_size, kv->d_flag};
  return true;
}
bool paged_ok(const KvView &v, int n_seq, int H) {
  const int64_t units = ((int64_t)v.table_pages * v.ps + PG_UNIT - 1) / PG_UNIT + PG_SETUP;
  return n_seq >= 0 && n_seq <= PG_MAX_SEQ && heads_ok(H, v.Hkv, v.hd) &&
         units * n_seq < ((int64_t)1 << 31);
}
int launched() { return cudaGetLastError() == cudaSuccess ? LLM_OK : LLM_ERR_CUDA; }

}  // namespace

extern "C" {

int llm_kernel_attention_packed_workspace(int64_t n_rows, int n_seq, int n_head, int backward,
                                          int64_t *bytes) {
  if (!bytes || !rows_ok(n_seq, n_rows) || n_head < 1 || n_head > 1024) return LLM_ERR_ARG;
  *bytes = pk_plan(nullptr, n_rows, n_seq, n_head, backward != 0).bytes;
  return LLM_OK;
}

int llm_kernel_attention_packed_fwd(const void *d_qkv, int64_t ld, int dtype, const int32_t *d_cu,
                                    int n_seq, int64_t n_rows, int n_head, int n_kv_head,
                                    int head_dim, void *d_o, float *d_lse, void *d_ws,
                                    int64_t ws_bytes, int32_t *d_flag, void *stream) {
  PkArgs a;
  if (!packed_args(&a, d_qkv, ld, dtype, d_cu, n_seq, n_rows, n_head, n_kv_head, head_dim, d_flag,
                   stream))
    return LLM_ERR_ARG;
  if (n_rows == 0 || n_seq == 0) return LLM_OK;
  const PkPlan p = pk_plan(d_ws, n_rows, n_seq, n_head, false);
  if (!aligned(d_o, elem(dtype)) || !aligned(d_lse, 4) || !aligned(d_ws, 16) || ws_bytes < p.bytes)
    return LLM_ERR_ARG;
  if (!claim_device(nullptr)) return LLM_ERR_ARG;  // one device per process
  g_launches = 0;
  int *flag = d_flag ? d_flag : p.n_tiles + 1;
  if (!packed_fwd_mma(a, p, d_o, d_lse) && !packed_fwd_tc(a, p, d_o, d_lse, flag) &&
      !packed_fwd_tile(a, p, d_o, d_lse))
    return LLM_ERR_CUDA;
  return launched();
}

int llm_kernel_attention_packed_bwd(const void *d_qkv, int64_t ld, int dtype, const int32_t *d_cu,
                                    int n_seq, int64_t n_rows, int n_head, int n_kv_head,
                                    int head_dim, const void *d_o, const float *d_lse,
                                    const void *d_dout, void *d_dqkv, int64_t dqkv_ld, void *d_ws,
                                    int64_t ws_bytes, int32_t *d_flag, void *stream) {
  PkArgs a;
  if (!packed_args(&a, d_qkv, ld, dtype, d_cu, n_seq, n_rows, n_head, n_kv_head, head_dim, d_flag,
                   stream) ||
      dqkv_ld < (int64_t)(n_head + 2 * n_kv_head) * head_dim)
    return LLM_ERR_ARG;
  if (n_rows == 0 || n_seq == 0) return LLM_OK;
  const PkPlan p = pk_plan(d_ws, n_rows, n_seq, n_head, true);
  const int e = elem(dtype);
  if (!aligned(d_o, e) || !aligned(d_lse, 4) || !aligned(d_dout, e) || !aligned(d_dqkv, e) ||
      !aligned(d_ws, 16) || ws_bytes < p.bytes)
    return LLM_ERR_ARG;
  // d_dqkv overlaps no input: its rows are written while those are still read
  const int64_t w = (int64_t)(n_head + 2 * n_kv_head) * head_dim * e,
                on = n_rows * n_head * head_dim * e;
  const uintptr_t dx = (uintptr_t)d_dqkv;
  if (rows_overlap(d_dqkv, dqkv_ld * e, d_qkv, ld * e, w, n_rows) ||
      overlap(dx, dqkv_ld * e, w, n_rows, (uintptr_t)d_o, on) ||
      overlap(dx, dqkv_ld * e, w, n_rows, (uintptr_t)d_dout, on) ||
      overlap(dx, dqkv_ld * e, w, n_rows, (uintptr_t)d_lse, 4 * n_rows * n_head))
    return LLM_ERR_ARG;
  if (!claim_device(nullptr)) return LLM_ERR_ARG;
  g_launches = 0;
  int *flag = d_flag ? d_flag : p.n_tiles + 1;
  if (!packed_bwd_mma(a, p, d_o, d_lse, d_dout, d_dqkv, dqkv_ld, true) &&
      !packed_bwd_tc(a, p, d_o, d_lse, d_dout, d_dqkv, dqkv_ld, flag) &&
      !packed_bwd_mma(a, p, d_o, d_lse, d_dout, d_dqkv, dqkv_ld, false) &&
      !packed_bwd_tile(a, p, d_o, d_lse, d_dout, d_dqkv, dqkv_ld))
    return LLM_ERR_CUDA;
  return launched();
}

int llm_kernel_kv_write(const llm_kv *kv, const void *d_qkv, int64_t ld, int dtype,
                        const int32_t *d_cu, const int32_t *d_start, int n_seq, int64_t n_rows,
                        int n_head, void *stream) {
  KvView v;
  if (!kv_view(kv, &v) || !dtype_ok(dtype) || !rows_ok(n_seq, n_rows) ||
      !heads_ok(n_head, v.Hkv, v.hd) || ld < (int64_t)(n_head + 2 * v.Hkv) * v.hd)
    return LLM_ERR_ARG;
  if (n_rows == 0 || n_seq == 0) return LLM_OK;
  if (!aligned(d_qkv, elem(dtype)) || !aligned(d_cu, 4) || (d_start && !aligned(d_start, 4)))
    return LLM_ERR_ARG;
  if (!claim_device(nullptr)) return LLM_ERR_ARG;
  g_launches = 0;
  kv_write(v, d_qkv, ld, (DType)dtype, d_cu, d_start, n_seq, n_rows, n_head, (cudaStream_t)stream);
  return launched();
}

int llm_kernel_kv_read(const llm_kv *kv, const int32_t *d_cu, const int32_t *d_start, int n_seq,
                       int64_t n_rows, void *d_k, void *d_v, int dtype, void *stream) {
  KvView v;
  if (!kv_view(kv, &v) || !dtype_ok(dtype) || !rows_ok(n_seq, n_rows)) return LLM_ERR_ARG;
  if (n_rows == 0 || n_seq == 0) return LLM_OK;
  if (!aligned(d_k, elem(dtype)) || !aligned(d_v, elem(dtype)) || !aligned(d_cu, 4) ||
      (d_start && !aligned(d_start, 4)))
    return LLM_ERR_ARG;
  if (!claim_device(nullptr)) return LLM_ERR_ARG;
  g_launches = 0;
  kv_read(v, d_cu, d_start, n_seq, n_rows, d_k, d_v, (DType)dtype, (cudaStream_t)stream);
  return launched();
}

int llm_kernel_attention_paged_workspace(const llm_kv *kv, int n_seq, int n_head, int64_t *bytes) {
  KvView v;
  if (!bytes || !kv_view(kv, &v) || !paged_ok(v, n_seq, n_head)) return LLM_ERR_ARG;
  *bytes = paged_ws_bytes(v, n_seq, n_head);
  return LLM_OK;
}

int llm_kernel_attention_paged(const llm_kv *kv, const void *d_q, int64_t q_ld, int dtype,
                               const int32_t *d_lens, int n_seq, int n_head, void *d_o,
                               float *d_lse, void *d_ws, int64_t ws_bytes, void *stream) {
  PagedArgs a;
  if (!kv_view(kv, &a.kv) || !dtype_ok(dtype) || !paged_ok(a.kv, n_seq, n_head) ||
      q_ld < (int64_t)n_head * a.kv.hd)
    return LLM_ERR_ARG;
  if (n_seq == 0) return LLM_OK;
  if (!aligned(d_q, elem(dtype)) || !aligned(d_lens, 4) || !aligned(d_o, elem(dtype)) ||
      (d_lse && !aligned(d_lse, 4)))
    return LLM_ERR_ARG;
  const int64_t need = paged_ws_bytes(a.kv, n_seq, n_head);
  if (need > 0 && (!aligned(d_ws, 16) || ws_bytes < need)) return LLM_ERR_ARG;
  if (!claim_device(nullptr)) return LLM_ERR_ARG;
  g_launches = 0;
  a.q = d_q;
  a.q_ld = q_ld;
  a.dt = (DType)dtype;
  a.lens = d_lens;
  a.n_seq = n_seq;
  a.H = n_head;
  a.o = d_o;
  a.lse = d_lse;
  a.ws = d_ws;
  a.s = (cudaStream_t)stream;
  if (!paged_attention(a)) return LLM_ERR_CUDA;
  return launched();
}

}  // extern "C"
