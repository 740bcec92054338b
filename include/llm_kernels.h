/*
 * llm_kernels.h -- single hot-path kernels of the training step exposed for
 * parity tests and micro-benchmarks.  Same conventions as llm.h: d_* are
 * caller-owned DEVICE pointers, work is enqueued on `stream` (a cudaStream_t),
 * return codes are the LLM_* values of llm.h, nothing is allocated.  The
 * one-device-per-process rule of llm.h holds here too (LLM_ERR_ARG when
 * another device than the process's is current).
 */
#ifndef LLM_KERNELS_H_
#define LLM_KERNELS_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* The projection matmuls of the step (Hephaistos, Architecture at a glance:
 * every projection is x W; the backward needs dy W^T and x^T dy):
 *   C[M,N] (float32, row-major, leading dimension ldc) = sum_k A(m,k) B(n,k)
 * with bfloat16 operands
 *   A(m,k) = a_kmajor ? A[m*lda + k] : A[k*lda + m]
 *   B(n,k) = b_kmajor ? B[n*ldb + k] : B[k*ldb + n]
 * and float32 accumulation.  tensor_cores = 1 runs the tcgen05/TMA kernel
 * (LLM_ERR_ARG if it does not cover the arguments: 16-byte aligned pointers,
 * lda and ldb multiples of 8, ldc a multiple of 4); 0 runs the CUDA-core
 * kernel.  d_flag: one device int the tcgen05 kernel ORs a time-out bit into
 * (LLM_ERR_TIMEOUT semantics of llm.h); it is never cleared here. */
int llm_kernel_gemm_bf16(int M, int N, int K, const void *d_A, int64_t lda, int a_kmajor,
                         const void *d_B, int64_t ldb, int b_kmajor, float *d_C, int64_t ldc,
                         int tensor_cores, int *d_flag, void *stream);

/* The same product with float32 operands (the float32 configurations):
 * tensor_cores = 1 runs the split-precision tensor-core kernel (3xTF32: each
 * operand split into a tf32 part and a float32 remainder, three tcgen05
 * kind::tf32 products accumulated in float32; relative error about 2^-21
 * per product), which first writes both parts of A and B, K-major, into
 * d_scratch: at least llm_kernel_gemm_f32_scratch_floats(M, N, K) floats,
 * 16-byte aligned, contents need no initialisation, LLM_ERR_ARG if smaller;
 * 0 runs the CUDA-core kernel (d_scratch unused).  d_flag as above. */
int llm_kernel_gemm_f32_scratch_floats(int M, int N, int K, int64_t *floats);
int llm_kernel_gemm_f32(int M, int N, int K, const float *d_A, int64_t lda, int a_kmajor,
                        const float *d_B, int64_t ldb, int b_kmajor, float *d_C, int64_t ldc,
                        int tensor_cores, float *d_scratch, int64_t scratch_floats, int *d_flag,
                        void *stream);

/* Causal self-attention of the step, bfloat16 operands and float32 softmax
 * (Hephaistos, Architecture at a glance: causal multi-head attention with a
 * numerically stable softmax; strata: n_head and n_kv_head independent,
 * flash-style forward and backward).  d_qkv: bf16 [batch*ctx, qkvw] with
 * qkvw = (n_head + 2*n_kv_head)*head_dim, per row all q heads, then k heads,
 * then v heads (RoPE already applied); query head h uses kv head
 * h / (n_head/n_kv_head); scale 1/sqrt(head_dim), the diagonal is kept.
 * Forward: d_o bf16 [batch*ctx, n_head*head_dim] (heads concatenated),
 * d_lse float32 [batch, n_head, ctx] = natural-log sum of exp of each score
 * row.  Backward: from d_o, d_lse and d_dout (bf16, like d_o) writes d_dqkv
 * (bf16, like d_qkv; every element written) and d_D float32 [batch, n_head,
 * ctx] = rowsum(dout * o) as scratch.  tensor_cores selects the kernels:
 * 2 = the tcgen05/TMEM kernels (head_dim 32 or 64; pointers 16-byte aligned),
 * 1 = the warp-level mma kernels (head_dim 32 or 64), 0 = the CUDA-core
 * kernels; LLM_ERR_ARG if the selection does not cover head_dim.  The calls
 * are asynchronous on `stream`.  The tcgen05 kernels bound every internal
 * wait (2 s); a wait that runs out ends the kernel early (outputs incomplete)
 * and is recorded only in a library-owned device word, which these entries do
 * not report (the training-step entries do report it, as LLM_ERR_TIMEOUT). */
int llm_kernel_attention_fwd_bf16(const void *d_qkv, void *d_o, float *d_lse, int batch, int ctx,
                                  int n_head, int n_kv_head, int head_dim, int tensor_cores,
                                  void *stream);
int llm_kernel_attention_bwd_bf16(const void *d_qkv, const void *d_o, const void *d_dout,
                                  const float *d_lse, float *d_D, void *d_dqkv, int batch,
                                  int ctx, int n_head, int n_kv_head, int head_dim,
                                  int tensor_cores, void *stream);

/* The same attention in float32 (the float32 configurations): d_qkv, d_o,
 * d_dout, d_dqkv float32 with the layouts above, d_lse and d_D as above.
 * tiled = 1 selects the tiled CUDA-core kernels (head_dim 32 or 64; rows
 * 16-byte aligned: pointers 16-byte aligned), 0 the one-warp-per-row
 * kernels (any head_dim); LLM_ERR_ARG otherwise.  Asynchronous on `stream`. */
int llm_kernel_attention_fwd_f32(const float *d_qkv, float *d_o, float *d_lse, int batch, int ctx,
                                 int n_head, int n_kv_head, int head_dim, int tiled, void *stream);
int llm_kernel_attention_bwd_f32(const float *d_qkv, const float *d_o, const float *d_dout,
                                 const float *d_lse, float *d_D, float *d_dqkv, int batch,
                                 int ctx, int n_head, int n_kv_head, int head_dim, int tiled,
                                 void *stream);

/* Embedding backward (Hephaistos, Architecture at a glance: token embedding;
 * its gradient is a scatter-add): dwte[v,:] = sum over positions i with
 * tokens[i] = v of dx[i,:], summed in increasing i (deterministic), zero for
 * ids that do not occur.  d_tokens: int32 [n_tokens] (ids outside
 * [0, vocab) are treated as 0); d_dx: float32 [n_tokens, d_model];
 * d_dwte: float32 [vocab, d_model], fully overwritten.  d_scratch: device
 * memory of at least llm_kernel_embed_bwd_scratch_bytes() bytes, 16-byte
 * aligned, used while the call's kernels run (its contents need no
 * initialisation).  LLM_ERR_ARG for null pointers, sizes < 1 or a small
 * scratch. */
int llm_kernel_embed_bwd_scratch_bytes(int64_t n_tokens, int vocab, int64_t *bytes);
int llm_kernel_embed_bwd(const int32_t *d_tokens, const float *d_dx, float *d_dwte,
                         int64_t n_tokens, int d_model, int vocab, void *d_scratch,
                         int64_t scratch_bytes, void *stream);

/* The embedding backward of llm_kernel_embed_bwd(), for callers that cannot
 * allocate device memory at call time: code running while a CUDA graph is
 * being captured, hooks inside an allocator, plug-ins whose host framework
 * owns all device memory, or loops that forbid allocation after start-up.
 * The source pages have no counterpart of this call; it exists for such
 * callers.  Same arguments, layout and result as llm_kernel_embed_bwd(),
 * without the scratch arguments: the scratch is one library-owned device
 * array of 1.5 MiB (394,307 int32) on every GPU that loads the library, kept
 * until the process exits.  Limits: n_tokens <= 65536 and vocab <= 65536,
 * else LLM_ERR_ARG with nothing launched.  The call allocates nothing (no
 * cudaMalloc, cudaFree or allocating library routine).  Its first call on a
 * device looks up the array's device address (cudaGetSymbolAddress, on the
 * current device) and caches it; make that first call before any stream
 * capture.  All calls on a device share the array: calls whose kernels
 * overlap on the GPU (different streams without ordering) race and give
 * wrong results; calls on one stream are ordered and safe.  Each call
 * re-initialises what it needs, so no state carries over between calls. */
int llm_kernel_embed_bwd_noalloc(const int32_t *d_tokens, const float *d_dx, float *d_dwte,
                                 int64_t n_tokens, int d_model, int vocab, void *stream);

/* Causal attention over packed sequences: several sequences of different
 * lengths end to end in one array, so that a batch of prompts or training
 * documents carries no padding (strata: n_head and n_kv_head independent,
 * flash-style attention; the operators above take one length for all).
 * dtype: LLM_FP32 or LLM_BF16, of d_qkv, d_o, d_dout and d_dqkv.
 *   d_qkv: [n_rows] rows of ld elements (ld >= qkvw), the layout of a row as
 *     in llm_kernel_attention_fwd_bf16 (q heads, k heads, v heads; RoPE
 *     applied; query head h uses kv head h / (n_head / n_kv_head); scale
 *     1/sqrt(head_dim)).
 *   d_cu: int32 [n_seq + 1], non-decreasing: sequence s is the rows
 *     [d_cu[s], d_cu[s+1]), and a row attends to the rows of its own sequence
 *     up to itself.  A sequence may have no rows.  Rows before d_cu[0] and
 *     from d_cu[n_seq] on belong to none: their outputs are left as they were,
 *     and their contents are not looked at (they may hold anything).
 *   Forward: d_o [n_rows, n_head*head_dim] (contiguous) and d_lse float32
 *     [n_head, n_rows], the natural-log sum of exp of each row's scores.
 *   Backward: from d_o, d_lse and d_dout (like d_o) writes d_dqkv (rows of
 *     dqkv_ld elements, the first qkvw of them written), no atomics: the same
 *     inputs give the same bits.  d_dqkv shares no byte with an input
 *     (LLM_ERR_ARG), as d_o and d_lse share none with d_qkv.
 *   d_ws: at least llm_kernel_attention_packed_workspace() bytes, 16-byte
 *     aligned, no initialisation needed; used while the call's kernels run, so
 *     calls that may overlap on the GPU need one each.
 *   d_flag: null, or one device int32 that gets bit 1 (LLM_PACKED_BAD_CU) OR-ed
 *     in when d_cu decreases or leaves [0, n_rows] -- its entries then count as
 *     clamped into the range and raised to the largest before them, so that
 *     nothing outside the rows is touched -- and bit 4 (LLM_PACKED_TIMEOUT)
 *     when a bounded wait of the tensor-core kernels gave up (the outputs are
 *     incomplete).  Never cleared here.
 * Which kernels run goes by n_rows / n_seq (empty sequences and rows of none
 * count), and in a captured call stays as it was captured: every choice serves
 * any offsets, but a long sequence among so many empty or short ones that the
 * mean is short (to 64 rows; 128 to 320 for small calls, heads to 32 and the
 * backward) runs at a half to a quarter of its rate.  Offsets padded to more
 * sequences than there are cost that where the rows are few.
 * A value that is not finite reaches rows of its own sequence only: in the
 * forward those behind it, and of those before it any in the same 128 rows of
 * the sequence; in the backward any of them.
 * Limits: n_rows <= 2^20, n_seq <= 65536, n_head <= 1024, an even head_dim of
 * 2 to 128.  n_rows = 0 or n_seq = 0 launches nothing.  LLM_ERR_ARG outside
 * them, for a null or misaligned pointer or a small workspace.  Asynchronous
 * on `stream`; may be captured into a graph. */
enum { LLM_PACKED_BAD_CU = 1, LLM_KV_BAD_PAGE = 2, LLM_PACKED_TIMEOUT = 4 };
int llm_kernel_attention_packed_workspace(int64_t n_rows, int n_seq, int n_head, int backward,
                                          int64_t *bytes);
int llm_kernel_attention_packed_fwd(const void *d_qkv, int64_t ld, int dtype, const int32_t *d_cu,
                                    int n_seq, int64_t n_rows, int n_head, int n_kv_head,
                                    int head_dim, void *d_o, float *d_lse, void *d_ws,
                                    int64_t ws_bytes, int32_t *d_flag, void *stream);
int llm_kernel_attention_packed_bwd(const void *d_qkv, int64_t ld, int dtype, const int32_t *d_cu,
                                    int n_seq, int64_t n_rows, int n_head, int n_kv_head,
                                    int head_dim, const void *d_o, const float *d_lse,
                                    const void *d_dout, void *d_dqkv, int64_t dqkv_ld, void *d_ws,
                                    int64_t ws_bytes, int32_t *d_flag, void *stream);

/* A paged key/value cache: the cache of llm_decode gives every sequence room
 * for ctx positions and keeps them at one position; here sequences of any
 * lengths share pages, and the values may be held in 8 bits.
 *   d_pages: [n_pages][2: k, v][n_kv_head][page_size][head_dim] elements of
 *     `format`; d_scales: float32 [n_pages][2][n_kv_head][page_size], one per
 *     row of head_dim elements and not negative, for the 8-bit formats
 *     (ignored otherwise).
 *   d_table: int32, row s (at d_table + s * table_ld) holds the pages of
 *     sequence s in order: position p is row p % page_size of page
 *     d_table[s * table_ld + p / page_size].  table_pages entries a row.
 *   d_flag: null, or one device int32 that gets bit 2 (LLM_KV_BAD_PAGE) OR-ed
 *     in when a position is needed that the table does not reach, or whose
 *     page is outside [0, n_pages); nothing is read or written there.
 * Formats: LLM_KV_F32, LLM_KV_BF16 (rounded to nearest);
 *   LLM_KV_E4M3: code = x / scale rounded to the nearest e4m3 number, scale
 *     the least power of two (2^-126 at least) with max|x| <= 448 scale over
 *     the row, so only the code rounds;
 *   LLM_KV_INT8: scale = max|x| / 127 rounded to float32 (the least normal
 *     number at least), code = x / scale rounded to the nearest integer, ties
 *     to even (codes -127 to 127).
 *   A value is code * scale.  A row that holds an infinity or a NaN gets a NaN
 *   scale and code 0: it reads back as NaN.
 * head_dim is even, 2 to 128; page_size 1 to 65536; n_kv_head <= 1024;
 * table_pages * page_size at most 2^30. */
enum { LLM_KV_F32 = 0, LLM_KV_BF16 = 1, LLM_KV_E4M3 = 2, LLM_KV_INT8 = 3 };
typedef struct {
  void *d_pages;
  float *d_scales;
  const int32_t *d_table;
  int64_t table_ld, n_pages;
  int32_t table_pages, format, n_kv_head, head_dim, page_size;
  int32_t *d_flag;
} llm_kv;

/* Packed rows (d_qkv, ld, dtype, d_cu, n_seq, n_rows, as above) into the cache:
 * row i of sequence s becomes position d_start[s] + i - d_cu[s] (d_start int32
 * [n_seq], null = all 0): a whole prompt, a later part of one, or one new
 * token each.  Offsets that decrease or leave the rows count as mended, as
 * above, with LLM_PACKED_BAD_CU in the cache's d_flag.  Two rows written to one
 * place (tables that share a page there) leave it with an undefined mix of both.
 * llm_kernel_kv_read is the inverse: d_k, d_v [n_rows, n_kv_head, head_dim] of
 * dtype get the values of those positions (rows without a place as zeros; rows
 * of no sequence are left as they were).  Limits as above; LLM_ERR_ARG
 * otherwise. */
int llm_kernel_kv_write(const llm_kv *kv, const void *d_qkv, int64_t ld, int dtype,
                        const int32_t *d_cu, const int32_t *d_start, int n_seq, int64_t n_rows,
                        int n_head, void *stream);
int llm_kernel_kv_read(const llm_kv *kv, const int32_t *d_cu, const int32_t *d_start, int n_seq,
                       int64_t n_rows, void *d_k, void *d_v, int dtype, void *stream);

/* Attention of one new token per sequence over its cached positions (the
 * attention of llm_decode for sequences of different lengths): d_q [n_seq]
 * rows of q_ld elements of dtype, n_head*head_dim of them used (a q|k|v row
 * will do); d_lens int32 [n_seq]: sequence s attends to positions 0 to
 * d_lens[s] - 1, its own new token among them once written.  d_o [n_seq,
 * n_head*head_dim] of dtype (contiguous), d_lse float32 [n_seq, n_head] (null:
 * not wanted).  A sequence of length 0 gets o = 0 and lse = -inf; a length
 * outside [0, table_pages * page_size] counts as clamped, and a position
 * without a place as not there (d_flag of the cache, LLM_KV_BAD_PAGE).  What
 * the pages hold past a sequence's length is not looked at.  d_ws: at least
 * llm_kernel_attention_paged_workspace() bytes, 16-byte aligned, no
 * initialisation needed, one per call that may overlap another on the GPU (not
 * looked at when that is 0: short tables, whose sequences are not split).
 * The lengths are read on the device: a captured call serves any.  The work is
 * split over the cached positions whatever the lengths are, and joined in a
 * fixed order: the same inputs give the same bits.  n_seq <= 8192. */
int llm_kernel_attention_paged_workspace(const llm_kv *kv, int n_seq, int n_head, int64_t *bytes);
int llm_kernel_attention_paged(const llm_kv *kv, const void *d_q, int64_t q_ld, int dtype,
                               const int32_t *d_lens, int n_seq, int n_head, void *d_o,
                               float *d_lse, void *d_ws, int64_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LLM_KERNELS_H_ */
