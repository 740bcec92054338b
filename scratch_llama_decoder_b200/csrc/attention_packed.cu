// Causal attention over packed sequences of different lengths: the work plan
// and the CUDA-core kernels.
//
//   s_ij = q_i . k_j / sqrt(hd)   j <= i in the same sequence
//   L_i  = ln sum_j exp(s_ij),    o_i = sum_j exp(s_ij - L_i) v_j
//   D_i  = dO_i . O_i,  P = exp(s - L),  dS = P (dO_i . v_j - D_i) / sqrt(hd)
//   dq_i = sum_j dS_ij k_j,  dk_j = sum dS_ij q_i,  dv_j = sum P_ij dO_i
// (the sums of dk, dv over the queries i >= j of every query head of the kv
// head, in a fixed order: no atomics).
#include "packed.cuh"

namespace llm {
namespace pk {

// ---------------------------------------------------------------- work plan
// The tiles of all sequences, most work first: a sequence of n blocks has one
// tile of each weight 1 .. n (block b, as a query tile, reads b + 1 key
// blocks), so weight c has cnt(c) = #{sequences of >= c blocks} tiles, the
// tiles of weight c start at off(c) = sum over c' > c of cnt(c'), and within a
// weight they go by the sequences' rank, longest first.  One block; offsets
// are clamped to a non-decreasing walk within [0, n_rows], so no tile reaches
// outside the rows and no two tiles share a row, whatever cu holds.
constexpr int PT = 1024;
constexpr int MAXC = (int)(PK_MAX_ROWS / PK_BLOCK);

// Inclusive scan over the block (sum or maximum).
template <bool MAX>
LLM_DEV int block_scan(int v, int *warp_tot) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = MAX ? max(v, t) : v + t;
  }
  __syncthreads();
  if (lane == 31) warp_tot[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int w = warp_tot[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w = MAX ? max(w, t) : w + t;
    }
    warp_tot[lane] = w;
  }
  __syncthreads();
  if (warp > 0) {
    const int t = warp_tot[warp - 1];
    v = MAX ? max(v, t) : v + t;
  }
  return v;
}

__global__ void __launch_bounds__(PT) k_plan(const int32_t *__restrict__ cu, int n_seq, int n_rows,
                                             int *__restrict__ n_tiles, PkTile *__restrict__ tiles,
                                             int *__restrict__ off, int *__restrict__ rank,
                                             int *flag) {
  __shared__ int hist[MAXC + 2];  // sequences of exactly n blocks; then cnt, then off
  pk_release();
  __shared__ int warp_tot[32];
  const int C = (n_rows + PK_BLOCK - 1) / PK_BLOCK;
  for (int i = threadIdx.x; i <= C + 1; i += PT) hist[i] = 0;
  // offsets: running maximum of the clamped entries
  int carry = 0;
  bool bad = false;
  for (int s0 = 0; s0 <= n_seq; s0 += PT) {
    const int s = s0 + threadIdx.x;
    const int c = s <= n_seq ? cu[s] : 0;
    const int v = max(block_scan<true>(min(max(c, 0), n_rows), warp_tot), carry);
    if (s <= n_seq) {
      off[s] = v;
      bad |= c != v;
    }
    __syncthreads();
    if (threadIdx.x == PT - 1) warp_tot[0] = v;
    __syncthreads();
    carry = warp_tot[0];
  }
  if (bad && flag) atomicOr(flag, PK_BAD_OFFSETS);
  __syncthreads();
  for (int s = threadIdx.x; s < n_seq; s += PT) {
    const int n = (off[s + 1] - off[s] + PK_BLOCK - 1) / PK_BLOCK;
    // the rank among sequences of as many blocks, completed below
    rank[s] = n ? atomicAdd(&hist[n], 1) : 0;
  }
  __syncthreads();
  // hist[n] -> cnt(n), scanned from the longest down
  carry = 0;
  for (int c0 = 0; c0 < C; c0 += PT) {
    const int n = C - (c0 + (int)threadIdx.x);
    const int v = carry + block_scan<false>(n >= 1 ? hist[n] : 0, warp_tot);
    __syncthreads();
    if (n >= 1) hist[n] = v;
    if (threadIdx.x == PT - 1) warp_tot[0] = v;
    __syncthreads();
    carry = warp_tot[0];
  }
  if (threadIdx.x == 0) hist[C + 1] = 0;
  __syncthreads();
  for (int s = threadIdx.x; s < n_seq; s += PT) {
    const int n = (off[s + 1] - off[s] + PK_BLOCK - 1) / PK_BLOCK;
    if (n) rank[s] += hist[n + 1];  // after every longer sequence
  }
  __syncthreads();
  // cnt(c) -> off(c): exclusive scan from the heaviest weight down
  carry = 0;
  for (int c0 = 0; c0 < C; c0 += PT) {
    const int c = C - (c0 + (int)threadIdx.x);
    const int own = c >= 1 ? hist[c] : 0;
    const int v = carry + block_scan<false>(own, warp_tot);
    __syncthreads();
    if (c >= 1) hist[c] = v - own;
    if (threadIdx.x == PT - 1) warp_tot[0] = v;
    __syncthreads();
    carry = warp_tot[0];
  }
  if (threadIdx.x == 0) {
    n_tiles[0] = carry;
    n_tiles[2] = 0;
  }
  __syncthreads();
  for (int s = threadIdx.x >> 5; s < n_seq; s += PT / 32) {
    const int row0 = off[s], len = off[s + 1] - row0, n = (len + PK_BLOCK - 1) / PK_BLOCK;
    for (int b = threadIdx.x & 31; b < n; b += 32)
      tiles[hist[b + 1] + rank[s]] = PkTile{row0, len, b, s};
  }
}

// The same plan for few sequences, where the scans' barriers would take longer
// than counting: off(c) = sum over the sequences of max(0, n - c), and a
// sequence's rank by comparing it with every other one.
constexpr int FEW = 256;
__global__ void __launch_bounds__(FEW) k_plan_few(const int32_t *__restrict__ cu, int n_seq,
                                                  int n_rows, int *__restrict__ n_tiles,
                                                  PkTile *__restrict__ tiles, int *flag) {
  __shared__ int off[FEW + 1], blocks[FEW], rank[FEW], base[MAXC + 1];
  __shared__ int warp_tot[FEW / 32];
  pk_release();
  const int t = threadIdx.x;
  const int mine = t <= n_seq ? cu[t] : 0, last = cu[n_seq];  // n_seq may be FEW: one entry more
  const int next = t < n_seq ? cu[t + 1] : 0;
  const bool bad = t < n_seq && (mine < 0 || mine > next || next > n_rows);
  if (t < n_seq) off[t] = mine;
  if (t == 0) off[n_seq] = last;
  if (__syncthreads_or(bad)) {  // running maximum of the clamped offsets
    if (flag && t == 0) atomicOr(flag, PK_BAD_OFFSETS);
    int v = min(max(t < n_seq ? mine : 0, 0), n_rows);
    const int lane = t & 31, warp = t >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v = max(v, x);
    }
    if (lane == 31) warp_tot[warp] = v;
    __syncthreads();
    for (int w = 0; w < warp; w++) v = max(v, warp_tot[w]);
    if (t < n_seq) off[t] = v;
    __syncthreads();
    if (t == 0) off[n_seq] = max(off[n_seq - 1], min(max(last, 0), n_rows));
    __syncthreads();
  }
  const int n = t < n_seq ? (off[t + 1] - off[t] + PK_BLOCK - 1) / PK_BLOCK : 0;
  if (t < n_seq) blocks[t] = n;
  __syncthreads();
  if (t < n_seq) {
    int r = 0;
    for (int s = 0; s < n_seq; s++) r += blocks[s] > n || (blocks[s] == n && s < t);
    rank[t] = r;
  }
  const int C = (n_rows + PK_BLOCK - 1) / PK_BLOCK;
  for (int c = t; c <= C; c += FEW) {
    int sum = 0;
    for (int s = 0; s < n_seq; s++) sum += max(0, blocks[s] - c);
    base[c] = sum;
  }
  __syncthreads();
  if (t == 0) {
    n_tiles[0] = base[0];
    n_tiles[2] = 0;
  }
  for (int s = t >> 5; s < n_seq; s += FEW / 32)
    for (int b = t & 31; b < blocks[s]; b += 32)
      tiles[base[b + 1] + rank[s]] = PkTile{off[s], off[s + 1] - off[s], b, s};
}

// --------------------------------------------------------- CUDA-core kernels
// 64 x 64 tiles, R x 4 results a thread (R = 8, or 4 at head 128 where the
// gradients' accumulators leave no room), 16 x 64 / R threads: tx = thread %
// 16, ty = thread / 16.  A thread's rows of a product are R ty .. R ty + R - 1
// of one tile, its columns rows tx + 16 c of the other; both are read along
// the head as float4 from tiles that lie row by row (padded by 4, so that the
// 16 tx fall on different banks), 12 loads to 128 multiply-adds at R = 8, two
// to an instruction (f32x2).  So no tile is transposed and float32 rows come
// by cp.async.  A tile of weights lies [row][column], the columns of odd ty
// with bit 4 turned (both ty of a warp would store to the same banks).  Head
// columns past hd are zero, so a head size runs on the next of 32, 64, 128.
// Against 4 x 4 results a thread from transposed tiles: training step of
// 16384 rows, 4 heads of 32, 538 -> 397 us (4 sequences of 2048 rows: forward 27,
// backward 22 TFLOP/s of the 74 of the FMA pipes).  What bounds it is the
// latency of 8 warps an SM: a thread's results take 173 to 232 registers, and
// cut to 168 or 128 for 3 or 4 blocks an SM they spill (422 and 557 us).
constexpr int TB = 64, LDP = TB + 4;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
// 2^x, the SFU's instruction alone (relative error 2^-22): exp2f adds the
// scaling of subnormal results, which no weight needs.
LLM_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <int HD> constexpr int rows_of() { return HD == 128 ? 4 : 8; }
template <int HD> constexpr int threads_of() { return 16 * TB / rows_of<HD>(); }
template <int HD> constexpr int tile_of() { return TB * (HD + 4); }  // floats

// Output column c of a thread: float4 groups 64 columns apart (head 128), so
// that the 16 threads of a row read consecutive float4.
template <int HD>
LLM_DEV int out_col(int tx, int c) {
  return HD == 32 ? tx * 2 + c : (c >> 2) * 64 + tx * 4 + (c & 3);
}
// 4 consecutive elements; elements at or past n read as 0.
LLM_DEV float4 read4(const float *p, bool vec, int n) {
  if (vec && n >= 4) return *reinterpret_cast<const float4 *>(p);
  return make_float4(n > 0 ? p[0] : 0.f, n > 1 ? p[1] : 0.f, n > 2 ? p[2] : 0.f,
                     n > 3 ? p[3] : 0.f);
}
LLM_DEV float4 read4(const __nv_bfloat16 *p, bool vec, int n) {
  if (vec && n >= 4) {
    const uint2 w = *reinterpret_cast<const uint2 *>(p);
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w.x));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w.y));
    return make_float4(a.x, a.y, b.x, b.y);
  }
  return make_float4(n > 0 ? to_f(p[0]) : 0.f, n > 1 ? to_f(p[1]) : 0.f,
                     n > 2 ? to_f(p[2]) : 0.f, n > 3 ? to_f(p[3]) : 0.f);
}
// Rows [0, nrows) of src (row stride ld), hd columns, into a tile; the rest 0.
// float32 rows of whole float4 by cp.async (the caller waits).
template <typename T, int HD>
LLM_DEV void load_tile(float *t, const T *src, int64_t ld, int nrows, int hd, bool vec) {
  for (int i = threadIdx.x; i < TB * HD / 4; i += threads_of<HD>()) {
    const int row = i / (HD / 4), c = i % (HD / 4) * 4;
    float *dst = t + row * (HD + 4) + c;
    const bool in = row < nrows && c < hd;
    if (sizeof(T) == 4 && vec) {  // vec: hd is a multiple of 4
      const T *p = in ? src + row * ld + c : src;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                       (uint32_t)__cvta_generic_to_shared(dst)),
                   "l"(p), "r"(in ? 16 : 0)
                   : "memory");
    } else {
      *reinterpret_cast<float4 *>(dst) =
          in ? read4(src + row * ld + c, vec, hd - c) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
}
LLM_DEV void tiles_ready() {
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
}
// s[r][c] = A[R ty + r] . B[tx + 16 c] for c in [C0, C1), 0 for the others.
template <int HD, int R, int C0 = 0, int C1 = 4>
LLM_DEV void dot(const float *A, const float *B, int tx, int ty, float (&s)[R][4]) {
  float2 acc[R][4];
#pragma unroll
  for (int r = 0; r < R; r++)
#pragma unroll
    for (int c = 0; c < 4; c++) acc[r][c] = make_float2(0.f, 0.f);
#pragma unroll 2
  for (int e = 0; e < HD; e += 4) {
    float4 b[4];
#pragma unroll
    for (int c = C0; c < C1; c++)
      b[c] = *reinterpret_cast<const float4 *>(B + (tx + 16 * c) * (HD + 4) + e);
#pragma unroll
    for (int r = 0; r < R; r++) {
      const float4 a = *reinterpret_cast<const float4 *>(A + (R * ty + r) * (HD + 4) + e);
#pragma unroll
      for (int c = C0; c < C1; c++) {
        acc[r][c] = __ffma2_rn(make_float2(a.x, a.y), make_float2(b[c].x, b[c].y), acc[r][c]);
        acc[r][c] = __ffma2_rn(make_float2(a.z, a.w), make_float2(b[c].z, b[c].w), acc[r][c]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; r++)
#pragma unroll
    for (int c = 0; c < 4; c++) s[r][c] = acc[r][c].x + acc[r][c].y;
}
// The warp's number within the block's rows: turned by the block, so that the
// warps with the most work of a diagonal tile do not all fall on one scheduler.
template <int HD>
LLM_DEV int row_warp() {
  return ((threadIdx.x >> 5) + (blockIdx.x >> 1)) & (threads_of<HD>() / 32 - 1);
}
template <int R>
LLM_DEV void put(float *P, const float (&p)[R][4], int tx, int ty) {
#pragma unroll
  for (int r = 0; r < R; r++)
#pragma unroll
    for (int c = 0; c < 4; c++) P[(R * ty + r) * LDP + ((tx + 16 * c) ^ ((ty & 1) * 16))] = p[r][c];
}
// out[r][c] += sum_k P[R ty + r][k] M[k][out_col(c)] over k in [k0, k1), multiples of 8
template <int HD, int R>
LLM_DEV void accumulate(const float *P, const float *M, int tx, int ty, float (&out)[R][HD / 16],
                        int k0, int k1) {
#pragma unroll 2
  for (int k = k0; k < k1; k += 4) {
    float4 p[R];
#pragma unroll
    for (int r = 0; r < R; r++)
      p[r] = *reinterpret_cast<const float4 *>(P + (R * ty + r) * LDP + (k ^ ((ty & 1) * 16)));
#pragma unroll
    for (int kk = 0; kk < 4; kk++) {
      float mv[HD / 16];
      const float *m = M + (k + kk) * (HD + 4);
      if constexpr (HD == 32) {
        const float2 v = *reinterpret_cast<const float2 *>(m + tx * 2);
        mv[0] = v.x; mv[1] = v.y;
      } else {
#pragma unroll
        for (int c = 0; c < HD / 16; c += 4) {
          const float4 v = *reinterpret_cast<const float4 *>(m + out_col<HD>(tx, c));
          mv[c] = v.x; mv[c + 1] = v.y; mv[c + 2] = v.z; mv[c + 3] = v.w;
        }
      }
#pragma unroll
      for (int r = 0; r < R; r++) {
        const float w = kk == 0 ? p[r].x : kk == 1 ? p[r].y : kk == 2 ? p[r].z : p[r].w;
#pragma unroll
        for (int c = 0; c < HD / 16; c++) out[r][c] = fmaf(w, mv[c], out[r][c]);
      }
    }
  }
}
LLM_DEV float half_max(float v) {
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
LLM_DEV float half_sum(float v) {
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <typename T, int HD>
LLM_DEV void put_row(T *dst, const float (&v)[HD / 16], float mul, int tx, int hd) {
#pragma unroll
  for (int c = 0; c < HD / 16; c++) {
    const int e = out_col<HD>(tx, c);
    if (e < hd) dst[e] = from_f<T>(v[c] * mul);
  }
}

// Shared memory: Q, K, V, P.
template <typename T, int HD>
__global__ void __launch_bounds__(threads_of<HD>())
    k_fwd(const T *__restrict__ qkv, int64_t ld, const PkTiles tl, T *__restrict__ o,
          float *__restrict__ lse, int64_t n_rows, int H, int Hkv, int hd, bool vec) {
  constexpr int R = rows_of<HD>();
  extern __shared__ float4 sm4[];
  float *Q = reinterpret_cast<float *>(sm4), *K = Q + tile_of<HD>(), *V = K + tile_of<HD>(),
        *P = V + tile_of<HD>();
  PkTile t;
  int h, half;
  if (!pk_item64(tl, H, t, h, half)) return;
  const int q0 = t.blk * PK_BLOCK + half * TB;
  if (q0 >= t.len) return;
  const int wr = row_warp<HD>(), tx = threadIdx.x & 15, ty = 2 * wr + (threadIdx.x >> 4 & 1);
  const int g = h / (H / Hkv), w0 = 2 * R * wr;  // the warp's first row: it has 2 R
  const float sl2 = LOG2E / sqrtf((float)hd);
  const T *base = qkv + (int64_t)t.row0 * ld;
  const T *kcol = base + (int64_t)(H + g) * hd, *vcol = base + (int64_t)(H + Hkv + g) * hd;
  const int nq = min(TB, t.len - q0);
  load_tile<T, HD>(Q, base + q0 * ld + (int64_t)h * hd, ld, nq, hd, vec);
  float m[R], l[R], acc[R][HD / 16];
#pragma unroll
  for (int r = 0; r < R; r++) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int c = 0; c < HD / 16; c++) acc[r][c] = 0.f;
  }
  for (int k0 = 0; k0 <= q0; k0 += TB) {
    __syncthreads();  // the previous tile's products are done with K and V
    const int nk = min(TB, t.len - k0);
    load_tile<T, HD>(K, kcol + k0 * ld, ld, nk, hd, vec);
    load_tile<T, HD>(V, vcol + k0 * ld, ld, nk, hd, vec);
    tiles_ready();
    if (w0 >= nq) continue;  // no row of the sequence
    // up to the warp's last row
    const bool diag = k0 == q0;
    float s[R][4];
    if (diag && w0 + 2 * R <= TB / 2) dot<HD, R, 0, 2>(Q, K, tx, ty, s);
    else dot<HD, R>(Q, K, tx, ty, s);
#pragma unroll
    for (int r = 0; r < R; r++) {
#pragma unroll
      for (int c = 0; c < 4; c++) {
        s[r][c] *= sl2;
        if (diag && tx + 16 * c > R * ty + r) s[r][c] = -INFINITY;
      }
      const float mn =
          fmaxf(m[r], half_max(fmaxf(fmaxf(s[r][0], s[r][1]), fmaxf(s[r][2], s[r][3]))));
      // a row whose scores are all -inf so far keeps the sums it has (0)
      const float ref = mn == -INFINITY ? 0.f : mn, corr = ex2(m[r] - ref);
#pragma unroll
      for (int c = 0; c < 4; c++) s[r][c] = ex2(s[r][c] - ref);
      l[r] = l[r] * corr + ((s[r][0] + s[r][1]) + (s[r][2] + s[r][3]));
      m[r] = mn;
#pragma unroll
      for (int c = 0; c < HD / 16; c++) acc[r][c] *= corr;
    }
    __syncwarp();  // P's rows are the warp's own
    put<R>(P, s, tx, ty);
    __syncwarp();
    accumulate<HD, R>(P, V, tx, ty, acc, 0, diag ? w0 + 2 * R : TB);
  }
#pragma unroll
  for (int r = 0; r < R; r++) {
    const float lt = half_sum(l[r]);
    const int q = q0 + R * ty + r;
    if (q >= t.len) continue;
    const int64_t row = (int64_t)t.row0 + q;
    put_row<T, HD>(o + row * ((int64_t)H * hd) + (int64_t)h * hd, acc[r], 1.f / lt, tx, hd);
    if (tx == 0) lse[(int64_t)h * n_rows + row] = (m[r] + log2f(lt)) * LN2;
  }
}

// dQ, and D = rowsum(dO o O) for the dK/dV kernel.  Shared memory: Q, dO, K,
// V, dS.
template <typename T, int HD>
__global__ void __launch_bounds__(threads_of<HD>())
    k_dq(const T *__restrict__ qkv, int64_t ld, const PkTiles tl, const T *__restrict__ o,
         const float *__restrict__ lse, const T *__restrict__ dout, float *__restrict__ D,
         T *__restrict__ dqkv, int64_t dld, int64_t n_rows, int H, int Hkv, int hd, bool vec) {
  constexpr int R = rows_of<HD>();
  extern __shared__ float4 sm4[];
  float *Q = reinterpret_cast<float *>(sm4), *G = Q + tile_of<HD>(), *K = G + tile_of<HD>(),
        *V = K + tile_of<HD>(), *S = V + tile_of<HD>();
  PkTile t;
  int h, half;
  if (!pk_item64(tl, H, t, h, half)) return;
  const int q0 = t.blk * PK_BLOCK + half * TB;
  if (q0 >= t.len) return;
  const int wr = row_warp<HD>(), tx = threadIdx.x & 15, ty = 2 * wr + (threadIdx.x >> 4 & 1);
  const int g = h / (H / Hkv), w0 = 2 * R * wr;  // the warp's first row: it has 2 R
  const int nq = min(TB, t.len - q0);
  const int64_t ow = (int64_t)H * hd;
  const float scale = 1.0f / sqrtf((float)hd), sl2 = scale * LOG2E;
  const T *base = qkv + (int64_t)t.row0 * ld;
  const T *kcol = base + (int64_t)(H + g) * hd, *vcol = base + (int64_t)(H + Hkv + g) * hd;
  const int64_t orow0 = ((int64_t)t.row0 + q0) * ow + (int64_t)h * hd;
  load_tile<T, HD>(Q, base + q0 * ld + (int64_t)h * hd, ld, nq, hd, vec);
  load_tile<T, HD>(G, dout + orow0, ow, nq, hd, vec);
  float Dr[R], Lr[R], dq[R][HD / 16];
#pragma unroll
  for (int r = 0; r < R; r++) {
    const int q = R * ty + r;
    float part = 0.f;
    if (q < nq)
#pragma unroll
      for (int c = 0; c < HD / 16; c++) {
        const int e = out_col<HD>(tx, c);
        if (e < hd) part += to_f(o[orow0 + q * ow + e]) * to_f(dout[orow0 + q * ow + e]);
      }
    Dr[r] = half_sum(part);
    const int64_t li = (int64_t)h * n_rows + t.row0 + q0 + q;
    Lr[r] = q < nq ? lse[li] * LOG2E : INFINITY;  // rows past the sequence: P = 0
    if (tx == 0 && q < nq) D[li] = Dr[r];
#pragma unroll
    for (int c = 0; c < HD / 16; c++) dq[r][c] = 0.f;
  }
  for (int k0 = 0; k0 <= q0; k0 += TB) {
    __syncthreads();
    const int nk = min(TB, t.len - k0);
    load_tile<T, HD>(K, kcol + k0 * ld, ld, nk, hd, vec);
    load_tile<T, HD>(V, vcol + k0 * ld, ld, nk, hd, vec);
    tiles_ready();
    if (w0 >= nq) continue;  // no row of the sequence
    const bool diag = k0 == q0;  // up to the warp's last row
    float s[R][4], dp[R][4];
    if (diag && w0 + 2 * R <= TB / 2) {
      dot<HD, R, 0, 2>(Q, K, tx, ty, s);
      dot<HD, R, 0, 2>(G, V, tx, ty, dp);
    } else {
      dot<HD, R>(Q, K, tx, ty, s);
      dot<HD, R>(G, V, tx, ty, dp);
    }
#pragma unroll
    for (int r = 0; r < R; r++)
#pragma unroll
      for (int c = 0; c < 4; c++) {
        const bool masked = diag && tx + 16 * c > R * ty + r;
        const float p = ex2(s[r][c] * sl2 - Lr[r]);
        s[r][c] = masked ? 0.f : p * (dp[r][c] - Dr[r]);
      }
    __syncwarp();  // S's rows are the warp's own
    put<R>(S, s, tx, ty);
    __syncwarp();
    accumulate<HD, R>(S, K, tx, ty, dq, 0, diag ? w0 + 2 * R : TB);
  }
#pragma unroll
  for (int r = 0; r < R; r++)
    if (R * ty + r < nq)
      put_row<T, HD>(dqkv + ((int64_t)t.row0 + q0 + R * ty + r) * dld + (int64_t)h * hd, dq[r],
                     scale, tx, hd);
}

// dK, dV of 64 keys: the query heads of the kv head in order, and for each
// the query tiles from the keys' own on.  Shared memory: K, V, Q, dO, a tile
// that holds P, then dS, and L and D of the queries.
template <typename T, int HD>
__global__ void __launch_bounds__(threads_of<HD>())
    k_dkv(const T *__restrict__ qkv, int64_t ld, const PkTiles tl, const float *__restrict__ lse,
          const T *__restrict__ dout, const float *__restrict__ D, T *__restrict__ dqkv,
          int64_t dld, int64_t n_rows, int H, int Hkv, int hd, bool vec) {
  constexpr int R = rows_of<HD>();
  extern __shared__ float4 sm4[];
  float *K = reinterpret_cast<float *>(sm4), *V = K + tile_of<HD>(), *Q = V + tile_of<HD>(),
        *G = Q + tile_of<HD>(), *P = G + tile_of<HD>(), *sL = P + TB * LDP, *sD = sL + TB;
  PkTile t;
  int g, half;
  if (!pk_item64(tl, Hkv, t, g, half)) return;
  const int n = (t.len + PK_BLOCK - 1) / PK_BLOCK;
  const int k0 = (n - 1 - t.blk) * PK_BLOCK + half * TB;
  if (k0 >= t.len) return;
  const int wr = row_warp<HD>(), tx = threadIdx.x & 15, ty = 2 * wr + (threadIdx.x >> 4 & 1);
  const int grp = H / Hkv, w0 = 2 * R * wr;  // the warp's first row: it has 2 R
  const int nk = min(TB, t.len - k0);
  const int64_t ow = (int64_t)H * hd;
  const float scale = 1.0f / sqrtf((float)hd), sl2 = scale * LOG2E;
  const T *base = qkv + (int64_t)t.row0 * ld;
  const T *kcol = base + (int64_t)(H + g) * hd, *vcol = base + (int64_t)(H + Hkv + g) * hd;
  load_tile<T, HD>(K, kcol + k0 * ld, ld, nk, hd, vec);
  load_tile<T, HD>(V, vcol + k0 * ld, ld, nk, hd, vec);
  float dk[R][HD / 16], dv[R][HD / 16];
#pragma unroll
  for (int r = 0; r < R; r++)
#pragma unroll
    for (int c = 0; c < HD / 16; c++) dk[r][c] = dv[r][c] = 0.f;
  for (int h = g * grp; h < (g + 1) * grp; h++) {
    for (int q0 = k0; q0 < t.len; q0 += TB) {
      __syncthreads();
      const int nq = min(TB, t.len - q0);
      load_tile<T, HD>(Q, base + q0 * ld + (int64_t)h * hd, ld, nq, hd, vec);
      load_tile<T, HD>(G, dout + ((int64_t)t.row0 + q0) * ow + (int64_t)h * hd, ow, nq, hd, vec);
      if (threadIdx.x < TB) {
        const int64_t li = (int64_t)h * n_rows + t.row0 + q0 + threadIdx.x;
        const bool in = (int)threadIdx.x < nq;
        sL[threadIdx.x] = in ? lse[li] * LOG2E : INFINITY;  // past the sequence: P = 0
        sD[threadIdx.x] = in ? ld_float(D + li) : 0.f;
      }
      tiles_ready();
      if (w0 >= nk) continue;  // no key of the sequence
      const bool diag = q0 == k0;  // from the warp's first key on
      float s[R][4], dp[R][4];  // rows keys, columns queries
      if (diag && w0 >= TB / 2) {
        dot<HD, R, 2, 4>(K, Q, tx, ty, s);
        dot<HD, R, 2, 4>(V, G, tx, ty, dp);
      } else {
        dot<HD, R>(K, Q, tx, ty, s);
        dot<HD, R>(V, G, tx, ty, dp);
      }
#pragma unroll
      for (int c = 0; c < 4; c++) {
        const float L = sL[tx + 16 * c], d = sD[tx + 16 * c];
#pragma unroll
        for (int r = 0; r < R; r++) {
          const bool masked = diag && R * ty + r > tx + 16 * c;
          const float e = masked ? 0.f : ex2(s[r][c] * sl2 - L);
          s[r][c] = e;
          dp[r][c] = masked ? 0.f : e * (dp[r][c] - d);
        }
      }
      __syncwarp();  // P's rows are the warp's own
      put<R>(P, s, tx, ty);
      __syncwarp();
      accumulate<HD, R>(P, G, tx, ty, dv, diag ? w0 : 0, TB);
      __syncwarp();  // one tile holds P, then dS
      put<R>(P, dp, tx, ty);
      __syncwarp();
      accumulate<HD, R>(P, Q, tx, ty, dk, diag ? w0 : 0, TB);
    }
  }
#pragma unroll
  for (int r = 0; r < R; r++) {
    if (R * ty + r >= nk) continue;
    T *dst = dqkv + ((int64_t)t.row0 + k0 + R * ty + r) * dld + (int64_t)(H + g) * hd;
    put_row<T, HD>(dst, dk[r], scale, tx, hd);
    put_row<T, HD>(dst + (int64_t)Hkv * hd, dv[r], 1.f, tx, hd);
  }
}

template <int HD> constexpr int fwd_smem() { return (3 * tile_of<HD>() + TB * LDP) * 4; }
template <int HD> constexpr int dq_smem() { return (4 * tile_of<HD>() + TB * LDP) * 4; }
template <int HD> constexpr int dkv_smem() { return (4 * tile_of<HD>() + TB * LDP + 2 * TB) * 4; }

template <typename T, int HD>
static bool fwd(const PkArgs &a, const PkPlan &p, void *o, float *lse, bool vec) {
  if (!smem_optin((const void *)k_fwd<T, HD>, fwd_smem<HD>())) return false;
  launch_dependent(
      k_fwd<T, HD>, dim3((unsigned)(2 * p.cap * a.H)), dim3(threads_of<HD>()), fwd_smem<HD>(), a.s,
      (const T *)a.qkv, a.ld, pk_tiles(a, p), (T *)o, lse, a.n_rows, a.H, a.Hkv, a.hd, vec);
  count_launch();
  return true;
}
template <typename T, int HD>
static bool bwd(const PkArgs &a, const PkPlan &p, const void *o, const float *lse,
                const void *dout, void *dqkv, int64_t dld, bool vec) {
  if (!smem_optin((const void *)k_dq<T, HD>, dq_smem<HD>()) ||
      !smem_optin((const void *)k_dkv<T, HD>, dkv_smem<HD>()))
    return false;
  launch_dependent(
      k_dq<T, HD>, dim3((unsigned)(2 * p.cap * a.H)), dim3(threads_of<HD>()), dq_smem<HD>(), a.s,
      (const T *)a.qkv, a.ld, pk_tiles(a, p), (const T *)o, lse, (const T *)dout, p.D,
      (T *)dqkv, dld, a.n_rows, a.H, a.Hkv, a.hd, vec);
  launch_dependent(
      k_dkv<T, HD>, dim3((unsigned)(2 * p.cap * a.Hkv)), dim3(threads_of<HD>()), dkv_smem<HD>(), a.s,
      (const T *)a.qkv, a.ld, pk_tiles(a, p), lse, (const T *)dout, p.D, (T *)dqkv, dld,
      a.n_rows, a.H, a.Hkv, a.hd, vec);
  count_launch(2);
  return true;
}
// 4-element loads need every row and head to start on one.
static bool vec4(const PkArgs &a, const void *p) {
  const int e = a.dt == DT_BF16 ? 2 : 4;
  return a.hd % 4 == 0 && a.ld % 4 == 0 && !((uintptr_t)p & (4 * e - 1));
}

}  // namespace pk

void packed_plan(const PkArgs &a, const PkPlan &p) {
  if (a.n_seq <= pk::FEW) {
    pk::k_plan_few<<<1, pk::FEW, 0, a.s>>>(a.cu, a.n_seq, (int)a.n_rows, p.n_tiles, p.tiles,
                                           a.flag);
    count_launch();
    return;
  }
  pk::k_plan<<<1, pk::PT, 0, a.s>>>(a.cu, a.n_seq, (int)a.n_rows, p.n_tiles, p.tiles, p.off,
                                    p.rank, a.flag);
  count_launch();
}

bool packed_fwd_tile(const PkArgs &a, const PkPlan &p, void *o, float *lse) {
  using namespace pk;
  if (pk_planned(a, p)) packed_plan(a, p);
  const bool v = vec4(a, a.qkv);
  if (a.dt == DT_BF16) {
    using T = __nv_bfloat16;
    return a.hd <= 32 ? fwd<T, 32>(a, p, o, lse, v)
                      : a.hd <= 64 ? fwd<T, 64>(a, p, o, lse, v) : fwd<T, 128>(a, p, o, lse, v);
  }
  return a.hd <= 32 ? fwd<float, 32>(a, p, o, lse, v)
                    : a.hd <= 64 ? fwd<float, 64>(a, p, o, lse, v)
                                 : fwd<float, 128>(a, p, o, lse, v);
}

bool packed_bwd_tile(const PkArgs &a, const PkPlan &p, const void *o, const float *lse,
                     const void *dout, void *dqkv, int64_t dld) {
  using namespace pk;
  if (pk_planned(a, p)) packed_plan(a, p);
  const bool v = vec4(a, a.qkv) && vec4(a, dout);
  if (a.dt == DT_BF16) {
    using T = __nv_bfloat16;
    return a.hd <= 32 ? bwd<T, 32>(a, p, o, lse, dout, dqkv, dld, v)
                      : a.hd <= 64 ? bwd<T, 64>(a, p, o, lse, dout, dqkv, dld, v)
                                   : bwd<T, 128>(a, p, o, lse, dout, dqkv, dld, v);
  }
  return a.hd <= 32 ? bwd<float, 32>(a, p, o, lse, dout, dqkv, dld, v)
                    : a.hd <= 64 ? bwd<float, 64>(a, p, o, lse, dout, dqkv, dld, v)
                                 : bwd<float, 128>(a, p, o, lse, dout, dqkv, dld, v);
}

}  // namespace llm
