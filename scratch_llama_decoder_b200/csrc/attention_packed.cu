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
                                             int block, int *flag) {
  __shared__ int hist[MAXC + 2];  // sequences of exactly n blocks; then cnt, then off
  pk_release();
  __shared__ int warp_tot[32];
  const int C = (n_rows + block - 1) / block;
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
    const int n = (off[s + 1] - off[s] + block - 1) / block;
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
    const int n = (off[s + 1] - off[s] + block - 1) / block;
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
    const int row0 = off[s], len = off[s + 1] - row0, n = (len + block - 1) / block;
    for (int b = threadIdx.x & 31; b < n; b += 32)
      tiles[hist[b + 1] + rank[s]] = PkTile{row0, len, b, 0};
  }
}

// The same plan for few sequences, where the scans' barriers would take longer
// than counting: off(c) = sum over the sequences of max(0, n - c), and a
// sequence's rank by comparing it with every other one.
constexpr int FEW = 256;
__global__ void __launch_bounds__(FEW) k_plan_few(const int32_t *__restrict__ cu, int n_seq,
                                                  int n_rows, int *__restrict__ n_tiles,
                                                  PkTile *__restrict__ tiles, int block, int *flag) {
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
  const int n = t < n_seq ? (off[t + 1] - off[t] + block - 1) / block : 0;
  if (t < n_seq) blocks[t] = n;
  __syncthreads();
  if (t < n_seq) {
    int r = 0;
    for (int s = 0; s < n_seq; s++) r += blocks[s] > n || (blocks[s] == n && s < t);
    rank[t] = r;
  }
  const int C = (n_rows + block - 1) / block;
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
      tiles[base[b + 1] + rank[s]] = PkTile{off[s], off[s + 1] - off[s], b, 0};
}

// --------------------------------------------------------- CUDA-core kernels
// 64 x 64 tiles in shared memory, 256 threads (tx, ty) of 4 x 4 scores each.
// Operands of a score product sit transposed ([column][row], rows padded by
// 4), operands of an accumulation row by row; a probability tile as
// [column][row] float4 slots, slot ty of column k at ty ^ (k / 4), so that a
// half-warp's float4 stores fall on different banks.  Head columns past hd
// are zero, so a head size runs on the next of 32, 64, 128.
constexpr int TB = 64, TLD = TB + 4, NT = 256;

LLM_DEV int slot(int k, int g4) { return k * TB + ((g4 ^ (k >> 2)) & 15) * 4; }
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
// Rows [0, nrows) of src (row stride ld), hd columns, times mul: transposed
// into At and/or row by row into Mr; the other rows read as 0.
template <typename T, int HD>
LLM_DEV void load_tile(const T *src, int64_t ld, int nrows, int hd, bool vec, float mul, float *At,
                       float *Mr) {
  for (int i = threadIdx.x; i < TB * HD / 4; i += NT) {
    const int row = i % TB, c = i / TB * 4;
    float4 v = row < nrows && c < hd ? read4(src + row * ld + c, vec, hd - c)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
    v.x *= mul; v.y *= mul; v.z *= mul; v.w *= mul;
    if (At) {
      At[(c + 0) * TLD + row] = v.x;
      At[(c + 1) * TLD + row] = v.y;
      At[(c + 2) * TLD + row] = v.z;
      At[(c + 3) * TLD + row] = v.w;
    }
    if (Mr) *reinterpret_cast<float4 *>(Mr + row * HD + c) = v;
  }
}
template <int HD>
LLM_DEV void dot(const float *At, const float *Bt, int tx, int ty, float (&acc)[4][4]) {
#pragma unroll 8
  for (int e = 0; e < HD; e++) {
    const float4 a = *reinterpret_cast<const float4 *>(At + e * TLD + ty * 4);
    const float4 b = *reinterpret_cast<const float4 *>(Bt + e * TLD + tx * 4);
    const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int r = 0; r < 4; r++)
#pragma unroll
      for (int c = 0; c < 4; c++) acc[r][c] = fmaf(av[r], bv[c], acc[r][c]);
  }
}
template <int HD>
LLM_DEV void accumulate(const float *P, const float *M, int tx, int ty, float (&out)[4][HD / 16]) {
#pragma unroll 4
  for (int k = 0; k < TB; k++) {
    const float4 p = *reinterpret_cast<const float4 *>(P + slot(k, ty));
    const float pv[4] = {p.x, p.y, p.z, p.w};
    float mv[HD / 16];
    if constexpr (HD == 32) {
      const float2 m = *reinterpret_cast<const float2 *>(M + k * HD + tx * 2);
      mv[0] = m.x; mv[1] = m.y;
    } else {
#pragma unroll
      for (int c = 0; c < HD / 16; c += 4) {
        const float4 m = *reinterpret_cast<const float4 *>(M + k * HD + out_col<HD>(tx, c));
        mv[c] = m.x; mv[c + 1] = m.y; mv[c + 2] = m.z; mv[c + 3] = m.w;
      }
    }
#pragma unroll
    for (int r = 0; r < 4; r++)
#pragma unroll
      for (int c = 0; c < HD / 16; c++) out[r][c] = fmaf(pv[r], mv[c], out[r][c]);
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
__global__ void __launch_bounds__(NT)
    k_fwd(const T *__restrict__ qkv, int64_t ld, const PkTiles tl, T *__restrict__ o, float *__restrict__ lse,
          int64_t n_rows, int H, int Hkv, int hd, bool vec) {
  extern __shared__ float4 sm4[];
  float *Qt = reinterpret_cast<float *>(sm4), *Kt = Qt + HD * TLD, *Vs = Kt + HD * TLD,
        *Pt = Vs + TB * HD;
  PkTile t;
  int h, half;
  if (!pk_item64(tl, H, t, h, half)) return;
  const int q0 = t.blk * PK_BLOCK + half * TB;
  if (q0 >= t.len) return;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, g = h / (H / Hkv);
  const T *base = qkv + (int64_t)t.row0 * ld;
  const T *kcol = base + (int64_t)(H + g) * hd, *vcol = base + (int64_t)(H + Hkv + g) * hd;
  load_tile<T, HD>(base + q0 * ld + (int64_t)h * hd, ld, min(TB, t.len - q0), hd, vec,
                   1.0f / sqrtf((float)hd), Qt, nullptr);
  float m[4], l[4], acc[4][HD / 16];
#pragma unroll
  for (int r = 0; r < 4; r++) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int c = 0; c < HD / 16; c++) acc[r][c] = 0.f;
  }
  for (int k0 = 0; k0 <= q0; k0 += TB) {
    __syncthreads();  // the previous tile's products are done with Kt, Vs and Pt
    const int nk = min(TB, t.len - k0);
    load_tile<T, HD>(kcol + k0 * ld, ld, nk, hd, vec, 1.f, Kt, nullptr);
    load_tile<T, HD>(vcol + k0 * ld, ld, nk, hd, vec, 1.f, nullptr, Vs);
    __syncthreads();
    float s[4][4] = {};
    dot<HD>(Qt, Kt, tx, ty, s);
    if (k0 == q0) {
#pragma unroll
      for (int r = 0; r < 4; r++)
#pragma unroll
        for (int c = 0; c < 4; c++)
          if (tx * 4 + c > ty * 4 + r) s[r][c] = -INFINITY;
    }
    float p[4][4];
#pragma unroll
    for (int r = 0; r < 4; r++) {
      const float mn =
          fmaxf(m[r], half_max(fmaxf(fmaxf(s[r][0], s[r][1]), fmaxf(s[r][2], s[r][3]))));
      // a row whose scores are all -inf so far keeps the sums it has (0)
      const float ref = mn == -INFINITY ? 0.f : mn;
      const float corr = expf(m[r] - ref);
      float ps = 0.f;
#pragma unroll
      for (int c = 0; c < 4; c++) {
        p[c][r] = expf(s[r][c] - ref);
        ps += p[c][r];
      }
      l[r] = l[r] * corr + ps;
      m[r] = mn;
#pragma unroll
      for (int c = 0; c < HD / 16; c++) acc[r][c] *= corr;
    }
#pragma unroll
    for (int c = 0; c < 4; c++)
      *reinterpret_cast<float4 *>(Pt + slot(tx * 4 + c, ty)) =
          make_float4(p[c][0], p[c][1], p[c][2], p[c][3]);
    __syncthreads();
    accumulate<HD>(Pt, Vs, tx, ty, acc);
  }
#pragma unroll
  for (int r = 0; r < 4; r++) {
    const float lt = half_sum(l[r]);
    const int q = q0 + ty * 4 + r;
    if (q >= t.len) continue;
    const int64_t row = (int64_t)t.row0 + q;
    T *orow = o + row * ((int64_t)H * hd) + (int64_t)h * hd;
#pragma unroll
    for (int c = 0; c < HD / 16; c++) {
      const int e = out_col<HD>(tx, c);
      if (e < hd) orow[e] = from_f<T>(acc[r][c] / lt);
    }
    if (tx == 0) lse[(int64_t)h * n_rows + row] = m[r] + logf(lt);
  }
}

// dQ, and D = rowsum(dO o O) for the dK/dV kernel.
template <typename T, int HD>
__global__ void __launch_bounds__(NT)
    k_dq(const T *__restrict__ qkv, int64_t ld, const PkTiles tl, const T *__restrict__ o, const float *__restrict__ lse,
         const T *__restrict__ dout, float *__restrict__ D, T *__restrict__ dqkv, int64_t dld,
         int64_t n_rows, int H, int Hkv, int hd, bool vec) {
  extern __shared__ float4 sm4[];
  float *Qt = reinterpret_cast<float *>(sm4), *dOt = Qt + HD * TLD, *Kt = dOt + HD * TLD,
        *Vt = Kt + HD * TLD, *Kr = Vt + HD * TLD, *dSt = Kr + TB * HD;
  PkTile t;
  int h, half;
  if (!pk_item64(tl, H, t, h, half)) return;
  const int q0 = t.blk * PK_BLOCK + half * TB;
  if (q0 >= t.len) return;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, g = h / (H / Hkv);
  const int nq = min(TB, t.len - q0);
  const int64_t ow = (int64_t)H * hd;
  const float scale = 1.0f / sqrtf((float)hd);
  const T *base = qkv + (int64_t)t.row0 * ld;
  const T *kcol = base + (int64_t)(H + g) * hd, *vcol = base + (int64_t)(H + Hkv + g) * hd;
  const int64_t orow0 = ((int64_t)t.row0 + q0) * ow + (int64_t)h * hd;
  load_tile<T, HD>(base + q0 * ld + (int64_t)h * hd, ld, nq, hd, vec, scale, Qt, nullptr);
  load_tile<T, HD>(dout + orow0, ow, nq, hd, vec, 1.f, dOt, nullptr);
  float Dr[4], Lr[4], dq[4][HD / 16];
#pragma unroll
  for (int r = 0; r < 4; r++) {
    const int q = ty * 4 + r;
    float part = 0.f;
    if (q < nq)
      for (int c = 0; c < HD / 16; c++) {
        const int e = out_col<HD>(tx, c);
        if (e < hd) part += to_f(o[orow0 + q * ow + e]) * to_f(dout[orow0 + q * ow + e]);
      }
    Dr[r] = half_sum(part);
    const int64_t li = (int64_t)h * n_rows + t.row0 + q0 + q;
    Lr[r] = q < nq ? lse[li] : INFINITY;  // rows past the sequence: P = 0
    if (tx == 0 && q < nq) D[li] = Dr[r];
#pragma unroll
    for (int c = 0; c < HD / 16; c++) dq[r][c] = 0.f;
  }
  for (int k0 = 0; k0 <= q0; k0 += TB) {
    __syncthreads();
    const int nk = min(TB, t.len - k0);
    load_tile<T, HD>(kcol + k0 * ld, ld, nk, hd, vec, 1.f, Kt, Kr);
    load_tile<T, HD>(vcol + k0 * ld, ld, nk, hd, vec, 1.f, Vt, nullptr);
    __syncthreads();
    float s[4][4] = {}, dp[4][4] = {};
    dot<HD>(Qt, Kt, tx, ty, s);
    dot<HD>(dOt, Vt, tx, ty, dp);
    float ds[4][4];
#pragma unroll
    for (int r = 0; r < 4; r++)
#pragma unroll
      for (int c = 0; c < 4; c++) {
        const bool masked = k0 == q0 && tx * 4 + c > ty * 4 + r;
        const float p = expf(s[r][c] - Lr[r]);
        ds[c][r] = masked ? 0.f : p * (dp[r][c] - Dr[r]);
      }
#pragma unroll
    for (int c = 0; c < 4; c++)
      *reinterpret_cast<float4 *>(dSt + slot(tx * 4 + c, ty)) =
          make_float4(ds[c][0], ds[c][1], ds[c][2], ds[c][3]);
    __syncthreads();
    accumulate<HD>(dSt, Kr, tx, ty, dq);
  }
#pragma unroll
  for (int r = 0; r < 4; r++) {
    const int q = ty * 4 + r;
    if (q >= nq) continue;
    T *dst = dqkv + ((int64_t)t.row0 + q0 + q) * dld + (int64_t)h * hd;
#pragma unroll
    for (int c = 0; c < HD / 16; c++) {
      const int e = out_col<HD>(tx, c);
      if (e < hd) dst[e] = from_f<T>(dq[r][c] * scale);
    }
  }
}

// dK, dV of 64 keys: the query heads of the kv head in order, and for each
// the query tiles from the keys' own on.
template <typename T, int HD>
__global__ void __launch_bounds__(NT)
    k_dkv(const T *__restrict__ qkv, int64_t ld, const PkTiles tl, const float *__restrict__ lse,
          const T *__restrict__ dout, const float *__restrict__ D, T *__restrict__ dqkv,
          int64_t dld, int64_t n_rows, int H, int Hkv, int hd, bool vec) {
  extern __shared__ float4 sm4[];
  float *Kt = reinterpret_cast<float *>(sm4), *Vt = Kt + HD * TLD, *Qt = Vt + HD * TLD,
        *dOt = Qt + HD * TLD, *Qr = dOt + HD * TLD, *dOr = Qr + TB * HD, *Ps = dOr + TB * HD,
        *sL = Ps + TB * TB, *sD = sL + TB;
  PkTile t;
  int g, half;
  if (!pk_item64(tl, Hkv, t, g, half)) return;
  const int n = (t.len + PK_BLOCK - 1) / PK_BLOCK;
  const int k0 = (n - 1 - t.blk) * PK_BLOCK + half * TB;
  if (k0 >= t.len) return;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, grp = H / Hkv;
  const int nk = min(TB, t.len - k0);
  const int64_t ow = (int64_t)H * hd;
  const float scale = 1.0f / sqrtf((float)hd);
  const T *base = qkv + (int64_t)t.row0 * ld;
  const T *kcol = base + (int64_t)(H + g) * hd, *vcol = base + (int64_t)(H + Hkv + g) * hd;
  load_tile<T, HD>(kcol + k0 * ld, ld, nk, hd, vec, 1.f, Kt, nullptr);
  load_tile<T, HD>(vcol + k0 * ld, ld, nk, hd, vec, 1.f, Vt, nullptr);
  float dk[4][HD / 16], dv[4][HD / 16];
#pragma unroll
  for (int r = 0; r < 4; r++)
#pragma unroll
    for (int c = 0; c < HD / 16; c++) dk[r][c] = dv[r][c] = 0.f;
  for (int h = g * grp; h < (g + 1) * grp; h++) {
    for (int q0 = k0; q0 < t.len; q0 += TB) {
      __syncthreads();
      const int nq = min(TB, t.len - q0);
      load_tile<T, HD>(base + q0 * ld + (int64_t)h * hd, ld, nq, hd, vec, scale, Qt, Qr);
      load_tile<T, HD>(dout + ((int64_t)t.row0 + q0) * ow + (int64_t)h * hd, ow, nq, hd, vec, 1.f,
                       dOt, dOr);
      if (threadIdx.x < TB) {
        const int64_t li = (int64_t)h * n_rows + t.row0 + q0 + threadIdx.x;
        const bool in = (int)threadIdx.x < nq;
        sL[threadIdx.x] = in ? lse[li] : INFINITY;  // queries past the sequence: P = 0
        sD[threadIdx.x] = in ? ld_float(D + li) : 0.f;
      }
      __syncthreads();
      float s[4][4] = {}, dp[4][4] = {};
      dot<HD>(Kt, Qt, tx, ty, s);  // rows keys, columns queries
      dot<HD>(Vt, dOt, tx, ty, dp);
      float p[4][4], ds[4][4];
#pragma unroll
      for (int r = 0; r < 4; r++)
#pragma unroll
        for (int c = 0; c < 4; c++) {
          const bool masked = q0 == k0 && ty * 4 + r > tx * 4 + c;
          const float e = masked ? 0.f : expf(s[r][c] - sL[tx * 4 + c]);
          p[c][r] = e;
          ds[c][r] = masked ? 0.f : e * (dp[r][c] - sD[tx * 4 + c]);
        }
#pragma unroll
      for (int c = 0; c < 4; c++)
        *reinterpret_cast<float4 *>(Ps + slot(tx * 4 + c, ty)) =
            make_float4(p[c][0], p[c][1], p[c][2], p[c][3]);
      __syncthreads();
      accumulate<HD>(Ps, dOr, tx, ty, dv);
      __syncthreads();  // one tile holds P, then dS: head 128 has no room for both
#pragma unroll
      for (int c = 0; c < 4; c++)
        *reinterpret_cast<float4 *>(Ps + slot(tx * 4 + c, ty)) =
            make_float4(ds[c][0], ds[c][1], ds[c][2], ds[c][3]);
      __syncthreads();
      accumulate<HD>(Ps, Qr, tx, ty, dk);  // Qr holds q / sqrt(hd)
    }
  }
#pragma unroll
  for (int r = 0; r < 4; r++) {
    if (ty * 4 + r >= nk) continue;
    T *dkr = dqkv + ((int64_t)t.row0 + k0 + ty * 4 + r) * dld + (int64_t)(H + g) * hd;
    T *dvr = dkr + (int64_t)Hkv * hd;
#pragma unroll
    for (int c = 0; c < HD / 16; c++) {
      const int e = out_col<HD>(tx, c);
      if (e < hd) {
        dkr[e] = from_f<T>(dk[r][c]);
        dvr[e] = from_f<T>(dv[r][c]);
      }
    }
  }
}

template <int HD> constexpr int fwd_smem() { return (2 * HD * TLD + TB * HD + TB * TB) * 4; }
template <int HD> constexpr int dq_smem() { return (4 * HD * TLD + TB * HD + TB * TB) * 4; }
template <int HD>
constexpr int dkv_smem() { return (4 * HD * TLD + 2 * TB * HD + TB * TB + 2 * TB) * 4; }

template <typename T, int HD>
static bool fwd(const PkArgs &a, const PkPlan &p, void *o, float *lse, bool vec) {
  if (!smem_optin((const void *)k_fwd<T, HD>, fwd_smem<HD>())) return false;
  launch_dependent(
      k_fwd<T, HD>, dim3((unsigned)(2 * p.cap * a.H)), dim3(NT), fwd_smem<HD>(), a.s,
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
      k_dq<T, HD>, dim3((unsigned)(2 * p.cap * a.H)), dim3(NT), dq_smem<HD>(), a.s,
      (const T *)a.qkv, a.ld, pk_tiles(a, p), (const T *)o, lse, (const T *)dout, p.D,
      (T *)dqkv, dld, a.n_rows, a.H, a.Hkv, a.hd, vec);
  launch_dependent(
      k_dkv<T, HD>, dim3((unsigned)(2 * p.cap * a.Hkv)), dim3(NT), dkv_smem<HD>(), a.s,
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

void packed_plan(const PkArgs &a, const PkPlan &p, int block) {
  if (a.n_seq <= pk::FEW) {
    pk::k_plan_few<<<1, pk::FEW, 0, a.s>>>(a.cu, a.n_seq, (int)a.n_rows, p.n_tiles, p.tiles,
                                           block, a.flag);
    count_launch();
    return;
  }
  pk::k_plan<<<1, pk::PT, 0, a.s>>>(a.cu, a.n_seq, (int)a.n_rows, p.n_tiles, p.tiles, p.off,
                                    p.rank, block, a.flag);
  count_launch();
}

bool packed_fwd_tile(const PkArgs &a, const PkPlan &p, void *o, float *lse) {
  using namespace pk;
  if (pk_planned(a, p)) packed_plan(a, p, PK_BLOCK);
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
  if (pk_planned(a, p)) packed_plan(a, p, PK_BLOCK);
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
