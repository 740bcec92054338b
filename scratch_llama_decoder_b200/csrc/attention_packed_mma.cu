// Backward of causal attention over packed sequences on warp-level mma tiles,
// for bfloat16 head sizes past 64 (the tcgen05 backward's accumulators of a
// 128-wide head do not fit TMEM beside its scores) that are multiples of 8.
//
//   D_i = dO_i . O_i,  P = exp(s - L),  dS = P (dO_i . v_j - D_i)
//   dq = c dS k,  dk = c dS^T q,  dv = P^T dO,  c = 1/sqrt(hd)
//
// 64 x 64 tiles, 4 warps of 16 rows; tiles of 64 rows x 128 columns in shared
// memory (rows padded by 16 bytes, so that the 8 rows of an ldmatrix fall on
// different banks), columns past the head's and rows past the sequence's end
// zero.  Scores go half a tile (32 columns) at a time, which keeps the
// accumulators of a 16 x 128 result in registers beside them.  The sums run in
// a fixed order without atomics; P and dS enter the products as bfloat16.
#include "packed.cuh"
#include "tcgen05.cuh"

namespace llm {
namespace pk_mma {

constexpr int HD = 128, LD = HD + 8, NT = 128, TB = 64;
constexpr int TILE = TB * LD;  // elements
constexpr float LOG2E = 1.4426950408889634f;
using bf16 = __nv_bfloat16;

LLM_DEV uint32_t sm(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
LLM_DEV void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
LLM_DEV void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
LLM_DEV void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Rows [0, n) of src (row stride ld elements, hd columns) into a tile.
LLM_DEV void load(bf16 *t, const bf16 *src, int64_t ld, int n, int hd) {
#pragma unroll
  for (int i = threadIdx.x; i < TB * (HD / 8); i += NT) {
    const int r = i / (HD / 8), c = (i % (HD / 8)) * 8;
    const bool ok = r < n && c < hd;
    const bf16 *p = ok ? src + r * ld + c : src;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sm(t + r * LD + c)), "l"(p),
                 "r"(ok ? 16 : 0)
                 : "memory");
  }
}
LLM_DEV void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
LLM_DEV void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// A fragment of rows [16 w, 16 w + 16), columns [16 k, 16 k + 16) of a tile.
LLM_DEV void afrag(const bf16 *t, int w, int k, uint32_t (&a)[4]) {
  const int lane = threadIdx.x & 31;
  ldsm4(sm(t + (16 * w + (lane & 15)) * LD + 16 * k + (lane >> 4) * 8), a);
}
// s += A . X^T over rows [x0, x0 + 32) of tile X; A in registers, or the rows
// of warp w of a tile.
LLM_DEV void abt_step(float (&s)[4][4], const uint32_t (&a)[4], const bf16 *x, int x0, int k) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int np = 0; np < 2; np++) {
    uint32_t b[4];
    ldsm4(sm(x + (x0 + 16 * np + (lane & 7) + (lane >> 4) * 8) * LD + 16 * k +
             ((lane >> 3) & 1) * 8), b);
    mma(s[2 * np], a, b[0], b[1]);
    mma(s[2 * np + 1], a, b[2], b[3]);
  }
}
// acc[16 x HD] += P . Y over rows [y0, y0 + 32) of tile Y, P as C fragments.
LLM_DEV void ab(float (&acc)[HD / 8][4], const float (&p)[4][4], const bf16 *y, int y0) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < 2; k++) {
    const uint32_t a[4] = {tc::pack_bf16(p[2 * k][0], p[2 * k][1]),
                           tc::pack_bf16(p[2 * k][2], p[2 * k][3]),
                           tc::pack_bf16(p[2 * k + 1][0], p[2 * k + 1][1]),
                           tc::pack_bf16(p[2 * k + 1][2], p[2 * k + 1][3])};
#pragma unroll
    for (int np = 0; np < HD / 16; np++) {
      uint32_t b[4];
      ldsm4t(sm(y + (y0 + 16 * k + (lane & 15)) * LD + 16 * np + (lane >> 4) * 8), b);
      mma(acc[2 * np], a, b[0], b[1]);
      mma(acc[2 * np + 1], a, b[2], b[3]);
    }
  }
}
// Row r (0: lane / 4, 1: 8 further) of a warp's 16 x HD result times mul to
// dst, hd columns.
LLM_DEV void store_row(bf16 *dst, const float (&acc)[HD / 8][4], int r, float mul, int hd) {
  const int t = (threadIdx.x & 3) * 2;
#pragma unroll
  for (int i = 0; i < HD / 8; i++)
    if (8 * i + t < hd)
      *reinterpret_cast<uint32_t *>(dst + 8 * i + t) =
          tc::pack_bf16(acc[i][2 * r] * mul, acc[i][2 * r + 1] * mul);
}

// dQ of 64 queries, and D for the dK/dV kernel.  Shared memory: Q, dO, then
// K and V twice.
__global__ void __launch_bounds__(NT)
    k_dq(const bf16 *__restrict__ qkv, int64_t ld, const PkTiles tl, const bf16 *__restrict__ o,
         const float *__restrict__ lse, const bf16 *__restrict__ dout, float *__restrict__ D,
         bf16 *__restrict__ dqkv, int64_t dld, int64_t n_rows, int H, int Hkv, int hd) {
  extern __shared__ __align__(16) bf16 smem[];
  bf16 *Ks = smem, *Vs = smem + 2 * TILE;  // [2] each; Q and dO pass through the second ones
  PkTile t;
  int h, half;
  if (!pk_item64(tl, H, t, h, half)) return;
  const int q0 = t.blk * PK_BLOCK + half * TB;
  if (q0 >= t.len) return;
  const int w = threadIdx.x / 32, lane = threadIdx.x & 31, g = h / (H / Hkv);
  const int nq = min(TB, t.len - q0);
  const int64_t ow = (int64_t)H * hd, orow0 = ((int64_t)t.row0 + q0) * ow + (int64_t)h * hd;
  const float scale = 1.0f / sqrtf((float)hd), sl2 = scale * LOG2E;
  const bf16 *base = qkv + (int64_t)t.row0 * ld;
  const bf16 *kcol = base + (int64_t)(H + g) * hd, *vcol = base + (int64_t)(H + Hkv + g) * hd;
  load(Ks + TILE, base + q0 * ld + (int64_t)h * hd, ld, nq, hd);
  load(Vs + TILE, dout + orow0, ow, nq, hd);
  commit();
  load(Ks, kcol, ld, min(TB, t.len), hd);
  load(Vs, vcol, ld, min(TB, t.len), hd);
  commit();
  wait<1>();
  __syncthreads();
  uint32_t qf[HD / 16][4], df[HD / 16][4];
#pragma unroll
  for (int k = 0; k < HD / 16; k++) {
    afrag(Ks + TILE, w, k, qf[k]);
    afrag(Vs + TILE, w, k, df[k]);
  }
  float L2[2], Dr[2];
#pragma unroll
  for (int r = 0; r < 2; r++) {
    const int q = 16 * w + (lane >> 2) + 8 * r;
    // rows past the sequence: P = 0
    L2[r] = q < nq ? lse[(int64_t)h * n_rows + t.row0 + q0 + q] * LOG2E : INFINITY;
    Dr[r] = 0.f;
    if (q0 > 0 && q < nq) {  // D from dO's fragments and O read the same way
      const bf16 *orow = o + orow0 + q * ow;
#pragma unroll
      for (int k = 0; k < HD / 16; k++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
          const int c = 16 * k + 8 * e + (lane & 3) * 2;
          if (c < hd) {
            const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(orow + c));
            const float2 b =
                __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&df[k][2 * e + r]));
            Dr[r] += a.x * b.x + a.y * b.y;
          }
        }
    }
  }
  if (q0 == 0) {
    // a sequence's first 64 rows: D = sum_j P_ij dP_ij / sum_j P_ij of their one
    // tile (the quotient, so that P's own errors cancel where dP is the same for
    // all).  dO . O takes O as it was rounded to bf16, and where O has few terms
    // that error is as large as dS's own.
    float l[2] = {0.f, 0.f};
    wait<0>();
    __syncthreads();
#pragma unroll
    for (int hf = 0; hf < 2; hf++) {
      float s[4][4] = {}, dp[4][4] = {};
#pragma unroll
      for (int k = 0; k < HD / 16; k++) {
        abt_step(s, qf[k], Ks, 32 * hf, k);
        abt_step(dp, df[k], Vs, 32 * hf, k);
      }
#pragma unroll
      for (int nt = 0; nt < 4; nt++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const int r = e >> 1, q = 16 * w + (lane >> 2) + 8 * r;
          const int key = 32 * hf + 8 * nt + (lane & 3) * 2 + (e & 1);
          if (key <= q) {
            const float p = tc::ex2(s[nt][e] * sl2 - L2[r]);
            Dr[r] += p * dp[nt][e];
            l[r] += p;
          }
        }
    }
#pragma unroll
    for (int r = 0; r < 2; r++) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      Dr[r] = l[r] > 0.f ? Dr[r] / l[r] : 0.f;  // 0: a row past the sequence
    }
  }
#pragma unroll
  for (int r = 0; r < 2; r++) {
    Dr[r] += __shfl_xor_sync(0xffffffffu, Dr[r], 1);
    Dr[r] += __shfl_xor_sync(0xffffffffu, Dr[r], 2);
    const int q = 16 * w + (lane >> 2) + 8 * r;
    if ((lane & 3) == 0 && q < nq) D[(int64_t)h * n_rows + t.row0 + q0 + q] = Dr[r];
  }
  float acc[HD / 8][4];
#pragma unroll
  for (int i = 0; i < HD / 8; i++) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  for (int k0 = 0, cur = 0; k0 <= q0; k0 += TB, cur ^= 1) {
    __syncthreads();  // the other buffers (and Q, dO in them) have been read
    if (k0 + TB <= q0) {
      const int n = min(TB, t.len - k0 - TB);
      load(Ks + (cur ^ 1) * TILE, kcol + (k0 + TB) * ld, ld, n, hd);
      load(Vs + (cur ^ 1) * TILE, vcol + (k0 + TB) * ld, ld, n, hd);
    }
    commit();
    wait<1>();
    __syncthreads();
    const bf16 *K = Ks + cur * TILE, *V = Vs + cur * TILE;
#pragma unroll
    for (int hf = 0; hf < 2; hf++) {
      float s[4][4] = {}, dp[4][4] = {};
#pragma unroll
      for (int k = 0; k < HD / 16; k++) {
        abt_step(s, qf[k], K, 32 * hf, k);
        abt_step(dp, df[k], V, 32 * hf, k);
      }
#pragma unroll
      for (int nt = 0; nt < 4; nt++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const int r = e >> 1, q = 16 * w + (lane >> 2) + 8 * r;
          const int key = 32 * hf + 8 * nt + (lane & 3) * 2 + (e & 1);
          const bool masked = k0 == q0 && key > q;
          const float p = tc::ex2(s[nt][e] * sl2 - L2[r]);
          s[nt][e] = masked ? 0.f : p * (dp[nt][e] - Dr[r]);
        }
      ab(acc, s, K, 32 * hf);
    }
  }
#pragma unroll
  for (int r = 0; r < 2; r++) {
    const int q = 16 * w + (lane >> 2) + 8 * r;
    if (q < nq)
      store_row(dqkv + ((int64_t)t.row0 + q0 + q) * dld + (int64_t)h * hd, acc, r, scale, hd);
  }
}

// dK, dV of 64 keys: the kv head's query heads in order, and for each the
// query tiles from the keys' own on.  Shared memory: K, V, then Q and dO twice,
// and their L and D.
__global__ void __launch_bounds__(NT)
    k_dkv(const bf16 *__restrict__ qkv, int64_t ld, const PkTiles tl,
          const float *__restrict__ lse, const bf16 *__restrict__ dout,
          const float *__restrict__ D, bf16 *__restrict__ dqkv, int64_t dld, int64_t n_rows, int H,
          int Hkv, int hd) {
  extern __shared__ __align__(16) bf16 smem[];
  bf16 *Ks = smem, *Vs = Ks + TILE, *Qs = Vs + TILE, *Gs = Qs + 2 * TILE;
  float *Ls = reinterpret_cast<float *>(Gs + 2 * TILE), *Ds = Ls + 2 * TB;
  PkTile t;
  int g, half;
  if (!pk_item64(tl, Hkv, t, g, half)) return;
  const int n = (t.len + PK_BLOCK - 1) / PK_BLOCK;
  const int k0 = (n - 1 - t.blk) * PK_BLOCK + half * TB;
  if (k0 >= t.len) return;
  const int w = threadIdx.x / 32, lane = threadIdx.x & 31, grp = H / Hkv;
  const int nk = min(TB, t.len - k0), nqt = (t.len - k0 + TB - 1) / TB, steps = grp * nqt;
  const int64_t ow = (int64_t)H * hd;
  const float scale = 1.0f / sqrtf((float)hd), sl2 = scale * LOG2E;
  const bf16 *base = qkv + (int64_t)t.row0 * ld;
  load(Ks, base + k0 * ld + (int64_t)(H + g) * hd, ld, nk, hd);
  load(Vs, base + k0 * ld + (int64_t)(H + Hkv + g) * hd, ld, nk, hd);
  auto issue = [&](int st, int buf) {
    const int h = g * grp + st / nqt, q0 = k0 + (st % nqt) * TB, nq = min(TB, t.len - q0);
    load(Qs + buf * TILE, base + q0 * ld + (int64_t)h * hd, ld, nq, hd);
    load(Gs + buf * TILE, dout + ((int64_t)t.row0 + q0) * ow + (int64_t)h * hd, ow, nq, hd);
    if (threadIdx.x < TB) {
      const int64_t li = (int64_t)h * n_rows + t.row0 + q0 + threadIdx.x;
      const bool in = (int)threadIdx.x < nq;
      Ls[buf * TB + threadIdx.x] = in ? lse[li] * LOG2E : INFINITY;  // past the end: P = 0
      Ds[buf * TB + threadIdx.x] = in ? ld_float(D + li) : 0.f;
    }
  };
  issue(0, 0);
  commit();
  float dk[HD / 8][4], dv[HD / 8][4];
#pragma unroll
  for (int i = 0; i < HD / 8; i++)
#pragma unroll
    for (int e = 0; e < 4; e++) dk[i][e] = dv[i][e] = 0.f;
  for (int st = 0; st < steps; st++) {
    const int cur = st & 1;
    __syncthreads();  // the other buffers have been read
    if (st + 1 < steps) issue(st + 1, cur ^ 1);
    commit();
    wait<1>();
    __syncthreads();
    const bf16 *Q = Qs + cur * TILE, *G = Gs + cur * TILE;
    const bool diag = st % nqt == 0;
#pragma unroll
    for (int hf = 0; hf < 2; hf++) {
      float s[4][4] = {}, dp[4][4] = {};  // S^T, dP^T: rows keys, columns 32 queries
#pragma unroll
      for (int k = 0; k < HD / 16; k++) {
        uint32_t a[4];
        afrag(Ks, w, k, a);
        abt_step(s, a, Q, 32 * hf, k);
        afrag(Vs, w, k, a);
        abt_step(dp, a, G, 32 * hf, k);
      }
#pragma unroll
      for (int nt = 0; nt < 4; nt++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const int key = 16 * w + (lane >> 2) + 8 * (e >> 1);
          const int q = 32 * hf + 8 * nt + (lane & 3) * 2 + (e & 1);
          const bool masked = diag && key > q;
          const float p = masked ? 0.f : tc::ex2(s[nt][e] * sl2 - Ls[cur * TB + q]);
          s[nt][e] = p;
          dp[nt][e] = masked ? 0.f : p * (dp[nt][e] - Ds[cur * TB + q]);
        }
      ab(dv, s, G, 32 * hf);
      ab(dk, dp, Q, 32 * hf);
    }
  }
#pragma unroll
  for (int r = 0; r < 2; r++) {
    const int key = 16 * w + (lane >> 2) + 8 * r;
    if (key >= nk) continue;
    bf16 *dst = dqkv + ((int64_t)t.row0 + k0 + key) * dld + (int64_t)(H + g) * hd;
    store_row(dst, dk, r, scale, hd);
    store_row(dst + (int64_t)Hkv * hd, dv, r, 1.f, hd);
  }
}

constexpr int DQ_SMEM = 4 * TILE * 2, DKV_SMEM = 6 * TILE * 2 + 4 * TB * 4;

}  // namespace pk_mma

bool packed_bwd_mma(const PkArgs &a, const PkPlan &p, const void *o, const float *lse,
                    const void *dout, void *dqkv, int64_t dld) {
  using namespace pk_mma;
  if (a.dt != DT_BF16 || a.hd % 8 || a.ld % 8 || dld % 2 ||
      (((uintptr_t)a.qkv | (uintptr_t)dout) & 15) || (((uintptr_t)o | (uintptr_t)dqkv) & 3))
    return false;
  if (!smem_optin((const void *)k_dq, DQ_SMEM) || !smem_optin((const void *)k_dkv, DKV_SMEM))
    return false;
  if (pk_planned(a, p)) packed_plan(a, p);
  launch_dependent(k_dq, dim3((unsigned)(2 * p.cap * a.H)), dim3(NT), DQ_SMEM, a.s,
                   (const bf16 *)a.qkv, a.ld, pk_tiles(a, p), (const bf16 *)o, lse,
                   (const bf16 *)dout, p.D, (bf16 *)dqkv, dld, a.n_rows, a.H, a.Hkv, a.hd);
  launch_dependent(k_dkv, dim3((unsigned)(2 * p.cap * a.Hkv)), dim3(NT), DKV_SMEM, a.s,
                   (const bf16 *)a.qkv, a.ld, pk_tiles(a, p), lse, (const bf16 *)dout, p.D,
                   (bf16 *)dqkv, dld, a.n_rows, a.H, a.Hkv, a.hd);
  count_launch(2);
  return true;
}

}  // namespace llm
