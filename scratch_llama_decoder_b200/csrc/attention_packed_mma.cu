// Causal attention over packed sequences on warp-level mma tiles, for bfloat16
// head sizes that are multiples of 8: both directions of short sequences, and
// the backward of head sizes past 64 (the tcgen05 backward is built for tiles of
// 64 columns; at 128 its S, dP, dK and dV take all 512 columns of TMEM, so P and
// dS would have to lie over S and dP, which it does not do).
//
//   o_i = sum_j P_ij v_j,  P = exp(s - L),  L_i = ln sum_j exp(s_ij)
//   D_i = dO_i . O_i,  dS = P (dO_i . v_j - D_i)
//   dq = c dS k,  dk = c dS^T q,  dv = P^T dO,  c = 1/sqrt(hd)
//
// 64 x 64 tiles, 4 warps of 16 rows; tiles of 64 rows x 32, 64 or 128 columns
// in shared memory (rows padded by 16 bytes, so that the 8 rows of an ldmatrix
// fall on different banks), columns past the head's and rows past the
// sequence's end zero.  Scores of the backward go half a tile (32 columns) at
// a time, which keeps the accumulators of a 16 x 128 result in registers
// beside them; halves that the mask empties are left out, and so are warps
// whose rows lie past the end.  The sums run in a fixed order without atomics;
// P and dS enter the products as bfloat16, their operands' type: each term is off
// by 2^-8 of itself at most, beside outputs that are rounded by as much (error of
// out and dqkv 0.0020 to 0.0023 against 0.0016 from the last rounding alone); a
// second term of each would double the products that take them.
//
// The tcgen05 kernels have one or two 128-row items in flight on an SM, each a
// chain of loads, products, softmax and store: 4 us an item (20 us forward and
// backward) however few rows it has.  These have 2 to 4 blocks of 64 rows, at a
// third of the rate.  So they win where sequences are short, by the mean of
// n_rows / n_seq (16384 rows, 8 heads, us, these and tcgen05's):
//   forward   heads of 32: 64 rows 28, 50; 192: 27, 35; 256: 28, 27
//             64: 64 rows 36, 50; 80: 45, 41   128: 64: 57, 63; 96: 67, 47
//             one wave of blocks (4 sequences), heads of 64: 128: 5.6, 7.0; 256:
//             9.8, 8.6; of 128: 128: 8.1, 7.8
//   backward  heads of 32: 64 rows 48, 160; 256: 61, 78; 320: 68, 105; 512: 89, 90
//             (2 kv heads 320: 80, 94; 384: 89, 75); 64: 64 rows 76, 166; 192: 95,
//             114; 256: 106, 84 (2 kv heads 128: 74, 66)
//             few blocks: 16 sequences, 2 kv heads of 32: 128: 21, 23; 256: 35, 33;
//             of 64: 64: 22, 23; 100: 38, 24
// Those are sequences of one length.  The mean is all that the host knows (the
// offsets lie on the device), so where empty slots or many short sequences stand
// beside a long one it is taken for short: 4096 rows alone and with 63 empty
// sequences, us, forward 51, 109, backward 223, 911 (8/2 heads of 64), 51, 80
// and 86, 187 (8 of 32); 16384 rows with 63 empty ones, 8 heads of 32, 390, 709
// and 1077, 1834; 12000 rows and 63 of 60, apart and in one call, 241, 411 and
// 618, 1029; 15876 and 127 of 4, 16 heads of 64, backward, 2258, 5717.  Where the
// mean is past the threshold all the same, nothing is lost: 16384 rows with 63
// empty ones, 16 heads of 64, 751, 754 and 2369, 2287.
#include "packed.cuh"
#include "tcgen05.cuh"

namespace llm {
namespace pk_mma {

constexpr int NT = 128, TB = 64;
// Blocks per SM that registers are cut for (5 at heads of 32: spills, twice the time).
constexpr int per_sm(int hd) { return hd == 32 ? 4 : hd == 64 ? 3 : 2; }
template <int HD> constexpr int LD = HD + 8;          // row of a tile
template <int HD> constexpr int TILE = TB * LD<HD>;  // elements
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
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
template <int HD>
LLM_DEV void load(bf16 *t, const bf16 *src, int64_t ld, int n, int hd) {
#pragma unroll
  for (int i = threadIdx.x; i < TB * (HD / 8); i += NT) {
    const int r = i / (HD / 8), c = (i % (HD / 8)) * 8;
    const bool ok = r < n && c < hd;
    const bf16 *p = ok ? src + r * ld + c : src;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sm(t + r * LD<HD> + c)), "l"(p),
                 "r"(ok ? 16 : 0)
                 : "memory");
  }
}
LLM_DEV void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
LLM_DEV void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// A fragment of rows [16 w, 16 w + 16), columns [16 k, 16 k + 16) of a tile.
template <int HD>
LLM_DEV void afrag(const bf16 *t, int w, int k, uint32_t (&a)[4]) {
  const int lane = threadIdx.x & 31;
  ldsm4(sm(t + (16 * w + (lane & 15)) * LD<HD> + 16 * k + (lane >> 4) * 8), a);
}
// s += A . X^T over rows [x0, x0 + 32) of tile X; A in registers, or the rows
// of warp w of a tile.
template <int HD>
LLM_DEV void abt_step(float (&s)[4][4], const uint32_t (&a)[4], const bf16 *x, int x0, int k) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int np = 0; np < 2; np++) {
    uint32_t b[4];
    ldsm4(sm(x + (x0 + 16 * np + (lane & 7) + (lane >> 4) * 8) * LD<HD> + 16 * k +
             ((lane >> 3) & 1) * 8), b);
    mma(s[2 * np], a, b[0], b[1]);
    mma(s[2 * np + 1], a, b[2], b[3]);
  }
}
// acc[16 x HD] += P . Y over rows [y0, y0 + 32) of tile Y, P as C fragments.
template <int HD>
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
      ldsm4t(sm(y + (y0 + 16 * k + (lane & 15)) * LD<HD> + 16 * np + (lane >> 4) * 8), b);
      mma(acc[2 * np], a, b[0], b[1]);
      mma(acc[2 * np + 1], a, b[2], b[3]);
    }
  }
}
// Row r (0: lane / 4, 1: 8 further) of a warp's 16 x HD result times mul to
// dst, hd columns.
template <int HD>
LLM_DEV void store_row(bf16 *dst, const float (&acc)[HD / 8][4], int r, float mul, int hd) {
  const int t = (threadIdx.x & 3) * 2;
#pragma unroll
  for (int i = 0; i < HD / 8; i++)
    if (8 * i + t < hd)
      *reinterpret_cast<uint32_t *>(dst + 8 * i + t) =
          tc::pack_bf16(acc[i][2 * r] * mul, acc[i][2 * r + 1] * mul);
}

// O and L of 64 queries.  Shared memory: K and V twice; Q passes through the
// second K.
template <int HD>
__global__ void __launch_bounds__(NT, per_sm(HD))
    k_fwd(const bf16 *__restrict__ qkv, int64_t ld, const PkTiles tl, bf16 *__restrict__ o,
          float *__restrict__ lse, int64_t n_rows, int H, int Hkv, int hd) {
  extern __shared__ __align__(16) bf16 smem[];
  bf16 *Ks = smem, *Vs = smem + 2 * TILE<HD>;
  PkTile t;
  int h, half;
  if (!pk_item64(tl, H, t, h, half)) return;
  const int q0 = t.blk * PK_BLOCK + half * TB;
  if (q0 >= t.len) return;
  const int w = threadIdx.x / 32, lane = threadIdx.x & 31, g = h / (H / Hkv);
  const int nq = min(TB, t.len - q0);
  const float sl2 = LOG2E / sqrtf((float)hd);
  const bf16 *base = qkv + (int64_t)t.row0 * ld;
  const bf16 *kcol = base + (int64_t)(H + g) * hd, *vcol = base + (int64_t)(H + Hkv + g) * hd;
  load<HD>(Ks + TILE<HD>, base + q0 * ld + (int64_t)h * hd, ld, nq, hd);
  load<HD>(Ks, kcol, ld, min(TB, t.len), hd);
  commit();
  load<HD>(Vs, vcol, ld, min(TB, t.len), hd);
  commit();
  wait<1>();
  __syncthreads();
  const int row = 16 * w + (lane >> 2);  // this thread's rows: this and 8 further
  uint32_t qf[HD / 16][4];
#pragma unroll
  for (int k = 0; k < HD / 16; k++) afrag<HD>(Ks + TILE<HD>, w, k, qf[k]);
  float acc[HD / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < HD / 8; i++) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  const bool rows = 16 * w < nq;  // the warp has rows of the sequence
  for (int k0 = 0, cur = 0; k0 <= q0; k0 += TB, cur ^= 1) {
    const bf16 *K = Ks + cur * TILE<HD>, *V = Vs + cur * TILE<HD>;
    const bool diag = k0 == q0, both = !diag || w >= 2;  // keys 32 and on before the last row
    float s[2][4][4] = {};
    if (rows) {
#pragma unroll
      for (int hf = 0; hf < 2; hf++)
        if (!hf || both)
#pragma unroll
          for (int k = 0; k < HD / 16; k++) abt_step<HD>(s[hf], qf[k], K, 32 * hf, k);
      float mn[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int hf = 0; hf < 2; hf++)
#pragma unroll
        for (int nt = 0; nt < 4; nt++)
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const int key = 32 * hf + 8 * nt + (lane & 3) * 2 + (e & 1);
            float &x = s[hf][nt][e];
            if (diag && key > row + (e & 2) * 4) x = -INFINITY;
            mn[e >> 1] = fmaxf(mn[e >> 1], x);
          }
#pragma unroll
      for (int r = 0; r < 2; r++) {
        mn[r] = fmaxf(mn[r], __shfl_xor_sync(0xffffffffu, mn[r], 1));
        mn[r] = fmaxf(mn[r], __shfl_xor_sync(0xffffffffu, mn[r], 2));
        const float top = fmaxf(m[r], mn[r] * sl2);
        const float ref = top == -INFINITY ? 0.f : top, corr = tc::ex2(m[r] - ref);
        m[r] = top;
        float2 lr = make_float2(l[r] * corr, 0.f);
#pragma unroll
        for (int i = 0; i < HD / 8; i++) {
          acc[i][2 * r] *= corr;
          acc[i][2 * r + 1] *= corr;
        }
#pragma unroll
        for (int hf = 0; hf < 2; hf++)
#pragma unroll
          for (int nt = 0; nt < 4; nt++) {
            float *x = s[hf][nt] + 2 * r;
            const float2 y = __ffma2_rn(make_float2(x[0], x[1]), make_float2(sl2, sl2),
                                        make_float2(-ref, -ref));
            x[0] = tc::ex2(y.x);
            x[1] = tc::ex2(y.y);
            lr = __fadd2_rn(lr, make_float2(x[0], x[1]));
          }
        l[r] = lr.x + lr.y;
      }
    }
    wait<0>();
    __syncthreads();  // this tile's V is there; the other K (and Q in it) has been read
    if (k0 + TB <= q0) {
      load<HD>(Ks + (cur ^ 1) * TILE<HD>, kcol + (k0 + TB) * ld, ld, min(TB, t.len - k0 - TB), hd);
      commit();
      load<HD>(Vs + (cur ^ 1) * TILE<HD>, vcol + (k0 + TB) * ld, ld, min(TB, t.len - k0 - TB), hd);
      commit();
    }
    if (rows) {
#pragma unroll
      for (int hf = 0; hf < 2; hf++)
        if (!hf || both) ab<HD>(acc, s[hf], V, 32 * hf);
    }
    if (k0 + TB <= q0) {
      wait<1>();
      __syncthreads();  // the next K is there
    }
  }
  if (!rows) return;
#pragma unroll
  for (int r = 0; r < 2; r++) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    const int q = row + 8 * r;
    if (q >= nq) continue;
    if ((lane & 3) == 0) lse[(int64_t)h * n_rows + t.row0 + q0 + q] = (m[r] + log2f(l[r])) * LN2;
    store_row<HD>(o + ((int64_t)t.row0 + q0 + q) * H * hd + (int64_t)h * hd, acc, r, 1.f / l[r], hd);
  }
}

// dQ of 64 queries, and D for the dK/dV kernel.  Shared memory: K and V twice;
// Q and dO pass through the second ones.
template <int HD>
__global__ void __launch_bounds__(NT, per_sm(HD))
    k_dq(const bf16 *__restrict__ qkv, int64_t ld, const PkTiles tl, const bf16 *__restrict__ o,
         const float *__restrict__ lse, const bf16 *__restrict__ dout, float *__restrict__ D,
         bf16 *__restrict__ dqkv, int64_t dld, int64_t n_rows, int H, int Hkv, int hd) {
  extern __shared__ __align__(16) bf16 smem[];
  bf16 *Ks = smem, *Vs = smem + 2 * TILE<HD>;  // [2] each; Q and dO pass through the second ones
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
  load<HD>(Ks + TILE<HD>, base + q0 * ld + (int64_t)h * hd, ld, nq, hd);
  load<HD>(Vs + TILE<HD>, dout + orow0, ow, nq, hd);
  commit();
  load<HD>(Ks, kcol, ld, min(TB, t.len), hd);
  load<HD>(Vs, vcol, ld, min(TB, t.len), hd);
  commit();
  const int row = 16 * w + (lane >> 2);  // this thread's rows: this and 8 further
  float L2[2], Dr[2] = {0.f, 0.f};
#pragma unroll
  for (int r = 0; r < 2; r++)  // rows past the sequence: P = 0
    L2[r] = row + 8 * r < nq ? lse[(int64_t)h * n_rows + t.row0 + q0 + row + 8 * r] * LOG2E
                             : INFINITY;
  wait<1>();
  __syncthreads();
  uint32_t qf[HD / 16][4], df[HD / 16][4];
#pragma unroll
  for (int k = 0; k < HD / 16; k++) {
    afrag<HD>(Ks + TILE<HD>, w, k, qf[k]);
    afrag<HD>(Vs + TILE<HD>, w, k, df[k]);
  }
  float acc[HD / 8][4];
#pragma unroll
  for (int i = 0; i < HD / 8; i++) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  // weights (0 past the row, where diag) and dP of the warp's rows and keys
  // [32 hf, 32 hf + 32) of a tile
  auto products = [&](float (&s)[4][4], float (&dp)[4][4], const bf16 *K, const bf16 *V, int hf,
                      bool diag) {
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int e = 0; e < 4; e++) s[i][e] = dp[i][e] = 0.f;
#pragma unroll
    for (int k = 0; k < HD / 16; k++) {
      abt_step<HD>(s, qf[k], K, 32 * hf, k);
      abt_step<HD>(dp, df[k], V, 32 * hf, k);
    }
#pragma unroll
    for (int nt = 0; nt < 4; nt++)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const float2 y =
            __ffma2_rn(make_float2(s[nt][e], s[nt][e + 1]), make_float2(sl2, sl2),
                       make_float2(-L2[e >> 1], -L2[e >> 1]));
        s[nt][e] = tc::ex2(y.x);
        s[nt][e + 1] = tc::ex2(y.y);
        if (diag) {
          const int after = 32 * hf + 8 * nt + (lane & 3) * 2 - row - e * 4;  // keys past the row
          if (after > 0) s[nt][e] = dp[nt][e] = 0.f;
          if (after > -1) s[nt][e + 1] = dp[nt][e + 1] = 0.f;
        }
      }
  };
  auto add_dq = [&](float (&s)[4][4], const float (&dp)[4][4], const bf16 *K, int hf) {
#pragma unroll
    for (int nt = 0; nt < 4; nt++)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const float2 y = __fmul2_rn(make_float2(s[nt][e], s[nt][e + 1]),
                                    __fadd2_rn(make_float2(dp[nt][e], dp[nt][e + 1]),
                                               make_float2(-Dr[e >> 1], -Dr[e >> 1])));
        s[nt][e] = y.x;
        s[nt][e + 1] = y.y;
      }
    ab<HD>(acc, s, K, 32 * hf);
  };
  auto quad = [&](float &x) {  // the row's sum over the 4 threads that hold it
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
  };
  const bool rows = 16 * w < nq;  // the warp has rows of the sequence
  if (q0 == 0) {
    // a sequence's first 64 rows: D = sum_j P_ij dP_ij / sum_j P_ij of their one
    // tile (the quotient, so that P's own errors cancel where dP is the same for
    // all).  dO . O takes O as it was rounded to bf16, and where O has few terms
    // that error is as large as dS's own.
    constexpr bool KEEP = HD <= 64;  // registers hold the tile's P and dP
    constexpr int N = KEEP ? 2 : 1;
    float s[N][4][4], dp[N][4][4], l[2] = {0.f, 0.f};
    wait<0>();
    __syncthreads();
    if (!rows) return;
#pragma unroll
    for (int hf = 0; hf < 2; hf++) {
      if (hf && w < 2) continue;  // behind the warp's last row
      products(s[hf % N], dp[hf % N], Ks, Vs, hf, true);
#pragma unroll
      for (int nt = 0; nt < 4; nt++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
          Dr[e >> 1] += s[hf % N][nt][e] * dp[hf % N][nt][e];
          l[e >> 1] += s[hf % N][nt][e];
        }
    }
#pragma unroll
    for (int r = 0; r < 2; r++) {
      quad(l[r]);
      quad(Dr[r]);
      Dr[r] = row + 8 * r < nq ? Dr[r] / l[r] : 0.f;
    }
#pragma unroll
    for (int hf = 0; hf < 2; hf++) {
      if (hf && w < 2) continue;
      if (!KEEP) products(s[0], dp[0], Ks, Vs, hf, true);
      add_dq(s[hf % N], dp[hf % N], Ks, hf);
    }
  } else {
#pragma unroll
    for (int r = 0; r < 2; r++) {  // D = dO . O from dO's fragments and O read the same way
      if (row + 8 * r < nq) {
        const bf16 *orow = o + orow0 + (row + 8 * r) * ow;
#pragma unroll
        for (int k = 0; k < HD / 16; k++)
#pragma unroll
          for (int e = 0; e < 2; e++) {
            const int c = 16 * k + 8 * e + (lane & 3) * 2;
            if (c < hd) {
              const float2 a =
                  __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(orow + c));
              const float2 b =
                  __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&df[k][2 * e + r]));
              Dr[r] += a.x * b.x + a.y * b.y;
            }
          }
      }
      quad(Dr[r]);
    }
    for (int k0 = 0, cur = 0; k0 <= q0; k0 += TB, cur ^= 1) {
      __syncthreads();  // the other buffers (and Q, dO in them) have been read
      if (k0 + TB <= q0) {
        const int n = min(TB, t.len - k0 - TB);
        load<HD>(Ks + (cur ^ 1) * TILE<HD>, kcol + (k0 + TB) * ld, ld, n, hd);
        load<HD>(Vs + (cur ^ 1) * TILE<HD>, vcol + (k0 + TB) * ld, ld, n, hd);
      }
      commit();
      wait<1>();
      __syncthreads();
      if (!rows) continue;
#pragma unroll
      for (int hf = 0; hf < 2; hf++) {
        if (hf && w < 2 && k0 == q0) continue;  // behind the warp's last row
        float s[4][4], dp[4][4];
        products(s, dp, Ks + cur * TILE<HD>, Vs + cur * TILE<HD>, hf, k0 == q0);
        add_dq(s, dp, Ks + cur * TILE<HD>, hf);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < 2; r++) {
    const int q = row + 8 * r;
    if (q >= nq) continue;
    if ((lane & 3) == 0) D[(int64_t)h * n_rows + t.row0 + q0 + q] = Dr[r];
    store_row<HD>(dqkv + ((int64_t)t.row0 + q0 + q) * dld + (int64_t)h * hd, acc, r, scale, hd);
  }
}

// dK, dV of 64 keys: the kv head's query heads in order, and for each the
// query tiles from the keys' own on.  Shared memory: K, V, then Q and dO twice,
// and their L and D.
template <int HD>
__global__ void __launch_bounds__(NT, per_sm(HD))
    k_dkv(const bf16 *__restrict__ qkv, int64_t ld, const PkTiles tl,
          const float *__restrict__ lse, const bf16 *__restrict__ dout,
          const float *__restrict__ D, bf16 *__restrict__ dqkv, int64_t dld, int64_t n_rows, int H,
          int Hkv, int hd) {
  extern __shared__ __align__(16) bf16 smem[];
  bf16 *Ks = smem, *Vs = Ks + TILE<HD>, *Qs = Vs + TILE<HD>, *Gs = Qs + 2 * TILE<HD>;
  float *Ls = reinterpret_cast<float *>(Gs + 2 * TILE<HD>), *Ds = Ls + 2 * TB;
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
  load<HD>(Ks, base + k0 * ld + (int64_t)(H + g) * hd, ld, nk, hd);
  load<HD>(Vs, base + k0 * ld + (int64_t)(H + Hkv + g) * hd, ld, nk, hd);
  auto issue = [&](int st, int buf) {
    const int h = g * grp + st / nqt, q0 = k0 + (st % nqt) * TB, nq = min(TB, t.len - q0);
    load<HD>(Qs + buf * TILE<HD>, base + q0 * ld + (int64_t)h * hd, ld, nq, hd);
    load<HD>(Gs + buf * TILE<HD>, dout + ((int64_t)t.row0 + q0) * ow + (int64_t)h * hd, ow, nq, hd);
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
  constexpr bool KEEP = HD <= 64;  // registers hold K's and V's fragments
  uint32_t kf[KEEP ? HD / 16 : 1][4], vf[KEEP ? HD / 16 : 1][4];
  const bool rows = 16 * w < nk;  // the warp has keys of the sequence
  for (int st = 0; st < steps; st++) {
    const int cur = st & 1;
    __syncthreads();  // the other buffers have been read
    if (st + 1 < steps) issue(st + 1, cur ^ 1);
    commit();
    wait<1>();
    __syncthreads();
    const bf16 *Q = Qs + cur * TILE<HD>, *G = Gs + cur * TILE<HD>;
    const bool diag = st % nqt == 0;
    if (!rows) continue;
    if (KEEP && st == 0) {
#pragma unroll
      for (int k = 0; k < HD / 16; k++) {
        afrag<HD>(Ks, w, k, kf[KEEP ? k : 0]);
        afrag<HD>(Vs, w, k, vf[KEEP ? k : 0]);
      }
    }
#pragma unroll
    for (int hf = 0; hf < 2; hf++) {
      if (diag && !hf && w >= 2) continue;  // before the warp's first key
      float s[4][4] = {}, dp[4][4] = {};  // S^T, dP^T: rows keys, columns 32 queries
#pragma unroll
      for (int k = 0; k < HD / 16; k++) {
        if (!KEEP) afrag<HD>(Ks, w, k, kf[0]);
        abt_step<HD>(s, kf[KEEP ? k : 0], Q, 32 * hf, k);
        if (!KEEP) afrag<HD>(Vs, w, k, vf[0]);
        abt_step<HD>(dp, vf[KEEP ? k : 0], G, 32 * hf, k);
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
      ab<HD>(dv, s, G, 32 * hf);
      ab<HD>(dk, dp, Q, 32 * hf);
    }
  }
#pragma unroll
  for (int r = 0; r < 2; r++) {
    const int key = 16 * w + (lane >> 2) + 8 * r;
    if (key >= nk) continue;
    bf16 *dst = dqkv + ((int64_t)t.row0 + k0 + key) * dld + (int64_t)(H + g) * hd;
    store_row<HD>(dst, dk, r, scale, hd);
    store_row<HD>(dst + (int64_t)Hkv * hd, dv, r, 1.f, hd);
  }
}

template <int HD> constexpr int DQ_SMEM = 4 * TILE<HD> * 2;
template <int HD> constexpr int DKV_SMEM = 6 * TILE<HD> * 2 + 4 * TB * 4;

template <int HD>
static bool launch_fwd(const PkArgs &a, const PkPlan &p, void *o, float *lse) {
  if (!smem_optin((const void *)k_fwd<HD>, DQ_SMEM<HD>)) return false;
  if (pk_planned(a, p)) packed_plan(a, p);
  launch_dependent(k_fwd<HD>, dim3((unsigned)(2 * p.cap * a.H)), dim3(NT), DQ_SMEM<HD>, a.s,
                   (const bf16 *)a.qkv, a.ld, pk_tiles(a, p), (bf16 *)o, lse, a.n_rows, a.H, a.Hkv,
                   a.hd);
  count_launch();
  return true;
}
template <int HD>
static bool launch(const PkArgs &a, const PkPlan &p, const void *o, const float *lse,
                   const void *dout, void *dqkv, int64_t dld) {
  if (!smem_optin((const void *)k_dq<HD>, DQ_SMEM<HD>) ||
      !smem_optin((const void *)k_dkv<HD>, DKV_SMEM<HD>))
    return false;
  if (pk_planned(a, p)) packed_plan(a, p);
  launch_dependent(k_dq<HD>, dim3((unsigned)(2 * p.cap * a.H)), dim3(NT), DQ_SMEM<HD>, a.s,
                   (const bf16 *)a.qkv, a.ld, pk_tiles(a, p), (const bf16 *)o, lse,
                   (const bf16 *)dout, p.D, (bf16 *)dqkv, dld, a.n_rows, a.H, a.Hkv, a.hd);
  launch_dependent(k_dkv<HD>, dim3((unsigned)(2 * p.cap * a.Hkv)), dim3(NT), DKV_SMEM<HD>, a.s,
                   (const bf16 *)a.qkv, a.ld, pk_tiles(a, p), lse, (const bf16 *)dout, p.D,
                   (bf16 *)dqkv, dld, a.n_rows, a.H, a.Hkv, a.hd);
  count_launch(2);
  return true;
}

}  // namespace pk_mma

bool packed_fwd_mma(const PkArgs &a, const PkPlan &p, void *o, float *lse) {
  using namespace pk_mma;
  const int64_t mean = a.n_rows / a.n_seq;
  if (mean > (a.hd <= 32 ? 256 : pk_planned(a, p) ? 64 : 128)) return false;
  if (a.dt != DT_BF16 || a.hd % 8 || a.ld % 8 || ((uintptr_t)a.qkv & 15) || ((uintptr_t)o & 3))
    return false;
  return a.hd <= 32   ? launch_fwd<32>(a, p, o, lse)
         : a.hd <= 64 ? launch_fwd<64>(a, p, o, lse)
                      : launch_fwd<128>(a, p, o, lse);
}

bool packed_bwd_mma(const PkArgs &a, const PkPlan &p, const void *o, const float *lse,
                    const void *dout, void *dqkv, int64_t dld, bool shorts) {
  using namespace pk_mma;
  if (shorts) {
    const int64_t mean = a.n_rows / a.n_seq, blocks = 2 * p.cap * a.Hkv;
    const bool narrow = a.hd <= 32;
    if (mean > (blocks > (narrow ? 2 : 8) * device_sms() ? (narrow ? 320 : 192) : narrow ? 128 : 64))
      return false;
  }
  if (a.dt != DT_BF16 || a.hd % 8 || a.ld % 8 || dld % 2 ||
      (((uintptr_t)a.qkv | (uintptr_t)dout) & 15) || (((uintptr_t)o | (uintptr_t)dqkv) & 3))
    return false;
  return a.hd <= 32   ? launch<32>(a, p, o, lse, dout, dqkv, dld)
         : a.hd <= 64 ? launch<64>(a, p, o, lse, dout, dqkv, dld)
                      : launch<128>(a, p, o, lse, dout, dqkv, dld);
}

}  // namespace llm
