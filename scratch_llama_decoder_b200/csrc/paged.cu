// The paged key/value cache: rows written (rounded or quantised) and read
// back, and the attention of one new token per sequence over its cached
// positions, split over their number and joined.
#include <cuda_fp8.h>
#include <limits.h>

#include "paged.cuh"

namespace llm {
namespace pg {

static inline unsigned cdiv(int64_t a, int64_t b) { return (unsigned)((a + b - 1) / b); }

// ------------------------------------------------------------ element types
// 8 consecutive elements; elements at or past n read as 0.
LLM_DEV void read8(const __nv_bfloat16 *p, bool vec, int n, float (&x)[8]) {
  if (vec) {
    const uint4 w = *reinterpret_cast<const uint4 *>(p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) x[i] = i < n ? to_f(p[i]) : 0.f;
  }
}
LLM_DEV void read8(const float *p, bool vec, int n, float (&x)[8]) {
  if (vec) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0];
    const float4 b = reinterpret_cast<const float4 *>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) x[i] = i < n ? p[i] : 0.f;
  }
}
LLM_DEV void write8(__nv_bfloat16 *p, bool vec, int n, const float (&x)[8]) {
  if (vec) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++)
      if (i < n) p[i] = __float2bfloat16_rn(x[i]);
  }
}
LLM_DEV void write8(float *p, bool vec, int n, const float (&x)[8]) {
  if (vec) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++)
      if (i < n) p[i] = x[i];
  }
}
LLM_DEV void write8(uint8_t *p, bool vec, int n, const uint32_t (&c)[2]) {
  if (vec) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(c[0], c[1]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++)
      if (i < n) p[i] = (uint8_t)(c[i >> 2] >> (8 * (i & 3)));
  }
}
LLM_DEV void read8(const uint8_t *p, bool vec, int n, uint32_t (&c)[2]) {
  if (vec) {
    const uint2 w = *reinterpret_cast<const uint2 *>(p);
    c[0] = w.x;
    c[1] = w.y;
  } else {
    c[0] = c[1] = 0;
#pragma unroll
    for (int i = 0; i < 8; i++)
      if (i < n) c[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
  }
}
// Two e4m3 codes (low 16 bits) as float32.
LLM_DEV float2 e4m3x2(uint32_t c) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c & 0xffff), __NV_E4M3);
  return __half22float2(__half2(h));
}
// 8 values of the codes, without their scale.
template <int FMT>
LLM_DEV void decode8(const uint32_t (&c)[2], float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const uint32_t w = c[i >> 2] >> (8 * (i & 3));
    if constexpr (FMT == KV_E4M3) {
      const float2 v = e4m3x2(w);
      x[i] = v.x;
      x[i + 1] = v.y;
    } else {
      x[i] = (float)(int8_t)(w & 0xff);
      x[i + 1] = (float)(int8_t)(w >> 8 & 0xff);
    }
  }
}
// 8 elements of a cached row as float32, without a scale.
template <int FMT>
LLM_DEV void kv_read8(const uint8_t *pages, int64_t elem, bool vec, int n, float (&x)[8]) {
  if constexpr (FMT == KV_F32) {
    read8(reinterpret_cast<const float *>(pages) + elem, vec, n, x);
  } else if constexpr (FMT == KV_BF16) {
    read8(reinterpret_cast<const __nv_bfloat16 *>(pages) + elem, vec, n, x);
  } else {
    uint32_t c[2];
    read8(pages + elem, vec, n, c);
    decode8<FMT>(c, x);
  }
}

// The scale of a row whose largest magnitude is amax.
//   e4m3: the least power of two s with amax <= 448 s (s >= 2^-126), so that
//     x / s and code * s are exact and the code is x / s rounded once;
//   int8: amax / 127 rounded to float32 (at least the least normal number).
// A row that holds an infinity or a NaN has a NaN scale: it reads back as
// NaN instead of as finite values.
template <int FMT>
LLM_DEV float row_scale(float amax) {
  if (!(amax < INFINITY)) return __uint_as_float(0x7fc00000u);
  if constexpr (FMT == KV_E4M3) {
    // amax / 448 <= 2^e: the exponent of the quotient, one more unless it is
    // a power of two itself.  The quotient is rounded up, so that amax <= 448 s
    // holds for the amax next above a power of two times 448, too.
    const uint32_t u = __float_as_uint(__fdiv_ru(amax, 448.f));
    const int e = (int)(u >> 23) - 127 + ((u & 0x7fffffu) ? 1 : 0);
    return __uint_as_float((uint32_t)(max(e, -126) + 127) << 23);
  } else {
    return fmaxf(__fdiv_rn(amax, 127.f), 1.17549435e-38f);
  }
}
// x / scale to the nearest code, ties to even.
template <int FMT>
LLM_DEV uint32_t encode4(const float *x, float scale, float inv) {
  if constexpr (FMT == KV_E4M3) {  // inv = 1 / scale, exact
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0] * inv, x[1] * inv),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2] * inv, x[3] * inv),
                                                 __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
  } else {
    // q = x / scale in float32 may land on the wrong side of a border between
    // two codes; the remainder r = x - q scale (one rounding, exact where it
    // decides) puts the code right: 2 |r| <= scale, and even on the border
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      float q = rintf(x[i] * inv);
      const float r2 = 2.f * fmaf(-q, scale, x[i]);
      if (r2 > scale || (r2 == scale && ((int)q & 1))) q += 1.f;
      else if (r2 < -scale || (r2 == -scale && ((int)q & 1))) q -= 1.f;
      w |= ((uint32_t)(int)fminf(fmaxf(q, -127.f), 127.f) & 0xffu) << (8 * i);
    }
    return w;
  }
}

// The sequence that holds packed row i (cu[s] <= i < cu[s + 1]), -1 for none.
LLM_DEV int seq_of(const int32_t *cu, int n_seq, int64_t i) {
  int lo = 0, hi = n_seq + 1;  // the first entry above i
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] > i) hi = mid;
    else lo = mid + 1;
  }
  return lo >= 1 && lo <= n_seq && cu[lo - 1] <= i ? lo - 1 : -1;
}
// The cache row of packed row i, -1 when it has none.
LLM_DEV int64_t place(const KvView &kv, const int32_t *cu, const int32_t *start, int n_seq,
                      int64_t i, int *seq) {
  const int s = seq_of(cu, n_seq, i);
  *seq = s;
  if (s < 0) return -1;
  const int64_t row = kv_row(kv, s, (start ? (int64_t)start[s] : 0) + i - cu[s]);
  if (row < 0 && kv.flag && (threadIdx.x & 31) == 0) atomicOr(kv.flag, PK_BAD_PAGE);
  return row;
}

// ------------------------------------------------------------------- write
// One warp per packed row: its k and v heads in groups of lanes, 8 elements a
// lane, so that a head's largest magnitude is a few shuffles away.
constexpr int RW_THREADS = 256;
template <typename T, int FMT>
__global__ void __launch_bounds__(RW_THREADS)
    k_write(const KvView kv, const T *__restrict__ qkv, int64_t ld, const int32_t *__restrict__ cu,
            const int32_t *__restrict__ start, int n_seq, int64_t n_rows, int H, int lph,
            bool vec) {
  const int64_t i = blockIdx.x * (int64_t)(RW_THREADS / 32) + threadIdx.x / 32;
  if (i >= n_rows) return;
  int s;
  const int64_t row = place(kv, cu, start, n_seq, i, &s);
  if (row < 0) return;
  const int lane = threadIdx.x & 31, sub = lane % lph, e = sub * 8;
  const T *src = qkv + i * ld + (int64_t)H * kv.hd;  // k heads, then v heads
  for (int h0 = 0; h0 < 2 * kv.Hkv; h0 += 32 / lph) {
    const int h = h0 + lane / lph;  // k or v and head: the pages' own order
    const bool on = h < 2 * kv.Hkv && e < kv.hd;
    float x[8];
    if (on) {
      read8(src + (int64_t)h * kv.hd + e, vec, kv.hd - e, x);
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++) x[j] = 0.f;
    }
    const int64_t dst = row + (int64_t)h * kv.ps;
    if constexpr (FMT == KV_F32) {
      if (on) write8(reinterpret_cast<float *>(kv.pages) + dst * kv.hd + e, vec, kv.hd - e, x);
    } else if constexpr (FMT == KV_BF16) {
      if (on)
        write8(reinterpret_cast<__nv_bfloat16 *>(kv.pages) + dst * kv.hd + e, vec, kv.hd - e, x);
    } else {
      // the largest magnitude by its bits: a NaN is above an infinity
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 8; j++) top = max(top, __float_as_uint(x[j]) & 0x7fffffffu);
      for (int o = 1; o < lph; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float scale = row_scale<FMT>(__uint_as_float(top));
      const bool bad = !(__uint_as_float(top) < INFINITY);
      const float inv = 1.f / scale;
      const uint32_t c[2] = {bad ? 0u : encode4<FMT>(x, scale, inv),
                             bad ? 0u : encode4<FMT>(x + 4, scale, inv)};
      if (on) {
        write8(kv.pages + dst * kv.hd + e, vec, kv.hd - e, c);
        if (sub == 0) kv.scales[dst] = scale;
      }
    }
  }
}

// -------------------------------------------------------------------- read
// One warp per packed row, as above; a row whose place does not exist reads
// as zeros, rows of no sequence are left alone.
template <typename T, int FMT>
__global__ void __launch_bounds__(RW_THREADS)
    k_read(const KvView kv, const int32_t *__restrict__ cu, const int32_t *__restrict__ start,
           int n_seq, int64_t n_rows, T *__restrict__ k, T *__restrict__ v, int lph, bool vec) {
  const int64_t i = blockIdx.x * (int64_t)(RW_THREADS / 32) + threadIdx.x / 32;
  if (i >= n_rows) return;
  int s;
  const int64_t row = place(kv, cu, start, n_seq, i, &s);
  if (s < 0) return;
  const int lane = threadIdx.x & 31, e = (lane % lph) * 8;
  const int64_t w = (int64_t)kv.Hkv * kv.hd;
  for (int h0 = 0; h0 < 2 * kv.Hkv; h0 += 32 / lph) {
    const int h = h0 + lane / lph;
    if (h >= 2 * kv.Hkv || e >= kv.hd) continue;
    float x[8] = {};
    if (row >= 0) {
      const int64_t src = row + (int64_t)h * kv.ps;
      kv_read8<FMT>(kv.pages, src * kv.hd + e, vec, kv.hd - e, x);
      if constexpr (FMT >= KV_E4M3) {
        const float sc = kv.scales[src];
#pragma unroll
        for (int j = 0; j < 8; j++) x[j] *= sc;
      }
    }
    T *dst = h < kv.Hkv ? k + i * w + (int64_t)h * kv.hd
                        : v + i * w + (int64_t)(h - kv.Hkv) * kv.hd;
    write8(dst + e, vec, kv.hd - e, x);
  }
}

// --------------------------------------------------------------- attention
// The work of a call is the (sequence, kv head) pairs in order, each
// ceil(len / 64) units of 64 positions: W units in a row, of which block i of
// N (at most W, so that none is empty) takes [W i / N, W (i + 1) / N) whatever
// the lengths are.  A pair that lies
// in one block is finished there; a pair cut between blocks leaves, per block,
// the running maximum, sum and weighted values of its part in the workspace,
// and a second kernel joins the parts in order.  A block's range cuts at most
// its first and its last pair: two slots per block.
constexpr int AT = 128;       // threads
constexpr int BLOCKS_SM = 4;  // blocks per SM that the split counts on
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

struct Sched {
  int n_seq, Hkv, N, direct;  // direct: block i is pair i, nothing is cut
};
LLM_DEV int clamped_len(const KvView &kv, const int32_t *lens, int s) {
  const int64_t cap = (int64_t)kv.table_pages * kv.ps;
  const int n = lens[s];
  const bool bad = n < 0 || n > cap;
  if (bad && kv.flag) atomicOr(kv.flag, PK_BAD_PAGE);
  return bad ? (n < 0 ? 0 : (int)cap) : n;
}
// pre[s] = units of the sequences before s, per kv head (n_seq + 1 entries).
LLM_DEV void unit_prefix(const KvView &kv, const int32_t *lens, int n_seq, int *pre) {
  __shared__ int tot[AT / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int carry = 0;
  for (int s0 = 0; s0 < n_seq; s0 += AT) {
    const int s = s0 + threadIdx.x;
    int v = s < n_seq ? (clamped_len(kv, lens, s) + PG_UNIT - 1) / PG_UNIT : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += t;
    }
    if (lane == 31) tot[warp] = v;
    __syncthreads();
    int before = carry;
    for (int w = 0; w < warp; w++) before += tot[w];
    if (s < n_seq) pre[s + 1] = before + v;
    for (int w = 0; w < AT / 32; w++) carry += tot[w];
    __syncthreads();
  }
  if (threadIdx.x == 0) pre[0] = 0;
  __syncthreads();
}
LLM_DEV int64_t block_begin(int64_t W, int i, int N) { return W * i / N; }
LLM_DEV int block_of(int64_t W, int64_t w, int N) { return (int)(((w + 1) * N - 1) / W); }
// The sequence whose units hold w (per-head units times Hkv).
LLM_DEV int seq_at(const int *pre, int n_seq, int64_t w, int Hkv) {
  int lo = 0, hi = n_seq;  // the first s with pre[s + 1] Hkv > w
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if ((int64_t)pre[mid + 1] * Hkv > w) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// 4 warps; a warp takes 4 positions at a time, 8 lanes each, a lane HD / 8 of
// the head's columns, and GT query heads of the kv head at once.
template <typename T, int FMT, int HD, int GT>
__global__ void __launch_bounds__(AT)
    k_attend(const KvView kv, const T *__restrict__ q, int64_t q_ld,
             const int32_t *__restrict__ lens, const Sched sc, int H, T *__restrict__ o,
             float *__restrict__ lse, int *__restrict__ pre_out, float *__restrict__ part,
             bool vec) {
  constexpr int EPL = HD / 8, NC = (EPL + 7) / 8;  // columns a lane, 8-element pieces
  extern __shared__ int pre[];
  __shared__ float sm[AT / 32][GT][HD + 2];
  unit_prefix(kv, lens, sc.n_seq, pre);
  if (!sc.direct && blockIdx.x == 0)
    for (int s = threadIdx.x; s <= sc.n_seq; s += AT) pre_out[s] = pre[s];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane & 7, ks = lane >> 3;
  const int grp = H / kv.Hkv, hd = kv.hd;
  const float sl2 = LOG2E / sqrtf((float)hd);
  const int64_t W = (int64_t)pre[sc.n_seq] * kv.Hkv;
  const int N = (int)min((int64_t)sc.N, W);
  if (!sc.direct && (int)blockIdx.x >= N) return;
  int64_t w = sc.direct ? 0 : block_begin(W, blockIdx.x, N);
  const int64_t end = sc.direct ? 1 : block_begin(W, blockIdx.x + 1, N);
  for (int piece = 0; w < end; piece++) {
    int s, g, u0, nu, units;
    if (sc.direct) {
      s = blockIdx.x / kv.Hkv;
      g = blockIdx.x % kv.Hkv;
      u0 = 0;
      nu = units = pre[s + 1] - pre[s];
      w = end;
    } else {
      s = seq_at(pre, sc.n_seq, w, kv.Hkv);
      units = pre[s + 1] - pre[s];
      const int64_t in = w - (int64_t)pre[s] * kv.Hkv;
      g = (int)(in / units);
      u0 = (int)(in % units);
      nu = (int)min((int64_t)(units - u0), end - w);
      w += nu;
    }
    const int len = min(max(lens[s], 0), (int)min((int64_t)kv.table_pages * kv.ps, (int64_t)INT_MAX));
    const int j0 = u0 * PG_UNIT, j1 = min(len, (u0 + nu) * PG_UNIT);
    for (int r0 = 0; r0 < grp; r0 += GT) {
      float qv[GT][EPL], acc[GT][EPL], m[GT], l[GT];
#pragma unroll
      for (int r = 0; r < GT; r++) {
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int c = 0; c < EPL; c++) {
          const int e = sub * EPL + c;
          qv[r][c] = r0 + r < grp && e < hd
                         ? to_f(q[s * q_ld + (int64_t)(g * grp + r0 + r) * hd + e]) * sl2
                         : 0.f;
          acc[r][c] = 0.f;
        }
      }
      for (int j = j0 + warp * 4; j < j1; j += AT / 32 * 4) {
        const int jj = j + ks;
        const int64_t row = jj < j1 ? kv_row(kv, s, jj) : -1;
        if (jj < j1 && row < 0 && kv.flag && sub == 0) atomicOr(kv.flag, PK_BAD_PAGE);
        const int64_t kr = row + (int64_t)g * kv.ps, vr = kr + (int64_t)kv.Hkv * kv.ps;
        float kx[8 * NC], vx[8 * NC], vs = 1.f, kscale = 1.f;
#pragma unroll
        for (int c = 0; c < NC; c++) {
          float a[8] = {}, b[8] = {};
          const int e = sub * EPL + 8 * c, n = min(hd - e, EPL - 8 * c);
          if (row >= 0 && n > 0) {
            kv_read8<FMT>(kv.pages, kr * hd + e, vec && n >= 8, n, a);
            kv_read8<FMT>(kv.pages, vr * hd + e, vec && n >= 8, n, b);
          }
#pragma unroll
          for (int i = 0; i < 8; i++) {
            kx[8 * c + i] = a[i];
            vx[8 * c + i] = b[i];
          }
        }
        if constexpr (FMT >= KV_E4M3) {
          if (row >= 0) {
            kscale = kv.scales[kr];
            vs = kv.scales[vr];
          }
        }
#pragma unroll
        for (int r = 0; r < GT; r++) {
          float t = 0.f;
#pragma unroll
          for (int c = 0; c < EPL; c++) t = fmaf(qv[r][c], kx[c], t);
#pragma unroll
          for (int x = 1; x < 8; x <<= 1) t += __shfl_xor_sync(0xffffffffu, t, x);
          t *= kscale;
          if (row < 0) t = -INFINITY;  // no such position: weight 0, v read as 0
          const float mn = fmaxf(m[r], t);
          const float ref = mn == -INFINITY ? 0.f : mn;
          const float corr = exp2f(m[r] - ref), p = exp2f(t - ref);
          l[r] = l[r] * corr + p;
          m[r] = mn;
          const float pv = p * vs;
#pragma unroll
          for (int c = 0; c < EPL; c++) acc[r][c] = fmaf(pv, vx[c], acc[r][c] * corr);
        }
      }
      // the warp's 4 position groups meet, then the 4 warps
#pragma unroll
      for (int x = 8; x < 32; x <<= 1)
#pragma unroll
        for (int r = 0; r < GT; r++) {
          const float mo = __shfl_xor_sync(0xffffffffu, m[r], x);
          const float mn = fmaxf(m[r], mo), ref = mn == -INFINITY ? 0.f : mn;
          const float a = exp2f(m[r] - ref), b = exp2f(mo - ref);
          l[r] = l[r] * a + __shfl_xor_sync(0xffffffffu, l[r], x) * b;
          m[r] = mn;
#pragma unroll
          for (int c = 0; c < EPL; c++)
            acc[r][c] = acc[r][c] * a + __shfl_xor_sync(0xffffffffu, acc[r][c], x) * b;
        }
      if (ks == 0) {
#pragma unroll
        for (int r = 0; r < GT; r++) {
#pragma unroll
          for (int c = 0; c < EPL; c++) sm[warp][r][sub * EPL + c] = acc[r][c];
          if (sub == 0) {
            sm[warp][r][HD] = m[r];
            sm[warp][r][HD + 1] = l[r];
          }
        }
      }
      __syncthreads();
      const bool whole = nu == units;
      float *rec = part + (int64_t)(2 * blockIdx.x + (piece > 0)) * grp * (hd + 2);
      for (int i = threadIdx.x; i < GT * HD; i += AT) {
        const int r = i / HD, e = i % HD;
        if (r0 + r >= grp || e >= hd) continue;
        float M = -INFINITY;
#pragma unroll
        for (int x = 0; x < AT / 32; x++) M = fmaxf(M, sm[x][r][HD]);
        const float ref = M == -INFINITY ? 0.f : M;
        float L = 0.f, v = 0.f;
#pragma unroll
        for (int x = 0; x < AT / 32; x++) {
          const float f = exp2f(sm[x][r][HD] - ref);
          L = fmaf(f, sm[x][r][HD + 1], L);
          v = fmaf(f, sm[x][r][e], v);
        }
        const int hq = g * grp + r0 + r;
        if (whole) {
          o[((int64_t)s * H + hq) * hd + e] = from_f<T>(L == 0.f ? 0.f : v / L);
          if (e == 0 && lse) lse[(int64_t)s * H + hq] = (M + log2f(L)) * LN2;
        } else {
          rec[(r0 + r) * (hd + 2) + 2 + e] = v;
          if (e == 0) {
            rec[(r0 + r) * (hd + 2)] = M;
            rec[(r0 + r) * (hd + 2) + 1] = L;
          }
        }
      }
      __syncthreads();
    }
  }
}

// Joins the parts of every cut pair, in order; a sequence of length 0 gets
// o = 0 and L = -inf.
template <typename T>
__global__ void __launch_bounds__(AT)
    k_join(const int *__restrict__ pre, const float *__restrict__ part, const Sched sc, int H,
           int hd, T *__restrict__ o, float *__restrict__ lse) {
  const int s = blockIdx.x / sc.Hkv, g = blockIdx.x % sc.Hkv, grp = H / sc.Hkv;
  const int units = pre[s + 1] - pre[s];
  const int64_t W = (int64_t)pre[sc.n_seq] * sc.Hkv;
  const int64_t w0 = (int64_t)pre[s] * sc.Hkv + (int64_t)g * units;
  if (units == 0) {
    for (int i = threadIdx.x; i < grp * hd; i += AT)
      o[((int64_t)s * H + g * grp) * hd + i] = from_f<T>(0.f);
    if (lse)
      for (int i = threadIdx.x; i < grp; i += AT) lse[(int64_t)s * H + g * grp + i] = -INFINITY;
    return;
  }
  const int N = (int)min((int64_t)sc.N, W);
  const int b0 = block_of(W, w0, N), b1 = block_of(W, w0 + units - 1, N);
  if (b0 == b1) return;
  // the pair's part in its first block follows another pair's there, or
  // begins the block's range; in every later block it begins the range
  const int first = block_begin(W, b0, N) < w0 ? 1 : 0;
  const int64_t step = (int64_t)grp * (hd + 2);
  for (int i = threadIdx.x; i < grp * hd; i += AT) {
    const int r = i / hd, e = i % hd;
    float M = -INFINITY, L = 0.f, v = 0.f;
    for (int b = b0; b <= b1; b++) {
      const float *rec = part + (2 * b + (b == b0 ? first : 0)) * step + r * (hd + 2);
      const float mn = fmaxf(M, rec[0]), ref = mn == -INFINITY ? 0.f : mn;
      const float a = exp2f(M - ref), f = exp2f(rec[0] - ref);
      L = L * a + rec[1] * f;
      v = v * a + rec[2 + e] * f;
      M = mn;
    }
    o[((int64_t)s * H + g * grp + r) * hd + e] = from_f<T>(L == 0.f ? 0.f : v / L);
    if (e == 0 && lse) lse[(int64_t)s * H + g * grp + r] = (M + log2f(L)) * LN2;
  }
}

template <typename T, int FMT, int HD>
static bool attend(const PagedArgs &a, const Sched &sc, int *pre, float *part, bool vec) {
  const int grp = a.H / a.kv.Hkv, smem = 4 * (a.n_seq + 1);
  auto go = [&](auto kern) {
    if (!smem_optin((const void *)kern, 4 * (PG_MAX_SEQ + 1))) return false;
    kern<<<sc.N, AT, smem, a.s>>>(a.kv, (const T *)a.q, a.q_ld, a.lens, sc, a.H, (T *)a.o, a.lse,
                                  pre, part, vec);
    count_launch();
    return true;
  };
  if (!(grp == 1 ? go(k_attend<T, FMT, HD, 1>) : go(k_attend<T, FMT, HD, 4>))) return false;
  if (!sc.direct) {
    k_join<T><<<a.n_seq * a.kv.Hkv, AT, 0, a.s>>>(pre, part, sc, a.H, a.kv.hd, (T *)a.o, a.lse);
    count_launch();
  }
  return true;
}
template <typename T, int FMT>
static bool attend_hd(const PagedArgs &a, const Sched &sc, int *pre, float *part, bool vec) {
  return a.kv.hd <= 32   ? attend<T, FMT, 32>(a, sc, pre, part, vec)
         : a.kv.hd <= 64 ? attend<T, FMT, 64>(a, sc, pre, part, vec)
                         : attend<T, FMT, 128>(a, sc, pre, part, vec);
}
template <typename T>
static bool attend_fmt(const PagedArgs &a, const Sched &sc, int *pre, float *part, bool vec) {
  switch (a.kv.fmt) {
    case KV_F32: return attend_hd<T, KV_F32>(a, sc, pre, part, vec);
    case KV_BF16: return attend_hd<T, KV_BF16>(a, sc, pre, part, vec);
    case KV_E4M3: return attend_hd<T, KV_E4M3>(a, sc, pre, part, vec);
    default: return attend_hd<T, KV_INT8>(a, sc, pre, part, vec);
  }
}

// Blocks of a call: the machine's worth of blocks, or one per pair when that
// cannot cut a pair worth the join.
static Sched schedule(const KvView &kv, int n_seq) {
  Sched sc{n_seq, kv.Hkv, 0, 0};
  const int64_t pairs = (int64_t)n_seq * kv.Hkv;
  const int64_t cap = (int64_t)kv.table_pages * kv.ps;
  sc.direct = cap <= 2 * PG_UNIT;
  sc.N = sc.direct ? (int)pairs : device_sms() * BLOCKS_SM;
  return sc;
}
static int64_t pre_bytes(int n_seq) { return (4 * ((int64_t)n_seq + 1) + 255) / 256 * 256; }

}  // namespace pg

void kv_write(const KvView &kv, const void *qkv, int64_t ld, DType dt, const int32_t *cu,
              const int32_t *start, int n_seq, int64_t n_rows, int H, cudaStream_t s) {
  using namespace pg;
  int lph = 1;  // lanes of a head
  while (lph * 8 < kv.hd) lph *= 2;
  const bool vec = kv.hd % 8 == 0 && ld % 8 == 0 && !((uintptr_t)qkv & 15) &&
                   !((uintptr_t)kv.pages & 15);
  const unsigned grid = cdiv(n_rows, RW_THREADS / 32);
#define GO(T, F)                                                                                 \
  k_write<T, F><<<grid, RW_THREADS, 0, s>>>(kv, (const T *)qkv, ld, cu, start, n_seq, n_rows, H, \
                                            lph, vec)
#define FMT(T)                                                                                 \
  switch (kv.fmt) {                                                                            \
    case KV_F32: GO(T, KV_F32); break;                                                         \
    case KV_BF16: GO(T, KV_BF16); break;                                                       \
    case KV_E4M3: GO(T, KV_E4M3); break;                                                       \
    default: GO(T, KV_INT8);                                                                   \
  }
  if (dt == DT_BF16) { FMT(__nv_bfloat16) } else { FMT(float) }
#undef GO
  count_launch();
}

void kv_read(const KvView &kv, const int32_t *cu, const int32_t *start, int n_seq, int64_t n_rows,
             void *k, void *v, DType dt, cudaStream_t s) {
  using namespace pg;
  int lph = 1;
  while (lph * 8 < kv.hd) lph *= 2;
  const bool vec = kv.hd % 8 == 0 && !(((uintptr_t)k | (uintptr_t)v | (uintptr_t)kv.pages) & 15);
  const unsigned grid = cdiv(n_rows, RW_THREADS / 32);
#define GO(T, F)                                                                                \
  k_read<T, F><<<grid, RW_THREADS, 0, s>>>(kv, cu, start, n_seq, n_rows, (T *)k, (T *)v, lph, vec)
  if (dt == DT_BF16) { FMT(__nv_bfloat16) } else { FMT(float) }
#undef GO
#undef FMT
  count_launch();
}

int64_t paged_ws_bytes(const KvView &kv, int n_seq, int H) {
  const pg::Sched sc = pg::schedule(kv, n_seq);
  if (sc.direct) return 256;
  return pg::pre_bytes(n_seq) + 4 * 2 * (int64_t)sc.N * (H / kv.Hkv) * (kv.hd + 2);
}

bool paged_attention(const PagedArgs &a) {
  using namespace pg;
  const Sched sc = schedule(a.kv, a.n_seq);
  int *pre = (int *)a.ws;
  float *part = (float *)((uint8_t *)a.ws + pre_bytes(a.n_seq));
  const bool vec = a.kv.hd % 8 == 0 && !((uintptr_t)a.kv.pages & 15);
  return a.dt == DT_BF16 ? attend_fmt<__nv_bfloat16>(a, sc, pre, part, vec)
                         : attend_fmt<float>(a, sc, pre, part, vec);
}

}  // namespace llm
