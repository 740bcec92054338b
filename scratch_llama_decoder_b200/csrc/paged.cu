// The paged key/value cache: rows written (rounded or quantised) and read
// back, and the attention of one new token per sequence over its cached
// positions, split over their number and joined.
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <limits.h>
#include <type_traits>

#include "paged.cuh"

namespace llm {
namespace pg {

__host__ __device__ static inline unsigned cdiv(int64_t a, int64_t b) {
  return (unsigned)((a + b - 1) / b);
}

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
    if constexpr (FMT == KV_E4M3) {
      const float2 v = e4m3x2(c[i >> 2] >> (8 * (i & 3)));
      x[i] = v.x;
      x[i + 1] = v.y;
    } else {
      // code + 128 as the low mantissa bits of 2^23 (a conversion runs at the SFU's rate)
      const uint32_t u = c[i >> 2] ^ 0x80808080u;
      x[i] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7540 + (i & 3))) - 8388736.f;
      x[i + 1] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7541 + (i & 3))) - 8388736.f;
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

// The scale of a row whose largest magnitude has the bits `top` (a NaN's are
// above an infinity's), and its reciprocal.
//   e4m3: the least power of two s with amax <= 448 s (s >= 2^-126), so that
//     x / s and code * s are exact and the code is x / s rounded once: 448 is
//     1.75 * 2^8, so the exponent is amax's less 8, or 7 past mantissa 1.75;
//   int8: amax / 127 rounded to float32 (at least the least normal number).
// A row that holds an infinity or a NaN has a NaN scale: it reads back as
// NaN instead of as finite values.
template <int FMT>
LLM_DEV float row_scale(uint32_t top, float *inv) {
  const bool bad = top >= 0x7f800000u;
  if constexpr (FMT == KV_E4M3) {
    const int f = max((int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0), 1);
    *inv = __uint_as_float((uint32_t)(254 - f) << 23);
    return bad ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)f << 23);
  } else {
    const float s = fmaxf(__fdiv_rn(__uint_as_float(top), 127.f), 1.17549435e-38f);
    *inv = __fdividef(1.f, s);  // to a few units: encode8 does not rely on it
    return bad ? __uint_as_float(0x7fc00000u) : s;
  }
}
// x / scale to the nearest code, ties to even, for 8 elements.
template <int FMT>
LLM_DEV void encode8(const float (&x)[8], float scale, float inv, uint32_t (&c)[2]) {
  if constexpr (FMT == KV_E4M3) {  // inv is exact
#pragma unroll
    for (int w = 0; w < 2; w++) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(
          make_float2(x[4 * w] * inv, x[4 * w + 1] * inv), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(
          make_float2(x[4 * w + 2] * inv, x[4 * w + 3] * inv), __NV_SATFINITE, __NV_E4M3);
      c[w] = lo | hi << 16;
    }
  } else {
    // q = x inv rounded to an integer by adding 1.5 * 2^23, whose low bits then
    // hold it.  inv is not exact, so q may lie on the wrong side of a border
    // between two codes; the remainder r = x - q scale (one rounding, exact
    // where it decides) tells: |2 r| < scale, or the element is looked at again.
    constexpr float MAGIC = 12582912.f;
    uint32_t t[8];
    bool close = false;
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const float m = fmaf(x[i], inv, MAGIC), q = m - MAGIC;
      t[i] = __float_as_uint(m);
      close |= fabsf(2.f * fmaf(-q, scale, x[i])) >= scale;
    }
    if (close) {  // on a border or past it by the rounding of inv: even, or the next
#pragma unroll
      for (int i = 0; i < 8; i++) {
        float q = (float)(int8_t)(t[i] & 0xff);
        const float r2 = 2.f * fmaf(-q, scale, x[i]);
        if (r2 > scale || (r2 == scale && (t[i] & 1))) q += 1.f;
        else if (r2 < -scale || (r2 == -scale && (t[i] & 1))) q -= 1.f;
        t[i] = (uint32_t)(int)q;
      }
    }
#pragma unroll
    for (int w = 0; w < 2; w++)
      c[w] = __byte_perm(__byte_perm(t[4 * w], t[4 * w + 1], 0x0040),
                         __byte_perm(t[4 * w + 2], t[4 * w + 3], 0x0040), 0x5410);
  }
}

// The sequence that holds packed row i (cu[s] <= i < cu[s + 1]), -1 for none, in
// offsets that do not decrease.  from: the first entry that may be above i (0, or
// that above an earlier row, where it is looked for near that); set to it.
LLM_DEV int seq_of(const int32_t *cu, int n_seq, int64_t i, int &from) {
  int lo = from, hi = n_seq + 1;  // the first entry above i
  if (lo > 0)
    for (int step = 1; lo + step < hi; step *= 2) {
      if (cu[lo + step - 1] > i) hi = lo + step - 1;
      else lo += step;
    }
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] > i) hi = mid;
    else lo = mid + 1;
  }
  from = lo;
  return lo >= 1 && lo <= n_seq && cu[lo - 1] <= i ? lo - 1 : -1;
}
// Whether cu decreases or leaves [0, n_rows] at entry s or every step-th further.
template <int UNROLL>
LLM_DEV bool bad_offsets(const int32_t *cu, int n_seq, int64_t n_rows, int s, int step) {
  bool bad = false;
#pragma unroll UNROLL
  for (; s <= n_seq; s += step) {
    const int a = cu[s], b = s < n_seq ? cu[s + 1] : a;
    bad |= a < 0 || a > b || a > n_rows;
  }
  return bad;
}
// seq_of in offsets of any contents, each clamped to [0, n_rows] and raised to
// the largest before it; *begin: the sequence's.  By a whole warp, a row each.
LLM_DEV int mended_seq_of(const int32_t *cu, int n_seq, int64_t n_rows, int64_t i, int *begin) {
  const int lane = threadIdx.x & 31;
  int s = -1, top = 0;
  for (int s0 = 0; s0 <= n_seq; s0 += 32) {
    int c = s0 + lane <= n_seq ? min(max(cu[s0 + lane], 0), (int)n_rows) : 0;
    c = max(c, top);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, c, o);
      if (lane >= o) c = max(c, t);
    }
#pragma unroll 1
    for (int k = 0; k < min(32, n_seq + 1 - s0); k++) {  // the last offset not above i
      const int t = __shfl_sync(0xffffffffu, c, k);
      if (t <= i) {
        s = s0 + k;
        *begin = t;
      }
    }
    top = __shfl_sync(0xffffffffu, c, 31);
  }
  return s < n_seq ? s : -1;
}
// ------------------------------------------------------------ write and read
// A block takes 32 packed rows.  One warp looks their places up (a chain of
// dependent loads: search, table) while the others have the rows' first loads
// in flight.  Then a warp takes 32 / LPH rows, LPH lanes of 8 elements each,
// and walks through their heads, a few at a time: a row's heads lie together
// where they are packed, and a head's rows, with their scales, in its page.
// Bound by memory, and next to it by instructions: 16001 rows of 16 heads of
// 64, bfloat16 to e4m3 (101 MB): write 23 us (4.3 TB/s), read 26.  (A warp per
// packed row, scattered 64-byte pieces: 39 and 26; rows and heads of a step
// found by division: 57 and 44.)
constexpr int RW_ROWS = 32, RW_THREADS = 256, RW_HEADS = 8;
constexpr int RW_LOOK = RW_THREADS - 32;  // threads that look at the offsets
constexpr int WU = 4, RU = 2;  // heads in flight: write, read (read with 4: 31 us)
constexpr int64_t NO_PLACE = -1, NO_SEQUENCE = -2;  // kv_row's; and a row of none
LLM_DEV int64_t place(const KvView &kv, const int32_t *start, int s, int64_t in) {
  if (s < 0) return NO_SEQUENCE;
  const int64_t row = kv_row(kv, s, (start ? (int64_t)start[s] : 0) + in);
  return row < 0 ? NO_PLACE : row;
}
// The places of 32 rows from i0 on, by warp 0, a row each: by bisection, which
// takes offsets that do not decrease, or in the mended ones.
LLM_DEV void find_places(const KvView &kv, const int32_t *cu, const int32_t *start, int n_seq,
                         int64_t n_rows, int64_t i0, int64_t *rows, int &from) {
  const int64_t i = i0 + threadIdx.x;
  const int s = i < n_rows ? seq_of(cu, n_seq, i, from) : -1;
  rows[threadIdx.x] = place(kv, start, s, s < 0 ? 0 : i - cu[s]);
}
LLM_DEV void find_mended(const KvView &kv, const int32_t *cu, const int32_t *start, int n_seq,
                         int64_t n_rows, int64_t i0, int64_t *rows) {
  const int64_t i = i0 + threadIdx.x;
  int begin = 0;
  const int s = mended_seq_of(cu, n_seq, n_rows, i, &begin);
  const int64_t row = i < n_rows ? place(kv, start, s, i - begin) : NO_SEQUENCE;
  rows[threadIdx.x] = row;
  if (kv.flag) {
    if (row == NO_PLACE) atomicOr(kv.flag, PK_BAD_PAGE);
    if (i == 0) atomicOr(kv.flag, PK_BAD_OFFSETS);
  }
}
LLM_DEV void flag_places(const KvView &kv, const int64_t *rows) {  // of the fast path
  if (threadIdx.x < 32 && kv.flag && rows[threadIdx.x] == NO_PLACE) atomicOr(kv.flag, PK_BAD_PAGE);
}

// Rows [i1, end) of this block in the mended offsets, a thread for each row and
// head.  (Calls of their own, so that they cost the fast path no registers.)
template <typename T, int FMT>
__device__ __noinline__ void write_mended(const KvView kv, const T *qkv, int64_t ld,
                                          const int32_t *cu, const int32_t *start, int n_seq,
                                          int64_t n_rows, int H, int64_t i1, int64_t end,
                                          int64_t *rows) {
  const int first = blockIdx.y * RW_HEADS, heads = min(2 * kv.Hkv, first + RW_HEADS);
#pragma unroll 1
  for (int64_t i0 = i1; i0 < end; i0 += RW_ROWS) {
    __syncthreads();
    if (threadIdx.x < 32) find_mended(kv, cu, start, n_seq, n_rows, i0, rows);
    __syncthreads();
    const int r = threadIdx.x / RW_HEADS, h = first + threadIdx.x % RW_HEADS;
    if (rows[r] < 0 || h >= heads) continue;
    const T *src = qkv + (i0 + r) * ld + (int64_t)(H + h) * kv.hd;
    const int64_t dst = rows[r] + (int64_t)h * kv.ps;
    float x[8], inv = 0.f, scale = 0.f;
    uint32_t top = 0;
    if constexpr (FMT >= KV_E4M3) {
#pragma unroll 1
      for (int c = 0; c < kv.hd; c++) top = max(top, __float_as_uint(to_f(src[c])) & 0x7fffffffu);
      scale = row_scale<FMT>(top, &inv);
      kv.scales[dst] = scale;
    }
#pragma unroll 1
    for (int c = 0; c < kv.hd; c += 8) {
      read8(src + c, false, kv.hd - c, x);
      if constexpr (FMT == KV_F32) {
        write8(reinterpret_cast<float *>(kv.pages) + dst * kv.hd + c, false, kv.hd - c, x);
      } else if constexpr (FMT == KV_BF16) {
        write8(reinterpret_cast<__nv_bfloat16 *>(kv.pages) + dst * kv.hd + c, false, kv.hd - c, x);
      } else {
        uint32_t code[2] = {0u, 0u};
        if (top < 0x7f800000u) encode8<FMT>(x, scale, inv, code);
        write8(kv.pages + dst * kv.hd + c, false, kv.hd - c, code);
      }
    }
  }
}
template <typename T, int FMT>
__device__ __noinline__ void read_mended(const KvView kv, const int32_t *cu, const int32_t *start,
                                         int n_seq, int64_t n_rows, T *k, T *v, int64_t i1,
                                         int64_t end, int64_t *rows) {
  const int first = blockIdx.y * RW_HEADS, heads = min(2 * kv.Hkv, first + RW_HEADS);
  const int64_t w = (int64_t)kv.Hkv * kv.hd;
#pragma unroll 1
  for (int64_t i0 = i1; i0 < end; i0 += RW_ROWS) {
    __syncthreads();
    if (threadIdx.x < 32) find_mended(kv, cu, start, n_seq, n_rows, i0, rows);
    __syncthreads();
    const int r = threadIdx.x / RW_HEADS, h = first + threadIdx.x % RW_HEADS;
    const int64_t row = rows[r], src = row + (int64_t)h * kv.ps;
    if (row == NO_SEQUENCE || h >= heads) continue;
    T *dst = (h < kv.Hkv ? k : v - w) + (i0 + r) * w + (int64_t)h * kv.hd;
    float x[8] = {}, sc = 1.f;
    if constexpr (FMT >= KV_E4M3) sc = row >= 0 ? kv.scales[src] : 0.f;
#pragma unroll 1
    for (int c = 0; c < kv.hd; c += 8) {
      if (row >= 0) kv_read8<FMT>(kv.pages, src * kv.hd + c, false, kv.hd - c, x);
      if constexpr (FMT >= KV_E4M3) {
#pragma unroll
        for (int j = 0; j < 8; j++) x[j] *= sc;
      }
      write8(dst + c, false, kv.hd - c, x);
    }
  }
}

// A block looks whether the offsets are bad while warp 0 searches (MANY, where it
// takes 32 rows several times: before); where they are, it leaves its rows to
// write_mended and read_mended.  (Blocks an SM: more registers and fewer blocks
// were 5 to 15% slower.)
template <typename T, int FMT, int LPH, bool VEC, bool MANY>
__global__ void __launch_bounds__(RW_THREADS, FMT < KV_E4M3 && !MANY && LPH < 16 ? 5 : 4)
    k_write(const KvView kv, const T *__restrict__ qkv, int64_t ld, const int32_t *__restrict__ cu,
            const int32_t *__restrict__ start, int n_seq, int64_t n_rows, int H) {
  __shared__ int64_t rows[RW_ROWS];
  const int64_t step = RW_ROWS * cdiv(n_rows, (int64_t)gridDim.x * RW_ROWS);  // MANY
  const int64_t i1 = blockIdx.x * (MANY ? step : RW_ROWS);
  const int64_t end = MANY ? min(i1 + step, n_rows) : min(i1 + RW_ROWS, n_rows);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = (lane % LPH) * 8;
  // k heads, then v heads: the pages' own order; RW_HEADS of them a block
  const int first = blockIdx.y * RW_HEADS, heads = min(2 * kv.Hkv, first + RW_HEADS);
  int from = 0;
  bool bad = MANY && __syncthreads_or(bad_offsets<8>(cu, n_seq, n_rows, threadIdx.x, RW_THREADS));
  // the first entries' loads ahead of the rows'
  const int s1 = !MANY && warp > 0 ? min((int)threadIdx.x - 32, n_seq) : n_seq;
  const int c0 = MANY ? 0 : cu[s1], c1 = MANY ? 0 : cu[min(s1 + 1, n_seq)];
  // every warp, before its first use of the places
  auto meet = [&] {
    if (MANY) {
      __syncthreads();
    } else {
      bad = c0 < 0 || c0 > c1 || c0 > n_rows;
      if (warp > 0) bad |= bad_offsets<1>(cu, n_seq, n_rows, s1 + RW_LOOK, RW_LOOK);
      bad = __syncthreads_or(bad);
    }
    if (!bad) flag_places(kv, rows);
  };
  int64_t i0 = i1;
  if (!bad) do {
    if (warp == 0) find_places(kv, cu, start, n_seq, n_rows, i0, rows, from);
    for (int g = warp; g < LPH; g += RW_THREADS / 32) {
      const int r = g * (32 / LPH) + lane / LPH;
      const bool in = i0 + r < n_rows && e < kv.hd;
      const T *src = qkv + (i0 + r) * ld + (int64_t)H * kv.hd + e;
      for (int h0 = first; h0 < heads; h0 += WU) {
        float x[WU][8];
#pragma unroll
        for (int k = 0; k < WU; k++) {
          if (in && h0 + k < heads) {
            read8(src + (h0 + k) * kv.hd, VEC, kv.hd - e, x[k]);
          } else {
#pragma unroll
            for (int j = 0; j < 8; j++) x[k][j] = 0.f;
          }
        }
        if (g == warp && h0 == first) meet();
        const int64_t row = rows[r];
        const bool on = in && row >= 0 && !bad;
#pragma unroll
        for (int k = 0; k < WU; k++) {
          if (h0 + k >= heads) break;
          const int64_t dst = row + (int64_t)(h0 + k) * kv.ps;
          if constexpr (FMT == KV_F32) {
            if (on)
              write8(reinterpret_cast<float *>(kv.pages) + dst * kv.hd + e, VEC, kv.hd - e, x[k]);
          } else if constexpr (FMT == KV_BF16) {
            if (on)
              write8(reinterpret_cast<__nv_bfloat16 *>(kv.pages) + dst * kv.hd + e, VEC, kv.hd - e,
                     x[k]);
          } else {
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < 8; j++) top = max(top, __float_as_uint(x[k][j]) & 0x7fffffffu);
#pragma unroll
            for (int o = 1; o < LPH; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            float inv;
            const float scale = row_scale<FMT>(top, &inv);
            uint32_t c[2] = {0u, 0u};
            if (top < 0x7f800000u) encode8<FMT>(x[k], scale, inv, c);
            if (on) {
              write8(kv.pages + dst * kv.hd + e, VEC, kv.hd - e, c);
              if (e == 0) kv.scales[dst] = scale;
            }
          }
        }
      }
    }
    if (warp >= LPH) meet();  // warps without rows
    if (MANY) __syncthreads();  // the places have been read
    i0 += RW_ROWS;
  } while (MANY && i0 < end);
  if (bad) write_mended<T, FMT>(kv, qkv, ld, cu, start, n_seq, n_rows, H, i1, end, rows);
}

// A row without a place reads as zeros, rows of no sequence are left alone.
template <typename T, int FMT, int LPH, bool VEC, bool MANY>
__global__ void __launch_bounds__(RW_THREADS, FMT == KV_INT8 && VEC && !MANY ? 8 : 6)
    k_read(const KvView kv, const int32_t *__restrict__ cu, const int32_t *__restrict__ start,
           int n_seq, int64_t n_rows, T *__restrict__ k, T *__restrict__ v) {
  __shared__ int64_t rows[RW_ROWS];
  const int64_t step = RW_ROWS * cdiv(n_rows, (int64_t)gridDim.x * RW_ROWS);  // MANY
  const int64_t i1 = blockIdx.x * (MANY ? step : RW_ROWS);
  const int64_t end = MANY ? min(i1 + step, n_rows) : min(i1 + RW_ROWS, n_rows);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = (lane % LPH) * 8;
  const int first = blockIdx.y * RW_HEADS, heads = min(2 * kv.Hkv, first + RW_HEADS);
  const int64_t w = (int64_t)kv.Hkv * kv.hd;
  int from = 0;
  bool bad = MANY && __syncthreads_or(bad_offsets<8>(cu, n_seq, n_rows, threadIdx.x, RW_THREADS));
  int64_t i0 = i1;
  if (!bad) do {
    if (warp == 0) find_places(kv, cu, start, n_seq, n_rows, i0, rows, from);
    if (MANY)
      __syncthreads();
    else
      bad = __syncthreads_or(warp > 0 &&
                             bad_offsets<4>(cu, n_seq, n_rows, threadIdx.x - 32, RW_LOOK));
    if (!bad) flag_places(kv, rows);
    for (int g = bad ? LPH : warp; g < LPH; g += RW_THREADS / 32) {
      const int r = g * (32 / LPH) + lane / LPH;
      const int64_t row = rows[r];
      if (row == NO_SEQUENCE || e >= kv.hd) continue;
      T *kd = k + (i0 + r) * w + e, *vd = v + (i0 + r) * w - w + e;  // v of head h - Hkv
      for (int h0 = first; h0 < heads; h0 += RU) {
        float x[RU][8], sc[RU];
#pragma unroll
        for (int m = 0; m < RU; m++) {
          sc[m] = 1.f;
          if (row >= 0 && h0 + m < heads) {
            const int64_t src = row + (int64_t)(h0 + m) * kv.ps;
            kv_read8<FMT>(kv.pages, src * kv.hd + e, VEC, kv.hd - e, x[m]);
            if constexpr (FMT >= KV_E4M3) sc[m] = kv.scales[src];
          } else {
#pragma unroll
            for (int j = 0; j < 8; j++) x[m][j] = 0.f;
          }
        }
#pragma unroll
        for (int m = 0; m < RU; m++) {
          const int h = h0 + m;
          if (h >= heads) break;
          if constexpr (FMT >= KV_E4M3) {
#pragma unroll
            for (int j = 0; j < 8; j++) x[m][j] *= sc[m];
          }
          write8((h < kv.Hkv ? kd : vd) + (int64_t)h * kv.hd, VEC, kv.hd - e, x[m]);
        }
      }
    }
    if (MANY) __syncthreads();  // the places have been read
    i0 += RW_ROWS;
  } while (MANY && i0 < end);
  if (bad) read_mended<T, FMT>(kv, cu, start, n_seq, n_rows, k, v, i1, end, rows);
}

// --------------------------------------------------------------- attention
// The work of a call is the (sequence, kv head) pairs in order, each
// ceil(len / 64) units of 64 positions behind PG_SETUP units that stand for what a
// pair costs before its first position (its queries, the first loads' latency,
// the warps' joining: about that of 3 units; without them the blocks that got
// many short sequences ran 1.4 times as long as the others): W units in a row,
// of which block i of N (at most W, so that none is empty) takes
// [W i / N, W (i + 1) / N) whatever the lengths are.  A pair that lies
// in one block is finished there; a pair cut between blocks leaves, per block,
// the running maximum, sum and weighted values of its part in the workspace,
// and a second kernel joins the parts in order.  A block's range cuts at most
// its first and its last pair: two slots per block.
constexpr int AT = 128;       // threads
constexpr int BLOCKS_SM = 4;  // most blocks per SM that the split counts on
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
LLM_DEV int units_of(int len) {
  return len > 0 ? PG_SETUP + (len + PG_UNIT - 1) / PG_UNIT : 0;
}
// pre[s] = units of the sequences before s, per kv head (n_seq + 1 entries).
LLM_DEV void unit_prefix(const KvView &kv, const int32_t *lens, int n_seq, int *pre) {
  __shared__ int tot[AT / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int carry = 0;
  for (int s0 = 0; s0 < n_seq; s0 += AT) {
    const int s = s0 + threadIdx.x;
    int v = s < n_seq ? units_of(clamped_len(kv, lens, s)) : 0;
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
// the head's columns, and GT query heads of the kv head at once; U such groups
// of positions have their loads in flight together.  The float32 form, and that
// of layouts the tensor-core kernel does not take.  32 sequences of 4096
// positions, 16 heads of 64 (float32 queries): float32 cache 165 us (6.5 TB/s;
// U = 1: 239), bfloat16 209 (U = 1: 319), 8-bit 257 (U = 4: 394, 1: 337), bound by
// the arithmetic a position costs (a dot product, 3 shuffles and an exponential
// for 8 lanes), as are grouped heads.
template <typename T, int FMT, int HD, int GT, bool VEC>
__global__ void __launch_bounds__(AT)
    k_attend(const KvView kv, const T *__restrict__ q, int64_t q_ld,
             const int32_t *__restrict__ lens, const Sched sc, int H, T *__restrict__ o,
             float *__restrict__ lse, int *__restrict__ pre_out, float *__restrict__ part) {
  constexpr int EPL = HD / 8, NC = (EPL + 7) / 8;  // columns a lane, 8-element pieces
  constexpr int U = FMT < KV_E4M3 && EPL * GT <= 8 ? 4 : EPL * GT <= 32 ? 2 : 1;
  extern __shared__ int pre[];
  __shared__ float sm[AT / 32][GT][HD + 2];
  pk_release();
  if (!sc.direct) {
    unit_prefix(kv, lens, sc.n_seq, pre);
    if (blockIdx.x == 0)
      for (int s = threadIdx.x; s <= sc.n_seq; s += AT) pre_out[s] = pre[s];
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane & 7, ks = lane >> 3;
  const int grp = H / kv.Hkv, hd = kv.hd;
  const float sl2 = LOG2E / sqrtf((float)hd);
  int64_t w = 0, end = 1;
  if (!sc.direct) {
    const int64_t W = (int64_t)pre[sc.n_seq] * kv.Hkv;
    const int N = (int)min((int64_t)sc.N, W);
    if ((int)blockIdx.x >= N) return;
    w = block_begin(W, blockIdx.x, N);
    end = block_begin(W, blockIdx.x + 1, N);
  }
  for (int piece = 0; w < end; piece++) {
    int s, g, u0, nu, units;
    if (sc.direct) {
      s = blockIdx.x / kv.Hkv;
      g = blockIdx.x % kv.Hkv;
      u0 = nu = units = 0;
      if (threadIdx.x == 0) clamped_len(kv, lens, s);  // a bad length is flagged
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
    const int j0 = sc.direct ? 0 : max(u0 - PG_SETUP, 0) * PG_UNIT;
    const int j1 = sc.direct ? len : min(len, max(u0 + nu - PG_SETUP, 0) * PG_UNIT);
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
      bool bad = false;  // a position without a place
      for (int j = j0 + warp * 4; j < j1; j += AT / 32 * 4 * U) {
        int64_t kr[U], row[U];
        float kx[U][8 * NC], vx[U][8 * NC], vs[U], kscale[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
          const int jj = j + u * (AT / 32 * 4) + ks;
          row[u] = jj < j1 ? kv_row(kv, s, jj) : -1;
          bad |= jj < j1 && row[u] < 0;
          kr[u] = row[u] + (int64_t)g * kv.ps;
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
          const int64_t vr = kr[u] + (int64_t)kv.Hkv * kv.ps;
#pragma unroll
          for (int c = 0; c < NC; c++) {
            float a[8] = {}, b[8] = {};
            const int e = sub * EPL + 8 * c, n = min(hd - e, EPL - 8 * c);
            if (row[u] >= 0 && n > 0) {
              kv_read8<FMT>(kv.pages, kr[u] * hd + e, VEC && EPL >= 8, n, a);
              kv_read8<FMT>(kv.pages, vr * hd + e, VEC && EPL >= 8, n, b);
            }
#pragma unroll
            for (int i = 0; i < 8; i++) {
              kx[u][8 * c + i] = a[i];
              vx[u][8 * c + i] = b[i];
            }
          }
          vs[u] = kscale[u] = 1.f;
          if constexpr (FMT >= KV_E4M3) {
            if (row[u] >= 0) {
              kscale[u] = kv.scales[kr[u]];
              vs[u] = kv.scales[vr];
            }
          }
        }
#pragma unroll
        for (int r = 0; r < GT; r++) {
          float t[U], mn = m[r];
#pragma unroll
          for (int u = 0; u < U; u++) {
            t[u] = 0.f;
#pragma unroll
            for (int c = 0; c < EPL; c++) t[u] = fmaf(qv[r][c], kx[u][c], t[u]);
#pragma unroll
            for (int x = 1; x < 8; x <<= 1) t[u] += __shfl_xor_sync(0xffffffffu, t[u], x);
            t[u] *= kscale[u];
            if (row[u] < 0) t[u] = -INFINITY;  // no such position: weight 0, v read as 0
            mn = fmaxf(mn, t[u]);
          }
          const float ref = mn == -INFINITY ? 0.f : mn, corr = exp2f(m[r] - ref);
          l[r] *= corr;
          m[r] = mn;
#pragma unroll
          for (int c = 0; c < EPL; c++) acc[r][c] *= corr;
#pragma unroll
          for (int u = 0; u < U; u++) {
            const float p = exp2f(t[u] - ref), pv = p * vs[u];
            l[r] += p;
#pragma unroll
            for (int c = 0; c < EPL; c++) acc[r][c] = fmaf(pv, vx[u][c], acc[r][c]);
          }
        }
      }
      if (bad && kv.flag && sub == 0) atomicOr(kv.flag, PK_BAD_PAGE);
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

// ------------------------------------------- bfloat16 queries, tensor cores
// The same work on mma.m16n8k16, the cached rows as the 16-row operand, so
// that a kv head's query heads fill the 8 columns (NT column tiles) and no
// row of a product is padding:
//   S^T [16 keys x 8 heads]  = K [16 x HD] q^T       (HD / 16 steps)
//   O^T [16 columns x 8] += V^T [16 x 16 keys] P^T   (HD / 16 tiles)
// Nothing passes through shared memory: a lane reads its operands of K and V
// from global memory in 16-byte (or row / 8) pieces, because the sums over
// head columns (S) and over keys (O) may take them in any order: lane (g, t) =
// (lane / 4, lane % 4) reads of key g a contiguous quarter of the row and
// calls its columns k-step s those that the fragment wants, and of keys
// 2t, 2t+1, 2t+8, 2t+9 an eighth of the row.  P^T comes from S^T's own
// registers by transposing 8 x 8 blocks (movmatrix).  Each of the 4 warps
// takes SB x 16 keys at a time with the next ones' loads in flight (K's issued
// as soon as S is formed, V's after O), so the kernel needs no barrier until
// the warps meet, and a block's latency is a few loads.  BIG: the SB x 16
// positions lie in one page (page sizes of a multiple of SB x 16), so one
// table entry and one address serve them; else each 8 positions have their
// own.  GC: query heads a lane holds of a column tile, 1 when the kv head has
// one query head (its second column, as the other lanes', is padding).
// 8-bit caches: codes become float16 exactly (e4m3 and 8-bit integers both
// fit); q is scaled per head by a power of two into [1, 2) so that it fits
// float16's range; K's row scale multiplies the scores.  V's row scale cannot
// be left to the products' end, so it joins the weight: 2^(s + log2 scale -
// mo), whose reference mo of its own (the running maximum of s + log2 scale)
// holds it within float16 whatever the scales are.
// The rounding of the weights to float16 (2^-12) is the only one below 32
// bits, and the sum l takes them unrounded; a bfloat16 cache takes each weight
// as two bfloat16 terms (2^-17: rounded to one, the outputs of a long context
// were 1.45 times as far off as their own rounding; the loads hide the second
// product).
// Measured: 32 sequences to 16384 positions, 16 heads of 64, e4m3, 280 MB: 55 us,
// 5.1 TB/s; one of 100001, bfloat16, 410 MB: 72 us, 5.7 TB/s, the loads' latency
// (10.7 of the 15 cycles between a warp's instructions) at 4 warps a scheduler,
// which is all that the operands' registers leave room for.
constexpr int NW = AT / 32;
// Blocks per SM: what the registers of a lane's operands leave room for.
constexpr int mma_blocks(int HD, int NT) { return NT == 2 ? 2 : HD == 128 ? 3 : 4; }
static_assert(mma_blocks(32, 1) <= BLOCKS_SM, "the workspace counts BLOCKS_SM");
// log2 units a maximum may grow before O is rescaled, and the log2 of a weight
// at its reference: a float16 weight is at most 2^(14 + 1), and those below
// 2^-14 keep steps of 2^-24, 2^-38 of the reference
template <bool BF> constexpr float LAZY = BF ? 8.f : 1.f;
constexpr float OFF16 = 14.f;

// W consecutive 32-bit words, read once.
template <int W>
LLM_DEV void ldg(const uint8_t *p, uint32_t *r) {
  if constexpr (W % 4 == 0) {
    asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "l"(p));
  } else if constexpr (W == 2) {
    asm volatile("ld.global.nc.L1::no_allocate.v2.b32 {%0,%1}, [%2];"
                 : "=r"(r[0]), "=r"(r[1]) : "l"(p));
  } else {
    asm volatile("ld.global.nc.L1::no_allocate.b32 %0, [%1];" : "=r"(r[0]) : "l"(p));
  }
}
template <bool BF>
LLM_DEV void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                 uint32_t b1) {
  if constexpr (BF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transposes the 8 x 8 matrix of 16-bit values the warp holds (row lane / 4,
// columns 2 (lane % 4) and the next).
LLM_DEV uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
template <bool BF>
LLM_DEV uint32_t pack16(float lo, float hi) {
  if constexpr (BF) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
  } else {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
}
LLM_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
LLM_DEV float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Codes in bytes (0, 1) of w, and (2, 3), as float16 pairs.
template <int FMT>
LLM_DEV void half_pairs(uint32_t w, uint32_t &lo, uint32_t &hi) {
  if constexpr (FMT == KV_E4M3) {
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n"
        " cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    // byte + 128 as the low mantissa bits of 1024: 0x6400 | (c + 128) = 1152 + c
    const uint32_t u = w ^ 0x80808080u, k = 0x64806480u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 kk = *reinterpret_cast<const __half2 *>(&k);
    const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&a), kk);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2 *>(&b), kk);
    lo = *reinterpret_cast<const uint32_t *>(&x);
    hi = *reinterpret_cast<const uint32_t *>(&y);
  }
}
// Joins the warps' parts of one piece (m, l and O, in sm [NW][8 NT][HD + 2])
// and writes the outputs, or the record of a cut pair: see k_attend.
template <int HD, int HEADS>
LLM_DEV void finish(const float *sm, int grp, int r0, int hd, bool whole, __nv_bfloat16 *o,
                    float *lse, float *rec) {
  for (int i = threadIdx.x; i < min(HEADS, grp - r0) * HD; i += AT) {
    const int r = i / HD, e = i % HD;
    float M = -INFINITY;
#pragma unroll
    for (int x = 0; x < NW; x++) M = fmaxf(M, sm[(x * HEADS + r) * (HD + 2) + HD]);
    const float ref = M == -INFINITY ? 0.f : M;
    float L = 0.f, v = 0.f;
#pragma unroll
    for (int x = 0; x < NW; x++) {
      const float *w = sm + (x * HEADS + r) * (HD + 2);
      const float f = exp2f(w[HD] - ref);
      L = fmaf(f, w[HD + 1], L);
      v = fmaf(f, w[e], v);
    }
    if (whole) {
      o[(r0 + r) * hd + e] = from_f<__nv_bfloat16>(L == 0.f ? 0.f : v / L);
      if (e == 0 && lse) lse[r0 + r] = (M + log2f(L)) * LN2;
    } else {
      rec[(r0 + r) * (hd + 2) + 2 + e] = v;
      if (e == 0) {
        rec[(r0 + r) * (hd + 2)] = M;
        rec[(r0 + r) * (hd + 2) + 1] = L;
      }
    }
  }
}

template <int FMT, int HD, int NT, int SB, int GC, bool BIG>
__global__ void __launch_bounds__(AT, mma_blocks(HD, NT))
    k_attend_mma(const KvView kv, const __nv_bfloat16 *__restrict__ q, int64_t q_ld,
                 const int32_t *__restrict__ lens, const Sched sc, int H,
                 __nv_bfloat16 *__restrict__ o, float *__restrict__ lse,
                 int *__restrict__ pre_out, float *__restrict__ part) {
  constexpr bool BF = FMT == KV_BF16;
  constexpr int ES = BF ? 2 : 1, KW = HD * ES / 16, VW = HD * ES / 32;  // words a lane and key
  constexpr int KC = KW < 4 ? KW : 4, VC = VW < 4 ? VW : 4;            // words of one load
  constexpr int KB = 16 * SB, GR = BIG ? 1 : 2 * SB, WI = 32 / GR, HEADS = 8 * NT;
  constexpr uint32_t ALL = (1u << GR) - 1;
  extern __shared__ int pre[];
  __shared__ float sm[NW * HEADS * (HD + 2)];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, lg = lane >> 2, lt = lane & 3;
  const int grp = H / kv.Hkv;
  const float sl2 = LOG2E / sqrtf((float)HD);
  int64_t w = 0, end = 1;
  if (!sc.direct) {
    pk_release();
    unit_prefix(kv, lens, sc.n_seq, pre);
    if (blockIdx.x == 0)
      for (int s = threadIdx.x; s <= sc.n_seq; s += AT) pre_out[s] = pre[s];
    const int64_t W = (int64_t)pre[sc.n_seq] * kv.Hkv;
    const int N = (int)min((int64_t)sc.N, W);
    if ((int)blockIdx.x >= N) return;
    w = block_begin(W, blockIdx.x, N);
    end = block_begin(W, blockIdx.x + 1, N);
  }
  for (int piece = 0; w < end; piece++) {
    int s, g, j0, j1;
    bool whole = true;
    if (sc.direct) {
      s = blockIdx.x / kv.Hkv;
      g = blockIdx.x % kv.Hkv;
      j0 = 0;
      j1 = clamped_len(kv, lens, s);
      w = end;
    } else {
      s = seq_at(pre, sc.n_seq, w, kv.Hkv);
      const int units = pre[s + 1] - pre[s];
      const int64_t in = w - (int64_t)pre[s] * kv.Hkv;
      g = (int)(in / units);
      const int u0 = (int)(in - (int64_t)g * units);
      const int nu = (int)min((int64_t)(units - u0), end - w);
      w += nu;
      whole = nu == units;
      const int64_t cap = (int64_t)kv.table_pages * kv.ps;
      j0 = max(u0 - PG_SETUP, 0) * PG_UNIT;
      j1 = (int)min(min((int64_t)lens[s], cap), (int64_t)max(u0 + nu - PG_SETUP, 0) * PG_UNIT);
    }
    const int32_t *table = kv.table + (int64_t)s * kv.table_ld;
    const int64_t vrows = (int64_t)kv.Hkv * kv.ps;  // from a key's row to its value's
    const int nit = (max(j1 - j0, 0) + NW * KB - 1) / (NW * KB);
    for (int r0 = 0; r0 < grp; r0 += HEADS) {
      // q^T fragments: head lg of each tile, columns as K's words hold them
      uint32_t qf[NT][HD / 16][2];
      float qs[NT][2];  // log2-score factor of this lane's heads 2 lt, 2 lt + 1
#pragma unroll
      for (int n = 0; n < NT; n++) {
        const int hh = r0 + n * 8 + lg;
        const __nv_bfloat16 *qr = q + s * q_ld + (int64_t)(g * grp + hh) * HD;
        float x[HD / 16][4], top = 0.f;
#pragma unroll
        for (int ks = 0; ks < HD / 16; ks++) {
          const int d = BF ? (ks / 2 * 4 + lt) * 8 + (ks & 1) * 4
                           : KW == 2 ? lt * 8 + ks * 4 : (ks / 4 * 4 + lt) * 16 + (ks & 3) * 4;
#pragma unroll
          for (int i = 0; i < 4; i++) {
            x[ks][i] = hh < grp ? to_f(qr[d + i]) : 0.f;
            top = fmaxf(top, fabsf(x[ks][i]));
          }
        }
        float up = 1.f, down = 1.f;
        if constexpr (!BF) {
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const int e = (int)(__float_as_uint(top) >> 23);  // top < 2^128: its exponent
          if (e > 0 && e < 255) {  // up = 2^-(e - 127), within [2^-126, 2^126]
            const int k = min(max(e - 127, -126), 126);
            up = __uint_as_float((uint32_t)(127 - k) << 23);
            down = __uint_as_float((uint32_t)(127 + k) << 23);
          }
        }
#pragma unroll
        for (int ks = 0; ks < HD / 16; ks++) {
          qf[n][ks][0] = pack16<BF>(x[ks][0] * up, x[ks][1] * up);
          qf[n][ks][1] = pack16<BF>(x[ks][2] * up, x[ks][3] * up);
        }
        // the factors of heads 2 lt and 2 lt + 1 sit in lanes of rows lg = those
        qs[n][0] = sl2 * __shfl_sync(0xffffffffu, down, 8 * lt);
        qs[n][1] = sl2 * __shfl_sync(0xffffffffu, down, 8 * lt + 4);
      }
      float acc[NT][HD / 16][4], m[NT][GC], mo[NT][GC], l[NT][GC];
#pragma unroll
      for (int n = 0; n < NT; n++) {
#pragma unroll
        for (int c = 0; c < GC; c++) {
          m[n][c] = mo[n][c] = -INFINITY;
          l[n][c] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < HD / 16; i++)
#pragma unroll
          for (int c = 0; c < 4; c++) acc[n][i][c] = 0.f;
      }
      uint32_t kr[SB][2][KW], vr[SB][4][VW];
      float kscale[SB][2], vscale[SB][2];
      // the window: first row of the positions that lane i looked up (group
      // i % GR of iteration i / GR from the window's first on), -1 for none
      int win = -1;
      uint32_t there = 0, there_next = 0;  // groups of the iteration whose page exists
      bool full = false, full_next = false;  // every position counts
      auto look_up = [&](int it) {
        if (it % WI == 0) {
          const int64_t key =
              j0 + ((int64_t)(it + lane / GR) * NW + warp) * KB + (lane % GR) * (KB / GR);
          win = -1;
          if (key < j1) {
            const uint32_t pg = (uint32_t)key / (uint32_t)kv.ps;
            const int64_t page = table[pg];
            if (page >= 0 && page < kv.n_pages)
              win = (int)(page * (2 * vrows)) + g * kv.ps + (int)((uint32_t)key - pg * kv.ps);
            else if (kv.flag)
              atomicOr(kv.flag, PK_BAD_PAGE);
          }
        }
      };
      const uint8_t *klane = kv.pages + lg * (HD * ES) + lt * (KC * 4);
      const uint8_t *vlane = kv.pages + (vrows + 2 * lt) * (HD * ES) + lg * (VC * 4);
      const float *slane = kv.scales + lg;
      auto load_k = [&](int it) {
        look_up(it);
        const int64_t key0 = j0 + ((int64_t)it * NW + warp) * KB;
        there_next = 0;
        int row[GR];
#pragma unroll
        for (int i = 0; i < GR; i++) {
          row[i] = __shfl_sync(0xffffffffu, win, (it % WI) * GR + i);
          there_next |= (uint32_t)(row[i] >= 0) << i;
        }
        full_next = there_next == ALL && key0 + KB <= j1;
#pragma unroll
        for (int b = 0; b < SB; b++)
#pragma unroll
          for (int hf = 0; hf < 2; hf++) {
            // BIG: positions in one page, consecutive rows
            const int64_t r = BIG ? (int64_t)row[0] + 16 * b + 8 * hf : row[(2 * b + hf) % GR];
            const bool on = full_next || (BIG ? there_next != 0 : r >= 0);
            if (on) {
#pragma unroll
              for (int c = 0; c < KW / KC; c++) ldg<KC>(klane + r * (HD * ES) + c * 64, &kr[b][hf][c * KC]);
              if constexpr (!BF) kscale[b][hf] = __ldg(slane + r);
            } else {
#pragma unroll
              for (int i = 0; i < KW; i++) kr[b][hf][i] = 0;
              kscale[b][hf] = 0.f;
            }
          }
      };
      auto load_v = [&](int it) {
        const int64_t key0 = j0 + ((int64_t)it * NW + warp) * KB;
        int row[GR];
#pragma unroll
        for (int i = 0; i < GR; i++) row[i] = __shfl_sync(0xffffffffu, win, (it % WI) * GR + i);
#pragma unroll
        for (int b = 0; b < SB; b++)
#pragma unroll
          for (int hf = 0; hf < 2; hf++) {
            const int64_t r = BIG ? (int64_t)row[0] + 16 * b + 8 * hf : row[(2 * b + hf) % GR];
            const uint8_t *p = vlane + r * (HD * ES);
            const int64_t key = key0 + 16 * b + 8 * hf;
            if (full_next) {
#pragma unroll
              for (int k = 0; k < 2; k++)
#pragma unroll
                for (int c = 0; c < VW / VC; c++)
                  ldg<VC>(p + k * (HD * ES) + c * 128, &vr[b][2 * hf + k][c * VC]);
              if constexpr (!BF) vscale[b][hf] = __ldg(slane + r + vrows);
            } else {  // zeros where no position counts: 0 weights meet numbers
              const bool page = BIG ? there_next != 0 : r >= 0;
#pragma unroll
              for (int k = 0; k < 2; k++) {
#pragma unroll
                for (int i = 0; i < VW; i++) vr[b][2 * hf + k][i] = 0;
                if (page && key + 2 * lt + k < j1)
#pragma unroll
                  for (int c = 0; c < VW / VC; c++)
                    ldg<VC>(p + k * (HD * ES) + c * 128, &vr[b][2 * hf + k][c * VC]);
              }
              if constexpr (!BF)
                vscale[b][hf] = page && key + lg < j1 ? __ldg(slane + r + vrows) : 0.f;
            }
          }
      };
      if (nit > 0) {
        load_k(0);
        load_v(0);
        there = there_next;
        full = full_next;
      }
      for (int it = 0; it < nit; it++) {
        float st[NT][SB][4];
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
          for (int b = 0; b < SB; b++)
#pragma unroll
            for (int c = 0; c < 4; c++) st[n][b][c] = 0.f;
#pragma unroll
        for (int b = 0; b < SB; b++)
#pragma unroll
          for (int ks = 0; ks < HD / 16; ks++) {
            uint32_t a[4];
            if constexpr (BF) {
              a[0] = kr[b][0][2 * ks];
              a[2] = kr[b][0][2 * ks + 1];
              a[1] = kr[b][1][2 * ks];
              a[3] = kr[b][1][2 * ks + 1];
            } else {
              half_pairs<FMT>(kr[b][0][ks], a[0], a[2]);
              half_pairs<FMT>(kr[b][1][ks], a[1], a[3]);
            }
#pragma unroll
            for (int n = 0; n < NT; n++)
              mma<BF>(st[n][b], a[0], a[1], a[2], a[3], qf[n][ks][0], qf[n][ks][1]);
          }
        // log2 scores x[n][b][hf][c] of keys 16 b + 8 hf + lg, heads 2 lt + c
        float x[NT][SB][2][GC], lv[SB][2];
#pragma unroll
        for (int b = 0; b < SB; b++)
#pragma unroll
          for (int hf = 0; hf < 2; hf++) {
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
              for (int c = 0; c < GC; c++)
                x[n][b][hf][c] = st[n][b][2 * hf + c] * (BF ? qs[n][c] : qs[n][c] * kscale[b][hf]);
            lv[b][hf] = BF ? 0.f : lg2(vscale[b][hf]);
          }
        if (!full) {  // keys past the end or without a page: weight 0
          const int64_t key0 = j0 + ((int64_t)it * NW + warp) * KB;
#pragma unroll
          for (int b = 0; b < SB; b++)
#pragma unroll
            for (int hf = 0; hf < 2; hf++)
              if (key0 + 16 * b + 8 * hf + lg >= j1 || !(there >> (BIG ? 0 : 2 * b + hf) & 1)) {
#pragma unroll
                for (int n = 0; n < NT; n++)
#pragma unroll
                  for (int c = 0; c < GC; c++) x[n][b][hf][c] = -INFINITY;
                lv[b][hf] = 0.f;
              }
        }
        if (it + 1 < nit) load_k(it + 1);
        // a maximum that grew by more than that moves its reference (in every
        // lane of the head: the lanes of its keys agree by shuffles)
        bool grew = false;
        float top[NT][GC], topo[NT][GC];
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
          for (int c = 0; c < GC; c++) {
            float a = -INFINITY, z = -INFINITY;
#pragma unroll
            for (int b = 0; b < SB; b++)
#pragma unroll
              for (int hf = 0; hf < 2; hf++) {
                a = fmaxf(a, x[n][b][hf][c]);
                if constexpr (!BF) z = fmaxf(z, x[n][b][hf][c] + lv[b][hf]);
              }
            top[n][c] = a;
            topo[n][c] = z;
            grew |= a > m[n][c] + LAZY<BF>;
            if constexpr (!BF) grew |= z > mo[n][c] + LAZY<BF>;
          }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int n = 0; n < NT; n++)
#pragma unroll
            for (int c = 0; c < GC; c++) {
              float a = top[n][c], z = topo[n][c];
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) {
                a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
                if constexpr (!BF) z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, o));
              }
              const float mn = fmaxf(m[n][c], a);
              const float corr = mn == -INFINITY ? 1.f : ex2(m[n][c] - mn);
              l[n][c] *= corr;
              m[n][c] = mn;
              float co = corr;
              if constexpr (!BF) {
                const float zn = fmaxf(mo[n][c], z);
                co = zn == -INFINITY ? 1.f : ex2(mo[n][c] - zn);
                mo[n][c] = zn;
              }
#pragma unroll
              for (int i = 0; i < HD / 16; i++) {
                acc[n][i][c] *= co;
                acc[n][i][2 + c] *= co;
              }
            }
        }
        // weights and their B fragments
        uint32_t pf[NT][SB][2], pl[NT][SB][2];  // pl: what pf's rounding left (bfloat16)
#pragma unroll
        for (int n = 0; n < NT; n++) {
          float ref[GC], refo[GC];
#pragma unroll
          for (int c = 0; c < GC; c++) {
            ref[c] = m[n][c] == -INFINITY ? 0.f : m[n][c];
            refo[c] = (mo[n][c] == -INFINITY ? 0.f : mo[n][c]) - OFF16;
          }
#pragma unroll
          for (int b = 0; b < SB; b++)
#pragma unroll
            for (int hf = 0; hf < 2; hf++) {
              float p[2] = {0.f, 0.f};
#pragma unroll
              for (int c = 0; c < GC; c++) {
                p[c] = ex2(x[n][b][hf][c] - ref[c]);
                l[n][c] += p[c];
                if constexpr (!BF) p[c] = ex2(x[n][b][hf][c] + (lv[b][hf] - refo[c]));
              }
              const uint32_t w = pack16<BF>(p[0], p[1]);
              pf[n][b][hf] = transpose8(w);
              if constexpr (BF)
                pl[n][b][hf] = transpose8(pack16<BF>(p[0] - __uint_as_float(w << 16),
                                                     p[1] - __uint_as_float(w & 0xffff0000u)));
            }
        }
        // O^T += V^T P^T: tile i holds columns d and d + 1 of word i (bf16), or
        // a pair of the four of a word of codes
#pragma unroll
        for (int b = 0; b < SB; b++) {
#pragma unroll
          for (int i = 0; i < VW; i++) {
            if constexpr (BF) {
              const uint32_t a0 = __byte_perm(vr[b][0][i], vr[b][1][i], 0x5410);
              const uint32_t a1 = __byte_perm(vr[b][0][i], vr[b][1][i], 0x7632);
              const uint32_t a2 = __byte_perm(vr[b][2][i], vr[b][3][i], 0x5410);
              const uint32_t a3 = __byte_perm(vr[b][2][i], vr[b][3][i], 0x7632);
#pragma unroll
              for (int n = 0; n < NT; n++) {
                mma<BF>(acc[n][i], a0, a1, a2, a3, pf[n][b][0], pf[n][b][1]);
                mma<BF>(acc[n][i], a0, a1, a2, a3, pl[n][b][0], pl[n][b][1]);
              }
            } else {
              uint32_t u[4], w[4];  // columns 0 .. 3 of the word: keys 2t, 2t+1; 2t+8, 2t+9
              half_pairs<FMT>(__byte_perm(vr[b][0][i], vr[b][1][i], 0x5140), u[0], u[1]);
              half_pairs<FMT>(__byte_perm(vr[b][0][i], vr[b][1][i], 0x7362), u[2], u[3]);
              half_pairs<FMT>(__byte_perm(vr[b][2][i], vr[b][3][i], 0x5140), w[0], w[1]);
              half_pairs<FMT>(__byte_perm(vr[b][2][i], vr[b][3][i], 0x7362), w[2], w[3]);
#pragma unroll
              for (int n = 0; n < NT; n++) {
                mma<BF>(acc[n][2 * i], u[0], u[1], w[0], w[1], pf[n][b][0], pf[n][b][1]);
                mma<BF>(acc[n][2 * i + 1], u[2], u[3], w[2], w[3], pf[n][b][0], pf[n][b][1]);
              }
            }
          }
        }
        if (it + 1 < nit) load_v(it + 1);
        there = there_next;
        full = full_next;
      }
      // the warp's O, in units of its maximum, and its sums to shared memory
#pragma unroll
      for (int n = 0; n < NT; n++)
#pragma unroll
        for (int c = 0; c < GC; c++) {
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], x);
          float f = 1.f;
          if constexpr (!BF) f = mo[n][c] == -INFINITY ? 1.f : exp2f(mo[n][c] - m[n][c] - OFF16);
          float *dst = sm + (warp * HEADS + n * 8 + 2 * lt + c) * (HD + 2);
#pragma unroll
          for (int i = 0; i < HD / 16; i++) {
            const int d = BF ? (VW == 2 ? lg * 4 + i * 2 : (i / 4 * 8 + lg) * 8 + (i & 3) * 2)
                             : lg * (HD / 8) + i * 2;
            dst[d] = acc[n][i][c] * f;
            dst[d + 1] = acc[n][i][2 + c] * f;
          }
          if (lg == 0) {
            dst[HD] = m[n][c];
            dst[HD + 1] = l[n][c];
          }
        }
      __syncthreads();
      finish<HD, HEADS>(sm, grp, r0, HD, whole, o + ((int64_t)s * H + g * grp) * HD,
                        lse ? lse + (int64_t)s * H + g * grp : nullptr,
                        part + (int64_t)(2 * blockIdx.x + (piece > 0)) * grp * (HD + 2));
      __syncthreads();
    }
  }
}

// Joins the parts of every cut pair, in order, AT outputs a block; a sequence
// of length 0 gets o = 0 and L = -inf.
template <typename T>
__global__ void __launch_bounds__(AT)
    k_join(const int *__restrict__ pre, const float *__restrict__ part, const Sched sc, int H,
           int hd, T *__restrict__ o, float *__restrict__ lse) {
  const int s = blockIdx.x / sc.Hkv, g = blockIdx.x % sc.Hkv, grp = H / sc.Hkv;
  const int i = blockIdx.y * AT + threadIdx.x;
  pk_wait();  // the parts and the prefix come from the kernel before
  if (i >= grp * hd) return;
  const int r = i / hd, e = i % hd;
  const int before = ld_int(pre + s), units = ld_int(pre + s + 1) - before;
  const int64_t W = (int64_t)ld_int(pre + sc.n_seq) * sc.Hkv;
  const int64_t w0 = (int64_t)before * sc.Hkv + (int64_t)g * units;
  if (units == 0) {
    o[((int64_t)s * H + g * grp) * hd + i] = from_f<T>(0.f);
    if (e == 0 && lse) lse[(int64_t)s * H + g * grp + r] = -INFINITY;
    return;
  }
  const int N = (int)min((int64_t)sc.N, W);
  const int b0 = block_of(W, w0, N), b1 = block_of(W, w0 + units - 1, N);
  if (b0 == b1) return;
  // the pair's part in its first block follows another pair's there, or
  // begins the block's range; in every later block it begins the range
  const int first = block_begin(W, b0, N) < w0 ? 1 : 0;
  const int64_t step = (int64_t)grp * (hd + 2);
  constexpr int U = 8;  // parts whose loads are in flight together
  float M = -INFINITY, L = 0.f, v = 0.f;
  for (int b = b0; b <= b1; b += U) {
    float pm[U], pl[U], pv[U], mn = M;
#pragma unroll
    for (int k = 0; k < U; k++) {
      const bool in = b + k <= b1;
      const float *rec = part + (2 * (in ? b + k : b0) + (b + k == b0 || !in ? first : 0)) * step +
                         r * (hd + 2);
      pm[k] = in ? ld_float(rec) : -INFINITY;
      pl[k] = ld_float(rec + 1);
      pv[k] = ld_float(rec + 2 + e);
    }
#pragma unroll
    for (int k = 0; k < U; k++) mn = fmaxf(mn, pm[k]);
    const float ref = mn == -INFINITY ? 0.f : mn, a = exp2f(M - ref);
    L *= a;
    v *= a;
#pragma unroll
    for (int k = 0; k < U; k++) {
      const float f = exp2f(pm[k] - ref);
      if (b + k <= b1) {
        L = fmaf(f, pl[k], L);
        v = fmaf(f, pv[k], v);
      }
    }
    M = mn;
  }
  o[((int64_t)s * H + g * grp) * hd + i] = from_f<T>(L == 0.f ? 0.f : v / L);
  if (e == 0 && lse) lse[(int64_t)s * H + g * grp + r] = (M + log2f(L)) * LN2;
}

template <typename T>
static void join(const PagedArgs &a, const Sched &sc, const int *pre, const float *part) {
  launch_dependent(k_join<T>,
                   dim3((unsigned)(a.n_seq * a.kv.Hkv), cdiv((int64_t)a.H / a.kv.Hkv * a.kv.hd, AT)),
                   dim3(AT), 0, a.s, pre, part, sc, a.H, a.kv.hd, (T *)a.o, a.lse);
  count_launch();
}
template <typename T, int FMT, int HD>
static bool attend(const PagedArgs &a, const Sched &sc, int *pre, float *part, bool vec) {
  const int grp = a.H / a.kv.Hkv, smem = 4 * (a.n_seq + 1);
  auto go = [&](auto kern) {
    if (!smem_optin((const void *)kern, 4 * (PG_MAX_SEQ + 1))) return false;
    kern<<<sc.N, AT, smem, a.s>>>(a.kv, (const T *)a.q, a.q_ld, a.lens, sc, a.H, (T *)a.o, a.lse,
                                  pre, part);
    count_launch();
    return true;
  };
  if (!(grp == 1 ? vec ? go(k_attend<T, FMT, HD, 1, true>) : go(k_attend<T, FMT, HD, 1, false>)
                 : vec ? go(k_attend<T, FMT, HD, 4, true>) : go(k_attend<T, FMT, HD, 4, false>)))
    return false;
  if (!sc.direct) {
    join<T>(a, sc, pre, part);
  }
  return true;
}
template <int FMT, int HD, int NT, int SB, int GC, bool BIG>
static bool attend_mma(const PagedArgs &a, Sched sc, int *pre, float *part) {
  using T = __nv_bfloat16;
  auto kern = k_attend_mma<FMT, HD, NT, SB, GC, BIG>;
  if (!smem_optin((const void *)kern, 4 * (PG_MAX_SEQ + 1))) return false;
  if (!sc.direct) sc.N = device_sms() * mma_blocks(HD, NT);
  kern<<<sc.N, AT, sc.direct ? 0 : 4 * (a.n_seq + 1), a.s>>>(
      a.kv, (const T *)a.q, a.q_ld, a.lens, sc, a.H, (T *)a.o, a.lse, pre, part);
  count_launch();
  if (!sc.direct) {
    join<T>(a, sc, pre, part);
  }
  return true;
}
template <int FMT, int HD, int SB>
static bool attend_mma_nt(const PagedArgs &a, const Sched &sc, int *pre, float *part) {
  const int grp = a.H / a.kv.Hkv;
  auto go = [&](auto big) {
    constexpr bool B = decltype(big)::value;
    return grp == 1   ? attend_mma<FMT, HD, 1, SB, 1, B>(a, sc, pre, part)
           : grp <= 8 ? attend_mma<FMT, HD, 1, SB, 2, B>(a, sc, pre, part)
                      : attend_mma<FMT, HD, 2, SB, 2, B>(a, sc, pre, part);
  };
  return a.kv.ps % (16 * SB) == 0 ? go(std::true_type()) : go(std::false_type());
}
template <int FMT>
static bool attend_mma_hd(const PagedArgs &a, const Sched &sc, int *pre, float *part) {
  switch (a.kv.hd) {
    case 32: return attend_mma_nt<FMT, 32, 4>(a, sc, pre, part);
    case 64: return attend_mma_nt<FMT, 64, 2>(a, sc, pre, part);
    default: return attend_mma_nt<FMT, 128, FMT == KV_BF16 ? 1 : 2>(a, sc, pre, part);
  }
}
// The tensor-core kernels: bfloat16 queries over a bfloat16 or 8-bit cache,
// head sizes 32, 64 and 128, pages of a multiple of 8 rows (8 consecutive
// positions lie in one page), 16-byte aligned, row numbers within 31 bits.
static bool mma_covers(const PagedArgs &a) {
  const KvView &kv = a.kv;
  return a.dt == DT_BF16 && kv.fmt != KV_F32 && (kv.hd == 32 || kv.hd == 64 || kv.hd == 128) &&
         kv.ps % 8 == 0 && !((uintptr_t)kv.pages & 15) &&
         kv.n_pages < ((int64_t)1 << 31) / (2 * (int64_t)kv.Hkv * kv.ps);
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

// Blocks of a call: the machine's worth of blocks, or one per pair where tables
// are short, which saves the prefix, the second kernel and the workspace (8
// heads, 2 kv heads of 64, bfloat16, lengths to the table's: 1 sequence of 512
// at most 4.9 us, split 8.0; of 1024, 10.1 and 7.4; 32 sequences of 1024, 10.4
// and 12.4, 128: 12.5 and 15.5; of 2048: 17.4 and 13.9, 24.4 and 20.9).
static Sched schedule(const KvView &kv, int n_seq) {
  Sched sc{n_seq, kv.Hkv, 0, 0};
  const int64_t pairs = (int64_t)n_seq * kv.Hkv;
  const int64_t cap = (int64_t)kv.table_pages * kv.ps;
  sc.direct = cap <= (pairs >= 64 ? 16 : 8) * PG_UNIT;
  sc.N = sc.direct ? (int)pairs : device_sms() * BLOCKS_SM;
  return sc;
}
static int64_t pre_bytes(int n_seq) { return (4 * ((int64_t)n_seq + 1) + 255) / 256 * 256; }

}  // namespace pg

namespace pg {
// A block for each 32 rows and RW_HEADS heads; where there are so many sequences
// that a block's look through their offsets costs as much as its rows, 8 blocks
// an SM with several times 32 rows each (2048 sequences, bfloat16 written: a
// block each 26 us, 8 an SM 33; 8192 sequences: 46 and 33).
constexpr int RW_SEQS = 4096;
static dim3 rw_grid(const KvView &kv, int64_t n_rows, bool many) {
  const unsigned x = cdiv(n_rows, RW_ROWS), y = cdiv(2 * kv.Hkv, RW_HEADS);
  const unsigned most = max(8 * device_sms() / y, 1u);
  return dim3(many && x > most ? most : x, y);
}
// Calls f with the element type, cache format, lanes of a head, vector access
// and MANY as constants.
template <typename F>
static void rw_dispatch(DType dt, int fmt, int hd, bool vec, bool many, F f) {
  const std::true_type yes;
  const std::false_type no;
  auto with = [&](auto t, auto m, auto l) {
    vec ? many ? f(t, m, l, yes, yes) : f(t, m, l, yes, no)
        : many ? f(t, m, l, no, yes) : f(t, m, l, no, no);
  };
  auto lanes = [&](auto t, auto m) {
    if (hd <= 8) with(t, m, std::integral_constant<int, 1>());
    else if (hd <= 16) with(t, m, std::integral_constant<int, 2>());
    else if (hd <= 32) with(t, m, std::integral_constant<int, 4>());
    else if (hd <= 64) with(t, m, std::integral_constant<int, 8>());
    else with(t, m, std::integral_constant<int, 16>());
  };
  auto format = [&](auto t) {
    switch (fmt) {
      case KV_F32: lanes(t, std::integral_constant<int, KV_F32>()); break;
      case KV_BF16: lanes(t, std::integral_constant<int, KV_BF16>()); break;
      case KV_E4M3: lanes(t, std::integral_constant<int, KV_E4M3>()); break;
      default: lanes(t, std::integral_constant<int, KV_INT8>());
    }
  };
  if (dt == DT_BF16) format(__nv_bfloat16());
  else format(float());
}
}  // namespace pg

void kv_write(const KvView &kv, const void *qkv, int64_t ld, DType dt, const int32_t *cu,
              const int32_t *start, int n_seq, int64_t n_rows, int H, cudaStream_t s) {
  using namespace pg;
  const bool vec = kv.hd % 8 == 0 && ld % 8 == 0 && !((uintptr_t)qkv & 15) &&
                   !((uintptr_t)kv.pages & 15);
  const bool many = n_seq > RW_SEQS;
  rw_dispatch(dt, kv.fmt, kv.hd, vec, many, [&](auto t, auto m, auto l, auto x, auto n) {
    using T = decltype(t);
    k_write<T, decltype(m)::value, decltype(l)::value, decltype(x)::value, decltype(n)::value>
        <<<rw_grid(kv, n_rows, many), RW_THREADS, 0, s>>>(kv, (const T *)qkv, ld, cu, start, n_seq,
                                                      n_rows, H);
  });
  count_launch();
}

void kv_read(const KvView &kv, const int32_t *cu, const int32_t *start, int n_seq, int64_t n_rows,
             void *k, void *v, DType dt, cudaStream_t s) {
  using namespace pg;
  const bool vec = kv.hd % 8 == 0 && !(((uintptr_t)k | (uintptr_t)v | (uintptr_t)kv.pages) & 15);
  const bool many = n_seq > RW_SEQS;
  rw_dispatch(dt, kv.fmt, kv.hd, vec, many, [&](auto t, auto m, auto l, auto x, auto n) {
    using T = decltype(t);
    k_read<T, decltype(m)::value, decltype(l)::value, decltype(x)::value, decltype(n)::value>
        <<<rw_grid(kv, n_rows, many), RW_THREADS, 0, s>>>(kv, cu, start, n_seq, n_rows, (T *)k,
                                                      (T *)v);
  });
  count_launch();
}

int64_t paged_ws_bytes(const KvView &kv, int n_seq, int H) {
  const pg::Sched sc = pg::schedule(kv, n_seq);
  if (sc.direct) return 0;
  return pg::pre_bytes(n_seq) + 4 * 2 * (int64_t)sc.N * (H / kv.Hkv) * (kv.hd + 2);
}

bool paged_attention(const PagedArgs &a) {
  using namespace pg;
  const Sched sc = schedule(a.kv, a.n_seq);
  int *pre = (int *)a.ws;
  float *part = (float *)((uint8_t *)a.ws + pre_bytes(a.n_seq));
  if (mma_covers(a)) {
    switch (a.kv.fmt) {
      case KV_BF16: return attend_mma_hd<KV_BF16>(a, sc, pre, part);
      case KV_E4M3: return attend_mma_hd<KV_E4M3>(a, sc, pre, part);
      default: return attend_mma_hd<KV_INT8>(a, sc, pre, part);
    }
  }
  const bool vec = a.kv.hd % 8 == 0 && !((uintptr_t)a.kv.pages & 15);
  return a.dt == DT_BF16 ? attend_fmt<__nv_bfloat16>(a, sc, pre, part, vec)
                         : attend_fmt<float>(a, sc, pre, part, vec);
}

}  // namespace llm
