// tcgen05 flash attention over packed sequences, forward (bf16 operands, fp32
// softmax and accumulators), for head sizes to 128 that are multiples of 8:
// the tiles are 64 or 128 columns wide and zero past the head's own
// (attn_tma.cuh).
//
// One CTA works on two 128-query tiles at once, streams A and B, each with
// items (query tile, head), key and value tiles of its own.  Per stream and
// key block of 128:
//   S = Q K_j^T         (M 128, N 128; operands K-major in shared memory)
//   P = 2^(S c - m)     softmax: 4 warps, a thread holds one row whole
//   O += P V_j          (M 128, N head size; A = P from TMEM, V MN-major)
// While one stream's threads wait for their products, the other's compute.
// The softmax bounds the kernel (1580 cycles a block and stream at 2 documents
// of 16384 rows, heads 64; the products take 512): the SFU gives 16
// exponentials a clock and SM, a block has 16384, of which NP of every 16
// pairs run as a polynomial on the FMA pipe (exp2_poly2; 0, 2, 6 and 8 of 16
// were 2 to 7% slower).  A row per thread needs no exchange between threads;
// its running maximum moves only when a block exceeds it by 2^8, and the
// thread then rescales its own row of O in TMEM.  Measured and dropped: two
// threads a row (16 softmax warps, 13% slower on long sequences), the streams
// taking turns at the exponentials (8%), weights formed on the old maximum
// while the block's own is found (17%).
// Items go to the streams from a queue, most work first (the plan clears its
// counter): dealt in a fixed snake the fullest CTA had 6% more at 24 sequences
// of 16001 rows in all; streams that share K and V (two heads of a kv head, or
// two blocks of a head) leave one idle where a sequence is short: 16 heads
// ragged 119 us against 115.
// Measured (heads of 64; 128): 2 documents of 16384 rows in all, 8 heads, 213
// us, 662 TFLOP/s; 2 x 8192 rows, 280 us, 982 TFLOP/s.
// P is rounded to bfloat16, V's type in the product (2^-8 of each term: out is off by
// 0.0020 where its own rounding makes 0.0016); a second term would add half again
// to the products.
// TMEM: S_A, S_B (128 columns each), O_A, O_B (head size each).  Heads to 64
// leave room for P beside S (SEP), so S_{j+1} is computed while block j's
// softmax runs; at head 128 P takes the first half of S's columns, and S_{j+1}
// follows O += P V_j.
// Warps: 0, 3 TMA producers of A and B; 1, 2 their MMA issuers (warp 1 also
// TMEM); 4-7 and 8-11 their softmax.  Every wait is bounded (FLAG_TIMEOUT).
// Rows of a tile past its sequence's end are another's: masked as keys, zeroed
// in V before they meet a zero weight, not stored.
#include "attn_tma.cuh"
#include "common.cuh"
#include "tcgen05.cuh"

namespace llm {
namespace attn_pk_tc {

using namespace tc;
using namespace attn_maps;

constexpr int SUB_BYTES = 128 * 64 * 2;  // 128 rows x 64 bf16, 128-byte swizzle
constexpr int NTHREADS = 384;
constexpr int SLOTS = 2;    // items handed out ahead
constexpr int READERS = 5;  // warps of a stream that take items from its producer
constexpr int TMEM_COLS = 512;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr float LAZY = 8.f;  // log2 units a row maximum may grow before O is rescaled
constexpr int NP = 4;        // polynomial pairs of every 16
constexpr int BAR_BYTES = 512;

template <int HD>
struct Cfg {
  static constexpr int SUB = HD / 64, TILE = SUB * SUB_BYTES;
  static constexpr bool SEP = HD == 64;
  static constexpr int QS = HD == 64 ? 2 : 1;   // Q slots of a stream
  static constexpr int KST = HD == 64 ? 2 : 1;  // K and V ring stages of a stream
  static constexpr int SMEM = (2 * QS + 4 * KST) * TILE + BAR_BYTES + 1024;
  // TMEM columns
  static constexpr int S(int x) { return 128 * x; }
  static constexpr int O(int x) { return 256 + HD * x; }
  static constexpr int P(int x) { return SEP ? 384 + 64 * x : 128 * x; }
};

// An item: query block q (of 128 rows) of a sequence, head h with kv head g, n
// key blocks.  t: the item's index and its tile (first row, length, block).
struct Work {
  int row0, T, q, h, g, n;
};
LLM_DEV Work work(int4 t, int H, int Hkv) {
  const int h = t.x % H;
  return Work{t.y, t.z, t.w, h, h / (H / Hkv), t.w + 1};
}

// Maxima that are NaN where an operand is.  exp2_poly2 takes a NaN for -126, so
// a score that is none has to reach the row through its maximum.
LLM_DEV float nmax(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
LLM_DEV float nmax3(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
template <int NPAIRS>
LLM_DEV float2 exp2_some(float2 x, int i) {
  return ((i & 15) * NPAIRS) % 16 < NPAIRS ? exp2_poly2(x) : make_float2(ex2(x.x), ex2(x.y));
}
// 32 scores to weights 2^(s sl2 - mr), packed; their sum is added to acc.
template <bool POLY>
LLM_DEV void weights(const float *sv, float sl2, float mr, uint32_t *w, float2 &acc) {
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    const float2 x = __ffma2_rn(make_float2(sv[i], sv[i + 1]), make_float2(sl2, sl2),
                                make_float2(-mr, -mr));
    const float2 p = POLY ? exp2_some<NP>(x, i / 2) : make_float2(ex2(x.x), ex2(x.y));
    acc = __fadd2_rn(acc, p);
    w[i / 2] = pack_bf16(p.x, p.y);
  }
}
LLM_DEV void tmem_st32u(uint32_t taddr, const uint32_t *w) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]),
      "r"(w[8]), "r"(w[9]), "r"(w[10]), "r"(w[11]), "r"(w[12]), "r"(w[13]), "r"(w[14]),
      "r"(w[15]), "r"(w[16]), "r"(w[17]), "r"(w[18]), "r"(w[19]), "r"(w[20]), "r"(w[21]),
      "r"(w[22]), "r"(w[23]), "r"(w[24]), "r"(w[25]), "r"(w[26]), "r"(w[27]), "r"(w[28]),
      "r"(w[29]), "r"(w[30]), "r"(w[31])
      : "memory");
}

template <int HD>
__global__ void __launch_bounds__(NTHREADS, 1)
    k_attn_fwd_streams(const __grid_constant__ CUtensorMap tm_qkv,
                    const __grid_constant__ CUtensorMap tm_o, float *__restrict__ lse, int H,
                    int Hkv, int hd, float scale, const PkView pk, int *gflag) {
  using C = Cfg<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  constexpr int RING = C::KST * C::TILE;  // bytes of a K or V ring
  uint8_t *sQ = smem, *sK = sQ + 2 * C::QS * C::TILE, *sV = sK + 2 * RING;
  uint64_t *bars = (uint64_t *)(sV + 2 * RING);
  uint32_t *tmem_sh = (uint32_t *)(bars + 48);
  volatile int *abort_sh = (volatile int *)(tmem_sh + 1);
  int4 *items = (int4 *)(bars + 50);  // [stream][SLOTS]
  const uint32_t b0 = smem_u32(bars);
  const uint32_t q_full = b0, q_empty = q_full + 16 * C::QS,  // [stream][slot]
                 s_full = q_empty + 16 * C::QS, s_free = s_full + 16, p_full = s_free + 16,
                 o_done = p_full + 16, drain = o_done + 16,  // [stream] each
                 rings = drain + 16;                         // then each stream's ring
  constexpr int RING_BARS = 4 * C::KST + 2 * SLOTS;
  static_assert(4 * C::QS + 10 + 2 * RING_BARS <= 48 &&
                    400 + 16 * 2 * SLOTS <= BAR_BYTES,
                "barriers overlap the TMEM address word or the items");
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    *abort_sh = 0;
    for (int i = 0; i < 2 * C::QS; i++) {
      mbar_init(q_full + 8 * i, 1);
      mbar_init(q_empty + 8 * i, 1 + 4);  // the last S product; each warp's part of O stored
    }
    for (int i = 0; i < 2; i++) {
      const uint32_t k_full = rings + 8 * RING_BARS * i, k_empty = k_full + 8 * C::KST,
                     v_full = k_empty + 8 * C::KST, v_empty = v_full + 8 * C::KST,
                     i_full = v_empty + 8 * C::KST, i_empty = i_full + 8 * SLOTS;
      for (int s = 0; s < C::KST; s++) {
        mbar_init(k_full + 8 * s, 1);
        mbar_init(k_empty + 8 * s, 1);
        mbar_init(v_full + 8 * s, 1);
        mbar_init(v_empty + 8 * s, 1);
      }
      for (int s = 0; s < SLOTS; s++) {
        mbar_init(i_full + 8 * s, 1);
        mbar_init(i_empty + 8 * s, READERS);
      }
    }
    for (int x = 0; x < 2; x++) {
      mbar_init(s_full + 8 * x, 1);
      mbar_init(s_free + 8 * x, 4);
      mbar_init(p_full + 8 * x, 4);
      mbar_init(o_done + 8 * x, 1);
      mbar_init(drain + 8 * x, 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_sh)),
                 "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_sh;
  if (pk.tiles) pk_wait();  // the plan comes from the kernel before
  // this warp's stream: its ring's barriers, K, V, items
  const int x = warp < 2 ? 0 : warp < 4 ? 1 : (warp - 4) >> 2;
  const uint32_t k_full = rings + 8 * RING_BARS * x, k_empty = k_full + 8 * C::KST,
                 v_full = k_empty + 8 * C::KST, v_empty = v_full + 8 * C::KST,
                 i_full = v_empty + 8 * C::KST, i_empty = i_full + 8 * SLOTS;
  sK += x * RING;
  sV += x * RING;
  items += x * SLOTS;
  // The it-th item of this warp's stream, from the producer; t.x < 0: no more (or a wait
  // gave up).  Whole warps; each takes every item once.
  auto take = [&](int it) {
    int4 t = make_int4(-1, 0, 0, 0);
    const int sl = it % SLOTS;
    if (warp_wait(i_full + 8 * sl, (it / SLOTS) & 1, abort_sh, gflag)) {
      t = items[sl];
      __syncwarp();
      if (lane == 0) mbar_arrive(i_empty + 8 * sl);
    }
    return t;
  };

  if (warp == 0 || warp == 3) {
    int4 only = make_int4(0, 0, 0, 0);
    if (!pk.tiles)
      only = pk_find(pk.cu, pk.n_seq, (int)pk.n_rows, PK_BLOCK, blockIdx.x / H, gflag);
    if (lane == 0) {
      // ------------------------------------------------------ TMA producer
      int gb = 0, nq = 0;  // key blocks, Q tiles issued
      bool ok = true;
      const int n_items = pk.tiles ? ld_int(pk.n_tiles) * H : only.w ? gridDim.x : 0;
      // (no plan: one item a block, the first stream's)
      int item = x * gridDim.x + blockIdx.x;
      for (int it = 0;; it++) {
        int4 t = make_int4(-1, 0, 0, 0);
        if (item < n_items) {
          const int4 u = pk.tiles ? ld_int4(pk.tiles + item / H) : only;
          t = make_int4(item, u.x, u.y, u.z);
        }
        const int is = it % SLOTS;
        if (!mbar_wait(i_empty + 8 * is, ((it / SLOTS) & 1) ^ 1, abort_sh, gflag)) break;
        items[is] = t;
        mbar_arrive(i_full + 8 * is);
        if (t.x < 0) break;
        // the next item, from the queue, while this one's tiles are loaded
        item = pk.tiles ? 2 * gridDim.x + atomicAdd(pk.n_tiles + 2, 1) : n_items;
        const Work w = work(t, H, Hkv);
        const int sl = nq % C::QS;
        const uint32_t qb = 8 * (x * C::QS + sl);
        if (!mbar_wait(q_empty + qb, ((nq / C::QS) & 1) ^ 1, abort_sh, gflag)) break;
        mbar_arrive_expect_tx(q_full + qb, C::TILE);
        for (int c = 0; c < C::SUB; c++)
          tma_load_3d(smem_u32(sQ + (x * C::QS + sl) * C::TILE + c * SUB_BYTES), &tm_qkv, 64 * c, w.h,
                      w.row0 + w.q * 128, q_full + qb);
        nq++;
        for (int j = 0; j < w.n && ok; j++, gb++) {
          const int s = gb % C::KST;
          const uint32_t ph = ((gb / C::KST) & 1) ^ 1;
          if (!mbar_wait(k_empty + 8 * s, ph, abort_sh, gflag)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(k_full + 8 * s, C::TILE);
          for (int c = 0; c < C::SUB; c++)
            tma_load_3d(smem_u32(sK + s * C::TILE + c * SUB_BYTES), &tm_qkv, 64 * c, H + w.g,
                        w.row0 + j * 128, k_full + 8 * s);
          if (!mbar_wait(v_empty + 8 * s, ph, abort_sh, gflag)) {
            ok = false;
            drain_wait(k_full + 8 * s, ph ^ 1);
            break;
          }
          mbar_arrive_expect_tx(v_full + 8 * s, C::TILE);
          for (int c = 0; c < C::SUB; c++)
            tma_load_3d(smem_u32(sV + s * C::TILE + c * SUB_BYTES), &tm_qkv, 64 * c, H + Hkv + w.g,
                        w.row0 + j * 128, v_full + 8 * s);
        }
        if (!ok) break;
      }
      // every copy this thread issued has landed before the CTA may exit
      for (int i = max(0, nq - C::QS); i < nq; i++)
        drain_wait(q_full + 8 * (x * C::QS + i % C::QS), (i / C::QS) & 1);
      for (int i = max(0, gb - C::KST); i < gb; i++) {
        drain_wait(k_full + 8 * (i % C::KST), (i / C::KST) & 1);
        drain_wait(v_full + 8 * (i % C::KST), (i / C::KST) & 1);
      }
    }
  } else if (warp == 1 || warp == 2) {
    // ------------------------------------- MMA issuer of the stream (whole warp)
    constexpr uint32_t ID_S = idesc_mn(128, 128, false, false);
    constexpr uint32_t ID_O = idesc_mn(128, HD, false, true);
    int gb = 0, nq = 0, cb = 0;  // the item's first ring block; Q tiles, blocks of the stream
    bool ok = true;
    auto wait = [&](uint32_t bar, int n) {  // the n-th phase of a barrier (n from 0)
      ok = ok && warp_wait(bar, n & 1, abort_sh, gflag);
      return ok;
    };
    for (int it = 0; ok; it++) {
      const int4 t = take(it);
      if (t.x < 0) break;
      const Work w = work(t, H, Hkv);
      const int n = w.n;
      const uint32_t qb = 8 * (x * C::QS + nq % C::QS);
      const uint64_t qd = sdesc(smem_u32(sQ + (x * C::QS + nq % C::QS) * C::TILE), 16, 1024);
      auto scores = [&](int j) {  // S = Q K_j^T
        const int s = (gb + j) % C::KST;
        if (!wait(k_full + 8 * s, (gb + j) / C::KST)) return;
        fence_after();
        const uint64_t kd = sdesc(smem_u32(sK + s * C::TILE), 16, 1024);
#pragma unroll
        for (int kk = 0; kk < HD / 16; kk++) {
          const uint64_t at = (uint64_t)((kk / 4) * (SUB_BYTES >> 4) + (kk % 4) * 2);
          mma_bf16_e(tmem + C::S(x), qd + at, kd + at, ID_S, kk > 0 ? 1u : 0u);
        }
        mma_commit_e(s_full + 8 * x);
        mma_commit_e(k_empty + 8 * s);
        if (j == n - 1) mma_commit_e(q_empty + qb);
      };
      if (!wait(q_full + qb, nq / C::QS)) break;
      // the buffer of the stream's previous block was read (P V done: P is in it)
      if (cb > 0 && !wait((C::SEP ? s_free : o_done) + 8 * x, cb - 1)) break;
      scores(0);
      for (int j = 0; j < n && ok; j++, cb++) {
        const int s = (gb + j) % C::KST;
        if (C::SEP && j + 1 < n) {
          if (!wait(s_free + 8 * x, cb)) break;
          scores(j + 1);
        }
        if (!wait(v_full + 8 * s, (gb + j) / C::KST) || !wait(p_full + 8 * x, cb)) break;
        fence_after();
        const uint64_t vd = sdesc(smem_u32(sV + s * C::TILE), SUB_BYTES, 1024);
#pragma unroll
        for (int kk = 0; kk < 8; kk++)
          mma_ts_e(tmem + C::O(x), tmem + C::P(x) + kk * 8, vd + (uint64_t)(kk * 128), ID_O,
                   (j > 0 || kk > 0) ? 1u : 0u);
        mma_commit_e(o_done + 8 * x);
        mma_commit_e(v_empty + 8 * s);
        if (!C::SEP && j + 1 < n) {
          if (!wait(o_done + 8 * x, cb)) break;
          scores(j + 1);
        }
      }
      nq++;
      gb += n;
    }
    mma_commit_e(drain + 8 * x);
    if (lane == 0) drain_wait(drain + 8 * x, 0);
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax
    const int quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_off + C::S(x), tP = tmem + lane_off + C::P(x),
                   tO = tmem + lane_off + C::O(x);
    const float sl2 = scale * LOG2E;
    int gb = 0, nq = 0, cb = 0, st_slot = -1;  // slot whose O store is still to be released
    bool ok = true;
    for (int it = 0; ok; it++) {
      const int4 t = take(it);
      if (t.x < 0) break;
      const Work w = work(t, H, Hkv);
      const int n = w.n, q0 = w.q * 128, T = w.T;
      float m = -INFINITY;
      float2 l2 = make_float2(0.f, 0.f);
      for (int j = 0; j < n; j++, cb++) {
        if (!(ok = warp_wait(s_full + 8 * x, cb & 1, abort_sh, gflag))) break;
        fence_after();
        float sv[128];
        {
          uint32_t u[4][32];
#pragma unroll
          for (int c = 0; c < 4; c++) tmem_ld_raw<32>(tS + 32 * c, u[c]);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 4; c++) {
            tmem_after_wait(u[c]);
#pragma unroll
            for (int i = 0; i < 32; i++) sv[32 * c + i] = __uint_as_float(u[c][i]);
          }
        }
        if constexpr (C::SEP) {  // the next block's scores may overwrite S
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(s_free + 8 * x);
        }
        const bool diag = j == n - 1;  // the row's own block: mask, and the sequence's end
        if (diag) {
          const int last = min(row, T - 1 - q0);  // keys up to the row itself
#pragma unroll
          for (int i = 0; i < 128; i++)
            if (i > last) sv[i] = -INFINITY;
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 128; i += 2) mx[(i >> 1) & 3] = nmax3(mx[(i >> 1) & 3], sv[i], sv[i + 1]);
        const float top = nmax(nmax(mx[0], mx[1]), nmax(mx[2], mx[3])) * sl2;
        // true on the first block with a key, and from a NaN on: it stays in m, l and O
        const bool need = !(top <= m + LAZY);
        if (j > 0 && __any_sync(0xffffffffu, need)) {
          // O is rescaled after the product of the block before
          if (!(ok = warp_wait(o_done + 8 * x, (cb - 1) & 1, abort_sh, gflag))) break;
          fence_after();
          const float corr = need ? ex2(m - top) : 1.f;
#pragma unroll 1
          for (int c = 0; c < HD; c += 16) {
            float v[16];
            uint32_t u[16];
            tmem_ld16(tO + c, v);
#pragma unroll
            for (int i = 0; i < 16; i++) u[i] = __float_as_uint(v[i] * corr);
            tmem_st16(tO + c, u);
          }
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        }
        if (need) {
          const float corr = m == -INFINITY ? 0.f : ex2(m - top);
          l2.x *= corr;
          l2.y *= corr;
          m = top;
        }
        const float mr = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int c = 0; c < 2; c++) {
          uint32_t pw[32];
          if (diag) {  // on the SFU alone: masked scores give exact zeros
#pragma unroll
            for (int d = 0; d < 2; d++) {
              if (2 * c + d <= quarter) {
                weights<false>(sv + 64 * c + 32 * d, sl2, mr, pw + 16 * d, l2);
              } else {
#pragma unroll
                for (int i = 0; i < 16; i++) pw[16 * d + i] = 0;
              }
            }
          } else {
            weights<true>(sv + 64 * c, sl2, mr, pw, l2);
            weights<true>(sv + 64 * c + 32, sl2, mr, pw + 16, l2);
          }
          if (C::SEP && c == 0 && cb > 0) {  // P is free once the product before has read it
            if (!(ok = warp_wait(o_done + 8 * x, (cb - 1) & 1, abort_sh, gflag))) break;
            fence_after();
          }
          tmem_st32u(tP + 32 * c, pw);
        }
        if (!ok) break;
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        if (diag && q0 + 128 > T) {  // V rows past the sequence's end must be numbers
          const int s = (gb + j) % C::KST;
          if (!(ok = warp_wait(v_full + 8 * s, ((gb + j) / C::KST) & 1, abort_sh, gflag))) break;
          if (q0 + row >= T) {
#pragma unroll
            for (int c = 0; c < C::SUB; c++) {
              uint4 *p = reinterpret_cast<uint4 *>(sV + s * C::TILE + c * SUB_BYTES + row * 128);
#pragma unroll
              for (int i = 0; i < 8; i++) p[i] = make_uint4(0, 0, 0, 0);
            }
          }
          fence_proxy_async();
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + 8 * x);
        if (st_slot >= 0) {  // the store of the item before has long read its tile
          if (lane == 0) {
            bulk_wait_read();
            mbar_arrive(q_empty + 8 * (x * C::QS + st_slot));
          }
          st_slot = -1;
        }
      }
      if (!ok) break;
      gb += n;
      // O = O / l: through the item's Q tile (its last S product is complete)
      // in the 128-byte-swizzle image of the store's boxes
      if (!(ok = warp_wait(o_done + 8 * x, (cb - 1) & 1, abort_sh, gflag))) break;
      fence_after();
      // a maximum that is not finite has no weights to it (an infinite one leaves
      // the polynomial's pairs finite): NaN, where finite ones add 0
      const float l = l2.x + l2.y, none = m - m, inv = 1.f / l + none;
      const int sl = nq % C::QS;
      uint8_t *tile = sQ + (x * C::QS + sl) * C::TILE;
#pragma unroll
      for (int c = 0; c < HD / 32; c++) {
        uint32_t u[32];
        tmem_ld_raw<32>(tO + 32 * c, u);
        tmem_wait_ld();
        tmem_after_wait(u);
        uint8_t *dst = tile + (c / 2) * SUB_BYTES + row * 128;
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const int ch = (c & 1) * 4 + i;
          uint32_t pw[4];
#pragma unroll
          for (int e = 0; e < 4; e++)
            pw[e] = pack_bf16(__uint_as_float(u[8 * i + 2 * e]) * inv,
                              __uint_as_float(u[8 * i + 2 * e + 1]) * inv);
          *reinterpret_cast<uint4 *>(dst + ((ch ^ (row & 7)) << 4)) =
              make_uint4(pw[0], pw[1], pw[2], pw[3]);
        }
      }
      fence_before();
      fence_proxy_async();
      __syncwarp();
      const int r0 = quarter * 32;  // the warp's rows: whole, or cut by the sequence's end
      if (q0 + r0 + 32 <= T) {
        if (lane == 0) {
          for (int c = 0; c < C::SUB; c++)
            tma_store_4d(&tm_o, smem_u32(tile + c * SUB_BYTES + r0 * 128), 64 * c, w.h,
                         w.row0 + q0 + r0, 0);
          bulk_commit();
        }
      } else {
        for (int rr = r0; rr < r0 + 32; rr += 8)
          for (int c = 0; c < C::SUB; c++)
            store_cut(tile + c * SUB_BYTES, rr, T - q0,
                      pk.out + (int64_t)(w.row0 + q0 + rr) * pk.out_ld + w.h * hd + 64 * c,
                      pk.out_ld, hd - 64 * c, lane);
      }
      if (q0 + row < T)
        lse[w.h * pk.n_rows + w.row0 + q0 + row] = (m + __log2f(l) + (m > 0.f ? none : 0.f)) * LN2;
      __syncwarp();
      if (C::QS > 1) {
        st_slot = sl;  // released after the next item's first block
      } else if (lane == 0) {  // the one slot is waited for
        bulk_wait_read();
        mbar_arrive(q_empty + 8 * (x * C::QS + sl));
      }
      nq++;
    }
    if (lane == 0) bulk_wait_all();
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 1) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(TMEM_COLS)
                 : "memory");
  }
}

template <int HD>
static bool launch(const PkArgs &a, const PkPlan &p, void *o, float *lse, int *flag) {
  auto kern = k_attn_fwd_streams<HD>;
  if (!smem_optin((const void *)kern, Cfg<HD>::SMEM)) return false;
  const int64_t dw = (int64_t)a.H * a.hd;
  CUtensorMap map, mo;
  if (!head_map_load(&map, a.qkv, a.hd, a.H + 2 * a.Hkv, a.n_rows, a.ld, 128) ||
      !head_map_store(&mo, o, a.hd, a.H, a.n_rows, 1, dw, 32))
    return false;
  const int64_t items = p.cap * a.H;
  // one item a block at most: no order to plan (300 rows, 8 heads: 11.3 us with
  // the plan's kernel, 9.7 without)
  const bool plan = items > device_sms() || a.n_seq > PK_FIND_SEQ;
  const PkView pk{p.n_tiles, plan ? p.tiles : nullptr, a.n_rows, (__nv_bfloat16 *)o, dw, a.cu,
                  a.n_seq, nullptr, 0};
  const dim3 grid((unsigned)(items < device_sms() ? items : device_sms()));
  if (plan) {
    packed_plan(a, p);
    launch_dependent(kern, grid, dim3(NTHREADS), Cfg<HD>::SMEM, a.s, map, mo, lse, a.H, a.Hkv, a.hd,
                     1.0f / sqrtf((float)a.hd), pk, flag);
  } else {
    kern<<<grid, NTHREADS, Cfg<HD>::SMEM, a.s>>>(map, mo, lse, a.H, a.Hkv, a.hd,
                                                 1.0f / sqrtf((float)a.hd), pk, flag);
  }
  count_launch();
  return true;
}

}  // namespace attn_pk_tc

bool packed_fwd_tc(const PkArgs &a, const PkPlan &p, void *o, float *lse, int *flag) {
  using namespace attn_pk_tc;
  if (a.dt != DT_BF16 || a.hd % 8) return false;
  return a.hd > 64 ? launch<128>(a, p, o, lse, flag) : launch<64>(a, p, o, lse, flag);
}

}  // namespace llm
