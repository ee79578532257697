// Attention of many query rows over the 4-bit cache (chunks of a prompt, many
// drafted tokens, large groups), bound by the matrix cores and the
// exponentials: 4 D multiply-adds and one exponential for each pair of a row
// and a key it sees.
//
// A workgroup of 8 waves takes 256 query rows (tokens times query heads) of
// one cache head, 32 rows a wave, and walks over the keys in tiles of KT
// tokens.  Each tile is dequantized once for all 256 rows, T[code] * a in fp32
// rounded to fp16, into one of two LDS buffers while the other is multiplied;
// one barrier a tile.
//  * Scores S^T = K Q^T and outputs O^T = V^T P^T with v_mfma_f32_32x32x16_f16.
//    A lane holds scores of one row, tokens 8 a + 4 h + b of 32 (h = lane / 32);
//    the values are stored in LDS in the order in which a lane has its weights,
//    so weights go from the first product to the second in registers, and
//    running maxima, sums and rescaling are of the lane's own row.
//  * Key and value scales are multiplied into the tiles, so no score needs
//    more than the exponential's own multiply-add.  A tile's keys are taken by
//    a power of two of their own to the top of fp16's range (their largest
//    scale becomes 2^14 .. 2^15), the values by a running one, weights by 2^14.
//    That power is shared by all tokens of the tile (of the tiles so far), seen
//    or not, so keys and values down to 2^-28 of the largest keep all of fp16's
//    bits, smaller ones lose them, and below 2^-39 nothing is left.
//  * bf16: one fp16 term each.  For the values T a that must not mean nearest
//    rounding: there are few distinct scales and 16 codes, so its errors have a
//    mean, which adds up over the keys while the values themselves cancel (normal
//    rows under equal weights: 7e-4 of the result at 2500 keys, 3e-3 at 34000,
//    5.5e-3 at 131072, where bf16 rounds by 1.7e-3).  They are rounded up or down
//    by a threshold that goes through the 16 sixteenths of a last place with the
//    token (dithered_pair): no mean, 2.7e-4 at each of these lengths.  fp16 (TWO):
//    keys, values and weights keep what fp16 leaves of them in second planes,
//    since the result would show it.
// Neighbouring workgroups take neighbouring cache heads, which puts a head's
// workgroups on one of the eight dies and its keys in that die's L2 cache; the
// rows that see most keys go first, over all sequences (three prompts 302 us
// sequence by sequence, 268 so).  Where there are few workgroups the keys are
// divided among several (splits), joined by prompt_join_kernel.
//
// Measured (64 query heads over 8 of 128, NF4 blocks of 128, bf16): 2048 tokens
// over 32768, 2.27e12 operations, 2.78 ms a call, 816 TFLOP/s of the 1194 that a
// large bf16 product reaches here; the vector unit (exponentials, conversions,
// dequantization) is active 56 % of the time and the matrix cores 34 %, and
// what the two do not overlap is the distance.  Three prompts of up to 2555
// tokens (7105 in all) with 32 query heads: 233 us a call, 596 TFLOP/s, less because the
// triangle's short rows leave units idle at the end.  The same in fp16, whose
// second planes make five products of two: 5.75 ms and 413 us.
// A sequence of few rows among prompts has its keys walked by one workgroup a
// head, whose other waves wait: a prompt of 512 tokens with 63 single tokens over
// 8000 each takes 493 us, the two in calls of their own 34 and 134 us.
#include <algorithm>

#include "qmv_attention_mfma.hpp"

namespace qmv {

constexpr int kPWaves = 8;
constexpr int kPThreads = 64 * kPWaves;
constexpr int kPRows = 32 * kPWaves;

struct PromptArgs {
  AttnArgs a;
  Partials part;
  int mtiles, splits;
};

// Tokens of a tile, so that two buffers of it and the table fit in LDS.
__host__ __device__ constexpr int prompt_tile(int D, bool two) { return D <= (two ? 96 : 128) ? 64 : 32; }
// Copies of the code table (float pairs).
__host__ __device__ constexpr int prompt_copies(int D, bool two) { return two && D > 128 ? 4 : 16; }

// lo and hi of tokens 2 j and 2 j + 1 of a group of 16 as an fp16 pair, a
// magnitude rounded up where what lies below its last fp16 place is at least 1
// minus the token's threshold of that place.  Thresholds (2 k + 1) / 32 with k
// the token's bits reversed: every sixteenth once, neighbours far apart.
constexpr uint32_t dither(int token) {
  const int k = (token & 1) << 3 | (token & 2) << 1 | (token & 4) >> 1 | (token & 8) >> 3;
  return (uint32_t)(2 * k + 1) << 8;  // fp16 drops 13 of fp32's bits
}
__device__ __forceinline__ uint32_t dithered_pair(float lo, float hi, int j) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(__uint_as_float(__float_as_uint(lo) + dither(2 * j)),
                                                                __uint_as_float(__float_as_uint(hi) + dither(2 * j + 1))));
}

template <int D, int DT, bool TWO>
__global__ __launch_bounds__(kPThreads, 2) void attention_prompt_kernel(PromptArgs pa) {
  constexpr int KT = prompt_tile(D, TWO);
  constexpr int COPIES = prompt_copies(D, TWO);
  constexpr int NU = KT * D / 32;        // 16-byte units of the keys of a tile, and of its values
  static_assert(2 * NU <= kPThreads && NU % 64 == 0, "one unit a thread, a role a wave");
  constexpr int KS = 2 * D + 16;         // row strides in bytes: 16 more keep rows off each other's banks
  constexpr int VS = 2 * KT + 16;
  constexpr int PL = TWO ? 2 : 1;
  constexpr int QS = D / 16, DTI = D / 32, TT = KT / 32;
  __shared__ __align__(16) uint8_t kbuf[2][PL][KT * KS];
  __shared__ __align__(16) uint8_t vbuf[2][PL][D * VS];
  __shared__ __align__(16) float2 lut[256 * COPIES];  // packed byte -> (T[byte >> 4], T[byte & 15])
  __shared__ __align__(16) uint32_t kmax[2][4], vmax[2][4];  // by wave of the role
  __shared__ __align__(4) uint8_t there[3][4];  // whether 16 tokens have a page: written two tiles ahead
  const AttnArgs &a = pa.a;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int heads = a.c.heads;
  const int h = (int)(blockIdx.x % (unsigned)heads);
  const unsigned rest = blockIdx.x / (unsigned)heads;
  const int b = (int)(rest % (unsigned)a.kb.batch);
  const int rest2 = (int)(rest / (unsigned)a.kb.batch);  // tiles of rows from the last on, then splits
  const int split = rest2 % pa.splits, mt = pa.mtiles - 1 - rest2 / pa.splits;
  const SeqRange s = seq_range(a.kb, b);
  const int n = s.n < a.kb.max_q ? s.n : a.kb.max_q;
  const int64_t rows = (int64_t)n * a.group;
  const int64_t m0 = (int64_t)mt * kPRows;
  if (m0 >= rows) return;
  {
    const uint32_t *tb = table_bits(a.qt);
    for (int i = tid; i < 256 * COPIES; i += kPThreads)
      lut[i] = make_float2(__uint_as_float(tb[i / COPIES >> 4]), __uint_as_float(tb[i / COPIES & 15]));
  }

  if (tid < 8) {  // roles of fewer than four waves
    kmax[tid >> 2][tid & 3] = 0u;
    vmax[tid >> 2][tid & 3] = 0u;
  }
  __syncthreads();

  // keys [lo, hi) of the workgroup's rows; tiles [t, t_to) of them
  int lo, hi, unused;
  const int last_row = (int)((rows - m0 < kPRows ? rows - m0 : kPRows) - 1);
  key_range(a, s, (int)(m0 / a.group), lo, unused);
  key_range(a, s, (int)((m0 + last_row) / a.group), unused, hi);
  lo &= ~15;
  const int tiles = hi > lo ? (hi - lo + KT - 1) / KT : 0;
  const int t_from = (int)((int64_t)tiles * split / pa.splits);
  const int t_to = (int)((int64_t)tiles * (split + 1) / pa.splits);

  // this lane's row and the keys it sees; the wave's rows all see [all_lo, all_hi)
  const int half = lane >> 5;
  const int rw = 32 * wave;
  const bool real = rw + (lane & 31) <= last_row;
  const bool busy = rw <= last_row;
  const int64_t m = m0 + (real ? rw + (lane & 31) : 0);
  const int i_row = (int)(m / a.group);
  const int h_row = h * a.group + (int)(m % a.group);
  int row_lo, row_hi, all_lo, all_hi, any_hi;
  key_range(a, s, i_row, row_lo, row_hi);
  if (!real) row_lo = row_hi = 0;
  key_range(a, s, (int)((m0 + rw) / a.group), unused, all_hi);
  key_range(a, s, (int)((m0 + (rw + 31 < last_row ? rw + 31 : last_row)) / a.group), all_lo, any_hi);

  // ---- queries in fp16, scaled by a power of two of their own ----
  f16x8_t qf[QS];
  float qscale;
  {
    const uint16_t *qrow = static_cast<const uint16_t *>(a.q.p) + (s.row0 + i_row) * a.q.ts + h_row * a.q.hs;
    uint4 raw[QS];
    float big = 0.f;
#pragma unroll
    for (int c = 0; c < QS; ++c) {
      raw[c] = *reinterpret_cast<const uint4 *>(qrow + 16 * c + 8 * half);
      float x[8];
      scales8<DT>(raw[c], x);
#pragma unroll
      for (int j = 0; j < 8; ++j) big = fmaxf(big, fabsf(x[j]));
    }
    uint32_t u = __float_as_uint(big), v = u;
    swap32(u, v);
    big = fmaxf(__uint_as_float(u), __uint_as_float(v));
    int e = exponent_of(big);
    e = e < -110 ? -110 : (e > 110 ? 110 : e);
    const float sign = a.scale < 0.f ? -1.f : 1.f;
#pragma unroll
    for (int c = 0; c < QS; ++c) {
      float x[8];
      scales8<DT>(raw[c], x);
      u32x4_t w;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = f16_pair(sign * ldexpf(x[2 * j], -e), sign * ldexpf(x[2 * j + 1], -e));
      qf[c] = __builtin_bit_cast(f16x8_t, w);
    }
    qscale = ldexpf(fabsf(a.scale) * 1.44269504088896340736f, e);
  }

  // ---- this thread's unit of every tile ----
  const bool isk = tid < NU, isv = !isk && tid < 2 * NU;
  const int u = isk ? tid : (isv ? tid - NU : 0);
  // keys: token u / (D / 32), chunk of 32 elements; values: 16 tokens, a pair of elements
  const int ktok = u / (D / 32), kch = u % (D / 32), vgrp = u / (D / 2), vpair = u % (D / 2);
  const int my_tok = isk ? ktok : 16 * vgrp;
  const int block = isk ? 32 * kch / a.c.bs : 2 * vpair / a.c.bs;
  const int ps = 1 << a.c.log2page;
  const uint32_t page_codes = (uint32_t)(heads << a.c.log2page) * (D / 2);
  const uint32_t page_scales = (uint32_t)(heads << a.c.log2page) * (uint32_t)(2 * (D / a.c.bs));
  const uint8_t *codes = (isk ? a.c.kc : a.c.vc) + (int64_t)(h << a.c.log2page) * (D / 2) +
                         (isk ? 16 * kch : 16 * vpair);
  const char *scales = reinterpret_cast<const char *>(isk ? a.c.ks : a.c.vs) +
                       (int64_t)(h << a.c.log2page) * (2 * (D / a.c.bs)) + ((int64_t)block << (a.c.log2page + 1));
  const int32_t *bt = a.kb.bt + (int64_t)b * a.kb.bt_stride;
  auto page_entry = [&](int t) {  // loaded unconditionally, judged where it is used
    const int i = (lo + t * KT + my_tok) >> a.c.log2page;
    return bt[i < a.kb.max_pages ? i : a.kb.max_pages - 1];
  };
  uint4 raw, s0, s1;
  bool page_ok;
  auto load_raw = [&](int t, int entry) {
    const int tok = lo + t * KT + my_tok;
    page_ok = tok < hi && (tok >> a.c.log2page) < a.kb.max_pages && entry >= 0 && entry < a.c.num_pages;
    const uint32_t page = page_ok ? entry : 0;
    const int at = tok & (ps - 1);
    raw = *reinterpret_cast<const uint4 *>(codes + (uint64_t)page * page_codes + at * (D / 2));
    const char *sp = scales + (uint64_t)page * page_scales + 2 * at;
    if (isk) {
      s0.x = *reinterpret_cast<const uint16_t *>(sp);
    } else {
      s0 = reinterpret_cast<const uint4 *>(sp)[0];
      s1 = reinterpret_cast<const uint4 *>(sp)[1];
    }
  };
  // scales of tokens that no row sees (which may hold anything) become 0; the
  // largest of the wave's is told to the others.  One that is not finite counts
  // for nothing there: it is the business of the rows that see it, and taking
  // the tile down by its exponent would leave zeros of all else.
  constexpr uint32_t kInf16 = DT == kF16 ? 0x7c00u : 0x7f80u;
  auto publish = [&](int t, int buf, int slot) {
    const int tok = lo + t * KT + my_tok;
    uint32_t big = 0;
    if (isk) {
      s0.x = page_ok ? s0.x & 0xffffu : 0u;
      big = s0.x < kInf16 ? s0.x : 0u;
      if (kch == 0 && (ktok & 15) == 0) there[slot][ktok >> 4] = page_ok;
    } else if (isv) {
      uint32_t w[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool k0 = page_ok && tok + 2 * j < hi, k1 = page_ok && tok + 2 * j + 1 < hi;
        w[j] &= (k0 ? 0x0000ffffu : 0u) | (k1 ? 0xffff0000u : 0u);
        big = max(big, max(w[j] & 0xffffu, w[j] >> 16));
      }
      s0 = make_uint4(w[0], w[1], w[2], w[3]);
      s1 = make_uint4(w[4], w[5], w[6], w[7]);
    }
    big = (uint32_t)wave_max_i32((int)big);
    if (big >= kInf16) {  // values: not looked at one by one above
      big = 0;
      const uint32_t w[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t a = w[j] & 0xffffu, b = w[j] >> 16;
        big = max(big, max(a < kInf16 ? a : 0u, b < kInf16 ? b : 0u));
      }
      big = (uint32_t)wave_max_i32((int)big);
    }
    if (lane == 0 && isk) kmax[buf][wave] = big;
    if (lane == 0 && isv) vmax[buf][wave - NU / 64] = big;
  };
  auto exponent16 = [&](const uint32_t (&x)[4]) {
    const uint4 w = *reinterpret_cast<const uint4 *>(x);
    const uint32_t big = max(max(w.x, w.y), max(w.z, w.w));
    int e = __builtin_amdgcn_readfirstlane(exponent_of(bits16_to_f32<DT>(big)));
    return e < -100 ? -100 : e;
  };
  // T[code] * scale of the unit into LDS
  const float2 *my_lut = lut + (lane & (COPIES - 1));
  auto dequantize = [&](int buf, int ek, int ev) {
    const uint32_t c[4] = {raw.x, raw.y, raw.z, raw.w};
    float2 tv[16];  // all table reads in flight before the first is used
#pragma unroll
    for (int j = 0; j < 16; ++j) tv[j] = my_lut[((c[j >> 2] >> (8 * (j & 3))) & 0xffu) * COPIES];
    __builtin_amdgcn_sched_barrier(0);
    if (isk) {
      const float f = ldexpf(bits16_to_f32<DT>(s0.x), 14 - ek);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        uint32_t w[4], y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 v = tv[4 * x + j];
          const float p0 = v.x * f, p1 = v.y * f;
          w[j] = f16_pair(p0, p1);
          if constexpr (TWO) {
            const f16x2v_t hv = __builtin_bit_cast(f16x2v_t, w[j]);
            y[j] = f16_pair(p0 - (float)hv[0], p1 - (float)hv[1]);
          }
        }
        uint8_t *dst = &kbuf[buf][0][ktok * KS + 64 * kch + 16 * x];
        *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
        if constexpr (TWO)
          *reinterpret_cast<uint4 *>(dst + KT * KS) = make_uint4(y[0], y[1], y[2], y[3]);
      }
    } else if (isv) {
      const uint32_t sw[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
      uint32_t w[2][8], y[2][8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {  // tokens 2 j, 2 j + 1
        const float f0 = ldexpf(bits16_to_f32<DT>(sw[j] & 0xffffu), 14 - ev);
        const float f1 = ldexpf(bits16_to_f32<DT>(sw[j] >> 16), 14 - ev);
        const float2 v0 = tv[2 * j], v1 = tv[2 * j + 1];
        const float e0 = v0.x * f0, e1 = v1.x * f1, o0 = v0.y * f0, o1 = v1.y * f1;
        w[0][j] = TWO ? f16_pair(e0, e1) : dithered_pair(e0, e1, j);
        w[1][j] = TWO ? f16_pair(o0, o1) : dithered_pair(o0, o1, j);
        if constexpr (TWO) {
          const f16x2v_t he = __builtin_bit_cast(f16x2v_t, w[0][j]), ho = __builtin_bit_cast(f16x2v_t, w[1][j]);
          y[0][j] = f16_pair(e0 - (float)he[0], e1 - (float)he[1]);
          y[1][j] = f16_pair(o0 - (float)ho[0], o1 - (float)ho[1]);
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        // tokens 0-3, 8-11 and then 4-7, 12-15: as the lanes hold their weights
        uint8_t *dst = &vbuf[buf][0][(2 * vpair + x) * VS + 32 * vgrp];
        *reinterpret_cast<uint4 *>(dst) = make_uint4(w[x][0], w[x][1], w[x][4], w[x][5]);
        *reinterpret_cast<uint4 *>(dst + 16) = make_uint4(w[x][2], w[x][3], w[x][6], w[x][7]);
        if constexpr (TWO) {
          *reinterpret_cast<uint4 *>(dst + D * VS) = make_uint4(y[x][0], y[x][1], y[x][4], y[x][5]);
          *reinterpret_cast<uint4 *>(dst + D * VS + 16) = make_uint4(y[x][2], y[x][3], y[x][6], y[x][7]);
        }
      }
    }
  };

  f32x16_t acc[DTI];
#pragma unroll
  for (int d = 0; d < DTI; ++d) acc[d] = f32x16_t{};
  float mx = kNoScore, l = 0.f;
  int ev = -100;
  bool far = false;  // a row's maximum is_far

  if (t_from < t_to) {
    const int t_last = t_to - 1;
    auto clip = [&](int t) { return t < t_last ? t : t_last; };
    int entry = page_entry(t_from);
    load_raw(t_from, entry);
    entry = page_entry(clip(t_from + 1));
    publish(t_from, 0, 0);
    __syncthreads();
    int ek = exponent16(kmax[0]), ek_next = 0;
    int ev_next = exponent16(vmax[0]);
    ev = ev_next;
    dequantize(0, ek, ev);
    load_raw(clip(t_from + 1), entry);
    entry = page_entry(clip(t_from + 2));
    publish(clip(t_from + 1), 1, 1);
    __syncthreads();
    for (int t = t_from, slot = 0; t < t_to; ++t) {
      const int buf = (t - t_from) & 1;
      // the next tile into the other buffer (after the last: once more the last)
      ek_next = exponent16(kmax[buf ^ 1]);
      const int e2 = exponent16(vmax[buf ^ 1]);
      ev_next = e2 > ev ? e2 : ev;
      const bool next = t + 1 < t_to;
      if (next) dequantize(buf ^ 1, ek_next, ev_next);
      const int t2 = clip(t + 2);
      load_raw(t2, entry);
      entry = page_entry(clip(t + 3));

      const int t0 = lo + t * KT;
      if (busy && t0 < any_hi) {
        // ---- scores ----
        f32x16_t sc[TT];
#pragma unroll
        for (int x = 0; x < TT; ++x) {
          sc[x] = f32x16_t{};
          const uint8_t *kr = &kbuf[buf][0][(32 * x + (lane & 31)) * KS + 16 * half];
#pragma unroll
          for (int c = 0; c < QS; ++c) {
            sc[x] = __builtin_amdgcn_mfma_f32_32x32x16_f16(*reinterpret_cast<const f16x8_t *>(kr + 32 * c), qf[c], sc[x], 0, 0, 0);
            if constexpr (TWO)
              sc[x] = __builtin_amdgcn_mfma_f32_32x32x16_f16(*reinterpret_cast<const f16x8_t *>(kr + KT * KS + 32 * c), qf[c], sc[x], 0, 0, 0);
          }
        }
        // fragments are read six ahead of the products that take them
        __builtin_amdgcn_sched_group_barrier(0x100, 6, 0);
#pragma unroll
        for (int x = 0; x < TT * QS * PL - 6; ++x) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, 6, 0);
        const uint32_t pages = *reinterpret_cast<const uint32_t *>(there[slot]) & (KT == 64 ? 0x01010101u : 0x0101u);
        if (!(t0 >= all_lo && t0 + KT <= all_hi && __all(pages == (KT == 64 ? 0x01010101u : 0x0101u)))) {
#pragma unroll
          for (int x = 0; x < TT; ++x)
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int at = 32 * x + 8 * (j >> 2) + 4 * half + (j & 3);
              const bool seen = (t0 + at >= row_lo) & (t0 + at < row_hi) & (pages >> (8 * (2 * x + (j >> 3))) & 1u);
              sc[x][j] = seen ? sc[x][j] : -INFINITY;
            }
        }
        // ---- running maximum of the row ----
        float top = sc[0][0];
#pragma unroll
        for (int x = 0; x < TT; ++x)
#pragma unroll
          for (int j = 0; j < 16; ++j) top = fmaxf(top, sc[x][j]);
        {
          uint32_t p = __float_as_uint(top), q = p;
          swap32(p, q);
          top = fmaxf(__uint_as_float(p), __uint_as_float(q));
        }
        const float f = fmaxf(ldexpf(qscale, ek - 14), 0x1p-100f);  // never 0: a masked score stays -inf
        top *= f;
        if (__any(top > mx)) {
          const float mn = fmaxf(mx, top);
          const float keep = __builtin_amdgcn_exp2f(mx - mn);
          mx = mn;
          far = __any(is_far(mx));
          l *= keep;
#pragma unroll
          for (int d = 0; d < DTI; ++d) acc[d] *= keep;
        }
        // ---- weights (times 2^14) and the products with the values ----
        if (far) {
#pragma unroll
          for (int x = 0; x < TT; ++x)
#pragma unroll
            for (int j = 0; j < 16; ++j) sc[x][j] = sc[x][j] * f - mx;
        }
        const float fm = far ? 1.f : f, shift = far ? 14.f : 14.f - mx;
        float sum = 0.f;
#pragma unroll
        for (int x = 0; x < TT; ++x)
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            sc[x][j] = __builtin_amdgcn_exp2f(fmaf(sc[x][j], fm, shift));
            sum += sc[x][j];
          }
        l += sum;
#pragma unroll
        for (int x = 0; x < TT; ++x)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            u32x4_t ph, pl;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float w0 = sc[x][8 * c + 2 * j], w1 = sc[x][8 * c + 2 * j + 1];
              const uint32_t pair = f16_pair(w0, w1);
              ph[j] = pair;
              if constexpr (TWO) {
                const f16x2v_t hv = __builtin_bit_cast(f16x2v_t, pair);
                pl[j] = f16_pair(w0 - (float)hv[0], w1 - (float)hv[1]);
              }
            }
            const f16x8_t pf = __builtin_bit_cast(f16x8_t, ph);
            const uint8_t *vr = &vbuf[buf][0][(lane & 31) * VS + 32 * (2 * x + c) + 16 * half];
#pragma unroll
            for (int d = 0; d < DTI; ++d) {
              const f16x8_t vf = *reinterpret_cast<const f16x8_t *>(vr + 32 * d * VS);
              acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf, pf, acc[d], 0, 0, 0);
              if constexpr (TWO) {
                acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf, __builtin_bit_cast(f16x8_t, pl), acc[d], 0, 0, 0);
                const f16x8_t vl = *reinterpret_cast<const f16x8_t *>(vr + D * VS + 32 * d * VS);
                acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vl, pf, acc[d], 0, 0, 0);
              }
            }
          }
      }
      if (next && ev_next != ev) {  // the next tile's values are scaled by another power of two
        const float keep = ldexpf(1.f, ev - ev_next);
#pragma unroll
        for (int d = 0; d < DTI; ++d) acc[d] *= keep;
        ev = ev_next;
      }
      ek = ek_next;
      publish(t2, buf, slot == 0 ? 2 : slot - 1);  // (slot + 2) % 3
      slot = slot == 2 ? 0 : slot + 1;
      __syncthreads();
    }
  }

  // ---- results: the row's sum over both halves of the wave ----
  {
    uint32_t p = __float_as_uint(l), q = p;
    swap32(p, q);
    l = __uint_as_float(p) + __uint_as_float(q);
  }
  if (!real) return;
  if (pa.splits == 1) {
    const float inv = l > 0.f ? ldexpf(1.f / l, ev - 14) : 0.f;
    uint16_t *orow = static_cast<uint16_t *>(a.out.p) + (s.row0 + i_row) * a.out.ts + h_row * a.out.hs;
#pragma unroll
    for (int d = 0; d < DTI; ++d)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint2 *>(orow + 32 * d + 8 * j + 4 * half) =
            make_uint2(cvt_pair<DT>(acc[d][4 * j] * inv, acc[d][4 * j + 1] * inv),
                       cvt_pair<DT>(acc[d][4 * j + 2] * inv, acc[d][4 * j + 3] * inv));
  } else {
    const float unit = ldexpf(1.f, ev - 14);
    const int64_t slot = ((s.row0 + i_row) * a.q.heads + h_row) * pa.splits + split;
    if (half == 0) pa.part.ml[slot] = make_float2(mx, l);
#pragma unroll
    for (int d = 0; d < DTI; ++d)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<float4 *>(pa.part.o + slot * D + 32 * d + 8 * j + 4 * half) =
            make_float4(acc[d][4 * j] * unit, acc[d][4 * j + 1] * unit, acc[d][4 * j + 2] * unit, acc[d][4 * j + 3] * unit);
  }
}

// A row's parts joined: a workgroup takes 256 / (dim / 4) rows of (token, query
// head); a thread sums four elements over the splits.  Latency: 4.7 us for 16
// sequences of one token, 64 heads of 128 and 4 splits.
template <int DT>
__global__ __launch_bounds__(256) void prompt_join_kernel(PromptArgs pa, int dim) {
  const AttnArgs &a = pa.a;
  const int quads = dim / 4, per = 256 / quads;
  const int k = threadIdx.x / quads, x = threadIdx.x - k * quads;
  if (k >= per) return;
  const int b = blockIdx.y;
  const SeqRange s = seq_range(a.kb, b);
  const int n = s.n < a.kb.max_q ? s.n : a.kb.max_q;
  const int64_t row = (int64_t)blockIdx.x * per + k;
  if (row >= (int64_t)n * a.q.heads) return;
  const int i = (int)(row / a.q.heads), h = (int)(row - (int64_t)i * a.q.heads);
  const int64_t slot = ((s.row0 + i) * a.q.heads + h) * pa.splits;
  float mx = kNoScore;
  for (int w = 0; w < pa.splits; ++w) mx = fmaxf(mx, pa.part.ml[slot + w].x);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
#pragma unroll 4
  for (int w = 0; w < pa.splits; ++w) {
    const float2 ml = pa.part.ml[slot + w];
    const float4 y = *reinterpret_cast<const float4 *>(pa.part.o + (slot + w) * dim + 4 * x);
    const float f = __builtin_amdgcn_exp2f(ml.x - mx);
    l = fmaf(f, ml.y, l);
    o.x = fmaf(f, y.x, o.x), o.y = fmaf(f, y.y, o.y), o.z = fmaf(f, y.z, o.z), o.w = fmaf(f, y.w, o.w);
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint16_t *dst = static_cast<uint16_t *>(a.out.p) + (s.row0 + i) * a.out.ts + h * a.out.hs + 4 * x;
  *reinterpret_cast<uint2 *>(dst) = make_uint2(cvt_pair<DT>(o.x * inv, o.y * inv), cvt_pair<DT>(o.z * inv, o.w * inv));
}

// Row tiles of a sequence, and the splits that give every compute unit a
// workgroup where the rows alone do not, of no fewer than 8 tiles of keys (a
// workgroup's start and its part of the join cost about as much).  16 sequences
// of about 4600 tokens, 32 rows of 4 heads of 128: 65 + 5 us with 4 splits.
static void prompt_plan(const KVCache &c, const KVBatch &kb, int group, int64_t max_kv, int64_t window, int *mtiles,
                        int *splits) {
  const int64_t rows = (int64_t)kb.max_q * group;
  *mtiles = (int)((rows + kPRows - 1) / kPRows);
  int64_t keys = max_kv;
  if (window > 0) keys = std::min<int64_t>(keys, window + kb.max_q + 15);
  const int64_t wgs = (int64_t)*mtiles * c.heads * kb.batch;
  const int64_t most = std::max<int64_t>(1, keys / (8 * prompt_tile(c.dim, false)));
  *splits = (int)std::max<int64_t>(1, std::min<int64_t>(most, device_cu_count() / wgs));
}

bool prompt_eligible(const KVCache &c) { return decode_eligible(c, 1); }

size_t prompt_workspace_bytes(const KVCache &c, const KVBatch &kb, int q_heads, int64_t max_kv, int64_t window) {
  int mtiles, splits;
  prompt_plan(c, kb, q_heads / c.heads, max_kv, window, &mtiles, &splits);
  return splits > 1 ? (size_t)kb.tokens * q_heads * splits * (c.dim + 2) * 4 : 0;
}

template <int DT>
static hipError_t launch_prompt_t(const PromptArgs &pa, hipStream_t st) {
  const AttnArgs &a = pa.a;
  const int64_t wgs = (int64_t)a.c.heads * pa.mtiles * pa.splits * a.kb.batch;
  if (!grid_fits(wgs, kPThreads)) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)wgs);
  constexpr bool two = DT == kF16;
#define QMV_P(D) hipLaunchKernelGGL((attention_prompt_kernel<D, DT, two>), grid, dim3(kPThreads), 0, st, pa)
  switch (a.c.dim) {
    case 64: QMV_P(64); break;
    case 96: QMV_P(96); break;
    case 128: QMV_P(128); break;
    case 192: QMV_P(192); break;
    default: QMV_P(256);
  }
#undef QMV_P
  return hipGetLastError();
}

hipError_t launch_attention_prompt(const AttnArgs &a, int dt, void *ws, hipStream_t st) {
  PromptArgs pa{a, {}, 1, 1};
  prompt_plan(a.c, a.kb, a.group, a.max_kv, a.window, &pa.mtiles, &pa.splits);
  pa.part.o = static_cast<float *>(ws);
  pa.part.ml = reinterpret_cast<float2 *>(pa.part.o + (size_t)a.kb.tokens * a.q.heads * pa.splits * a.c.dim);
  const hipError_t e = dt == kBF16 ? launch_prompt_t<kBF16>(pa, st) : launch_prompt_t<kF16>(pa, st);
  if (e != hipSuccess || pa.splits == 1) return e;
  const int per = 256 / (a.c.dim / 4);
  const int64_t rows = (int64_t)a.kb.max_q * a.q.heads;
  const dim3 grid((unsigned)((rows + per - 1) / per), (unsigned)a.kb.batch);
  if (dt == kBF16) hipLaunchKernelGGL((prompt_join_kernel<kBF16>), grid, dim3(256), 0, st, pa, a.c.dim);
  else hipLaunchKernelGGL((prompt_join_kernel<kF16>), grid, dim3(256), 0, st, pa, a.c.dim);
  return hipGetLastError();
}

}  // namespace qmv
