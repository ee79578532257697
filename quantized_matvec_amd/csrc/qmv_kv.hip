// The 4-bit key/value cache: appending keys and values (the position rotation
// applied on the way) and reading them back.
//
// A row (one token's head) is quantized as quantize_4bit quantizes a run of
// head_dim elements: per block of bs elements a = max |x|, the code nearest to
// x / a, exactly.  Rows have 16-bit elements, and that makes the exact search
// cheap: a code is the number of midpoints m with x above a m, and with at
// most 11 significant bits in x and a, no x lies between a m and fp32(a m) (an
// exhaustive check over all pairs of 11-bit significands and every midpoint of
// both tables is in the tests), so one fp32 product and comparison decides as
// the exact comparison does, ties included.  Blocks with a < 2^-100 are scaled
// up by 2^100 first (exactly), so the product is never subnormal.
#include <algorithm>

#include "qmv_attention.hpp"

#pragma clang fp contract(off)

namespace qmv {

struct Mids32 {
  float m[15];
};

// Code of x against the thresholds a m_j (ascending; NF4: 7 negative, 8
// positive; FP4: the 7 positive ones, on magnitudes).
template <int QT>
__device__ __forceinline__ uint32_t nearest_code(float x, const float (&thr)[15]) {
  uint32_t r = 0;
  if constexpr (QT == kNF4) {
#pragma unroll
    for (int j = 0; j < 7; ++j) r += x >= thr[j] ? 1u : 0u;
#pragma unroll
    for (int j = 7; j < 15; ++j) r += x > thr[j] ? 1u : 0u;
  } else {
    const float ax = fabsf(x);
#pragma unroll
    for (int j = 0; j < 7; ++j) r += ax > thr[j] ? 1u : 0u;
    r |= (x < 0.f && r) ? 8u : 0u;
  }
  return r;
}

template <int DT>
__device__ __forceinline__ void unpack8(const uint4 &w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bits16_to_f32<DT>(u[i] & 0xffffu);
    x[2 * i + 1] = bits16_to_f32<DT>(u[i] >> 16);
  }
}

// The rotation of elements e0 .. e0 + 7 of a token's rows: the angles are
// fetched once.  An element e of the rotated part becomes
// x_e c + sign x_partner s, sign -1 for the first of a pair (rounded as
// x c - partner s, since negation is exact).
template <int DT>
struct Turn {
  float c[8], s[8];  // cos, and sin with the sign
  uint32_t turned;   // bit i: element e0 + i is of the rotated part
  int off;           // partner run's distance (halves), 0: pairs inside the run or no whole run
  int first;         // halves without a whole run: e0, else -1
  int half;
  bool zero;         // no such position in the table: zeros
  bool inter, any;

  __device__ __forceinline__ void load(const Rope &rope, int e0, int64_t pos) {
    half = rope.half;
    inter = rope.interleaved;
    any = rope.table != nullptr && e0 < 2 * half;
    zero = rope.table != nullptr && (pos < 0 || pos >= rope.max_pos);
    off = 0;
    first = -1;
    turned = 0;
    if (!any || zero) return;
    const float2 *cs = rope.table + pos * half;
    const bool whole = half % 8 == 0;  // a run's partners are one aligned run
    if (!inter && whole) off = e0 < half ? half : -half;
    if (!inter && !whole) first = e0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = e0 + i;
      const bool in = e < 2 * half;
      const bool lead = inter ? (e & 1) == 0 : e < half;
      const int p = inter ? e >> 1 : (lead ? e : e - half);
      const float2 v = cs[in ? p : 0];
      c[i] = v.x;
      s[i] = lead ? -v.y : v.y;
      turned |= in ? 1u << i : 0u;
    }
  }
  // The run that holds the partners (p: this run); itself where there is none.
  __device__ __forceinline__ uint4 partner(const uint16_t *p) const {
    return *reinterpret_cast<const uint4 *>(p + off);
  }
  __device__ __forceinline__ void apply(const uint16_t *p, const uint4 &other, float (&x)[8]) const {
    if (zero) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 0.f;
      return;
    }
    if (!any) return;
    float y[8];
    if (inter) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = x[i ^ 1];
    } else if (first < 0) {
      unpack8<DT>(other, y);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = first + i;
        y[i] = e < 2 * half ? bits16_to_f32<DT>(p[i + (e < half ? half : -half)]) : 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float r = x[i] * c[i] + y[i] * s[i];
      x[i] = turned >> i & 1u ? r : x[i];
    }
  }
};

// What a thread works on.  A row takes LPR lanes of a wave, 8 elements each; a
// workgroup has 256 / LPR rows at a time: TG tokens side by side for each of
// HS rows h, and goes through `iters` such sets of rows, so that positions,
// pages and angles are fetched once.  With TG = 1 (few tokens) the rows of one token fill the
// workgroup; otherwise TG places of one group of 16 cache positions do, and
// one workgroup writes all bytes of a value group and of a group's scales
// (2532 tokens of three chunks, 32 + 32 + 32 heads of 64: 28.3 us one by one,
// 23.6 us in groups, one set of rows a thread both times).
template <int LPR, int TG>
struct Place {
  static constexpr int RPW = 256 / LPR, HS = RPW / TG;
  int i;   // token of the sequence, or negative: none
  int h;   // the first row h; further ones HS apart
  int end; // rows of this workgroup end before
  __device__ __forceinline__ Place(unsigned x, int rows, int iters, const SeqRange &s, int most) {
    const int blocks = (rows + HS * iters - 1) / (HS * iters);  // along the rows of a token
    const int group = (int)(x / (unsigned)blocks), block = (int)(x - (unsigned)group * blocks);
    const int slot = threadIdx.x / LPR;
    h = block * HS * iters + slot / TG;
    end = (block + 1) * HS * iters < rows ? (block + 1) * HS * iters : rows;
    const int64_t place = (int64_t)group * TG + slot % TG;
    const int64_t t = place - (s.pos0 & (TG - 1));
    i = t >= 0 && t < s.n && t < most ? (int)t : -1;
  }
};

struct AppendArgs {
  KVCache c;
  KVBatch kb;
  Heads k, v, q, qo;  // q.heads 0: no queries
  Rope rope;          // table NULL: not turned
  Mids32 mids;
};

// What a workgroup takes, so that its loop over rows is one code for all its
// waves.
enum : int { kQueries, kKeys, kValues };

// Tokens side by side for queries, which need no whole groups: four make longer
// runs of a token's heads (16 for queries too 78.7 us at 7375 tokens of 64
// query heads, 19.3 at 2532 of 32; 4: 73.9 and 19.8; 1: 82.7 and 22.5).
constexpr int query_tokens(int tg) { return tg < 4 ? tg : 4; }

template <int DT, int QT, int LPR, int TG, int WHAT>
__device__ __forceinline__ void append_rows(const AppendArgs &a, unsigned place, int iters) {
  using P = Place<LPR, TG>;
  const int b = blockIdx.y;
  const SeqRange s = seq_range(a.kb, b);
  const Heads &src = WHAT == kQueries ? a.q : (WHAT == kKeys ? a.k : a.v);
  const P pl(place, src.heads, iters, s, a.kb.max_q);
  const int e0 = 8 * (int)(threadIdx.x % LPR);
  if (pl.i < 0 || pl.h >= pl.end) return;
  const int pos = s.pos0 + pl.i;
  const int64_t t = s.row0 + pl.i;
  const bool mine = e0 < a.c.dim;
  int64_t page = 0;
  if constexpr (WHAT != kQueries) {
    page = page_of(a.kb, a.c, b, pos);
    if (page < 0) return;  // the same for the whole row
  }
  const int at = pos & ((1 << a.c.log2page) - 1);
  const uint16_t *in = static_cast<const uint16_t *>(src.p) + t * src.ts + pl.h * src.hs + (mine ? e0 : 0);
  Turn<DT> turn;
  if constexpr (WHAT != kValues) turn.load(a.rope, e0, pos);
  uint16_t *out = nullptr;  // queries
  uint8_t *codes = nullptr;
  uint16_t *scales = nullptr;
  const int64_t head_bytes = (int64_t)(a.c.dim >> 1) << a.c.log2page, head_scales = (int64_t)(a.c.dim / a.c.bs) << a.c.log2page;
  if constexpr (WHAT == kQueries) {
    out = static_cast<uint16_t *>(a.qo.p) + t * a.qo.ts + pl.h * a.qo.hs + e0;
  } else {
    const int64_t first = page * a.c.heads + pl.h;
    codes = (WHAT == kValues ? a.c.vc + (int64_t)(at >> 4) * a.c.dim * 8 + (e0 >> 1) * 16 + (at & 15)
                             : a.c.kc + (int64_t)at * (a.c.dim >> 1) + (e0 >> 1)) + first * head_bytes;
    scales = (WHAT == kValues ? a.c.vs : a.c.ks) + first * head_scales + ((int64_t)(e0 / a.c.bs) << a.c.log2page) + at;
  }
  for (int h = pl.h; h < pl.end; h += P::HS) {
    const uint4 raw = *reinterpret_cast<const uint4 *>(in);
    float x[8];
    unpack8<DT>(raw, x);
    if constexpr (WHAT != kValues) turn.apply(in, turn.partner(in), x);
    in += P::HS * src.hs;
    uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    if constexpr (WHAT != kValues) {
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = cvt_pair<DT>(x[2 * j], x[2 * j + 1]);
    }
    if constexpr (WHAT == kQueries) {
      if (mine) *reinterpret_cast<uint4 *>(out) = make_uint4(w[0], w[1], w[2], w[3]);
      out += P::HS * a.qo.hs;
    } else {
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // what is quantized: the row as the cache's type holds it
        x[2 * j] = bits16_to_f32<DT>(w[j] & 0xffffu);
        x[2 * j + 1] = bits16_to_f32<DT>(w[j] >> 16);
        m = fmaxf(m, fmaxf(fabsf(x[2 * j]), fabsf(x[2 * j + 1])));
      }
      m = group_max(m, a.c.bs >> 3);  // (lanes past the row's end repeat its first run, in blocks of their own)
      const float up = m < 0x1p-100f ? 0x1p100f : 1.f;
      float thr[15];
#pragma unroll
      for (int j = 0; j < 15; ++j) thr[j] = (m * up) * a.mids.m[j];
      uint32_t word = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t code = nearest_code<QT>(x[j] * up, thr);
        word |= code << (8 * (j >> 1) + (j & 1 ? 0 : 4));  // even element: high nibble
      }
      if (mine) {
        if constexpr (WHAT == kValues) {
#pragma unroll
          for (int j = 0; j < 4; ++j) codes[16 * j] = (uint8_t)(word >> (8 * j));
        } else {
          *reinterpret_cast<uint32_t *>(codes) = word;
        }
        if ((e0 & (a.c.bs - 1)) == 0) *scales = (uint16_t)f32_to_bits16<DT>(m);
      }
      codes += P::HS * head_bytes;
      scales += P::HS * head_scales;
    }
  }
}

// Bound by memory in large calls, where a value byte is a store of its own, and
// by the fifteen comparisons of an element.  7375 tokens of 5 prompts, 64 + 8 +
// 8 heads of 128, bf16: 74 us for 280 MB, 3.8 TB/s, of which the queries are
// 242 MB; 2532 tokens, 32 + 32 + 32 heads of 64, fp16: 18.6 us; 32 single
// tokens: 5.1 us, mostly the chain length -> page -> write.  Queries, keys and
// values are in workgroups of their own, since one loop with all three kept the
// registers of each (144 and 28 us, with one set of rows a thread).  Values,
// which take longest, come first, and no part's grid is padded to another's
// (queries first and padded: 84.5 us instead of 79).
template <int DT, int QT, int LPR, int TG>
__global__ __launch_bounds__(256) void kv_append_kernel(AppendArgs a, int q_iters, int kv_iters, unsigned kv_grid) {
  const unsigned x = blockIdx.x;
  if (x < kv_grid) append_rows<DT, QT, LPR, TG, kValues>(a, x, kv_iters);
  else if (x < 2 * kv_grid) append_rows<DT, QT, LPR, TG, kKeys>(a, x - kv_grid, kv_iters);
  else append_rows<DT, QT, LPR, query_tokens(TG), kQueries>(a, x - 2 * kv_grid, q_iters);
}

// Lanes of a row: head_dim / 8 rounded up to a power of two.
static int row_lanes(int dim) { return dim <= 32 ? 4 : dim <= 64 ? 8 : dim <= 128 ? 16 : 32; }

// Calls with fewer new tokens of a sequence take them one by one (append and
// read back of 64 sequences, 32 + 8 + 8 rows of 128, one by one and in groups: 4
// tokens 9.7 us and 14.1, 8 tokens 15.8 and 14.8, 12 tokens 17.5 and 17.9, 16 tokens
// 19.8 and 20.0, 20 tokens 22.8 and 22.1, 24 tokens 25.4 and 22.8, 64 tokens 51 and
// 39; of 16 sequences, 32 + 32 + 32 heads of 64, 15 tokens 11.5 and 11.8, 24 tokens
// 14.8 and 13.7; chunks of 1000 tokens at Place).
constexpr int kGroupFrom = 16;

// Grid and sets of rows of a workgroup: as many sets (up to 16) as leave 8
// workgroups for each compute unit (the two large calls above, all parts in
// groups of 16, with 4, 8 and 16: 85.6 and 18.7, 85.4 and 18.1, 82.4 and 20.9
// us; at most 32 sets: 87.2 and 19.5 against 79.1 and 19.1).
template <int LPR, int TG>
static int64_t append_grid(const KVBatch &kb, int rows, int *iters) {
  constexpr int HS = 256 / LPR / TG;
  const int64_t groups = ((int64_t)kb.max_q + 2 * (TG - 1)) / TG;  // a group may begin TG - 1 places early
  const int64_t sets = (rows + HS - 1) / HS;
  *iters = (int)std::min<int64_t>(std::max<int64_t>(groups * kb.batch * sets * 3 / (8 * device_cu_count()), 1),
                                  std::min<int64_t>(sets, 16));
  return groups * ((rows + HS * *iters - 1) / (HS * *iters));
}

template <int DT, int QT, int LPR, int TG>
static hipError_t launch_append_g(const AppendArgs &a, hipStream_t st) {
  int q_iters = 1, kv_iters;
  const int64_t kv_grid = append_grid<LPR, TG>(a.kb, a.c.heads, &kv_iters);
  const int64_t q_grid = a.q.heads ? append_grid<LPR, query_tokens(TG)>(a.kb, a.q.heads, &q_iters) : 0;
  if (!grid_fits(2 * kv_grid + q_grid, 256)) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)(2 * kv_grid + q_grid), (unsigned)a.kb.batch);
  hipLaunchKernelGGL((kv_append_kernel<DT, QT, LPR, TG>), grid, dim3(256), 0, st, a, q_iters, kv_iters, (unsigned)kv_grid);
  return hipGetLastError();
}

template <int DT, int QT>
static hipError_t launch_append_t(const AppendArgs &a, hipStream_t st) {
  const bool few = a.kb.max_q < kGroupFrom;
  switch (row_lanes(a.c.dim)) {
    case 4: return few ? launch_append_g<DT, QT, 4, 1>(a, st) : launch_append_g<DT, QT, 4, 16>(a, st);
    case 8: return few ? launch_append_g<DT, QT, 8, 1>(a, st) : launch_append_g<DT, QT, 8, 16>(a, st);
    case 16: return few ? launch_append_g<DT, QT, 16, 1>(a, st) : launch_append_g<DT, QT, 16, 16>(a, st);
    default: return few ? launch_append_g<DT, QT, 32, 1>(a, st) : launch_append_g<DT, QT, 32, 8>(a, st);
  }
}

hipError_t launch_kv_append(const KVCache &c, int dt, int qt, const Midpoints4 &mids,
                            const KVBatch &kb, const Heads &k, const Heads &v, const Rope &rope,
                            const Heads &q, const Heads &qo, hipStream_t st) {
  AppendArgs a{c, kb, k, v, q, qo, rope, {}};
  for (int j = 0; j < 15; ++j) a.mids.m[j] = (float)mids.mid[qt == kNF4 ? j : std::min(7 + j, 13)];
  if (dt == kBF16) {
    return qt == kNF4 ? launch_append_t<kBF16, kNF4>(a, st) : launch_append_t<kBF16, kFP4>(a, st);
  }
  return qt == kNF4 ? launch_append_t<kF16, kNF4>(a, st) : launch_append_t<kF16, kFP4>(a, st);
}

// ---------------------------------------------------------------------------
// Reading back: fp32(T[code] * a) rounded to the cache's type.  A byte becomes
// both values by one table read.  Rows go through it as through the append, with
// the same places and sets.  Bound by the 16-bit writes and, for values, by
// loads of single bytes 16 apart: the 7375 tokens (8 + 8 heads of 128) 20.6 us
// for 38 MB, the 2532 tokens (32 + 32 heads of 64) 11.0 us for 27 MB, 32 single
// tokens 3.6 us.
// ---------------------------------------------------------------------------
struct ReadArgs {
  KVCache c;
  KVBatch kb;
  Heads k, v;
};

template <int DT, int LPR, int TG>
__global__ __launch_bounds__(256) void kv_dequantize_kernel(ReadArgs a, int qt, int iters) {
  using P = Place<LPR, TG>;
  __shared__ float2 lut[256];  // packed byte -> (T[byte >> 4], T[byte & 15])
  {
    const uint32_t *tb = table_bits(qt);
    lut[threadIdx.x] = make_float2(__uint_as_float(tb[threadIdx.x >> 4]),
                                   __uint_as_float(tb[threadIdx.x & 15]));
  }
  __syncthreads();
  const int b = blockIdx.y;
  const SeqRange s = seq_range(a.kb, b);
  const bool isv = blockIdx.z != 0;
  const P pl(blockIdx.x, a.c.heads, iters, s, a.kb.max_q);
  const int e0 = 8 * (int)(threadIdx.x % LPR);
  if (pl.i < 0 || e0 >= a.c.dim || pl.h >= pl.end) return;
  const int pos = s.pos0 + pl.i;
  const int64_t t = s.row0 + pl.i;
  const int64_t page = page_of(a.kb, a.c, b, pos);
  const int at = pos & ((1 << a.c.log2page) - 1);
  const int64_t head_bytes = (int64_t)(a.c.dim >> 1) << a.c.log2page, head_scales = (int64_t)(a.c.dim / a.c.bs) << a.c.log2page;
  const int64_t first = page < 0 ? 0 : page * a.c.heads + pl.h;
  const uint8_t *src = (isv ? a.c.vc + (int64_t)(at >> 4) * a.c.dim * 8 + (e0 >> 1) * 16 + (at & 15)
                            : a.c.kc + (int64_t)at * (a.c.dim >> 1) + (e0 >> 1)) + first * head_bytes;
  const uint16_t *sc = (isv ? a.c.vs : a.c.ks) + first * head_scales + ((int64_t)(e0 / a.c.bs) << a.c.log2page) + at;
  const Heads &dst = isv ? a.v : a.k;
  uint16_t *out = static_cast<uint16_t *>(dst.p) + t * dst.ts + pl.h * dst.hs + e0;
  const int step = isv ? 16 : 1;  // bytes from one pair of elements to the next
  for (int h = pl.h; h < pl.end; h += P::HS) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = src[j * step];
    const float m = bits16_to_f32<DT>(sc[0]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 v = lut[w[j]];
      w[j] = page >= 0 ? cvt_pair<DT>(v.x * m, v.y * m) : 0u;
    }
    *reinterpret_cast<uint4 *>(out) = make_uint4(w[0], w[1], w[2], w[3]);
    src += P::HS * head_bytes;
    sc += P::HS * head_scales;
    out += P::HS * dst.hs;
  }
}

template <int DT, int LPR, int TG>
static hipError_t launch_read_g(const ReadArgs &a, int qt, hipStream_t st) {
  int iters;
  const int64_t x = append_grid<LPR, TG>(a.kb, a.c.heads, &iters);
  if (!grid_fits(x, 256)) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)x, (unsigned)a.kb.batch, 2);  // keys, values
  hipLaunchKernelGGL((kv_dequantize_kernel<DT, LPR, TG>), grid, dim3(256), 0, st, a, qt, iters);
  return hipGetLastError();
}

template <int DT>
static hipError_t launch_read_t(const ReadArgs &a, int qt, hipStream_t st) {
  const bool few = a.kb.max_q < kGroupFrom;
  switch (row_lanes(a.c.dim)) {
    case 4: return few ? launch_read_g<DT, 4, 1>(a, qt, st) : launch_read_g<DT, 4, 16>(a, qt, st);
    case 8: return few ? launch_read_g<DT, 8, 1>(a, qt, st) : launch_read_g<DT, 8, 16>(a, qt, st);
    case 16: return few ? launch_read_g<DT, 16, 1>(a, qt, st) : launch_read_g<DT, 16, 16>(a, qt, st);
    default: return few ? launch_read_g<DT, 32, 1>(a, qt, st) : launch_read_g<DT, 32, 8>(a, qt, st);
  }
}

hipError_t launch_kv_dequantize(const KVCache &c, int dt, int qt, const KVBatch &kb,
                                const Heads &k, const Heads &v, hipStream_t st) {
  const ReadArgs a{c, kb, k, v};
  return dt == kBF16 ? launch_read_t<kBF16>(a, qt, st) : launch_read_t<kF16>(a, qt, st);
}

}  // namespace qmv
