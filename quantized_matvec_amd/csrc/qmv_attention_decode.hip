// Attention of a few query rows (up to 48, in tiles of 16: new tokens times
// query heads of a cache head) over the 4-bit cache: the serving step, bound by
// reading the cache once.
//
// A wave takes 64 tokens a step.  Scores are S = Q K^T with
// v_mfma_f32_16x16x32_f16 (16 query rows by 16 tokens), outputs O^T = V^T P^T
// (16 pairs of elements by 16 query rows).  Lane l has column r = l % 16 and
// row group g = l / 16.
//  * A lane gets rows 4 g .. 4 g + 3 of a score tile, column r.  Query row i
//    is put at tile row 4 (i / RJ) + i % RJ, so with up to 4, 8 or 16 rows a
//    lane has RJ = 1, 2 or 4 that mean anything, and the exponentials, sums
//    and scales are computed for those alone.
//  * Column r of score tile i is token 4 r + i: a lane's four tokens are
//    neighbours, their scales one 8-byte load a block, and their weights one
//    8-byte write to LDS, from where the second product takes 16 tokens of a
//    row as two 16-byte reads.
//  * The keys' bytes come as 16-byte loads, whose four words belong to four
//    different k-steps; a 4 x 4 transpose among the rows of 16 lanes (four
//    lane swaps for 32 values) gives each k-step 32 consecutive elements, all
//    of one scale block, so a block's scale multiplies finished fp32 sums.
//  * The values' bytes lie 16 tokens side by side, so a 16-byte load is a pair
//    of elements of 16 tokens in the order in which the weights are read.  The
//    value scale multiplies the weight before the weight is rounded to fp16.
//  * Codes become fp16 pairs by one table read for two.  The NF4 values are
//    not fp16 numbers: for the values the rest below fp16 comes from a second
//    table and is multiplied too (LO), because its sum over a long sequence
//    does not cancel while the values' own does; in the scores it is a shift
//    common to all keys, to which the softmax is blind, and a random part of
//    6e-5 of the score.
// Queries are scaled by a power of two of their own (exact) into fp16's range
// and the products p a by one common to the wave, which keeps the largest
// finite block scale that any of its rows has seen so far in [2^14, 2^15): a
// weight loses nothing above 2^-38 of the largest.
//
// Work is divided by steps, whatever the lengths are (they are read here, on
// the device): each workgroup takes an equal run of the order (sequence, head,
// step), each of its waves an equal part of the run, and a wave goes through
// its heads by itself.  A workgroup whose run lies in one head adds its waves'
// sums up in LDS.  A head that no wave (or workgroup) holds whole is left as
// partial sums in the workspace, which attention_join_kernel adds up.
//
// Measured (32 query heads over 8 of 128, NF4 blocks of 64, bf16, one token,
// unless said otherwise), kernel and join:
//  * 196611 tokens, 64 query heads: 57 + 7 us for 214 MB.  In its steady state
//    it read 9 bytes a cycle and compute unit, 5.6 TB/s of the 6.4 that a
//    reading loop reaches (when the whole took 55 us); the table, the first loads
//    and the uneven ends are some 6000 cycles around it.
//  * 64 sequences of up to 8170 tokens: 73 + 6 us for 316 MB.
//  * 24 sequences of up to 8799, 4 tokens with a window of 4096, 32 heads over
//    32 of 64, FP4 blocks of 32, fp16: 51 + 6 us for 195 MB.
//  * one sequence of 1001: 11 + 5 us, launch, table and the chain of dependent
//    loads length -> page -> keys -> values.
#include <algorithm>

#include "qmv_attention_mfma.hpp"

namespace qmv {

constexpr int kStep = 64;      // tokens of a wave's step
constexpr int kJoinWaves = 4;
constexpr int kMaxRuns = 1024;  // workgroups of a call

struct DecodeArgs {
  AttnArgs a;
  Partials part;
  int runs;   // workgroups
  int tiles;  // of 16 query rows; the division of work takes a head's tiles for heads
};

// Steps of sequence b for each cache head: at least one, which writes the
// zeros of an empty sequence; none without tokens.
struct SeqSteps {
  SeqRange s;
  int n;        // tokens of this call that are worked on
  int lo, hi;   // keys [lo, hi) that any of them sees, lo a multiple of 16
  int steps;
};
__device__ __forceinline__ SeqSteps seq_steps(const AttnArgs &a, int b) {
  SeqSteps q;
  q.s = seq_range(a.kb, b);
  q.n = q.s.n < a.kb.max_q ? q.s.n : a.kb.max_q;
  int unused;
  key_range(a, q.s, 0, q.lo, unused);
  key_range(a, q.s, q.n - 1, unused, q.hi);
  q.lo &= ~15;
  const int keys = q.hi > q.lo ? q.hi - q.lo : 0;
  q.steps = q.n <= 0 ? 0 : (keys ? (keys + kStep - 1) / kStep : 1);
  return q;
}

// The same value in every lane, in scalar registers.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ SeqSteps uniform(const SeqSteps &q) {
  SeqSteps u;
  u.s.row0 = ((int64_t)uniform((int)(q.s.row0 >> 32)) << 32) | (uint32_t)uniform((int)q.s.row0);
  u.s.n = uniform(q.s.n);
  u.s.pos0 = uniform(q.s.pos0);
  u.s.len = uniform(q.s.len);
  u.n = uniform(q.n);
  u.lo = uniform(q.lo);
  u.hi = uniform(q.hi);
  u.steps = uniform(q.steps);
  return u;
}

// Sum of v over a workgroup of W waves, and the sum over the threads before
// this one.  tmp is free again after the next barrier.
template <int W>
__device__ __forceinline__ int scan(int v, int *tmp, int &before) {
  const int wave = threadIdx.x >> 6;
  int x = v;
  x += dpp_fill<0x111, 0xf>(x, 0);  // row_shr:1
  x += dpp_fill<0x112, 0xf>(x, 0);
  x += dpp_fill<0x114, 0xf>(x, 0);
  x += dpp_fill<0x118, 0xf>(x, 0);
  x += dpp_fill<0x142, 0xa>(x, 0);  // row_bcast:15
  x += dpp_fill<0x143, 0xc>(x, 0);  // row_bcast:31
  if ((threadIdx.x & 63) == 63) tmp[wave] = x;
  __syncthreads();
  int total = 0, base = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w < wave) base += tmp[w];
    total += tmp[w];
  }
  before = base + x - v;
  return total;
}

// The runs: workgroup k takes steps [k per, (k + 1) per) of total, its wave w
// of W the part [per w / W, per (w + 1) / W) of them.  Steps of all sequences
// and heads fit in 31 bits (checked on the host).
struct Runs {
  int total, per;
  __device__ __forceinline__ Runs(int total_, int runs) : total(total_), per((total_ + runs - 1) / runs) {}
  __device__ __forceinline__ int from(int k) const { return k * per < total ? k * per : total; }
  template <int W>
  __device__ __forceinline__ int wave_from(int k, int w) const {
    const int a = from(k), n = from(k + 1) - a;
    return a + (int)((uint32_t)n * (uint32_t)w / W);
  }
};

__device__ __forceinline__ uint32_t &word_of(uint4 &w, int i) {  // i: a constant
  return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
}

// Scale i of 4 (i a constant) as fp32.
template <int DT>
__device__ __forceinline__ float scale_at(const uint2 &s, int i) {
  const uint32_t w = i & 2 ? s.y : s.x;
  if constexpr (DT == kBF16) return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  else return bits16_to_f32<DT>(i & 1 ? w >> 16 : w & 0xffffu);
}

typedef __attribute__((ext_vector_type(2))) uint16_t u16x2_t;

// Maximum and sum over a row of 16 lanes.
template <int CTRL>
__device__ __forceinline__ float dpp_f32(float x) {
  return __uint_as_float(dpp_u32<CTRL>(__float_as_uint(x)));
}
__device__ __forceinline__ float row16_max(float v) {
  v = fmaxf(v, dpp_f32<0xb1>(v));
  v = fmaxf(v, dpp_f32<0x4e>(v));
  v = fmaxf(v, dpp_f32<0x141>(v));
  return fmaxf(v, dpp_f32<0x140>(v));
}
__device__ __forceinline__ float row16_sum(float v) {
  v += dpp_f32<0xb1>(v);
  v += dpp_f32<0x4e>(v);
  v += dpp_f32<0x141>(v);
  return v + dpp_f32<0x140>(v);
}

// Entries of the block table for a step: the page of the 16 tokens whose value
// bytes a lane loads (g), and of those whose key bytes and scales it loads
// (r / 4).
struct StepPages {
  int pg, pk;
};

// Waves of a workgroup, which has a compute unit to itself: three waves of a
// SIMD share its registers, two or one where rows are long and three or two
// would spill.  With the join: heads of 64: 57 us with 12, 59 with 8 (the 24
// sequences above); of 128: 62 and 81 us with 8, 71 and 90 with 12 (the long
// sequence, the 64); of 256: 69 us with 4, 75 with 8 (16 of the 64), in blocks of
// 32 100 and 120.  Between these neither number is always the better one.  Of 96:
// 70 us with 12, 68 with 8 (the 64), 104 and 106 (24 sequences of 4 tokens, 32
// cache heads), 69 and 58 (the same with 8).  Of 192: 137 us with 4, 115 with 8 (the
// 64), 91 and 82 (the 24 with 8 cache heads), but with blocks of 32 102 and 167,
// spilled: taken is the number whose worst case is the smaller.
__host__ __device__ constexpr int decode_waves(int D) { return D <= 96 ? 12 : D <= 128 ? 8 : 4; }

template <int D, int CB, int RJ, int DT, bool LO>
__global__ __launch_bounds__(64 * decode_waves(D), decode_waves(D) / 4) void attention_decode_kernel(DecodeArgs da) {
  constexpr int kWaves = decode_waves(D), kThreads = 64 * kWaves;
  constexpr int KU = D / 32;       // k-steps of a score, groups of 16 pairs of a value row
  constexpr int NB = KU / CB;      // scale blocks of a row
  constexpr int QR = 4 * RJ;       // query rows
  constexpr int JW = 32 + 4;       // row stride of the join buffer (floats)
  constexpr int PB = DT == kF16 ? 2 : 1;  // fp16 terms of a weight
  constexpr uint32_t kInf16 = DT == kF16 ? 0x7c00u : 0x7f80u;
  constexpr int row_bytes = D / 2;
  __shared__ __align__(256) uint32_t lut[kLutBytes / 4];
  union Scratch {
    uint16_t p[kWaves][PB][QR][64];  // weights of a step and block
    float join[kWaves][QR][JW];      // partial outputs, 32 elements at a time
  };
  __shared__ __align__(16) Scratch sh;
  __shared__ float jm[kWaves][QR], jl[kWaves][QR];
  __shared__ int tmp[2][kWaves];
  struct Start {
    SeqSteps q;
    int b, first;  // the sequence, and its first step
  };
  __shared__ Start starts[kWaves];
  const AttnArgs &a = da.a;
  const int tid = threadIdx.x;
  const int wave = uniform(tid >> 6);

  // this wave's steps [cur, end) of the order (sequence, head, step): the
  // lengths are summed up, and the thread whose sequence holds a wave's first
  // step tells it
  const int heads = a.c.heads, units = heads * da.tiles;
  SeqSteps q = {};
  if (tid < a.kb.batch) q = seq_steps(a, tid);
  fill_lut<LO, kThreads>(lut, a.qt, tid);
  int before, total = scan<kWaves>(q.steps, tmp[0], before);
  for (int b0 = kThreads; b0 < a.kb.batch; b0 += kThreads) {
    int unused;
    __syncthreads();
    total += scan<kWaves>(b0 + tid < a.kb.batch ? seq_steps(a, b0 + tid).steps : 0, tmp[0], unused);
  }
  const Runs runs(uniform(total) * units, da.runs);
  const int run_from = runs.from(blockIdx.x), run_to = runs.from(blockIdx.x + 1);
  if (run_from >= run_to) return;
  for (int b0 = 0, base = 0; b0 < a.kb.batch; b0 += kThreads) {
    int sum = 0;
    if (a.kb.batch > kThreads) {
      q = SeqSteps{};
      if (b0 + tid < a.kb.batch) q = seq_steps(a, b0 + tid);
      __syncthreads();
      sum = scan<kWaves>(q.steps, tmp[1], before);
    }
    const int first = (base + before) * units, last = first + q.steps * units;
    if (first < run_to && last > run_from) {
      for (int w = 0; w < kWaves; ++w) {
        const int at = runs.wave_from<kWaves>(blockIdx.x, w);
        if (at >= first && at < last) starts[w] = Start{q, b0 + tid, first};
      }
    }
    base += sum;
  }
  __syncthreads();
  const int wave_run = runs.wave_from<kWaves>(blockIdx.x, wave);
  const int end = runs.wave_from<kWaves>(blockIdx.x, wave + 1);
  int cur = wave_run;
  // whether the run lies in one head, and which
  const int run_steps = uniform(starts[0].q.steps), run_first = uniform(starts[0].first);
  const int run_unit = (run_from - run_first) / run_steps;
  const int run_head0 = run_first + run_unit * run_steps;
  const bool joined = run_to <= run_head0 + run_steps;
  // (a wave of a joined run takes part in it also without a step of its own)
  if (!joined && cur >= end) return;
  const Start &start = starts[joined ? 0 : wave];
  q = uniform(start.q);
  int b = uniform(start.b), first = uniform(start.first);
  const int ps = 1 << a.c.log2page;
  // a page's bytes fit in 31 bits (checked on the host), its number times them
  // does not
  const uint32_t page_codes = (uint32_t)(heads << a.c.log2page) * row_bytes;
  const uint32_t page_scales = (uint32_t)(heads << a.c.log2page) * (2 * NB);

  for (;;) {
    while (q.steps == 0) {  // sequences without tokens
      if (++b >= a.kb.batch) return;
      q = uniform(seq_steps(a, b));
    }
    // what depends on the lane is found anew for each segment: kept over the
    // loop, its registers are spilled
    int lane = tid & 63;
    asm volatile("" : "+v"(lane));
    const int r = lane & 15, g = lane >> 4;
    const uint32_t copy = lut_copy<LO>(lane);
    int koff[KU];  // of key load L: (score tile i, k-step c) = 4 L + g
#pragma unroll
    for (int L = 0; L < KU; ++L) {
      const int i = (4 * L + g) / KU, c = 4 * L + g - i * KU;
      koff[L] = (4 * (r & 3) + i) * row_bytes + 16 * c;
    }
    const int unit = joined ? run_unit : (cur - first) / q.steps;
    const int h = unit / da.tiles, base_row = (unit - h * da.tiles) * 16;
    const int head0 = first + unit * q.steps;
    const int t_from = cur - head0;
    const int t_to = end - head0 < q.steps ? end - head0 : q.steps;
    const int all_rows = q.n * a.group - base_row;  // none in a tile past this sequence's rows
    const int rows = all_rows < 0 ? 0 : (all_rows < 16 ? all_rows : 16);

    // ---- loads of a step ----
    // entries of the block table, loaded unconditionally (a branch around a
    // load waits for it there) and looked at only where they are used
    auto pages = [&](int t) {
      const int t0 = q.lo + t * kStep;
      const int last = a.kb.max_pages - 1;
      const int ig = (t0 + 16 * g) >> a.c.log2page, ik = (t0 + 16 * (r >> 2)) >> a.c.log2page;
      const int32_t *bt = a.kb.bt + (int64_t)b * a.kb.bt_stride;
      return StepPages{bt[ig < last ? ig : last], bt[ik < last ? ik : last]};
    };
    // whether the 16 tokens from tok on have page p
    auto here = [&](int p, int tok) {
      return tok < q.hi && (tok >> a.c.log2page) < a.kb.max_pages && p >= 0 && p < a.c.num_pages;
    };
    const int64_t head_codes = (int64_t)(h << a.c.log2page) * row_bytes;
    const int64_t head_scales = (int64_t)(h << a.c.log2page) * (2 * NB);
    uint4 kc[KU], vc[KU];      // key and value bytes
    uint2 ks[NB], vs[NB];      // scales of the lane's four tokens
    auto load_keys = [&](int t, StepPages p) {
      const int tk = q.lo + t * kStep + 16 * (r >> 2);
      const uint32_t page = here(p.pk, tk) ? p.pk : 0;
      const int at = tk & (ps - 1);
      const uint8_t *base = a.c.kc + head_codes + (uint64_t)page * page_codes + at * row_bytes;
#pragma unroll
      for (int L = 0; L < KU; ++L) kc[L] = *reinterpret_cast<const uint4 *>(base + koff[L]);
      const char *sb = reinterpret_cast<const char *>(a.c.ks) + head_scales + (uint64_t)page * page_scales +
                       2 * at + 8 * (r & 3);
#pragma unroll
      for (int n = 0; n < NB; ++n) ks[n] = *reinterpret_cast<const uint2 *>(sb + 2 * n * ps);
    };
    auto load_values = [&](int t, StepPages p) {
      const int tg = q.lo + t * kStep + 16 * g, tk = q.lo + t * kStep + 16 * (r >> 2);
      const uint32_t page = here(p.pg, tg) ? p.pg : 0, spage = here(p.pk, tk) ? p.pk : 0;
      const uint8_t *base = a.c.vc + head_codes + (uint64_t)page * page_codes + (tg & (ps - 1)) * row_bytes + 16 * r;
#pragma unroll
      for (int c = 0; c < KU; ++c) vc[c] = *reinterpret_cast<const uint4 *>(base + 256 * c);
      const char *sb = reinterpret_cast<const char *>(a.c.vs) + head_scales + (uint64_t)spage * page_scales +
                       2 * (tk & (ps - 1)) + 8 * (r & 3);
#pragma unroll
      for (int n = 0; n < NB; ++n) vs[n] = *reinterpret_cast<const uint2 *>(sb + 2 * n * ps);
    };

    int t = t_from;
    const int t_last = t_to > t_from ? t_to - 1 : t_from;
    StepPages p = pages(t);
    StepPages pn = pages(t + 1 < t_last ? t + 1 : t_last);
    // ---- queries: tile row r, 8 elements of each k-step, in fp16; the scale
    // that takes a product back to powers of two of the softmax ----
    auto query = [&](int row) {
      return static_cast<const uint16_t *>(a.q.p) + (q.s.row0 + row / a.group) * a.q.ts +
             (h * a.group + row % a.group) * a.q.hs;
    };
    const int mine = (r >> 2) * RJ + (r & 3);
    const bool real = (r & 3) < RJ && mine < rows;
    const uint16_t *qrow = query(real ? base_row + mine : 0);
    uint4 raw[KU];
#pragma unroll
    for (int c = 0; c < KU; ++c) raw[c] = *reinterpret_cast<const uint4 *>(qrow + 32 * c + 8 * g);
    float big = 0.f;
    f16x8_t qf[KU];
    {
#pragma unroll
      for (int c = 0; c < KU; ++c) {
        float x[8];
        scales8<DT>(raw[c], x);
#pragma unroll
        for (int j = 0; j < 8; ++j) big = fmaxf(big, fabsf(x[j]));
      }
      big = rows_max(big);
      int e = exponent_of(big);
      e = e < -110 ? -110 : (e > 110 ? 110 : e);
      const float sign = a.scale < 0.f ? -1.f : 1.f;
#pragma unroll
      for (int c = 0; c < KU; ++c) {
        float x[8];
        scales8<DT>(raw[c], x);
        u32x4_t w;
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = f16_pair(sign * ldexpf(x[2 * j], -e), sign * ldexpf(x[2 * j + 1], -e));
        qf[c] = __builtin_bit_cast(f16x8_t, w);
      }
      // at least 2^-100, so that a masked score stays -inf when the scale is 0
      big = fmaxf(ldexpf(fabsf(a.scale) * 1.44269504088896340736f / half_factor(a.qt), e), 0x1p-100f);
    }
    // rows g RJ + j of this lane's scores: their scale, and the keys they see
    float qscale[RJ];
    int lo[RJ], hi[RJ];
#pragma unroll
    for (int j = 0; j < RJ; ++j) {
      qscale[j] = __shfl(big, 4 * g + j);
      const int row = g * RJ + j;
      key_range(a, q.s, row < rows ? (base_row + row) / a.group : 0, lo[j], hi[j]);
      if (row >= rows) lo[j] = hi[j] = 0;
    }
    int all_lo, all_hi, unused;
    key_range(a, q.s, 0, unused, all_hi);        // every row sees keys below all_hi
    key_range(a, q.s, q.n - 1, all_lo, unused);  // and from all_lo on


    load_keys(t, p);
    load_values(t, p);
    f32x4_t acc[KU][2];
#pragma unroll
    for (int c = 0; c < KU; ++c) acc[c][0] = acc[c][1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    float m[RJ], l[RJ];
#pragma unroll
    for (int j = 0; j < RJ; ++j) m[j] = kNoScore, l[j] = 0.f;
    int ev = 100;      // weights are scaled by 2^ev
    bool far = false;  // a row's maximum is_far
    {
      for (; t < t_to; ++t) {
        const int t0 = q.lo + t * kStep;
        const int tn = t + 1 < t_last ? t + 1 : t_last;
        const int tnn = t + 2 < t_last ? t + 2 : t_last;
        const StepPages pnn = pages(tnn);
        // ---- scores of the lane's rows and four tokens ----
        float s[RJ][4];
#pragma unroll
        for (int L = 0; L < KU; ++L) transpose_rows(kc[L]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
          for (int n = 0; n < NB; ++n) {
            f32x4_t x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = n * CB; c < (n + 1) * CB; ++c)
              x = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                  qf[c], lut8(lut, word_of(kc[(i * KU + c) >> 2], (i * KU + c) & 3), copy), x, 0, 0, 0);
            const float f = scale_at<DT>(ks[n], i);
#pragma unroll
            for (int j = 0; j < RJ; ++j) s[j][i] = n == 0 ? x[j] * f : fmaf(x[j], f, s[j][i]);
          }
        }
        // the next step's loads go where this step's words are done with, and
        // not before: a second set of registers would be copied, and a copy
        // waits for the load
        __builtin_amdgcn_sched_barrier(0);
        load_keys(tn, pn);
        __builtin_amdgcn_sched_barrier(0);
        // ---- masks: an unseen token has no score, and its value scale (which
        // may be anything, a NaN too) is 0 ----
        const bool there = here(p.pk, t0 + 16 * (r >> 2));
        const bool whole = t0 >= all_lo && t0 + kStep <= all_hi;
        if (!(whole && __all(there))) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int tok = t0 + 4 * r + i;
            bool any = false;
#pragma unroll
            for (int j = 0; j < RJ; ++j) {
              const bool seen = there && tok >= lo[j] && tok < hi[j];
              s[j][i] = seen ? s[j][i] : -INFINITY;
              any |= seen;
            }
            const uint32_t keep = any ? 0xffffffffu : (i & 1 ? 0x0000ffffu : 0xffff0000u);
#pragma unroll
            for (int n = 0; n < NB; ++n) (i & 2 ? vs[n].y : vs[n].x) &= keep;
          }
        }
        // ---- running maxima ----
        u16x2_t vm = {0, 0};  // magnitudes compare as their bits
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          vm = __builtin_elementwise_max(vm, __builtin_bit_cast(u16x2_t, (uint32_t)vs[n].x));
          vm = __builtin_elementwise_max(vm, __builtin_bit_cast(u16x2_t, (uint32_t)vs[n].y));
        }
        const float vmax = bits16_to_f32<DT>(vm[0] > vm[1] ? vm[0] : vm[1]);
        const bool high = !(ldexpf(vmax, ev) < 0x1p15f);
        bool odd = false;  // the step has a value scale that is not finite: 0 times it is 0
        float top[RJ];
        bool grows = high;
#pragma unroll
        for (int j = 0; j < RJ; ++j) {
          top[j] = fmaxf(fmaxf(s[j][0], s[j][1]), fmaxf(s[j][2], s[j][3]));
          top[j] = row16_max(top[j]) * qscale[j];
          grows |= top[j] > m[j];
        }
        if (__any(grows)) {
          int en = ev;
          if (__any(high)) {
            // a power of two with the largest scale in [2^14, 2^15).  One that is
            // not finite counts for nothing: it is the business of the rows that
            // see it, and its exponent would leave zeros of all else
            odd = __any(vm[0] >= kInf16 || vm[1] >= kInf16);
            uint32_t most = 0;
#pragma unroll
            for (int n = 0; n < NB; ++n) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t x = (i & 2 ? vs[n].y : vs[n].x) >> (i & 1 ? 16 : 0) & 0xffffu;
                most = x < kInf16 && x > most ? x : most;
              }
            }
            const float big = rows_max(group_max(bits16_to_f32<DT>(most), 16));
            if (ldexpf(big, ev) >= 0x1p15f) en = 14 - exponent_of(big);
            en = en < -100 ? -100 : (en > 100 ? 100 : en);
          }
#pragma unroll
          for (int j = 0; j < RJ; ++j) {
            const float mn = fmaxf(m[j], top[j]);
            const float keep = ldexpf(__builtin_amdgcn_exp2f(m[j] - mn), en - ev);
            m[j] = mn;
            l[j] *= keep;
            if (r == 0) jm[wave][g * RJ + j] = keep;
          }
          ev = en;
          far = false;
#pragma unroll
          for (int j = 0; j < RJ; ++j) far |= is_far(m[j]);
          far = __any(far);
          const float keep = jm[wave][r % QR];  // of the output's column
#pragma unroll
          for (int c = 0; c < KU; ++c) {
            acc[c][0] *= keep;
            acc[c][1] *= keep;
          }
        }
        // ---- weights, and the products with the values ----
        if (far) {
#pragma unroll
          for (int j = 0; j < RJ; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[j][i] = s[j][i] * qscale[j] - m[j];
        }
#pragma unroll
        for (int j = 0; j < RJ; ++j) {
          const float f = far ? 1.f : qscale[j], shift = far ? (float)ev : (float)ev - m[j];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[j][i] = __builtin_amdgcn_exp2f(fmaf(s[j][i], f, shift));
            l[j] += s[j][i];
          }
        }
#pragma unroll
        for (int n = 0; n < NB; ++n) {
#pragma unroll
          for (int j = 0; j < RJ; ++j) {
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = s[j][i] * scale_at<DT>(vs[n], i);
            if (odd) {
#pragma unroll
              for (int i = 0; i < 4; ++i) w[i] = s[j][i] == 0.f ? 0.f : w[i];
              asm volatile("" : "+v"(w[0]));  // a branch that is hardly ever taken, not eight selects
            }
            const uint32_t h0 = f16_pair(w[0], w[1]), h1 = f16_pair(w[2], w[3]);
            *reinterpret_cast<uint2 *>(&sh.p[wave][0][g * RJ + j][4 * r]) = make_uint2(h0, h1);
            if constexpr (DT == kF16) {
              // an fp16 result would show the weights' rounding (as large as
              // its own): they keep the bits below fp16 in a second product
              const f16x2v_t a0 = __builtin_bit_cast(f16x2v_t, h0), a1 = __builtin_bit_cast(f16x2v_t, h1);
              *reinterpret_cast<uint2 *>(&sh.p[wave][PB - 1][g * RJ + j][4 * r]) =
                  make_uint2(f16_pair(w[0] - (float)a0[0], w[1] - (float)a0[1]),
                             f16_pair(w[2] - (float)a1[0], w[3] - (float)a1[1]));
            }
          }
          // the wave's own writes, read back in order: 16 tokens of row r
          f16x8_t pf[PB][2];
#pragma unroll
          for (int k = 0; k < PB; ++k)
#pragma unroll
            for (int x = 0; x < 2; ++x)
              pf[k][x] = *reinterpret_cast<const f16x8_t *>(&sh.p[wave][k][r % QR][16 * g + 8 * x]);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int c = n * CB; c < (n + 1) * CB; ++c) {
              const uint32_t w0 = x ? vc[c].z : vc[c].x, w1 = x ? vc[c].w : vc[c].y;
              Pair8 val, rest;
              lut8x2<LO>(lut, w0, w1, copy, val, rest);
#pragma unroll
              for (int k = 0; k < PB; ++k) {
                acc[c][0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(val.even, pf[k][x], acc[c][0], 0, 0, 0);
                acc[c][1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(val.odd, pf[k][x], acc[c][1], 0, 0, 0);
              }
              if constexpr (LO) {
                acc[c][0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(rest.even, pf[0][x], acc[c][0], 0, 0, 0);
                acc[c][1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(rest.odd, pf[0][x], acc[c][1], 0, 0, 0);
              }
            }
          }
        }
        __builtin_amdgcn_sched_barrier(0);
        load_values(tn, pn);
        __builtin_amdgcn_sched_barrier(0);
        p = pn;
        pn = pnn;
      }
    }

    // ---- this segment's sums: l over the lanes, column r's maximum and sum ----
#pragma unroll
    for (int j = 0; j < RJ; ++j) {
      l[j] = ldexpf(row16_sum(l[j]), -ev);
      if (r == 0) {
        jm[wave][g * RJ + j] = m[j];
        jl[wave][g * RJ + j] = l[j];
      }
    }
    const float factor = ldexpf(1.f / half_factor(a.qt), -ev);
    auto out_row = [&](int r) {
      const int row = base_row + r;
      return static_cast<uint16_t *>(a.out.p) + (q.s.row0 + row / a.group) * a.out.ts +
             (h * a.group + row % a.group) * a.out.hs;
    };
    if (joined) {
      // ---- the run lies in this head: its waves' sums together, 32 elements
      // at a time ----
      const bool whole = run_from == head0 && run_to == head0 + q.steps;
      __syncthreads();
      float top = kNoScore;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) top = fmaxf(top, jm[w][r % QR]);
      const float f = factor * __builtin_amdgcn_exp2f(jm[wave][r % QR] - top);
      const int64_t part = (int64_t)(2 * kWaves) * blockIdx.x * QR;
#pragma unroll
      for (int c = 0; c < KU; ++c) {
        if (r < QR) {
          float4 *dst = reinterpret_cast<float4 *>(&sh.join[wave][r][8 * g]);
          dst[0] = make_float4(acc[c][0][0] * f, acc[c][1][0] * f, acc[c][0][1] * f, acc[c][1][1] * f);
          dst[1] = make_float4(acc[c][0][2] * f, acc[c][1][2] * f, acc[c][0][3] * f, acc[c][1][3] * f);
        }
        __syncthreads();
        const int row = tid >> 3, d = 4 * (tid & 7);
        if (row < rows) {
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
          float mx = kNoScore, sum = 0.f;
#pragma unroll
          for (int w = 0; w < kWaves; ++w) {
            const float4 y = *reinterpret_cast<const float4 *>(&sh.join[w][row][d]);
            o.x += y.x, o.y += y.y, o.z += y.z, o.w += y.w;
            mx = fmaxf(mx, jm[w][row]);
          }
#pragma unroll
          for (int w = 0; w < kWaves; ++w) sum += jl[w][row] * __builtin_amdgcn_exp2f(jm[w][row] - mx);
          if (whole) {
            const float inv = sum > 0.f ? 1.f / sum : 0.f;
            *reinterpret_cast<uint2 *>(out_row(row) + 32 * c + d) =
                make_uint2(cvt_pair<DT>(o.x * inv, o.y * inv), cvt_pair<DT>(o.z * inv, o.w * inv));
          } else {
            *reinterpret_cast<float4 *>(da.part.o + (part + row) * D + 32 * c + d) = o;
            if (c == 0 && d == 0) da.part.ml[part + row] = make_float2(mx, sum);
          }
        }
        __syncthreads();
      }
      return;
    }
    // ---- the wave writes them itself ----
    const bool whole = t_from == 0 && t_to == q.steps;
    const float sum = jl[wave][r % QR];
    const float f = factor * (whole ? (sum > 0.f ? 1.f / sum : 0.f) : 1.f);
    const int part = 2 * (kWaves * blockIdx.x + wave) + (cur == wave_run ? 0 : 1);
    if (r < rows) {
#pragma unroll
      for (int c = 0; c < KU; ++c) {
        const float o[8] = {acc[c][0][0] * f, acc[c][1][0] * f, acc[c][0][1] * f, acc[c][1][1] * f,
                            acc[c][0][2] * f, acc[c][1][2] * f, acc[c][0][3] * f, acc[c][1][3] * f};
        if (whole) {
          *reinterpret_cast<uint4 *>(out_row(r) + 32 * c + 8 * g) =
              make_uint4(cvt_pair<DT>(o[0], o[1]), cvt_pair<DT>(o[2], o[3]), cvt_pair<DT>(o[4], o[5]),
                         cvt_pair<DT>(o[6], o[7]));
        } else {
          float4 *dst = reinterpret_cast<float4 *>(da.part.o + ((int64_t)part * QR + r) * D + 32 * c + 8 * g);
          dst[0] = make_float4(o[0], o[1], o[2], o[3]);
          dst[1] = make_float4(o[4], o[5], o[6], o[7]);
        }
      }
      if (!whole && g == 0) da.part.ml[(int64_t)part * QR + r] = make_float2(jm[wave][r], sum);
    }
    cur = head0 + t_to;
    if (cur >= end) return;
    if (cur == first + q.steps * units) {
      first = cur;
      if (++b >= a.kb.batch) return;
      q = uniform(seq_steps(a, b));
    }
  }
}

// The partial sums of a tile of rows joined: grid (cache heads times tiles,
// sequences, sets of `set` query rows).  What a wave or workgroup held whole is
// written.  Bound by latency (the lengths again, then where the parts lie, then
// the parts): 6 to 7 us at the sizes above, 12 to 16 for 32 and 48 rows.  A
// thread sums four elements of a row over every `lists`-th part.
template <int DT>
__global__ __launch_bounds__(64 * kJoinWaves) void attention_join_kernel(DecodeArgs da, int dim, int qr, int set) {
  constexpr int kThreads = 64 * kJoinWaves;
  __shared__ int tmp[3][kJoinWaves];
  __shared__ __align__(16) float4 acc[kThreads];
  __shared__ float acc_l[kThreads];
  __shared__ int where[kMaxRuns + 32];
  __shared__ float row_max[16];
  const AttnArgs &a = da.a;
  const int unit = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const int h = unit / da.tiles, base_row = (unit - h * da.tiles) * 16, units = a.c.heads * da.tiles;
  const SeqSteps q = seq_steps(a, b);
  const int row0 = blockIdx.z * set;
  const int all_rows = q.n * a.group - base_row < 16 ? q.n * a.group - base_row : 16;
  const int rows = all_rows - row0 < set ? all_rows - row0 : set;
  int mine = 0, prior = 0, unused;
  for (int x = tid; x < a.kb.batch; x += kThreads) {
    const int st = seq_steps(a, x).steps;
    mine += st;
    if (x < b) prior += st;
  }
  const int W = decode_waves(dim);
  const Runs runs(scan<kJoinWaves>(mine, tmp[0], unused) * units, da.runs);
  const int start = scan<kJoinWaves>(prior, tmp[1], unused) * units + unit * q.steps, stop = start + q.steps;
  if (rows <= 0) return;
  const int k0 = start / runs.per, k1 = (stop - 1) / runs.per;
  // the parts: up to W waves of the first and of the last workgroup (or one,
  // where its run lies in this head), one of each between
  const int places = 2 * W + (k1 - k0 > 1 ? k1 - k0 - 1 : 0);
  auto part = [&](int x) {
    const int k = x < W ? k0 : (x < 2 * W ? k1 : k0 + 1 + x - 2 * W);
    const int w = x < W ? x : (x < 2 * W ? x - W : 0);
    if (x >= places || (x >= W && x < 2 * W && k0 == k1)) return -1;
    if (runs.from(k) >= start && runs.from(k + 1) <= stop) return w == 0 ? 2 * W * k : -1;
    const int from = runs.from(k), n = runs.from(k + 1) - from;
    const int at = from + (int)((uint32_t)n * (uint32_t)w / W), to = from + (int)((uint32_t)n * (uint32_t)(w + 1) / W);
    if (at >= to || to <= start || at >= stop) return -1;
    return 2 * (W * k + w) + (at >= start ? 0 : 1);
  };
  // at most 2 W + kMaxRuns places: one or two for a thread
  int count = 0;
  for (int x0 = 0; x0 < places; x0 += kThreads) {
    const int p = part(x0 + tid);
    int before;
    if (x0 > 0) __syncthreads();
    const int found = scan<kJoinWaves>(p >= 0, tmp[2], before);
    if (p >= 0) where[count + before] = p;
    count += found;
  }
  if (count <= 1) return;  // written whole
  __syncthreads();
  const int quads = dim / 4, items = rows * quads;
  const int lists = items >= kThreads ? 1 : kThreads / items;
  // rows' maxima: a wave for each row
  for (int row = tid >> 6; row < rows; row += kJoinWaves) {
    float mx = kNoScore;
    for (int k = tid & 63; k < count; k += 64) mx = fmaxf(mx, da.part.ml[(int64_t)where[k] * qr + row0 + row].x);
    mx = rows_max(row16_max(mx));
    if ((tid & 63) == 0) row_max[row] = mx;
  }
  __syncthreads();
  for (int i0 = 0; i0 < items; i0 += kThreads) {
    const int item = i0 + tid % (lists > 1 ? items : kThreads), list = lists > 1 ? tid / items : 0;
    const bool busy = item < items && list < lists;
    const int row = busy ? item / quads : 0, x4 = busy ? item - row * quads : 0;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    if (busy) {
      const float mx = row_max[row];
#pragma unroll 8
      for (int k = list; k < count; k += lists) {
        const int64_t at = (int64_t)where[k] * qr + row0 + row;
        const float2 ml = da.part.ml[at];
        const float4 y = *reinterpret_cast<const float4 *>(da.part.o + at * dim + 4 * x4);
        const float f = __builtin_amdgcn_exp2f(ml.x - mx);
        l = fmaf(f, ml.y, l);
        o.x = fmaf(f, y.x, o.x), o.y = fmaf(f, y.y, o.y), o.z = fmaf(f, y.z, o.z), o.w = fmaf(f, y.w, o.w);
      }
    }
    if (lists > 1) {  // one round: items < kThreads
      acc[tid] = o;
      acc_l[tid] = l;
      __syncthreads();
      if (busy && list == 0) {
        for (int k = 1; k < lists; ++k) {
          const float4 y = acc[k * items + item];
          o.x += y.x, o.y += y.y, o.z += y.z, o.w += y.w;
          l += acc_l[k * items + item];
        }
      }
    }
    if (busy && list == 0) {
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const int m = base_row + row0 + row;
      uint16_t *dst = static_cast<uint16_t *>(a.out.p) + (q.s.row0 + m / a.group) * a.out.ts +
                      (h * a.group + m % a.group) * a.out.hs + 4 * x4;
      *reinterpret_cast<uint2 *>(dst) = make_uint2(cvt_pair<DT>(o.x * inv, o.y * inv), cvt_pair<DT>(o.z * inv, o.w * inv));
    }
  }
}

// Up to 48 query rows are three tiles, each of which goes over the keys by
// itself (mostly out of the caches); the prompt kernel's time is about the same
// for any number of rows up to 256.  Kernels and join, here against there, 16
// sequences of about 4600 tokens, 64 heads over 4 of 128: 16 rows 32 us / 65,
// 32 rows 48 / 66, 48 rows 63 / 68, 64 rows 71 / 69, so no fourth tile; 24
// sequences of 40 rows, 8 heads of 128: 119 / 260, 32 heads of 64 with fp16 and
// a window of 4096: 185 / 384; heads of 256 in the first call, 32 rows in fp16
// 94 / 311, 48 rows in bf16 118 / 194.  Where there are hardly any keys the join
// costs more than it saves (32 prompts of 44 tokens: 14 / 10), the price of a
// rule that does not look at max_kv.  The tiles are those of the largest sequence,
// and one without rows of its own still goes over its keys: one sequence of 48
// rows among 15 of 16 (4600 tokens, 32 heads over 8 of 128) takes 78 us, 16 of 48
// rows 83, 16 of 16 rows 41.
bool decode_eligible(const KVCache &c, int64_t rows) {
  return rows <= 48 && (c.dim == 64 || c.dim == 96 || c.dim == 128 || c.dim == 192 || c.dim == 256);
}

// Query rows that a call's kernel has room for.
static int decode_rows(int rows) { return rows <= 4 ? 4 : rows <= 8 ? 8 : 16; }

static int decode_tiles(int rows) { return (rows + 15) / 16; }

// Workgroups of a call: one for each compute unit, fewer where there cannot be
// that many steps.
static int decode_runs(const KVCache &c, const KVBatch &kb, int rows, int64_t max_kv, int64_t window) {
  int64_t keys = max_kv;
  if (window > 0) keys = std::min<int64_t>(keys, window + kb.max_q + 15);
  const int64_t steps = (int64_t)kb.batch * c.heads * decode_tiles(rows) * ((keys + kStep - 1) / kStep + 1);
  return (int)std::max<int64_t>(1, std::min<int64_t>(std::min(device_cu_count(), kMaxRuns), steps));
}

size_t decode_workspace_bytes(const KVCache &c, const KVBatch &kb, int rows, int64_t max_kv, int64_t window) {
  const size_t parts = (size_t)decode_runs(c, kb, rows, max_kv, window) * 2 * decode_waves(c.dim);
  return parts * decode_rows(rows) * (c.dim + 2) * 4;
}

template <int RJ, int DT, bool LO>
static hipError_t launch_decode_t(const DecodeArgs &da, hipStream_t st) {
  const dim3 grid((unsigned)da.runs);
#define QMV_D(D, CB) hipLaunchKernelGGL((attention_decode_kernel<D, CB, RJ, DT, LO>), grid, dim3(64 * decode_waves(D)), 0, st, da)
  const int cb = da.a.c.bs / 32;
  switch (da.a.c.dim) {
    case 64:
      if (cb == 1) QMV_D(64, 1); else QMV_D(64, 2);
      break;
    case 96: QMV_D(96, 1); break;
    case 128:
      if (cb == 1) QMV_D(128, 1); else if (cb == 2) QMV_D(128, 2); else QMV_D(128, 4);
      break;
    case 192:
      if (cb == 1) QMV_D(192, 1); else QMV_D(192, 2);
      break;
    default:
      if (cb == 1) QMV_D(256, 1); else if (cb == 2) QMV_D(256, 2); else if (cb == 4) QMV_D(256, 4); else QMV_D(256, 8);
  }
#undef QMV_D
  return hipGetLastError();
}

template <int DT>
static hipError_t launch_decode_d(const DecodeArgs &da, hipStream_t st) {
  const int rows = da.a.kb.max_q * da.a.group;
  if (da.a.qt == kNF4) {
    if (rows <= 4) return launch_decode_t<1, DT, true>(da, st);
    if (rows <= 8) return launch_decode_t<2, DT, true>(da, st);
    return launch_decode_t<4, DT, true>(da, st);
  }
  if (rows <= 4) return launch_decode_t<1, DT, false>(da, st);
  if (rows <= 8) return launch_decode_t<2, DT, false>(da, st);
  return launch_decode_t<4, DT, false>(da, st);
}

hipError_t launch_attention_decode(const AttnArgs &a, int dt, void *ws, hipStream_t st) {
  const int rows = a.kb.max_q * a.group;
  DecodeArgs da{a, {}, decode_runs(a.c, a.kb, rows, a.max_kv, a.window), decode_tiles(rows)};
  da.part.o = static_cast<float *>(ws);
  const int qr = decode_rows(rows);
  da.part.ml = reinterpret_cast<float2 *>(da.part.o + (size_t)da.runs * 2 * decode_waves(a.c.dim) * qr * a.c.dim);
  const hipError_t e = dt == kBF16 ? launch_decode_d<kBF16>(da, st) : launch_decode_d<kF16>(da, st);
  if (e != hipSuccess) return e;
  // all rows of a head together, or, where there are few heads and so many
  // parts of each, one by one (196611 tokens, 8 heads of 8 rows: 7 us against 12)
  const int units = a.c.heads * da.tiles, most = std::min(rows, 16);
  const int set = (int64_t)units * a.kb.batch >= device_cu_count() ? most : 1;
  const dim3 grid((unsigned)units, (unsigned)a.kb.batch, (unsigned)((most + set - 1) / set));
  if (dt == kBF16) hipLaunchKernelGGL((attention_join_kernel<kBF16>), grid, dim3(64 * kJoinWaves), 0, st, da, a.c.dim, qr, set);
  else hipLaunchKernelGGL((attention_join_kernel<kF16>), grid, dim3(64 * kJoinWaves), 0, st, da, a.c.dim, qr, set);
  return hipGetLastError();
}

}  // namespace qmv
