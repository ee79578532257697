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
__device__ __forceinline__ void load8(const uint16_t *p, float (&x)[8]) {
  const uint4 w = *reinterpret_cast<const uint4 *>(p);
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bits16_to_f32<DT>(u[i] & 0xffffu);
    x[2 * i + 1] = bits16_to_f32<DT>(u[i] >> 16);
  }
}

// Elements e0 .. e0 + 7 of a row turned by the table row cs (half pairs), or
// zeros where there is no table row.
template <int DT>
__device__ __forceinline__ void turn8(const uint16_t *row, int e0, const Rope &rope, int64_t pos,
                                      float (&x)[8]) {
  if (pos < 0 || pos >= rope.max_pos) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
    return;
  }
  const float2 *cs = rope.table + pos * rope.half;
  const int half = rope.half;
  if (rope.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = (e0 >> 1) + i;
      if (p < half) {
        const float2 v = cs[p];
        const float a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = a * v.x - b * v.y;
        x[2 * i + 1] = b * v.x + a * v.y;
      }
    }
  } else if (e0 < 2 * half) {
    float y[8];
    const bool whole = half % 8 == 0;  // the run's partners are one aligned run
    if (whole) load8<DT>(row + (e0 < half ? e0 + half : e0 - half), y);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = e0 + i;
      if (e >= 2 * half) continue;
      const bool first = e < half;
      const float o = whole ? y[i] : bits16_to_f32<DT>(row[first ? e + half : e - half]);
      const float2 v = cs[first ? e : e - half];
      x[i] = first ? x[i] * v.x - o * v.y : x[i] * v.x + o * v.y;
    }
  }
}

// Token of the sequence (and row h of it) that this thread's LPR lanes take:
// rows are numbered through over the tokens, in 64 bits.
template <int LPR>
__device__ __forceinline__ int unit_token(int rows, int &h) {
  const int64_t first = (int64_t)blockIdx.x * (256 / LPR);
  const int64_t i0 = first / rows;
  const uint32_t u = (uint32_t)(first - i0 * rows) + threadIdx.x / LPR;
  h = (int)(u % (uint32_t)rows);
  return (int)(i0 + u / (uint32_t)rows);
}

struct AppendArgs {
  KVCache c;
  KVBatch kb;
  Heads k, v, q, qo;  // q.heads 0: no queries
  Rope rope;          // table NULL: not turned
  Mids32 mids;
};

// A row takes LPR lanes of a wave, 8 elements each (the first head_dim / 8
// lanes hold some); rows of a token: its queries, its keys, its values.
template <int DT, int QT, int LPR>
__global__ __launch_bounds__(256) void kv_append_kernel(AppendArgs a) {
  const int b = blockIdx.y;
  const SeqRange s = seq_range(a.kb, b);
  const int rows = a.q.heads + 2 * a.c.heads;
  int h;
  const int i = unit_token<LPR>(rows, h);
  if (i >= s.n || i >= a.kb.max_q) return;
  const int l = threadIdx.x % LPR;
  const int e0 = 8 * l;
  const int pos = s.pos0 + i;
  const int64_t t = s.row0 + i;
  const bool isq = h < a.q.heads;
  if (!isq) h -= a.q.heads;
  const bool isv = !isq && h >= a.c.heads;
  if (isv) h -= a.c.heads;
  const Heads &src = isq ? a.q : (isv ? a.v : a.k);
  const uint16_t *row = static_cast<const uint16_t *>(src.p) + t * src.ts + h * src.hs;
  const bool mine = e0 < a.c.dim;

  float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (mine) {
    load8<DT>(row + e0, x);
    if (!isv && a.rope.table) turn8<DT>(row, e0, a.rope, pos, x);
  }
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = cvt_pair<DT>(x[2 * j], x[2 * j + 1]);
  if (isq) {
    if (mine)
      *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.qo.p) + t * a.qo.ts + h * a.qo.hs + e0) =
          make_uint4(w[0], w[1], w[2], w[3]);
    return;
  }
  const int64_t page = page_of(a.kb, a.c, b, pos);
  if (page < 0) return;  // the same for the whole row
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {  // what is quantized: the row as the cache's type holds it
    x[2 * j] = bits16_to_f32<DT>(w[j] & 0xffffu);
    x[2 * j + 1] = bits16_to_f32<DT>(w[j] >> 16);
    m = fmaxf(m, fmaxf(fabsf(x[2 * j]), fabsf(x[2 * j + 1])));
  }
  m = group_max(m, a.c.bs >> 3);
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
  if (!mine) return;
  const int at = pos & ((1 << a.c.log2page) - 1);
  const int64_t cb = code_base(a.c, page, h);
  if (isv) {
    uint8_t *dst = a.c.vc + cb + (int64_t)(at >> 4) * a.c.dim * 8 + (e0 >> 1) * 16 + (at & 15);
#pragma unroll
    for (int j = 0; j < 4; ++j) dst[16 * j] = (uint8_t)(word >> (8 * j));
  } else {
    *reinterpret_cast<uint32_t *>(a.c.kc + cb + (int64_t)at * (a.c.dim >> 1) + (e0 >> 1)) = word;
  }
  if ((e0 & (a.c.bs - 1)) == 0) {
    uint16_t *sc = isv ? a.c.vs : a.c.ks;
    sc[scale_base(a.c, page, h) + ((int64_t)(e0 / a.c.bs) << a.c.log2page) + at] =
        (uint16_t)f32_to_bits16<DT>(m);
  }
}

// Lanes of a row: head_dim / 8 rounded up to a power of two.
static int row_lanes(int dim) { return dim <= 32 ? 4 : dim <= 64 ? 8 : dim <= 128 ? 16 : 32; }

template <int DT, int QT>
static void launch_append_t(const AppendArgs &a, hipStream_t st) {
  const int lpr = row_lanes(a.c.dim);
  const int64_t units = (int64_t)a.kb.max_q * (a.q.heads + 2 * a.c.heads);
  const dim3 grid((unsigned)((units * lpr + 255) / 256), (unsigned)a.kb.batch);
  switch (lpr) {
    case 4: hipLaunchKernelGGL((kv_append_kernel<DT, QT, 4>), grid, dim3(256), 0, st, a); break;
    case 8: hipLaunchKernelGGL((kv_append_kernel<DT, QT, 8>), grid, dim3(256), 0, st, a); break;
    case 16: hipLaunchKernelGGL((kv_append_kernel<DT, QT, 16>), grid, dim3(256), 0, st, a); break;
    default: hipLaunchKernelGGL((kv_append_kernel<DT, QT, 32>), grid, dim3(256), 0, st, a);
  }
}

hipError_t launch_kv_append(const KVCache &c, int dt, int qt, const Midpoints4 &mids,
                            const KVBatch &kb, const Heads &k, const Heads &v, const Rope &rope,
                            const Heads &q, const Heads &qo, hipStream_t st) {
  AppendArgs a{c, kb, k, v, q, qo, rope, {}};
  for (int j = 0; j < 15; ++j) a.mids.m[j] = (float)mids.mid[qt == kNF4 ? j : std::min(7 + j, 13)];
  if (dt == kBF16) {
    if (qt == kNF4) launch_append_t<kBF16, kNF4>(a, st);
    else launch_append_t<kBF16, kFP4>(a, st);
  } else {
    if (qt == kNF4) launch_append_t<kF16, kNF4>(a, st);
    else launch_append_t<kF16, kFP4>(a, st);
  }
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Reading back: fp32(T[code] * a) rounded to the cache's type.
// ---------------------------------------------------------------------------
struct ReadArgs {
  KVCache c;
  KVBatch kb;
  Heads k, v;
};

template <int DT, int LPR>
__global__ __launch_bounds__(256) void kv_dequantize_kernel(ReadArgs a, int qt) {
  __shared__ float2 lut[256];  // packed byte -> (T[byte >> 4], T[byte & 15])
  {
    const uint32_t *tb = table_bits(qt);
    lut[threadIdx.x] = make_float2(__uint_as_float(tb[threadIdx.x >> 4]),
                                   __uint_as_float(tb[threadIdx.x & 15]));
  }
  __syncthreads();
  const int b = blockIdx.y;
  const SeqRange s = seq_range(a.kb, b);
  const int rows = 2 * a.c.heads;
  int h;
  const int i = unit_token<LPR>(rows, h);
  const int e0 = 8 * (threadIdx.x % LPR);
  if (i >= s.n || i >= a.kb.max_q || e0 >= a.c.dim) return;
  const bool isv = h >= a.c.heads;
  if (isv) h -= a.c.heads;
  const int pos = s.pos0 + i;
  const int64_t page = page_of(a.kb, a.c, b, pos);
  uint32_t out[4] = {0, 0, 0, 0};
  if (page >= 0) {
    const int at = pos & ((1 << a.c.log2page) - 1);
    const int64_t cb = code_base(a.c, page, h);
    uint32_t word = 0;
    if (isv) {
      const uint8_t *src = a.c.vc + cb + (int64_t)(at >> 4) * a.c.dim * 8 + (e0 >> 1) * 16 + (at & 15);
#pragma unroll
      for (int j = 0; j < 4; ++j) word |= (uint32_t)src[16 * j] << (8 * j);
    } else {
      word = *reinterpret_cast<const uint32_t *>(a.c.kc + cb + (int64_t)at * (a.c.dim >> 1) + (e0 >> 1));
    }
    const uint16_t *sc = isv ? a.c.vs : a.c.ks;
    const float m = bits16_to_f32<DT>(
        sc[scale_base(a.c, page, h) + ((int64_t)(e0 / a.c.bs) << a.c.log2page) + at]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 v = lut[(word >> (8 * j)) & 0xffu];
      out[j] = cvt_pair<DT>(v.x * m, v.y * m);
    }
  }
  const Heads &dst = isv ? a.v : a.k;
  *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(dst.p) + (s.row0 + i) * dst.ts + h * dst.hs + e0) =
      make_uint4(out[0], out[1], out[2], out[3]);
}

template <int DT>
static void launch_read_t(const ReadArgs &a, int qt, hipStream_t st) {
  const int lpr = row_lanes(a.c.dim);
  const int64_t units = (int64_t)a.kb.max_q * 2 * a.c.heads;
  const dim3 grid((unsigned)((units * lpr + 255) / 256), (unsigned)a.kb.batch);
  switch (lpr) {
    case 4: hipLaunchKernelGGL((kv_dequantize_kernel<DT, 4>), grid, dim3(256), 0, st, a, qt); break;
    case 8: hipLaunchKernelGGL((kv_dequantize_kernel<DT, 8>), grid, dim3(256), 0, st, a, qt); break;
    case 16: hipLaunchKernelGGL((kv_dequantize_kernel<DT, 16>), grid, dim3(256), 0, st, a, qt); break;
    default: hipLaunchKernelGGL((kv_dequantize_kernel<DT, 32>), grid, dim3(256), 0, st, a, qt);
  }
}

hipError_t launch_kv_dequantize(const KVCache &c, int dt, int qt, const KVBatch &kb,
                                const Heads &k, const Heads &v, hipStream_t st) {
  const ReadArgs a{c, kb, k, v};
  if (dt == kBF16) launch_read_t<kBF16>(a, qt, st);
  else launch_read_t<kF16>(a, qt, st);
  return hipGetLastError();
}

}  // namespace qmv
