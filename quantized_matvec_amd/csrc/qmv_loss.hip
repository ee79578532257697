// Losses over a 4-bit vocabulary projection (include/qmv/tuning.h): softmax
// cross entropy, and the divergence from a teacher's largest logits.
//
// With l = W^ x / tau and a target distribution p on a few ids,
//   loss = sum_j p_j (log p_j - l_j) + log sum_v exp l_v
//   dx   = dloss / tau (sum_v q_v W^_v - sum_j p_j W^_j),   q = softmax(l).
// The vocabulary is taken in pieces.  A piece's logits are a product, kept in
// fp32; over the pieces run the maximum m and the sum s of exp(l - m), and,
// with a gradient, D = sum_v exp(l_v - m) W^_v, which is multiplied by
// exp(m_old - m_new) before a piece is added (one pass: the logits are computed
// once).  The target ids stay out of m, s and D: their logits are kept, and
// at the end q_j - p_j times their rows is added in fp32.  So the gradient of a
// token whose target is all but certain keeps its precision (1 - q is
// computed from s, not by subtracting), and a type with few exponent bits
// does not flush the rest of the vocabulary against the target's logit.
#include "qmv_tile.hpp"

namespace qmv {

constexpr int kSegment = 8192;   // columns of a logits row that a workgroup takes
constexpr int64_t kTokens = 4096;  // most tokens taken at a time
constexpr int kTail = 64;
constexpr int kMostPiece = 32768;   // of the tile product's pieces
constexpr int64_t kTiledFrom = 448;  // tokens from which it is used
constexpr int64_t kLogits = (int64_t)1 << 26;  // logits of a piece where it is not, all slices of the sum together

// What exp(l - m) is multiplied by before its rounding.  fp16 has no normal
// numbers below 2^-14: with 2^14 (sums are fp32, and D is divided by it at the
// end) terms keep their 11 bits down to 2^-28 of the largest.
template <int DT>
constexpr float kGain = DT == kF16 ? 16384.f : 1.f;

struct RowState {
  float *m, *s, *f;  // running maximum, sum, and the factor of what D held before this piece
  float *lt;         // [T, k] logits of the target ids
  float *tail;       // [T, 64] logits of the last V % 64 columns (-inf: none, or a target)
};

// ---------------------------------------------------------------------------
// Which tokens count (an id in [0, V) with a logit above -inf): one wave a token,
// then the tokens that do, in order, followed by the others, and their number.
// Many tokens: the others are left out of the products.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float teacher_logit(const void *teacher, int dt, int64_t i) {
  return dt == kF32 ? static_cast<const float *>(teacher)[i]
         : dt == kF16 ? bits16_to_f32<kF16>(static_cast<const uint16_t *>(teacher)[i])
                      : bits16_to_f32<kBF16>(static_cast<const uint16_t *>(teacher)[i]);
}

__global__ __launch_bounds__(256) void loss_live_kernel(const int64_t *__restrict__ ids, const void *teacher,
                                                        int teacher_dt, int k, int64_t V, int T, int32_t *__restrict__ live) {
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (t >= T) return;
  bool any = false;
  for (int j = lane; j < k; j += 64) {
    const int64_t v = ids[(int64_t)t * k + j];
    if (v >= 0 && v < V) any |= !teacher || !(teacher_logit(teacher, teacher_dt, (int64_t)t * k + j) == -INFINITY);
  }
  const bool on = __ballot(any) != 0;
  if (lane == 0) live[t] = on;
}

__global__ __launch_bounds__(1024) void loss_order_kernel(const int32_t *__restrict__ live, int T,
                                                          int32_t *__restrict__ list, int32_t *__restrict__ count) {
  __shared__ int before[17];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int each = (T + 1023) / 1024, t0 = threadIdx.x * each, t1 = min(t0 + each, T);
  int mine = 0;
  for (int t = t0; t < t1; ++t) mine += live[t];
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 63) before[wave + 1] = upto;
  if (threadIdx.x == 0) before[0] = 0;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int w = 0; w < 16; ++w) before[w + 1] += before[w];
  __syncthreads();
  const int total = before[16];
  int at = before[wave] + upto - mine;  // tokens before t0 that count
  for (int t = t0; t < t1; ++t) {
    const bool on = live[t];
    list[on ? at : total + t - at] = t;
    at += on;
  }
  if (threadIdx.x == 0) *count = total;
}

template <class F>
__device__ __forceinline__ float block_reduce(float v, float *buf, F op) {  // 256 threads
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) buf[wave] = v;
  __syncthreads();
  v = op(op(buf[0], buf[1]), op(buf[2], buf[3]));
  __syncthreads();
  return v;
}

// ---------------------------------------------------------------------------
// Few tokens: a token's logits are shared out among workgroups of 8192 columns.
// loss_part_kernel leaves each segment's maximum and sum (and takes the target ids'
// logits); loss_merge_kernel puts them together with what was before the piece
// and, with a gradient, writes P = exp(l - m) in 16 bits, [T, np] with np the
// multiple of 64 below n (the columns from np on go to `tail`).  Two launches,
// but no workgroup reads more than 32 kB: 17 tokens x 32000 5.9 and 2.5 us, 96 x 32003 with P 7.4 and 11.7.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void mark_ids(uint32_t *out, const int64_t *ids, int k, int64_t v0, int n) {  // one barrier
  for (int j = threadIdx.x; j < k; j += 256) {
    const int64_t c = ids[j] - v0;
    if (c >= 0 && c < n) atomicOr(&out[c >> 5], 1u << (c & 31));
  }
  __syncthreads();
}

__global__ __launch_bounds__(256) void loss_part_kernel(const float *__restrict__ logits, int64_t v0, int n,
                                                        const int64_t *__restrict__ ids, int k, float inv_tau,
                                                        float *__restrict__ lt, float2 *__restrict__ segments) {
  __shared__ uint32_t out[kSegment / 32];  // columns of target ids
  __shared__ float buf[4];
  const int64_t t = blockIdx.y;
  const int c0 = blockIdx.x * kSegment, cols = min(n - c0, kSegment);
  const float *row = logits + t * n + c0;
  out[threadIdx.x] = 0;
  float l[32];
#pragma unroll
  for (int q = 0; q < 32; ++q) l[q] = row[min(256 * q + (int)threadIdx.x, cols - 1)] * inv_tau;
  __syncthreads();
  mark_ids(out, ids + t * k, k, v0 + c0, cols);
  for (int j = threadIdx.x; j < k; j += 256) {
    const int64_t c = ids[t * k + j] - v0 - c0;
    if (c >= 0 && c < cols) lt[t * k + j] = row[c] * inv_tau;
  }
  float m = -INFINITY;
#pragma unroll
  for (int q = 0; q < 32; ++q) {
    const int c = 256 * q + threadIdx.x;
    if (c >= cols || (out[c >> 5] >> (c & 31) & 1)) l[q] = -INFINITY;
    m = fmaxf(m, l[q]);
  }
  m = block_reduce(wave_max(m), buf, [](float a, float b) { return fmaxf(a, b); });
  const float ref = m == -INFINITY ? 0.f : m;
  float s = 0.f;
#pragma unroll
  for (int q = 0; q < 32; ++q) s += __expf(l[q] - ref);
  s = block_reduce(wave_sum(s), buf, [](float a, float b) { return a + b; });
  if (threadIdx.x == 0) segments[t * gridDim.x + blockIdx.x] = make_float2(m, s);
}

// before, after: (maximum, sum) of each token before and after this piece
template <int DT, bool GRAD>
__global__ __launch_bounds__(256) void loss_merge_kernel(const float *__restrict__ logits, int64_t v0, int n, int np,
                                                         const int64_t *__restrict__ ids, int k, float inv_tau, bool first,
                                                         const float2 *__restrict__ segments, int n_segments,
                                                         const float2 *__restrict__ before, float2 *__restrict__ after,
                                                         RowState rs, uint16_t *__restrict__ P) {
  __shared__ uint32_t out[kSegment / 32];
  const int64_t t = blockIdx.y;
  const int c0 = blockIdx.x * kSegment, cols = min(n - c0, kSegment);
  const float *row = logits + t * n + c0;
  const float2 old = first ? make_float2(-INFINITY, 0.f) : before[t];
  float m = old.x;
  for (int i = 0; i < n_segments; ++i) m = fmaxf(m, segments[t * n_segments + i].x);
  const float ref = m == -INFINITY ? 0.f : m;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    const float f = __expf(old.x - ref);  // 0 at first
    float s = old.y * f;
    for (int i = 0; i < n_segments; ++i) {
      const float2 seg = segments[t * n_segments + i];
      s += seg.y * __expf(seg.x - ref);
    }
    after[t] = make_float2(m, s);
    rs.m[t] = m;
    rs.s[t] = s;
    rs.f[t] = f;
  }
  if constexpr (GRAD) {
    out[threadIdx.x] = 0;
    __syncthreads();
    mark_ids(out, ids + t * k, k, v0 + c0, cols);
#pragma unroll 8
    for (int q = 0; q < 32; ++q) {
      const int c = 256 * q + threadIdx.x;
      if (c >= cols) break;
      const bool gone = out[c >> 5] >> (c & 31) & 1;
      const float l = gone ? -INFINITY : row[c] * inv_tau;
      if (c0 + c < np) P[t * np + c0 + c] = (uint16_t)f32_to_bits16<DT>(__expf(l - ref) * kGain<DT>);
      else rs.tail[t * kTail + c0 + c - np] = l;
    }
    if (c0 + cols == n && (int)threadIdx.x < np - n) P[t * np + n + threadIdx.x] = 0;
  }
}

// D = D f + what a piece adds (nothing: NULL), f of the row; `first`: D = 0
__global__ __launch_bounds__(256) void loss_add_kernel(float *__restrict__ D, const float *__restrict__ add,
                                                       const float *__restrict__ f, int64_t K, bool first) {
  const int64_t t = blockIdx.x;
  const float ft = f[t];
  for (int64_t c = threadIdx.x; c < K; c += 256) {
    const int64_t i = t * K + c;
    D[i] = first ? 0.f : fmaf(D[i], ft, add ? add[i] : 0.f);
  }
}

// The loss of a token, and its row of dx from D: a workgroup a token.  Bound by D's read for one id (4096 tokens x 4096
// 37 us), by the ids' rows of codes, scattered over the weight, for many (2048 tokens x 64 ids x 4096 161 us: 268 MB).
template <int DT, int LDT, bool DQ>
__global__ __launch_bounds__(256) void loss_finish_kernel(const int64_t *__restrict__ ids, const void *teacher,
                                                          int teacher_dt, int k, float inv_tau, int64_t V, RowState rs,
                                                          int tail_n, const float *__restrict__ D, int parts,
                                                          int64_t part, int64_t K, const int32_t *list,
                                                          const uint8_t *__restrict__ packed, Scales sc, int log2bs,
                                                          CodeValues table, const float *__restrict__ dloss,
                                                          typename Storage<LDT>::type *__restrict__ loss,
                                                          uint16_t *__restrict__ dx) {
  __shared__ float z[128], p[128], lt[128], each[128], coef[128 + kTail], tab[16], buf[4], by_block[64][64];
  __shared__ int64_t id[128 + kTail];
  const int64_t i = blockIdx.x;             // its place among the rows of D and rs
  const int64_t t = list ? list[i] : i;
  const int tid = threadIdx.x;
  if (tid < 16) tab[tid] = table.v[tid];
  // the target distribution; an entry that repeats an earlier id lends that
  // one its p, and is no entry of its own for q
  bool there = false, own = false;
  if (tid < k) {
    const int64_t v = ids[t * k + tid];
    there = v >= 0 && v < V;
    id[tid] = there ? v : -1;
    z[tid] = !there ? -INFINITY : teacher ? teacher_logit(teacher, teacher_dt, t * k + tid) : 0.f;
  }
  __syncthreads();
  const auto most = [](float a, float b) { return fmaxf(a, b); };
  const auto both = [](float a, float b) { return a + b; };
  const float mz = tid < k ? z[tid] : -INFINITY;
  if (!__syncthreads_or(!(mz == -INFINITY))) {  // no entry (a NaN counts, and p is NaN then)
    if (tid == 0) store_elem<LDT>(loss, t, 0.f);
    if (dx)
      for (int64_t c = tid; c < K; c += 256) dx[t * K + c] = 0;
    return;
  }
  const float ml = there ? rs.lt[i * k + tid] : -INFINITY;
  const float zm = block_reduce(wave_max(mz), buf, most);
  // the difference before the temperature: a type's lowest value may not be divided by it
  const float dz = (mz - zm) * inv_tau, ez = tid < k ? expf(dz) : 0.f;
  const float zs = block_reduce(wave_sum(ez), buf, both);
  if (tid < k) {
    lt[tid] = ml;
    p[tid] = ez / zs;
    own = there;
#pragma unroll 8
    for (int j = 0; j < tid; ++j) own &= id[j] != id[tid];
  }
  // the loss
  const float m = rs.m[i];
  const float M = fmaxf(m, block_reduce(wave_max(ml), buf, most));
  const float rest = rs.s[i] * (m == -INFINITY ? 0.f : expf(m - M));
  const float mine = own ? expf(ml - M) : 0.f;
  const float targets = block_reduce(wave_sum(mine), buf, both);
  const float Z = rest + targets;
  if (!teacher) {
    // (M - l) + log Z; where the target is the largest that is log(1 + rest)
    if (tid == 0) store_elem<LDT>(loss, t, lt[0] == M ? log1pf(rest) : (M - lt[0]) + logf(Z));
  } else {
    float part = 0.f;
    if (tid < k && p[tid] != 0.f) part = p[tid] * ((dz - logf(zs)) - (ml - M) + logf(Z));
    part = block_reduce(wave_sum(part), buf, both);
    if (tid == 0) store_elem<LDT>(loss, t, part);
  }
  if (!dx) return;
  // q - p of every id; by the complements where both are near 1
  if (tid < k) each[tid] = mine;
  __syncthreads();
  if (tid < k) {
    float c = 0.f;
    if (own) {
      float pj = 0.f, others_p = 0.f, others_q = rest;
#pragma unroll 4
      for (int j = 0; j < k; ++j) {
        const bool same = id[j] == id[tid];
        pj += same ? p[j] : 0.f;
        others_p += same ? 0.f : p[j];
        others_q += same ? 0.f : each[j];
      }
      c = pj > 0.5f ? others_p - others_q / Z : mine / Z - pj;
    }
    coef[tid] = c;
  }
  if (tid >= 128 && tid < 128 + kTail) {
    const int j = tid - 128;
    const float l = j < tail_n ? rs.tail[i * kTail + j] : -INFINITY;
    coef[k + j] = l == -INFINITY ? 0.f : expf(l - M) / Z;
    id[k + j] = V - tail_n + j;
  }
  __syncthreads();
  const float gain = dloss[t] * inv_tau;
  const float scale = m == -INFINITY ? 0.f : expf(m - M) / Z / kGain<DT>;
  const float offset = DQ ? sc.offset[0] : 0.f;
  const int entries = k + tail_n;
  // 2048 columns at a time, 8 a thread; 64 entries at a time have their coefficients
  // times the scales of their blocks (32 columns at least) in LDS, eight rows are in flight
  for (int64_t base = 0; base < K; base += 2048) {
    const int64_t c = base + tid * 8;
    const bool in = c < K;
    float acc[8] = {};
    if (in) {
      for (int s = 0; s < parts; ++s) {
        const float4 *d = reinterpret_cast<const float4 *>(D + s * part + i * K + c);
        const float4 u = d[0], v = d[1];
        acc[0] += u.x, acc[1] += u.y, acc[2] += u.z, acc[3] += u.w;
        acc[4] += v.x, acc[5] += v.y, acc[6] += v.z, acc[7] += v.w;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] *= scale;
    }
    const int log2sub = log2bs < 11 ? log2bs : 11, log2n = 11 - log2sub;  // blocks in the columns: 2^log2n
    for (int j0 = 0; j0 < entries; j0 += 64) {
      const int some = min(entries - j0, 64);
      __syncthreads();
#pragma unroll 4
      for (int b = tid; b < some << log2n; b += 256) {
        const int at = b & ((1 << log2n) - 1), j = j0 + (b >> log2n);
        const int64_t col = base + ((int64_t)at << log2sub);
        const float cj = coef[j];
        by_block[b >> log2n][at] =
            cj == 0.f || col >= K ? 0.f : cj * block_scale<DQ>(sc, (id[j] * K + col) >> log2bs, offset);
      }
      __syncthreads();
      if (!in) continue;
      for (int j1 = 0; j1 < some; j1 += 8) {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int j = j1 + e;
          w[e] = j < some && coef[j0 + j] != 0.f ? *reinterpret_cast<const uint32_t *>(packed + (id[j0 + j] * K + c) / 2) : 0;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float a = j1 + e < some ? by_block[j1 + e][(8 * tid) >> log2sub] : 0.f;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            acc[2 * x] = fmaf(a, tab[w[e] >> (8 * x + 4) & 15], acc[2 * x]);
            acc[2 * x + 1] = fmaf(a, tab[w[e] >> (8 * x) & 15], acc[2 * x + 1]);
          }
        }
      }
    }
    if (!in) continue;
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = cvt_pair<DT>(acc[2 * e] * gain, acc[2 * e + 1] * gain);
    *reinterpret_cast<uint4 *>(dx + t * K + c) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// ---------------------------------------------------------------------------
// Many tokens: a piece's logits and D by the tile product.
//
// One row of a piece in the registers of a workgroup of 256, 512 or 1024 threads,
// 32 columns each; rows are those that count, list[i] the token of row i.  One read of
// the logits: 2867 rows x 16384 59.5 us with P, 282 MB at 4.7 TB/s; 2048 rows without 31 us.
// ---------------------------------------------------------------------------
template <int DT, bool GRAD>
__global__ __launch_bounds__(1024) void loss_rows_kernel(const float *__restrict__ logits, int64_t ld, int64_t v0, int n,
                                                         int np, const int64_t *__restrict__ ids, int k, float inv_tau,
                                                         bool first, RowState rs, const int32_t *__restrict__ list,
                                                         const int32_t *__restrict__ count, uint16_t *__restrict__ P) {
  __shared__ uint32_t out[kMostPiece / 32];  // columns of target ids
  __shared__ float buf[2][16];
  const int64_t i = blockIdx.x;
  if (i >= *count) return;
  const int64_t t = list[i];
  const int tid = threadIdx.x, threads = blockDim.x, waves = threads >> 6;
  const float *row = logits + i * ld;
  for (int c = tid; c < threads; c += threads) out[c] = 0;  // 32 columns a thread
  float l[8][4];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int c = 4 * (q * threads + tid);
    float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    if (c + 3 < n) {
      v = *reinterpret_cast<const float4 *>(row + c);
    } else if (c < n) {
      v.x = row[c];
      if (c + 1 < n) v.y = row[c + 1];
      if (c + 2 < n) v.z = row[c + 2];
    }
    l[q][0] = v.x * inv_tau, l[q][1] = v.y * inv_tau, l[q][2] = v.z * inv_tau, l[q][3] = v.w * inv_tau;
  }
  __syncthreads();
  for (int j = tid; j < k; j += threads) {
    const int64_t c = ids[t * k + j] - v0;
    if (c >= 0 && c < n) {
      atomicOr(&out[c >> 5], 1u << (c & 31));
      rs.lt[i * k + j] = row[c] * inv_tau;
    }
  }
  __syncthreads();
  float m = -INFINITY;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int c = 4 * (q * threads + tid);
    const uint32_t gone = out[c >> 5] >> (c & 31) & 15;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (gone >> e & 1) l[q][e] = -INFINITY;
      m = fmaxf(m, l[q][e]);
    }
  }
  m = wave_max(m);
  if ((tid & 63) == 0) buf[0][tid >> 6] = m;
  __syncthreads();
  for (int w = 0; w < waves; ++w) m = fmaxf(m, buf[0][w]);
  const float m_old = first ? -INFINITY : rs.m[i];
  m = fmaxf(m, m_old);
  const float ref = m == -INFINITY ? 0.f : m;  // no column yet: exp(-inf) = 0
  float s = 0.f;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int c = 4 * (q * threads + tid);
    float e[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      e[x] = __expf(l[q][x] - ref);
      s += e[x];
    }
    if constexpr (GRAD)
      if (c < np)  // np is a multiple of 64; past n: zeros
        *reinterpret_cast<uint2 *>(P + i * np + c) = make_uint2(cvt_pair<DT>(e[0] * kGain<DT>, e[1] * kGain<DT>),
                                                                cvt_pair<DT>(e[2] * kGain<DT>, e[3] * kGain<DT>));
  }
  s = wave_sum(s);
  if ((tid & 63) == 0) buf[1][tid >> 6] = s;
  __syncthreads();
  if (tid == 0) {
    s = 0.f;
    for (int w = 0; w < waves; ++w) s += buf[1][w];
    const float f = m_old == -INFINITY ? 0.f : __expf(m_old - m);
    rs.s[i] = (first ? 0.f : rs.s[i] * f) + s;
    rs.m[i] = m;
    rs.f[i] = f;
  }
}

// D = D f + sums, the part of this workgroup's terms
struct EpilogueAdd : EpilogueBase {
  static constexpr bool kPlain = true, kAdds = true;
  float *C;
  const float *f;
  int64_t ld, part;
  bool first;
  __device__ __forceinline__ float *row(int m) const { return C + blockIdx.y * part + m * ld; }
  __device__ __forceinline__ void store(float *, int, float) const {}
};

// ---------------------------------------------------------------------------
struct LossPlan {
  bool tiled, mixed;
  int64_t tokens, Kp;  // taken at a time; K up to a multiple of 64
  int piece, parts, split;
  size_t x, logits, m, s, f, lt, tail, P, D, add, back, segments, carry, live, list, count, W, Wt, total;
};

static LossPlan loss_plan(int64_t T, int64_t V, int64_t K, int log2bs, int k, bool grad) {
  LossPlan p{};
  Carver c;
  // The tile product from many tokens on: both sides, us with the gradient, by it / by gemm_4bit's kernels: 256 tokens
  // x 128256 x 4096 1488 / 848, 448 tokens 1663 / 1584, 512 tokens 1680 / 1665, and the latter grows with every
  // token.  Fewer tokens where the backward has no kernel that divides the sum: gemm_4bit's logits, and D by the
  // tile product: 1 token x 29158 x 640 87 / 404, 223 tokens x 56425 x 1152 263 / 832.
  const int64_t turns = (T + kTokens - 1) / kTokens;
  p.tokens = (T + turns - 1) / turns;
  p.tiled = K <= 65536 && T >= kTiledFrom;
  p.mixed = K <= 65536 && !p.tiled && grad && !fast_backward(p.tokens, V & ~(int64_t)63, K, log2bs);
  const size_t n = (size_t)p.tokens;
  // few tiles of D: the piece's terms in parts, each with a D of its own
  auto d_parts = [&]() {
    const int64_t tiles = ((p.tokens + kTileM - 1) / kTileM) * ((K + kTileN - 1) / kTileN);
    p.parts = (int)(tiles >= 256 ? 1 : 256 / tiles);
    if (p.parts > p.piece / 1024) p.parts = p.piece / 1024 > 0 ? p.piece / 1024 : 1;
    p.split = (int)to64((p.piece + p.parts - 1) / p.parts);
    p.parts = (int)((to64(p.piece) + p.split - 1) / p.split);
  };
  p.m = c.take(n * 4), p.s = c.take(n * 4), p.f = c.take(n * 4), p.lt = c.take(n * k * 4);
  if (p.tiled) {
    // 512 tiles of logits or more
    const int64_t rows = (p.tokens + kTileM - 1) / kTileM;
    p.piece = rows >= 8 ? 16384 : kMostPiece;
    while (p.piece > 8192 && p.piece / 2 >= V) p.piece /= 2;
    d_parts();
    p.Kp = to64(K);
    if (p.Kp != K) p.x = c.take(n * p.Kp * 2);
    p.logits = c.take(n * p.piece * 4);
    p.live = c.take(n * 4), p.list = c.take(n * 4), p.count = c.take(4);
    p.W = c.take((size_t)p.piece * p.Kp * 2);
    if (grad) {
      p.Wt = c.take((size_t)to64(p.piece) * K * 2);
      p.P = c.take(n * to64(p.piece) * 2);
      p.D = c.take(n * K * 4 * p.parts);
    }
  } else {
    p.parts = 1;
    const int64_t slices = skinny_fits(p.tokens, K, log2bs) ? skinny_parts(K) : 1;  // each with logits of its own
    int64_t piece = (kLogits / (p.tokens * slices)) & ~(int64_t)4095;  // rows_of wants 4096 rows
    if (piece < 4096) piece = 4096;
    if (p.mixed && piece > kMostPiece) piece = kMostPiece;
    p.piece = (int)(V < piece ? V : piece);
    if (p.mixed) d_parts();
    p.logits = c.take(n * p.piece * 4 * slices);
    p.segments = c.take(n * ((p.piece + kSegment - 1) / kSegment) * 8);
    p.carry = c.take(n * 16);
    if (grad) {
      p.P = c.take(n * to64(p.piece) * 2);
      p.D = c.take(n * K * 4 * p.parts);
    }
    if (p.mixed) {
      p.Wt = c.take((size_t)to64(p.piece) * K * 2);
    } else if (grad) {
      p.tail = c.take(n * kTail * 4);
      if (p.piece < V) p.add = c.take(n * K * 4);
      size_t most = 0;  // the product's own workspace, over all sizes that come up
      for (int64_t m : {p.tokens, T % p.tokens})
        for (int64_t v : {(int64_t)p.piece & ~63ll, (V % p.piece) & ~63ll})
          if (m > 0 && v > 0) {
            const size_t b = gemm_backward_workspace_bytes(m, v, K, log2bs);
            most = b > most ? b : most;
          }
      p.back = c.take(most);
    }
  }
  p.total = c.at;
  return p;
}

size_t loss_workspace(int64_t T, int64_t V, int64_t K, int log2bs, int k, bool grad) {
  return loss_plan(T, V, K, log2bs, k, grad).total;
}

// D = D f + P Wt^T, in the plan's parts
template <int DT>
static void add_to_D(const LossPlan &p, const uint16_t *P, int np, const uint16_t *Wt, int64_t m, int64_t K,
                     const int32_t *count, const float *f, float *D, bool first, hipStream_t st) {
  TileArgs b = tile_args(P, np, Wt, np, m, K, np);
  b.count = count, b.split = p.split;
  EpilogueAdd add;
  add.C = D, add.f = f, add.ld = K, add.part = p.tokens * K, add.first = first;
  hipLaunchKernelGGL((tile_kernel<DT, EpilogueAdd>), dim3(b.ncol * b.nrow, p.parts), dim3(256), 0, st, b, add);
}

// m tokens by the tile product; what is left for loss_finish_kernel is in rs and D
template <int DT>
static hipError_t pieces_tiled(const LossPlan &p, const uint16_t *x, int64_t m, const Weight4 &w, const Targets &tg,
                               const int64_t *ids, const void *teacher, bool grad, const RowState &rs, float *D,
                               char *ws, hipStream_t st) {
  float *logits = reinterpret_cast<float *>(ws + p.logits);
  uint16_t *P = reinterpret_cast<uint16_t *>(ws + p.P), *W = reinterpret_cast<uint16_t *>(ws + p.W);
  uint16_t *Wt = grad ? reinterpret_cast<uint16_t *>(ws + p.Wt) : nullptr;
  int32_t *live = reinterpret_cast<int32_t *>(ws + p.live), *list = reinterpret_cast<int32_t *>(ws + p.list);
  int32_t *count = reinterpret_cast<int32_t *>(ws + p.count);
  hipLaunchKernelGGL(loss_live_kernel, dim3((unsigned)((m + 3) / 4)), dim3(256), 0, st, ids, teacher, tg.teacher_dt, tg.k,
                     w.N, (int)m, live);
  hipLaunchKernelGGL(loss_order_kernel, dim3(1), dim3(1024), 0, st, live, (int)m, list, count);
  if (p.Kp != w.K) {
    uint16_t *padded = reinterpret_cast<uint16_t *>(ws + p.x);
    const hipError_t e = launch_pad_rows(x, m, w.K, p.Kp, padded, st);
    if (e != hipSuccess) return e;
    x = padded;
  }
  for (int64_t v = 0; v < w.N; v += p.piece) {
    const int n = (int)(w.N - v < p.piece ? w.N - v : p.piece), np = (n + 63) & ~63;
    const hipError_t e = grad ? launch_decode_piece(rows_of(w, v, n), DT, 0, w.K, W, p.Kp, Wt, np, st)
                              : launch_decode_rows(rows_of(w, v, n), DT, W, p.Kp, st);
    if (e != hipSuccess) return e;
    TileArgs a = tile_args(x, p.Kp, W, p.Kp, m, n, p.Kp);
    a.rows = list, a.count = count;
    EpilogueF32 keep;
    keep.C = logits, keep.ld = p.piece;
    hipLaunchKernelGGL((tile_kernel<DT, EpilogueF32>), dim3(a.ncol * a.nrow), dim3(256), 0, st, a, keep);
    const int threads = p.piece / 32;
    if (!grad) {
      hipLaunchKernelGGL((loss_rows_kernel<DT, false>), dim3((unsigned)m), dim3(threads), 0, st, logits, (int64_t)p.piece, v,
                         n, np, ids, tg.k, tg.inv_tau, v == 0, rs, list, count, P);
      continue;
    }
    hipLaunchKernelGGL((loss_rows_kernel<DT, true>), dim3((unsigned)m), dim3(threads), 0, st, logits, (int64_t)p.piece, v,
                       n, np, ids, tg.k, tg.inv_tau, v == 0, rs, list, count, P);
    add_to_D<DT>(p, P, np, Wt, m, w.K, count, rs.f, D, v == 0, st);
  }
  return hipGetLastError();
}

// m tokens by the products of gemm_4bit and its backward
template <int DT>
static hipError_t pieces_plain(const LossPlan &p, const uint16_t *x, int64_t m, const Weight4 &w, const Targets &tg,
                               const int64_t *ids, bool grad, const RowState &rs, float *D, int *tail_n, char *ws,
                               hipStream_t st) {
  float *logits = reinterpret_cast<float *>(ws + p.logits), *add = reinterpret_cast<float *>(ws + p.add);
  uint16_t *P = reinterpret_cast<uint16_t *>(ws + p.P);
  float2 *segments = reinterpret_cast<float2 *>(ws + p.segments), *carry = reinterpret_cast<float2 *>(ws + p.carry);
  int turn = 0;
  for (int64_t v = 0; v < w.N; v += p.piece, turn ^= 1) {
    const int n = (int)(w.N - v < p.piece ? w.N - v : p.piece);
    const int np = p.mixed ? (int)to64(n) : n & ~63, n_segments = (n + kSegment - 1) / kSegment;
    const Weight4 c = rows_of(w, v, n);
    const bool skinny = skinny_fits(m, w.K, w.log2bs);
    hipError_t e = skinny ? launch_skinny(x, DT, m, c, logits, st)
                          : launch_gemm_4bit(x, DT, m, n, w.K, c.packed, c.sc, c.dq, c.log2bs, c.qt, logits, kF32, nullptr, st);
    if (e != hipSuccess) return e;
    if (skinny && skinny_parts(w.K) > 1)
      e = launch_sum_parts(logits, skinny_parts(w.K), m * n, st);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(loss_part_kernel, dim3(n_segments, (unsigned)m), dim3(256), 0, st, logits, v, n, ids, tg.k, tg.inv_tau,
                       rs.lt, segments);
    float2 *before = carry + (turn ? p.tokens : 0), *after = carry + (turn ? 0 : p.tokens);
    if (!grad) {
      hipLaunchKernelGGL((loss_merge_kernel<DT, false>), dim3(1, (unsigned)m), dim3(64), 0, st, logits, v, n, np, ids, tg.k,
                         tg.inv_tau, v == 0, segments, n_segments, before, after, rs, P);
      continue;
    }
    hipLaunchKernelGGL((loss_merge_kernel<DT, true>), dim3(n_segments, (unsigned)m), dim3(256), 0, st, logits, v, n, np, ids,
                       tg.k, tg.inv_tau, v == 0, segments, n_segments, before, after, rs, P);
    if (p.mixed) {
      uint16_t *Wt = reinterpret_cast<uint16_t *>(ws + p.Wt);
      e = launch_decode_piece(c, DT, 0, w.K, nullptr, 0, Wt, np, st);
      if (e != hipSuccess) return e;
      add_to_D<DT>(p, P, np, Wt, m, w.K, nullptr, rs.f, D, v == 0, st);
      continue;
    }
    if (np) {
      e = launch_gemm_4bit_backward(P, DT, m, np, w.K, c.packed, c.sc, c.dq, c.log2bs, c.qt, v == 0 ? D : add, kF32,
                                    ws + p.back, st);
      if (e != hipSuccess) return e;
    }
    if (v > 0 || !np)
      hipLaunchKernelGGL(loss_add_kernel, dim3((unsigned)m), dim3(256), 0, st, D, np ? add : nullptr, rs.f, w.K, v == 0);
    *tail_n = n - np;
  }
  return hipGetLastError();
}

template <int DT>
static hipError_t loss_t(const uint16_t *x, int64_t T, const Weight4 &w, const Targets &tg, const float *dloss,
                         void *loss, int loss_dt, uint16_t *dx, char *ws, hipStream_t st) {
  const LossPlan p = loss_plan(T, w.N, w.K, w.log2bs, tg.k, dx != nullptr);
  float *D = reinterpret_cast<float *>(ws + p.D);
  const RowState rs{reinterpret_cast<float *>(ws + p.m), reinterpret_cast<float *>(ws + p.s),
                    reinterpret_cast<float *>(ws + p.f), reinterpret_cast<float *>(ws + p.lt),
                    reinterpret_cast<float *>(ws + p.tail)};
  const size_t tsize = tg.teacher_dt == kF32 ? 4 : 2, lsize = loss_dt == kF32 ? 4 : 2;
  for (int64_t t = 0; t < T; t += p.tokens) {
    const int64_t m = T - t < p.tokens ? T - t : p.tokens;
    const int64_t *ids = tg.ids + t * tg.k;
    const void *teacher = tg.teacher ? static_cast<const char *>(tg.teacher) + t * tg.k * tsize : nullptr;
    int tail_n = 0;
    const hipError_t e = p.tiled ? pieces_tiled<DT>(p, x + t * w.K, m, w, tg, ids, teacher, dx != nullptr, rs, D, ws, st)
                                 : pieces_plain<DT>(p, x + t * w.K, m, w, tg, ids, dx != nullptr, rs, D, &tail_n, ws, st);
    if (e != hipSuccess) return e;
    const int32_t *list = p.tiled ? reinterpret_cast<int32_t *>(ws + p.list) : nullptr;
    char *lp = static_cast<char *>(loss) + t * lsize;
#define QMV_L(LDT, DQV)                                                                                              \
  hipLaunchKernelGGL((loss_finish_kernel<DT, LDT, DQV>), dim3((unsigned)m), dim3(256), 0, st, ids, teacher,          \
                     tg.teacher_dt, tg.k, tg.inv_tau, w.N, rs, tail_n, D, p.parts, p.tokens * w.K, w.K, list,        \
                     w.packed, w.sc, w.log2bs, code_values(w.qt), dloss ? dloss + t : nullptr,                       \
                     reinterpret_cast<typename Storage<LDT>::type *>(lp), dx ? dx + t * w.K : nullptr)
    if (loss_dt == kF32) {
      if (w.dq) QMV_L(kF32, true);
      else QMV_L(kF32, false);
    } else {
      if (w.dq) QMV_L(DT, true);
      else QMV_L(DT, false);
    }
#undef QMV_L
  }
  return hipGetLastError();
}

hipError_t launch_loss(const void *x, int dt, int64_t T, const Weight4 &w, const Targets &tg, const float *dloss,
                       void *loss, int loss_dt, void *dx, char *ws, hipStream_t st) {
  const uint16_t *xp = static_cast<const uint16_t *>(x);
  uint16_t *d = static_cast<uint16_t *>(dx);
  return dt == kF16 ? loss_t<kF16>(xp, T, w, tg, dloss, loss, loss_dt, d, ws, st)
                    : loss_t<kBF16>(xp, T, w, tg, dloss, loss, loss_dt, d, ws, st);
}

}  // namespace qmv
