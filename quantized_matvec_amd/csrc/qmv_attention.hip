// Attention over the 4-bit cache:
//   out[t] = sum_j p_j v^_j / sum_j p_j,  p_j = exp(scale q_t . k^_j - m)
// over the keys j that token t sees, k^ = T[code] a and v^ likewise, m the
// running maximum of the scores; m and both sums are fp32.
#include <algorithm>

#include "qmv_attention_mfma.hpp"

namespace qmv {

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// ---------------------------------------------------------------------------
// One wave for each (token, query head), 64 keys a step: a lane scores one
// key, then each lane sums over the keys for two pairs of elements.  Bound by
// the vector unit (each query head dequantizes the cache for itself).  It
// serves the head sizes that the matrix-core kernels are not built for: 64
// sequences as in attention_decode_kernel's comment take 470, 1315 and 1545 us
// with heads of 32, 160 and 224.  With heads of 128 it took 1224 us for them (73
// there), and 132 ms for the chunk of attention_prompt_kernel's (2.8).
// ---------------------------------------------------------------------------
template <int DT>
__global__ __launch_bounds__(64) void attention_rows_kernel(AttnArgs a, float scale_log2) {
  __shared__ float2 lut[256];
  __shared__ float qs[256];
  __shared__ float w[8][64];     // p_j a_j of each value block
  __shared__ int64_t pages[64];
  const int lane = threadIdx.x;
  const int b = blockIdx.y;
  const SeqRange s = seq_range(a.kb, b);
  const int i = blockIdx.x / a.q.heads;
  const int h = blockIdx.x - i * a.q.heads;
  if (i >= s.n || i >= a.kb.max_q) return;
  const int kh = h / a.group;
  const int dim = a.c.dim, nb = dim / a.c.bs, ps = 1 << a.c.log2page;
  const uint32_t *tb = table_bits(a.qt);
  for (int e = lane; e < 256; e += 64)
    lut[e] = make_float2(__uint_as_float(tb[e >> 4]), __uint_as_float(tb[e & 15]));
  const uint16_t *qrow = static_cast<const uint16_t *>(a.q.p) + (s.row0 + i) * a.q.ts + h * a.q.hs;
  for (int e = lane; e < dim; e += 64) qs[e] = bits16_to_f32<DT>(qrow[e]) * scale_log2;
  __syncthreads();

  int lo, hi;
  key_range(a, s, i, lo, hi);
  float m = -INFINITY, l = 0.f;
  float o[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
  for (int t0 = lo & ~15; t0 < hi; t0 += 64) {
    const int j = t0 + lane;
    const int64_t page = j < hi ? page_of(a.kb, a.c, b, j) : -1;
    const bool seen = page >= 0 && j >= lo;
    const int at = j & (ps - 1);
    float score = -INFINITY;
    if (seen) {
      const uint4 *src = reinterpret_cast<const uint4 *>(a.c.kc + code_base(a.c, page, kh) +
                                                         (int64_t)at * (dim >> 1));
      const uint16_t *ks = a.c.ks + scale_base(a.c, page, kh) + at;
      score = 0.f;
      for (int ch = 0; ch < dim / 32; ++ch) {
        const uint4 v = src[ch];
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          const float2 t = lut[(u[n >> 2] >> (8 * (n & 3))) & 0xffu];
          sum = fmaf(t.x, qs[32 * ch + 2 * n], sum);
          sum = fmaf(t.y, qs[32 * ch + 2 * n + 1], sum);
        }
        score = fmaf(sum, bits16_to_f32<DT>(ks[(int64_t)(32 * ch / a.c.bs) << a.c.log2page]), score);
      }
    }
    const float top = fmaxf(m, wave_max(score));
    const float p = seen ? exp2f(score - top) : 0.f;
    const float keep = m == -INFINITY ? 0.f : exp2f(m - top);
    m = top;
    l = l * keep + wave_sum(p);
    __syncthreads();
    for (int n = 0; n < nb; ++n)
      w[n][lane] = seen ? p * bits16_to_f32<DT>(a.c.vs[scale_base(a.c, page, kh) +
                                                       ((int64_t)n << a.c.log2page) + at]) : 0.f;
    pages[lane] = page;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int P = lane + 64 * r;  // elements 2 P and 2 P + 1
      if (2 * P >= dim) continue;
      const float *wn = w[2 * P / a.c.bs];
      float s0 = o[r][0] * keep, s1 = o[r][1] * keep;
      for (int g = 0; g < 4; ++g) {
        const int64_t pg = pages[16 * g];
        if (pg < 0) continue;  // 16 tokens share a page; none of a missing one is seen
        const uint4 v = *reinterpret_cast<const uint4 *>(
            a.c.vc + code_base(a.c, pg, kh) +
            (int64_t)(((t0 + 16 * g) & (ps - 1)) >> 4) * dim * 8 + P * 16);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          const float2 t = lut[(u[n >> 2] >> (8 * (n & 3))) & 0xffu];
          s0 = fmaf(t.x, wn[16 * g + n], s0);
          s1 = fmaf(t.y, wn[16 * g + n], s1);
        }
      }
      o[r][0] = s0;
      o[r][1] = s1;
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint16_t *orow = static_cast<uint16_t *>(a.out.p) + (s.row0 + i) * a.out.ts + h * a.out.hs;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int P = lane + 64 * r;
    if (2 * P < dim) reinterpret_cast<uint32_t *>(orow)[P] = cvt_pair<DT>(o[r][0] * inv, o[r][1] * inv);
  }
}

hipError_t launch_attention_rows(const AttnArgs &a, int dt, hipStream_t st) {
  if (!grid_fits((int64_t)a.kb.max_q * a.q.heads, 64)) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)(a.kb.max_q * a.q.heads), (unsigned)a.kb.batch);
  const float sl = a.scale * 1.44269504088896340736f;
  if (dt == kBF16) hipLaunchKernelGGL((attention_rows_kernel<kBF16>), grid, dim3(64), 0, st, a, sl);
  else hipLaunchKernelGGL((attention_rows_kernel<kF16>), grid, dim3(64), 0, st, a, sl);
  return hipGetLastError();
}

size_t attention_workspace_bytes(const KVCache &c, const KVBatch &kb, int q_heads, int64_t max_kv,
                                 int64_t window) {
  const int64_t rows = (int64_t)kb.max_q * (q_heads / c.heads);
  if (decode_eligible(c, rows))
    return decode_workspace_bytes(c, kb, (int)rows, max_kv, window);
  return prompt_eligible(c) ? prompt_workspace_bytes(c, kb, q_heads, max_kv, window) : 0;
}

hipError_t launch_attention(const KVCache &c, int dt, int qt, const KVBatch &kb, const Heads &q,
                            int64_t max_kv, float scale, bool causal, int64_t window,
                            const Heads &out, void *ws, hipStream_t st) {
  const AttnArgs a{c, kb, q, out, q.heads / c.heads, scale, (int)max_kv,
                   (int)std::min<int64_t>(window, INT32_MAX), causal, qt};
  const int64_t rows = (int64_t)kb.max_q * a.group;
  if (decode_eligible(c, rows)) return launch_attention_decode(a, dt, ws, st);
  return prompt_eligible(c) ? launch_attention_prompt(a, dt, ws, st) : launch_attention_rows(a, dt, st);
}

}  // namespace qmv
