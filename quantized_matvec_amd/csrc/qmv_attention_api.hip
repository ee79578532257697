// The C ABI of include/qmv/attention.h: argument validation on the host, then
// a launch on the caller's stream.
#include <math.h>

#include "qmv/attention.h"
#include "qmv_attention.hpp"

using namespace qmv;

namespace {

constexpr int64_t kMost = (int64_t)1 << 31;  // tokens, positions and heads stay below

bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool is_pow2(int64_t v) { return v > 0 && (v & (v - 1)) == 0; }
int launch_status(hipError_t e) {
  return e == hipSuccess ? QMV_OK : (e == hipErrorInvalidConfiguration ? QMV_ERR_TOO_LARGE : QMV_ERR_LAUNCH);
}

// The strides of a dimension of one count for nothing.
int check_heads(const qmv_heads *h, int64_t tokens, int size, Heads *out) {
  if (!h || !h->data || h->heads <= 0 || h->heads > 65535) return QMV_ERR_INVALID_ARG;
  Heads v{h->data, tokens > 1 ? h->token_stride : 0, h->heads > 1 ? h->head_stride : 0, h->heads};
  if (v.ts < 0 || v.hs < 0) return QMV_ERR_INVALID_ARG;
  if (v.ts > INT64_MAX / (kMost * 8) || v.hs > INT64_MAX / (kMost * 8)) return QMV_ERR_INVALID_ARG;
  if (!aligned(v.p, 16) || v.ts * size % 16 || v.hs * size % 16) return QMV_ERR_ALIGNMENT;
  *out = v;
  return QMV_OK;
}

int check_rope(const qmv_rope *r, int32_t head_dim, Rope *out) {
  if (!r->table || r->max_pos <= 0 || r->rot_dim < 2 || r->rot_dim % 2 || r->rot_dim > head_dim)
    return QMV_ERR_INVALID_ARG;
  if (r->max_pos > INT64_MAX / 4096) return QMV_ERR_INVALID_ARG;
  if (!aligned(r->table, 16)) return QMV_ERR_ALIGNMENT;
  *out = Rope{reinterpret_cast<const float2 *>(r->table), r->max_pos, r->rot_dim / 2,
              r->interleaved != 0};
  return QMV_OK;
}

// Sizes of the cache, and whether its arrays are there where `arrays` is set.
int check_cache(const qmv_kv_cache *c, bool arrays, KVCache *out) {
  if (!c || c->num_pages <= 0 || c->num_pages > INT32_MAX || c->heads <= 0 || c->heads > 65535)
    return QMV_ERR_INVALID_ARG;
  if (c->quant_type != QMV_NF4 && c->quant_type != QMV_FP4) return QMV_ERR_INVALID_ARG;
  if (c->dtype != QMV_F32 && c->dtype != QMV_F16 && c->dtype != QMV_BF16) return QMV_ERR_INVALID_ARG;
  if (c->dtype == QMV_F32) return QMV_ERR_UNSUPPORTED;
  if (!is_pow2(c->page_size) || c->page_size < 16 || c->page_size > 1024) return QMV_ERR_UNSUPPORTED;
  if (c->head_dim < 32 || c->head_dim > 256 || c->head_dim % 32) return QMV_ERR_UNSUPPORTED;
  if (!is_pow2(c->blocksize) || c->blocksize < 32 || c->head_dim % c->blocksize)
    return QMV_ERR_UNSUPPORTED;
  // offsets inside a page fit in 31 bits (num_pages < 2^31: all of them in 64)
  if ((int64_t)c->heads * c->page_size * c->head_dim >= kMost) return QMV_ERR_TOO_LARGE;
  if (arrays) {
    if (!c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales) return QMV_ERR_INVALID_ARG;
    if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, 16) ||
        !aligned(c->v_scales, 16))
      return QMV_ERR_ALIGNMENT;
  }
  *out = KVCache{c->k_codes, c->v_codes, static_cast<uint16_t *>(c->k_scales),
                 static_cast<uint16_t *>(c->v_scales), c->num_pages, c->heads,
                 log2_exact(c->page_size), c->head_dim, c->blocksize};
  return QMV_OK;
}

int check_batch(const qmv_kv_batch *b, int64_t tokens, bool arrays, KVBatch *out) {
  if (!b || tokens <= 0 || tokens >= kMost || b->batch <= 0 || b->max_pages <= 0 || b->max_q <= 0)
    return QMV_ERR_INVALID_ARG;
  if (b->batch > 65535) return QMV_ERR_UNSUPPORTED;
  if (b->table_stride < b->max_pages && b->batch > 1) return QMV_ERR_INVALID_ARG;
  if (b->table_stride > INT64_MAX / kMost) return QMV_ERR_INVALID_ARG;
  if (arrays) {
    if (!b->block_table || !b->kv_len) return QMV_ERR_INVALID_ARG;
    if (!aligned(b->block_table, 4) || !aligned(b->kv_len, 4) || !aligned(b->cu_q, 4))
      return QMV_ERR_ALIGNMENT;
    if (!b->cu_q && tokens != b->batch) return QMV_ERR_INVALID_ARG;
  }
  const int32_t most = b->cu_q ? (int32_t)(b->max_q < tokens ? b->max_q : tokens) : 1;
  *out = KVBatch{b->block_table, b->batch > 1 ? b->table_stride : 0, b->kv_len, b->cu_q, b->batch,
                 b->max_pages, most, tokens};
  return QMV_OK;
}

// Keys a call can reach: the caller's bound, and the block table's.
int64_t reach(const KVCache &c, const KVBatch &b, int64_t max_kv) {
  const int64_t all = (int64_t)b.max_pages << c.log2page;
  const int64_t most = max_kv > 0 && max_kv < all ? max_kv : all;
  return most < kMost - 1024 ? most : kMost - 1024;
}

Midpoints4 code_midpoints(int qt) {
  float t[16];
  qmv_code_table((qmv_quant_type)qt, t);
  Midpoints4 m{};
  if (qt == QMV_NF4) {
    for (int j = 0; j < 15; ++j) m.mid[j] = 0.5 * ((double)t[j] + (double)t[j + 1]);
  } else {
    for (int j = 0; j < 7; ++j) {
      m.mid[7 + j] = 0.5 * ((double)t[j] + (double)t[j + 1]);
      m.mid[6 - j] = -m.mid[7 + j];
    }
  }
  return m;
}

}  // namespace

extern "C" {

int qmv_rope_frequencies(int32_t rot_dim, double theta, qmv_rope_scaling scaling, double factor,
                         int64_t original_len, double beta_fast, double beta_slow, double *freqs) {
  if (!freqs || rot_dim < 2 || rot_dim % 2 || !(theta > 0.0) || !isfinite(theta))
    return QMV_ERR_INVALID_ARG;
  if (scaling != QMV_ROPE_PLAIN && scaling != QMV_ROPE_LINEAR && scaling != QMV_ROPE_BASE &&
      scaling != QMV_ROPE_BANDS)
    return QMV_ERR_INVALID_ARG;
  if (scaling != QMV_ROPE_PLAIN && (!(factor >= 1.0) || !isfinite(factor))) return QMV_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925;
  double first = 0.0, last = 0.0;
  if (scaling == QMV_ROPE_BASE) {
    if (rot_dim <= 2) return QMV_ERR_INVALID_ARG;
    theta *= pow(factor, (double)rot_dim / (rot_dim - 2));
  }
  if (scaling == QMV_ROPE_BANDS) {
    if (original_len <= 0 || !(beta_slow > 0.0) || !(beta_fast > beta_slow) || !isfinite(beta_fast) ||
        !(theta > 1.0))
      return QMV_ERR_INVALID_ARG;
    // pair i turns original_len theta^(-2 i / rot_dim) / (2 pi) times: the
    // (real) index at which that is beta
    auto index = [&](double beta) {
      return 0.5 * rot_dim * log((double)original_len / (two_pi * beta)) / log(theta);
    };
    // not clipped to the pairs there are: that would turn the line between
    first = floor(index(beta_fast));
    last = ceil(index(beta_slow));
    if (last <= first) last = first + 1e-3;
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = pow(theta, -2.0 * i / rot_dim);
    if (scaling == QMV_ROPE_LINEAR) f /= factor;
    if (scaling == QMV_ROPE_BANDS) {
      const double slow = fmin(fmax((i - first) / (last - first), 0.0), 1.0);
      f = f * (1.0 - slow) + f / factor * slow;
    }
    freqs[i] = f;
  }
  return QMV_OK;
}

int qmv_rope_table(const double *freqs, int32_t rot_dim, int64_t max_pos, double gain, float *table,
                   void *stream) {
  if (!freqs || !table || rot_dim < 2 || rot_dim % 2 || max_pos <= 0 || !isfinite(gain))
    return QMV_ERR_INVALID_ARG;
  if (rot_dim > 256) return QMV_ERR_UNSUPPORTED;
  if (max_pos > INT64_MAX / 4096) return QMV_ERR_INVALID_ARG;
  for (int i = 0; i < rot_dim / 2; ++i)
    if (!isfinite(freqs[i])) return QMV_ERR_INVALID_ARG;
  if (!aligned(table, 16)) return QMV_ERR_ALIGNMENT;
  return launch_status(launch_rope_table(freqs, rot_dim / 2, max_pos, gain, table, (hipStream_t)stream));
}

int qmv_rotary(const qmv_heads *q, const qmv_heads *q_out, const qmv_heads *k,
               const qmv_heads *k_out, qmv_dtype dtype, int64_t tokens, int32_t head_dim,
               const int64_t *positions, const qmv_rope *rope, int32_t inverse, void *stream) {
  if (!rope || !positions || tokens <= 0 || tokens >= kMost || head_dim <= 0 || !k != !k_out)
    return QMV_ERR_INVALID_ARG;
  if (dtype != QMV_F32 && dtype != QMV_F16 && dtype != QMV_BF16) return QMV_ERR_INVALID_ARG;
  if (head_dim % 8 || head_dim > 4096) return QMV_ERR_UNSUPPORTED;
  const int size = dtype == QMV_F32 ? 4 : 2;
  Rope r{};
  Heads hq{}, hqo{}, hk{}, hko{};
  int rc = check_rope(rope, head_dim, &r);
  if (rc == QMV_OK) rc = check_heads(q, tokens, size, &hq);
  if (rc == QMV_OK) rc = check_heads(q_out, tokens, size, &hqo);
  if (rc == QMV_OK && k) rc = check_heads(k, tokens, size, &hk);
  if (rc == QMV_OK && k) rc = check_heads(k_out, tokens, size, &hko);
  if (rc != QMV_OK) return rc;
  if (hq.heads != hqo.heads || hk.heads != hko.heads) return QMV_ERR_INVALID_ARG;
  if (!aligned(positions, 8)) return QMV_ERR_ALIGNMENT;
  // workgroups of 256 pairs or more are counted in 31 bits
  if (tokens > kMost * 255 / ((int64_t)(hq.heads + hk.heads) * head_dim)) return QMV_ERR_TOO_LARGE;
  return launch_status(launch_rotary(hq, hqo, hk, hko, dtype, tokens, head_dim, positions, r,
                                     inverse != 0, (hipStream_t)stream));
}

int qmv_kv_append_4bit(const qmv_kv_cache *cache, const qmv_kv_batch *batch, int64_t tokens,
                       const qmv_heads *k, const qmv_heads *v, const qmv_rope *rope,
                       const qmv_heads *q, const qmv_heads *q_out, void *stream) {
  KVCache c;
  KVBatch kb;
  Heads hk{}, hv{}, hq{}, hqo{};
  Rope r{};
  if (!q != !q_out || (q && !rope)) return QMV_ERR_INVALID_ARG;
  int rc = check_cache(cache, true, &c);
  if (rc == QMV_OK) rc = check_batch(batch, tokens, true, &kb);
  if (rc == QMV_OK) rc = check_heads(k, tokens, 2, &hk);
  if (rc == QMV_OK) rc = check_heads(v, tokens, 2, &hv);
  if (rc == QMV_OK && rope) rc = check_rope(rope, c.dim, &r);
  if (rc == QMV_OK && q) rc = check_heads(q, tokens, 2, &hq);
  if (rc == QMV_OK && q) rc = check_heads(q_out, tokens, 2, &hqo);
  if (rc != QMV_OK) return rc;
  if (hk.heads != c.heads || hv.heads != c.heads || hq.heads != hqo.heads) return QMV_ERR_INVALID_ARG;
  if (kb.max_q > kMost * 5 / (hq.heads + 2 * (int64_t)c.heads)) return QMV_ERR_TOO_LARGE;
  return launch_status(launch_kv_append(c, cache->dtype, cache->quant_type,
                                        code_midpoints(cache->quant_type), kb, hk, hv, r, hq, hqo,
                                        (hipStream_t)stream));
}

int qmv_kv_dequantize_4bit(const qmv_kv_cache *cache, const qmv_kv_batch *batch, int64_t tokens,
                           const qmv_heads *k_out, const qmv_heads *v_out, void *stream) {
  KVCache c;
  KVBatch kb;
  Heads hk{}, hv{};
  int rc = check_cache(cache, true, &c);
  if (rc == QMV_OK) rc = check_batch(batch, tokens, true, &kb);
  if (rc == QMV_OK) rc = check_heads(k_out, tokens, 2, &hk);
  if (rc == QMV_OK) rc = check_heads(v_out, tokens, 2, &hv);
  if (rc != QMV_OK) return rc;
  if (hk.heads != c.heads || hv.heads != c.heads) return QMV_ERR_INVALID_ARG;
  if (kb.max_q > kMost * 7 / (2 * (int64_t)c.heads)) return QMV_ERR_TOO_LARGE;
  return launch_status(launch_kv_dequantize(c, cache->dtype, cache->quant_type, kb, hk, hv,
                                            (hipStream_t)stream));
}

size_t qmv_attention_4bit_workspace(const qmv_kv_cache *cache, const qmv_kv_batch *batch,
                                    int64_t tokens, int32_t q_heads, int64_t max_kv,
                                    int64_t window) {
  KVCache c;
  KVBatch kb;
  if (check_cache(cache, false, &c) != QMV_OK || check_batch(batch, tokens, false, &kb) != QMV_OK)
    return 0;
  if (q_heads <= 0 || q_heads > 65535 || q_heads % c.heads || max_kv < 0 || window < 0) return 0;
  return attention_workspace_bytes(c, kb, q_heads, reach(c, kb, max_kv), window);
}

int qmv_attention_4bit(const qmv_heads *q, const qmv_kv_cache *cache, const qmv_kv_batch *batch,
                       int64_t tokens, int64_t max_kv, float scale, int32_t causal, int64_t window,
                       const qmv_heads *out, void *workspace, size_t workspace_bytes, void *stream) {
  KVCache c;
  KVBatch kb;
  Heads hq{}, ho{};
  int rc = check_cache(cache, true, &c);
  if (rc == QMV_OK) rc = check_batch(batch, tokens, true, &kb);
  if (rc == QMV_OK) rc = check_heads(q, tokens, 2, &hq);
  if (rc == QMV_OK) rc = check_heads(out, tokens, 2, &ho);
  if (rc != QMV_OK) return rc;
  if (hq.heads != ho.heads || hq.heads % c.heads || max_kv < 0 || window < 0 ||
      (window > 0 && !causal) || !isfinite(scale))
    return QMV_ERR_INVALID_ARG;
  if (kb.max_q > (kMost - 1) / hq.heads) return QMV_ERR_TOO_LARGE;
  const int64_t most = reach(c, kb, max_kv);
  // steps of 64 tokens over all sequences, heads and (up to three) row tiles
  // are counted in 31 bits
  if ((most / 64 + 2) * 3 * c.heads >= kMost / kb.batch) return QMV_ERR_TOO_LARGE;
  // workgroups of 256 query rows (and a row's parts, at most one for each
  // compute unit, only where there are fewer workgroups than units)
  if (((int64_t)kb.max_q * (hq.heads / c.heads) / 256 + 1) * c.heads >= kMost / kb.batch) return QMV_ERR_TOO_LARGE;
  const size_t need = attention_workspace_bytes(c, kb, hq.heads, most, window);
  if (need && (!workspace || workspace_bytes < need)) return QMV_ERR_WORKSPACE;
  if (need && !aligned(workspace, 16)) return QMV_ERR_ALIGNMENT;
  return launch_status(launch_attention(c, cache->dtype, cache->quant_type, kb, hq, most, scale,
                                        causal != 0, window, ho, workspace, (hipStream_t)stream));
}

}  // extern "C"
