/*
 * qmv/attention.h -- C ABI of libqmv.so, continued: rotary positions, a paged
 * key/value cache held in the library's 4-bit blockwise codes, and attention
 * over it.
 *
 * The conventions of qmv.h hold here too: every array is the caller's, device
 * arrays are 16-byte aligned, work is enqueued on ``stream`` and nothing
 * synchronizes the host, and every argument the host can see is checked
 * before anything is launched.  QMV_ERR_TOO_LARGE: a call's sizes pass the
 * limits named at each structure and call, or need a grid of 2^32 threads along
 * a dimension (at the earliest: rotary at 2^32 elements, an append or a read back
 * at 2^34, attention at 2^23 tiles of 256 query rows, or with head sizes of 32,
 * 160 and 224 at 2^26 query rows of a sequence).  What only the device sees
 * (positions, lengths, offsets and page numbers) is checked by the kernels: a
 * value out of range never reaches memory, and what it means is stated at each
 * call.
 */
#ifndef QMV_ATTENTION_H
#define QMV_ATTENTION_H

#include "../qmv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Head vectors [tokens, heads, head_dim] with unit stride in head_dim.
 * Strides are in elements; for more than one token (head) the token (head)
 * stride is a multiple of 16 bytes (QMV_ERR_ALIGNMENT), so the heads of one
 * fused projection are taken as they are.  Outputs must not overlap
 * themselves. */
typedef struct {
  void *data;
  int64_t token_stride;
  int64_t head_stride;
  int32_t heads;
} qmv_heads;

/*
 * The rotation of a position: cos and sin of position * frequency i, for the
 * rot_dim / 2 pairs that are turned.
 *   table        [max_pos, rot_dim / 2, 2] device fp32 (qmv_rope_table fills one)
 *   rot_dim      even, 2 .. head_dim: the first rot_dim elements of a head are
 *                turned, the others are copied
 *   interleaved  0: pair i is elements (i, i + rot_dim / 2); 1: (2 i, 2 i + 1)
 * With pair (a, b) and (c, s) the result is (a c - b s, b c + a s): products
 * and sums rounded separately in fp32, then one rounding to the heads' type.
 * A token whose position is outside [0, max_pos) becomes a row of zeros.
 */
typedef struct {
  const float *table;
  int64_t max_pos;
  int32_t rot_dim;
  int32_t interleaved;
} qmv_rope;

typedef enum {
  QMV_ROPE_PLAIN = 0,   /* theta^(-2 i / rot_dim) */
  QMV_ROPE_LINEAR = 1,  /* plain / factor: positions are compressed by factor */
  QMV_ROPE_BASE = 2,    /* the base grows to theta * factor^(rot_dim / (rot_dim - 2)): the slowest pair
                           is stretched by factor, the fastest not at all */
  QMV_ROPE_BANDS = 3    /* pairs that turn more than beta_fast times in original_len positions keep
                           their frequency, those that turn fewer than beta_slow times are divided by
                           factor, in between the two are mixed linearly in the pair's index (from the
                           last index of the first kind to the first of the second, also where these
                           lie outside the pairs) */
} qmv_rope_scaling;

/* Host-side: freqs [rot_dim / 2] float64 out.  factor >= 1 (ignored for
 * QMV_ROPE_PLAIN); original_len and 0 < beta_slow < beta_fast are read for
 * QMV_ROPE_BANDS only. */
int qmv_rope_frequencies(int32_t rot_dim, double theta, qmv_rope_scaling scaling, double factor,
                         int64_t original_len, double beta_fast, double beta_slow, double *freqs);

/* table [max_pos, rot_dim / 2, 2] device fp32 out: gain * (cos, sin) of
 * position * freqs[i], computed in float64 and rounded once.
 *   freqs  [rot_dim / 2] HOST float64, rot_dim at most 256
 *   gain   the factor some long-context scalings put on queries and keys (1) */
int qmv_rope_table(const double *freqs, int32_t rot_dim, int64_t max_pos, double gain, float *table,
                   void *stream);

/*
 * rotary: the position rotation of queries and keys in one pass.
 *   q, q_out   heads of any of the three types; q_out may be q itself (same
 *              pointer and strides), but must not overlap it otherwise
 *   k, k_out   both NULL, or as q with a head count of their own
 *   head_dim   a multiple of 8, at most 4096, else QMV_ERR_UNSUPPORTED; heads at most 65535
 *   positions  [tokens] device int64, 8-byte aligned
 *   inverse    1: the rotation by minus the angle.  It is the backward pass:
 *              with dY the gradient of the outputs, the gradient of the inputs
 *              is the inverse rotation of dY (the table's gain included, since
 *              it multiplies both).
 */
int qmv_rotary(const qmv_heads *q, const qmv_heads *q_out, const qmv_heads *k,
               const qmv_heads *k_out, qmv_dtype dtype, int64_t tokens, int32_t head_dim,
               const int64_t *positions, const qmv_rope *rope, int32_t inverse, void *stream);

/*
 * A paged cache.  Page p holds page_size consecutive tokens of one sequence:
 *   k_codes   [num_pages, heads, page_size, head_dim / 2] uint8
 *   v_codes   [num_pages, heads, page_size / 16, head_dim / 2, 16] uint8: the
 *             16 tokens of a byte lie side by side, the order in which the
 *             matrix cores take the values
 *   k_scales, v_scales  [num_pages, heads, head_dim / blocksize, page_size] dtype
 * A row (one token's head) is quantized as by qmv_quantize_4bit with blocks of
 * `blocksize` consecutive elements: the same codes, two to a byte with the
 * even element in the high nibble, and the same block maxima, which a 16-bit
 * type holds exactly because they are magnitudes of its own values.
 *   page_size  power of two in [16, 1024]
 *   head_dim   a multiple of 32 in [32, 256]
 *   blocksize  power of two, at least 32, dividing head_dim
 *   dtype      QMV_F16 or QMV_BF16: the type of keys, values and queries
 * else QMV_ERR_UNSUPPORTED.
 *   heads      1 .. 65535, num_pages 1 .. 2^31 - 1 (QMV_ERR_INVALID_ARG)
 * heads * page_size * head_dim, a page's elements, is below 2^31, else
 * QMV_ERR_TOO_LARGE; offsets of pages are 64-bit.
 */
typedef struct {
  uint8_t *k_codes;
  uint8_t *v_codes;
  void *k_scales;
  void *v_scales;
  int64_t num_pages;
  int32_t heads;
  int32_t page_size;
  int32_t head_dim;
  int32_t blocksize;
  qmv_quant_type quant_type;
  qmv_dtype dtype;
} qmv_kv_cache;

/*
 * The sequences of a call and the tokens that it adds to each or asks for.
 *   block_table  [batch, max_pages] device int32, row stride table_stride:
 *                page of tokens [i page_size, (i + 1) page_size); an entry
 *                outside [0, num_pages) is a page that is not there
 *   kv_len       [batch] device int32: tokens of each sequence in the cache,
 *                those of this call included
 *   cu_q         [batch + 1] device int32 offsets (cu_q[0] = 0, ascending) of
 *                each sequence's tokens among the call's `tokens`, or NULL:
 *                one token for each sequence (tokens = batch)
 *   max_q        at least the most tokens of one sequence in this call; the
 *                tokens of a sequence beyond it are not worked on
 *   batch        1 .. 65535, else QMV_ERR_UNSUPPORTED
 * max_q times the heads of a token, and the 64-token steps of the longest
 * sequence times batch and heads, have to fit in 31 bits (attention counts
 * three row tiles for each head), else QMV_ERR_TOO_LARGE.
 * Token i of a sequence's n tokens has position kv_len - n + i.
 */
typedef struct {
  const int32_t *block_table;
  int64_t table_stride;
  const int32_t *kv_len;
  const int32_t *cu_q;
  int32_t batch;
  int32_t max_pages;
  int32_t max_q;
} qmv_kv_batch;

/*
 * kv_append_4bit: the keys and values of `tokens` new tokens, the keys turned
 * by their positions first, quantized into the cache.  The turned key is
 * rounded to the cache's type, then quantized, so the cache holds exactly
 * what qmv_rotary and qmv_quantize_4bit give one after the other.
 *   k, v      [tokens, cache heads, head_dim]
 *   rope      NULL: the keys are taken as they are
 *   q, q_out  both NULL, or the queries of the same tokens, turned in the same
 *             launch (needs rope; q_out may be q itself)
 * A token whose page is not there, or whose position is negative or past the
 * block table, is not written.  Two tokens of one call must not be the same
 * position of the same page.
 */
int qmv_kv_append_4bit(const qmv_kv_cache *cache, const qmv_kv_batch *batch, int64_t tokens,
                       const qmv_heads *k, const qmv_heads *v, const qmv_rope *rope,
                       const qmv_heads *q, const qmv_heads *q_out, void *stream);

/*
 * kv_dequantize_4bit: the cached keys and values of the batch's tokens (with
 * cu_q, the last ones of each sequence), as qmv_dequantize_4bit gives them.
 *   k_out, v_out  [tokens, cache heads, head_dim] of the cache's type
 * A token whose page is not there is a row of zeros.
 */
int qmv_kv_dequantize_4bit(const qmv_kv_cache *cache, const qmv_kv_batch *batch, int64_t tokens,
                           const qmv_heads *k_out, const qmv_heads *v_out, void *stream);

/*
 * attention_4bit: out = softmax(scale q K^T) V over the cached keys of each
 * token's sequence, with fp32 statistics and sums.
 *   q, out    [tokens, q_heads, head_dim] of the cache's type; q_heads a
 *             multiple of the cache's heads, q head h reading head
 *             h / (q_heads / heads)
 *   max_kv    an upper bound of kv_len on the host (keys beyond it are not
 *             read); 0: max_pages * page_size
 *   scale     finite; usually 1 / sqrt(head_dim)
 *   causal    1: position p sees keys j <= p; 0: every cached key
 *   window    0, or with causal: only keys j > p - window
 * A row that sees no key (an empty sequence, a negative position, pages that
 * are not there) is zeros.  Codes and scales of tokens past kv_len may hold
 * anything.  A key or value that is not finite concerns the rows that see it,
 * with one exception: where a sequence has more than 48 query rows of a cache
 * head (max_q times q_heads / heads), a value's block of elements may be NaN in
 * rows that do not see it too.
 * Keys and values are taken to fp16 by a power of two that is shared by 64
 * tokens or more, seen or not: those below 2^-28 of the largest lose bits,
 * those below 2^-38 count as zeros.  (Keys up to 48 query rows are exempt.)
 * 2^100 and more is outside the range of values.
 *   workspace  device scratch of at least qmv_attention_4bit_workspace(...)
 *              bytes for the same arguments, 16-byte aligned, any contents
 *              (NULL when that is 0): partial results where the keys of a
 *              sequence are divided among workgroups.  Calls that share a
 *              workspace must not overlap.
 * The division depends on the arguments only, so results repeat bit for bit.
 */
size_t qmv_attention_4bit_workspace(const qmv_kv_cache *cache, const qmv_kv_batch *batch,
                                    int64_t tokens, int32_t q_heads, int64_t max_kv,
                                    int64_t window);
int qmv_attention_4bit(const qmv_heads *q, const qmv_kv_cache *cache, const qmv_kv_batch *batch,
                       int64_t tokens, int64_t max_kv, float scale, int32_t causal, int64_t window,
                       const qmv_heads *out, void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* QMV_ATTENTION_H */
