// Kernel-side views shared by the rotary, cache and attention kernels, and
// their host launchers (internal to libqmv.so).  Launchers assume that the C
// ABI layer checked their arguments.
#pragma once

#include "qmv_launch.hpp"

namespace qmv {

// Head vectors [tokens, heads, head_dim]; strides in elements.
struct Heads {
  void *p;
  int64_t ts, hs;
  int heads;
};

struct Rope {
  const float2 *table;  // [max_pos, half] (cos, sin)
  int64_t max_pos;
  int half;             // pairs
  bool interleaved;
};

struct KVCache {
  uint8_t *kc, *vc;
  uint16_t *ks, *vs;
  int64_t num_pages;
  int heads;
  int log2page;
  int dim;
  int bs;
};

struct KVBatch {
  const int32_t *bt;
  int64_t bt_stride;
  const int32_t *kv_len;
  const int32_t *cu;  // NULL: one token for each sequence
  int batch, max_pages, max_q;
  int64_t tokens;
};

// The tokens of sequence b: the first one's row among the call's tokens, how
// many there are, and the position of the first.  Offsets are held inside
// [0, tokens], so nothing that cu says leads out of the operands.
struct SeqRange {
  int64_t row0;
  int n;
  int pos0;
  int len;
};
__device__ __forceinline__ SeqRange seq_range(const KVBatch &kb, int b) {
  SeqRange s;
  if (kb.cu) {
    int64_t lo = kb.cu[b], hi = kb.cu[b + 1];
    lo = lo < 0 ? 0 : (lo > kb.tokens ? kb.tokens : lo);
    hi = hi < lo ? lo : (hi > kb.tokens ? kb.tokens : hi);
    s.row0 = lo;
    s.n = (int)(hi - lo);
  } else {
    s.row0 = b;
    s.n = b < kb.tokens ? 1 : 0;
  }
  const int len = kb.kv_len[b];
  s.len = len < 0 ? 0 : len;
  s.pos0 = s.len - s.n;  // above -2^31: n <= tokens < 2^31
  return s;
}

// Page of position pos of sequence b, or -1 where there is none.
__device__ __forceinline__ int64_t page_of(const KVBatch &kb, const KVCache &c, int b, int pos) {
  const int i = pos >> c.log2page;
  if (pos < 0 || i >= kb.max_pages) return -1;
  const int p = kb.bt[(int64_t)b * kb.bt_stride + i];
  return p >= 0 && p < c.num_pages ? p : -1;
}

// Byte offsets of a page's head in the code arrays (head_dim / 2 bytes a
// token) and element offsets in the scale arrays, in 64 bits: a long cache
// passes 2^32 bytes.
__device__ __forceinline__ int64_t code_base(const KVCache &c, int64_t page, int h) {
  return ((page * c.heads + h) << c.log2page) * (c.dim >> 1);
}
__device__ __forceinline__ int64_t scale_base(const KVCache &c, int64_t page, int h) {
  return ((page * c.heads + h) << c.log2page) * (c.dim / c.bs);
}

// HIP takes fewer than 2^32 threads along a dimension of a grid.  The launchers
// return hipErrorInvalidConfiguration, and launch nothing, where a call needs more.
inline bool grid_fits(int64_t workgroups, int threads) { return workgroups * threads < ((int64_t)1 << 32); }

hipError_t launch_rope_table(const double *freqs, int half, int64_t max_pos, double gain,
                             float *table, hipStream_t st);
hipError_t launch_rotary(const Heads &q, const Heads &qo, const Heads &k, const Heads &ko, int dt,
                         int64_t tokens, int dim, const int64_t *positions, const Rope &rope,
                         bool inverse, hipStream_t st);
// mids: midpoints of the code table; rope.table NULL: keys not turned.
hipError_t launch_kv_append(const KVCache &c, int dt, int qt, const Midpoints4 &mids,
                            const KVBatch &kb, const Heads &k, const Heads &v, const Rope &rope,
                            const Heads &q, const Heads &qo, hipStream_t st);
hipError_t launch_kv_dequantize(const KVCache &c, int dt, int qt, const KVBatch &kb,
                                const Heads &k, const Heads &v, hipStream_t st);

size_t attention_workspace_bytes(const KVCache &c, const KVBatch &kb, int q_heads, int64_t max_kv,
                                 int64_t window);
hipError_t launch_attention(const KVCache &c, int dt, int qt, const KVBatch &kb, const Heads &q,
                            int64_t max_kv, float scale, bool causal, int64_t window,
                            const Heads &out, void *ws, hipStream_t st);

}  // namespace qmv
