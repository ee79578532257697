// Shared by the kernels of include/qmv/tuning.h: low-rank adapters beside a
// 4-bit projection, and losses over a 4-bit vocabulary.
#pragma once

#include "qmv_launch.hpp"

namespace qmv {

struct Weight4 {
  const uint8_t *packed;
  Scales sc;
  bool dq;
  int64_t N, K;
  int log2bs, qt;
};

// Rows [first, first + n).  first * K / blocksize has to be a multiple of the
// second-level group: first a multiple of 4096, the largest group, always is.
inline Weight4 rows_of(const Weight4 &w, int64_t first, int64_t n) {
  Weight4 r = w;
  const int64_t block = (first * w.K) >> w.log2bs;
  r.packed += first * w.K / 2;
  if (w.dq) {
    r.sc.q += block;
    r.sc.absmax2 += block >> w.sc.log2bs2;
  } else {
    r.sc.absmax += block;
  }
  r.N = n;
  return r;
}

// Rows of a weight and its columns [c0, c0 + cols) as 16-bit values W [N, ldw] and
// their transpose Wt [cols, ldt], either NULL; ldw and ldt reach over cols and N up to
// a multiple of 64, with zeros.
hipError_t launch_decode_piece(const Weight4 &w, int dt, int64_t c0, int64_t cols, void *W, int64_t ldw, void *Wt,
                               int64_t ldt, hipStream_t st);
hipError_t launch_pad_rows(const void *in, int64_t T, int64_t L, int64_t Lp, void *out, hipStream_t st);

// All of W alone: dequantize_4bit's kernel, where no zeros are needed.
inline hipError_t launch_decode_rows(const Weight4 &w, int dt, void *W, int64_t ldw, hipStream_t st) {
  if (ldw != w.K) return launch_decode_piece(w, dt, 0, w.K, W, ldw, nullptr, 0, st);
  return launch_dequantize_4bit(w.packed, w.sc, w.dq, w.N * w.K, w.log2bs, w.qt, W, dt, st);
}

inline int64_t to64(int64_t v) { return (v + 63) & ~(int64_t)63; }

// Whether gemm_4bit_backward is the quickest way to M rows of [N, K] of up to some hundred rows: it has to take its
// kernel that divides the sum among workgroups, and the last workgroup of each 128 x 256 tile then adds up all parts of
// it, about 1.2 us each (19 rows of 4608 x 768: 98 us, 84 of them for 72 parts).  The other way decodes the weight and
// multiplies that (qmv_tile.hpp).  The rule is a line between 2.5 us for each of 256 / tiles parts (also where N / 64
// is less, the most there can be) and 1 us for 2^20 weights and 24 us.  Both sides, us of lora_4bit_backward with rank 16
// by gemm_4bit_backward / by the other: 19 rows of 4608 x 768 135 / 73, 200 rows of 8192 x 4096 101 / 112.  Over
// K from 256 to 8192, N from 512 to 32768 and 19 to 600 rows it is 3 % above the faster side on average; farthest are
// 600 rows (14336 x 4096 237 / 171: takes the first) and small weights (64 rows of 512 x 768, a loss with its gradient,
// 51 / 61: takes the second).
inline bool fast_backward(int64_t M, int64_t N, int64_t K, int log2bs) {
  if (N % 64 || K % 256 || log2bs < 6) return false;
  return (N * K >> 20) >= 166000 / (K * ((M + 127) / 128)) - 24;
}

// Sums that came in parts, n values apart: added up in order, the sum left in the first.
hipError_t launch_sum_parts(float *sums, int parts, int64_t n, hipStream_t st);

// Up to 64 rows times a weight, in fp32, in parts [skinny_parts][M][N] that the caller adds up.
bool skinny_fits(int64_t M, int64_t K, int log2bs);
int skinny_parts(int64_t K);
hipError_t launch_skinny(const void *A, int dt, int64_t M, const Weight4 &w, float *parts, hipStream_t st);

struct Lora {
  const uint16_t *down, *up;
  const float *scale;
  int count, rank;
};

// fp32 values of the 16 codes, as a kernel argument.
struct CodeValues {
  float v[16];
};
inline CodeValues code_values(int qt) {
  CodeValues t;
  for (int c = 0; c < 16; ++c) t.v[c] = __builtin_bit_cast(float, table_bits(qt)[c]);
  return t;
}

// A workspace is handed out from its start in pieces of 256 bytes.
struct Carver {
  size_t at = 0;
  size_t take(size_t bytes) {
    const size_t p = at;
    at += (bytes + 255) & ~(size_t)255;
    return p;
  }
};

size_t lora_workspace(int64_t T, int64_t N, int64_t K, int log2bs, int count, int rank, bool backward);
hipError_t launch_lora(const void *x, int dt, int64_t T, const Weight4 &w, const Lora &l, const int32_t *index,
                       const void *bias, void *y, int y_dt, char *ws, hipStream_t st);
hipError_t launch_lora_backward(const void *dy, const void *x, int dt, int64_t T, const Weight4 &w, const Lora &l,
                                const int32_t *index, void *dx, void *d_down, void *d_up, int grad_dt, char *ws,
                                hipStream_t st);

// What a loss is taken against: one target a token (teacher NULL), or k ids
// with a teacher's logits.
struct Targets {
  const int64_t *ids;
  const void *teacher;
  int teacher_dt, k;
  float inv_tau;
};

size_t loss_workspace(int64_t T, int64_t V, int64_t K, int log2bs, int k, bool grad);
hipError_t launch_loss(const void *x, int dt, int64_t T, const Weight4 &w, const Targets &tg, const float *dloss,
                       void *loss, int loss_dt, void *dx, char *ws, hipStream_t st);

// Sums and maxima over a wave, every lane's result the same: a fixed tree.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}

// The two 16-bit elements of a word.
template <int DT>
__device__ __forceinline__ float lo16(uint32_t w) {
  if constexpr (DT == kBF16) return __uint_as_float(w << 16);
  else return (float)__builtin_bit_cast(_Float16, (uint16_t)w);
}
template <int DT>
__device__ __forceinline__ float hi16(uint32_t w) {
  if constexpr (DT == kBF16) return __uint_as_float(w & 0xffff0000u);
  else return (float)__builtin_bit_cast(_Float16, (uint16_t)(w >> 16));
}
template <int DT>
__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]) {
  f[0] = lo16<DT>(v.x), f[1] = hi16<DT>(v.x), f[2] = lo16<DT>(v.y), f[3] = hi16<DT>(v.y);
  f[4] = lo16<DT>(v.z), f[5] = hi16<DT>(v.z), f[6] = lo16<DT>(v.w), f[7] = hi16<DT>(v.w);
}

}  // namespace qmv
