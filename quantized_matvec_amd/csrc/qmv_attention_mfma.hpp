// Building blocks of the matrix-core attention kernels: 4-bit codes to fp16
// operands, lane moves, and what one call passes to its kernels.
#pragma once

#include "qmv_attention.hpp"

namespace qmv {

typedef __attribute__((ext_vector_type(8))) _Float16 f16x8_t;
typedef __attribute__((ext_vector_type(4))) float f32x4_t;
typedef __attribute__((ext_vector_type(16))) float f32x16_t;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4_t;

struct AttnArgs {
  KVCache c;
  KVBatch kb;
  Heads q, out;
  int group;    // query heads of a cache head
  float scale;
  int max_kv;
  int window;   // 0: none
  bool causal;
  int qt;
};

// Keys [lo, hi) that token i of the sequence sees.  Both are within max_kv (below
// 2^31 - 1024, so positions a step past them do not overflow), whatever kv_len says.
__device__ __forceinline__ void key_range(const AttnArgs &a, const SeqRange &s, int i, int &lo,
                                          int &hi) {
  const int pos = s.pos0 + i;
  const int len = s.len < a.max_kv ? s.len : a.max_kv;
  hi = a.causal ? (pos + 1 < len ? pos + 1 : len) : len;
  lo = a.window > 0 && pos >= a.window ? pos - a.window + 1 : 0;
  lo = lo < len ? lo : len;
}

// The code values in fp16, times a factor: with 11 significant bits the NF4
// values alone are off by 1.6e-4 of their norm, times 1.6776895 by 6.2e-5 (the
// smallest over [1, 2)); the FP4 values times 6 are exact.  Scores and outputs
// are divided by the factor in fp32.
struct HalfTables {
  uint16_t value[2][16];   // by quant type and code
  uint16_t rest[16];       // what fp16 leaves of the NF4 values (to 3e-8)
  uint32_t pair[3][256];   // packed byte -> values of both codes, the even element low; [2]: rests
};
constexpr HalfTables half_tables() {
  HalfTables t{{{0xbeb6, 0xbcac, 0xbb0c, 0xb94d, 0xb7a3, 0xb4f6, 0xb0e3, 0x0000, 0x3046, 0x3452,
                 0x369b, 0x3889, 0x39ea, 0x3b8d, 0x3cda, 0x3eb6},
                {0x0000, 0x3800, 0x3c00, 0x3e00, 0x4000, 0x4200, 0x4400, 0x4600, 0x8000, 0xb800,
                 0xbc00, 0xbe00, 0xc000, 0xc200, 0xc400, 0xc600}},
               {0x02f0, 0x81c2, 0x834a, 0x0331, 0x05f1, 0x0456, 0x82dc, 0x0000, 0x8238, 0x81e1, 0x03d1, 0x0175, 0x07a1, 0x0335, 0x006a, 0x82f0},
               {}};
  for (int e = 0; e < 256; ++e) {
    t.pair[kNF4][e] = (uint32_t)t.value[kNF4][e >> 4] | ((uint32_t)t.value[kNF4][e & 15] << 16);
    t.pair[kFP4][e] = (uint32_t)t.value[kFP4][e >> 4] | ((uint32_t)t.value[kFP4][e & 15] << 16);
    t.pair[2][e] = (uint32_t)t.rest[e >> 4] | ((uint32_t)t.rest[e & 15] << 16);
  }
  return t;
}
__device__ constexpr HalfTables kHalf = half_tables();
__host__ __device__ inline float half_factor(int qt) { return qt == kNF4 ? 1.677689552307129f : 6.f; }

// A table in LDS from a packed byte to the fp16 pair of its two values (even
// element in the low half), and with REST the pair of what fp16 leaves of them
// beside it.  Byte e's entry is 256 bytes, a copy for each of 64 lanes (32
// with REST), so lanes never meet in a bank, and the address of (byte n of w,
// copy) is one byte permute of the two.
constexpr int kLutBytes = 256 * 256;

template <bool REST, int THREADS>
__device__ __forceinline__ void fill_lut(uint32_t *lut, int qt, int tid) {
  constexpr int N = (kLutBytes / 16 + THREADS - 1) / THREADS;
  uint32_t v[N], w[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int e = (tid + k * THREADS) / 16 & 255;
    v[k] = kHalf.pair[qt][e];
    w[k] = REST ? kHalf.pair[2][e] : v[k];
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int i = tid + k * THREADS;  // neighbours write neighbouring 16 bytes
    if (i < kLutBytes / 16) reinterpret_cast<uint4 *>(lut)[i] = make_uint4(v[k], w[k], v[k], w[k]);
  }
}
// The lane's copy, as a byte offset.
template <bool REST>
__device__ __forceinline__ uint32_t lut_copy(int lane) { return REST ? 8u * (lane & 31) : 4u * lane; }

// The entry of byte N of w.
template <int N>
__device__ __forceinline__ const uint32_t *lut_entry(const uint32_t *lut, uint32_t w, uint32_t copy) {
  const uint32_t off = __builtin_amdgcn_perm(w, copy, 0x0c0c0400u + (N << 8));
  return reinterpret_cast<const uint32_t *>(reinterpret_cast<const char *>(lut) + off);
}

// 8 codes (4 bytes) to 8 fp16 values in order.
__device__ __forceinline__ f16x8_t lut8(const uint32_t *lut, uint32_t w, uint32_t copy) {
  const u32x4_t v = {*lut_entry<0>(lut, w, copy), *lut_entry<1>(lut, w, copy),
                     *lut_entry<2>(lut, w, copy), *lut_entry<3>(lut, w, copy)};
  return __builtin_bit_cast(f16x8_t, v);
}

// Two elements (2 P, 2 P + 1) of 8 tokens, a byte each: the operands of both
// elements, 8 tokens in order, and those of the rests.
struct Pair8 {
  f16x8_t even, odd;
};
__device__ __forceinline__ Pair8 split_pairs(const uint32_t (&p)[8]) {
  u32x4_t e, o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    e[i] = __builtin_amdgcn_perm(p[2 * i + 1], p[2 * i], 0x05040100u);
    o[i] = __builtin_amdgcn_perm(p[2 * i + 1], p[2 * i], 0x07060302u);
  }
  return Pair8{__builtin_bit_cast(f16x8_t, e), __builtin_bit_cast(f16x8_t, o)};
}
template <bool REST>
__device__ __forceinline__ void lut8x2(const uint32_t *lut, uint32_t w0, uint32_t w1, uint32_t copy,
                                       Pair8 &value, Pair8 &rest) {
  const uint32_t *at[8] = {lut_entry<0>(lut, w0, copy), lut_entry<1>(lut, w0, copy),
                           lut_entry<2>(lut, w0, copy), lut_entry<3>(lut, w0, copy),
                           lut_entry<0>(lut, w1, copy), lut_entry<1>(lut, w1, copy),
                           lut_entry<2>(lut, w1, copy), lut_entry<3>(lut, w1, copy)};
  uint32_t v[8], x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (REST) {
      const uint2 y = *reinterpret_cast<const uint2 *>(at[i]);
      v[i] = y.x;
      x[i] = y.y;
    } else {
      v[i] = *at[i];
    }
  }
  value = split_pairs(v);
  if constexpr (REST) rest = split_pairs(x);
}

// v_permlane32_swap: the upper half of a changes places with the lower half
// of b; v_permlane16_swap: the odd rows of 16 lanes of a with the even ones of b.
__device__ __forceinline__ void swap32(uint32_t &a, uint32_t &b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ void swap16(uint32_t &a, uint32_t &b) {
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}

// Transposes the 4 x 4 grid of (register, row of 16 lanes).
__device__ __forceinline__ void transpose_rows(uint4 &w) {
  swap32(w.x, w.z);
  swap32(w.y, w.w);
  swap16(w.x, w.y);
  swap16(w.z, w.w);
}

// Maximum over the four rows of 16 lanes (lanes of equal l % 16).
__device__ __forceinline__ float rows_max(float v) {
  uint32_t a = __float_as_uint(v), b = a;
  swap32(a, b);
  v = fmaxf(__uint_as_float(a), __uint_as_float(b));
  a = b = __float_as_uint(v);
  swap16(a, b);
  return fmaxf(__uint_as_float(a), __uint_as_float(b));
}
__device__ __forceinline__ uint32_t f16_pair(float lo, float hi) {
  const f32x2_t v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2v_t));
}

// The 16 bytes of 8 cached scales as fp32.
template <int DT>
__device__ __forceinline__ void scales8(const uint4 &w, float (&s)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == kBF16) {
      s[2 * i] = __uint_as_float(u[i] << 16);
      s[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    } else {
      s[2 * i] = bits16_to_f32<DT>(u[i] & 0xffffu);
      s[2 * i + 1] = bits16_to_f32<DT>(u[i] >> 16);
    }
  }
}

// floor(log2 x) of a normal x > 0 (-127 below).
__device__ __forceinline__ int exponent_of(float x) {
  return (int)((__float_as_uint(x) >> 23) & 0xffu) - 127;
}

constexpr float kNoScore = -3e38f;  // running maximum of a row that has seen nothing

// A score's exponent s f - m is one multiply-add.  Its product is not rounded
// and m, the largest product, is, so all weights of a row carry a factor of up to
// 2^(|m| 2^-24): nothing below this |m|, past it more than fp16 has room for.
// There products are rounded before m is taken from them.
constexpr float kFarScore = 0x1p20f;
__device__ __forceinline__ bool is_far(float m) { return fabsf(m) >= kFarScore && m > kNoScore; }

// Results of a part of a row's keys: running maximum (in powers of two), sum of
// weights, and the weighted sum of values (not divided).
struct Partials {
  float *o;
  float2 *ml;
};

// The generic kernel: head sizes without a matrix-core kernel.
hipError_t launch_attention_rows(const AttnArgs &a, int dt, hipStream_t st);
// Up to 48 query rows (tokens times group) of a cache head.
bool decode_eligible(const KVCache &c, int64_t rows);
size_t decode_workspace_bytes(const KVCache &c, const KVBatch &kb, int rows, int64_t max_kv, int64_t window);
hipError_t launch_attention_decode(const AttnArgs &a, int dt, void *ws, hipStream_t st);
// Any number of query rows.
bool prompt_eligible(const KVCache &c);
size_t prompt_workspace_bytes(const KVCache &c, const KVBatch &kb, int q_heads, int64_t max_kv, int64_t window);
hipError_t launch_attention_prompt(const AttnArgs &a, int dt, void *ws, hipStream_t st);

}  // namespace qmv
