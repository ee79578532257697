// Rotary positions: the table of cosines and sines, and the rotation of
// queries and keys by it, forward and inverse.
//
// A pair (a, b) of a head's elements at position p, with (c, s) the table's
// entry of p and of the pair, becomes (a c - b s, b c + a s).  The rotation is
// orthogonal (times the table's gain), so its backward is the rotation by
// (c, -s).  Products and sums are rounded one by one in fp32 (no fused
// multiply-add), so the result is a function of the operands alone and the
// cache append gets the same bits; the one rounding to the heads' type comes
// last.
#include <algorithm>

#include "qmv_attention.hpp"

#pragma clang fp contract(off)

namespace qmv {

struct Freqs {
  double f[128];
};

// Angles in float64: at position 2^20 an fp32 angle would be off by 2^-4.  Bound
// by the float64 sines, once for a model: 131072 positions of 64 pairs 32 us.
__global__ __launch_bounds__(256) void rope_table_kernel(Freqs fr, int half, int64_t n, double gain,
                                                         float2 *__restrict__ table) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t pos = i / half;
    double s, c;
    sincos((double)pos * fr.f[i - pos * half], &s, &c);
    table[i] = make_float2((float)(gain * c), (float)(gain * s));
  }
}

hipError_t launch_rope_table(const double *freqs, int half, int64_t max_pos, double gain,
                             float *table, hipStream_t st) {
  Freqs fr{};
  for (int i = 0; i < half; ++i) fr.f[i] = freqs[i];
  const int64_t n = max_pos * half;
  const unsigned grid = (unsigned)std::min<int64_t>((n + 255) / 256, 16384);
  hipLaunchKernelGGL(rope_table_kernel, dim3(grid), dim3(256), 0, st, fr, half, n, gain,
                     reinterpret_cast<float2 *>(table));
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// rotary
//
// Bound by memory: every element is read and written once.  A unit of work is
// what one thread loads and stores: V pairs as two runs of V elements (halves),
// V / 2 pairs as one run (interleaved), or V elements that are only copied.
// Each unit reads its own elements only, so the output may be the input.
// V is the widest run that the pair count allows: 8 elements, else 4 (half of
// the rotated part a multiple of 4), else single pairs.
// 16384 tokens of 32 + 8 heads of 128 in bf16 (336 MB): 63.5 us, 5.3 TB/s, the
// rate of a large copy; 8198 tokens of 64 + 8 heads, 64 of 128 elements turned
// as neighbours, fp16: 60.3 us, 5.0 TB/s.  16 tokens: 3.3 us, a launch.
// ---------------------------------------------------------------------------
template <int DT, int V>
__device__ __forceinline__ void load_run(const void *base, int64_t at, float (&x)[V]) {
  if constexpr (DT == kF32) {
    const float *p = static_cast<const float *>(base) + at;
    if constexpr (V % 4 == 0) {
#pragma unroll
      for (int i = 0; i < V / 4; ++i) {
        const float4 v = reinterpret_cast<const float4 *>(p)[i];
        x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = p[i];
    }
  } else {
    const uint16_t *p = static_cast<const uint16_t *>(base) + at;
    if constexpr (V == 1) {
      x[0] = bits16_to_f32<DT>(p[0]);
    } else {
      typedef uint32_t words __attribute__((ext_vector_type(V / 2)));
      uint32_t w[V / 2];
      __builtin_memcpy(w, __builtin_assume_aligned(p, sizeof(words)), sizeof(words));
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        x[2 * i] = bits16_to_f32<DT>(w[i] & 0xffffu);
        x[2 * i + 1] = bits16_to_f32<DT>(w[i] >> 16);
      }
    }
  }
}

template <int DT, int V>
__device__ __forceinline__ void store_run(void *base, int64_t at, const float (&x)[V]) {
  if constexpr (DT == kF32) {
    float *p = static_cast<float *>(base) + at;
    if constexpr (V % 4 == 0) {
#pragma unroll
      for (int i = 0; i < V / 4; ++i)
        reinterpret_cast<float4 *>(p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) p[i] = x[i];
    }
  } else {
    uint16_t *p = static_cast<uint16_t *>(base) + at;
    if constexpr (V == 1) {
      store_elem<DT>(p, 0, x[0]);
    } else {
      uint32_t w[V / 2];
#pragma unroll
      for (int i = 0; i < V / 2; ++i) w[i] = cvt_pair<DT>(x[2 * i], x[2 * i + 1]);
      __builtin_memcpy(__builtin_assume_aligned(p, 2 * V), w, sizeof(w));
    }
  }
}

struct RotaryArgs {
  Heads q, qo, k, ko;
  Rope rope;
  const int64_t *positions;
  int64_t tokens;
  int dim;
  int per_head;   // units of a head
  int head_sets;  // threads along the heads of a token
  int per_token;  // threads of a token: head_sets * per_head
};

// A thread takes the same unit of HP heads of a token (head_sets apart): the
// position and the angles are fetched once, and HP heads' elements are in
// flight together.
template <int DT, int V, bool INTER, int HP>
__global__ __launch_bounds__(256) void rotary_kernel(RotaryArgs a, float sign) {
  const int64_t base = (int64_t)blockIdx.x * 256;
  const int64_t t0 = base / a.per_token;
  const uint32_t u = (uint32_t)(base - t0 * a.per_token) + threadIdx.x;
  const int64_t t = t0 + u / (uint32_t)a.per_token;
  if (t >= a.tokens) return;
  const uint32_t w = u % (uint32_t)a.per_token;
  const int h0 = (int)(w / (uint32_t)a.per_head);
  const int i = (int)(w % (uint32_t)a.per_head);
  const int half = a.rope.half;
  const int64_t pos = a.positions[t];
  const bool there = pos >= 0 && pos < a.rope.max_pos;
  const float2 *cs = a.rope.table + (there ? pos : 0) * half;

  constexpr int NP = INTER ? V / 2 : V;  // pairs of a unit
  const int turned = half / NP;          // units that turn
  const bool turns = i < turned;
  const int at = turns ? i * V : 2 * half + (i - turned) * V;
  const int at2 = !INTER && turns ? half + i * V : at;  // the run of the pairs' second elements
  const void *xp[HP];
  void *yp[HP];
  int64_t xo[HP], yo[HP];
  bool real[HP];
#pragma unroll
  for (int n = 0; n < HP; ++n) {
    int h = h0 + n * a.head_sets;
    real[n] = h < a.q.heads + a.k.heads;
    h = real[n] ? h : h0;  // one that is there
    const bool isk = h >= a.q.heads;
    if (isk) h -= a.q.heads;
    const Heads &x = isk ? a.k : a.q;
    const Heads &y = isk ? a.ko : a.qo;
    xp[n] = x.p, yp[n] = y.p;
    xo[n] = t * x.ts + h * x.hs;
    yo[n] = t * y.ts + h * y.hs;
  }
  float e[HP][V], f[HP][V];
#pragma unroll
  for (int n = 0; n < HP; ++n) {
    load_run<DT, V>(xp[n], xo[n] + at, e[n]);
    if constexpr (!INTER) load_run<DT, V>(xp[n], xo[n] + at2, f[n]);
  }
  float c[NP], s[NP];
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    const float2 v = cs[turns ? i * NP + j : 0];
    c[j] = v.x;
    s[j] = sign * v.y;
  }
#pragma unroll
  for (int n = 0; n < HP; ++n) {
    if (!real[n]) continue;
    float r[V], g[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if constexpr (INTER) {
        const float o = e[n][j ^ 1];
        r[j] = j & 1 ? e[n][j] * c[j / 2] + o * s[j / 2] : e[n][j] * c[j / 2] - o * s[j / 2];
      } else {
        r[j] = e[n][j] * c[j] - f[n][j] * s[j];
        g[j] = f[n][j] * c[j] + e[n][j] * s[j];
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      r[j] = there ? (turns ? r[j] : e[n][j]) : 0.f;
      if constexpr (!INTER) g[j] = there ? g[j] : 0.f;
    }
    store_run<DT, V>(yp[n], yo[n] + at, r);
    if constexpr (!INTER) {
      if (turns) store_run<DT, V>(yp[n], yo[n] + at2, g);
    }
  }
}

template <int DT, int V, bool INTER>
static hipError_t launch_rotary_t(RotaryArgs &a, float sign, hipStream_t st) {
  constexpr int HP = 4;
  const int half = a.rope.half, heads = a.q.heads + a.k.heads;
  a.per_head = half / (INTER ? V / 2 : V) + (a.dim - 2 * half) / V;
  // Four heads a thread where that leaves 8 workgroups for each compute unit:
  // the two large calls above take 64 and 60 us so, 74 and 79 us with one head
  // a thread.  With few workgroups there is nothing to hide latency behind: 64
  // tokens of 40 heads of 128 4.4 us with four, 3.2 with one, 512 tokens 5.1 and
  // 5.0.  The rule is on the safe side, the two being even from about 1500 tokens
  // on (2048: 10.5 and 11.2, 6144, just below it: 22.7 and 26).
  const bool many = a.tokens * a.per_head * heads >= (int64_t)HP * 256 * 8 * device_cu_count() && heads >= HP;
  a.head_sets = many ? (heads + HP - 1) / HP : heads;
  a.per_token = a.per_head * a.head_sets;
  const int64_t wgs = (a.tokens * a.per_token + 255) / 256;
  if (!grid_fits(wgs, 256)) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)wgs);
  if (many) hipLaunchKernelGGL((rotary_kernel<DT, V, INTER, HP>), grid, dim3(256), 0, st, a, sign);
  else hipLaunchKernelGGL((rotary_kernel<DT, V, INTER, 1>), grid, dim3(256), 0, st, a, sign);
  return hipGetLastError();
}

template <int DT>
static hipError_t launch_rotary_d(RotaryArgs &a, float sign, hipStream_t st) {
  const int half = a.rope.half;
  if (a.rope.interleaved) {
    if (half % 4 == 0) return launch_rotary_t<DT, 8, true>(a, sign, st);
    return launch_rotary_t<DT, 2, true>(a, sign, st);
  }
  if (half % 8 == 0) return launch_rotary_t<DT, 8, false>(a, sign, st);
  if (half % 4 == 0) return launch_rotary_t<DT, 4, false>(a, sign, st);
  return launch_rotary_t<DT, 1, false>(a, sign, st);
}

hipError_t launch_rotary(const Heads &q, const Heads &qo, const Heads &k, const Heads &ko, int dt,
                         int64_t tokens, int dim, const int64_t *positions, const Rope &rope,
                         bool inverse, hipStream_t st) {
  RotaryArgs a{q, qo, k, ko, rope, positions, tokens, dim, 0, 0, 0};
  const float sign = inverse ? -1.f : 1.f;
  if (dt == kF32) return launch_rotary_d<kF32>(a, sign, st);
  return dt == kF16 ? launch_rotary_d<kF16>(a, sign, st) : launch_rotary_d<kBF16>(a, sign, st);
}

}  // namespace qmv
