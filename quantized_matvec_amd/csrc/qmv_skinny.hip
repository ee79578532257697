// C[s][M, N] = A[M, K_s] W^[N, K_s]^T for up to 64 rows, in fp32, a part for each
// slice K_s of the sum: the projection of a decode step with adapters, and the
// logits of a few tokens, whose next kernels add the parts up in order.
#include "qmv_tile.hpp"

namespace qmv {

// ---------------------------------------------------------------------------
// A workgroup of 8 waves keeps a slice of 512 terms of A in LDS, in the order of
// the matrix cores' operands, and goes over columns, 32 a wave at a time: the next
// columns' packed weights (16 bytes a lane for 64 terms) and scales are on their
// way while these are decoded and multiplied, 64 terms at a step.  A byte is one
// v_perm_b32 (its address) and one LDS read of both its table values, from a
// table that every lane has a copy of in a bank of its own.  Blocks are 64 terms
// or more, so a step's products are sums of rounded table value times activation,
// and the block's scale, which is its column's, is applied to the sum in fp32.
//
// One workgroup a compute unit (its LDS), which reads its rows of A once: a
// kernel that takes all of K for 32 columns reads 256 KB of A (32 rows of 4096)
// for each 64 KB of weights.  14336 x 4096, 32 rows 20 us (26 by gemm_4bit's kernel): one turn
// of loads, decoding and stores that wait for each other, 1.5 TB/s of codes and 14.7 MB of parts.
// ---------------------------------------------------------------------------
constexpr int kSlice = 512, kSteps = kSlice / 64;

template <int DT, bool DQ, int MT>
__global__ __launch_bounds__(512, 2) void skinny_4bit_kernel(const uint16_t *__restrict__ A, int M, int64_t N, int64_t K,
                                                             const uint8_t *__restrict__ packed, Scales sc, int log2bs,
                                                             CodeValues table, float *__restrict__ parts) {
  typedef __attribute__((ext_vector_type(4))) uint32_t u32x4_t;
  __shared__ uint32_t lut[256 * 64];  // byte, lane -> table values of its high and low nibble, 16 bits each
  __shared__ u32x4_t rows[MT][kSteps * 8 * 32];
  __shared__ float code2[256];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l32 = lane & 31, h = lane >> 5;
  const int64_t k0 = (int64_t)blockIdx.y * kSlice;
  const int steps = (int)((K - k0 < kSlice ? K - k0 : kSlice) / 64);
  struct Group {  // 32 columns' weights and scales; steps past the end take the last one's
    u32x4_t w[kSteps];
    float s[kSteps];
    uint32_t q[kSteps];
  };
  const int64_t groups = (N + 31) / 32, stride = (int64_t)gridDim.x * 8;
  auto load = [&](int64_t group, Group &g) __attribute__((always_inline)) {
    const int64_t n = 32 * group + l32, row0 = (n < N ? n : N - 1) * K + k0;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int64_t e = row0 + 64 * min(i, steps - 1);
      g.w[i] = *reinterpret_cast<const u32x4_t *>(packed + (e + 32 * h) / 2);
      if constexpr (DQ) {
        g.q[i] = sc.q[e >> log2bs];
        g.s[i] = sc.absmax2[(e >> log2bs) >> sc.log2bs2];
      } else {
        g.s[i] = sc.absmax[e >> log2bs];
      }
    }
  };
  int64_t group = (int64_t)blockIdx.x * 8 + wave;
  Group g0, g1;
  load(group < groups ? group : groups - 1, g0);
  {  // rows: 16-byte chunk kc of row m to chunk ((kc / 8 * 4 + kc % 4) * 2 + kc / 4 % 2) * 32 + m; then the tables
    u32x4_t v[MT][kSteps / 2];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int i = 0; i < kSteps / 2; ++i) {
        const int m = 32 * t + (tid >> 4), kc = 16 * i + (tid & 15);
        v[t][i] = *reinterpret_cast<const u32x4_t *>(A + (int64_t)min(m, M - 1) * K + k0 + 8 * min(kc, 8 * steps - 1));
        v[t][i] &= m < M ? ~0u : 0u;
      }
    const uint32_t hi = f32_to_bits16<DT>(table.v[(tid >> 5) & 15]);  // 32 threads an entry of 16 high nibbles
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const uint32_t both = hi | f32_to_bits16<DT>(table.v[q]) << 16;
      // entry 16 (tid / 32) + q, copies 2 (tid % 32) and + 1
      *reinterpret_cast<uint2 *>(&lut[(16 * (tid >> 5) + q) * 64 + 2 * (tid & 31)]) = make_uint2(both, both);
    }
    if (DQ && tid < 256) code2[tid] = sc.code2[tid];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int i = 0; i < kSteps / 2; ++i) {
        const int kc = 16 * i + (tid & 15);
        rows[t][((kc / 8 * 4 + (kc & 3)) * 2 + ((kc >> 2) & 1)) * 32 + (tid >> 4)] = v[t][i];
      }
  }
  const float offset = DQ ? sc.offset[0] : 0.f;
  __syncthreads();
  const uint32_t lane4 = (uint32_t)lane << 2;
  const char *lut_b = reinterpret_cast<const char *>(lut);
  auto multiply = [&](int64_t group, const Group &g) __attribute__((always_inline)) {
    tile_acc_t acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[t][r] = 0.f;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      if (i >= steps) break;
      tile_acc_t sum[MT];
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) sum[t][r] = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t b[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)  // byte e of the word, times 256, and this lane's copy
          b[e] = *reinterpret_cast<const uint32_t *>(lut_b + __builtin_amdgcn_perm(g.w[i][j], lane4, 0x0c0c0000u | ((4u + e) << 8)));
        const frag_t bf = __builtin_bit_cast(frag_t, make_uint4(b[0], b[1], b[2], b[3]));
#pragma unroll
        for (int t = 0; t < MT; ++t)
          sum[t] = tile_mma<DT>(__builtin_bit_cast(frag_t, rows[t][((4 * i + j) * 2 + h) * 32 + l32]), bf, sum[t]);
      }
      float a = g.s[i];
      if constexpr (DQ) {
#pragma clang fp contract(off)
        const float p = code2[g.q[i]] * a;
        a = p + offset;
      }
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[t][r] = fmaf(a, sum[t][r], acc[t][r]);
    }
    const int64_t n = 32 * group + l32;
    if (n >= N) return;
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int m = 32 * t + 8 * (r >> 2) + 4 * h + (r & 3);
        if (m < M) parts[((int64_t)blockIdx.y * M + m) * N + n] = acc[t][r];
      }
  };
  if constexpr (MT > 1) {  // a second set does not fit the registers: the other wave of the SIMD multiplies meanwhile
    for (; group < groups; group += stride) {
      multiply(group, g0);
      load(min(group + stride, groups - 1), g0);
    }
    return;
  }
  for (; group < groups; group += 2 * stride) {  // past the end: the last columns again, not multiplied
    load(min(group + stride, groups - 1), g1);
    multiply(group, g0);
    load(min(group + 2 * stride, groups - 1), g0);
    if (group + stride < groups) multiply(group + stride, g1);
  }
}

int skinny_parts(int64_t K) {
  return (int)((K + kSlice - 1) / kSlice);
}

// Both sides, us without the adding up of parts / gemm_4bit: 14336 x 4096, 16 rows 19.1 / 18.2, 17 rows 19.5 / 21.1,
// 32 rows 20.2 / 26.4, 64 rows 25.7 / 44.9; 128256 x 4096, 16 rows 109 / 120, 32 rows 119 / 182
bool skinny_fits(int64_t M, int64_t K, int log2bs) {
  return M > 16 && M <= 64 && K % 64 == 0 && log2bs >= 6 && skinny_parts(K) <= 16;
}


hipError_t launch_skinny(const void *A, int dt, int64_t M, const Weight4 &w, float *parts, hipStream_t st) {
  const int64_t wanted = (w.N + 255) / 256;  // workgroups for one turn of 32 columns a wave
  int64_t each = device_cu_count() / skinny_parts(w.K);
  if (each < 1) each = 1;
  const dim3 grid((unsigned)(wanted < each ? wanted : each), (unsigned)skinny_parts(w.K));
  const uint16_t *a = static_cast<const uint16_t *>(A);
#define QMV_S(DT, DQV, MT)                                                                                          \
  hipLaunchKernelGGL((skinny_4bit_kernel<DT, DQV, MT>), grid, dim3(512), 0, st, a, (int)M, w.N, w.K, w.packed, w.sc, \
                     w.log2bs, code_values(w.qt), parts)
#define QMV_SD(DT)                    \
  if (M <= 32) {                      \
    if (w.dq) QMV_S(DT, true, 1);     \
    else QMV_S(DT, false, 1);         \
  } else {                            \
    if (w.dq) QMV_S(DT, true, 2);     \
    else QMV_S(DT, false, 2);         \
  }
  if (dt == kF16) { QMV_SD(kF16); }
  else { QMV_SD(kBF16); }
#undef QMV_SD
#undef QMV_S
  return hipGetLastError();
}

}  // namespace qmv
