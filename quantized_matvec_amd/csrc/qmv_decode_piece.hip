// Pieces of a 4-bit weight as 16-bit operands of the tile product (qmv_tile.hpp).
#include "qmv_tuning.hpp"

namespace qmv {

// ---------------------------------------------------------------------------
// W[v][c] = round(T[code] a) of rows v and columns c0 + c, exactly as
// dequantize_4bit returns them in DT, and its transpose Wt[c][v], both up to a
// multiple of 64 along the sum with zeros: each where it is wanted, from one read
// of the codes.
//
// A workgroup takes 64 rows x 128 columns.  A thread decodes 8 columns of four
// rows (4 bytes of codes, one block), 16 threads a row, and stores their 16
// bytes of W; the transpose goes through LDS, whose 16-byte chunks are swizzled
// by row / 8, so that 8 lanes can take 8 rows each of a column, from 8 different
// bank groups, and store one whole line of it.  Bound by the writes: 4 bytes
// for each half byte read: 16384 x 4096, both forms, 68 us (4.4 TB/s); 4096 x 14336, the
// transpose alone, 45 us.
// ---------------------------------------------------------------------------
template <int DT, bool DQ>
__global__ __launch_bounds__(256) void decode_piece_kernel(const uint8_t *__restrict__ packed, Scales sc, int log2bs,
                                                           CodeValues table, int64_t K, int64_t c0, int64_t cols, int n,
                                                           uint16_t *__restrict__ W, int64_t ldw,
                                                           uint16_t *__restrict__ Wt, int64_t ldt) {
  __shared__ float tab[16];
  __shared__ __attribute__((aligned(16))) uint16_t tile[64][128];
  const int tid = threadIdx.x, row = tid >> 4, col = 8 * (tid & 15);
  const int64_t c = (int64_t)blockIdx.x * 128 + col;
  if (tid < 16) tab[tid] = table.v[tid];
  uint32_t w[4] = {};
  float a[4] = {};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t v = (int64_t)blockIdx.y * 64 + 16 * q + row;
    if (v < n && c < cols) {  // cols is a multiple of 32: a thread's 8 columns are all there or none is
      const int64_t e = v * K + c0 + c;
      w[q] = *reinterpret_cast<const uint32_t *>(packed + (e >> 1));
      a[q] = block_scale<DQ>(sc, e >> log2bs, DQ ? sc.offset[0] : 0.f);
    }
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t v = (int64_t)blockIdx.y * 64 + 16 * q + row;
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = cvt_pair<DT>(tab[w[q] >> (8 * i + 4) & 15] * a[q], tab[w[q] >> (8 * i) & 15] * a[q]);
    const uint4 out = make_uint4(o[0], o[1], o[2], o[3]);
    if (W && v < n && c < ldw) *reinterpret_cast<uint4 *>(W + v * ldw + c) = out;  // past cols: zeros
    *reinterpret_cast<uint4 *>(&tile[16 * q + row][col ^ (8 * ((16 * q + row) >> 3 & 7))]) = out;
  }
  if (!Wt) return;
  __syncthreads();
  const int r8 = tid & 7;  // rows 8 r8 .. + 7
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int oc = 32 * q + (tid >> 3);
    const int64_t at = (int64_t)blockIdx.x * 128 + oc;
    if (at >= cols) return;
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = tile[8 * r8 + 2 * i][oc ^ (8 * r8)] | (uint32_t)tile[8 * r8 + 2 * i + 1][oc ^ (8 * r8)] << 16;
    *reinterpret_cast<uint4 *>(Wt + at * ldt + blockIdx.y * 64 + 8 * r8) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

hipError_t launch_decode_piece(const Weight4 &w, int dt, int64_t c0, int64_t cols, void *W, int64_t ldw, void *Wt,
                               int64_t ldt, hipStream_t st) {
  const int n = (int)w.N, np = (n + 63) & ~63;
  const dim3 grid((unsigned)((cols + 127) / 128), (unsigned)(np / 64));
#define QMV_D(DT, DQV)                                                                                              \
  hipLaunchKernelGGL((decode_piece_kernel<DT, DQV>), grid, dim3(256), 0, st, w.packed, w.sc, w.log2bs,              \
                     code_values(w.qt), w.K, c0, cols, n, static_cast<uint16_t *>(W), ldw, static_cast<uint16_t *>(Wt), ldt)
  if (dt == kF16) {
    if (w.dq) QMV_D(kF16, true);
    else QMV_D(kF16, false);
  } else {
    if (w.dq) QMV_D(kBF16, true);
    else QMV_D(kBF16, false);
  }
#undef QMV_D
  return hipGetLastError();
}

// Rows [T, L] with zeros up to Lp elements (multiples of 8, L of 32): a sum's last
// 32 terms must not meet what lies behind a row.
__global__ __launch_bounds__(256) void pad_rows_kernel(const uint4 *__restrict__ in, int64_t T, int L8, int Lp8,
                                                       uint4 *__restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= T * Lp8) return;
  const int64_t t = i / Lp8;
  const int c = (int)(i % Lp8);
  out[i] = c < L8 ? in[t * L8 + c] : make_uint4(0, 0, 0, 0);
}

hipError_t launch_pad_rows(const void *in, int64_t T, int64_t L, int64_t Lp, void *out, hipStream_t st) {
  hipLaunchKernelGGL(pad_rows_kernel, dim3((unsigned)((T * (Lp / 8) + 255) / 256)), dim3(256), 0, st,
                     static_cast<const uint4 *>(in), T, (int)(L / 8), (int)(Lp / 8), static_cast<uint4 *>(out));
  return hipGetLastError();
}

__global__ __launch_bounds__(256) void sum_parts_kernel(float *__restrict__ sums, int parts, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * 1024 + threadIdx.x;
  float sum[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) sum[q] = i + 256 * q < n ? sums[i + 256 * q] : 0.f;
#pragma unroll 4
  for (int s = 1; s < parts; ++s)
#pragma unroll
    for (int q = 0; q < 4; ++q) sum[q] += sums[s * n + min(i + 256 * q, n - 1)];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (i + 256 * q < n) sums[i + 256 * q] = sum[q];
}

hipError_t launch_sum_parts(float *sums, int parts, int64_t n, hipStream_t st) {
  hipLaunchKernelGGL(sum_parts_kernel, dim3((unsigned)((n + 1023) / 1024)), dim3(256), 0, st, sums, parts, n);
  return hipGetLastError();
}

}  // namespace qmv
