// Pieces of a 4-bit weight as 16-bit operands of the tile product (qmv_tile.hpp).
#include "qmv_tuning.hpp"

namespace qmv {

// ---------------------------------------------------------------------------
// W[v][c] = round(T[code] a) of rows v and columns c0 + c, exactly as
// dequantize_4bit returns them in DT, and its transpose Wt[c][v], rows past the
// last as zeros there: each where it is wanted, from one read of the codes.
//
// A workgroup takes 64 rows x 64 columns.  A thread decodes 16 columns of a row
// (8 bytes of codes, one block) and stores its 32 bytes of W; the transpose goes
// through LDS, from which lane c of wave w takes column c's rows 16 w .. + 15.
// Bound by the writes: 4 bytes for each half byte read.
// ---------------------------------------------------------------------------
template <int DT, bool DQ>
__global__ __launch_bounds__(256) void decode_piece_kernel(const uint8_t *__restrict__ packed, Scales sc, int log2bs,
                                                           CodeValues table, int64_t K, int64_t c0, int n,
                                                           uint16_t *__restrict__ W, int64_t ldw,
                                                           uint16_t *__restrict__ Wt, int64_t ldt) {
  __shared__ float tab[16];
  __shared__ __attribute__((aligned(16))) uint16_t tile[64][72];
  const int tid = threadIdx.x, row = tid >> 2, col = 16 * (tid & 3);
  const int v = blockIdx.y * 64 + row, c = blockIdx.x * 64 + col;
  if (tid < 16) tab[tid] = table.v[tid];
  __syncthreads();
  uint32_t out[8] = {};
  if (v < n && c0 + c < K) {  // K is a multiple of 32: a thread's 16 columns are all there or none is
    const int64_t e = (int64_t)v * K + c0 + c;
    const float a = block_scale<DQ>(sc, e >> log2bs, DQ ? sc.offset[0] : 0.f);
    const uint2 w = *reinterpret_cast<const uint2 *>(packed + (e >> 1));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t b = (i < 4 ? w.x : w.y) >> (8 * (i & 3));
      out[i] = cvt_pair<DT>(tab[b >> 4 & 15] * a, tab[b & 15] * a);
    }
    if (W) {
      uint4 *dst = reinterpret_cast<uint4 *>(W + (int64_t)v * ldw + c);
      dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
      dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
    }
  }
  if (!Wt) return;
  uint4 *t = reinterpret_cast<uint4 *>(&tile[row][col]);
  t[0] = make_uint4(out[0], out[1], out[2], out[3]);
  t[1] = make_uint4(out[4], out[5], out[6], out[7]);
  __syncthreads();
  const int lane = tid & 63, wave = tid >> 6;
  const int64_t oc = (int64_t)blockIdx.x * 64 + lane;
  if (c0 + oc >= K) return;
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    o[i] = tile[16 * wave + 2 * i][lane] | (uint32_t)tile[16 * wave + 2 * i + 1][lane] << 16;
  uint4 *dst = reinterpret_cast<uint4 *>(Wt + oc * ldt + blockIdx.y * 64 + 16 * wave);
  dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
  dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

hipError_t launch_decode_piece(const Weight4 &w, int dt, int64_t c0, int64_t cols, void *W, int64_t ldw, void *Wt,
                               int64_t ldt, hipStream_t st) {
  const int n = (int)w.N, np = (n + 63) & ~63;
  const dim3 grid((unsigned)((cols + 63) / 64), (unsigned)(np / 64));
#define QMV_D(DT, DQV)                                                                                              \
  hipLaunchKernelGGL((decode_piece_kernel<DT, DQV>), grid, dim3(256), 0, st, w.packed, w.sc, w.log2bs,              \
                     code_values(w.qt), w.K, c0, n, static_cast<uint16_t *>(W), ldw, static_cast<uint16_t *>(Wt), ldt)
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

}  // namespace qmv
