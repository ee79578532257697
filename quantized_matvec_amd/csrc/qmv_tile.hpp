// C[M, N] = A[M, L] B[N, L]^T for 16-bit operands whose rows run along the sum:
// the product behind the large calls of include/qmv/tuning.h, where a piece of
// a 4-bit weight is decoded once into a 16-bit workspace and then multiplied by
// many rows.
#pragma once

#include <type_traits>

#include "qmv_tuning.hpp"

namespace qmv {

typedef __attribute__((__vector_size__(8 * sizeof(__bf16)))) __bf16 frag_t;
typedef __attribute__((__vector_size__(8 * sizeof(_Float16)))) _Float16 frag_h_t;
typedef __attribute__((__vector_size__(16 * sizeof(float)))) float tile_acc_t;

template <int DT>
__device__ __forceinline__ tile_acc_t tile_mma(const frag_t &a, const frag_t &b, const tile_acc_t &c) {
  if constexpr (DT == kBF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(frag_h_t, a), __builtin_bit_cast(frag_h_t, b), c, 0, 0, 0);
}

constexpr int kTileM = 256, kTileN = 256, kTileL = 64;

struct TileArgs {
  const uint16_t *A, *B;
  int64_t lda, ldb;      // elements, multiples of 8; 256 rows of either are less than 2^31 bytes
  int M, N, L;           // L a multiple of 64
  const int32_t *rows;   // NULL, or [M]: row m of the product is row rows[m] of A (all of A: less than 2^31 bytes)
  const int32_t *count;  // NULL, or how many of the M rows there are (on the device)
  int split;             // terms of a workgroup along the grid's y, a multiple of 64 (L: all)
  int ncol, nrow;        // tiles
};
inline TileArgs tile_args(const uint16_t *A, int64_t lda, const uint16_t *B, int64_t ldb, int64_t M, int64_t N, int64_t L) {
  return TileArgs{A, B, lda, ldb, (int)M, (int)N, (int)L, nullptr, nullptr, (int)L,
                  (int)((N + kTileN - 1) / kTileN), (int)((M + kTileM - 1) / kTileM)};
}

// Tile of workgroup id.  Workgroups go to the 8 XCDs in turn, and an XCD's
// 32 compute units work on neighbouring ids / 8 at a time: each XCD takes one
// run of the tiles, in strips of 4 row tiles, so that the tiles it has in work
// share their rows and columns in its L2.
__host__ __device__ inline void tile_of(int id, int ncol, int nrow, int &rb, int &cb) {
  const int n = ncol * nrow, xcd = id & 7, each = n >> 3, more = n & 7;
  const int at = xcd * each + (xcd < more ? xcd : more) + (id >> 3);
  const int strip = at / (4 * ncol), rows = nrow - 4 * strip < 4 ? nrow - 4 * strip : 4;
  const int in = at - strip * 4 * ncol;
  rb = 4 * strip + in % rows;
  cb = in / rows;
}

// Four waves of 128 x 128, one a SIMD with all of its registers: 64 products of 32 x 32 x 16 for
// 32 LDS reads of 16 bytes and 16 loads a stage, so the matrix cores bound it.  Half-size stages would load
// half lines; 64 terms a row are whole ones.  All of the next stage's first operands are read
// behind the last quarter of this one's products, and what is loaded has two stages to land.  Measured
// (bf16, fp32 / bf16 outputs, TFLOP/s): 4096 x 4096 of 8192 terms 1382 / 1417, 4096 x 14336 of 4096 1149 / 1297,
// 8192 x 8192 of 8192 1371 / 1429; no LDS bank conflicts.  Short sums pay for filling the ring and for the stores:
// 4096 x 4096 of 1088 920 / 1022.
template <int DT, class Epi>
__global__ __launch_bounds__(256, 1) void tile_kernel(TileArgs g, Epi epi) {
  // a ring of units, 64 terms of 256 rows: A and B of the stage in use, A and B of
  // the next, A of the one after; one array each, so that the compiler can tell
  // a load into one from reads of another
  __shared__ uint4 u0[2048], u1[2048], u2[2048], u3[2048], u4[2048];
  typedef __attribute__((address_space(3))) void lds_t;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // the tiles that there are take the first workgroups, so that each XCD has its share of them
  const int M = g.count ? min(g.M, *g.count) : g.M, nrow = (M + kTileM - 1) / kTileM;
  if ((int)blockIdx.x >= nrow * g.ncol) return;
  int rb, cb;
  tile_of((int)blockIdx.x, g.ncol, nrow, rb, cb);
  const int m0 = rb * kTileM, n0 = cb * kTileN;
  const int l0 = (int)blockIdx.y * g.split;
  const int KT = (g.L - l0 < g.split ? g.L - l0 : g.split) / kTileL;  // none: zeros
  // loads: wave w moves rows 64 w .. + 63 of A and of B, 8 rows an instruction;
  // lane l brings chunk (l % 8) ^ (row / 2 % 8) of row l / 8 to place l % 8 of it:
  // then 16 rows of a fragment read at one chunk lie in 16 different bank groups
  const int mrows = M - m0 < kTileM ? M - m0 : kTileM, ncols = g.N - n0 < kTileN ? g.N - n0 : kTileN;
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(g.rows ? g.A : g.A + m0 * g.lda, 0x7fffffffu);
  const __amdgpu_buffer_rsrc_t rbs = make_rsrc(g.B + n0 * g.ldb, 0x7fffffffu);
  uint32_t aoff[8], boff[8];
#pragma unroll
  for (int d = 0; d < 8; ++d) {
    const int r = 64 * wave + 8 * d + (lane >> 3);
    const uint32_t c = 16u * ((lane & 7) ^ ((r >> 1) & 7));
    const int ar = !g.rows ? r : r < mrows ? g.rows[m0 + r] : 0;
    aoff[d] = r < mrows ? (uint32_t)(ar * g.lda * 2) + c : 0x80000000u;  // past the end: zeros
    boff[d] = r < ncols ? (uint32_t)(r * g.ldb * 2) + c : 0x80000000u;
  }
  auto issue = [&](const __amdgpu_buffer_rsrc_t &rs, const uint32_t (&off)[8], int kt, uint4 *st) __attribute__((always_inline)) {
    const int so = (l0 + (kt < KT ? kt : KT - 1) * kTileL) * 2;  // past the end: the last stage again
#pragma unroll
    for (int d = 0; d < 8; ++d)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_t *)(st + (8 * wave + d) * 64), 16, off[d], so, 0, 0);
  };
  // wave (wm, wn) has rows 128 wm .. + 127 and columns 128 wn .. + 127 of the tile, in 32 x 32
  // accumulators: column lane % 32, rows 8 (r / 4) + 4 (lane / 32) + r % 4
  const int wm = wave >> 1, wn = wave & 1, h = lane >> 5, l32 = lane & 31;
  const int mw = m0 + 128 * wm + 4 * h, nw = n0 + 128 * wn + l32;
  tile_acc_t acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  struct Frags {
    frag_t a[4], b[4];
  };
  const int arow = 128 * wm + l32, brow = 128 * wn + l32;
  const int swz = (l32 >> 1) & 7;
  // in the order in which the products want them
  auto read = [&](const uint4 *a, const uint4 *b, int s, Frags &f) __attribute__((always_inline)) {
    const int c = (2 * s + h) ^ swz;
    f.a[0] = __builtin_bit_cast(frag_t, a[arow * 8 + c]);
#pragma unroll
    for (int j = 0; j < 4; ++j) f.b[j] = __builtin_bit_cast(frag_t, b[(brow + 32 * j) * 8 + c]);
#pragma unroll
    for (int i = 1; i < 4; ++i) f.a[i] = __builtin_bit_cast(frag_t, a[(arow + 32 * i) * 8 + c]);
  };
  auto mma = [&](const Frags &f) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = tile_mma<DT>(f.a[i], f.b[j], acc[i][j]);
  };
  Frags f0, f1;
  auto weave = [&](auto loads) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if constexpr (decltype(loads)::value) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  // stage kt in (a, b), the next in (na, nb), the next A after that in c
  auto step = [&](int kt, uint4 *a, uint4 *b, uint4 *na, uint4 *nb, uint4 *c) __attribute__((always_inline)) {
    __builtin_amdgcn_sched_barrier(0);
    read(a, b, 1, f1);
    issue(ra, aoff, kt + 2, c);
    mma(f0);
    weave(std::true_type{});
    read(a, b, 2, f0);
    mma(f1);
    weave(std::false_type{});
    read(a, b, 3, f1);
    mma(f0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, 8, 0);
    __builtin_amdgcn_sched_barrier(0);
    // all of stage kt is in registers, and stage kt + 1 has landed: open may be A of kt + 2
    __builtin_amdgcn_s_waitcnt((8 & 15) | (7 << 4) | (0 << 8) | ((8 >> 4) << 14));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read(na, nb, 0, f0);
    issue(rbs, boff, kt + 2, a);
    mma(f1);
    weave(std::true_type{});
  };
  if (KT > 0) {
    issue(ra, aoff, 0, u0), issue(rbs, boff, 0, u1);
    issue(ra, aoff, 1, u2), issue(rbs, boff, 1, u3);
    __builtin_amdgcn_s_waitcnt((16 & 15) | (7 << 4) | (15 << 8) | ((16 >> 4) << 14));  // stage 0 has landed
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read(u0, u1, 0, f0);
    int kt = 0;
    for (; kt + 5 <= KT; kt += 5) {
      step(kt, u0, u1, u2, u3, u4);
      step(kt + 1, u2, u3, u4, u0, u1);
      step(kt + 2, u4, u0, u1, u2, u3);
      step(kt + 3, u1, u2, u3, u4, u0);
      step(kt + 4, u3, u4, u0, u1, u2);
    }
    if (kt < KT) step(kt, u0, u1, u2, u3, u4);
    if (kt + 1 < KT) step(kt + 1, u2, u3, u4, u0, u1);
    if (kt + 2 < KT) step(kt + 2, u4, u0, u1, u2, u3);
    if (kt + 3 < KT) step(kt + 3, u1, u2, u3, u4, u0);
    __builtin_amdgcn_s_waitcnt((7 << 4) | (15 << 8));  // no load into LDS outlives the kernel
  }
  const int mfirst = m0 + 128 * wm, mpast = mfirst + 128 < M ? mfirst + 128 : M;  // of this wave
  const bool more = epi.begin(acc, g.N, mfirst, mpast, n0 + 128 * wn, lane);
  if constexpr (Epi::kPlain) {
    // C = sums, or C f[row] + sums, in parts of 32 x 128: bounded resources (what is not there, or
    // no rows yet, reads as 0 and is not written), so no branches, and the loads of a part are in
    // flight together; no part's loads before the last part's stores, which would not fit the registers
    const __amdgpu_buffer_rsrc_t ro = make_rsrc(epi.row(m0) + n0, 0x7fffffffu);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __builtin_amdgcn_sched_barrier(0);
      auto place = [&](int r, int j) __attribute__((always_inline)) {
        const int m = mw - m0 + 32 * i + 8 * (r >> 2) + (r & 3), n = nw - n0 + 32 * j;
        return m < mrows && n < ncols ? (uint32_t)((m * (int)epi.ld + n) * 4) : 0x80000000u;
      };
      if constexpr (Epi::kAdds) {
        const __amdgpu_buffer_rsrc_t rc = make_rsrc(epi.row(m0) + n0, epi.first ? 0 : 0x7fffffffu);
        const __amdgpu_buffer_rsrc_t rf = make_rsrc(epi.f + m0, epi.first ? 0 : (uint32_t)mrows * 4);
        float f[16], old[16][4];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          f[r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rf, (uint32_t)(mw - m0 + 32 * i + 8 * (r >> 2) + (r & 3)) * 4, 0, 0));
#pragma unroll
          for (int j = 0; j < 4; ++j) old[r][j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rc, place(r, j), 0, 0));
        }
#pragma unroll
        for (int r = 0; r < 16; ++r)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(fmaf(old[r][j], f[r], acc[i][j][r])), ro, place(r, j), 0, 0);
      } else {
#pragma unroll
        for (int r = 0; r < 16; ++r)
#pragma unroll
          for (int j = 0; j < 4; ++j) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(acc[i][j][r]), ro, place(r, j), 0, 0);
      }
    }
    return;
  }
  auto store = [&](auto whole) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int m = mw + 32 * i + 8 * (r >> 2) + (r & 3);
        if (!decltype(whole)::value && m >= M) continue;
        const auto row = epi.row(m);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (decltype(whole)::value || nw + 32 * j < g.N) epi.store(row, nw + 32 * j, acc[i][j][r]);
      }
  };
  if (mrows == kTileM && ncols == kTileN) store(std::true_type{});
  else store(std::false_type{});
  if (more) epi.end(g.N, mfirst, mpast, n0 + 128 * wn, lane);
}

// What becomes of the sums: begin() may add to them, row() gives what store() needs of a row, and end() follows
// the stores where begin() asks for it.  Both get the tile product's columns, the wave's rows and its first column.
struct EpilogueBase {
  static constexpr bool kPlain = false;  // into C in fp32 as they are, of rows C, ld apart (256 of them: below 2^31 bytes)
  static constexpr bool kAdds = false;   // plain, C f + sums, but for `first`
  __device__ __forceinline__ bool begin(tile_acc_t (&)[4][4], int, int, int, int, int) const { return false; }
  __device__ __forceinline__ void end(int, int, int, int, int) const {}
};
struct EpilogueF32 : EpilogueBase {
  static constexpr bool kPlain = true;
  float *C;
  int64_t ld, part = 0;  // the sums' parts along the grid's y
  __device__ __forceinline__ float *row(int m) const { return C + blockIdx.y * part + m * ld; }
  __device__ __forceinline__ void store(float *, int, float) const {}
};

}  // namespace qmv
