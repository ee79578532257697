// Low-rank adapters beside a 4-bit projection (include/qmv/tuning.h):
//   y[t] = W^ x[t] + bias + up[a] u[t],   u[t] = scale[a] down[a] x[t],   a = index[t]
// and the gradients of x, down and up.
//
// u and v = scale up^T dy are a handful of values a token, held in fp32.  For a
// few tokens their long sums are cut into pieces, one workgroup each, whose
// results the next kernel adds up in order.
#include "qmv_tuning.hpp"

namespace qmv {

// ---------------------------------------------------------------------------
// u[s][t][r] = scale[a] * sum over piece s of x[t][k] down[a][r][k]
//
// A workgroup of 4 waves takes one token and one piece; a wave goes through
// every fourth r, its lanes along k (16-byte loads).
// ---------------------------------------------------------------------------
template <int DT>
__global__ __launch_bounds__(256) void lora_down_kernel(const uint16_t *__restrict__ x, int64_t K, int piece,
                                                        const uint16_t *__restrict__ down,
                                                        const float *__restrict__ scale, int count, int R,
                                                        const int32_t *__restrict__ index, float *__restrict__ u,
                                                        int64_t T) {
  const int64_t t = blockIdx.x;
  const int a = index[t];
  if (a < 0 || a >= count) return;  // nothing reads this token's u
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t k0 = (int64_t)blockIdx.y * piece;
  const int64_t k1 = k0 + piece < K ? k0 + piece : K;
  const float s = scale[a];
  for (int r = wave; r < R; r += 4) {
    const uint16_t *row = down + ((int64_t)a * R + r) * K;
    float acc = 0.f;
    for (int64_t k = k0 + 8 * lane; k < k1; k += 512) {
      float xf[8], af[8];
      unpack8<DT>(*reinterpret_cast<const uint4 *>(x + t * K + k), xf);
      unpack8<DT>(*reinterpret_cast<const uint4 *>(row + k), af);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc = fmaf(xf[i], af[i], acc);
    }
    acc = wave_sum(acc);
    if (lane == 0) u[((int64_t)blockIdx.y * T + t) * R + r] = s * acc;
  }
}

// v[s][t][r] = scale[a] * sum over piece s of dy[t][n] up[a][n][r]: lanes take 8
// r's of one n, the rows of a workgroup are added up in LDS.
template <int DT>
__global__ __launch_bounds__(256) void lora_down_t_kernel(const uint16_t *__restrict__ dy, int64_t N, int piece,
                                                          const uint16_t *__restrict__ up,
                                                          const float *__restrict__ scale, int count, int R,
                                                          const int32_t *__restrict__ index, float *__restrict__ v,
                                                          int64_t T) {
  __shared__ float part[256][9];
  const int64_t t = blockIdx.x;
  const int a = index[t];
  if (a < 0 || a >= count) return;
  const int groups = R / 8, rows = 256 / groups;
  const int g = threadIdx.x % groups, row = threadIdx.x / groups;
  const int64_t n0 = (int64_t)blockIdx.y * piece;
  const int64_t n1 = n0 + piece < N ? n0 + piece : N;
  float acc[8] = {};
  if (row < rows)
    for (int64_t n = n0 + row; n < n1; n += rows) {
      const float d = bits16_to_f32<DT>(dy[t * N + n]);
      float b[8];
      unpack8<DT>(*reinterpret_cast<const uint4 *>(up + ((int64_t)a * N + n) * R + 8 * g), b);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = fmaf(d, b[i], acc[i]);
    }
#pragma unroll
  for (int i = 0; i < 8; ++i) part[threadIdx.x][i] = acc[i];
  __syncthreads();
  if ((int)threadIdx.x < R) {
    float sum = 0.f;
    for (int j = 0; j < rows; ++j) sum += part[j * groups + threadIdx.x / 8][threadIdx.x % 8];
    v[((int64_t)blockIdx.y * T + t) * R + threadIdx.x] = scale[a] * sum;
  }
}

// The pieces of u (v), added up in order, into LDS; returns whether the token
// has an adapter.  One barrier.
__device__ __forceinline__ bool gather_u(const float *__restrict__ u, int pieces, int64_t T, int64_t t, int R, int a,
                                         int count, float *dst) {
  const bool there = a >= 0 && a < count;
  if (there)
    for (int r = threadIdx.x; r < R; r += blockDim.x) {
      float sum = 0.f;
      for (int s = 0; s < pieces; ++s) sum += u[((int64_t)s * T + t) * R + r];
      dst[r] = sum;
    }
  __syncthreads();
  return there;
}

// out[t][n] = round(base[t][n] + bias[n] + sum_r up[a][n][r] u[t][r])
template <int DT, int ODT>
__global__ __launch_bounds__(256) void lora_up_kernel(const float *__restrict__ base, int64_t N,
                                                      const uint16_t *__restrict__ up, int count, int R,
                                                      const int32_t *__restrict__ index, const float *__restrict__ u,
                                                      int pieces, int64_t T, const uint16_t *__restrict__ bias,
                                                      typename Storage<ODT>::type *__restrict__ out) {
  __shared__ float us[128];
  const int64_t t = blockIdx.y;
  const int a = index[t];
  const bool there = gather_u(u, pieces, T, t, R, a, count, us);
  const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (n >= N) return;
  float acc = 0.f;
  if (there) {
    const uint16_t *row = up + ((int64_t)a * N + n) * R;
    for (int r = 0; r < R; r += 8) {
      float b[8];
      unpack8<DT>(*reinterpret_cast<const uint4 *>(row + r), b);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc = fmaf(us[r + i], b[i], acc);
    }
  }
  acc += base[t * N + n];
  if (bias) acc += bits16_to_f32<DT>(bias[n]);
  store_elem<ODT>(out, t * N + n, acc);
}

// out[t][k] = round(base[t][k] + sum_r down[a][r][k] v[t][r]): 8 columns a thread
template <int DT, int ODT>
__global__ __launch_bounds__(256) void lora_up_t_kernel(const float *__restrict__ base, int64_t K,
                                                        const uint16_t *__restrict__ down, int count, int R,
                                                        const int32_t *__restrict__ index,
                                                        const float *__restrict__ v, int pieces, int64_t T,
                                                        typename Storage<ODT>::type *__restrict__ out) {
  __shared__ float vs[128];
  const int64_t t = blockIdx.y;
  const int a = index[t];
  const bool there = gather_u(v, pieces, T, t, R, a, count, vs);
  const int64_t k = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (k >= K) return;
  float acc[8] = {};
  if (there)
    for (int r = 0; r < R; ++r) {
      float d[8];
      unpack8<DT>(*reinterpret_cast<const uint4 *>(down + ((int64_t)a * R + r) * K + k), d);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = fmaf(vs[r], d[i], acc[i]);
    }
#pragma unroll
  for (int i = 0; i < 8; ++i) store_elem<ODT>(out, t * K + k + i, acc[i] + base[t * K + k + i]);
}

// u[t][r] = the sum of its pieces, in order
__global__ void lora_sum_kernel(const float *__restrict__ parts, int pieces, int64_t n, float *__restrict__ u) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float sum = 0.f;
  for (int s = 0; s < pieces; ++s) sum += parts[s * n + i];
  u[i] = sum;
}

// sum over the tokens t of adapter a of g[t][w] h[t][r]: at [a][w][r] (UP) or [a][r][w]
template <int DT, int ODT, bool UP>
__global__ __launch_bounds__(64) void lora_grad_kernel(const uint16_t *__restrict__ g, int64_t W,
                                                       const float *__restrict__ h, int R,
                                                       const int32_t *__restrict__ index, int64_t T,
                                                       typename Storage<ODT>::type *__restrict__ out) {
  const int64_t w = (int64_t)blockIdx.x * 64 + threadIdx.x;
  const int r0 = 8 * blockIdx.y, a = blockIdx.z;
  float acc[8] = {};
  for (int64_t t = 0; t < T; ++t) {
    if (index[t] != a) continue;
    const float gv = w < W ? bits16_to_f32<DT>(g[t * W + w]) : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = fmaf(gv, h[t * R + r0 + i], acc[i]);
  }
  if (w >= W) return;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    store_elem<ODT>(out, UP ? ((int64_t)a * W + w) * R + r0 + i : ((int64_t)a * R + r0 + i) * W + w, acc[i]);
}

// ---------------------------------------------------------------------------
constexpr int64_t kRows = 4096;  // tokens whose projection is in the workspace at a time
constexpr int kPiece = 512;      // terms of a piece of u and v for few tokens

static int pieces_of(int64_t T, int64_t width) { return T <= 64 ? (int)((width + kPiece - 1) / kPiece) : 1; }

struct LoraPlan {
  size_t base, u, v, parts, back, total;
};

static LoraPlan lora_plan(int64_t T, int64_t N, int64_t K, int log2bs, int R, bool backward) {
  LoraPlan p{};
  Carver c;
  const int64_t rows = T < kRows ? T : kRows;
  p.base = c.take((size_t)rows * (backward ? K : N) * 4);
  p.u = c.take((size_t)T * R * 4 * pieces_of(T, K));
  if (backward) {
    p.v = c.take((size_t)T * R * 4 * pieces_of(T, N));
    p.parts = c.take((size_t)T * R * 4 * 2);
    const size_t a = gemm_backward_workspace_bytes(rows, N, K, log2bs);
    const size_t b = T > kRows && T % kRows ? gemm_backward_workspace_bytes(T % kRows, N, K, log2bs) : 0;
    p.back = c.take(a > b ? a : b);
  }
  p.total = c.at;
  return p;
}

size_t lora_workspace(int64_t T, int64_t N, int64_t K, int log2bs, int, int rank, bool backward) {
  return lora_plan(T, N, K, log2bs, rank, backward).total;
}

template <int DT>
static hipError_t lora_t(const uint16_t *x, int64_t T, const Weight4 &w, const Lora &l, const int32_t *index,
                         const uint16_t *bias, void *y, int y_dt, char *ws, hipStream_t st) {
  const LoraPlan p = lora_plan(T, w.N, w.K, w.log2bs, l.rank, false);
  float *base = reinterpret_cast<float *>(ws + p.base), *u = reinterpret_cast<float *>(ws + p.u);
  const int pieces = pieces_of(T, w.K), piece = pieces > 1 ? kPiece : (int)w.K;
  hipLaunchKernelGGL(lora_down_kernel<DT>, dim3((unsigned)T, (unsigned)pieces), dim3(256), 0, st, x, w.K, piece, l.down,
                     l.scale, l.count, l.rank, index, u, T);
  for (int64_t t = 0; t < T; t += kRows) {
    const int64_t m = T - t < kRows ? T - t : kRows;
    const hipError_t e = launch_gemm_4bit(x + t * w.K, DT, m, w.N, w.K, w.packed, w.sc, w.dq, w.log2bs, w.qt, base, kF32,
                                          nullptr, st);
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)((w.N + 255) / 256), (unsigned)m);
    if (y_dt == kF32)
      hipLaunchKernelGGL((lora_up_kernel<DT, kF32>), grid, dim3(256), 0, st, base, w.N, l.up, l.count, l.rank, index + t,
                         u + t * l.rank, pieces, T, bias, static_cast<float *>(y) + t * w.N);
    else
      hipLaunchKernelGGL((lora_up_kernel<DT, DT>), grid, dim3(256), 0, st, base, w.N, l.up, l.count, l.rank, index + t,
                         u + t * l.rank, pieces, T, bias, static_cast<uint16_t *>(y) + t * w.N);
  }
  return hipGetLastError();
}

template <int DT>
static hipError_t lora_backward_t(const uint16_t *dy, const uint16_t *x, int64_t T, const Weight4 &w, const Lora &l,
                                  const int32_t *index, uint16_t *dx, void *d_down, void *d_up, int grad_dt, char *ws,
                                  hipStream_t st) {
  const LoraPlan p = lora_plan(T, w.N, w.K, w.log2bs, l.rank, true);
  float *base = reinterpret_cast<float *>(ws + p.base);
  float *u = reinterpret_cast<float *>(ws + p.u), *v = reinterpret_cast<float *>(ws + p.v);
  const int R = l.rank, pu = pieces_of(T, w.K), pv = pieces_of(T, w.N);
  hipLaunchKernelGGL(lora_down_kernel<DT>, dim3((unsigned)T, (unsigned)pu), dim3(256), 0, st, x, w.K,
                     pu > 1 ? kPiece : (int)w.K, l.down, l.scale, l.count, R, index, u, T);
  hipLaunchKernelGGL(lora_down_t_kernel<DT>, dim3((unsigned)T, (unsigned)pv), dim3(256), 0, st, dy, w.N,
                     pv > 1 ? kPiece : (int)w.N, l.up, l.scale, l.count, R, index, v, T);
  for (int64_t t = 0; t < T; t += kRows) {
    const int64_t m = T - t < kRows ? T - t : kRows;
    const hipError_t e = launch_gemm_4bit_backward(dy + t * w.N, DT, m, w.N, w.K, w.packed, w.sc, w.dq, w.log2bs, w.qt,
                                                   base, kF32, ws + p.back, st);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((lora_up_t_kernel<DT, DT>), dim3((unsigned)((w.K + 2047) / 2048), (unsigned)m), dim3(256), 0, st,
                       base, w.K, l.down, l.count, R, index + t, v + t * R, pv, T, dx + t * w.K);
  }
  float *us = reinterpret_cast<float *>(ws + p.parts), *vs = us + T * R;
  const dim3 sum_grid((unsigned)((T * R + 255) / 256));
  hipLaunchKernelGGL(lora_sum_kernel, sum_grid, dim3(256), 0, st, u, pu, T * R, us);
  hipLaunchKernelGGL(lora_sum_kernel, sum_grid, dim3(256), 0, st, v, pv, T * R, vs);
  const dim3 gd((unsigned)((w.K + 63) / 64), (unsigned)(R / 8), (unsigned)l.count);
  const dim3 gu((unsigned)((w.N + 63) / 64), (unsigned)(R / 8), (unsigned)l.count);
  if (grad_dt == kF32) {
    hipLaunchKernelGGL((lora_grad_kernel<DT, kF32, false>), gd, dim3(64), 0, st, x, w.K, vs, R, index, T,
                       static_cast<float *>(d_down));
    hipLaunchKernelGGL((lora_grad_kernel<DT, kF32, true>), gu, dim3(64), 0, st, dy, w.N, us, R, index, T,
                       static_cast<float *>(d_up));
  } else {
    hipLaunchKernelGGL((lora_grad_kernel<DT, DT, false>), gd, dim3(64), 0, st, x, w.K, vs, R, index, T,
                       static_cast<uint16_t *>(d_down));
    hipLaunchKernelGGL((lora_grad_kernel<DT, DT, true>), gu, dim3(64), 0, st, dy, w.N, us, R, index, T,
                       static_cast<uint16_t *>(d_up));
  }
  return hipGetLastError();
}

hipError_t launch_lora(const void *x, int dt, int64_t T, const Weight4 &w, const Lora &l, const int32_t *index,
                       const void *bias, void *y, int y_dt, char *ws, hipStream_t st) {
  const uint16_t *xp = static_cast<const uint16_t *>(x), *b = static_cast<const uint16_t *>(bias);
  return dt == kF16 ? lora_t<kF16>(xp, T, w, l, index, b, y, y_dt, ws, st)
                    : lora_t<kBF16>(xp, T, w, l, index, b, y, y_dt, ws, st);
}

hipError_t launch_lora_backward(const void *dy, const void *x, int dt, int64_t T, const Weight4 &w, const Lora &l,
                                const int32_t *index, void *dx, void *d_down, void *d_up, int grad_dt, char *ws,
                                hipStream_t st) {
  const uint16_t *g = static_cast<const uint16_t *>(dy), *xp = static_cast<const uint16_t *>(x);
  uint16_t *o = static_cast<uint16_t *>(dx);
  return dt == kF16 ? lora_backward_t<kF16>(g, xp, T, w, l, index, o, d_down, d_up, grad_dt, ws, st)
                    : lora_backward_t<kBF16>(g, xp, T, w, l, index, o, d_down, d_up, grad_dt, ws, st);
}

}  // namespace qmv
