// Losses over a 4-bit vocabulary projection (include/qmv/tuning.h): softmax
// cross entropy, and the divergence from a teacher's largest logits.
//
// With l = W^ x / tau and a target distribution p on a few ids,
//   loss = sum_j p_j (log p_j - l_j) + log sum_v exp l_v
//   dx   = dloss / tau (sum_v q_v W^_v - sum_j p_j W^_j),   q = softmax(l).
// The vocabulary is taken in pieces.  A piece's logits are a product, kept in
// fp32; over the pieces run the maximum m and the sum s of exp(l - m), and,
// with a gradient, D = sum_v exp(l_v - m) W^_v, which is multiplied by
// exp(m_old - m_new) before a piece is added (one pass: the logits are computed
// once).  The target ids stay out of m, s and D: their logits are kept, and
// at the end q_j - p_j times their rows is added in fp32.  So the gradient of a
// token whose target is all but certain keeps its precision (1 - q is
// computed from s, not by subtracting), and a type with few exponent bits
// does not flush the rest of the vocabulary against the target's logit.
#include "qmv_tuning.hpp"

namespace qmv {

constexpr int kPieceV = 8192;    // columns of a piece: a multiple of 4096 (rows_of)
constexpr int64_t kTokens = 4096;  // tokens taken at a time
constexpr int kTail = 32;

// What exp(l - m) is multiplied by before its rounding.  fp16 has no normal
// numbers below 2^-14: with 2^14 (sums are fp32, and D is divided by it at the
// end) terms keep their 11 bits down to 2^-28 of the largest.
template <int DT>
constexpr float kGain = DT == kF16 ? 16384.f : 1.f;

struct RowState {
  float *m, *s, *f;  // running maximum, sum, and the factor of what D held before this piece
  float *lt;         // [T, k] logits of the target ids
  float *tail;       // [T, 32] logits of the last V % 32 columns (-inf: none, or a target)
};

template <class F>
__device__ __forceinline__ float block_reduce(float v, float *buf, F op) {  // 256 threads
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) buf[wave] = v;
  __syncthreads();
  v = op(op(buf[0], buf[1]), op(buf[2], buf[3]));
  __syncthreads();
  return v;
}

// One piece's columns [v0, v0 + n) of one token: m, s, f, the target ids'
// logits and, with a gradient, P = exp(l - m) in 16 bits, [T, np] with np the
// multiple of 32 below n (the columns from np on go to `tail`).
template <int DT, bool GRAD>
__global__ __launch_bounds__(256) void loss_piece_kernel(const float *__restrict__ logits, int64_t ld, int64_t v0, int n,
                                                         int np, const int64_t *__restrict__ ids, int k, float inv_tau,
                                                         bool first, RowState rs, uint16_t *__restrict__ P) {
  __shared__ uint32_t out[kPieceV / 32];  // columns of target ids
  __shared__ float buf[4];
  const int64_t t = blockIdx.x;
  const float *row = logits + t * ld;
  for (int i = threadIdx.x; i < kPieceV / 32; i += 256) out[i] = 0;
  __syncthreads();
  for (int j = threadIdx.x; j < k; j += 256) {
    const int64_t c = ids[t * k + j] - v0;
    if (c >= 0 && c < n) {
      atomicOr(&out[c >> 5], 1u << (c & 31));
      rs.lt[t * k + j] = row[c] * inv_tau;
    }
  }
  __syncthreads();
  auto held = [&](int c) { return (out[c >> 5] >> (c & 31) & 1) == 0; };
  float m = -INFINITY;
  for (int c = threadIdx.x; c < n; c += 256)
    if (held(c)) m = fmaxf(m, row[c] * inv_tau);
  m = block_reduce(wave_max(m), buf, [](float a, float b) { return fmaxf(a, b); });
  const float m_old = first ? -INFINITY : rs.m[t];
  m = fmaxf(m, m_old);
  float s = 0.f;
  for (int c = threadIdx.x; c < n; c += 256) {
    const float l = row[c] * inv_tau;
    const float e = held(c) ? expf(l - m) : 0.f;
    s += e;
    if constexpr (GRAD) {
      if (c < np) P[t * np + c] = (uint16_t)f32_to_bits16<DT>(e * kGain<DT>);
      else rs.tail[t * kTail + c - np] = held(c) ? l : -INFINITY;
    }
  }
  s = block_reduce(wave_sum(s), buf, [](float a, float b) { return a + b; });
  if (threadIdx.x == 0) {
    const float f = m_old == -INFINITY ? 0.f : expf(m_old - m);
    rs.s[t] = (first ? 0.f : rs.s[t] * f) + s;
    rs.m[t] = m;
    rs.f[t] = f;
  }
}

// D = D f + what a piece adds (f of the row; the first piece stores)
__global__ __launch_bounds__(256) void loss_add_kernel(float *__restrict__ D, const float *__restrict__ add,
                                                       const float *__restrict__ f, int64_t K, bool first) {
  const int64_t t = blockIdx.x;
  const float ft = f[t];
  for (int64_t c = threadIdx.x; c < K; c += 256) {
    const int64_t i = t * K + c;
    D[i] = (first ? 0.f : D[i] * ft) + (add ? add[i] : 0.f);
  }
}

// The loss of a token, and its row of dx from D.
template <int DT, int LDT, bool DQ>
__global__ __launch_bounds__(256) void loss_finish_kernel(const int64_t *__restrict__ ids, const void *teacher,
                                                          int teacher_dt, int k, float inv_tau, int64_t V, RowState rs,
                                                          int tail_n, const float *__restrict__ D, int64_t K,
                                                          const uint8_t *__restrict__ packed, Scales sc, int log2bs,
                                                          CodeValues table, const float *__restrict__ dloss,
                                                          typename Storage<LDT>::type *__restrict__ loss,
                                                          uint16_t *__restrict__ dx) {
  __shared__ float z[128], p[128], lt[128], coef[128 + kTail], tab[16], buf[4];
  __shared__ int64_t id[128 + kTail];
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x;
  if (tid < 16) tab[tid] = table.v[tid];
  // the target distribution; an entry that repeats an earlier id lends that
  // one its p, and is no entry of its own for q
  bool there = false, own = false;
  if (tid < k) {
    const int64_t v = ids[t * k + tid];
    there = v >= 0 && v < V;
    id[tid] = there ? v : -1;
    lt[tid] = there ? rs.lt[t * k + tid] : -INFINITY;
    z[tid] = !there ? -INFINITY
             : !teacher ? 0.f
             : teacher_dt == kF32 ? static_cast<const float *>(teacher)[t * k + tid] * inv_tau
             : teacher_dt == kF16 ? bits16_to_f32<kF16>(static_cast<const uint16_t *>(teacher)[t * k + tid]) * inv_tau
                                  : bits16_to_f32<kBF16>(static_cast<const uint16_t *>(teacher)[t * k + tid]) * inv_tau;
  }
  __syncthreads();
  float zm = -INFINITY, zs = 0.f;
  for (int j = 0; j < k; ++j) zm = fmaxf(zm, z[j]);
  const bool live = zm > -INFINITY;  // with a NaN in z: not so, or p is NaN
  if (!live && !(zm != zm)) {
    bool nan = false;
    for (int j = 0; j < k; ++j) nan |= z[j] != z[j];
    if (!nan) {
      if (tid == 0) store_elem<LDT>(loss, t, 0.f);
      if (dx)
        for (int64_t c = tid; c < K; c += 256) dx[t * K + c] = 0;
      return;
    }
  }
  for (int j = 0; j < k; ++j) zs += expf(z[j] - zm);
  if (tid < k) {
    p[tid] = expf(z[tid] - zm) / zs;
    own = there;
    for (int j = 0; j < tid; ++j) own = own && id[j] != id[tid];
  }
  __syncthreads();
  // the loss
  float M = rs.m[t];
  for (int j = 0; j < k; ++j) M = fmaxf(M, lt[j]);
  const float rest = rs.s[t] * (rs.m[t] == -INFINITY ? 0.f : expf(rs.m[t] - M));
  const float mine = own ? expf(lt[tid] - M) : 0.f;
  const float targets = block_reduce(wave_sum(mine), buf, [](float a, float b) { return a + b; });
  const float Z = rest + targets;
  if (!teacher) {
    // (M - l) + log Z; where the target is the largest that is log(1 + rest)
    if (tid == 0) store_elem<LDT>(loss, t, lt[0] == M ? log1pf(rest) : (M - lt[0]) + logf(Z));
  } else {
    float part = 0.f;
    if (tid < k && p[tid] != 0.f) part = p[tid] * ((z[tid] - zm - logf(zs)) - (lt[tid] - M) + logf(Z));
    part = block_reduce(wave_sum(part), buf, [](float a, float b) { return a + b; });
    if (tid == 0) store_elem<LDT>(loss, t, part);
  }
  if (!dx) return;
  // q - p of every id; by the complements where both are near 1
  if (tid < k) {
    float c = 0.f;
    if (own) {
      float pj = 0.f, others_p = 0.f, others_q = rest;
      for (int j = 0; j < k; ++j) {
        if (id[j] == id[tid]) {
          pj += p[j];
        } else {
          others_p += p[j];
          bool seen = id[j] < 0;
          for (int i = 0; i < j; ++i) seen = seen || id[i] == id[j];
          if (!seen) others_q += expf(lt[j] - M);
        }
      }
      const float q = mine / Z;
      c = pj > 0.5f ? others_p - others_q / Z : q - pj;
    }
    coef[tid] = c;
  }
  if (tid >= 128 && tid < 128 + kTail) {
    const int j = tid - 128;
    const float l = j < tail_n ? rs.tail[t * kTail + j] : -INFINITY;
    coef[k + j] = l == -INFINITY ? 0.f : expf(l - M) / Z;
    id[k + j] = V - tail_n + j;
  }
  __syncthreads();
  const float gain = dloss[t] * inv_tau;
  const float scale = rs.m[t] == -INFINITY ? 0.f : expf(rs.m[t] - M) / Z / kGain<DT>;
  const float offset = DQ ? sc.offset[0] : 0.f;
  for (int64_t c = tid * 8; c < K; c += 2048) {
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = D[t * K + c + i] * scale;
    for (int j = 0; j < k + tail_n; ++j) {
      const float cj = coef[j];
      if (cj == 0.f) continue;
      const int64_t e = id[j] * K + c;
      const float a = cj * block_scale<DQ>(sc, e >> log2bs, offset);
      const uint32_t w = *reinterpret_cast<const uint32_t *>(packed + e / 2);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[2 * i] = fmaf(a, tab[w >> (8 * i + 4) & 15], acc[2 * i]);
        acc[2 * i + 1] = fmaf(a, tab[w >> (8 * i) & 15], acc[2 * i + 1]);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) store_elem<DT>(dx, t * K + c + i, acc[i] * gain);
  }
}

// ---------------------------------------------------------------------------
struct LossPlan {
  int64_t tokens;
  int piece;
  size_t logits, m, s, f, lt, tail, P, D, add, back, total;
};

static LossPlan loss_plan(int64_t T, int64_t V, int64_t K, int log2bs, int k, bool grad) {
  LossPlan p{};
  Carver c;
  p.tokens = T < kTokens ? T : kTokens;
  p.piece = (int)(V < kPieceV ? V : kPieceV);
  const size_t n = (size_t)p.tokens;
  p.logits = c.take(n * p.piece * 4);
  p.m = c.take(n * 4), p.s = c.take(n * 4), p.f = c.take(n * 4), p.lt = c.take(n * k * 4);
  if (grad) {
    p.tail = c.take(n * kTail * 4);
    p.P = c.take(n * p.piece * 2);
    p.D = c.take(n * K * 4);
    p.add = c.take(n * K * 4);
    size_t most = 0;  // the product's own workspace, over all sizes that come up
    for (int64_t m : {p.tokens, T % p.tokens})
      for (int64_t v : {(int64_t)p.piece & ~31ll, (V % p.piece) & ~31ll})
        if (m > 0 && v > 0) {
          const size_t b = gemm_backward_workspace_bytes(m, v, K, log2bs);
          most = b > most ? b : most;
        }
    p.back = c.take(most);
  }
  p.total = c.at;
  return p;
}

size_t loss_workspace(int64_t T, int64_t V, int64_t K, int log2bs, int k, bool grad) {
  return loss_plan(T, V, K, log2bs, k, grad).total;
}

template <int DT>
static hipError_t loss_t(const uint16_t *x, int64_t T, const Weight4 &w, const Targets &tg, const float *dloss,
                         void *loss, int loss_dt, uint16_t *dx, char *ws, hipStream_t st) {
  const LossPlan p = loss_plan(T, w.N, w.K, w.log2bs, tg.k, dx != nullptr);
  float *logits = reinterpret_cast<float *>(ws + p.logits);
  uint16_t *P = reinterpret_cast<uint16_t *>(ws + p.P);
  float *D = reinterpret_cast<float *>(ws + p.D), *add = reinterpret_cast<float *>(ws + p.add);
  const RowState rs{reinterpret_cast<float *>(ws + p.m), reinterpret_cast<float *>(ws + p.s),
                    reinterpret_cast<float *>(ws + p.f), reinterpret_cast<float *>(ws + p.lt),
                    reinterpret_cast<float *>(ws + p.tail)};
  const size_t tsize = tg.teacher_dt == kF32 ? 4 : 2, lsize = loss_dt == kF32 ? 4 : 2;
  for (int64_t t = 0; t < T; t += p.tokens) {
    const int64_t m = T - t < p.tokens ? T - t : p.tokens;
    const int64_t *ids = tg.ids + t * tg.k;
    int tail_n = 0;
    for (int64_t v = 0; v < w.N; v += p.piece) {
      const int n = (int)(w.N - v < p.piece ? w.N - v : p.piece), np = n & ~31;
      const Weight4 c = rows_of(w, v, n);
      hipError_t e = launch_gemm_4bit(x + t * w.K, DT, m, n, w.K, c.packed, c.sc, c.dq, c.log2bs, c.qt, logits, kF32,
                                      nullptr, st);
      if (e != hipSuccess) return e;
      if (!dx) {
        hipLaunchKernelGGL((loss_piece_kernel<DT, false>), dim3((unsigned)m), dim3(256), 0, st, logits, (int64_t)n, v, n, n,
                           ids, tg.k, tg.inv_tau, v == 0, rs, P);
        continue;
      }
      hipLaunchKernelGGL((loss_piece_kernel<DT, true>), dim3((unsigned)m), dim3(256), 0, st, logits, (int64_t)n, v, n, np,
                         ids, tg.k, tg.inv_tau, v == 0, rs, P);
      if (np) {
        e = launch_gemm_4bit_backward(P, DT, m, np, w.K, c.packed, c.sc, c.dq, c.log2bs, c.qt, add, kF32, ws + p.back, st);
        if (e != hipSuccess) return e;
      }
      hipLaunchKernelGGL(loss_add_kernel, dim3((unsigned)m), dim3(256), 0, st, D, np ? add : nullptr, rs.f, w.K, v == 0);
      tail_n = n - np;
    }
    const void *teacher = tg.teacher ? static_cast<const char *>(tg.teacher) + t * tg.k * tsize : nullptr;
    char *lp = static_cast<char *>(loss) + t * lsize;
#define QMV_L(LDT, DQV)                                                                                              \
  hipLaunchKernelGGL((loss_finish_kernel<DT, LDT, DQV>), dim3((unsigned)m), dim3(256), 0, st, ids, teacher,          \
                     tg.teacher_dt, tg.k, tg.inv_tau, w.N, rs, tail_n, D, w.K, w.packed, w.sc, w.log2bs,             \
                     code_values(w.qt), dloss ? dloss + t : nullptr, reinterpret_cast<typename Storage<LDT>::type *>(lp), \
                     dx ? dx + t * w.K : nullptr)
    if (loss_dt == kF32) {
      if (w.dq) QMV_L(kF32, true);
      else QMV_L(kF32, false);
    } else {
      if (w.dq) QMV_L(DT, true);
      else QMV_L(DT, false);
    }
#undef QMV_L
  }
  return hipGetLastError();
}

hipError_t launch_loss(const void *x, int dt, int64_t T, const Weight4 &w, const Targets &tg, const float *dloss,
                       void *loss, int loss_dt, void *dx, char *ws, hipStream_t st) {
  const uint16_t *xp = static_cast<const uint16_t *>(x);
  uint16_t *d = static_cast<uint16_t *>(dx);
  return dt == kF16 ? loss_t<kF16>(xp, T, w, tg, dloss, loss, loss_dt, d, ws, st)
                    : loss_t<kBF16>(xp, T, w, tg, dloss, loss, loss_dt, d, ws, st);
}

}  // namespace qmv
