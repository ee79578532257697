// The C ABI of include/qmv/tuning.h: argument validation on the host, then
// launches on the caller's stream.
#include <math.h>

#include "qmv/tuning.h"
#include "qmv_tuning.hpp"

using namespace qmv;

namespace {

constexpr int64_t kMost = (int64_t)1 << 31;

bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool valid_dtype(int d) { return d == QMV_F32 || d == QMV_F16 || d == QMV_BF16; }
bool is_pow2(int64_t v) { return v > 0 && (v & (v - 1)) == 0; }
bool valid_blocksize(int64_t bs) { return is_pow2(bs) && bs >= 32 && bs <= 4096; }
int launch_status(hipError_t e) { return e == hipSuccess ? QMV_OK : QMV_ERR_LAUNCH; }

int check_sizes(int64_t T, int64_t N, int64_t K, int32_t blocksize) {
  if (T <= 0 || N <= 0 || K <= 0) return QMV_ERR_INVALID_ARG;
  if (!valid_blocksize(blocksize) || K % 32 || K % blocksize) return QMV_ERR_UNSUPPORTED;
  // tokens are counted, and a row tile's and a weight tile's offsets held, in 32 bits
  if (T >= kMost / 2 || N >= kMost || K >= (1 << 22)) return QMV_ERR_UNSUPPORTED;
  return QMV_OK;
}

int check_weight(const qmv_weight_4bit *w, int64_t T, Weight4 *out) {
  if (!w || (w->quant_type != QMV_NF4 && w->quant_type != QMV_FP4)) return QMV_ERR_INVALID_ARG;
  const int rc = check_sizes(T, w->rows, w->cols, w->blocksize);
  if (rc != QMV_OK) return rc;
  const qmv_absmax &s = w->scales;
  const bool plain = s.absmax != nullptr;
  const bool any = s.absmax_q || s.absmax2 || s.code2 || s.offset, all = s.absmax_q && s.absmax2 && s.code2 && s.offset;
  if (!w->packed || plain == any || (!plain && !all)) return QMV_ERR_INVALID_ARG;
  if (!plain && !valid_blocksize(s.blocksize2)) return QMV_ERR_UNSUPPORTED;
  if (!aligned(w->packed, 16) || !aligned(s.absmax, 16) || !aligned(s.absmax_q, 16) || !aligned(s.absmax2, 16) ||
      !aligned(s.code2, 16) || !aligned(s.offset, 16))
    return QMV_ERR_ALIGNMENT;
  Scales sc{};
  sc.absmax = s.absmax;
  if (!plain) sc = Scales{nullptr, s.absmax_q, s.absmax2, s.code2, s.offset, log2_exact(s.blocksize2)};
  *out = Weight4{w->packed, sc, !plain, w->rows, w->cols, log2_exact(w->blocksize), w->quant_type};
  return QMV_OK;
}

int check_rank(int32_t count, int32_t rank) {
  if (count <= 0 || rank <= 0) return QMV_ERR_INVALID_ARG;
  return count > 4096 || rank % 8 || rank > 128 ? QMV_ERR_UNSUPPORTED : QMV_OK;
}

// the adapters' kernels have a grid dimension along the outputs
bool wide(int64_t N) { return N >= (1 << 22); }
// the backward puts all tokens in order at once, and each 256 of them count all
bool many(int64_t T) { return T >= (1 << 22); }

int check_lora(const qmv_lora *l, Lora *out) {
  if (!l || !l->down || !l->up || !l->scale) return QMV_ERR_INVALID_ARG;
  const int rc = check_rank(l->count, l->rank);
  if (rc != QMV_OK) return rc;
  if (!aligned(l->down, 16) || !aligned(l->up, 16) || !aligned(l->scale, 4)) return QMV_ERR_ALIGNMENT;
  *out = Lora{static_cast<const uint16_t *>(l->down), static_cast<const uint16_t *>(l->up), l->scale, l->count, l->rank};
  return QMV_OK;
}

// 16-bit activations, and an output of their type or fp32
int check_types(int dtype, int out_dtype) {
  if (!valid_dtype(dtype) || !valid_dtype(out_dtype)) return QMV_ERR_INVALID_ARG;
  return dtype == QMV_F32 || (out_dtype != dtype && out_dtype != QMV_F32) ? QMV_ERR_UNSUPPORTED : QMV_OK;
}

int check_workspace(const void *ws, size_t bytes, size_t need) {
  return need > 0 && (!ws || bytes < need || !aligned(ws, 16)) ? QMV_ERR_WORKSPACE : QMV_OK;
}

int loss(const void *x, int dtype, int64_t T, const qmv_weight_4bit *w, const Targets &tg, const float *dloss,
         void *out, int out_dtype, void *dx, void *ws, size_t bytes, void *stream) {
  if (!x || !tg.ids || !out || (dloss == nullptr) != (dx == nullptr)) return QMV_ERR_INVALID_ARG;
  int rc = check_types(dtype, out_dtype);
  if (rc != QMV_OK) return rc;
  Weight4 wt;
  rc = check_weight(w, T, &wt);
  if (rc != QMV_OK) return rc;
  if (!aligned(x, 16) || !aligned(dx, 16) || !aligned(tg.ids, 8) || !aligned(dloss, 4) ||
      !aligned(out, out_dtype == QMV_F32 ? 4 : 2) || !aligned(tg.teacher, tg.teacher_dt == QMV_F32 ? 4 : 2))
    return QMV_ERR_ALIGNMENT;
  rc = check_workspace(ws, bytes, loss_workspace(T, wt.N, wt.K, wt.log2bs, tg.k, dx != nullptr));
  if (rc != QMV_OK) return rc;
  return launch_status(launch_loss(x, dtype, T, wt, tg, dloss, out, out_dtype, dx, static_cast<char *>(ws),
                                   (hipStream_t)stream));
}

}  // namespace

extern "C" {

size_t qmv_lora_4bit_workspace(int64_t T, int64_t N, int64_t K, int32_t blocksize, int32_t count, int32_t rank) {
  if (check_sizes(T, N, K, blocksize) != QMV_OK || check_rank(count, rank) != QMV_OK || wide(N)) return 0;
  return lora_workspace(T, N, K, log2_exact(blocksize), count, rank, false);
}

int qmv_lora_4bit(const void *x, qmv_dtype dtype, int64_t T, const qmv_weight_4bit *w, const qmv_lora *lora,
                  const int32_t *index, const void *bias, void *y, qmv_dtype y_dtype, void *workspace,
                  size_t workspace_bytes, void *stream) {
  if (!x || !y || !index) return QMV_ERR_INVALID_ARG;
  int rc = check_types(dtype, y_dtype);
  if (rc != QMV_OK) return rc;
  Weight4 wt;
  Lora l;
  if ((rc = check_weight(w, T, &wt)) != QMV_OK || (rc = check_lora(lora, &l)) != QMV_OK) return rc;
  if (wide(wt.N)) return QMV_ERR_UNSUPPORTED;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(index, 4) || !aligned(bias, 2)) return QMV_ERR_ALIGNMENT;
  rc = check_workspace(workspace, workspace_bytes, lora_workspace(T, wt.N, wt.K, wt.log2bs, l.count, l.rank, false));
  if (rc != QMV_OK) return rc;
  return launch_status(launch_lora(x, dtype, T, wt, l, index, bias, y, y_dtype, static_cast<char *>(workspace),
                                   (hipStream_t)stream));
}

size_t qmv_lora_4bit_backward_workspace(int64_t T, int64_t N, int64_t K, int32_t blocksize, int32_t count,
                                        int32_t rank) {
  if (check_sizes(T, N, K, blocksize) != QMV_OK || check_rank(count, rank) != QMV_OK || wide(N) || N % 32 || many(T)) return 0;
  return lora_workspace(T, N, K, log2_exact(blocksize), count, rank, true);
}

int qmv_lora_4bit_backward(const void *dy, const void *x, qmv_dtype dtype, int64_t T, const qmv_weight_4bit *w,
                           const qmv_lora *lora, const int32_t *index, void *dx, void *d_down, void *d_up,
                           qmv_dtype grad_dtype, void *workspace, size_t workspace_bytes, void *stream) {
  if (!dy || !x || !index || !dx || !d_down || !d_up) return QMV_ERR_INVALID_ARG;
  int rc = check_types(dtype, grad_dtype);
  if (rc != QMV_OK) return rc;
  Weight4 wt;
  Lora l;
  if ((rc = check_weight(w, T, &wt)) != QMV_OK || (rc = check_lora(lora, &l)) != QMV_OK) return rc;
  if (wt.N % 32 || wide(wt.N) || many(T)) return QMV_ERR_UNSUPPORTED;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(dx, 16) || !aligned(d_down, 16) || !aligned(d_up, 16) ||
      !aligned(index, 4))
    return QMV_ERR_ALIGNMENT;
  rc = check_workspace(workspace, workspace_bytes, lora_workspace(T, wt.N, wt.K, wt.log2bs, l.count, l.rank, true));
  if (rc != QMV_OK) return rc;
  return launch_status(launch_lora_backward(dy, x, dtype, T, wt, l, index, dx, d_down, d_up, grad_dtype,
                                            static_cast<char *>(workspace), (hipStream_t)stream));
}

size_t qmv_cross_entropy_4bit_workspace(int64_t T, int64_t V, int64_t K, int32_t blocksize, int32_t grad) {
  return qmv_distill_4bit_workspace(T, V, K, blocksize, 1, grad);
}

int qmv_cross_entropy_4bit(const void *x, qmv_dtype dtype, int64_t T, const qmv_weight_4bit *w, const int64_t *target,
                           const float *dloss, void *loss_out, qmv_dtype loss_dtype, void *dx, void *workspace,
                           size_t workspace_bytes, void *stream) {
  return loss(x, dtype, T, w, Targets{target, nullptr, QMV_F32, 1, 1.f}, dloss, loss_out, loss_dtype, dx, workspace,
              workspace_bytes, stream);
}

size_t qmv_distill_4bit_workspace(int64_t T, int64_t V, int64_t K, int32_t blocksize, int32_t k, int32_t grad) {
  if (check_sizes(T, V, K, blocksize) != QMV_OK || k < 1 || k > 128) return 0;
  return loss_workspace(T, V, K, log2_exact(blocksize), k, grad != 0);
}

int qmv_distill_4bit(const void *x, qmv_dtype dtype, int64_t T, const qmv_weight_4bit *w, const int64_t *ids,
                     const void *teacher, qmv_dtype teacher_dtype, int32_t k, float temperature, const float *dloss,
                     void *loss_out, qmv_dtype loss_dtype, void *dx, void *workspace, size_t workspace_bytes,
                     void *stream) {
  if (!teacher || !valid_dtype(teacher_dtype) || k < 1 || !(temperature > 0.f) || !isfinite(temperature) ||
      !isfinite(1.f / temperature))
    return QMV_ERR_INVALID_ARG;
  if (k > 128) return QMV_ERR_UNSUPPORTED;
  return loss(x, dtype, T, w, Targets{ids, teacher, teacher_dtype, k, 1.f / temperature}, dloss, loss_out, loss_dtype,
              dx, workspace, workspace_bytes, stream);
}

}  // extern "C"
