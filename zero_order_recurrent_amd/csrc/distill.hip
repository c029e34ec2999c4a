// Host side of cdrge_distill_losses and cdrge_distill_grad (include/cdrge.h).
#include <hip/hip_runtime.h>

#include <cmath>

#include "cdrge.h"
#include "host_common.h"
#include "kernels_distill.h"

using namespace cdrge;

namespace {

cdrge_status check(const cdrge_distill_config* c, int64_t n_rows, const void* logits, int64_t stride, const void* ids,
                   const void* teacher, const void* row_losses) {
  if (!c || c->abi_version != CDRGE_ABI_VERSION) return CDRGE_ERR_INVALID_ARG;
  if (c->dtype != CDRGE_F32 && c->dtype != CDRGE_BF16) return CDRGE_ERR_INVALID_ARG;
  if (c->vocab < 1 || c->top_k < 1 || c->n_models < 1 || n_rows < 0) return CDRGE_ERR_INVALID_ARG;
  if (!std::isfinite(c->temperature) || !(c->temperature > 0.f)) return CDRGE_ERR_INVALID_ARG;
  if (n_rows % c->n_models != 0 || stride < c->vocab) return CDRGE_ERR_INVALID_ARG;
  if (n_rows > 0 && (!logits || !ids || !teacher || !row_losses)) return CDRGE_ERR_INVALID_ARG;
  // beyond these the scaled logits or the loss's tau^2 leave float32's range for ordinary logits
  if (c->temperature < 0x1p-60f || c->temperature > 0x1p60f) return CDRGE_ERR_UNSUPPORTED;
  if (c->vocab > (1 << 24) || c->top_k > 1024 || c->n_models > (1 << 20) || n_rows > (int64_t(1) << 30))
    return CDRGE_ERR_UNSUPPORTED;
  return CDRGE_OK;
}

template <class T, bool kGrad, int kTeam, int kPieces>
void launch(const DistillArgs& a, hipStream_t s) {
  constexpr int kThreads = distill_threads(kTeam), kRows = kThreads / kTeam;
  const size_t lds = size_t(8) * ((a.top_k + 3) & ~3) * kRows;
  hipLaunchKernelGGL((k_distill<T, kGrad, kTeam, kPieces>), grid_of((a.n_rows + kRows - 1) / kRows, kThreads),
                     dim3(kThreads), lds, s, a);
}

// Threads of a row and pieces a thread: the fewest threads that hold the row in at most 8 pieces each, so that short rows share a workgroup and long ones have enough loads in flight.
// A team of 16 holds at most 256 teacher entries in its registers while the gradient is written.
template <class T, bool kGrad>
void launch_team(const DistillArgs& a, hipStream_t s) {
  const int pieces = (a.vocab + DistillRow<T>::kPer - 1) / DistillRow<T>::kPer;
  if (pieces <= 16 * 4 && a.top_k <= 256) return pieces <= 16 ? launch<T, kGrad, 16, 1>(a, s) : launch<T, kGrad, 16, 4>(a, s);
  if (pieces <= 64 * 2) return launch<T, kGrad, 64, 2>(a, s);
  if (pieces <= 64 * 8) return launch<T, kGrad, 64, 8>(a, s);
  if (pieces <= 256 * 4) return launch<T, kGrad, 256, 4>(a, s);
  if (pieces <= 256 * 8) return launch<T, kGrad, 256, 8>(a, s);
  if (pieces <= 512 * 8) return launch<T, kGrad, 512, 8>(a, s);
  if (pieces <= 1024 * 8) return launch<T, kGrad, 1024, 8>(a, s);
  return launch<T, kGrad, 1024, 0>(a, s);
}

template <bool kGrad>
cdrge_status enqueue(const cdrge_distill_config* c, const DistillArgs& a, float* losses, hipStream_t s) {
  if (a.n_rows > 0) {
    if (c->dtype == CDRGE_F32)
      launch_team<float, kGrad>(a, s);
    else
      launch_team<uint16_t, kGrad>(a, s);
    CDRGE_HIP(hipGetLastError());
  }
  if (losses) {
    hipLaunchKernelGGL(k_distill_mean, dim3(c->n_models), dim3(256), 0, s, a.row_losses, a.n_rows / c->n_models, losses);
    CDRGE_HIP(hipGetLastError());
  }
  return CDRGE_OK;
}

}  // namespace

extern "C" {

cdrge_status cdrge_distill_losses(const cdrge_distill_config* cfg, int64_t n_rows, const void* logits,
                                  int64_t logits_stride, const int32_t* ids, const float* teacher,
                                  float* row_losses, float* losses, void* stream) {
  const cdrge_status st = check(cfg, n_rows, logits, logits_stride, ids, teacher, row_losses);
  if (st != CDRGE_OK) return st;
  const DistillArgs a{logits, logits_stride, ids, teacher, nullptr, row_losses, nullptr, 0, n_rows,
                      cfg->vocab, cfg->top_k, cfg->temperature};
  return enqueue<false>(cfg, a, losses, static_cast<hipStream_t>(stream));
}

cdrge_status cdrge_distill_grad(const cdrge_distill_config* cfg, int64_t n_rows, const void* logits,
                                int64_t logits_stride, const int32_t* ids, const float* teacher,
                                const float* row_grad, float* row_losses, float* losses, void* dlogits,
                                int64_t dlogits_stride, void* stream) {
  const cdrge_status st = check(cfg, n_rows, logits, logits_stride, ids, teacher, row_losses);
  if (st != CDRGE_OK) return st;
  if (dlogits_stride < cfg->vocab || (n_rows > 0 && !dlogits)) return CDRGE_ERR_INVALID_ARG;
  if (dlogits == logits && dlogits_stride != logits_stride) return CDRGE_ERR_INVALID_ARG;
  const DistillArgs a{logits, logits_stride, ids, teacher, row_grad, row_losses, dlogits, dlogits_stride, n_rows,
                      cfg->vocab, cfg->top_k, cfg->temperature};
  return enqueue<true>(cfg, a, losses, static_cast<hipStream_t>(stream));
}

}  // extern "C"
