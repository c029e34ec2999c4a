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
  if (c->vocab > (1 << 24) || c->top_k > 1024 || c->n_models > (1 << 20) || n_rows > (int64_t(1) << 30))
    return CDRGE_ERR_UNSUPPORTED;
  return CDRGE_OK;
}

template <class T, bool kGrad, int kTeam>
void launch(const DistillArgs& a, hipStream_t s) {
  constexpr int kRows = kTeam == 64 ? 4 : 1;
  const size_t lds = size_t(8) * a.top_k * kRows;
  hipLaunchKernelGGL((k_distill<T, kGrad, kTeam>), dim3(static_cast<uint32_t>((a.n_rows + kRows - 1) / kRows)),
                     dim3(kTeam == 64 ? 256 : kTeam), lds, s, a);
}

template <class T, bool kGrad>
void launch_team(const DistillArgs& a, hipStream_t s) {
  if (a.vocab <= 2048)
    launch<T, kGrad, 64>(a, s);
  else
    launch<T, kGrad, 256>(a, s);
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
    hipLaunchKernelGGL(k_distill_mean, dim3(c->n_models), dim3(256), 0, s, a.row_losses, a.ids, a.teacher, a.top_k,
                       a.n_rows / c->n_models, losses);
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
