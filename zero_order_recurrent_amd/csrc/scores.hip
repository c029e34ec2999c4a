// Host side of cdrge_token_scores and cdrge_token_scores_grad (include/cdrge.h).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "cdrge.h"
#include "host_common.h"
#include "kernels_scores.h"

using namespace cdrge;

namespace {

cdrge_status check(const cdrge_score_config* c, int64_t n_rows, const void* logits, int64_t stride) {
  if (!c || c->abi_version != CDRGE_ABI_VERSION) return CDRGE_ERR_INVALID_ARG;
  if (c->dtype != CDRGE_F32 && c->dtype != CDRGE_BF16) return CDRGE_ERR_INVALID_ARG;
  if (c->vocab < 1 || c->top_k < 0 || c->top_k > c->vocab || n_rows < 0) return CDRGE_ERR_INVALID_ARG;
  if (!std::isfinite(c->temperature) || !(c->temperature > 0.f)) return CDRGE_ERR_INVALID_ARG;
  if (stride < c->vocab || (n_rows > 0 && !logits)) return CDRGE_ERR_INVALID_ARG;
  // beyond these the scaled logits or the gradient leave float32's range for ordinary logits
  if (c->temperature < 0x1p-60f || c->temperature > 0x1p60f) return CDRGE_ERR_UNSUPPORTED;
  if (c->vocab > (1 << 24) || c->top_k > 1024 || n_rows > (int64_t(1) << 30)) return CDRGE_ERR_UNSUPPORTED;
  return CDRGE_OK;
}

template <class T, int kMode, int kTeam, int kPieces>
cdrge_status launch(const ScoreArgs& a, hipStream_t s) {
  constexpr int kThreads = distill_threads(kTeam), kRows = kThreads / kTeam;
  const size_t lds = kMode == kScoreTop ? score_lds(a.cap, kTeam) * kRows : 0;
  hipLaunchKernelGGL((k_scores<T, kMode, kTeam, kPieces>), grid_of((a.n_rows + kRows - 1) / kRows, kThreads), dim3(kThreads),
                     lds, s, a);
  CDRGE_HIP(hipGetLastError());
  return CDRGE_OK;
}

// Threads of a row and pieces a thread: as for the distillation loss the fewest threads that hold the row in at most 8
// pieces each, but where alternatives are asked for no fewer than there are of them, as far as the row has pieces, so that
// the threads' largest logits bound them.
template <class T, int kMode>
cdrge_status launch_team(const ScoreArgs& a, hipStream_t s) {
  const int pieces = (a.vocab + DistillRow<T>::kPer - 1) / DistillRow<T>::kPer, least = std::min(a.top_k, pieces);
  if (least <= 16 && pieces <= 16 * 4 && a.top_k <= 64)
    return pieces <= 16 ? launch<T, kMode, 16, 1>(a, s) : launch<T, kMode, 16, 4>(a, s);
  if (least <= 64 && pieces <= 64 * 2) return launch<T, kMode, 64, 2>(a, s);
  if (least <= 64 && pieces <= 64 * 8) return launch<T, kMode, 64, 8>(a, s);
  if (least <= 256 && pieces <= 256 * 4) return launch<T, kMode, 256, 4>(a, s);
  if (least <= 256 && pieces <= 256 * 8) return launch<T, kMode, 256, 8>(a, s);
  if (least <= 512 && pieces <= 512 * 8) return launch<T, kMode, 512, 8>(a, s);
  if (pieces <= 1024 * 8) return launch<T, kMode, 1024, 8>(a, s);
  if (pieces <= 1024 * 16) return launch<T, kMode, 1024, 16>(a, s);
  return launch<T, kMode, 1024, 0>(a, s);
}

template <int kMode>
cdrge_status enqueue(const cdrge_score_config* c, ScoreArgs& a, hipStream_t s) {
  if (a.n_rows == 0) return CDRGE_OK;
  a.vocab = c->vocab;
  a.tau = c->temperature;
  a.top_k = kMode == kScoreTop ? c->top_k : 0;
  a.cap = std::min(c->vocab, std::max(4 * a.top_k, 128));
  if (a.cap > 512)  // sorted as a power of two
    for (int n = 1024;; n *= 2)
      if (n >= a.cap) {
        a.cap = n;
        break;
      }
  return c->dtype == CDRGE_F32 ? launch_team<float, kMode>(a, s) : launch_team<uint16_t, kMode>(a, s);
}

}  // namespace

extern "C" {

cdrge_status cdrge_token_scores(const cdrge_score_config* cfg, int64_t n_rows, const void* logits,
                                int64_t logits_stride, const int32_t* tokens, float* logprobs, float* entropy,
                                int32_t* top_ids, float* top_logprobs, void* stream) {
  const cdrge_status st = check(cfg, n_rows, logits, logits_stride);
  if (st != CDRGE_OK) return st;
  if (n_rows > 0 && logprobs && !tokens) return CDRGE_ERR_INVALID_ARG;
  if (n_rows > 0 && cfg->top_k > 0 && (!top_ids || !top_logprobs)) return CDRGE_ERR_INVALID_ARG;
  ScoreArgs a{};
  a.logits = logits;
  a.logits_stride = logits_stride;
  a.tokens = tokens;
  a.logprobs = logprobs;
  a.entropy = entropy;
  a.top_ids = top_ids;
  a.top_logprobs = top_logprobs;
  a.n_rows = n_rows;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return cfg->top_k > 0 ? enqueue<kScoreTop>(cfg, a, s) : enqueue<kScoreOnly>(cfg, a, s);
}

cdrge_status cdrge_token_scores_grad(const cdrge_score_config* cfg, int64_t n_rows, const void* logits,
                                     int64_t logits_stride, const int32_t* tokens, const float* d_logprob,
                                     const float* d_entropy, void* dlogits, int64_t dlogits_stride, void* stream) {
  const cdrge_status st = check(cfg, n_rows, logits, logits_stride);
  if (st != CDRGE_OK) return st;
  if (dlogits_stride < cfg->vocab || (n_rows > 0 && (!dlogits || (d_logprob && !tokens)))) return CDRGE_ERR_INVALID_ARG;
  if (n_rows > 0 && dlogits == logits && dlogits_stride != logits_stride) return CDRGE_ERR_INVALID_ARG;
  ScoreArgs a{};
  a.logits = logits;
  a.logits_stride = logits_stride;
  a.tokens = tokens;
  a.d_logprob = d_logprob;
  a.d_entropy = d_entropy;
  a.dlogits = dlogits;
  a.dlogits_stride = dlogits_stride;
  a.n_rows = n_rows;
  return enqueue<kScoreGrad>(cfg, a, static_cast<hipStream_t>(stream));
}

}  // extern "C"
