// Host side of cdrge_adapter_project (include/cdrge.h).
#include <hip/hip_runtime.h>

#include "cdrge.h"
#include "host_common.h"
#include "kernels_adapters.h"

using namespace cdrge;

namespace {

cdrge_status check(const cdrge_adapter_config* c, int64_t n_rows) {
  if (!c || c->abi_version != CDRGE_ABI_VERSION) return CDRGE_ERR_INVALID_ARG;
  if (c->dtype != CDRGE_F32 && c->dtype != CDRGE_BF16) return CDRGE_ERR_INVALID_ARG;
  if (c->in_features < 1 || c->out_features < 1 || c->n_adapters < 0 || c->max_rank < 1 || n_rows < 0)
    return CDRGE_ERR_INVALID_ARG;
  constexpr int kMost = 1 << 20;
  if (c->in_features > kMost || c->out_features > kMost || c->n_adapters > kMost || c->max_rank > 128 ||
      n_rows > (int64_t(1) << 30))
    return CDRGE_ERR_UNSUPPORTED;
  return CDRGE_OK;
}

size_t workspace(const cdrge_adapter_config* c, int64_t n_rows) {
  return align_up(sizeof(float) * static_cast<size_t>(n_rows) * c->max_rank);
}

template <class T>
cdrge_status enqueue(const AdapterArgs& a, hipStream_t s) {
  const uint32_t tiles = static_cast<uint32_t>((a.n_rows + 15) / 16);
  if (a.row_adapter && a.A > 0) {
    hipLaunchKernelGGL(k_adapter_down<T>, dim3(tiles), dim3(64), 0, s, a);
    CDRGE_HIP(hipGetLastError());
  }
  hipLaunchKernelGGL(k_adapter_project<T>, dim3(tiles, (a.O + 63) / 64), dim3(64), 0, s, a);
  CDRGE_HIP(hipGetLastError());
  return CDRGE_OK;
}

}  // namespace

extern "C" {

cdrge_status cdrge_adapter_workspace_bytes(const cdrge_adapter_config* cfg, int64_t n_rows, size_t* bytes_out) {
  if (!bytes_out) return CDRGE_ERR_INVALID_ARG;
  const cdrge_status st = check(cfg, n_rows);
  if (st != CDRGE_OK) return st;
  *bytes_out = workspace(cfg, n_rows);
  return CDRGE_OK;
}

cdrge_status cdrge_adapter_project(const cdrge_adapter_config* cfg, const cdrge_adapter_weights* weights,
                                   int64_t n_rows, const void* x, int64_t x_stride, const int32_t* row_adapter,
                                   const float* row_scale, void* y, int64_t y_stride, void* ws,
                                   size_t workspace_bytes, void* stream) {
  const cdrge_status st = check(cfg, n_rows);
  if (st != CDRGE_OK) return st;
  const int K = cfg->in_features, O = cfg->out_features;
  if (!weights || !weights->weight || weights->weight_stride < K || x_stride < K || y_stride < O)
    return CDRGE_ERR_INVALID_ARG;
  if (row_adapter && cfg->n_adapters > 0 && (!weights->down || !weights->up)) return CDRGE_ERR_INVALID_ARG;
  if (n_rows == 0) return CDRGE_OK;
  if (!x || !y) return CDRGE_ERR_INVALID_ARG;
  const size_t need = workspace(cfg, n_rows);
  if (row_adapter && (!ws || workspace_bytes < need || reinterpret_cast<uintptr_t>(ws) % kAlign != 0))
    return workspace_error("cdrge_adapter_project", need, ws ? workspace_bytes : 0);
  const AdapterArgs a{x, x_stride, weights->weight, weights->weight_stride, weights->bias, weights->down, weights->up,
                      weights->ranks, row_adapter, row_scale, y, y_stride, static_cast<float*>(ws), n_rows,
                      K, O, cfg->n_adapters, cfg->max_rank};
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return cfg->dtype == CDRGE_F32 ? enqueue<float>(a, s) : enqueue<uint16_t>(a, s);
}

}  // extern "C"
