// Host side of cdrge_mx_quantize, cdrge_mx_dequantize and cdrge_mx_project (include/cdrge.h).
#include <hip/hip_runtime.h>

#include "cdrge.h"
#include "host_common.h"
#include "kernels_mx.h"

using namespace cdrge;

namespace {

cdrge_status check(const cdrge_mx_config* c, int64_t n_rows) {
  if (!c || c->abi_version != CDRGE_ABI_VERSION) return CDRGE_ERR_INVALID_ARG;
  if (c->dtype != CDRGE_F32 && c->dtype != CDRGE_BF16) return CDRGE_ERR_INVALID_ARG;
  if (c->in_features < 1 || c->out_features < 1 || n_rows < 0) return CDRGE_ERR_INVALID_ARG;
  constexpr int kMost = 1 << 20;
  if (c->in_features > kMost || c->out_features > kMost || n_rows > (int64_t(1) << 30)) return CDRGE_ERR_UNSUPPORTED;
  return CDRGE_OK;
}

bool aligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

int blocks_of(const cdrge_mx_config* c) { return (c->in_features + 31) / 32; }

cdrge_status check_rows(const cdrge_mx_config* c, int64_t n_rows, const void* x, int64_t stride, const uint8_t* codes,
                        const uint8_t* scales) {
  const cdrge_status st = check(c, n_rows);
  if (st != CDRGE_OK) return st;
  if (stride < c->in_features || (n_rows > 0 && (!x || !codes || !scales)) || !aligned(codes, 16)) return CDRGE_ERR_INVALID_ARG;
  return CDRGE_OK;
}

// Workgroups of the kernels that take a quarter of a block a thread; parts: workgroups of a row.
int64_t quarter_groups(int64_t n_rows, int quarters, int* parts) {
  *parts = (quarters + 255) / 256;
  if (*parts > 1) return n_rows * *parts;
  const int each = 256 / quarters;
  return (n_rows + each - 1) / each;
}

constexpr int64_t kMostGroups = int64_t(1) << 35;  // 2^20 by 2^15 of a grid

cdrge_status quantize(const cdrge_mx_config* c, int64_t n_rows, const void* x, int64_t stride, uint8_t* codes,
                      uint8_t* scales, hipStream_t s) {
  int parts = 1;
  const int quarters = 4 * blocks_of(c);
  const int64_t n = quarter_groups(n_rows, quarters, &parts);
  if (n > kMostGroups) return CDRGE_ERR_UNSUPPORTED;
  if (n == 0) return CDRGE_OK;
  if (c->dtype == CDRGE_F32)
    hipLaunchKernelGGL(k_mx_quantize<float>, grid_of(n, 256), dim3(256), 0, s, static_cast<const float*>(x), stride, n_rows,
                       c->in_features, quarters, parts, codes, scales);
  else
    hipLaunchKernelGGL(k_mx_quantize<uint16_t>, grid_of(n, 256), dim3(256), 0, s, static_cast<const uint16_t*>(x), stride,
                       n_rows, c->in_features, quarters, parts, codes, scales);
  CDRGE_HIP(hipGetLastError());
  return CDRGE_OK;
}

struct Plan {
  size_t codes, scales, total;
};

Plan make_plan(const cdrge_mx_config* c, int64_t n_rows) {
  Plan p{};
  const size_t blocks = static_cast<size_t>(n_rows) * blocks_of(c);
  p.scales = align_up(16 * blocks);
  p.total = align_up(p.scales + blocks);
  return p;
}

int64_t project_groups(const cdrge_mx_config* c, int64_t n_rows) {
  return (n_rows + 63) / 64 * ((c->out_features + 15) / 16);
}

}  // namespace

extern "C" {

cdrge_status cdrge_mx_quantize(const cdrge_mx_config* cfg, int64_t n_rows, const void* x, int64_t x_stride,
                               uint8_t* codes, uint8_t* scales, void* stream) {
  const cdrge_status st = check_rows(cfg, n_rows, x, x_stride, codes, scales);
  if (st != CDRGE_OK) return st;
  return quantize(cfg, n_rows, x, x_stride, codes, scales, static_cast<hipStream_t>(stream));
}

cdrge_status cdrge_mx_dequantize(const cdrge_mx_config* cfg, int64_t n_rows, const uint8_t* codes,
                                 const uint8_t* scales, void* x, int64_t x_stride, void* stream) {
  const cdrge_status st = check_rows(cfg, n_rows, x, x_stride, codes, scales);
  if (st != CDRGE_OK) return st;
  int parts = 1;
  const int quarters = 4 * blocks_of(cfg);
  const int64_t n = quarter_groups(n_rows, quarters, &parts);
  if (n > kMostGroups) return CDRGE_ERR_UNSUPPORTED;
  if (n == 0) return CDRGE_OK;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (cfg->dtype == CDRGE_F32)
    hipLaunchKernelGGL(k_mx_dequantize<float>, grid_of(n, 256), dim3(256), 0, s, codes, scales, n_rows, cfg->in_features,
                       quarters, parts, static_cast<float*>(x), x_stride);
  else
    hipLaunchKernelGGL(k_mx_dequantize<uint16_t>, grid_of(n, 256), dim3(256), 0, s, codes, scales, n_rows, cfg->in_features,
                       quarters, parts, static_cast<uint16_t*>(x), x_stride);
  CDRGE_HIP(hipGetLastError());
  return CDRGE_OK;
}

cdrge_status cdrge_mx_workspace_bytes(const cdrge_mx_config* cfg, int64_t n_rows, size_t* bytes_out) {
  if (!bytes_out) return CDRGE_ERR_INVALID_ARG;
  const cdrge_status st = check(cfg, n_rows);
  if (st != CDRGE_OK) return st;
  if (project_groups(cfg, n_rows) > kMostGroups) return CDRGE_ERR_UNSUPPORTED;
  *bytes_out = make_plan(cfg, n_rows).total;
  return CDRGE_OK;
}

cdrge_status cdrge_mx_project(const cdrge_mx_config* cfg, const uint8_t* w_codes, const uint8_t* w_scales,
                              const void* bias, int64_t n_rows, const void* x, int64_t x_stride, void* y,
                              int64_t y_stride, void* workspace, size_t workspace_bytes, void* stream) {
  size_t need = 0;
  cdrge_status st = cdrge_mx_workspace_bytes(cfg, n_rows, &need);
  if (st != CDRGE_OK) return st;
  if (!w_codes || !w_scales || !aligned(w_codes, 16)) return CDRGE_ERR_INVALID_ARG;
  if (x_stride < cfg->in_features || y_stride < cfg->out_features) return CDRGE_ERR_INVALID_ARG;
  if (n_rows == 0) return CDRGE_OK;
  if (!x || !y) return CDRGE_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < need || !aligned(workspace, kAlign))
    return workspace_error("cdrge_mx_project", need, workspace ? workspace_bytes : 0);
  const Plan p = make_plan(cfg, n_rows);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  uint8_t* const codes = static_cast<uint8_t*>(workspace) + p.codes;
  uint8_t* const scales = static_cast<uint8_t*>(workspace) + p.scales;
  st = quantize(cfg, n_rows, x, x_stride, codes, scales, s);
  if (st != CDRGE_OK) return st;
  const MxArgs a{w_codes, w_scales, bias, codes, scales, y, y_stride, n_rows, cfg->out_features, blocks_of(cfg)};
  const int o_tiles = (a.O + 15) / 16;
  const dim3 grid = grid_of(project_groups(cfg, n_rows), 512);
  if (cfg->dtype == CDRGE_F32)
    hipLaunchKernelGGL(k_mx_rows<float>, grid, dim3(512), 0, s, a, o_tiles);
  else
    hipLaunchKernelGGL(k_mx_rows<uint16_t>, grid, dim3(512), 0, s, a, o_tiles);
  CDRGE_HIP(hipGetLastError());
  return CDRGE_OK;
}

}  // extern "C"
