// Host side of cdrge_scan_prompt and cdrge_scan_step (include/cdrge.h).
#include <hip/hip_runtime.h>

#include "cdrge.h"
#include "host_common.h"
#include "kernels_scan.h"

using namespace cdrge;

namespace {

int64_t channels(const cdrge_scan_config* c) {
  return int64_t(c->n_heads) * c->head_dim + int64_t(2) * c->n_groups * c->state_dim;
}

cdrge_status check_config(const cdrge_scan_config* c) {
  if (!c || c->abi_version != CDRGE_ABI_VERSION) return CDRGE_ERR_INVALID_ARG;
  if (c->dtype != CDRGE_F32 && c->dtype != CDRGE_BF16) return CDRGE_ERR_INVALID_ARG;
  if (c->n_heads < 1 || c->head_dim < 1 || c->n_groups < 1 || c->state_dim < 1 || c->conv_width < 1)
    return CDRGE_ERR_INVALID_ARG;
  if (c->n_heads % c->n_groups != 0) return CDRGE_ERR_INVALID_ARG;
  if (c->head_dim > 256 || c->state_dim > kScanMaxState || c->conv_width < 2 || c->conv_width > kScanMaxConv ||
      c->n_heads > (1 << 16))
    return CDRGE_ERR_UNSUPPORTED;
  return CDRGE_OK;
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

cdrge_status check_io(const cdrge_scan_config* c, const cdrge_scan_weights* w, const cdrge_scan_io* io) {
  if (!w || !io || !w->conv_weight || !w->decay) return CDRGE_ERR_INVALID_ARG;
  if (io->n_tokens < 0 || io->n_seqs < 1) return CDRGE_ERR_INVALID_ARG;
  const int64_t d = int64_t(c->n_heads) * c->head_dim;
  if (io->xbc_stride < channels(c) || io->dt_stride < c->n_heads || io->y_stride < d || (io->z && io->z_stride < d))
    return CDRGE_ERR_INVALID_ARG;
  if (io->n_tokens > 0 && (!io->xbc || !io->dt || !io->y)) return CDRGE_ERR_INVALID_ARG;
  const int states = !!io->conv_in + !!io->conv_out + !!io->ssm_in + !!io->ssm_out;
  if (states != 0 && states != 4) return CDRGE_ERR_INVALID_ARG;
  if (states == 0 && (io->slots || io->positions)) return CDRGE_ERR_INVALID_ARG;
  if (states == 4) {
    if (io->n_slots < 1 || (!io->slots && io->n_slots < io->n_seqs)) return CDRGE_ERR_INVALID_ARG;
    if (!aligned16(io->conv_in) || !aligned16(io->conv_out) || !aligned16(io->ssm_in) || !aligned16(io->ssm_out))
      return CDRGE_ERR_INVALID_ARG;
  }
  if (!io->offsets && io->n_tokens % io->n_seqs != 0) return CDRGE_ERR_INVALID_ARG;
  if (io->n_tokens > (int64_t(1) << 30) || io->n_seqs > (1 << 20)) return CDRGE_ERR_UNSUPPORTED;
  return CDRGE_OK;
}

ScanArgs make_args(const cdrge_scan_config* c, const cdrge_scan_weights* w, const cdrge_scan_io* io) {
  ScanArgs a;
  a.xbc = io->xbc;
  a.xbc_stride = io->xbc_stride;
  a.dt = io->dt;
  a.dt_stride = io->dt_stride;
  a.z = io->z;
  a.z_stride = io->z_stride;
  a.y = io->y;
  a.y_stride = io->y_stride;
  a.n_tokens = io->n_tokens;
  a.offsets = io->offsets;
  a.slots = io->slots;
  a.positions = io->positions;
  a.conv_in = io->conv_in;
  a.conv_out = io->conv_out;
  a.ssm_in = io->ssm_in;
  a.ssm_out = io->ssm_out;
  a.conv_weight = w->conv_weight;
  a.conv_bias = w->conv_bias;
  a.decay = w->decay;
  a.skip = w->skip;
  a.dt_bias = w->dt_bias;
  a.n_seqs = io->n_seqs;
  a.n_slots = io->n_slots;
  a.H = c->n_heads;
  a.P = c->head_dim;
  a.G = c->n_groups;
  a.N = c->state_dim;
  a.W = c->conv_width;
  a.C = static_cast<int>(channels(c));
  a.ptiles = 1;
  return a;
}

constexpr int64_t kMostBlocks = (int64_t(1) << 31) - 1;

template <class T, int kLanes, int kRpt>
cdrge_status launch_step(ScanArgs a, hipStream_t s) {
  constexpr int kTile = 256 / kLanes * kRpt;
  a.ptiles = (a.P + kTile - 1) / kTile;
  const int64_t n = int64_t(a.n_seqs) * a.H * a.ptiles;
  if (n > kMostBlocks) return CDRGE_ERR_UNSUPPORTED;
  hipLaunchKernelGGL((k_scan_step<T, kLanes, kRpt>), dim3(static_cast<uint32_t>(n)), dim3(256), 0, s, a);
  CDRGE_HIP(hipGetLastError());
  return CDRGE_OK;
}

template <class T>
cdrge_status enqueue_step(const ScanArgs& a, hipStream_t s) {
  if (a.N <= 16) return launch_step<T, 4, 1>(a, s);
  if (a.N <= 32) return launch_step<T, 8, 2>(a, s);
  if (a.N <= 64) return launch_step<T, 16, 4>(a, s);
  if (a.N <= 128) return launch_step<T, 32, 8>(a, s);
  return launch_step<T, 64, 8>(a, s);
}

template <class T, int kQuarter>
cdrge_status launch_walk(ScanArgs a, hipStream_t s) {
  a.ptiles = (a.P + 63) / 64;
  const int64_t n = int64_t(a.n_seqs) * a.H * a.ptiles;
  if (n > kMostBlocks) return CDRGE_ERR_UNSUPPORTED;
  hipLaunchKernelGGL((k_scan_walk<T, kQuarter>), dim3(static_cast<uint32_t>(n)), dim3(256), 0, s, a);
  CDRGE_HIP(hipGetLastError());
  if (a.conv_in) {
    const int cblocks = (a.C + 255) / 256;
    hipLaunchKernelGGL(k_scan_ring<T>, dim3(static_cast<uint32_t>(a.n_seqs) * cblocks), dim3(256), 0, s, a, cblocks);
    CDRGE_HIP(hipGetLastError());
  }
  return CDRGE_OK;
}

template <class T>
cdrge_status enqueue_prompt(const ScanArgs& a, hipStream_t s) {
  if (a.N <= 16) return launch_walk<T, 4>(a, s);
  if (a.N <= 64) return launch_walk<T, 16>(a, s);
  if (a.N <= 128) return launch_walk<T, 32>(a, s);
  return launch_walk<T, 64>(a, s);
}

}  // namespace

extern "C" {

cdrge_status cdrge_scan_workspace_bytes(const cdrge_scan_config* cfg, int64_t n_tokens, int32_t n_seqs,
                                        size_t* bytes_out) {
  if (!bytes_out || n_tokens < 0 || n_seqs < 1) return CDRGE_ERR_INVALID_ARG;
  const cdrge_status st = check_config(cfg);
  if (st != CDRGE_OK) return st;
  *bytes_out = 256;
  return CDRGE_OK;
}

cdrge_status cdrge_scan_prompt(const cdrge_scan_config* cfg, const cdrge_scan_weights* weights,
                               const cdrge_scan_io* io, void* workspace, size_t workspace_bytes, void* stream) {
  cdrge_status st = check_config(cfg);
  if (st == CDRGE_OK) st = check_io(cfg, weights, io);
  if (st != CDRGE_OK) return st;
  size_t need = 0;
  st = cdrge_scan_workspace_bytes(cfg, io->n_tokens, io->n_seqs, &need);
  if (st != CDRGE_OK) return st;
  if (!workspace || workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % kAlign != 0)
    return workspace_error("cdrge_scan_prompt", need, workspace ? workspace_bytes : 0);
  const ScanArgs a = make_args(cfg, weights, io);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return cfg->dtype == CDRGE_F32 ? enqueue_prompt<float>(a, s) : enqueue_prompt<uint16_t>(a, s);
}

cdrge_status cdrge_scan_step(const cdrge_scan_config* cfg, const cdrge_scan_weights* weights,
                             const cdrge_scan_io* io, void* stream) {
  cdrge_status st = check_config(cfg);
  if (st == CDRGE_OK) st = check_io(cfg, weights, io);
  if (st != CDRGE_OK) return st;
  if (io->offsets || io->n_tokens != io->n_seqs || !io->ssm_in || !io->positions) return CDRGE_ERR_INVALID_ARG;
  const ScanArgs a = make_args(cfg, weights, io);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return cfg->dtype == CDRGE_F32 ? enqueue_step<float>(a, s) : enqueue_step<uint16_t>(a, s);
}

}  // extern "C"
