// Host side of cdrge_delta_prompt and cdrge_delta_step (include/cdrge.h).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "cdrge.h"
#include "host_common.h"
#include "kernels_delta.h"

using namespace cdrge;

namespace {

constexpr int64_t kMostBlocks = (int64_t(1) << 31) - 1;

cdrge_status check_config(const cdrge_delta_config* c) {
  if (!c || c->abi_version != CDRGE_ABI_VERSION) return CDRGE_ERR_INVALID_ARG;
  if (c->dtype != CDRGE_F32 && c->dtype != CDRGE_BF16) return CDRGE_ERR_INVALID_ARG;
  if (c->n_heads < 1 || c->value_dim < 1 || c->n_groups < 1 || c->key_dim < 1) return CDRGE_ERR_INVALID_ARG;
  if (c->n_heads % c->n_groups != 0) return CDRGE_ERR_INVALID_ARG;
  if (!std::isfinite(c->q_scale) || !std::isfinite(c->norm_eps) || !(c->norm_eps > 0.f)) return CDRGE_ERR_INVALID_ARG;
  if (c->value_dim > 256 || c->key_dim > kScanMaxState || c->n_heads > (1 << 16)) return CDRGE_ERR_UNSUPPORTED;
  if (std::fabs(c->q_scale) > 0x1p60f || c->norm_eps < 0x1p-60f || c->norm_eps > 1.f) return CDRGE_ERR_UNSUPPORTED;
  return CDRGE_OK;
}

bool aligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

cdrge_status check_io(const cdrge_delta_config* c, const cdrge_delta_weights* w, const cdrge_delta_io* io) {
  if (!w || !io || !w->decay) return CDRGE_ERR_INVALID_ARG;
  if (io->n_tokens < 0 || io->n_seqs < 1) return CDRGE_ERR_INVALID_ARG;
  const int64_t keys = int64_t(c->n_groups) * c->key_dim, values = int64_t(c->n_heads) * c->value_dim;
  if (io->q_stride < keys || io->k_stride < keys || io->v_stride < values || io->y_stride < values ||
      io->dt_stride < c->n_heads || io->beta_stride < c->n_heads)
    return CDRGE_ERR_INVALID_ARG;
  if (io->n_tokens > 0 && (!io->q || !io->k || !io->v || !io->dt || !io->beta || !io->y)) return CDRGE_ERR_INVALID_ARG;
  if (!io->state_in != !io->state_out) return CDRGE_ERR_INVALID_ARG;
  if (!io->state_in && (io->slots || io->positions)) return CDRGE_ERR_INVALID_ARG;
  if (io->state_in) {
    if (io->n_slots < 1 || (!io->slots && io->n_slots < io->n_seqs)) return CDRGE_ERR_INVALID_ARG;
    const size_t piece = c->key_dim % 4 == 0 ? 16 : 4;
    if (!aligned(io->state_in, piece) || !aligned(io->state_out, piece)) return CDRGE_ERR_INVALID_ARG;
  }
  if (!io->offsets && io->n_tokens % io->n_seqs != 0) return CDRGE_ERR_INVALID_ARG;
  if (io->n_tokens > (int64_t(1) << 30) || io->n_seqs > (1 << 20)) return CDRGE_ERR_UNSUPPORTED;
  return CDRGE_OK;
}

DeltaArgs make_args(const cdrge_delta_config* c, const cdrge_delta_weights* w, const cdrge_delta_io* io) {
  DeltaArgs a{};
  a.s.dt = io->dt;
  a.s.dt_stride = io->dt_stride;
  a.s.y = io->y;
  a.s.y_stride = io->y_stride;
  a.s.n_tokens = io->n_tokens;
  a.s.offsets = io->offsets;
  a.s.slots = io->slots;
  a.s.positions = io->positions;
  a.s.ssm_in = io->state_in;
  a.s.ssm_out = io->state_out;
  a.s.decay = w->decay;
  a.s.dt_bias = w->dt_bias;
  a.s.n_seqs = io->n_seqs;
  a.s.n_slots = io->n_slots;
  a.s.H = c->n_heads;
  a.s.P = c->value_dim;
  a.s.G = c->n_groups;
  a.s.N = c->key_dim;
  a.s.ptiles = 1;
  a.q = io->q;
  a.q_stride = io->q_stride;
  a.k = io->k;
  a.k_stride = io->k_stride;
  a.v = io->v;
  a.v_stride = io->v_stride;
  a.beta = io->beta;
  a.beta_stride = io->beta_stride;
  a.q_scale = c->q_scale;
  a.norm_eps = c->norm_eps;
  return a;
}

// How a prompt call is cut up and where its workspace's parts lie; by sizes alone.
struct Plan {
  int max_blocks;
  size_t slots, counts, start, bounds, block_of, piece_of, total;
};

Plan make_plan(int64_t n_tokens, int32_t n_seqs, bool equal) {
  Plan p{};
  const int64_t blocks = equal ? int64_t(n_seqs) * scan_blocks_of(n_tokens / n_seqs) : n_tokens / kScanBlock + n_seqs;
  p.max_blocks = static_cast<int>(blocks);
  size_t at = 0;
  auto region = [&](size_t bytes) {
    const size_t here = at;
    at = align_up(at + bytes);
    return here;
  };
  p.slots = region(sizeof(int32_t) * n_seqs);
  if (!equal) {
    p.counts = region(2 * sizeof(int32_t));
    p.start = region(sizeof(int2) * n_seqs);
    p.bounds = region(sizeof(int2) * n_seqs);
    p.block_of = region(sizeof(int2) * blocks);
    p.piece_of = region(sizeof(int2) * n_seqs);
  }
  p.total = at;
  return p;
}

ScanWork make_work(const Plan& p, void* ws) {
  char* const at = static_cast<char*>(ws);
  ScanWork w{};
  w.slots = reinterpret_cast<int32_t*>(at + p.slots);
  w.counts = reinterpret_cast<int32_t*>(at + p.counts);
  w.start = reinterpret_cast<int2*>(at + p.start);
  w.bounds = reinterpret_cast<int2*>(at + p.bounds);
  w.block_of = reinterpret_cast<int2*>(at + p.block_of);
  w.piece_of = reinterpret_cast<int2*>(at + p.piece_of);
  w.piece_blocks = 1 << 30;  // a sequence is one piece
  w.max_blocks = p.max_blocks;
  return w;
}

template <class T, int kLanes, int kRpt, bool kStep>
cdrge_status launch_tokens(DeltaArgs a, const ScanWork& w, hipStream_t s) {
  constexpr int kTile = 256 / kLanes * kRpt;
  a.s.ptiles = (a.s.P + kTile - 1) / kTile;
  const int64_t n = int64_t(a.s.n_seqs) * a.s.H * a.s.ptiles;
  if (n > kMostBlocks) return CDRGE_ERR_UNSUPPORTED;
  a.s.owned = scan_owned(a.s.slots, a.s.n_seqs, n);
  if (a.s.owned) {
    if (kStep)
      hipLaunchKernelGGL(k_scan_mark<T>, dim3((a.s.n_seqs + 63) / 64), dim3(64 * kScanOwnerWaves), 0, s, a.s, kTile);
    else
      hipLaunchKernelGGL(k_scan_owners, dim3((a.s.n_seqs + 63) / 64), dim3(64 * kScanOwnerWaves), 0, s, a.s, w.slots);
    CDRGE_HIP(hipGetLastError());
  }
  hipLaunchKernelGGL((k_delta_tokens<T, kLanes, kRpt, kStep>), grid_of(n, 256), dim3(256), 0, s, a, w);
  CDRGE_HIP(hipGetLastError());
  return CDRGE_OK;
}

template <class T, bool kStep>
cdrge_status enqueue_tokens(const DeltaArgs& a, const ScanWork& w, hipStream_t s) {
  if (a.s.N <= 16) return launch_tokens<T, 4, 1, kStep>(a, w, s);
  if (a.s.N <= 32) return launch_tokens<T, 8, 2, kStep>(a, w, s);
  if (a.s.N <= 64) return launch_tokens<T, 16, 4, kStep>(a, w, s);
  if (a.s.N <= 128) return launch_tokens<T, 32, 8, kStep>(a, w, s);
  return launch_tokens<T, 64, 8, kStep>(a, w, s);
}

template <class T>
cdrge_status enqueue_prompt(const DeltaArgs& a, const ScanWork& w, hipStream_t s) {
  if (a.s.offsets) {
    hipLaunchKernelGGL(k_scan_map, dim3(1), dim3(1024), 0, s, a.s, w);
    CDRGE_HIP(hipGetLastError());
  }
  return enqueue_tokens<T, false>(a, w, s);
}

// Whether the call's sizes fit the kernels' 32-bit counts.
bool fits(const cdrge_delta_config* c, int64_t n_tokens, int32_t n_seqs) {
  const int64_t blocks = n_tokens / kScanBlock + n_seqs, tiles = (c->value_dim + 15) / 16;
  return n_tokens <= (int64_t(1) << 30) && n_seqs <= (1 << 20) && blocks * c->n_heads * tiles <= kMostBlocks;
}

}  // namespace

extern "C" {

cdrge_status cdrge_delta_workspace_bytes(const cdrge_delta_config* cfg, int64_t n_tokens, int32_t n_seqs,
                                         size_t* bytes_out) {
  if (!bytes_out || n_tokens < 0 || n_seqs < 1) return CDRGE_ERR_INVALID_ARG;
  const cdrge_status st = check_config(cfg);
  if (st != CDRGE_OK) return st;
  if (!fits(cfg, n_tokens, n_seqs)) return CDRGE_ERR_UNSUPPORTED;
  *bytes_out = make_plan(n_tokens, n_seqs, false).total;
  if (n_tokens % n_seqs == 0) *bytes_out = std::max(*bytes_out, make_plan(n_tokens, n_seqs, true).total);
  return CDRGE_OK;
}

cdrge_status cdrge_delta_prompt(const cdrge_delta_config* cfg, const cdrge_delta_weights* weights,
                                const cdrge_delta_io* io, void* workspace, size_t workspace_bytes, void* stream) {
  cdrge_status st = check_config(cfg);
  if (st == CDRGE_OK) st = check_io(cfg, weights, io);
  if (st != CDRGE_OK) return st;
  size_t need = 0;
  st = cdrge_delta_workspace_bytes(cfg, io->n_tokens, io->n_seqs, &need);
  if (st != CDRGE_OK) return st;
  if (!workspace || workspace_bytes < need || !aligned(workspace, kAlign))
    return workspace_error("cdrge_delta_prompt", need, workspace ? workspace_bytes : 0);
  const DeltaArgs a = make_args(cfg, weights, io);
  const ScanWork w = make_work(make_plan(io->n_tokens, io->n_seqs, !io->offsets), workspace);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return cfg->dtype == CDRGE_F32 ? enqueue_prompt<float>(a, w, s) : enqueue_prompt<uint16_t>(a, w, s);
}

cdrge_status cdrge_delta_step(const cdrge_delta_config* cfg, const cdrge_delta_weights* weights,
                              const cdrge_delta_io* io, void* stream) {
  cdrge_status st = check_config(cfg);
  if (st == CDRGE_OK) st = check_io(cfg, weights, io);
  if (st != CDRGE_OK) return st;
  if (io->offsets || io->n_tokens != io->n_seqs || !io->state_in || !io->positions) return CDRGE_ERR_INVALID_ARG;
  const DeltaArgs a = make_args(cfg, weights, io);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return cfg->dtype == CDRGE_F32 ? enqueue_tokens<float, true>(a, ScanWork{}, s) : enqueue_tokens<uint16_t, true>(a, ScanWork{}, s);
}

}  // extern "C"
