// Host side of cdrge_scan_prompt and cdrge_scan_step (include/cdrge.h).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>

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

bool aligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

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
    // rings are read by element; rows of whole pieces of the state by piece
    const size_t element = c->dtype == CDRGE_F32 ? 4 : 2, piece = c->state_dim % 4 == 0 ? 16 : 4;
    if (!aligned(io->conv_in, element) || !aligned(io->conv_out, element) || !aligned(io->ssm_in, piece) || !aligned(io->ssm_out, piece))
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
  a.owned = false;
  return a;
}

constexpr int64_t kMostBlocks = (int64_t(1) << 31) - 1;

template <class T, int kLanes, int kRpt>
cdrge_status launch_step(ScanArgs a, hipStream_t s) {
  constexpr int kTile = 256 / kLanes * kRpt;
  a.ptiles = (a.P + kTile - 1) / kTile;
  const int64_t n = int64_t(a.n_seqs) * a.H * a.ptiles;
  if (n > kMostBlocks) return CDRGE_ERR_UNSUPPORTED;
  a.owned = scan_owned(a.slots, a.n_seqs, n);
  if (a.owned) {
    hipLaunchKernelGGL(k_scan_mark<T>, dim3((a.n_seqs + 63) / 64), dim3(64 * kScanOwnerWaves), 0, s, a, kTile);
    CDRGE_HIP(hipGetLastError());
  }
  hipLaunchKernelGGL((k_scan_step<T, kLanes, kRpt>), grid_of(n, 256), dim3(256), 0, s, a);
  CDRGE_HIP(hipGetLastError());
  return CDRGE_OK;
}

// Few rows take small tiles: the call's time is then the way of one workgroup, a quarter of the loads long
// (N 128, one row of 16 heads: 6.6 us against 8.8). Past four workgroups a compute unit the convolution of B
// and C, which every tile repeats, costs more (8 x 16 heads 7.7 against 9.3 us, 16 x 16 10.0 against 9.9,
// 64 x 64 95 against 56).
template <class T, int kLanes, int kRpt>
cdrge_status launch_step_tiles(const ScanArgs& a, hipStream_t s) {
  constexpr int kSmall = 256 / kLanes * (kRpt / 4);
  if (int64_t(a.n_seqs) * a.H * ((a.P + kSmall - 1) / kSmall) <= 1024) return launch_step<T, kLanes, kRpt / 4>(a, s);
  return launch_step<T, kLanes, kRpt>(a, s);
}

template <class T>
cdrge_status enqueue_step(const ScanArgs& a, hipStream_t s) {
  if (a.N <= 16) return launch_step<T, 4, 1>(a, s);
  if (a.N <= 32) return launch_step<T, 8, 2>(a, s);
  if (a.N <= 64) return launch_step_tiles<T, 16, 4>(a, s);
  if (a.N <= 128) return launch_step_tiles<T, 32, 8>(a, s);
  return launch_step_tiles<T, 64, 8>(a, s);
}

// How a prompt call is cut up and where its workspace's parts lie; by sizes alone.
struct Plan {
  int kn;  // state_dim as the kernels have it
  int ptiles, max_blocks, max_pieces, piece_blocks;
  size_t blocks, steps, rests, totals, slots, counts, start, bounds, block_of, piece_of, states, fades, total;
};

constexpr int kPieceWorkgroups = 512;  // two for each of 256 compute units

size_t block_bytes(int kn) {
  switch (kn) {
    case 32: return ScanBlock<32>::kBytes;
    case 64: return ScanBlock<64>::kBytes;
    case 128: return ScanBlock<128>::kBytes;
    default: return ScanBlock<256>::kBytes;
  }
}

// Whether a sequence may have more than one piece.
bool cut(const Plan& p, int64_t n_tokens, int32_t n_seqs, bool equal) {
  return scan_blocks_of(equal ? n_tokens / n_seqs : n_tokens) > p.piece_blocks;
}

// equal: every sequence has n_tokens / n_seqs rows.
Plan make_plan(const cdrge_scan_config* c, int64_t n_tokens, int32_t n_seqs, bool equal) {
  Plan p{};
  p.kn = c->state_dim <= 32 ? 32 : (c->state_dim <= 64 ? 64 : (c->state_dim <= 128 ? 128 : 256));
  p.ptiles = (c->head_dim + 63) / 64;
  const int64_t blocks = equal ? int64_t(n_seqs) * scan_blocks_of(n_tokens / n_seqs) : n_tokens / kScanBlock + n_seqs;
  p.max_blocks = static_cast<int>(blocks);
  const int64_t share = blocks * c->n_heads * p.ptiles / kPieceWorkgroups;
  p.piece_blocks = static_cast<int>(std::max<int64_t>(4, share));
  const int64_t pieces = equal ? int64_t(n_seqs) * ((scan_blocks_of(n_tokens / n_seqs) + p.piece_blocks - 1) / p.piece_blocks)
                               : blocks / p.piece_blocks + n_seqs;
  p.max_pieces = static_cast<int>(pieces);
  size_t at = 0;
  auto region = [&](size_t bytes) {
    const size_t here = at;
    at = align_up(at + bytes);
    return here;
  };
  p.blocks = region(block_bytes(p.kn) * blocks * c->n_groups);
  p.steps = region(sizeof(float4) * 64 * blocks * c->n_heads);
  p.rests = region(sizeof(float) * 64 * blocks * c->n_heads);
  p.totals = region(sizeof(float4) * blocks * c->n_heads);
  p.slots = region(sizeof(int32_t) * n_seqs);
  if (!equal) {
    p.counts = region(2 * sizeof(int32_t));
    p.start = region(sizeof(int2) * n_seqs);
    p.bounds = region(sizeof(int2) * n_seqs);
    p.block_of = region(sizeof(int2) * blocks);
    p.piece_of = region(sizeof(int2) * pieces);
  }
  if (cut(p, n_tokens, n_seqs, equal)) {
    p.states = region(sizeof(float) * 64 * p.kn * p.ptiles * c->n_heads * pieces);
    p.fades = region(sizeof(float) * c->n_heads * pieces);
  }
  p.total = at;
  return p;
}

ScanWork make_work(const Plan& p, void* ws) {
  char* const at = static_cast<char*>(ws);
  ScanWork w;
  w.blocks = at + p.blocks;
  w.steps = reinterpret_cast<float4*>(at + p.steps);
  w.rests = reinterpret_cast<float*>(at + p.rests);
  w.totals = reinterpret_cast<float4*>(at + p.totals);
  w.slots = reinterpret_cast<int32_t*>(at + p.slots);
  w.counts = reinterpret_cast<int32_t*>(at + p.counts);
  w.start = reinterpret_cast<int2*>(at + p.start);
  w.bounds = reinterpret_cast<int2*>(at + p.bounds);
  w.block_of = reinterpret_cast<int2*>(at + p.block_of);
  w.piece_of = reinterpret_cast<int2*>(at + p.piece_of);
  w.states = reinterpret_cast<float*>(at + p.states);
  w.fades = reinterpret_cast<float*>(at + p.fades);
  w.piece_blocks = p.piece_blocks;
  w.max_blocks = p.max_blocks;
  w.max_pieces = p.max_pieces;
  return w;
}

template <class T, int kN>
cdrge_status launch_prompt(ScanArgs a, const Plan& p, const ScanWork& w, bool pieces, hipStream_t s) {
  a.ptiles = p.ptiles;
  if (a.offsets) {
    hipLaunchKernelGGL(k_scan_map, dim3(1), dim3(1024), 0, s, a, w);
    CDRGE_HIP(hipGetLastError());
  }
  a.owned = scan_owned(a.slots, a.n_seqs, int64_t(p.max_blocks) * a.G);
  if (a.owned) {
    hipLaunchKernelGGL(k_scan_owners, dim3((a.n_seqs + 63) / 64), dim3(64 * kScanOwnerWaves), 0, s, a, w.slots);
    CDRGE_HIP(hipGetLastError());
  }
  constexpr size_t kLds = sizeof(float) * kScanBlock * (2 * kN + 2);
  if (kLds > 64 * 1024) {
    static std::atomic<uint64_t> ready{0};  // devices on which the kernel may use this much LDS
    int dev = 0;
    CDRGE_HIP(hipGetDevice(&dev));
    if (!(ready.load(std::memory_order_relaxed) >> (dev & 63) & 1)) {
      CDRGE_HIP(hipFuncSetAttribute(reinterpret_cast<const void*>(k_scan_blocks<T, kN>),
                                    hipFuncAttributeMaxDynamicSharedMemorySize, kLds));
      ready.fetch_or(uint64_t(1) << (dev & 63), std::memory_order_relaxed);
    }
  }
  const int parts = 1 + (a.H / a.G + 8 * kScanHeads - 1) / (8 * kScanHeads);
  hipLaunchKernelGGL((k_scan_blocks<T, kN>), grid_of(int64_t(p.max_blocks) * a.G * parts, 512), dim3(512), kLds, s, a, w, parts);
  CDRGE_HIP(hipGetLastError());
  const dim3 grid = grid_of(int64_t(p.max_pieces) * a.H * p.ptiles, 256);
  if (pieces) {
    hipLaunchKernelGGL((k_scan_heads<T, kN, true>), grid, dim3(256), 0, s, a, w);
    CDRGE_HIP(hipGetLastError());
  }
  hipLaunchKernelGGL((k_scan_heads<T, kN, false>), grid, dim3(256), 0, s, a, w);
  CDRGE_HIP(hipGetLastError());
  if (a.conv_in) {
    const int cblocks = (a.C + 255) / 256;
    hipLaunchKernelGGL(k_scan_ring<T>, grid_of(int64_t(a.n_seqs) * cblocks, 256), dim3(256), 0, s, a, w, cblocks);
    CDRGE_HIP(hipGetLastError());
  }
  return CDRGE_OK;
}

template <class T>
cdrge_status enqueue_prompt(const ScanArgs& a, const Plan& p, const ScanWork& w, bool pieces, hipStream_t s) {
  switch (p.kn) {
    case 32: return launch_prompt<T, 32>(a, p, w, pieces, s);
    case 64: return launch_prompt<T, 64>(a, p, w, pieces, s);
    case 128: return launch_prompt<T, 128>(a, p, w, pieces, s);
    default: return launch_prompt<T, 256>(a, p, w, pieces, s);
  }
}

template <class T, int kN>
cdrge_status launch_short(ScanArgs a, hipStream_t s) {
  a.ptiles = (a.P + 63) / 64;
  const int parts = (a.H / a.G * a.ptiles + kScanUnits - 1) / kScanUnits;
  hipLaunchKernelGGL((k_scan_short<T, kN>), grid_of(int64_t(a.n_seqs) * a.G * parts, 256), dim3(256), 0, s, a, parts);
  CDRGE_HIP(hipGetLastError());
  return CDRGE_OK;
}

template <class T>
cdrge_status enqueue_short(const ScanArgs& a, hipStream_t s) {
  if (a.N <= 32) return launch_short<T, 32>(a, s);
  if (a.N <= 64) return launch_short<T, 64>(a, s);
  if (a.N <= 128) return launch_short<T, 128>(a, s);
  return launch_short<T, 256>(a, s);
}

// Whether the call's sizes fit the kernels' 32-bit counts.
bool fits(const cdrge_scan_config* c, int64_t n_tokens, int32_t n_seqs) {
  const int64_t blocks = n_tokens / kScanBlock + n_seqs, ptiles = (c->head_dim + 63) / 64;
  return n_tokens <= (int64_t(1) << 30) && n_seqs <= (1 << 20) && blocks * c->n_heads * (ptiles + 1) <= kMostBlocks &&
         int64_t(n_seqs) * ((channels(c) + 255) / 256) <= kMostBlocks;
}

}  // namespace

extern "C" {

cdrge_status cdrge_scan_workspace_bytes(const cdrge_scan_config* cfg, int64_t n_tokens, int32_t n_seqs,
                                        size_t* bytes_out) {
  if (!bytes_out || n_tokens < 0 || n_seqs < 1) return CDRGE_ERR_INVALID_ARG;
  const cdrge_status st = check_config(cfg);
  if (st != CDRGE_OK) return st;
  if (!fits(cfg, n_tokens, n_seqs)) return CDRGE_ERR_UNSUPPORTED;
  // ragged sequences may take more blocks than equal ones, equal ones more pieces
  *bytes_out = make_plan(cfg, n_tokens, n_seqs, false).total;
  if (n_tokens % n_seqs == 0) *bytes_out = std::max(*bytes_out, make_plan(cfg, n_tokens, n_seqs, true).total);
  return CDRGE_OK;
}

cdrge_status cdrge_scan_prompt(const cdrge_scan_config* cfg, const cdrge_scan_weights* weights,
                               const cdrge_scan_io* io, void* workspace, size_t workspace_bytes, void* stream) {
  cdrge_status st = check_config(cfg);
  if (st == CDRGE_OK) st = check_io(cfg, weights, io);
  if (st != CDRGE_OK) return st;
  if (!fits(cfg, io->n_tokens, io->n_seqs)) return CDRGE_ERR_UNSUPPORTED;
  const bool equal = !io->offsets;
  const ScanArgs a = make_args(cfg, weights, io);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (equal && !io->ssm_in && io->n_tokens > 0 && io->n_tokens / io->n_seqs <= kScanShort)
    return cfg->dtype == CDRGE_F32 ? enqueue_short<float>(a, s) : enqueue_short<uint16_t>(a, s);
  size_t need = 0;
  st = cdrge_scan_workspace_bytes(cfg, io->n_tokens, io->n_seqs, &need);
  if (st != CDRGE_OK) return st;
  if (!workspace || workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % kAlign != 0)
    return workspace_error("cdrge_scan_prompt", need, workspace ? workspace_bytes : 0);
  const Plan p = make_plan(cfg, io->n_tokens, io->n_seqs, equal);
  const ScanWork w = make_work(p, workspace);
  const bool pieces = cut(p, io->n_tokens, io->n_seqs, equal);
  return cfg->dtype == CDRGE_F32 ? enqueue_prompt<float>(a, p, w, pieces, s) : enqueue_prompt<uint16_t>(a, p, w, pieces, s);
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
