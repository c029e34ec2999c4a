// Host side of cdrge_delta_prompt and cdrge_delta_step (include/cdrge.h).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
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
  bool tokens, long_ones;  // k_delta_tokens, the kernels of blocks
  int short_len;           // as in DeltaArgs
  int kn;       // key_dim as the kernels of blocks have it
  int max_blocks;
  bool direct;  // as in DeltaWork
  bool pair;    // kPair of k_delta_heads
  size_t group_bytes;
  size_t slots, counts, start, bounds, block_of, piece_of, groups, heads, total;
};

// Sequences that are taken token by token. A block of 64 tokens costs the same however few it holds. 32 heads of 128 x 128,
// bf16, 32 tokens: one sequence 24 us and 19 by blocks, 8 of them 45 and 43, 64 244 and 253, 256 916 and 1,038; 40 tokens: 8
// 53 and 43, 64 297 and 262. In float32, where blocks take twice as long, with 256 keys too (32 heads of 128 values): 32 tokens,
// one sequence 32 us and 33, 8 68 and 96, 64 436 and 871. In bf16 with 256 keys 16 tokens: one 30 and 23, 8 48 and 55, 64 362 and
// 413; 24 tokens: 8 68 and 55, 64 507 and 417. The border does not go by the number of sequences: one would be 5 us quicker by
// blocks at it, and many narrow or float32 ones of 33 to 64 tokens token by token (256 sequences of 16 heads of 64 x 64, float32,
// 40 tokens: 211 us so and 635 by blocks; bf16 214 and 326).
int short_len(const cdrge_delta_config* c) { return c->key_dim <= 128 || c->dtype == CDRGE_F32 ? 32 : 16; }

// A ragged batch may hold both kinds, which the host does not see: up to this many tokens a sequence on average either
// path is launched and leaves the other's sequences alone. 255 single tokens beside a prompt of 512 (32 heads of 128 x 128,
// bf16) take 375 us so and 1,044 by blocks alone, beside one of 4,096 888 and 1,734. Lengths that differ less lose by the second
// launch: 64 sequences of 8 heads, 2,000 tokens together, 107 and 78 us, 7,000 168 and 145, 256 with 20,000 429 and 411; 64 with
// 12,000, past the border, 214 and 190.
constexpr int kMixed = 128;

constexpr int kCus = 256;

template <class T>
void block_bytes(int kn, size_t* keys, size_t* head) {
  *keys = kn == 128 ? DeltaBlock<T, 128>::kKeys : DeltaBlock<T, 256>::kKeys;
  *head = kn == 128 ? DeltaBlock<T, 128>::kHeadBytes : DeltaBlock<T, 256>::kHeadBytes;
}

Plan make_plan(const cdrge_delta_config* c, int64_t n_tokens, int32_t n_seqs, bool equal) {
  Plan p{};
  p.short_len = short_len(c);
  const int64_t longest = equal ? n_tokens / n_seqs : n_tokens;
  p.long_ones = longest > p.short_len;
  p.tokens = !p.long_ones || (!equal && n_tokens <= int64_t(kMixed) * n_seqs);
  if (!p.tokens) p.short_len = -1;
  p.kn = c->key_dim <= 128 ? 128 : 256;
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
  if (p.long_ones) {
    size_t keys = 0, head = 0;
    if (c->dtype == CDRGE_F32)
      block_bytes<float>(p.kn, &keys, &head);
    else
      block_bytes<uint16_t>(p.kn, &keys, &head);
    p.pair = (c->dtype == CDRGE_BF16 || p.kn == 128) && int64_t(n_seqs) * c->n_heads * ((c->value_dim + 15) / 16) > kCus;
    p.direct = c->dtype == CDRGE_BF16 && c->key_dim == 128 && !p.pair;
    p.group_bytes = (p.direct ? 1 : 3) * keys;
    p.groups = region(p.group_bytes * c->n_groups * blocks);
    p.heads = region(head * c->n_heads * blocks);
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

template <class T, int kLanes, int kQuads, int kRpt, bool kStep>
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
  hipLaunchKernelGGL((k_delta_tokens<T, kLanes, kQuads, kRpt, kStep>), grid_of(n, 256), dim3(256), 0, s, a, w);
  CDRGE_HIP(hipGetLastError());
  return CDRGE_OK;
}

// Few rows take tiles of 16 rows of the state, more of them tiles of 64, by how many columns of 64 the small tiles hold.
// Single tokens, 32 heads of 128 x 128: one row 6.9 us with small tiles and 7.1 with large ones, 4 rows 8.7 and 7.9, 16 rows
// 19.3 and 14.4; of 256 x 256 2 rows 10.8 and 11.8; of 64 x 64 8 rows 8.1 and 6.8.
template <class T, int kQuads, bool kStep>
cdrge_status launch_tiles(const DeltaArgs& a, const ScanWork& w, hipStream_t s) {
  if (int64_t(a.s.n_seqs) * a.s.H * ((a.s.P + 15) / 16) <= 256 * kQuads) return launch_tokens<T, 16, kQuads, 1, kStep>(a, w, s);
  return launch_tokens<T, 16, kQuads, 4, kStep>(a, w, s);
}

template <class T, bool kStep>
cdrge_status enqueue_tokens(const DeltaArgs& a, const ScanWork& w, hipStream_t s) {
  if (a.s.N <= 16) return launch_tokens<T, 4, 1, 1, kStep>(a, w, s);
  if (a.s.N <= 32) return launch_tokens<T, 8, 1, 2, kStep>(a, w, s);
  if (a.s.N <= 64) return launch_tiles<T, 1, kStep>(a, w, s);
  if (a.s.N <= 128) return launch_tiles<T, 2, kStep>(a, w, s);
  return launch_tiles<T, 4, kStep>(a, w, s);
}

template <class T, int kN>
cdrge_status launch_blocks(DeltaArgs a, const ScanWork& w, const DeltaWork& d, bool pair, hipStream_t s) {
  using Block = DeltaBlock<T, kN>;
  a.s.ptiles = (a.s.P + 15) / 16;
  const int64_t n = int64_t(a.s.n_seqs) * a.s.H * a.s.ptiles;
  a.s.owned = scan_owned(a.s.slots, a.s.n_seqs, n);
  if (a.s.owned) {
    hipLaunchKernelGGL(k_scan_owners, dim3((a.s.n_seqs + 63) / 64), dim3(64 * kScanOwnerWaves), 0, s, a.s, w.slots);
    CDRGE_HIP(hipGetLastError());
  }
  constexpr size_t kLds = 1024 * 4 * (kN / 32) * Block::kRaw + sizeof(float) * 2 * 64 * kDeltaRow;
  if (kLds > 64 * 1024) {
    static std::atomic<uint64_t> ready{0};  // devices on which the kernel may use this much LDS
    int dev = 0;
    CDRGE_HIP(hipGetDevice(&dev));
    if (!(ready.load(std::memory_order_relaxed) >> (dev & 63) & 1)) {
      CDRGE_HIP(hipFuncSetAttribute(reinterpret_cast<const void*>(k_delta_blocks<T, kN>),
                                    hipFuncAttributeMaxDynamicSharedMemorySize, kLds));
      ready.fetch_or(uint64_t(1) << (dev & 63), std::memory_order_relaxed);
    }
  }
  hipLaunchKernelGGL((k_delta_blocks<T, kN>), grid_of(int64_t(w.max_blocks) * a.s.H, 256), dim3(256), kLds, s, a, w, d);
  CDRGE_HIP(hipGetLastError());
  constexpr bool kPair = sizeof(T) == 2 || kN == 128, kDirect = sizeof(T) == 2 && kN == 128;
  if (kPair && pair)
    hipLaunchKernelGGL((k_delta_heads<T, kN, false, kPair>), grid_of(n, 512), dim3(512), 0, s, a, w, d);
  else if (kDirect && d.direct)
    hipLaunchKernelGGL((k_delta_heads<T, kN, kDirect, false>), grid_of(n, 512), dim3(512), 0, s, a, w, d);
  else
    hipLaunchKernelGGL((k_delta_heads<T, kN, false, false>), grid_of(n, 512), dim3(512), 0, s, a, w, d);
  CDRGE_HIP(hipGetLastError());
  return CDRGE_OK;
}

template <class T>
cdrge_status enqueue_prompt(DeltaArgs a, const Plan& p, void* ws, hipStream_t s) {
  a.short_len = p.short_len;
  const ScanWork w = make_work(p, ws);
  if (a.s.offsets) {
    hipLaunchKernelGGL(k_scan_map, dim3(1), dim3(1024), 0, s, a.s, w);
    CDRGE_HIP(hipGetLastError());
  }
  if (p.tokens) {
    const cdrge_status st = enqueue_tokens<T, false>(a, w, s);
    if (st != CDRGE_OK || !p.long_ones) return st;
  }
  const DeltaWork d{static_cast<char*>(ws) + p.groups, static_cast<char*>(ws) + p.heads, static_cast<int64_t>(p.group_bytes), p.direct};
  return p.kn == 128 ? launch_blocks<T, 128>(a, w, d, p.pair, s) : launch_blocks<T, 256>(a, w, d, p.pair, s);
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
  *bytes_out = make_plan(cfg, n_tokens, n_seqs, false).total;
  if (n_tokens % n_seqs == 0) *bytes_out = std::max(*bytes_out, make_plan(cfg, n_tokens, n_seqs, true).total);
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
  const Plan p = make_plan(cfg, io->n_tokens, io->n_seqs, !io->offsets);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return cfg->dtype == CDRGE_F32 ? enqueue_prompt<float>(a, p, workspace, s) : enqueue_prompt<uint16_t>(a, p, workspace, s);
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
