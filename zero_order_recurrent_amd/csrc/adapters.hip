// Host side of cdrge_adapter_project (include/cdrge.h).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>

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

// How a call is cut up. It goes by the sizes alone, so that the workspace is known without pointers.
struct Cut {
  bool few;              // k_adapter_few, which needs no workspace
  bool rows;             // k_adapter_rows (up to 64 rows)
  int side;              // of the tiles of the shared product (k_adapter_tiles)
  int tiles_r, tiles_o, slices, slice_cols;
  int v_slices, v_cols, v_slots;
  bool packed;           // v as operand rows
  int vq_row, o_pad;
  size_t off_partial, total;
};

constexpr int kWorkgroups = 512;  // two for each of 256 compute units

int ceil_div(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

// Cuts n columns into at most `want` slices of a multiple of `unit` columns; returns a slice's columns.
int slice_columns(int n, int want, int unit) { return ceil_div(ceil_div(n, unit), std::max(1, want)) * unit; }

Cut make_cut(const cdrge_adapter_config* c, int64_t n_rows) {
  Cut p{};
  const int K = c->in_features, O = c->out_features;
  const int step = c->dtype == CDRGE_F32 ? 32 : 64;  // columns of 128 bytes
  p.o_pad = (O + 63) / 64 * 64;
  // A row or a few in one launch. Each workgroup repeats the down product (tiles of 16 rows of D), which pays while
  // that is little: one row of rank 16, K x O = 1024 x 4096 6.6 us against 12.7 in two launches, 4096 x 4096 12.6
  // against 17.5, but 5888 x 5888 34 against 26; two rows at 4096 x 1024 15.8 against 13.8. Without adapters, 16 rows
  // at 4096 x 4096 9.9 against 15.5 and at 5888 x 5888 30 against 26; up to four rows 21 against 23 there, and at
  // 512 x 65536, where W's rows are short, 24.6 against 19.4.
  const int tiles = c->n_adapters > 0 ? static_cast<int>(std::min<int64_t>(n_rows, kFewTiles + 1)) * ceil_div(c->max_rank, 16) : 0;
  const int64_t load = int64_t(std::max(tiles, 1)) * K;
  p.few = n_rows <= 16 && tiles <= kFewTiles &&
          ((load <= 4096 && load * O <= (1 << 24)) || (tiles == 0 && n_rows <= 4 && K >= 1024));
  if (p.few) return p;
  p.rows = n_rows <= 64;
  int want;
  if (p.rows) {
    p.tiles_r = 1;
    p.tiles_o = p.o_pad / 64;
    // the down product's workgroups (up to kMostVSlices * 16) take part in the same round
    want = std::max(1, (kWorkgroups - 64) / p.tiles_o);
    // four waves share a slice: at least two steps of 64 bytes each for every wave
    want = std::min(want, ceil_div(K, 4 * step));
  } else {
    // 256 x 256 tiles where they fill the chip (rows x K x O of 8192 x 4096 x 4096 in bf16: 263 us, 330 with 128 x 128;
    // 4096 x 2048 x 3584: 85 against 109); 128 x 128, in slices of at least 8 steps where the tiles alone
    // leave compute units idle; 64 x 64 where K is too short for slices (1279 x 128 x 512: 17 against 27)
    auto tiles = [&](int side) { return int64_t(ceil_div(n_rows, side)) * ceil_div(O, side); };
    p.side = tiles(256) >= 192 ? 256 : (tiles(128) >= 192 || K >= 16 * step ? 128 : 64);
    p.tiles_r = ceil_div(n_rows, p.side);
    p.tiles_o = ceil_div(O, p.side);
    want = p.side != 128 || tiles(128) >= 256 ? 1 : std::min(ceil_div(kWorkgroups, tiles(128)), ceil_div(K, 8 * step));
  }
  p.slice_cols = slice_columns(K, want, p.rows ? 4 * step / 2 : step);
  p.slices = ceil_div(K, p.slice_cols);
  const int v_tiles = ceil_div(n_rows, 64);
  // as many workgroups for the adapters as fill the chip, beside up to 64 rows one for each that they can name
  p.v_slots = std::max(1, std::min({c->n_adapters, p.rows ? static_cast<int>(n_rows) : 16, ceil_div(256, v_tiles)}));
  p.v_cols = slice_columns(K, p.rows || p.slices > 1 ? kMostVSlices : 1, 4 * step);
  p.v_slices = ceil_div(K, p.v_cols);
  p.packed = !p.rows && p.slices == 1;
  p.vq_row = (c->max_rank + 31) / 32 * 32 * (c->dtype == CDRGE_F32 ? 1 : 2);
  const size_t v_row = p.packed ? p.vq_row * (c->dtype == CDRGE_F32 ? 4 : 2) : sizeof(float) * p.v_slices * c->max_rank;
  p.off_partial = c->n_adapters > 0 ? align_up(v_row * static_cast<size_t>(n_rows)) : 0;
  p.total = p.off_partial;
  if (p.rows || p.slices > 1) p.total = align_up(p.total + sizeof(float) * p.slices * static_cast<size_t>(n_rows) * p.o_pad);
  return p;
}

constexpr int64_t kMostBlocks = (int64_t(1) << 31) - 1;

template <class T, int kTiles>
void launch_rows(const AdapterArgs& a, int blocks, hipStream_t s) {
  hipLaunchKernelGGL((k_adapter_rows<T, kTiles>), dim3(blocks), dim3(256), 0, s, a);
}

template <class T, int kSide, int kWavesR, int kWavesO, bool kDirect>
cdrge_status launch_tiles(const AdapterArgs& a, int64_t blocks, hipStream_t s) {
  constexpr size_t kLds = 2 * 2 * kSide * 128;
  const void* f = reinterpret_cast<const void*>(k_adapter_tiles<T, kSide, kSide, kWavesR, kWavesO, kDirect>);
  static std::atomic<uint64_t> ready{0};  // devices on which the kernel may use this much LDS
  int dev = 0;
  CDRGE_HIP(hipGetDevice(&dev));
  if (!(ready.load(std::memory_order_relaxed) >> (dev & 63) & 1)) {
    CDRGE_HIP(hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, kLds));
    ready.fetch_or(uint64_t(1) << (dev & 63), std::memory_order_relaxed);
  }
  hipLaunchKernelGGL((k_adapter_tiles<T, kSide, kSide, kWavesR, kWavesO, kDirect>), 
                     grid_of(blocks, 64 * kWavesR * kWavesO), dim3(64 * kWavesR * kWavesO), kLds, s, a);
  CDRGE_HIP(hipGetLastError());
  return CDRGE_OK;
}

template <class T, bool kDirect>
cdrge_status launch_side(AdapterArgs a, int side, bool low, hipStream_t s) {
  // chunks that pass through registers leave no room for the products of the largest tiles
  if (!kDirect && side == 256) {
    side = 128;
    a.tiles_r = ceil_div(a.n_rows, side);
    a.tiles_o = ceil_div(a.O, side);
  }
  const int64_t down = low && a.slices > 1 ? int64_t(ceil_div(a.n_rows, 64)) * a.v_slices * a.v_slots : 0;
  const int64_t blocks = int64_t(a.tiles_r) * a.tiles_o * a.slices + down;
  if (side == 64) return launch_tiles<T, 64, 4, 1, kDirect>(a, blocks, s);
  if (side == 128) return launch_tiles<T, 128, 2, 2, kDirect>(a, blocks, s);
  if constexpr (kDirect) return launch_tiles<T, 256, 2, 4, true>(a, blocks, s);
  return CDRGE_ERR_UNSUPPORTED;
}

template <class T>
cdrge_status enqueue(const AdapterArgs& a, const Cut& p, hipStream_t s) {
  const bool low = a.row_adapter && a.A > 0;
  if (p.few) {
    const int tiles = low ? static_cast<int>(a.n_rows) * ceil_div(a.R, 16) : 0;
    const dim3 grid(ceil_div(a.O, 16));
    if (tiles == 0)
      hipLaunchKernelGGL((k_adapter_few<T, 0>), grid, dim3(512), 0, s, a);
    else if (tiles == 1)
      hipLaunchKernelGGL((k_adapter_few<T, 1>), grid, dim3(512), 0, s, a);
    else if (tiles == 2)
      hipLaunchKernelGGL((k_adapter_few<T, 2>), grid, dim3(512), 0, s, a);
    else
      hipLaunchKernelGGL((k_adapter_few<T, kFewTiles>), grid, dim3(512), 0, s, a);
    CDRGE_HIP(hipGetLastError());
    return CDRGE_OK;
  }
  if (p.rows) {
    const int blocks = a.tiles_o * a.slices + (low ? a.v_slices * a.v_slots : 0);
    switch ((a.n_rows + 15) / 16) {
      case 1: launch_rows<T, 1>(a, blocks, s); break;
      case 2: launch_rows<T, 2>(a, blocks, s); break;
      case 3: launch_rows<T, 3>(a, blocks, s); break;
      default: launch_rows<T, 4>(a, blocks, s); break;
    }
    CDRGE_HIP(hipGetLastError());
  } else {
    if (low && a.slices == 1) {
      const int64_t blocks = int64_t(ceil_div(a.n_rows, 64)) * a.v_slots;
      hipLaunchKernelGGL(k_adapter_down<T>, grid_of(blocks, 1024), dim3(1024), 0, s, a);
      CDRGE_HIP(hipGetLastError());
    }
    constexpr int kPer = 16 / sizeof(T), kStep = 128 / sizeof(T);
    const bool direct = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && reinterpret_cast<uintptr_t>(a.weight) % 16 == 0 &&
                        a.x_stride % kPer == 0 && a.weight_stride % kPer == 0 && a.K % kStep == 0 &&
                        std::max(a.x_stride, a.weight_stride) <= int64_t(1 << 23) / int64_t(sizeof(T));
    const cdrge_status st = direct ? launch_side<T, true>(a, p.side, low, s) : launch_side<T, false>(a, p.side, low, s);
    if (st != CDRGE_OK || a.slices == 1) return st;
  }
  hipLaunchKernelGGL(k_adapter_finish<T>, dim3(a.o_pad / 64, static_cast<uint32_t>((a.n_rows + 15) / 16)), dim3(256), 0, s, a);
  CDRGE_HIP(hipGetLastError());
  return CDRGE_OK;
}

}  // namespace

extern "C" {

cdrge_status cdrge_adapter_workspace_bytes(const cdrge_adapter_config* cfg, int64_t n_rows, size_t* bytes_out) {
  if (!bytes_out) return CDRGE_ERR_INVALID_ARG;
  const cdrge_status st = check(cfg, n_rows);
  if (st != CDRGE_OK) return st;
  *bytes_out = n_rows > 0 ? make_cut(cfg, n_rows).total : 0;
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
  const Cut p = make_cut(cfg, n_rows);
  if (int64_t(ceil_div(n_rows, 64)) * ceil_div(O, 64) * p.slices > kMostBlocks / 2 ||
      int64_t(ceil_div(n_rows, 64)) * p.v_slices * p.v_slots > kMostBlocks / 2)
    return CDRGE_ERR_UNSUPPORTED;
  if (p.total > 0 && (!ws || workspace_bytes < p.total || reinterpret_cast<uintptr_t>(ws) % kAlign != 0))
    return workspace_error("cdrge_adapter_project", p.total, ws ? workspace_bytes : 0);
  const bool low = row_adapter && cfg->n_adapters > 0;  // vq is set only where there are rows' adapters to read
  float* const vp = static_cast<float*>(ws);
  float* const partial = reinterpret_cast<float*>(static_cast<char*>(ws) + p.off_partial);
  const AdapterArgs a{x, x_stride, weights->weight, weights->weight_stride, weights->bias, weights->down, weights->up,
                      weights->ranks, row_adapter, row_scale, y, y_stride, vp, p.packed && low ? ws : nullptr, p.vq_row, partial, n_rows,
                      K, O, cfg->n_adapters, cfg->max_rank, p.v_slices, p.v_cols, p.v_slots, p.slices, p.slice_cols,
                      p.o_pad, p.tiles_r, p.tiles_o};
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return cfg->dtype == CDRGE_F32 ? enqueue<float>(a, p, s) : enqueue<uint16_t>(a, p, s);
}

}  // extern "C"
