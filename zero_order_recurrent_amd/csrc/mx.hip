// Host side of cdrge_mx_quantize, cdrge_mx_dequantize and cdrge_mx_project (include/cdrge.h).
#include <hip/hip_runtime.h>

#include <atomic>

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

// Workgroups of the kernels that take a quarter of a block a thread; parts: as in mx_place.
int64_t quarter_groups(int64_t n_rows, int quarters, int* parts) {
  *parts = (quarters + 255) / 256;
  const int each = *parts > 1 ? 1 : 256 / quarters;
  return (n_rows + each - 1) / each * *parts;
}

constexpr int64_t kMostGroups = int64_t(1) << 35;  // 2^20 by 2^15 of a grid

// kMxSteps: with the weights' scales (w_scales to w_tiled) in the same launch
template <class T, int kLayout>
cdrge_status quantize(const cdrge_mx_config* c, int64_t n_rows, const void* x, int64_t stride, uint8_t* codes,
                      uint8_t* scales, const uint8_t* w_scales, uint8_t* w_tiled, hipStream_t s) {
  constexpr int kStep = kLayout == kMxSteps ? 8 : kLayout == kMxOperands ? 4 : 1;  // blocks
  int parts = 1;
  const int blocks = blocks_of(c), steps = (blocks + kStep - 1) / kStep, quarters = 4 * kStep * steps;
  const int64_t n = quarter_groups(n_rows, quarters, &parts);
  const int64_t first = kLayout == kMxSteps ? (int64_t(c->out_features) * steps + 255) / 256 : 0;
  if (n + first > kMostGroups) return CDRGE_ERR_UNSUPPORTED;
  if (n == 0) return CDRGE_OK;
  hipLaunchKernelGGL((k_mx_quantize<T, kLayout>), grid_of(n + first, 256), dim3(256), 0, s, static_cast<const T*>(x), stride, n_rows,
                     c->in_features, quarters, parts, codes, scales, static_cast<int>(first), w_scales, c->out_features, blocks,
                     w_tiled);
  CDRGE_HIP(hipGetLastError());
  return CDRGE_OK;
}

// How a call is cut up and where its workspace's parts lie; by sizes alone.
struct Plan {
  int side;    // of the tiles of k_mx_tiles; 0: k_mx_rows
  bool fused;  // which quantises the rows itself, without a workspace
  int blocks, steps, tiles_r, tiles_o;
  size_t codes, scales, w_scales, total;
};

// Up to four rows are quantised by every workgroup of k_mx_rows, which saves a launch, where their codes fit in 34 KB:
// 4096 -> 4096, one row 7.1 us and 10.2 with a launch for it, four 8.5 and 10.2, eight 10.3 both; 16384 -> 4096, one row
// 14.8 and 17.6, four (2,048 blocks) 21.3 and 17.6.
constexpr int kFusedBlocks = 2000;

Plan make_plan(const cdrge_mx_config* c, int64_t n_rows) {
  Plan p{};
  p.blocks = blocks_of(c);
  p.steps = (p.blocks + 7) / 8;
  const int64_t r128 = (n_rows + 127) / 128, o128 = (c->out_features + 127) / 128;
  // k_mx_rows takes up to 64 rows, whose codes every one of its workgroups reads, for 16 outputs: 64 rows, 4096 -> 4096, 11 us,
  // and 21 by tiles, which are too few to fill the chip. With outputs for 256 tiles these are quicker: 4096 -> 32768, 17 rows
  // 25 us by tiles and 28 by rows, 64 rows 26 and 37; -> 16384, 64 rows 23 both. Large tiles read half as much, but leave
  // CUs idle below 256 of them: 8192 rows, 4096 -> 4096, 101 us and 112 with small ones, 2048 rows 45 and 34.
  p.fused = n_rows <= 4 && n_rows * p.blocks <= kFusedBlocks;
  if (n_rows > 64 || (n_rows > 16 && o128 >= 256)) p.side = r128 * o128 >= 1024 ? 256 : 128;
  if (p.side > 0) {
    p.tiles_r = static_cast<int>((n_rows + p.side - 1) / p.side);
    p.tiles_o = (c->out_features + p.side - 1) / p.side;
  }
  // blocks of the rows: k_mx_tiles has whole steps of 8, k_mx_rows of 4 and tiles of 16 rows
  const size_t blocks = p.side > 0 ? size_t(8) * p.steps * n_rows : size_t((p.blocks + 3) / 4 * 4) * ((n_rows + 15) / 16 * 16);
  p.scales = align_up(16 * blocks);
  p.w_scales = align_up(p.scales + blocks);
  p.total = p.fused ? 0 : p.side > 0 ? align_up(p.w_scales + size_t(8) * p.steps * c->out_features) : p.w_scales;
  return p;
}

// Whether the call's sizes fit the kernels' counts.
bool fits(const cdrge_mx_config* c, int64_t n_rows) {
  return (n_rows + 127) / 128 * ((c->out_features + 127) / 128) < (int64_t(1) << 31);
}

template <class T, int kSide>
cdrge_status launch_tiles(const MxTileArgs& a, hipStream_t s) {
  constexpr size_t kLds = size_t(2) * 2 * kSide * 128;
  static std::atomic<uint64_t> ready{0};  // devices on which the kernel may use this much LDS
  int dev = 0;
  CDRGE_HIP(hipGetDevice(&dev));
  if (!(ready.load(std::memory_order_relaxed) >> (dev & 63) & 1)) {
    CDRGE_HIP(hipFuncSetAttribute(reinterpret_cast<const void*>(k_mx_tiles<T, kSide>), hipFuncAttributeMaxDynamicSharedMemorySize, kLds));
    ready.fetch_or(uint64_t(1) << (dev & 63), std::memory_order_relaxed);
  }
  hipLaunchKernelGGL((k_mx_tiles<T, kSide>), grid_of(int64_t(a.tiles_r) * a.tiles_o, 2 * kSide), dim3(2 * kSide), kLds, s, a);
  CDRGE_HIP(hipGetLastError());
  return CDRGE_OK;
}

template <class T, int kTiles, bool kFused>
cdrge_status launch_rows(const MxArgs& a, hipStream_t s) {
  const size_t lds = kFused ? size_t(68) * a.n_rows * ((a.blocks + 3) / 4) : 0;
  hipLaunchKernelGGL((k_mx_rows<T, kTiles, kFused>), grid_of((a.O + 15) / 16, 512), dim3(512), lds, s, a);
  CDRGE_HIP(hipGetLastError());
  return CDRGE_OK;
}

template <class T>
cdrge_status project(const cdrge_mx_config* c, const uint8_t* w_codes, const uint8_t* w_scales, const void* bias, int64_t n_rows,
                     const void* x, int64_t x_stride, void* y, int64_t y_stride, const Plan& p, void* workspace, hipStream_t s) {
  uint8_t* const codes = static_cast<uint8_t*>(workspace) + p.codes;
  uint8_t* const scales = static_cast<uint8_t*>(workspace) + p.scales;
  uint8_t* const w_tiled = static_cast<uint8_t*>(workspace) + p.w_scales;
  const MxArgs a{w_codes, w_scales, bias, x, x_stride, codes, scales, y, y_stride, n_rows, c->in_features, c->out_features, p.blocks};
  if (p.fused) return launch_rows<T, 1, true>(a, s);
  if (p.side > 0) {
    const cdrge_status st = quantize<T, kMxSteps>(c, n_rows, x, x_stride, codes, scales, w_scales, w_tiled, s);
    if (st != CDRGE_OK) return st;
    const MxTileArgs t{w_codes, w_tiled, codes, scales, bias, y, y_stride, n_rows, c->out_features, p.blocks, p.steps, p.tiles_r, p.tiles_o};
    return p.side == 256 ? launch_tiles<T, 256>(t, s) : launch_tiles<T, 128>(t, s);
  }
  const cdrge_status st = quantize<T, kMxOperands>(c, n_rows, x, x_stride, codes, scales, nullptr, nullptr, s);
  if (st != CDRGE_OK) return st;
  if (n_rows <= 16) return launch_rows<T, 1, false>(a, s);
  if (n_rows <= 32) return launch_rows<T, 2, false>(a, s);
  return n_rows <= 48 ? launch_rows<T, 3, false>(a, s) : launch_rows<T, 4, false>(a, s);
}

}  // namespace

extern "C" {

cdrge_status cdrge_mx_quantize(const cdrge_mx_config* cfg, int64_t n_rows, const void* x, int64_t x_stride,
                               uint8_t* codes, uint8_t* scales, void* stream) {
  const cdrge_status st = check_rows(cfg, n_rows, x, x_stride, codes, scales);
  if (st != CDRGE_OK) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return cfg->dtype == CDRGE_F32 ? quantize<float, kMxRows>(cfg, n_rows, x, x_stride, codes, scales, nullptr, nullptr, s)
                                 : quantize<uint16_t, kMxRows>(cfg, n_rows, x, x_stride, codes, scales, nullptr, nullptr, s);
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
  if (!fits(cfg, n_rows)) return CDRGE_ERR_UNSUPPORTED;
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
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, kAlign)))
    return workspace_error("cdrge_mx_project", need, workspace ? workspace_bytes : 0);
  const Plan p = make_plan(cfg, n_rows);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return cfg->dtype == CDRGE_F32
             ? project<float>(cfg, w_codes, w_scales, bias, n_rows, x, x_stride, y, y_stride, p, workspace, s)
             : project<uint16_t>(cfg, w_codes, w_scales, bias, n_rows, x, x_stride, y, y_stride, p, workspace, s);
}

}  // extern "C"
