// Microscaled 4-bit floating point: quantisation, the values back, and the product of quantised rows with quantised
// weights (E2M1 elements, a power of two for each 32 of them along the reduction).
#pragma once
#include <type_traits>

#include "operators_common.h"

namespace cdrge {

typedef __attribute__((ext_vector_type(8))) int i32x8;
typedef __attribute__((ext_vector_type(4))) int i32x4;

// 16 x 16 x 128 of 4-bit operands: lane l holds row (column) l % 16 of A (B), the block of 32 values l / 16, 16 bytes,
// and that block's scale byte; of the result column l % 16 and rows 4 (l / 16) + 0..3.
__device__ __forceinline__ f32x4 mma_mx(i32x4 a, int ea, i32x4 b, int eb, f32x4 c) {
  const i32x8 wa = {a[0], a[1], a[2], a[3], 0, 0, 0, 0}, wb = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wa, wb, c, 4, 4, 0, ea, 0, eb);
}

// Eight elements of a row from column c on; zeros past its end. kOnce: past the caches.
template <class T>
struct MxQuarter {
  T e[8];
  template <bool kOnce>
  __device__ __forceinline__ void load(const T* row, int c, int K) {
    if (c + 8 <= K) {
      if (kOnce)
        load_once(e, row + c);
      else
        __builtin_memcpy(e, row + c, sizeof(e));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = c + i < K ? row[c + i] : T(0);
    }
  }
};

// The scale byte of a block from its largest magnitude's bits, which are those of a NaN if it has one.
__device__ __forceinline__ int mx_scale(uint32_t most) {
  const int e = static_cast<int>(most >> 23);
  return e == 255 ? 255 : max(e - 2, 0);
}

// Eight values as codes. Scaling by a power of two is exact, or leaves less than the smallest code's half.
__device__ __forceinline__ uint32_t mx_codes(const float (&v)[8], int scale) {
  if (scale == 255) return 0;
  const float f = __uint_as_float(static_cast<uint32_t>(254 - scale) << 23);  // mx_scale is at most 252 else
  uint32_t w = 0;
  float m[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) m[i] = fminf(fmaxf(v[i] * f, -6.f), 6.f);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, m[0], m[1], 1.f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, m[2], m[3], 1.f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, m[4], m[5], 1.f, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, m[6], m[7], 1.f, 3);
}

// The largest of the four lanes of a block.
__device__ __forceinline__ uint32_t quad_most(uint32_t v) {
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0xb1, 0xf, 0xf, false)));
  return max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x4e, 0xf, 0xf, false)));
}

// Where a thread of k_mx_quantize and k_mx_dequantize works: a quarter of a block, `quarters` to a row; `parts` groups of
// 256 threads take a row, or rows lie side by side in a group where they are short.
struct MxPlace {
  int64_t row;
  int quarter;
};
__device__ __forceinline__ MxPlace mx_place(int64_t group, int quarters, int parts) {
  if (parts > 1) {
    const int64_t row = group >> 32 ? group / parts : static_cast<uint32_t>(group) / static_cast<uint32_t>(parts);
    return {row, static_cast<int>(group - row * parts) * 256 + static_cast<int>(threadIdx.x)};
  }
  const int each = 256 / quarters;  // rows of a group
  const int r = threadIdx.x / quarters;
  return {r < each ? group * each + r : (int64_t(1) << 62), static_cast<int>(threadIdx.x) % quarters};
}

// Where the codes and scales of a row go. kMxSteps, for k_mx_tiles: steps of 8 blocks (zeros past K), [step][row][8]; the
// first workgroups lay out the weights' scales in the same way, the last block's in the place of those past it (which meet
// zeros). kMxOperands, for k_mx_rows: steps of 4 blocks (zeros past K), [step][tile of 16 rows][lane], the places past the
// last row left as they are (their products are dropped).
enum MxLayout { kMxRows, kMxSteps, kMxOperands };
template <int kLayout>
__device__ __forceinline__ int64_t mx_at(int64_t row, int64_t n_rows, int block, int blocks) {  // a block's place
  if (kLayout == kMxSteps) return ((block / 8) * n_rows + row) * 8 + block % 8;
  if (kLayout == kMxOperands) return ((block / 4) * ((n_rows + 15) / 16) + row / 16) * 64 + row % 16 + 16 * (block % 4);
  return row * blocks + block;
}

// A quarter of a block a thread, the block's largest magnitude by two lane permutations. Bound by reading x: 8192 x 4096 bf16
// with back again 40 us, 4.2 TB/s; the rows of a product in the layout of kMxSteps 20 us. Two quarters a thread: the same.
template <class T, int kLayout>
__global__ __launch_bounds__(256) void k_mx_quantize(const T* __restrict__ x, int64_t stride, int64_t n_rows, int K, int quarters,
                                                     int parts, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                                                     int first, const uint8_t* __restrict__ w_scales, int O, int blocks,
                                                     uint8_t* __restrict__ w_tiled) {
  const int64_t block = block_number() - first;
  if (kLayout == kMxSteps && block < 0) {
    const int steps = (blocks + 7) / 8;
    const uint32_t id = static_cast<uint32_t>(block_number()) * 256 + threadIdx.x;
    const int o = id / steps, step = id % steps;
    if (o >= O) return;
    const uint8_t* const from = w_scales + static_cast<int64_t>(o) * blocks + 8 * step;
    uint8_t v[8];
    if (8 * step + 8 <= blocks) {
      __builtin_memcpy(v, from, 8);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = from[min(i, blocks - 1 - 8 * step)];
    }
    __builtin_memcpy(w_tiled + (static_cast<int64_t>(step) * O + o) * 8, v, 8);
    return;
  }
  const MxPlace at = mx_place(block, quarters, parts);
  if (at.row >= n_rows || at.quarter >= quarters) return;  // whole blocks
  MxQuarter<T> raw;
  raw.template load<true>(x + at.row * stride, at.quarter * 8, K);
  float v[8];
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = to_float(raw.e[i]);
    most = max(most, __float_as_uint(v[i]) & 0x7fffffffu);
  }
  const int e = mx_scale(quad_most(most));
  const int64_t to = mx_at<kLayout>(at.row, n_rows, at.quarter / 4, quarters / 4);
  reinterpret_cast<uint32_t*>(codes)[to * 4 + at.quarter % 4] = mx_codes(v, e);
  if (at.quarter % 4 == 0) scales[to] = static_cast<uint8_t>(e);
}

// The value of a code with the scale byte e.
__device__ __forceinline__ float mx_value(uint32_t code, int e) {
  const uint32_t m = code & 7;
  const float size = m < 2 ? 0.5f * m : __uint_as_float(((m >> 1) + 126) << 23 | (m & 1) << 22);
  return e == 255 ? __builtin_nanf("") : ldexpf(code & 8 ? -size : size, e - 127);
}

// A quarter of a block a thread. Bound by writing x: 8192 x 4096 bf16 22 us, 3.8 TB/s with the codes; 5887 x 4099 float32 29.
template <class T>
__global__ __launch_bounds__(256) void k_mx_dequantize(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                       int64_t n_rows, int K, int quarters, int parts, T* __restrict__ x, int64_t stride) {
  const MxPlace at = mx_place(block_number(), quarters, parts);
  if (at.row >= n_rows || at.quarter >= quarters) return;
  const uint32_t w = reinterpret_cast<const uint32_t*>(codes)[at.row * quarters + at.quarter];
  const int e = scales[(at.row * quarters + at.quarter) / 4], c = at.quarter * 8;
  T v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = from_float<T>(mx_value(w >> (4 * i) & 15, e));
  T* const to = x + at.row * stride + c;
  if (c + 8 <= K) {
    __builtin_memcpy(to, v, sizeof(v));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < K) to[i] = v[i];
  }
}

struct MxArgs {
  const uint8_t* w_codes;
  const uint8_t* w_scales;
  const void* bias;
  const void* x;  // the rows themselves, for kFused, and otherwise their codes and scales as kMxOperands
  int64_t x_stride;
  const uint8_t* x_codes;
  const uint8_t* x_scales;
  void* y;
  int64_t y_stride;
  int64_t n_rows;
  int K, O, blocks;  // blocks of 32 along the reduction
};

// 16 outputs of up to 16 kTiles rows by a workgroup of eight waves, which share the reduction; each wave's sums are joined
// in their order. Bound by reading W, with a request a wave in flight: 32768 x 4096, one row 20.5 us (3.5 TB/s), 16 rows 25;
// with few outputs by the launches and the loads' latency: 4096 x 4096, one row 7.0 us, 64 rows 11. Requests of two or three
// steps at a time: one row 7.6, 64 rows 12.9. kFused: every workgroup quantises the rows itself, into LDS, while its first
// weights are on their way.
template <class T, int kTiles, bool kFused>
__global__ __launch_bounds__(512) void k_mx_rows(MxArgs a) {
  __shared__ f32x4 sums[8][kTiles][64];
  extern __shared__ __align__(16) uint8_t rows[];  // kFused: codes [row][steps][4][16], then scales [row][steps][4]
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l16 = lane & 15, q = lane >> 4;
  const int o0 = static_cast<int>(block_number()) * 16;
  if (o0 >= a.O) return;
  const int steps = (a.blocks + 3) / 4, each = (steps + 7) / 8, end = min(steps, wave * each + each), n_rows = static_cast<int>(a.n_rows);
  const int64_t wrow = static_cast<int64_t>(min(o0 + l16, a.O - 1)) * a.blocks;
  f32x4 acc[kTiles] = {};
  i32x4 w, x[kTiles];
  int we, xe[kTiles];
  auto request_w = [&](int s) {
    // past the last block: the last one's weights, which meet zeros
    const int at = min(4 * min(s, steps - 1) + q, a.blocks - 1);
    w = *reinterpret_cast<const i32x4*>(a.w_codes + (wrow + at) * 16);
    we = a.w_scales[wrow + at];
  };
  auto request_x = [&](int s) {
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      if (kFused) {
        const int from = (min(l16, n_rows - 1) * steps + s) * 4 + q;
        x[t] = reinterpret_cast<const i32x4*>(rows)[from];
        xe[t] = rows[n_rows * steps * 64 + from];
      } else {
        const uint32_t from = (s * static_cast<uint32_t>((n_rows + 15) / 16) + t) * 64 + lane;
        x[t] = reinterpret_cast<const i32x4*>(a.x_codes)[from];
        xe[t] = a.x_scales[from];
      }
    }
  };
  int s = wave * each;
  request_w(s);
  if (kFused) {
    const int quarters = 16 * steps;
    for (int i = tid; i < n_rows * quarters; i += 512) {
      const int row = i / quarters;
      MxQuarter<T> raw;
      raw.template load<false>(static_cast<const T*>(a.x) + row * a.x_stride, (i - row * quarters) * 8, a.K);
      float v[8];
      uint32_t most = 0;
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        v[n] = to_float(raw.e[n]);
        most = max(most, __float_as_uint(v[n]) & 0x7fffffffu);
      }
      const int e = mx_scale(quad_most(most));
      reinterpret_cast<uint32_t*>(rows)[i] = mx_codes(v, e);
      if (i % 4 == 0) rows[n_rows * steps * 64 + i / 4] = static_cast<uint8_t>(e);
    }
    __syncthreads();
  }
  for (; s < end; ++s) {
    request_x(s);
#pragma unroll
    for (int t = 0; t < kTiles; ++t) acc[t] = mma_mx(w, we, x[t], xe[t], acc[t]);
    if (s + 1 < end) request_w(s + 1);
  }
#pragma unroll
  for (int t = 0; t < kTiles; ++t) sums[wave][t][lane] = acc[t];
  __syncthreads();
  if (wave >= kTiles) return;
  f32x4 sum = sums[0][wave][lane];
#pragma unroll
  for (int v = 1; v < 8; ++v) sum += sums[v][wave][lane];
  const int row = 16 * wave + l16;
  if (row >= a.n_rows) return;
  T* const y = static_cast<T*>(a.y) + row * a.y_stride;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int o = o0 + 4 * q + e;
    if (o < a.O) y[o] = from_float<T>(sum[e] + (a.bias ? to_float(static_cast<const T*>(a.bias)[o]) : 0.f));
  }
}

// ---------------------------------------------------------------------------------------------
// Many rows: tiles of kSide x kSide outputs, a wave 64 outputs by kSide / 2 rows of them, in products of 32 x 32 x 64. A
// step is 256 values (128 bytes) of each row, in two buffers of LDS that are loaded without passing through registers, the
// next step's while this one's products run. Rows lie there as eight chunks of 16 bytes, chunk c of row i at place c ^ f(i)
// (mx_place_of), so that the eight rows that a read touches at a time take all eight.
// The order along the reduction is free: lane group h of a wave takes the step's blocks 4 h .. 4 h + 3, whose scales are
// one word. Outputs lie along the lanes, so that a store fills 64 bytes of a row (bf16); with rows along the lanes and 16
// bytes of each a store the products below took 48 us more.
// 8192 x 4096 -> 4096, bf16: 80 us, 3.4 PFLOP/s, where 4-bit products with nothing else reach 6.5 to 7.5. What is left is the
// start and end of each of two rounds of tiles, in which no products run, and the stores (67 MB, 14 us at the memory's rate).
// ---------------------------------------------------------------------------------------------
typedef __attribute__((ext_vector_type(16))) float f32x16;

struct MxTileArgs {
  const uint8_t* w_codes;  // [O][blocks][16]
  const uint8_t* w_scales;  // [step][O][8]
  const uint8_t* x_codes;  // [step][row][8][16]
  const uint8_t* x_scales;  // [step][row][8]
  const void* bias;
  void* y;
  int64_t y_stride;
  int64_t n_rows;
  int O, blocks, steps, tiles_r, tiles_o;
};

__device__ __forceinline__ int mx_place_of(int row) { return row & 7; }

template <class T, int kSide>
__global__ __launch_bounds__(kSide * 2, 2) void k_mx_tiles(MxTileArgs a) {
  constexpr int kThreads = kSide * 2, kRT = kSide / 64;  // row tiles of a wave
  constexpr int kLoads = kSide * 8 / kThreads;           // chunks of either operand that a thread loads a step
  constexpr int kBuf = 2 * kSide * 8;
  extern __shared__ uint4 stage[];  // [2][kBuf]: W's rows, then x's
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l32 = lane & 31, half = lane >> 5;
  const int wo = wave >> 1, wr = wave & 1;

  // Workgroups go round the eight XCDs, each of which has its own L2: XCD i gets the i-th eighth of the tiles, walked in
  // columns of up to four row tiles.
  const int n_tiles = a.tiles_r * a.tiles_o;
  uint32_t id = static_cast<uint32_t>(block_number());
  if (id >= static_cast<uint32_t>(n_tiles)) return;
  {
    const uint32_t per = n_tiles >> 3, left = n_tiles & 7, xcd = id & 7;
    id = xcd * per + min(xcd, left) + (id >> 3);
  }
  const int band = id / (4 * a.tiles_o), in_band = id % (4 * a.tiles_o);
  const int band_rows = min(4, a.tiles_r - 4 * band);
  const int64_t r0 = static_cast<int64_t>(4 * band + in_band % band_rows) * kSide;
  const int o0 = in_band / band_rows * kSide;
  const int last_r = static_cast<int>(a.n_rows - r0 < kSide ? a.n_rows - r0 : kSide) - 1, last_o = min(kSide, a.O - o0) - 1;

  // load i of a thread: place tid % 8 of row tid / 8 + i kThreads / 8; rows past the last are read from it
  const char* const wb = reinterpret_cast<const char*>(a.w_codes) + static_cast<int64_t>(o0) * a.blocks * 16;
  const char* const xb = reinterpret_cast<const char*>(a.x_codes) + r0 * 128;
  const int c = (tid & 7) ^ mx_place_of(tid >> 3);
  uint32_t w_at[kLoads], x_at[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int row = (tid >> 3) + i * (kThreads / 8);
    w_at[i] = (min(row, last_o) * a.blocks + c) * 16;
    x_at[i] = min(row, last_r) * 128 + c * 16;
  }
  auto fetch = [&](int step, int buf) {
    uint4* const to = stage + buf * kBuf + wave * 64;
    if (8 * step + 8 <= a.blocks) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) load_to_lds(wb + step * 128, w_at[i], to + i * kThreads);
    } else {
      // W's blocks past the last meet zeros of x: the last one is read in their place
      const int more = (min(8 * step + c, a.blocks - 1) - c) * 16;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) load_to_lds(wb, w_at[i] + more, to + i * kThreads);
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) load_to_lds(xb + step * a.n_rows * 128, x_at[i], to + kSide * 8 + i * kThreads);
  };
  int ew[2], ex[kRT], ew_next[2], ex_next[kRT];
  uint32_t ew_at[2], ex_at[kRT];
#pragma unroll
  for (int t = 0; t < 2; ++t) ew_at[t] = min(wo * 64 + 32 * t + l32, last_o) * 8 + 4 * half;
#pragma unroll
  for (int t = 0; t < kRT; ++t) ex_at[t] = min(wr * (kSide / 2) + 32 * t + l32, last_r) * 8 + 4 * half;
  auto fetch_scales = [&](int step) {
    const uint8_t* const w = a.w_scales + (static_cast<int64_t>(step) * a.O + o0) * 8;
    const uint8_t* const x = a.x_scales + (step * a.n_rows + r0) * 8;
#pragma unroll
    for (int t = 0; t < 2; ++t) ew_next[t] = *reinterpret_cast<const int*>(w + ew_at[t]);
#pragma unroll
    for (int t = 0; t < kRT; ++t) ex_next[t] = *reinterpret_cast<const int*>(x + ex_at[t]);
  };

  f32x16 acc[2][kRT];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int r = 0; r < kRT; ++r)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[t][r][e] = 0.f;

  fetch(0, 0);
  fetch_scales(0);
  for (int step = 0; step < a.steps; ++step) {
    __builtin_amdgcn_s_waitcnt(kWaitLoads);
    __syncthreads();
#pragma unroll
    for (int t = 0; t < 2; ++t) ew[t] = ew_next[t];
#pragma unroll
    for (int t = 0; t < kRT; ++t) ex[t] = ex_next[t];
    const uint4* const w = stage + (step & 1) * kBuf;
    const uint4* const x = w + kSide * 8;
    // operands of blocks s and 4 + s, requested while the products of the ones before them run
    uint4 wf[2][2], xf[2][kRT];
    auto request = [&](int s) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int row = wo * 64 + 32 * t + l32;
        wf[s & 1][t] = w[row * 8 + ((4 * half + s) ^ mx_place_of(row))];
      }
#pragma unroll
      for (int t = 0; t < kRT; ++t) {
        const int row = wr * (kSide / 2) + 32 * t + l32;
        xf[s & 1][t] = x[row * 8 + ((4 * half + s) ^ mx_place_of(row))];
      }
    };
    auto operand = [](uint4 v) {
      return i32x8{static_cast<int>(v.x), static_cast<int>(v.y), static_cast<int>(v.z), static_cast<int>(v.w), 0, 0, 0, 0};
    };
    auto products = [&](auto s_) {
      constexpr int s = decltype(s_)::value;
      if (s < 3) request(s + 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int r = 0; r < kRT; ++r)
#pragma unroll
        for (int t = 0; t < 2; ++t)
          acc[t][r] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(xf[s & 1][r]), operand(wf[s & 1][t]), acc[t][r], 4, 4, s, ex[r], s, ew[t]);
      __builtin_amdgcn_sched_barrier(0);
    };
    request(0);
    if (step + 1 < a.steps) {
      fetch(step + 1, ~step & 1);
      fetch_scales(step + 1);
    }
    products(std::integral_constant<int, 0>{});
    products(std::integral_constant<int, 1>{});
    products(std::integral_constant<int, 2>{});
    products(std::integral_constant<int, 3>{});
  }

  // lane: an output, and rows 8 (e / 4) + 4 half + e % 4 of each tile
  const bool whole = last_r == kSide - 1;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int o = o0 + wo * 64 + 32 * t + l32;
    if (o >= a.O) continue;
    const float bias = a.bias ? to_float(static_cast<const T*>(a.bias)[o]) : 0.f;
    const int first = wr * (kSide / 2) + 4 * half;
    T* const y = static_cast<T*>(a.y) + (r0 + first) * a.y_stride + o;
#pragma unroll
    for (int r = 0; r < kRT; ++r)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int row = 32 * r + 8 * (e >> 2) + (e & 3);
        if (whole || first + row <= last_r) __builtin_nontemporal_store(from_float<T>(acc[t][r][e] + bias), y + row * a.y_stride);
      }
  }
}

}  // namespace cdrge
