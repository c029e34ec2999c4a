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

// Eight elements of a row from column c on; zeros past its end.
template <class T>
__device__ __forceinline__ void mx_load(float (&v)[8], const T* row, int c, int K) {
  T e[8];
  if (c + 8 <= K) {
    __builtin_memcpy(e, row + c, sizeof(e));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = c + i < K ? row[c + i] : T(0);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = to_float(e[i]);
}

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

// Where a thread of k_mx_quantize and k_mx_dequantize works: a quarter of a block, `quarters` to a row, rows side by side
// in a workgroup where they are short.
struct MxPlace {
  int64_t row;
  int quarter;
};
__device__ __forceinline__ MxPlace mx_place(int quarters, int parts) {
  const int64_t id = block_number();
  if (parts > 1) return {id / parts, static_cast<int>(id % parts) * 256 + static_cast<int>(threadIdx.x)};
  const int each = 256 / quarters;  // rows of a workgroup
  const int r = threadIdx.x / quarters;
  return {r < each ? id * each + r : (int64_t(1) << 62), static_cast<int>(threadIdx.x) % quarters};
}

// kTiled: rows of whole steps of 8 blocks (zeros past K) and scales by step, as k_mx_tiles reads them; the workgroups past
// the rows' lay out the weights' scales in the same way, the last block's in the place of those past it (which meet zeros).
template <class T, bool kTiled>
__global__ __launch_bounds__(256) void k_mx_quantize(const T* __restrict__ x, int64_t stride, int64_t n_rows, int K, int quarters,
                                                     int parts, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                                                     int64_t groups, const uint8_t* __restrict__ w_scales, int O, int blocks,
                                                     uint8_t* __restrict__ w_tiled) {
  if (kTiled && block_number() >= groups) {
    const int64_t id = (block_number() - groups) * 256 + threadIdx.x;
    const int o = static_cast<int>(id % O), step = static_cast<int>(id / O);
    if (8 * step >= blocks) return;
    const uint8_t* const from = w_scales + static_cast<int64_t>(o) * blocks;
    uint8_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = from[min(8 * step + i, blocks - 1)];
    __builtin_memcpy(w_tiled + id * 8, v, 8);
    return;
  }
  const MxPlace at = mx_place(quarters, parts);
  if (at.row >= n_rows || at.quarter >= quarters) return;  // whole blocks
  float v[8];
  mx_load(v, x + at.row * stride, at.quarter * 8, K);
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) most = max(most, __float_as_uint(v[i]) & 0x7fffffffu);
  const int e = mx_scale(quad_most(most));
  reinterpret_cast<uint32_t*>(codes)[at.row * quarters + at.quarter] = mx_codes(v, e);
  const int b = at.quarter / 4;
  if (at.quarter % 4 == 0) scales[kTiled ? ((b / 8) * n_rows + at.row) * 8 + b % 8 : at.row * (quarters / 4) + b] = static_cast<uint8_t>(e);
}

// The value of a code with the scale byte e.
__device__ __forceinline__ float mx_value(uint32_t code, int e) {
  const uint32_t m = code & 7;
  const float size = m < 2 ? 0.5f * m : __uint_as_float(((m >> 1) + 126) << 23 | (m & 1) << 22);
  return e == 255 ? __builtin_nanf("") : ldexpf(code & 8 ? -size : size, e - 127);
}

template <class T>
__global__ __launch_bounds__(256) void k_mx_dequantize(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                       int64_t n_rows, int K, int quarters, int parts, T* __restrict__ x, int64_t stride) {
  const MxPlace at = mx_place(quarters, parts);
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
  const uint8_t* x_codes;
  const uint8_t* x_scales;
  void* y;
  int64_t y_stride;
  int64_t n_rows;
  int O, blocks;  // blocks of 32 along the reduction
};

// 16 outputs of up to 64 rows by a workgroup of eight waves, which share the reduction; each wave's sums are joined in
// their order.
template <class T>
__global__ __launch_bounds__(512) void k_mx_rows(MxArgs a, int o_tiles) {
  __shared__ f32x4 sums[8][4][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l16 = lane & 15, q = lane >> 4;
  const int64_t id = block_number();
  const int64_t row0 = id / o_tiles * 64;
  const int o0 = static_cast<int>(id % o_tiles) * 16;
  if (row0 >= a.n_rows) return;
  const int tiles = static_cast<int>(min<int64_t>(4, (a.n_rows - row0 + 15) / 16));
  const int steps = (a.blocks + 3) / 4, each = (steps + 7) / 8;
  const int64_t wrow = min(o0 + l16, a.O - 1);
  f32x4 acc[4] = {};
  for (int s = wave * each; s < min(steps, wave * each + each); ++s) {
    const int b = 4 * s + q;
    const bool have = b < a.blocks;
    const i32x4 none = {0, 0, 0, 0};
    const i32x4 w = have ? *reinterpret_cast<const i32x4*>(a.w_codes + (wrow * a.blocks + b) * 16) : none;
    const int we = have ? a.w_scales[wrow * a.blocks + b] : 127;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (t >= tiles) break;
      const int64_t row = min(row0 + 16 * t + l16, a.n_rows - 1);
      const i32x4 x = have ? *reinterpret_cast<const i32x4*>(a.x_codes + (row * a.blocks + b) * 16) : none;
      const int xe = have ? a.x_scales[row * a.blocks + b] : 127;
      acc[t] = mma_mx(w, we, x, xe, acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < 4; ++t) sums[wave][t][lane] = acc[t];
  __syncthreads();
  if (wave >= tiles) return;
  f32x4 sum = sums[0][wave][lane];
#pragma unroll
  for (int v = 1; v < 8; ++v) sum += sums[v][wave][lane];
  const int64_t row = row0 + 16 * wave + l16;
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
// (see place_w and place_x), so that the eight rows that a read touches at a time take all eight.
// The order along the reduction is free: lane group h of a wave takes the step's blocks 4 h .. 4 h + 3, whose scales are
// one word. So is that of a tile's outputs: a lane holds 32 adjacent ones of a row, which leave it in whole pieces.
// ---------------------------------------------------------------------------------------------
typedef __attribute__((ext_vector_type(16))) float f32x16;

struct MxTileArgs {
  const uint8_t* w_codes;  // [O][blocks][16]
  const uint8_t* w_scales;  // [step][O][8]
  const uint8_t* x_codes;  // [row][steps][8][16]
  const uint8_t* x_scales;  // [step][row][8]
  const void* bias;
  void* y;
  int64_t y_stride;
  int64_t n_rows;
  int O, blocks, steps, tiles_r, tiles_o;
};

__device__ __forceinline__ int mx_place_x(int row) { return row & 7; }
__device__ __forceinline__ int mx_place_w(int row) { return (row & 3) | ((row >> 3) & 4); }

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
  const char* const xb = reinterpret_cast<const char*>(a.x_codes) + r0 * a.steps * 128;
  auto fetch = [&](int step, int buf) {
    uint4* const to = stage + buf * kBuf + (tid & ~63);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int row = (tid >> 3) + i * (kThreads / 8), c = (tid & 7) ^ mx_place_w(row);
      // W's blocks past the last meet zeros of x: the last one is read in their place
      load_to_lds(wb, (min(row, last_o) * a.blocks + min(8 * step + c, a.blocks - 1)) * 16, to + i * kThreads);
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int row = (tid >> 3) + i * (kThreads / 8), c = (tid & 7) ^ mx_place_x(row);
      load_to_lds(xb + step * 128, min(row, last_r) * a.steps * 128 + c * 16, to + kSide * 8 + i * kThreads);
    }
  };
  // W's rows of a wave: row m of tile t is output 32 (m / 4 % 2) + 16 t + 4 (m / 8) + m % 4 of its 64
  int w_row[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) w_row[t] = wo * 64 + 32 * (l32 >> 2 & 1) + 16 * t + 4 * (l32 >> 3) + (l32 & 3);
  int ew[2], ex[kRT], ew_next[2], ex_next[kRT];
  auto fetch_scales = [&](int step) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
      ew_next[t] = *reinterpret_cast<const int*>(a.w_scales + (static_cast<int64_t>(step) * a.O + o0 + min(w_row[t], last_o)) * 8 + 4 * half);
#pragma unroll
    for (int t = 0; t < kRT; ++t)
      ex_next[t] = *reinterpret_cast<const int*>(a.x_scales + (step * a.n_rows + r0 + min(wr * (kSide / 2) + 32 * t + l32, last_r)) * 8 + 4 * half);
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
    if (step + 1 < a.steps) {
      fetch(step + 1, ~step & 1);
      fetch_scales(step + 1);
    }
    auto products = [&](auto s_) {
      constexpr int s = decltype(s_)::value;
      i32x8 wf[2], xf[kRT];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint4 v = w[w_row[t] * 8 + ((4 * half + s) ^ mx_place_w(w_row[t]))];
        wf[t] = i32x8{static_cast<int>(v.x), static_cast<int>(v.y), static_cast<int>(v.z), static_cast<int>(v.w), 0, 0, 0, 0};
      }
#pragma unroll
      for (int t = 0; t < kRT; ++t) {
        const int row = wr * (kSide / 2) + 32 * t + l32;
        const uint4 v = x[row * 8 + ((4 * half + s) ^ mx_place_x(row))];
        xf[t] = i32x8{static_cast<int>(v.x), static_cast<int>(v.y), static_cast<int>(v.z), static_cast<int>(v.w), 0, 0, 0, 0};
      }
#pragma unroll
      for (int r = 0; r < kRT; ++r)
#pragma unroll
        for (int t = 0; t < 2; ++t)
          acc[t][r] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wf[t], xf[r], acc[t][r], 4, 4, s, ew[t], s, ex[r]);
    };
    products(std::integral_constant<int, 0>{});
    products(std::integral_constant<int, 1>{});
    products(std::integral_constant<int, 2>{});
    products(std::integral_constant<int, 3>{});
  }

  const int o = o0 + wo * 64 + 32 * half;  // this lane's 32 outputs
  if (o >= a.O) return;
  const bool whole = o + 32 <= a.O;
#pragma unroll
  for (int r = 0; r < kRT; ++r) {
    const int row = wr * (kSide / 2) + 32 * r + l32;
    if (row > last_r) continue;
    T* const y = static_cast<T*>(a.y) + (r0 + row) * a.y_stride + o;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      T v[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float sum = acc[t][r][e];
        if (a.bias && o + 16 * t + e < a.O) sum += to_float(static_cast<const T*>(a.bias)[o + 16 * t + e]);
        v[e] = from_float<T>(sum);
      }
      if (whole) {
        __builtin_memcpy(y + 16 * t, v, sizeof(v));
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (o + 16 * t + e < a.O) y[16 * t + e] = v[e];
      }
    }
  }
}

}  // namespace cdrge
