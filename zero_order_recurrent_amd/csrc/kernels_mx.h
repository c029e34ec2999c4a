// Microscaled 4-bit floating point: quantisation, the values back, and the product of quantised rows with quantised
// weights (E2M1 elements, a power of two for each 32 of them along the reduction).
#pragma once
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

template <class T>
__global__ __launch_bounds__(256) void k_mx_quantize(const T* __restrict__ x, int64_t stride, int64_t n_rows, int K, int quarters,
                                                     int parts, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const MxPlace at = mx_place(quarters, parts);
  if (at.row >= n_rows || at.quarter >= quarters) return;  // whole blocks
  float v[8];
  mx_load(v, x + at.row * stride, at.quarter * 8, K);
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) most = max(most, __float_as_uint(v[i]) & 0x7fffffffu);
  const int e = mx_scale(quad_most(most));
  reinterpret_cast<uint32_t*>(codes)[at.row * quarters + at.quarter] = mx_codes(v, e);
  if (at.quarter % 4 == 0) scales[(at.row * quarters + at.quarter) / 4] = static_cast<uint8_t>(e);
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

}  // namespace cdrge
