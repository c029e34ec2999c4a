// A projection shared by all rows beside a low-rank adapter by row:
//   y_r = W x_r + b + s_r U_a (D_a x_r),  a = row_adapter[r].
//
// Two launches: k_adapter_down forms v_r = s_r D_a x_r (float32, max_rank values a row), then
// k_adapter_project forms W x_r and adds U_a v_r from the same matrix-core tiles. Rows need no
// order: a tile of 16 rows runs the low-rank product once for each adapter that it meets and keeps,
// of each, the rows that name it (a selection, so that what one adapter holds cannot reach
// another's rows, NaN included).
//
// Both element types run on the matrix cores with 16 bytes of a row in each lane: for bf16 that
// is one 16x16x32 product over 32 columns, for float32 four 16x16x4 products over 16 columns, in
// which product t takes element t of every lane - a permutation of the reduction index that both
// operands share.
#pragma once
#include "operators_common.h"

namespace cdrge {

struct AdapterArgs {
  const void* x;
  int64_t x_stride;
  const void* weight;
  int64_t weight_stride;
  const void* bias;
  const void* down;
  const void* up;
  const int32_t* ranks;
  const int32_t* row_adapter;
  const float* row_scale;
  void* y;
  int64_t y_stride;
  float* v;  // [n_rows][R]
  int64_t n_rows;
  int K, O, A, R;
};

template <class T>
struct Frag;  // 16 bytes of a row per lane
template <>
struct Frag<uint16_t> {
  static constexpr int kCols = 32, kPer = 8;
  bf16x8 v;
};
template <>
struct Frag<float> {
  static constexpr int kCols = 16, kPer = 4;
  f32x4 v;
};

__device__ __forceinline__ f32x4 mma(const Frag<uint16_t>& a, const Frag<uint16_t>& b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(const Frag<float>& a, const Frag<float>& b, f32x4 c) {
#pragma unroll
  for (int t = 0; t < 4; ++t) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[t], b.v[t], c, 0, 0, 0);
  return c;
}

// Columns k .. k + kPer - 1 of a row of n columns (zero past its end, and everywhere if !ok).
template <class T>
__device__ __forceinline__ Frag<T> load_frag(const T* row, int k, int n, bool ok) {
  Frag<T> f;
  T e[Frag<T>::kPer];
#pragma unroll
  for (int i = 0; i < Frag<T>::kPer; ++i) e[i] = (ok && k + i < n) ? row[k + i] : T(0);
  __builtin_memcpy(&f.v, e, 16);
  return f;
}

__device__ __forceinline__ int rank_of(const AdapterArgs& a, int ad) {
  return a.ranks ? min(max(a.ranks[ad], 0), a.R) : a.R;
}

// v of a tile of 16 rows, one wave. grid: tiles.
template <class T>
__global__ __launch_bounds__(64) void k_adapter_down(AdapterArgs a) {
  const int lane = threadIdx.x, l16 = lane & 15, q = lane >> 4;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * 16, r = r0 + l16;
  const bool rok = r < a.n_rows;
  int ad = rok ? a.row_adapter[r] : -1;
  const T* x = static_cast<const T*>(a.x) + (rok ? r : 0) * a.x_stride;
  uint32_t todo = static_cast<uint32_t>(__ballot(ad >= 0 && ad < a.A)) & 0xffffu;
  while (todo) {
    const int cur = __shfl(ad, __builtin_ctz(todo));
    todo &= ~static_cast<uint32_t>(__ballot(ad == cur));
    const int rank = rank_of(a, cur);
    for (int j0 = 0; j0 < rank; j0 += 16) {
      const T* d = static_cast<const T*>(a.down) + (static_cast<int64_t>(cur) * a.R + min(j0 + l16, rank - 1)) * a.K;
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
      for (int k = 0; k < a.K; k += Frag<T>::kCols)
        acc = mma(load_frag<T>(d, k + q * Frag<T>::kPer, a.K, j0 + l16 < rank),
                  load_frag<T>(x, k + q * Frag<T>::kPer, a.K, rok), acc);
      // acc[e]: rank index j0 + 4 q + e of row l16
      if (rok && ad == cur) {
        const float s = a.row_scale ? a.row_scale[r] : 1.f;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (j0 + 4 * q + e < rank) a.v[r * a.R + j0 + 4 * q + e] = s * acc[e];
      }
    }
  }
}

// v of row r as a fragment (bf16: the high or the low half of its value).
__device__ __forceinline__ Frag<float> v_frag(const float* v, int k, int n, bool ok, Frag<float>& low) {
  low.v = f32x4{0.f, 0.f, 0.f, 0.f};
  return load_frag<float>(v, k, n, ok);
}
__device__ __forceinline__ Frag<uint16_t> v_frag(const float* v, int k, int n, bool ok, Frag<uint16_t>& low) {
  Frag<uint16_t> hi;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float f = (ok && k + i < n) ? v[k + i] : 0.f;
    const __bf16 h = static_cast<__bf16>(f);
    hi.v[i] = h;
    // an infinite v has no low half (inf - inf would turn it into NaN)
    low.v[i] = static_cast<__bf16>(fabsf(f) <= 3.38953139e38f ? f - static_cast<float>(h) : 0.f);
  }
  return hi;
}

// y of 16 rows x 64 outputs a wave: the operands are W (16 outputs) and x (16 rows), so that a lane
// holds four adjacent outputs of one row. grid: (row tiles of 16, output tiles of 64).
template <class T>
__global__ __launch_bounds__(64) void k_adapter_project(AdapterArgs a) {
  const int lane = threadIdx.x, l16 = lane & 15, q = lane >> 4;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * 16 + l16;
  const int o0 = blockIdx.y * 64;
  const bool rok = r < a.n_rows;
  const T* x = static_cast<const T*>(a.x) + (rok ? r : 0) * a.x_stride;
  const T* w = static_cast<const T*>(a.weight);
  f32x4 acc[4];
  for (int t = 0; t < 4; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int k = 0; k < a.K; k += Frag<T>::kCols) {
    const Frag<T> xf = load_frag<T>(x, k + q * Frag<T>::kPer, a.K, rok);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int o = o0 + 16 * t + l16;
      acc[t] = mma(load_frag<T>(w + static_cast<int64_t>(min(o, a.O - 1)) * a.weight_stride, k + q * Frag<T>::kPer, a.K, o < a.O),
                   xf, acc[t]);
    }
  }
  const int ad = (rok && a.row_adapter) ? a.row_adapter[r] : -1;
  uint32_t todo = static_cast<uint32_t>(__ballot(ad >= 0 && ad < a.A)) & 0xffffu;
  while (todo) {
    const int cur = __shfl(ad, __builtin_ctz(todo));
    todo &= ~static_cast<uint32_t>(__ballot(ad == cur));
    const int rank = rank_of(a, cur);
    const bool mine = ad == cur;
    f32x4 low[4];
    for (int t = 0; t < 4; ++t) low[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < rank; k += Frag<T>::kCols) {
      Frag<T> vl;
      const Frag<T> vh = v_frag(a.v + (rok ? r : 0) * a.R, k + q * Frag<T>::kPer, rank, mine, vl);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int o = o0 + 16 * t + l16;
        const T* u = static_cast<const T*>(a.up) + (static_cast<int64_t>(cur) * a.O + min(o, a.O - 1)) * a.R;
        const Frag<T> uf = load_frag<T>(u, k + q * Frag<T>::kPer, rank, o < a.O);
        low[t] = mma(uf, vh, low[t]);
        if (sizeof(T) == 2) low[t] = mma(uf, vl, low[t]);
      }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[t][e] = mine ? acc[t][e] + low[t][e] : acc[t][e];
  }
  if (!rok) return;
  T* y = static_cast<T*>(a.y) + r * a.y_stride;
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int o = o0 + 16 * t + 4 * q + e;
      if (o >= a.O) continue;
      float f = acc[t][e];
      if (a.bias) f += to_float(static_cast<const T*>(a.bias)[o]);
      if (ad >= a.A) f = __builtin_nanf("");
      y[o] = from_float<T>(f);
    }
}

}  // namespace cdrge
