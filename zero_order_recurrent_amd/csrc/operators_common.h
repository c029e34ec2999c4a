// What the kernels of the scan, the adapters and the distillation loss share: element types,
// conversions, matrix-core fragments in 32-bit and split 16-bit precision, reductions over a wave.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace cdrge {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;

// Tensors of type T hold float, or uint16_t bit patterns of bf16.
__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

// Nearest bf16, ties to even: the cast is one conversion instruction on gfx950.
__device__ __forceinline__ uint16_t bf16_bits(float x) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x)); }
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
  const bf16x2 v = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
  return __builtin_bit_cast(uint32_t, v);
}

template <class T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ uint16_t from_float<uint16_t>(float v) {
  return bf16_bits(v);
}

// e^x and the logistic function on the exponential unit (relative error a few 2^-23). Both ends
// saturate by themselves: e^-x = inf gives a logistic value of 0.
__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896340736f); }
__device__ __forceinline__ float silu(float x) { return x * __builtin_amdgcn_rcpf(1.f + exp_fast(-x)); }
__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))); }

// Whole pieces of 16 bytes, at any element's alignment, past the caches: for what is read or written once.
typedef __attribute__((ext_vector_type(4), aligned(2))) uint32_t u32x4;
template <class A>
__device__ __forceinline__ void load_once(A& to, const void* from) {
  static_assert(sizeof(A) % 16 == 0, "whole pieces");
  u32x4 v[sizeof(A) / 16];
#pragma unroll
  for (int i = 0; i < int(sizeof(A) / 16); ++i) v[i] = __builtin_nontemporal_load(static_cast<const u32x4*>(from) + i);
  __builtin_memcpy(&to, v, sizeof(A));
}
template <class A>
__device__ __forceinline__ void store_once(void* to, const A& from) {
  static_assert(sizeof(A) % 16 == 0, "whole pieces");
  u32x4 v[sizeof(A) / 16];
  __builtin_memcpy(v, &from, sizeof(A));
#pragma unroll
  for (int i = 0; i < int(sizeof(A) / 16); ++i) __builtin_nontemporal_store(v[i], static_cast<u32x4*>(to) + i);
}

// Workgroups in one row, or in rows of 2^20 where a dimension's limit of 2^32 threads does not hold them; then the
// last row has some too many, which a kernel sends home by their number.
inline dim3 grid_of(int64_t blocks, int threads) {
  if (blocks * threads < (int64_t(1) << 32)) return dim3(static_cast<uint32_t>(blocks));
  return dim3(1u << 20, static_cast<uint32_t>((blocks + (1 << 20) - 1) >> 20));
}
__device__ __forceinline__ int64_t block_number() { return static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x; }

// Sum and maximum over a wave, in every lane. Within a row of 16 lanes the partner is reached by a lane
// permutation of the vector unit (quads, then mirrored halves and rows), across rows by a swap.
template <int kControl>
__device__ __forceinline__ float lane_move(float v) {
  const int i = __float_as_int(v);
  return __int_as_float(__builtin_amdgcn_update_dpp(i, i, kControl, 0xf, 0xf, false));
}
template <class F>
__device__ __forceinline__ float wave_reduce(float v, F op) {
  v = op(v, lane_move<0xb1>(v));   // lane ^ 1
  v = op(v, lane_move<0x4e>(v));   // lane ^ 2
  v = op(v, lane_move<0x141>(v));  // half-row mirror: 7 - lane
  v = op(v, lane_move<0x140>(v));  // row mirror: 15 - lane
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = op(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return op(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float wave_sum(float v) {
  return wave_reduce(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float wave_max(float v) {
  return wave_reduce(v, [](float a, float b) { return fmaxf(a, b); });
}

}  // namespace cdrge
