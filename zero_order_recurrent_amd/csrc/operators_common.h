// What the operators' kernels share (scan, adapters, distillation loss, delta rule, token scores, 4-bit projections): element
// types, conversions, matrix-core fragments, loads past the caches and into LDS, grids, reductions over a wave.
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

// s_waitcnt operand: no vector memory load in flight (vmcnt 0), the other counters not waited for
constexpr int kWaitLoads = 0x0f70;

// 16 bytes a lane from base + offset into LDS, lane by lane behind `to` (base and to are the same for
// the whole wave). The load has no register result. It is written as an instruction because the
// compiler, which cannot tell the two buffers apart, would wait for every load of this kind before any
// read of LDS; the wait that is needed stands before the step's barrier.
// m0 is written, and named so that no other use of it is moved across; clang warns that it never allocates m0 itself.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_to_lds(const char* base, uint32_t offset, uint4* to) {
  const uint32_t at = __builtin_amdgcn_readfirstlane(
      static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) void*)to)));
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(offset), "s"(base), "s"(at) : "memory", "m0");
}
#pragma clang diagnostic pop

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
