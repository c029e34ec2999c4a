// Gated delta rule.
//
//   q' = q_scale q / sqrt(q.q + eps),  k' = k / sqrt(k.k + eps)
//   a_t = exp(decay softplus(dt_t + dt_bias)),  b_t = 1 / (1 + exp(-beta_t))
//   S_t = a_t S_{t-1} + b_t (v_t - a_t S_{t-1} k'_t) k'_t^T,   y_t = S_t q'_t
//
// Sequences, slots and blocks of tokens are the scan's: DeltaArgs holds its arguments, with value_dim for
// head_dim and key_dim for state_dim, beside the delta rule's own.
#pragma once
#include "kernels_scan.h"

namespace cdrge {

struct DeltaArgs {
  ScanArgs s;
  const void* q;
  int64_t q_stride;
  const void* k;
  int64_t k_stride;
  const void* v;
  int64_t v_stride;
  const void* beta;
  int64_t beta_stride;
  float q_scale, norm_eps;
};

__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + expf(-x)); }

// What brings a row of the sum of squares ss to length one; a sum past float32 makes the row NaN.
__device__ __forceinline__ float delta_norm(float ss, float eps) {
  return ss < __builtin_inff() ? 1.f / sqrtf(ss + eps) : __builtin_nanf("");
}

template <int kLanes>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int m = kLanes / 2; m > 0; m >>= 1) v += __shfl_xor(v, m);
  return v;
}

// Token after token, with the state in registers: kLanes lanes side by side hold four of its columns each, a thread
// kRpt of its rows. One token for each sequence (kStep) is bound by memory, which the state crosses twice.
// With S the state before a token, its prediction of v is a S k' and y = a S q' + (k'.q') b (v - a S k'), so that both
// products of S run before its update.
template <class T, int kLanes, int kRpt, bool kStep>
__global__ __launch_bounds__(256) void k_delta_tokens(DeltaArgs a, ScanWork w) {
  constexpr int kTile = 256 / kLanes * kRpt;
  const ScanArgs& s = a.s;
  const int tid = threadIdx.x;
  const uint32_t id = static_cast<uint32_t>(block_number());
  const int tile = id % s.ptiles, h = id / s.ptiles % s.H, i = id / (s.ptiles * s.H);
  if (i >= s.n_seqs) return;
  const int p0 = tile * kTile, np = min(kTile, s.P - p0);
  int64_t first = i;
  int len = 1, slot = -1, pos = 0, taken = 0;
  T* y = static_cast<T*>(s.y) + static_cast<int64_t>(h) * s.P + p0;
  if (kStep) {
    slot = s.slots ? s.slots[i] : i;
    pos = max(s.positions[i], 0);
    if (slot < 0) return;
    if (slot >= s.n_slots)
      taken = 1;
    else if (s.owned)
      taken = !(to_float(y[i * s.y_stride]) == 0.f);
    else if (s.slots)
      for (int j = tid; j < i; j += 256) taken |= s.slots[j] == slot;
    taken = __syncthreads_or(taken);
  } else {
    const ScanSeq sq = scan_seq(s, w, i);
    first = sq.first;
    len = sq.len;
    if (s.ssm_in) {
      slot = s.owned ? w.slots[i] : scan_slot(s, i);
      taken = slot == -2;
      if (slot >= 0 && s.positions) pos = max(s.positions[i], 0);
    }
  }
  y += first * s.y_stride;
  if (taken) {
    for (int t = 0; t < len; ++t)
      if (tid < np) y[t * s.y_stride + tid] = from_float<T>(__builtin_nanf(""));
    return;
  }
  const int N = s.N, g = h / (s.H / s.G);
  const int ln = tid % kLanes, n0 = ln * 4, have = N - n0, r0 = tid / kLanes * kRpt;
  const bool vec = N % 4 == 0;
  const int64_t sbase = (static_cast<int64_t>(max(slot, 0)) * s.H + h) * s.P + p0;
  float st[kRpt][4];
#pragma unroll
  for (int r = 0; r < kRpt; ++r) {
#pragma unroll
    for (int e = 0; e < 4; ++e) st[r][e] = 0.f;
    if (slot >= 0 && pos > 0 && r0 + r < np && have > 0) {
      const float* const from = s.ssm_in + (sbase + r0 + r) * N + n0;
      if (vec) {
        const f32x4 x = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(from));
#pragma unroll
        for (int e = 0; e < 4; ++e) st[r][e] = x[e];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e < have) st[r][e] = from[e];
      }
    }
  }
  const T* const qp = static_cast<const T*>(a.q) + first * a.q_stride + static_cast<int64_t>(g) * N + n0;
  const T* const kp = static_cast<const T*>(a.k) + first * a.k_stride + static_cast<int64_t>(g) * N + n0;
  const T* const vp = static_cast<const T*>(a.v) + first * a.v_stride + static_cast<int64_t>(h) * s.P + p0 + r0;
  const T* const dp = static_cast<const T*>(s.dt) + first * s.dt_stride + h;
  const T* const bp = static_cast<const T*>(a.beta) + first * a.beta_stride + h;
  const float bias = s.dt_bias ? s.dt_bias[h] : 0.f, decay = s.decay[h];
  for (int t = 0; t < len; ++t) {
    Four<T> qv, kv;
    qv.load(qp + t * a.q_stride, have);
    kv.load(kp + t * a.k_stride, have);
    float v[kRpt];
#pragma unroll
    for (int r = 0; r < kRpt; ++r) v[r] = r0 + r < np ? to_float(vp[t * a.v_stride + r]) : 0.f;
    const float step = softplus(to_float(dp[t * s.dt_stride]) + bias), b = sigmoid(to_float(bp[t * a.beta_stride]));
    const float fade = expf(step * decay);
    float q[4], k[4], qq = 0.f, kk = 0.f, kq = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      q[e] = qv.at(e);
      k[e] = kv.at(e);
      qq += q[e] * q[e];
      kk += k[e] * k[e];
    }
    const float rq = a.q_scale * delta_norm(lanes_sum<kLanes>(qq), a.norm_eps), rk = delta_norm(lanes_sum<kLanes>(kk), a.norm_eps);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      q[e] *= rq;
      k[e] *= rk;
      kq += k[e] * q[e];
    }
    kq = lanes_sum<kLanes>(kq);
    float mine = 0.f;
#pragma unroll
    for (int r = 0; r < kRpt; ++r) {
      float sk = 0.f, sq = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        st[r][e] *= fade;
        sk += st[r][e] * k[e];
        sq += st[r][e] * q[e];
      }
      sk = lanes_sum<kLanes>(sk);
      sq = lanes_sum<kLanes>(sq);
      const float add = b * (v[r] - sk);
#pragma unroll
      for (int e = 0; e < 4; ++e) st[r][e] += add * k[e];
      const float out = sq + add * kq;
      if (kRpt <= kLanes) {
        if (ln == r) mine = out;
      } else if (ln == 0 && r0 + r < np) {
        y[t * s.y_stride + r0 + r] = from_float<T>(out);
      }
    }
    if (kRpt <= kLanes && ln < kRpt && r0 + ln < np) y[t * s.y_stride + r0 + ln] = from_float<T>(mine);
  }
  if (slot < 0) return;
#pragma unroll
  for (int r = 0; r < kRpt; ++r) {
    if (r0 + r >= np || have <= 0) continue;
    float* const to = s.ssm_out + (sbase + r0 + r) * N + n0;
    if (vec) {
      __builtin_nontemporal_store(f32x4{st[r][0], st[r][1], st[r][2], st[r][3]}, reinterpret_cast<f32x4*>(to));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < have) to[e] = st[r][e];
    }
  }
}

}  // namespace cdrge
