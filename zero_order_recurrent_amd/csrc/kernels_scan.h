// Selective state space scan with its short causal convolution.
//
//   u_q = silu(conv_bias + sum_j conv_weight[:, j] xbc_{q - W + 1 + j}),  u = [x | B | C]
//   step_q = softplus(dt_q + dt_bias),  S_q = exp(step_q decay) S_{q-1} + step_q x_q B_q^T
//   y_q = S_q C_q + skip x_q, times silu(z_q)
//
// The convolution's memory is a ring of W rows of xbc by slot, row q at entry q mod W. A token's
// convolution reads the W - 1 entries before its own and writes its own, so that within one launch
// the workgroups that read a ring never meet the one that updates it in place.
#pragma once
#include "operators_common.h"

namespace cdrge {

constexpr int kScanMaxState = 256;
constexpr int kScanMaxConv = 4;

struct ScanArgs {
  const void* xbc;
  int64_t xbc_stride;
  const void* dt;
  int64_t dt_stride;
  const void* z;
  int64_t z_stride;
  void* y;
  int64_t y_stride;
  int64_t n_tokens;
  const int32_t* offsets;
  const int32_t* slots;
  const int32_t* positions;
  const void* conv_in;
  void* conv_out;
  const float* ssm_in;
  float* ssm_out;
  const void* conv_weight;
  const void* conv_bias;
  const float* decay;
  const float* skip;
  const float* dt_bias;
  int n_seqs, n_slots;
  int H, P, G, N, W, C;  // C: channels = H P + 2 G N
  int ptiles;            // column tiles of a head
};

// Slot of sequence i: -1 if it keeps no state, -2 if the slot is out of range or an earlier
// sequence of the call has it. Called by a whole workgroup.
__device__ __forceinline__ int scan_slot(const ScanArgs& a, int i) {
  const int s = a.slots ? a.slots[i] : i;
  if (s < 0) return -1;
  if (s >= a.n_slots) return -2;
  int taken = 0;
  if (a.slots)
    for (int j = threadIdx.x; j < i; j += blockDim.x) taken |= a.slots[j] == s;
  return __syncthreads_or(taken) ? -2 : s;
}

// ---------------------------------------------------------------------------------------------
// One token for each sequence. A workgroup owns kRpt * (256 / kLanes) channels of one head of one
// row: kLanes lanes side by side hold four columns of the state each, so a state row is read and
// written in whole lines. Bound by memory: the state is read and written once.
// ---------------------------------------------------------------------------------------------
template <class T, int kLanes, int kRpt>
__global__ __launch_bounds__(256) void k_scan_step(ScanArgs a) {
  constexpr int kRows = 256 / kLanes;
  constexpr int kTile = kRows * kRpt;
  __shared__ float sb[kScanMaxState], sc[kScanMaxState], sx[kTile], sy[kTile];
  const int tid = threadIdx.x;
  const int tile = blockIdx.x % a.ptiles, h = (blockIdx.x / a.ptiles) % a.H, i = blockIdx.x / (a.ptiles * a.H);
  const int slot = scan_slot(a, i);
  if (slot == -1) return;
  const int p0 = tile * kTile, np = min(kTile, a.P - p0);
  T* y = static_cast<T*>(a.y) + i * a.y_stride + static_cast<int64_t>(h) * a.P + p0;
  if (slot < 0) {
    if (tid < np) y[tid] = from_float<T>(__builtin_nanf(""));
    return;
  }
  const int pos = max(a.positions[i], 0);
  const int N = a.N, ln = tid % kLanes, n0 = ln * 4, pr = tid / kLanes;
  const int64_t sbase = ((static_cast<int64_t>(slot) * a.H + h) * a.P + p0) * N;
  const bool vec = N % 4 == 0;
  float st[kRpt][4];
#pragma unroll
  for (int k = 0; k < kRpt; ++k) {
    const int p = pr + k * kRows;
#pragma unroll
    for (int e = 0; e < 4; ++e) st[k][e] = 0.f;
    if (pos > 0 && p < np && n0 < N) {
      const float* s = a.ssm_in + sbase + static_cast<int64_t>(p) * N + n0;
      if (vec) {
        const float4 v = *reinterpret_cast<const float4*>(s);
        st[k][0] = v.x; st[k][1] = v.y; st[k][2] = v.z; st[k][3] = v.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n0 + e < N) st[k][e] = s[e];
      }
    }
  }
  // convolution of this tile's x and of the group's B and C
  const int g = h / (a.H / a.G);
  const bool owns_bc = tile == 0 && h % (a.H / a.G) == 0;
  const T* x = static_cast<const T*>(a.xbc) + i * a.xbc_stride;
  const T* ring = static_cast<const T*>(a.conv_in) + static_cast<int64_t>(slot) * a.W * a.C;
  T* ring_out = static_cast<T*>(a.conv_out) + static_cast<int64_t>(slot) * a.W * a.C;
  const bool in_place = a.conv_in == a.conv_out;
  for (int idx = tid; idx < np + 2 * N; idx += 256) {
    const int c = idx < np ? h * a.P + p0 + idx
                           : (idx < np + N ? a.H * a.P + g * N + idx - np : a.H * a.P + a.G * N + g * N + idx - np - N);
    const T* w = static_cast<const T*>(a.conv_weight) + static_cast<int64_t>(c) * a.W;
    const T now = x[c];
    float u = a.conv_bias ? to_float(static_cast<const T*>(a.conv_bias)[c]) : 0.f;
    for (int j = 1; j < a.W; ++j)
      if (pos - j >= 0) u += to_float(w[a.W - 1 - j]) * to_float(ring[static_cast<int64_t>((pos - j) % a.W) * a.C + c]);
    u = silu(u + to_float(w[a.W - 1]) * to_float(now));
    if (idx < np)
      sx[idx] = u;
    else if (idx < np + N)
      sb[idx - np] = u;
    else
      sc[idx - np - N] = u;
    if (idx < np || owns_bc) {
      if (!in_place)
        for (int e = 0; e < a.W; ++e) ring_out[static_cast<int64_t>(e) * a.C + c] = ring[static_cast<int64_t>(e) * a.C + c];
      ring_out[static_cast<int64_t>(pos % a.W) * a.C + c] = now;
    }
  }
  const float dt = softplus(to_float(static_cast<const T*>(a.dt)[i * a.dt_stride + h]) + (a.dt_bias ? a.dt_bias[h] : 0.f));
  const float fade = expf(dt * a.decay[h]);
  __syncthreads();
  float b[4], c[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    b[e] = n0 + e < N ? sb[n0 + e] : 0.f;
    c[e] = n0 + e < N ? sc[n0 + e] : 0.f;
  }
#pragma unroll
  for (int k = 0; k < kRpt; ++k) {
    const int p = pr + k * kRows;
    const float xd = p < np ? dt * sx[p] : 0.f;
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      st[k][e] = st[k][e] * fade + xd * b[e];
      sum += n0 + e < N ? st[k][e] * c[e] : 0.f;
    }
#pragma unroll
    for (int m = kLanes / 2; m > 0; m >>= 1) sum += __shfl_xor(sum, m);
    if (ln == 0) sy[p] = sum;
    if (p < np && n0 < N) {
      float* s = a.ssm_out + sbase + static_cast<int64_t>(p) * N + n0;
      if (vec) {
        *reinterpret_cast<float4*>(s) = make_float4(st[k][0], st[k][1], st[k][2], st[k][3]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n0 + e < N) s[e] = st[k][e];
      }
    }
  }
  __syncthreads();
  if (tid < np) {
    float v = sy[tid] + (a.skip ? a.skip[h] * sx[tid] : 0.f);
    if (a.z) v *= silu(to_float(static_cast<const T*>(a.z)[i * a.z_stride + static_cast<int64_t>(h) * a.P + p0 + tid]));
    y[tid] = from_float<T>(v);
  }
}

// ---------------------------------------------------------------------------------------------
// Prompts, token by token: a workgroup walks one sequence for 64 channels of one head; thread
// (p, quarter) holds a quarter of the state row of channel p.
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ void scan_bounds(const ScanArgs& a, int i, int64_t& first, int64_t& len) {
  if (!a.offsets) {
    len = a.n_tokens / a.n_seqs;
    first = i * len;
    return;
  }
  first = min(max(static_cast<int64_t>(a.offsets[i]), int64_t(0)), a.n_tokens);
  len = max(min(static_cast<int64_t>(a.offsets[i + 1]), a.n_tokens) - first, int64_t(0));
}

template <class T>
__device__ __forceinline__ float scan_conv(const ScanArgs& a, int c, int64_t first, int64_t t, int pos, const T* ring) {
  const T* w = static_cast<const T*>(a.conv_weight) + static_cast<int64_t>(c) * a.W;
  float u = a.conv_bias ? to_float(static_cast<const T*>(a.conv_bias)[c]) : 0.f;
  for (int j = 0; j < a.W; ++j) {
    const int64_t back = t - (a.W - 1 - j);
    if (back >= 0)
      u += to_float(w[j]) * to_float(static_cast<const T*>(a.xbc)[(first + back) * a.xbc_stride + c]);
    else if (ring && pos + back >= 0)
      u += to_float(w[j]) * to_float(ring[((pos + back) % a.W) * a.C + c]);
  }
  return silu(u);
}

template <class T, int kQuarter>
__global__ __launch_bounds__(256) void k_scan_walk(ScanArgs a) {
  __shared__ float sx[64], sb[kScanMaxState], sc[kScanMaxState];
  const int tid = threadIdx.x;
  const int tile = blockIdx.x % a.ptiles, h = (blockIdx.x / a.ptiles) % a.H, i = blockIdx.x / (a.ptiles * a.H);
  const int slot = a.ssm_in ? scan_slot(a, i) : -1;
  int64_t first, len;
  scan_bounds(a, i, first, len);
  const int p0 = tile * 64, np = min(64, a.P - p0), p = tid >> 2, n0 = (tid & 3) * kQuarter, N = a.N;
  T* y = static_cast<T*>(a.y) + static_cast<int64_t>(h) * a.P + p0;
  if (slot == -2) {
    for (int64_t t = 0; t < len; ++t)
      if (tid < np) y[(first + t) * a.y_stride + tid] = from_float<T>(__builtin_nanf(""));
    return;
  }
  const int pos = (slot >= 0 && a.positions) ? max(a.positions[i], 0) : 0;
  const T* ring = slot >= 0 ? static_cast<const T*>(a.conv_in) + static_cast<int64_t>(slot) * a.W * a.C : nullptr;
  const int64_t sbase = ((static_cast<int64_t>(max(slot, 0)) * a.H + h) * a.P + p0 + p) * N;
  float st[kQuarter];
#pragma unroll
  for (int n = 0; n < kQuarter; ++n) st[n] = (pos > 0 && p < np && n0 + n < N) ? a.ssm_in[sbase + n0 + n] : 0.f;
  const int g = h / (a.H / a.G);
  for (int64_t t = 0; t < len; ++t) {
    __syncthreads();
    for (int idx = tid; idx < np + 2 * N; idx += 256) {
      const int c = idx < np ? h * a.P + p0 + idx
                             : (idx < np + N ? a.H * a.P + g * N + idx - np : a.H * a.P + a.G * N + g * N + idx - np - N);
      const float u = scan_conv<T>(a, c, first, t, pos, ring);
      if (idx < np)
        sx[idx] = u;
      else if (idx < np + N)
        sb[idx - np] = u;
      else
        sc[idx - np - N] = u;
    }
    const float dt = softplus(to_float(static_cast<const T*>(a.dt)[(first + t) * a.dt_stride + h]) + (a.dt_bias ? a.dt_bias[h] : 0.f));
    const float fade = expf(dt * a.decay[h]);
    __syncthreads();
    const float x = p < np ? sx[p] : 0.f;
    float sum = 0.f;
#pragma unroll
    for (int n = 0; n < kQuarter; ++n)
      if (n0 + n < N) {
        st[n] = st[n] * fade + dt * x * sb[n0 + n];
        sum += st[n] * sc[n0 + n];
      }
    sum += __shfl_xor(sum, 1);
    sum += __shfl_xor(sum, 2);
    if ((tid & 3) == 0 && p < np) {
      float v = sum + (a.skip ? a.skip[h] * x : 0.f);
      if (a.z) v *= silu(to_float(static_cast<const T*>(a.z)[(first + t) * a.z_stride + static_cast<int64_t>(h) * a.P + p0 + p]));
      y[(first + t) * a.y_stride + p] = from_float<T>(v);
    }
  }
  if (slot >= 0 && p < np) {
#pragma unroll
    for (int n = 0; n < kQuarter; ++n)
      if (n0 + n < N) a.ssm_out[sbase + n0 + n] = st[n];
  }
}

// The rings after a prompt call, a launch of its own: in place, every reader of the old rings is
// done. grid: (channel blocks of 256, sequences).
template <class T>
__global__ __launch_bounds__(256) void k_scan_ring(ScanArgs a, int cblocks) {
  const int i = blockIdx.x / cblocks, c = (blockIdx.x % cblocks) * 256 + threadIdx.x;
  const int slot = scan_slot(a, i);
  if (slot < 0 || c >= a.C) return;
  int64_t first, len;
  scan_bounds(a, i, first, len);
  const int pos = a.positions ? max(a.positions[i], 0) : 0;
  const T* ring = static_cast<const T*>(a.conv_in) + static_cast<int64_t>(slot) * a.W * a.C + c;
  T* out = static_cast<T*>(a.conv_out) + static_cast<int64_t>(slot) * a.W * a.C + c;
  for (int e = 0; e < a.W; ++e) {
    // the newest of this call's tokens whose place is e modulo W
    const int64_t last = pos + len - 1;
    const int64_t q = last - (((last - e) % a.W) + a.W) % a.W;
    if (q >= pos)
      out[static_cast<int64_t>(e) * a.C] = static_cast<const T*>(a.xbc)[(first + q - pos) * a.xbc_stride + c];
    else if (a.conv_in != a.conv_out)
      out[static_cast<int64_t>(e) * a.C] = ring[static_cast<int64_t>(e) * a.C];
  }
}

}  // namespace cdrge
