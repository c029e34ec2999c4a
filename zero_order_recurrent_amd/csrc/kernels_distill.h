// Distillation from a teacher's top logits: row loss, its gradient, and the mean by model.
//
// With z = logits / tau, M the row's largest logit and S = sum_v exp((logit_v - M) / tau):
//   log q_v = (logit_v - M) / tau - log S,   row_loss = tau^2 sum_j p_j (log p_j + (M - logit_{id_j}) / tau + log S),
//   d row_loss / d logit_v = tau (exp((logit_v - M) / tau) / S - sum_{j: id_j = v} p_j).
// The work is one read of the logits (and one write of the gradient): bound by memory.
#pragma once
#include "operators_common.h"

namespace cdrge {

struct DistillArgs {
  const void* logits;
  int64_t logits_stride;
  const int32_t* ids;
  const float* teacher;
  const float* row_grad;
  float* row_losses;
  void* dlogits;
  int64_t dlogits_stride;
  int64_t n_rows;
  int vocab, top_k;
  float tau;
};

// Sum or maximum over the kTeam threads that share a row. part: kTeam / 64 floats of LDS.
template <int kTeam, bool kMax>
__device__ __forceinline__ float team_reduce(float v, float* part) {
  v = kMax ? wave_max(v) : wave_sum(v);
  if (kTeam == 64) return v;
  const int wave = threadIdx.x >> 6;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[wave] = v;
  __syncthreads();
  float r = part[0];
#pragma unroll
  for (int i = 1; i < kTeam / 64; ++i) r = kMax ? fmaxf(r, part[i]) : r + part[i];
  return r;
}

// Orders the team's memory accesses before it against those after it.
template <int kTeam>
__device__ __forceinline__ void team_sync() {
  if (kTeam == 64) {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
    __builtin_amdgcn_wave_barrier();
  } else {
    __syncthreads();
  }
}

// One row by kTeam threads (64: four rows by a workgroup of 256).
template <class T, bool kGrad, int kTeam>
__global__ __launch_bounds__(kTeam == 64 ? 256 : kTeam) void k_distill(DistillArgs a) {
  extern __shared__ float lds[];  // per row of the workgroup: top_k probabilities, top_k ids
  __shared__ float part[16];
  const int lane = kTeam == 64 ? (threadIdx.x & 63) : threadIdx.x;
  const int team = kTeam == 64 ? (threadIdx.x >> 6) : 0;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kTeam == 64 ? 4 : 1) + team;
  if (row >= a.n_rows) return;  // a whole wave, which waits for nobody below
  float* prob = lds + 2 * team * a.top_k;
  int* id = reinterpret_cast<int*>(prob + a.top_k);
  const T* x = static_cast<const T*>(a.logits) + row * a.logits_stride;
  const int V = a.vocab, k = a.top_k;
  const float inv_tau = 1.f / a.tau, scale = 1.44269504088896340736f / a.tau;
  const float ninf = -__builtin_inff();

  // teacher: softmax over the present entries
  float tmax = ninf;
  int bad = 0, present = 0;
  for (int j = lane; j < k; j += kTeam) {
    const int v = a.ids[row * k + j];
    const float t = a.teacher[row * k + j];
    const bool have = v >= 0 && !(t == ninf);
    bad |= (have && v >= V) ? 1 : 0;
    present |= have ? 1 : 0;
    id[j] = have ? v : -1;
    prob[j] = t;
    if (have) tmax = fmaxf(tmax, t);
  }
  tmax = team_reduce<kTeam, true>(tmax, part);
  bad = team_reduce<kTeam, true>(static_cast<float>(bad), part) > 0.f;
  present = team_reduce<kTeam, true>(static_cast<float>(present), part) > 0.f;

  // student: largest logit, then the sum of exponentials
  float xmax = ninf;
  for (int v = lane; v < V; v += kTeam) xmax = fmaxf(xmax, to_float(x[v]));
  xmax = team_reduce<kTeam, true>(xmax, part);
  const float base = xmax == ninf ? 0.f : xmax;
  float sum = 0.f;
  for (int v = lane; v < V; v += kTeam) sum += __builtin_amdgcn_exp2f((to_float(x[v]) - base) * scale);
  sum = team_reduce<kTeam, false>(sum, part);
  const float log_sum = logf(sum);

  team_sync<kTeam>();
  float mass = 0.f;
  for (int j = lane; j < k; j += kTeam) mass += id[j] >= 0 ? expf((prob[j] - tmax) * inv_tau) : 0.f;
  mass = team_reduce<kTeam, false>(mass, part);
  const float log_mass = logf(mass);
  float loss = 0.f;
  for (int j = lane; j < k; j += kTeam) {
    const float lp = (prob[j] - tmax) * inv_tau - log_mass;
    const float p = id[j] >= 0 ? expf(lp) : 0.f;
    // a probability that underflows contributes its limit, zero
    if (id[j] >= 0 && id[j] < V && !(p == 0.f)) loss += p * (lp + (base - to_float(x[id[j]])) * inv_tau + log_sum);
    prob[j] = p;
  }
  loss = team_reduce<kTeam, false>(loss, part) * a.tau * a.tau;
  if (bad) loss = __builtin_nanf("");
  if (!present) loss = 0.f;
  if (lane == 0) a.row_losses[row] = loss;

  if (kGrad) {
    const float g = (a.row_grad ? a.row_grad[row] : 1.f) * a.tau;
    const float up = bad ? __builtin_nanf("") : g;
    const float inv_sum = 1.f / sum;
    T* d = static_cast<T*>(a.dlogits) + row * a.dlogits_stride;
    // the teacher's entries first (from logits that an update in place is about to overwrite),
    // held by the threads that own them, written once the row's other entries are
    float fix[(1024 + kTeam - 1) / kTeam];
#pragma unroll
    for (int i = 0; i < (1024 + kTeam - 1) / kTeam; ++i) {
      const int j = lane + i * kTeam;
      fix[i] = 0.f;
      if (j < k && id[j] >= 0 && id[j] < V) {
        float p = 0.f;
        for (int o = 0; o < k; ++o) p += id[o] == id[j] ? prob[o] : 0.f;
        fix[i] = up * (__builtin_amdgcn_exp2f((to_float(x[id[j]]) - base) * scale) * inv_sum - p);
      }
    }
    team_sync<kTeam>();
    for (int v = lane; v < V; v += kTeam)
      d[v] = from_float<T>(present ? up * (__builtin_amdgcn_exp2f((to_float(x[v]) - base) * scale) * inv_sum) : 0.f);
    team_sync<kTeam>();
    if (present) {
#pragma unroll
      for (int i = 0; i < (1024 + kTeam - 1) / kTeam; ++i) {
        const int j = lane + i * kTeam;
        if (j < k && id[j] >= 0 && id[j] < V) d[id[j]] = from_float<T>(fix[i]);
      }
    }
  }
}

// losses[m]: mean over the scored rows of model m, in a fixed order, in double. One workgroup a model.
static __global__ __launch_bounds__(256) void k_distill_mean(const float* __restrict__ row_losses, const int32_t* __restrict__ ids,
                                                      const float* __restrict__ teacher, int top_k, int64_t rows_per_model,
                                                      float* __restrict__ losses) {
  __shared__ double part[256];
  __shared__ double cnt[256];
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * rows_per_model;
  double s = 0.0, n = 0.0;
  for (int64_t i = threadIdx.x; i < rows_per_model; i += 256) {
    const int64_t r = r0 + i;
    s += static_cast<double>(row_losses[r]);
    int have = 0;
    for (int j = 0; j < top_k && !have; ++j)
      have = ids[r * top_k + j] >= 0 && !(teacher[r * top_k + j] == -__builtin_inff());
    n += have;
  }
  part[threadIdx.x] = s;
  cnt[threadIdx.x] = n;
  __syncthreads();
  for (int w = 128; w > 0; w >>= 1) {
    if (static_cast<int>(threadIdx.x) < w) {
      part[threadIdx.x] += part[threadIdx.x + w];
      cnt[threadIdx.x] += cnt[threadIdx.x + w];
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) losses[blockIdx.x] = static_cast<float>(part[0] / cnt[0]);
}

}  // namespace cdrge
