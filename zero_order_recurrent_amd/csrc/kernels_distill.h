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

// kN sums or maxima over the kTeam threads that share a row. part: kN * kTeam / 64 floats of LDS
// that no other reduction of the row uses, so that one barrier does.
template <int kTeam, bool kMax, int kN>
__device__ __forceinline__ void team_reduce(float (&v)[kN], float* part) {
#pragma unroll
  for (int m = (kTeam < 64 ? kTeam : 64) / 2; m > 0; m >>= 1)
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      const float o = __shfl_xor(v[n], m);
      v[n] = kMax ? fmaxf(v[n], o) : v[n] + o;
    }
  if (kTeam <= 64) return;
  constexpr int kWaves = kTeam / 64;
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int n = 0; n < kN; ++n) part[n * kWaves + (threadIdx.x >> 6)] = v[n];
  __syncthreads();
#pragma unroll
  for (int n = 0; n < kN; ++n) {
    v[n] = part[n * kWaves + (threadIdx.x & (kWaves - 1))];
#pragma unroll
    for (int m = kWaves / 2; m > 0; m >>= 1) {
      const float o = __shfl_xor(v[n], m);
      v[n] = kMax ? fmaxf(v[n], o) : v[n] + o;
    }
  }
}

// Orders the team's memory accesses before it against those after it (a team of at most one wave
// runs in step).
template <int kTeam>
__device__ __forceinline__ void team_sync() {
  if (kTeam <= 64) {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
    __builtin_amdgcn_wave_barrier();
  } else {
    __syncthreads();
  }
}

// A row as pieces of 16 bytes, wherever it starts (global memory takes such accesses at any element's
// alignment). Sums group by piece, so a row's results do not depend on where it lies. Elements past
// the row's end read as minus infinity and are neither loaded nor stored.
template <class T>
struct DistillRow {
  static constexpr int kPer = 16 / sizeof(T);
  int V, pieces;
  __device__ __forceinline__ DistillRow(int vocab) : V(vocab), pieces((vocab + kPer - 1) / kPer) {}
  // kOnce: the row is read only this once, past the caches.
  template <bool kOnce = false>
  __device__ __forceinline__ uint4 load(const T* x, int b) const {
    uint4 r;
    if ((b + 1) * kPer <= V) {
      if (kOnce)
        load_once(r, x + b * kPer);
      else
        __builtin_memcpy(&r, x + b * kPer, 16);
      return r;
    }
    T e[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) e[i] = b * kPer + i < V ? x[b * kPer + i] : from_float<T>(-__builtin_inff());
    __builtin_memcpy(&r, e, 16);
    return r;
  }
  __device__ __forceinline__ void store(T* d, int b, uint4 r) const {
    if ((b + 1) * kPer <= V) {
      store_once(d + b * kPer, r);
      return;
    }
    T e[kPer];
    __builtin_memcpy(e, &r, 16);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (b * kPer + i < V) d[b * kPer + i] = e[i];
  }
};

template <class T>
__device__ __forceinline__ void piece_max(uint4 r, float& m) {
  T e[16 / sizeof(T)];
  __builtin_memcpy(e, &r, 16);
#pragma unroll
  for (int i = 0; i < int(16 / sizeof(T)); ++i) m = fmaxf(m, to_float(e[i]));
}
template <class T>
__device__ __forceinline__ float piece_sum(uint4 r, float most, float scale) {
  T e[16 / sizeof(T)];
  __builtin_memcpy(e, &r, 16);
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < int(16 / sizeof(T)); ++i) s += __builtin_amdgcn_exp2f((to_float(e[i]) - most) * scale);
  return s;
}
template <class T>
__device__ __forceinline__ uint4 piece_grad(uint4 r, float most, float scale, float up) {
  T e[16 / sizeof(T)];
  __builtin_memcpy(e, &r, 16);
#pragma unroll
  for (int i = 0; i < int(16 / sizeof(T)); ++i)
    e[i] = from_float<T>(up * __builtin_amdgcn_exp2f((to_float(e[i]) - most) * scale));
  __builtin_memcpy(&r, e, 16);
  return r;
}

constexpr int distill_threads(int team) { return team < 256 ? 256 : team; }

// Waves a SIMD should hold: rows wait for memory, then for each other's sums, so several have to be in flight.
constexpr int distill_waves(int team, int pieces) { return team <= 64 ? 4 : (pieces == 8 && team < 1024 ? 6 : 8); }

// One row by kTeam threads. kPieces > 0: the row stays in registers, kPieces pieces a thread, and is
// read once. kPieces = 0 (rows too long for that): the row is read again, from the caches, for the sum and for the
// gradient. Otherwise reads and writes go past the caches: 4,096 rows of 32,768 in bf16, loss and gradient, take 109 us
// (4.9 TB/s; 117 through the caches), 301 rows of 30,011 in float32 19.9 us (21.8), 10,240 rows of 50 7.2 us, of which
// two launches.
template <class T, bool kGrad, int kTeam, int kPieces>
__global__ __launch_bounds__(distill_threads(kTeam), distill_waves(kTeam, kPieces)) void k_distill(DistillArgs a) {
  extern __shared__ float lds[];  // per row of the workgroup: kPad probabilities, as many ids
  __shared__ float part[3 * 4 * 16];
  constexpr int kRows = distill_threads(kTeam) / kTeam;
  constexpr int kOwn = (kTeam == 16 ? 256 : 1024 + kTeam - 1) / kTeam;  // teacher entries of a thread
  const int lane = threadIdx.x % kTeam, team = threadIdx.x / kTeam;
  const int64_t row = block_number() * kRows + team;
  if (row >= a.n_rows) return;  // whole teams, of one wave at most, which wait for nobody below
  const int V = a.vocab, k = a.top_k, k4 = (k + 3) & ~3;
  float* prob = lds + 2 * team * k4;
  int* id = reinterpret_cast<int*>(prob + k4);
  const T* x = static_cast<const T*>(a.logits) + row * a.logits_stride;
  const DistillRow<T> at(V);
  const float inv_tau = 1.f / a.tau, scale = 1.44269504088896340736f / a.tau;
  const float ninf = -__builtin_inff();

  uint4 held[kPieces > 0 ? kPieces : 1];
  if (kPieces > 0) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int b = lane + i * kTeam;
      if (b < at.pieces) held[i] = at.template load<true>(x, b);
    }
  }

  // the teacher's and the student's largest logits, whether an entry is present, whether one is bad
  float most[4] = {ninf, ninf, 0.f, 0.f};
  for (int j = lane; j < k4; j += kTeam) {
    const int v = j < k ? a.ids[row * k + j] : -1;
    const float t = j < k ? a.teacher[row * k + j] : ninf;
    const bool have = v >= 0 && !(t == ninf);
    id[j] = have ? v : -1;
    prob[j] = t;
    if (have) {
      most[0] = fmaxf(most[0], t);
      most[2] = 1.f;
      if (v >= V) most[3] = 1.f;
    }
  }
  if (kPieces > 0) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      if (lane + i * kTeam < at.pieces) piece_max<T>(held[i], most[1]);
  } else {
    for (int b = lane; b < at.pieces; b += kTeam) piece_max<T>(at.load(x, b), most[1]);
  }
  team_reduce<kTeam, true, 4>(most, part);
  const bool present = most[2] > 0.f, bad = most[3] > 0.f;
  const float tmax = most[0];
  // Logits enter as (x - M) scale, in units of log 2, the largest at zero. As x scale - M scale, one instruction less,
  // all would be off by the rounding of M scale, which at |M| / tau of 2^31 passes the exponents' whole range.
  const float top = most[1] == ninf ? 0.f : most[1];

  float sums[2] = {0.f, 0.f};  // the student's exponentials, the teacher's
  if (kPieces > 0) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      if (lane + i * kTeam < at.pieces) sums[0] += piece_sum<T>(held[i], top, scale);
      __builtin_amdgcn_sched_barrier(0);  // piece by piece: temporaries of one, not of all
    }
  } else {
    for (int b = lane; b < at.pieces; b += kTeam) sums[0] += piece_sum<T>(at.load(x, b), top, scale);
  }
  for (int j = lane; j < k; j += kTeam) sums[1] += id[j] >= 0 ? expf((prob[j] - tmax) * inv_tau) : 0.f;
  team_reduce<kTeam, false, 2>(sums, part + 4 * 16);
  const float log_sum = logf(sums[0]), log_mass = logf(sums[1]);

  float loss[1] = {0.f}, mine[kOwn];  // mine: (x - M) scale at this thread's teacher entries
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const int j = lane + i * kTeam;
    if (j >= k) continue;
    const float lp = (prob[j] - tmax) * inv_tau - log_mass;
    const float p = id[j] >= 0 ? expf(lp) : 0.f;
    if (id[j] >= 0 && id[j] < V) {
      mine[i] = (to_float(x[id[j]]) - top) * scale;
      // a probability that underflows contributes its limit, zero
      if (!(p == 0.f)) loss[0] += p * (lp - mine[i] * 0.693147180559945309417f + log_sum);
    }
    prob[j] = p;
  }
  team_reduce<kTeam, false, 1>(loss, part + 8 * 16);
  // rows that are not scored are marked for the mean by the sign of their zero
  if (lane == 0) a.row_losses[row] = !present ? -0.f : (bad ? __builtin_nanf("") : loss[0] * a.tau * a.tau + 0.f);

  if (kGrad) {
    T* d = static_cast<T*>(a.dlogits) + row * a.dlogits_stride;
    if (!present) {
      for (int b = lane; b < at.pieces; b += kTeam) at.store(d, b, make_uint4(0, 0, 0, 0));
      return;  // for the whole team
    }
    const float up = bad ? __builtin_nanf("") : (a.row_grad ? a.row_grad[row] : 1.f) * a.tau;
    const float up_q = up / sums[0];
    // every read of the row at the teacher's ids is done (they lie before the last reduction, and in
    // `mine`), so an update in place may begin; the teacher's entries are written over it afterwards
    if (kPieces > 0) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int b = lane + i * kTeam;
        if (b < at.pieces) at.store(d, b, piece_grad<T>(held[i], top, scale, up_q));
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
      for (int b = lane; b < at.pieces; b += kTeam) at.store(d, b, piece_grad<T>(at.load(x, b), top, scale, up_q));
    }
    team_sync<kTeam>();
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int j = lane + i * kTeam;
      if (j >= k || id[j] < 0 || id[j] >= V) continue;
      const int v = id[j];
      float p = 0.f;  // an id that comes twice has the sum, whoever writes it
      for (int o = 0; o < k4; o += 4) {
        const int4 io = *reinterpret_cast<const int4*>(id + o);
        const float4 po = *reinterpret_cast<const float4*>(prob + o);
        p += (io.x == v ? po.x : 0.f) + (io.y == v ? po.y : 0.f) + (io.z == v ? po.z : 0.f) + (io.w == v ? po.w : 0.f);
      }
      d[v] = from_float<T>(up_q * __builtin_amdgcn_exp2f(mine[i]) - up * p);
    }
  }
}

// losses[m]: mean over the scored rows of model m, in a fixed order, in double. One workgroup a model.
static __global__ __launch_bounds__(256) void k_distill_mean(const float* __restrict__ row_losses, int64_t rows_per_model,
                                                             float* __restrict__ losses) {
  __shared__ double part[256];
  __shared__ int cnt[256];
  const float* r = row_losses + static_cast<int64_t>(blockIdx.x) * rows_per_model;
  double s = 0.0;
  int n = 0;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < rows_per_model; i += 256) {
    const float v = r[i];
    s += static_cast<double>(v);
    n += __float_as_uint(v) != 0x80000000u;
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
  if (threadIdx.x == 0) losses[blockIdx.x] = static_cast<float>(part[0] / static_cast<double>(cnt[0]));
}

}  // namespace cdrge
