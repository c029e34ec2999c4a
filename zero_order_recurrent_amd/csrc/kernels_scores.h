// Log probabilities of given tokens, entropy and the top alternatives, or the gradient of the former two.
//
// With M the row's largest logit, d_v = (logit_v - M) / tau and S1 = sum_v exp(d_v) - 1, in which the largest logit
// itself is left out and not subtracted again:
//   log p_v = d_v - log1p(S1),   entropy = log1p(S1) - sum_v exp(d_v) d_v / (1 + S1),
// sums of terms of one sign, so that what a sure row has left over keeps its bits. The work is one read of the logits
// (and one write of the gradient): bound by memory.
#pragma once
#include "kernels_distill.h"

namespace cdrge {

struct ScoreArgs {
  const void* logits;
  int64_t logits_stride;
  const int32_t* tokens;
  float* logprobs;
  float* entropy;
  int32_t* top_ids;
  float* top_logprobs;
  const float* d_logprob;
  const float* d_entropy;
  void* dlogits;
  int64_t dlogits_stride;
  int64_t n_rows;
  int vocab, top_k, cap;
  float tau;
};

// An alternative's place in the order: its logit, then its id from the lowest on. Larger is earlier; all differ.
__device__ __forceinline__ uint64_t score_key(float x, int id) {
  const uint32_t bits = __float_as_uint(x + 0.f);  // both zeros are one
  const uint32_t up = bits & 0x80000000u ? ~bits : bits | 0x80000000u;
  return static_cast<uint64_t>(up) << 32 | static_cast<uint32_t>(~id);
}
__device__ __forceinline__ float score_value(uint64_t key) {
  const uint32_t up = static_cast<uint32_t>(key >> 32);
  return __uint_as_float(up & 0x80000000u ? up & 0x7fffffffu : ~up);
}

// LDS of a row: the candidates, the groups' largest logits, how many candidates there are and their bound.
__host__ __device__ constexpr size_t score_lds(int cap, int team) { return size_t(8) * cap + 4 * team + 16; }

// One row by kTeam threads, in registers or, with kPieces = 0, read again for each pass (as in k_distill).
//
// Alternatives: the threads form at least 2 k groups where they are that many, and the k-th largest of the groups'
// largest logits bounds the k largest of all from below. What lies above the bound, 1.4 k logits of a row without order,
// goes into LDS and takes its place by counting. Where more lie above it than LDS holds (rows of ties, falling rows) or
// there are fewer threads than k, the bound is searched for by halving the range of logit and id, which ends as all
// differ.
template <class T, bool kGrad, int kTeam, int kPieces>
__global__ __launch_bounds__(distill_threads(kTeam), distill_waves(kTeam, kPieces)) void k_scores(ScoreArgs a) {
  extern __shared__ __align__(16) char lds[];
  __shared__ float part[(2 + 3 + 1 + 1) * 16];
  constexpr int kRows = distill_threads(kTeam) / kTeam, kPer = DistillRow<T>::kPer;
  const int lane = threadIdx.x % kTeam, team = threadIdx.x / kTeam;
  const int64_t row = block_number() * kRows + team;
  if (row >= a.n_rows) return;  // whole teams, of one wave at most, which wait for nobody below
  const int V = a.vocab, k = a.top_k;
  const T* x = static_cast<const T*>(a.logits) + row * a.logits_stride;
  T* dx = kGrad ? static_cast<T*>(a.dlogits) + row * a.dlogits_stride : nullptr;
  const DistillRow<T> at(V);
  const float ninf = -__builtin_inff(), nan = __builtin_nanf("");
  const float inv_tau = 1.f / a.tau, scale = 1.44269504088896340736f / a.tau;
  const int token = a.tokens ? a.tokens[row] : -1;
  const bool inside = token >= 0 && token < V;
  const float chosen = inside ? to_float(x[token]) : 0.f;
  float up_l = 0.f, up_h = 0.f;
  if (kGrad) {
    up_l = token >= 0 && a.d_logprob ? a.d_logprob[row] : 0.f;
    up_h = a.d_entropy ? a.d_entropy[row] : 0.f;
    if (up_l == 0.f && up_h == 0.f) {
      for (int b = lane; b < at.pieces; b += kTeam) at.store(dx, b, make_uint4(0, 0, 0, 0));
      return;  // for the whole team
    }
  }

  uint4 held[kPieces > 0 ? kPieces : 1];
  if (kPieces > 0) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int b = lane + i * kTeam;
      if (b < at.pieces) held[i] = at.template load<true>(x, b);
    }
  }
  // f(piece, its number) for each of this thread's pieces
  auto each = [&](auto f) {
    if (kPieces > 0) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        if (lane + i * kTeam < at.pieces) f(held[i], lane + i * kTeam);
        __builtin_amdgcn_sched_barrier(0);  // piece by piece: temporaries of one, not of all
      }
    } else {
      for (int b = lane; b < at.pieces; b += kTeam) f(at.load(x, b), b);
    }
  };

  float most[1] = {ninf};
  each([&](uint4 r, int) { piece_max<T>(r, most[0]); });
  const float mine = most[0];
  team_reduce<kTeam, true, 1>(most, part);
  const float top = most[0];
  // sum of exponentials and of those times their exponents, without the largest logit; how often that one comes
  float sums[3] = {0.f, 0.f, 0.f};
  each([&](uint4 r, int) {
    T v[kPer];
    __builtin_memcpy(v, &r, 16);
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const float z = to_float(v[e]);
      float d = (z - top) * scale;
      d = d < -1000.f ? -1000.f : d;  // nothing there in float32; keeps NaN, and zero times it is zero
      const float p = __builtin_amdgcn_exp2f(d);
      sums[0] += z == top ? 0.f : p;
      sums[1] += p * d;
      sums[2] += z == top ? 1.f : 0.f;
    }
  });
  team_reduce<kTeam, false, 3>(sums, part + 2 * 16);
  constexpr float kLn2 = 0.693147180559945309417f;
  const float rest = sums[0] + (sums[2] - 1.f), total = 1.f + rest, log_total = log1pf(rest);
  const bool bad = !(fabsf(top) < __builtin_inff()) || !(rest < __builtin_inff());
  const float entropy = bad ? nan : log_total - kLn2 * (sums[1] / total);
  const float logprob = token < 0 ? 0.f : (bad || !inside ? nan : (chosen - top) * inv_tau - log_total);

  if (kGrad) {
    const bool spoilt = bad || (up_l != 0.f && !inside);
    // -p (up_l + up_h (log p + entropy)) / tau, with log p = d ln 2 - log_total
    const float c0 = spoilt ? nan : -inv_tau / total * (up_l + up_h * (entropy - log_total)), c1 = -inv_tau / total * up_h * kLn2;
    each([&](uint4 r, int b) {
      T v[kPer];
      __builtin_memcpy(v, &r, 16);
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        float d = (to_float(v[e]) - top) * scale;
        d = d < -1000.f ? -1000.f : d;
        v[e] = from_float<T>(__builtin_amdgcn_exp2f(d) * (c0 + c1 * d));
      }
      __builtin_memcpy(&r, v, 16);
      at.store(dx, b, r);
    });
    // the given token's, by the thread that has just written its piece: 1 - p is not formed by subtraction
    if (inside && !spoilt && up_l != 0.f && lane == token / kPer % kTeam)
      dx[token] = from_float<T>(-inv_tau * (up_l * expm1f(logprob) + up_h * expf(logprob) * (logprob == ninf ? 0.f : logprob + entropy)));
    return;
  }
  if (lane == 0) {
    if (a.logprobs) a.logprobs[row] = logprob;
    if (a.entropy) a.entropy[row] = entropy;
  }
  if (k == 0) return;

  int32_t* const ids = a.top_ids + row * k;
  float* const lps = a.top_logprobs + row * k;
  if (bad) {
    for (int j = lane; j < k; j += kTeam) {
      ids[j] = -1;
      lps[j] = nan;
    }
    return;
  }
  char* const base = lds + team * score_lds(a.cap, kTeam);
  uint64_t* const cand = reinterpret_cast<uint64_t*>(base);
  float* const group_most = reinterpret_cast<float*>(base + size_t(8) * a.cap);
  int* const count = reinterpret_cast<int*>(group_most + kTeam);
  float* const bound = reinterpret_cast<float*>(count + 1);
  int size = 1;  // threads of a group
  while (size < 64 && size < kTeam && kTeam / (2 * size) >= 2 * k) size *= 2;
  const int groups = kTeam / size;
  float gm = mine;
  for (int m = 1; m < size; m <<= 1) gm = fmaxf(gm, __shfl_xor(gm, m));
  if (lane % size == 0) group_most[lane / size] = gm;
  if (lane == 0) {
    *count = 0;
    *bound = ninf;
  }
  team_sync<kTeam>();
  if (groups >= k && lane < groups) {
    const float own = group_most[lane];
    int rank = 0;
    for (int o = 0; o < groups; ++o) rank += group_most[o] > own || (group_most[o] == own && o < lane);
    if (rank == k - 1) *bound = own;
  }
  team_sync<kTeam>();
  const float floor = *bound;
  auto collect = [&](uint64_t least) {
    each([&](uint4 r, int b) {
      T v[kPer];
      __builtin_memcpy(v, &r, 16);
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const float z = to_float(v[e]);
        if (z >= floor && z > ninf) {
          const uint64_t key = score_key(z, b * kPer + e);
          if (key >= least) {
            const int n = atomicAdd(count, 1);
            if (n < a.cap) cand[n] = key;
          }
        }
      }
    });
  };
  collect(0);
  team_sync<kTeam>();
  int n = *count;
  if (n > a.cap) {
    uint64_t lo = score_key(floor == ninf ? -3.402823466e38f : floor, -1), hi = score_key(top, -1) | 0xffffffffu;
    // as many as `lo` or above are more than LDS holds, as many as `hi` or above less than k
    while (n < k || n > a.cap) {
      const uint64_t mid = lo + (hi - lo) / 2;
      float c[1] = {0.f};
      each([&](uint4 r, int b) {
        T v[kPer];
        __builtin_memcpy(v, &r, 16);
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          const float z = to_float(v[e]);
          c[0] += z >= floor && z > ninf && score_key(z, b * kPer + e) >= mid ? 1.f : 0.f;
        }
      });
      team_sync<kTeam>();  // the last reduction's places are read
      team_reduce<kTeam, false, 1>(c, part + 5 * 16);
      n = static_cast<int>(c[0]);
      if (n > a.cap) lo = mid;
      else if (n < k) hi = mid;
      else lo = mid;
    }
    if (lane == 0) *count = 0;
    team_sync<kTeam>();
    collect(lo);
    team_sync<kTeam>();
    n = *count;
  }
  for (int c = lane; c < n; c += kTeam) {
    const uint64_t own = cand[c];
    int rank = 0;
    for (int o = 0; o < n; ++o) rank += cand[o] > own;
    if (rank < k) {
      ids[rank] = static_cast<int32_t>(~static_cast<uint32_t>(own));
      lps[rank] = (score_value(own) - top) * inv_tau - log_total;
    }
  }
  for (int j = n + lane; j < k; j += kTeam) {
    ids[j] = -1;
    lps[j] = ninf;
  }
}

}  // namespace cdrge
