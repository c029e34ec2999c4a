// Log probabilities of given tokens, entropy and the top alternatives, or the gradient of the former two.
//
// With M the row's largest logit, d_v = (logit_v - M) / tau and S1 = sum_v exp(d_v) - 1, in which the largest logit
// itself is left out and not subtracted again:
//   log p_v = d_v - log1p(S1),   entropy = log1p(S1) - sum_v exp(d_v) d_v / (1 + S1),
// sums of terms of one sign, so that what a sure row has left over keeps its bits. The work is one read of the logits
// (and one write of the gradient): bound by memory.
#pragma once
#include <type_traits>

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

// The largest of three, or NaN if there is one among them.
__device__ __forceinline__ float score_most(float a, float b, float c) {
  return __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, b), c);
}

// LDS of a row: the candidates, the threads' largest logits, how many candidates there are and their bound.
__host__ __device__ constexpr size_t score_lds(int cap, int team) { return size_t(8) * cap + 4 * team + 16; }

// Waves a SIMD should hold; see distill_waves. 16 pieces take 64 registers.
constexpr int score_waves(int team, int pieces) { return pieces == 16 ? 4 : distill_waves(team, pieces); }

enum ScoreMode { kScoreOnly, kScoreTop, kScoreGrad };  // what a launch writes: no alternatives, those too, the gradient

// One row by kTeam threads, in registers or, with kPieces = 0, read again for each pass (as in k_distill). 4,096 rows of
// 32,768 bf16 logits: 70 us (3.8 TB/s), of which the exponentials' instructions overlap the reading; with 64 alternatives 104;
// gradient 112 (4.8 TB/s); in float32 98, 209 and 193. 10,240 rows of 50 float32 logits: 7.0 us with five alternatives; 48 rows
// of 32,768 with 20: 14 us, a row's latency. Rows of more than 16 pieces for each of 1,024 threads are read up to three times, by
// one CU each: 64 rows of 300,007 bf16 logits with 20 alternatives 71 us, 0.5 TB/s. With alternatives, 1,024 threads with 8
// pieces each (32,769 to 65,536 bf16 logits, half as many in float32, or more than 512 alternatives) keep 14 to 16 registers in
// scratch, 256 and 512 threads of a bf16 row 2.
//
// Alternatives: the k-th largest of the threads' largest logits, or one a little below it, bounds the k largest of all from
// below. What lies above the bound, 1.1 to 1.6 k logits of a row without order, goes into LDS and takes its place by
// counting. Where more lie above it than LDS holds (rows of ties, falling rows) or there are fewer threads than k, the bound
// is searched for by halving the range of logit and id, which ends as all differ.
template <class T, int kMode, int kTeam, int kPieces>
__global__ __launch_bounds__(distill_threads(kTeam), score_waves(kTeam, kPieces)) void k_scores(ScoreArgs a) {
  constexpr bool kGrad = kMode == kScoreGrad;
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
  // f(piece, its number) for each of this thread's pieces. A pass takes pieces and their numbers for new ones: the compiler
  // would otherwise keep all elements, converted by the first pass, and all their places, and spill them.
  auto each = [&](auto f) {
    if (kPieces > 0) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        int b = lane + i * kTeam;
        asm("" : "+v"(held[i].x), "+v"(held[i].y), "+v"(held[i].z), "+v"(held[i].w), "+v"(b));
        if (b < at.pieces) f(held[i], b);
        __builtin_amdgcn_sched_barrier(0);  // piece by piece: temporaries of one, not of all
      }
    } else {
      for (int b = lane; b < at.pieces; b += kTeam) f(at.load(x, b), b);
    }
  };

  float mine = ninf;
  auto top_of = [](uint4 r) {
    T v[kPer];
    __builtin_memcpy(v, &r, 16);
    float m = to_float(v[0]);
#pragma unroll
    for (int e = 1; e + 1 < kPer; e += 2) m = score_most(m, to_float(v[e]), to_float(v[e + 1]));
    return __builtin_elementwise_maximum(m, to_float(v[kPer - 1]));
  };
  // each piece's, which says later where alternatives are
  float piece_top[kMode == kScoreTop && kPieces > 0 ? kPieces : 1];
  if (kPieces > 0) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const float m = lane + i * kTeam < at.pieces ? top_of(held[i]) : ninf;
      if (kMode == kScoreTop) piece_top[i] = m;
      mine = __builtin_elementwise_maximum(mine, m);
    }
  } else {
    each([&](uint4 r, int) { mine = __builtin_elementwise_maximum(mine, top_of(r)); });
  }
  if (!(mine == mine)) mine = __builtin_inff();  // a row with a NaN is as bad as one with plus infinity
  float most[1] = {mine};
  team_reduce<kTeam, true, 1>(most, part);
  const float top = most[0];
  // sum of exponentials and of those times their exponents, without the largest logit; how often that one comes
  float sums[3] = {0.f, 0.f, 0.f};
  auto sum_up = [&](auto has_top) {
    each([&](uint4 r, int) {
      T v[kPer];
      __builtin_memcpy(v, &r, 16);
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const float z = to_float(v[e]);
        const float d = fmaxf((z - top) * scale, -1000.f);  // nothing there in float32, and zero times it is zero
        const float p = __builtin_amdgcn_exp2f(d);
        sums[1] += p * d;
        if (decltype(has_top)::value) {
          sums[0] += z == top ? 0.f : p;
          sums[2] += z == top ? 1.f : 0.f;
        } else {
          sums[0] += p;
        }
      }
    });
  };
  // few threads hold the largest logit and have to look for it
  if (mine == top)
    sum_up(std::true_type{});
  else
    sum_up(std::false_type{});
  team_reduce<kTeam, false, 3>(sums, part + 2 * 16);
  constexpr float kLn2 = 0.693147180559945309417f;
  const float rest = sums[0] + (sums[2] - 1.f), total = 1.f + rest, log_total = log1pf(rest);
  const bool bad = !(fabsf(top) < __builtin_inff()) || !(rest < __builtin_inff());
  const float apart = -kLn2 * (sums[1] / total);  // the mean distance from the largest: log p_v + entropy = d_v + apart
  const float entropy = bad ? nan : log_total + apart;
  const float logprob = token < 0 ? 0.f : (bad || !inside ? nan : (chosen - top) * inv_tau - log_total);

  if (kGrad) {
    const bool spoilt = bad || (up_l != 0.f && !inside);
    // -p (up_l + up_h (log p + entropy)) / tau, without log_total, in which the distances of a flat row would be lost
    const float c0 = spoilt ? nan : -inv_tau / total * (up_l + up_h * apart), c1 = -inv_tau / total * up_h * kLn2;
    each([&](uint4 r, int b) {
      T v[kPer];
      __builtin_memcpy(v, &r, 16);
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const float d = fmaxf((to_float(v[e]) - top) * scale, -1000.f);
        v[e] = from_float<T>(__builtin_amdgcn_exp2f(d) * (c0 + c1 * d));
      }
      __builtin_memcpy(&r, v, 16);
      at.store(dx, b, r);
    });
    // the given token's, by the thread that has just written its piece: 1 - p is not formed by subtraction
    if (inside && !spoilt && up_l != 0.f && lane == token / kPer % kTeam)
      dx[token] = from_float<T>(-inv_tau * (up_l * expm1f(logprob) + up_h * expf(logprob) * (logprob == ninf ? 0.f : (chosen - top) * inv_tau + apart)));
    return;
  }
  if (lane == 0) {
    if (a.logprobs) a.logprobs[row] = logprob;
    if (a.entropy) a.entropy[row] = entropy;
  }
  if (kMode != kScoreTop) return;

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
  float* const thread_most = reinterpret_cast<float*>(base + size_t(8) * a.cap);
  int* const count = reinterpret_cast<int*>(thread_most + kTeam);
  float* const bound = reinterpret_cast<float*>(count + 1);
  thread_most[lane] = mine;
  if (lane == 0) {
    *count = 0;
    *bound = ninf;
  }
  team_sync<kTeam>();
  if (kTeam < 64 && kTeam >= k) {
    int rank = 0;
#pragma unroll
    for (int o = 0; o < kTeam; ++o) rank += thread_most[o] > mine || (thread_most[o] == mine && o < lane);
    if (rank == k - 1) *bound = mine;
  } else if (kTeam >= k && lane < 64) {
    // one wave halves the range of their keys until k of them, or some more, are above the bound
    constexpr int kOwn = kTeam < 64 ? 1 : kTeam / 64;
    uint32_t own[kOwn], least = ~0u;
#pragma unroll
    for (int n = 0; n < kOwn; ++n) {
      own[n] = static_cast<uint32_t>(score_key(thread_most[n * 64 + lane], 0) >> 32);
      least = min(least, own[n]);
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) least = min(least, static_cast<uint32_t>(__shfl_xor(static_cast<int>(least), m)));
    uint32_t lo = __builtin_amdgcn_readfirstlane(least), hi = static_cast<uint32_t>(score_key(top, 0) >> 32);
    while (lo < hi) {  // at least k have `lo`; more than `hi` has none
      const uint32_t mid = lo + (hi - lo) / 2 + 1;
      int c = 0;
#pragma unroll
      for (int n = 0; n < kOwn; ++n) c += __popcll(__ballot(own[n] >= mid));
      if (c >= k) lo = mid;
      else hi = mid - 1;
      if (c >= k && c <= k + k / 4 + 4) break;
    }
    if (lane == 0) *bound = score_value(static_cast<uint64_t>(lo) << 32);
  }
  team_sync<kTeam>();
  const float floor = fmaxf(*bound, -3.402823466e38f);  // minus infinity is no alternative
  // f(piece, its number) for those of this thread's pieces that have an element of `floor` or above, few of all
  auto each_hit = [&](auto f) {
    if (kPieces > 0) {
      uint32_t hits = 0;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) hits |= piece_top[i] >= floor ? 1u << i : 0u;
      while (hits) {
        const int i = __builtin_ctz(hits);
        hits &= hits - 1;
        uint4 r = make_uint4(0, 0, 0, 0);  // held[i], picked out bit by bit: an index would put the row into memory
#pragma unroll
        for (int o = 0; o < kPieces; ++o) {
          const uint32_t is = i == o ? ~0u : 0u;
          r = make_uint4(r.x | (held[o].x & is), r.y | (held[o].y & is), r.z | (held[o].z & is), r.w | (held[o].w & is));
        }
        f(r, lane + i * kTeam);
      }
    } else {
      for (int b = lane; b < at.pieces; b += kTeam) {
        const uint4 r = at.load(x, b);
        if (top_of(r) >= floor) f(r, b);
      }
    }
  };
  // as many as `least` or above may be more than LDS holds, as many as `past` or above are less than k
  uint64_t least = 0, past = score_key(top, -1) | 0xffffffffu;
  auto key_of = [&](T v, int id) {  // zero for what is no candidate
    const uint64_t key = score_key(to_float(v), id);
    return to_float(v) >= floor && key >= least ? key : 0;
  };
  int n;
  while (true) {
    each_hit([&](uint4 r, int b) {
      T v[kPer];
      __builtin_memcpy(v, &r, 16);
      uint64_t key[kPer];
      int own = 0;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        key[e] = key_of(v[e], b * kPer + e);
        own += key[e] != 0;
      }
      int to = atomicAdd(count, own);
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        if (key[e] != 0 && to < a.cap) cand[to] = key[e];
        to += key[e] != 0;
      }
    });
    team_sync<kTeam>();
    n = *count;
    if (n <= a.cap) break;
    if (least == 0) least = score_key(floor, -1);
    do {
      const uint64_t mid = least + (past - least) / 2;
      float c[1] = {0.f};
      each_hit([&](uint4 r, int b) {
        T v[kPer];
        __builtin_memcpy(v, &r, 16);
#pragma unroll
        for (int e = 0; e < kPer; ++e) c[0] += key_of(v[e], b * kPer + e) >= mid ? 1.f : 0.f;
      });
      team_sync<kTeam>();  // the last reduction's places are read
      team_reduce<kTeam, false, 1>(c, part + 5 * 16);
      n = static_cast<int>(c[0]);
      (n < k ? past : least) = mid;
    } while (n < k || n > a.cap);
    if (lane == 0) *count = 0;
    team_sync<kTeam>();
  }
  auto put = [&](int rank, uint64_t key) {
    ids[rank] = static_cast<int32_t>(~static_cast<uint32_t>(key));
    lps[rank] = (score_value(key) - top) * inv_tau - log_total;
  };
  if (kTeam < 64) {
    for (int c = lane; c < n; c += kTeam) {
      const uint64_t own = cand[c];
      int rank = 0;
#pragma unroll 8
      for (int o = 0; o < n; ++o) rank += cand[o] > own;
      if (rank < k) put(rank, own);
    }
  } else if (n <= 512) {
    // every wave has all of them, 64 at a time, and counts for its share how many are larger (1,024 rows of 32,768 with 100
    // alternatives: 42 us, sorted 59; with 300, some 400 candidates, 65 and 63)
    constexpr int kWaves = kTeam < 64 ? 1 : kTeam / 64;
    const int l64 = lane & 63, wave = __builtin_amdgcn_readfirstlane(lane >> 6);
    uint64_t all[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) all[j] = 64 * j + l64 < n ? cand[64 * j + l64] : 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (64 * j >= n) break;
      int mine_rank = k;
      for (int l = wave; l < min(64, n - 64 * j); l += kWaves) {
        const uint64_t key = static_cast<uint64_t>(__builtin_amdgcn_readlane(static_cast<int>(all[j] >> 32), l)) << 32 |
                             static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(all[j]), l));
        int rank = 0;
#pragma unroll
        for (int o = 0; o < 8; ++o)
          if (64 * o < n) rank += __popcll(__ballot(all[o] > key));
        if (l64 == l) mine_rank = rank;
      }
      if (mine_rank < k) put(mine_rank, all[j]);
    }
  } else {  // counting takes n^2 steps: many are sorted, as a power of two of them, halves of rising runs merged
    int size = 1024;
    while (size < n) size *= 2;
    for (int c = n + lane; c < size; c += kTeam) cand[c] = 0;
    for (int run = 2; run <= size; run *= 2)
      for (int apart = run / 2; apart > 0; apart /= 2) {
        team_sync<kTeam>();
        for (int i = lane; i < size / 2; i += kTeam) {
          const int c = 2 * i - (i & (apart - 1));
          const uint64_t x0 = cand[c], x1 = cand[c + apart];
          if ((x0 < x1) == ((c & run) == 0)) {
            cand[c] = x1;
            cand[c + apart] = x0;
          }
        }
      }
    team_sync<kTeam>();
    for (int c = lane; c < min(n, k); c += kTeam) put(c, cand[c]);
  }
  for (int j = n + lane; j < k; j += kTeam) {
    ids[j] = -1;
    lps[j] = ninf;
  }
}

}  // namespace cdrge
