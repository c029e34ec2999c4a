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
  int short_len;  // prompts: k_delta_tokens takes sequences of up to so many tokens, the kernels of blocks longer ones
};

__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + expf(-x)); }

// What brings a row of the sum of squares ss to length one; a sum past float32 makes the row NaN.
__device__ __forceinline__ float delta_norm(float ss, float eps) {
  return ss < __builtin_inff() ? __builtin_amdgcn_rsqf(ss + eps) : __builtin_nanf("");  // off by 2^-23 at most
}

// Sum over kLanes (4, 8 or 16) lanes side by side, in each of them.
template <int kControl>
__device__ __forceinline__ float add_lane(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kControl, 0xf, 0xf, true));
}
template <int kLanes>
__device__ __forceinline__ float lanes_sum(float v) {
  v = add_lane<0xb1>(v);                   // lane ^ 1
  v = add_lane<0x4e>(v);                   // lane ^ 2
  if (kLanes > 4) v = add_lane<0x141>(v);  // half-row mirror
  if (kLanes > 8) v = add_lane<0x140>(v);  // row mirror
  return v;
}

// What a thread reads of a token: four entries each of q and k from column 4 (its lane + kLanes n) on, kRpt of v.
template <class T, int kQuads, int kRpt>
struct DeltaToken {
  Four<T> q[kQuads], k[kQuads];
  T v[kRpt];
};

// Token after token, with the state in registers: kLanes lanes side by side hold 4 kQuads of its columns each, a thread
// kRpt of its rows. One token for each sequence (kStep) is bound by memory, which the state crosses twice, past the caches;
// all that is read is requested together, the check for a repeated slot beside it. 256 rows, 32 heads of 128 x 128, bf16:
// 196 us, 5.4 TB/s; one row of 8 heads: 4.2 us, a launch and two loads one after the other. In prompts a token is requested
// while the one before it is worked on, and 64 tokens' gates are formed at a time, a token a thread: bound by the sums over
// lanes, 29 us for a token of 256 sequences of the same sizes.
// With S the state before a token, its prediction of v is a S k' and y = a S q' + (k'.q') b (v - a S k'), so that both
// products of S run before its update, and, as the norms are factors, beside theirs.
template <class T, int kLanes, int kQuads, int kRpt, bool kStep>
__global__ __launch_bounds__(256) void k_delta_tokens(DeltaArgs a, ScanWork w) {
  constexpr int kTile = 256 / kLanes * kRpt;
  __shared__ float2 gates[64];
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
  } else {
    const ScanSeq sq = scan_seq(s, w, i);
    first = sq.first;
    len = sq.len;
    if (len > a.short_len) return;
    if (s.ssm_in) {
      slot = s.owned ? w.slots[i] : scan_slot(s, i);
      taken = slot == -2;
      if (slot >= 0 && s.positions) pos = max(s.positions[i], 0);
    }
  }
  y += first * s.y_stride;
  const int N = s.N, g = h / (s.H / s.G);
  const int ln = tid % kLanes, n0 = ln * 4, have = N - n0, r0 = tid / kLanes * kRpt;
  const bool vec = N % 4 == 0, held = slot >= 0 && !(kStep && slot >= s.n_slots);
  const int64_t sbase = (static_cast<int64_t>(held ? slot : 0) * s.H + h) * s.P + p0;
  f32x4 st[kRpt][kQuads];
#pragma unroll
  for (int r = 0; r < kRpt; ++r)
#pragma unroll
    for (int n = 0; n < kQuads; ++n) {
      st[r][n] = f32x4{0.f, 0.f, 0.f, 0.f};
      const int left = have - 4 * kLanes * n;
      if (held && pos > 0 && r0 + r < np && left > 0) {
        const float* const from = s.ssm_in + (sbase + r0 + r) * N + n0 + 4 * kLanes * n;
        if (vec) {
          st[r][n] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(from));
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (e < left) st[r][n][e] = from[e];
        }
      }
    }
  const T* const qp = static_cast<const T*>(a.q) + first * a.q_stride + static_cast<int64_t>(g) * N + n0;
  const T* const kp = static_cast<const T*>(a.k) + first * a.k_stride + static_cast<int64_t>(g) * N + n0;
  const T* const vp = static_cast<const T*>(a.v) + first * a.v_stride + static_cast<int64_t>(h) * s.P + p0 + r0;
  const T* const dp = static_cast<const T*>(s.dt) + first * s.dt_stride + h;
  const T* const bp = static_cast<const T*>(a.beta) + first * a.beta_stride + h;
  const float bias = s.dt_bias ? s.dt_bias[h] : 0.f, decay = s.decay[h];
  auto load = [&](int64_t t) {
    DeltaToken<T, kQuads, kRpt> x;
#pragma unroll
    for (int n = 0; n < kQuads; ++n) {
      x.q[n].load(qp + t * a.q_stride + 4 * kLanes * n, have - 4 * kLanes * n);
      x.k[n].load(kp + t * a.k_stride + 4 * kLanes * n, have - 4 * kLanes * n);
    }
#pragma unroll
    for (int r = 0; r < kRpt; ++r) x.v[r] = r0 + r < np ? vp[t * a.v_stride + r] : T(0);
    return x;
  };
  auto gate = [&](int64_t t) {  // the state's fade and the strength
    return make_float2(expf(softplus(to_float(dp[t * s.dt_stride]) + bias) * decay), sigmoid(to_float(bp[t * a.beta_stride])));
  };
  DeltaToken<T, kQuads, kRpt> next;
  if (len > 0) next = load(0);
  float2 only;
  if (kStep) {
    only = gate(0);
    taken = __syncthreads_or(taken);
  }
  if (taken) {
    for (int64_t t = 0; t < len; ++t)
      if (tid < np) y[t * s.y_stride + tid] = from_float<T>(__builtin_nanf(""));
    return;
  }
  for (int t = 0; t < len; ++t) {
    const DeltaToken<T, kQuads, kRpt> x = next;
    if (!kStep) {
      if (t + 1 < len) next = load(t + 1);
      if (t % 64 == 0) {
        __syncthreads();
        if (tid < min(64, len - t)) gates[tid] = gate(t + tid);
        __syncthreads();
      }
    }
    const float2 now = kStep ? only : gates[t % 64];
    float qq = 0.f, kk = 0.f, kq = 0.f, sk[kRpt], sq[kRpt];
#pragma unroll
    for (int n = 0; n < kQuads; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float q = x.q[n].at(e), k = x.k[n].at(e);
        qq += q * q;
        kk += k * k;
        kq += k * q;
      }
    qq = lanes_sum<kLanes>(qq);
    kk = lanes_sum<kLanes>(kk);
    kq = lanes_sum<kLanes>(kq);
#pragma unroll
    for (int r = 0; r < kRpt; ++r) {
      sk[r] = sq[r] = 0.f;
#pragma unroll
      for (int n = 0; n < kQuads; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          st[r][n][e] *= now.x;
          sk[r] += st[r][n][e] * x.k[n].at(e);
          sq[r] += st[r][n][e] * x.q[n].at(e);
        }
      sk[r] = lanes_sum<kLanes>(sk[r]);
      sq[r] = lanes_sum<kLanes>(sq[r]);
    }
    const float rq = a.q_scale * delta_norm(qq, a.norm_eps), rk = delta_norm(kk, a.norm_eps);
    float mine = 0.f;
#pragma unroll
    for (int r = 0; r < kRpt; ++r) {
      const float add = now.y * (to_float(x.v[r]) - sk[r] * rk) * rk;
#pragma unroll
      for (int n = 0; n < kQuads; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) st[r][n][e] += add * x.k[n].at(e);
      const float out = (sq[r] + add * kq) * rq;
      if (ln == r) mine = out;
    }
    if (ln < kRpt && r0 + ln < np) y[t * s.y_stride + r0 + ln] = from_float<T>(mine);
  }
  if (slot < 0) return;
#pragma unroll
  for (int r = 0; r < kRpt; ++r)
#pragma unroll
    for (int n = 0; n < kQuads; ++n) {
      const int left = have - 4 * kLanes * n;
      if (r0 + r >= np || left <= 0) continue;
      float* const to = s.ssm_out + (sbase + r0 + r) * N + n0 + 4 * kLanes * n;
      if (vec) {
        __builtin_nontemporal_store(st[r][n], reinterpret_cast<f32x4*>(to));
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e < left) to[e] = st[r][n][e];
      }
    }
}

// ---------------------------------------------------------------------------------------------
// Prompts. With G_i the sum of log decays over a block's tokens up to i, S the state before the block, and K, Q, V the
// block's rows as they come (k' = r k, q' = s q), what the tokens write, N, solves a triangular system:
//
//   N_i = b_i (v_i - e^G_i S k'_i - sum_{j < i} e^(G_i - G_j) (k'_i.k'_j) N_j)
//   N = T diag(b) (V - diag(e^G r) K S^T),  T = (1 + L)^-1,  L_ij = b_i e^(G_i - G_j) k'_i.k'_j  (j < i)
//
// and with N' = diag(r) N, U = diag(r) T diag(b), P_ij = e^(G_i - G_j) s_i q_i.k_j (j <= i):
//
//   N' = U (V - diag(e^G r) K S^T),  Y = diag(e^G s) Q S^T + P N',  S' = e^G_last S + (diag(e^(G_last - G)) N')^T K
//
// k_delta_blocks forms U, P and the factors for all blocks at once, and K and Q as operands where they are not such as
// they lie; k_delta_heads walks a sequence's blocks for 16 values of one head. Four of its waves share the keys and hold S
// in their registers; what a block's products leave is joined through LDS three times: the waves' parts of K S^T, V's
// rest, and N'. Four further waves form y from S and N', beside that chain.
//
// Operands of the matrix cores are bf16 (K, Q of bf16 tensors as they are), others the sum of three bf16 parts, which
// hold 24 bits whatever the magnitude; of two such operands the six products that reach 2^-24 are taken. So is y in bf16,
// which comes out as a neighbour of the value nearest to the exact one in 0.014 % of its elements, 2.4e-5 of y in the 2-norm,
// as for single tokens. With two parts for what y is formed of that was 0.33 % and 1.2e-4, and one sequence of 8,192 tokens
// (below) took 343 us instead of 368, 32 of 512 632 instead of 649. Parts end where float32 does: magnitudes past 2^100 may
// come out infinite, and below 2^-100 some bits are lost.
//
// Along a reduction the order is free if both operands have it, and so is that of a result's rows. Keys: entry e of lane
// group q is key 8 q + e of 32, and row m of a state's tile t is key 8 (m / 4) + 4 t + m % 4. Tokens: entry e of lane
// group q is token 16 (e / 4) + 4 q + e % 4. So a product's result is the next one's operand in the lane where it lies.
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ f32x4 mma_bf16(bf16x8 a, bf16x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }

// An operand as the sum of kParts of bf16, two entries to a word.
template <int kParts>
struct Parts {
  uint32_t w[kParts][4];
  __device__ __forceinline__ void set(int pair, float v0, float v1) {
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      w[p][pair] = bf16_pair(v0, v1);
      if (p + 1 < kParts) asm("" : "+v"(w[p][pair]));  // one conversion, not another for each half
      v0 -= __uint_as_float(w[p][pair] << 16);
      v1 -= __uint_as_float(w[p][pair] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ bf16x8 part(int p) const {
    bf16x8 v;
    __builtin_memcpy(&v, w[p], 16);
    return v;
  }
};

// c[m] + a[m] b for kM operands a, the products of parts that reach 2^-24, small ones first. Products with sums of their own
// stand next to each other.
template <int kM, int kA>
__device__ __forceinline__ void mma_parts(const bf16x8 (&a)[kM][kA], const Parts<3>& b, f32x4 (&c)[kM]) {
#pragma unroll
  for (int s = 2; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < kA; ++i)
#pragma unroll
      for (int m = 0; m < kM; ++m)
        if (s - i >= 0) c[m] = mma_bf16(a[m][i], b.part(s - i), c[m]);
}

// What k_delta_blocks leaves, as operands of 1 KB (16 bytes a lane).
//   for a block and group  kt     [tile kN / 16][step 2][part]: keys of a state's tile, tokens of the step
//                          k, q   [strip 4][step kN / 32][part]: token 16 strip + l16, keys of the step (not for `direct`)
//   for a block and head   u, p   [pair 6][part]: token 16 strip + l16, tokens of the step; pairs (strip, step) with
//                                 step <= strip / 2, in order
//                          factors: e^G r, e^G s and e^(G_last - G) of 64 tokens each, e^G_last
template <class T, int kN>
struct DeltaBlock {
  static constexpr int kRaw = sizeof(T) == 2 ? 1 : 3;         // parts of K and Q; all other operands have three
  static constexpr int kKeys = 1024 * (kN / 32) * 4 * kRaw;  // of kt, of k and of q
  static constexpr int kOffP = 6 * 3 * 1024, kOffFactors = 2 * kOffP, kHeadBytes = kOffFactors + 1024;
};
__host__ __device__ constexpr int delta_pair(int strip, int step) { return strip + (strip > 2) + step; }

struct DeltaWork {
  char* groups;  // [block][group]
  char* heads;   // [block][head]
  int64_t group_bytes;
  // K and Q in bf16 with rows of 128 keys are operands as they lie: k_delta_heads reads the tensors (one sequence of 8,192
  // tokens, 32 heads of 128 x 128: 368 us, and 399 by way of the workspace). Rows of 256 keys, which are twice the addresses,
  // go by way of it (one of 4,096, 16 heads of 256 x 256: 196 us, and 220 as they lie; one of 8,192, 8 heads: 323 and 388)
  bool direct;
};

constexpr int kDeltaRow = 68;  // floats of a row of a 64 x 64 matrix in LDS

// d = sum over 4 kSteps indices of a[l16][k] b[k][l16 of the result's column], in float32
template <int kSteps>
__device__ __forceinline__ f32x4 mma_lds(const float* a, const float* b, f32x4 d) {
  const int l16 = threadIdx.x & 15, q = threadIdx.x >> 4 & 3;
#pragma unroll
  for (int k = 0; k < kSteps; ++k)
    d = __builtin_amdgcn_mfma_f32_16x16x4f32(a[l16 * kDeltaRow + 4 * k + q], b[(4 * k + q) * kDeltaRow + l16], d, 0, 0, 0);
  return d;
}
__device__ __forceinline__ void store_lds(float* to, f32x4 d, float sign) {
  const int l16 = threadIdx.x & 15, q = threadIdx.x >> 4 & 3;
#pragma unroll
  for (int r = 0; r < 4; ++r) to[(4 * q + r) * kDeltaRow + l16] = sign * d[r];
}

// One block of a head: a wave takes 16 tokens. The first head of a group writes the group's operands. The inverse goes from
// blocks of 16, by substitution in registers, to 32 and 64 by products in float32, as its entries grow with the block where
// keys are alike. 128 blocks of 32 heads of 128 x 128, bf16: 88 us; float32, 160 blocks of 14 heads of 40 x 100: 125 us,
// with six products for one. Bound by its dependent steps and nine barriers, not by memory: LDS holds three workgroups a CU in
// bf16 (two with more than 128 keys) and one in float32.
template <class T, int kN>
__global__ __launch_bounds__(256) void k_delta_blocks(DeltaArgs a, ScanWork w, DeltaWork d) {
  using Block = DeltaBlock<T, kN>;
  constexpr int kRaw = Block::kRaw, kSteps = kN / 32;
  extern __shared__ __align__(16) char lds[];
  bf16x8* const kl = reinterpret_cast<bf16x8*>(lds);  // [strip][step][part][lane]
  float* const lm = reinterpret_cast<float*>(lds + 4 * kSteps * kRaw * 1024);
  float* const tm = lm + 64 * kDeltaRow;
  __shared__ __align__(16) float sg[64], sgl[64], sb[64], srk[64], srq[64];
  const ScanArgs& s = a.s;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l16 = lane & 15, q = lane >> 4;
  const uint32_t id = static_cast<uint32_t>(block_number());
  const int h = id % s.H, block = id / s.H, rep = s.H / s.G, g = h / rep;
  const int2 at = scan_find(s, w, block, false);
  if (at.x < 0) return;
  const ScanSeq sq = scan_seq(s, w, at.x);
  const int64_t row0 = sq.first + static_cast<int64_t>(at.y) * kScanBlock;
  const int L = min(kScanBlock, sq.len - at.y * kScanBlock);
  if (sq.len <= max(a.short_len, 0)) return;
  char* const group = d.groups + (static_cast<int64_t>(block) * s.G + g) * d.group_bytes;
  char* const head = d.heads + (static_cast<int64_t>(block) * s.H + h) * Block::kHeadBytes;
  const bool first = h % rep == 0;

  // this wave's rows of K and Q
  const int i = 16 * wave + l16, N = s.N;
  bf16x8 kf[kSteps][kRaw];
  Parts<kRaw> kq[kSteps], qq[kSteps];
  float k2 = 0.f, q2 = 0.f;
  {
    const int64_t row = row0 + min(i, L - 1);
    const T* const kp = static_cast<const T*>(a.k) + row * a.k_stride + static_cast<int64_t>(g) * N;
    const T* const qp = static_cast<const T*>(a.q) + row * a.q_stride + static_cast<int64_t>(g) * N;
#pragma unroll
    for (int n = 0; n < kSteps; ++n) {
      const int c = 32 * n + 8 * q, have = i < L ? N - c : 0;
      Four<T> kv[2], qv[2];
      kv[0].load(kp + c, have);
      kv[1].load(kp + c + 4, have - 4);
      qv[0].load(qp + c, have);
      qv[1].load(qp + c + 4, have - 4);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float k0 = kv[e >> 2].at(e & 3), k1 = kv[e >> 2].at((e & 3) + 1);
        const float q0 = qv[e >> 2].at(e & 3), q1 = qv[e >> 2].at((e & 3) + 1);
        k2 += k0 * k0 + k1 * k1;
        q2 += q0 * q0 + q1 * q1;
        kq[n].set(e >> 1, k0, k1);
        qq[n].set(e >> 1, q0, q1);
      }
    }
  }
#pragma unroll
  for (int n = 0; n < kSteps; ++n)
#pragma unroll
    for (int p = 0; p < kRaw; ++p) {
      kf[n][p] = kq[n].part(p);
      kl[((wave * kSteps + n) * kRaw + p) * 64 + lane] = kf[n][p];
      if (first && !d.direct) {
        bf16x8* const to = reinterpret_cast<bf16x8*>(group + Block::kKeys) + ((wave * kSteps + n) * kRaw + p) * 64 + lane;
        to[0] = kf[n][p];
        to[Block::kKeys / 16] = qq[n].part(p);
      }
    }
  k2 += __shfl_xor(k2, 16);
  q2 += __shfl_xor(q2, 16);
  k2 += __shfl_xor(k2, 32);
  q2 += __shfl_xor(q2, 32);
  const float rk = i < L ? delta_norm(k2, a.norm_eps) : 0.f, rq = i < L ? a.q_scale * delta_norm(q2, a.norm_eps) : 0.f;
  if (q == 0) {
    srk[i] = rk;
    srq[i] = rq;
  }
  if (wave == 0) {  // gates, lane = token
    const bool ok = lane < L;
    const int64_t row = row0 + min(lane, L - 1);
    const float step = softplus(to_float(static_cast<const T*>(s.dt)[row * s.dt_stride + h]) + (s.dt_bias ? s.dt_bias[h] : 0.f));
    const float b = sigmoid(to_float(static_cast<const T*>(a.beta)[row * a.beta_stride + h]));
    double sum = ok ? scan_log_decay(step, s.decay[h]) : 0.0;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const double o = __shfl_up(sum, m);
      if (lane >= m) sum += o;
    }
    const float hi = static_cast<float>(sum);
    sg[lane] = hi;
    sgl[lane] = static_cast<float>(sum - static_cast<double>(hi));
    sb[lane] = ok ? b : 0.f;
  }
  __syncthreads();
  if (wave == 3) {
    float* const to = reinterpret_cast<float*>(head + Block::kOffFactors);
    const float grown = __builtin_amdgcn_exp2f(sg[lane] + sgl[lane]);
    to[lane] = grown * srk[lane];
    to[64 + lane] = grown * srq[lane];
    to[128 + lane] = lane < L ? __builtin_amdgcn_exp2f((sg[63] - sg[lane]) + (sgl[63] - sgl[lane])) : 0.f;
    if (lane == 63) to[192] = grown;
  }

  // lane: token i and, of the strips up to this wave's, tokens j = 16 strip + 4 q + r
  {
    const float gi = sg[i], gli = sgl[i], bi = sb[i] * rk;
    for (int strip = 0; strip <= (wave | 1); ++strip) {
      f32x4 kkt = {0.f, 0.f, 0.f, 0.f}, qkt = kkt;
      if (strip <= wave) {
        f32x4 sum[2][2] = {{kkt, kkt}, {kkt, kkt}};
#pragma unroll
        for (int n = 0; n < kSteps; ++n) {
          bf16x8 kj[kRaw];
#pragma unroll
          for (int p = 0; p < kRaw; ++p) kj[p] = kl[((strip * kSteps + n) * kRaw + p) * 64 + lane];
#pragma unroll
          for (int p = kRaw - 1; p >= 0; --p)
#pragma unroll
            for (int o = 0; o < kRaw; ++o)
              if (p - o >= 0) {
                sum[0][n & 1] = mma_bf16(kj[o], kq[n].part(p - o), sum[0][n & 1]);
                sum[1][n & 1] = mma_bf16(kj[o], qq[n].part(p - o), sum[1][n & 1]);
              }
        }
        kkt = sum[0][0] + sum[0][1];
        qkt = sum[1][0] + sum[1][1];
      }
      f32x4 low;
      float p[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int j = 16 * strip + 4 * q + r;
        const float fall = j <= i ? __builtin_amdgcn_exp2f((gi - sg[j]) + (gli - sgl[j])) : 0.f;
        low[r] = j < i ? bi * srk[j] * kkt[r] * fall : 0.f;
        p[r] = j <= i ? rq * qkt[r] * fall : 0.f;
      }
      if (strip <= wave) *reinterpret_cast<f32x4*>(lm + i * kDeltaRow + 16 * strip + 4 * q) = low;
      Parts<3> pp;
      pp.set(0, p[0], p[1]);
      pp.set(1, p[2], p[3]);
#pragma unroll
      for (int o = 0; o < 3; ++o)
        __builtin_memcpy(head + Block::kOffP + (delta_pair(wave, strip >> 1) * 3 + o) * 1024 + lane * 16 + 8 * (strip & 1), pp.w[o], 8);
    }
  }
  if (first) {  // K on its side
    const uint16_t* const kb = reinterpret_cast<const uint16_t*>(kl);
    for (int f = wave; f < kN / 8; f += 4) {
      const int tile = f >> 1, nn = 8 * (l16 >> 2) + 4 * (tile & 1) + (l16 & 3);  // of the step's 32 keys
#pragma unroll
      for (int p = 0; p < kRaw; ++p) {
        uint16_t v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int t = 32 * (f & 1) + 16 * (e >> 2) + 4 * q + (e & 3);
          v[e] = kb[((((t >> 4) * kSteps + (tile >> 1)) * kRaw + p) * 64 + (t & 15) + 16 * (nn >> 3)) * 8 + (nn & 7)];
        }
        __builtin_memcpy(group + (f * kRaw + p) * 1024 + lane * 16, v, 16);
      }
    }
  }
  __syncthreads();

  // (1 + L)^-1: blocks of 16 on the diagonal by substitution, lane = column
  {
    float x[16];
    const float* const l = lm + 16 * wave * (kDeltaRow + 1);
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      float v[2] = {r == l16 ? 1.f : 0.f, 0.f};
#pragma unroll
      for (int m = 0; m < r; ++m) v[m & 1] -= l[r * kDeltaRow + m] * x[m];
      x[r] = v[0] + v[1];
    }
    if (q == 0)
#pragma unroll
      for (int r = 0; r < 16; ++r) tm[(16 * wave + r) * kDeltaRow + 16 * wave + l16] = x[r];
  }
  __syncthreads();
  // then those of 32, X = L_21 T_11 in the place of L_21, T_21 = -T_22 X
  constexpr int kDown = 16 * kDeltaRow;
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  f32x4 x = zero;
  const int corner = 32 * wave * (kDeltaRow + 1);
  if (wave < 2) x = mma_lds<4>(lm + corner + kDown, tm + corner, zero);
  __syncthreads();
  if (wave < 2) store_lds(lm + corner + kDown, x, 1.f);
  __syncthreads();
  if (wave < 2) store_lds(tm + corner + kDown, mma_lds<4>(tm + corner + kDown + 16, lm + corner + kDown, zero), -1.f);
  __syncthreads();
  // and the last of 64, a tile of 16 x 16 a wave
  const int tr = wave >> 1, tc = wave & 1;
  x = mma_lds<4>(lm + (2 + tr) * kDown + 16, tm + kDown + 16 * tc, zero);
  if (tc == 0) x = mma_lds<4>(lm + (2 + tr) * kDown, tm, x);
  __syncthreads();
  store_lds(lm + (2 + tr) * kDown + 16 * tc, x, 1.f);
  __syncthreads();
  x = mma_lds<4>(tm + (2 + tr) * kDown + 32, lm + 2 * kDown + 16 * tc, zero);
  if (tr == 1) x = mma_lds<4>(tm + 3 * kDown + 48, lm + 3 * kDown + 16 * tc, x);
  store_lds(tm + (2 + tr) * kDown + 16 * tc, x, -1.f);
  __syncthreads();

#pragma unroll
  for (int step = 0; step < 2; ++step) {
    if (step > wave >> 1) break;
    Parts<3> u;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int strip = 2 * step + half, j = 16 * strip + 4 * q;
      const f32x4 v = strip <= wave ? *reinterpret_cast<const f32x4*>(tm + i * kDeltaRow + j) : zero;
      u.set(2 * half, rk * v[0] * sb[j], rk * v[1] * sb[j + 1]);
      u.set(2 * half + 1, rk * v[2] * sb[j + 2], rk * v[3] * sb[j + 3]);
    }
#pragma unroll
    for (int p = 0; p < 3; ++p) *reinterpret_cast<bf16x8*>(head + (delta_pair(wave, step) * 3 + p) * 1024 + lane * 16) = u.part(p);
  }
}

// Where a lane's rows of a tensor lie, one block of tokens after the other: rows at(r) of the block and column `col`;
// past the sequence's end its last row.
template <class T, int kRows>
struct DeltaRows {
  const T* ptr[kRows];
  int64_t block;  // elements of a block's rows
  template <class At>
  __device__ __forceinline__ DeltaRows(const T* from, int64_t stride, int len, int64_t col, At at) : block(stride * kScanBlock) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) ptr[r] = from + min(at(r), max(len - 1, 0)) * stride + col;
  }
  // to block b of `blocks`, from the one before it
  template <class At>
  __device__ __forceinline__ void to(int b, int blocks, const T* from, int64_t stride, int len, int64_t col, At at) {
    if ((b + 1) * kScanBlock <= len) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) ptr[r] += block;
    } else if (b < blocks) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) ptr[r] = from + static_cast<int64_t>(min(b * kScanBlock + at(r), len - 1)) * stride + col;
    }
  }
};

// The blocks of a sequence for 16 values of a head (see above). Wave n of the first four holds the state at keys
// 32 (kW n + t / 2) + 8 q + 4 (t % 2) + r, tile t, and value l16, and takes a block's tokens 16 n + 4 q + r, as does wave 4 + n
// for y. An operand is requested again, for the next block, when this block has used it. 16 values of a head are a
// workgroup, since the rows of S do not wait for each other: 32 heads of 128 values fill the 256 CUs with one sequence.
// One sequence of 8,192 tokens, 32 heads of 128 x 128, bf16: 272 us, 2.1 us a block. That is the chain: with y of two parts,
// whose waves hold it up less, it took 4,500 clocks a block, of which one wave's instructions, the trips through LDS and three
// barriers took 3,300 and waits for the next operands the rest (0.2 GB of them by way of L2); its products alone would take
// 600. With sequences enough to hide the chain it is the operands, 84 KB of a block in bf16 and 180 in float32, which every
// workgroup of 16 values reads again.
// A sequence's workgroups follow each other in the order that fills an XCD after the other, so that one long sequence among
// short ones has 32 CUs: 4,096 tokens beside 255 single ones, 32 heads of 128 x 128, bf16, take 888 us, alone 176.
// kPair, where there are more workgroups than CUs: two of them share a CU, in 128 registers each, so that one's steps hide
// the other's waits. Operands are requested within the block then, and Q and K come by way of the workspace, whose addresses
// are fewer; 4 registers go to scratch in float32, 6 with 256 keys. 32 heads of 128 x 128, bf16: 32 sequences of 512 tokens
// 649 us, without 832 and with Q and K by way of the workspace 863; 2 of 4,096 320 and 366, but one of 8,192 400 and 368; with
// 256 keys 8 of 1,024 475 and 548; in float32 32 of 512 1,348 and 1,482, but with 256 keys, whose operands do not fit, 32 of
// 256 2,237 and 1,311. It goes by the call's sequences, though not all of a ragged batch need have blocks: the 4,096 tokens
// beside 255 single ones take 1,222 us without, one of 8,192 beside a single one 517 and 607.
template <class T, int kN, bool kDirect, bool kPair>
__global__ __launch_bounds__(512, kPair ? 4 : 2) void k_delta_heads(DeltaArgs a, ScanWork w, DeltaWork d) {
  using Block = DeltaBlock<T, kN>;
  constexpr int kRaw = Block::kRaw, kW = kN / 128, kSteps = kN / 32;
  __shared__ f32x4 ks_parts[4][4][64];           // [wave][strip]: parts of K S^T
  __shared__ uint4 state[kSteps][3][64];      // S as y's operand
  __shared__ uint4 rest[2][3][64], wide[2][3][64];  // [step][part]: V's rest, N' faded
  __shared__ f32x4 news[4][64];                  // [strip]: N'
  const ScanArgs& s = a.s;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l16 = lane & 15, q = lane >> 4;

  // workgroups go round the eight XCDs: the slices of a head, which share its operands, stay on one
  uint32_t id = static_cast<uint32_t>(block_number());
  {
    const uint32_t n = gridDim.x * gridDim.y, per = n >> 3, left = n & 7, xcd = id & 7;
    id = xcd * per + min(xcd, left) + (id >> 3);
  }
  const int tile = id % s.ptiles, h = id / s.ptiles % s.H, i = id / (s.ptiles * s.H);
  if (i >= s.n_seqs) return;
  const ScanSeq sq = scan_seq(s, w, i);
  if (sq.len <= a.short_len) return;
  const int p0 = 16 * tile, np = min(16, s.P - p0), g = h / (s.H / s.G), N = s.N;
  const bool mine = l16 < np;
  T* const y = static_cast<T*>(s.y) + sq.first * s.y_stride + static_cast<int64_t>(h) * s.P + p0;
  int slot = -1, pos = 0;
  if (s.ssm_in) {
    slot = s.owned ? w.slots[i] : scan_slot(s, i);
    if (slot == -2) {
      for (int64_t t = tid >> 4; t < sq.len; t += 32)
        if (mine) y[t * s.y_stride + l16] = from_float<T>(__builtin_nanf(""));
      return;
    }
    if (slot >= 0 && s.positions) pos = max(s.positions[i], 0);
  }

  const int blocks = sq.len > 0 ? sq.blocks : 0;
  const char* group = d.groups + (static_cast<int64_t>(sq.block0) * s.G + g) * d.group_bytes;
  const char* head = d.heads + (static_cast<int64_t>(sq.block0) * s.H + h) * Block::kHeadBytes;
  const int64_t group_next = s.G * d.group_bytes, head_next = static_cast<int64_t>(s.H) * Block::kHeadBytes;

  if (wave < 4) {
    f32x4 st[2 * kW];
    const int key0 = 32 * kW * wave + 8 * q;
    const int64_t place = ((static_cast<int64_t>(max(slot, 0)) * s.H + h) * s.P + p0 + l16) * N + key0;
    const bool vec = N % 4 == 0;
#pragma unroll
    for (int t = 0; t < 2 * kW; ++t) {
      st[t] = f32x4{0.f, 0.f, 0.f, 0.f};
      const int more = 32 * (t >> 1) + 4 * (t & 1), have = mine ? N - key0 - more : 0;
      if (slot >= 0 && pos > 0 && have > 0) {
        const float* const from = s.ssm_in + place + more;
        if (vec) {
          st[t] = *reinterpret_cast<const f32x4*>(from);
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (r < have) st[t][r] = from[r];
        }
      }
    }

    const T* const k_rows = static_cast<const T*>(a.k) + sq.first * a.k_stride + static_cast<int64_t>(g) * N;
    const T* const v_rows = static_cast<const T*>(a.v) + sq.first * a.v_stride + static_cast<int64_t>(h) * s.P + p0;
    auto key_row = [&](int r) { return 16 * r + l16; };
    auto value_row = [&](int r) { return 16 * wave + 4 * q + r; };
    // columns past the head's last value read that one's rows, and are dropped
    const int v_col = min(l16, np - 1);
    DeltaRows<T, kDirect ? 4 : 1> keys(k_rows, a.k_stride, sq.len, key0, key_row);
    DeltaRows<T, 4> values(v_rows, a.v_stride, sq.len, v_col, value_row);
    // K and its turned form together would take 192 registers for float32 and wide states: there they are requested when
    // the other one is done with
    constexpr bool kAhead = kRaw * kW <= 3 && !kPair;
    bf16x8 kf[kW][4][kRaw], kt[2 * kW][2][kRaw], u[2][3];
    T vv[4];
    f32x4 fk, fe;
    float fade = 0.f;
    auto load_keys = [&](const char* group) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        if (kDirect) {
#pragma unroll
          for (int n = 0; n < kW; ++n) __builtin_memcpy(&kf[n][t][0], keys.ptr[kDirect ? t : 0] + 32 * n, 16);
        } else {
          const bf16x8* const from = reinterpret_cast<const bf16x8*>(group + Block::kKeys) + (t * kSteps + kW * wave) * kRaw * 64;
#pragma unroll
          for (int n = 0; n < kW; ++n)
#pragma unroll
            for (int o = 0; o < kRaw; ++o) kf[n][t][o] = from[(n * kRaw + o) * 64 + lane];
        }
      }
    };
    auto load_kt = [&](const char* group, const char* head) {
      const bf16x8* const from = reinterpret_cast<const bf16x8*>(group) + 2 * kW * wave * 2 * kRaw * 64;
#pragma unroll
      for (int t = 0; t < 2 * kW; ++t)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int o = 0; o < kRaw; ++o) kt[t][n][o] = from[((t * 2 + n) * kRaw + o) * 64 + lane];
      fade = *reinterpret_cast<const float*>(head + Block::kOffFactors + 768);
    };
    auto load_u = [&](const char* head) {
      const bf16x8* const from = reinterpret_cast<const bf16x8*>(head) + delta_pair(wave, 0) * 3 * 64;
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int o = 0; o < 3; ++o)
          if (n <= wave >> 1) u[n][o] = from[(n * 3 + o) * 64 + lane];
      fe = *reinterpret_cast<const f32x4*>(head + Block::kOffFactors + 512 + (16 * wave + 4 * q) * 4);
    };
    auto load_values = [&](const char* head) {
      fk = *reinterpret_cast<const f32x4*>(head + Block::kOffFactors + (16 * wave + 4 * q) * 4);
#pragma unroll
      for (int r = 0; r < 4; ++r) vv[r] = *values.ptr[r];
    };
    if (blocks > 0) {
      if (kAhead) {
        load_keys(group);
        load_kt(group, head);
      }
      load_values(head);
      if (!kPair) load_u(head);
    }
    for (int b = 0; b < blocks; ++b) {
      const bool more = b + 1 < blocks;
      const char* const group_then = more ? group + group_next : group;
      const char* const head_then = more ? head + head_next : head;
      if (!kAhead) load_keys(group);
      {
        f32x4 ks[4];
#pragma unroll
        for (int n = 0; n < kW; ++n) {
          Parts<3> sp;
#pragma unroll
          for (int e = 0; e < 8; e += 2) sp.set(e >> 1, st[2 * n + (e >> 2)][e & 3], st[2 * n + (e >> 2)][(e & 3) + 1]);
#pragma unroll
          for (int o = 0; o < 3; ++o) __builtin_memcpy(&state[kW * wave + n][o][lane], sp.w[o], 16);
          if (n == 0)
#pragma unroll
            for (int t = 0; t < 4; ++t) ks[t] = f32x4{0.f, 0.f, 0.f, 0.f};
          mma_parts(kf[n], sp, ks);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) ks_parts[wave][t][lane] = ks[t];
      }
      if (kAhead) {
        if (kDirect) keys.to(b + 1, blocks, k_rows, a.k_stride, sq.len, key0, key_row);
        load_keys(group_then);
      } else if (!kPair) {
        load_kt(group, head);
      }
      if (kPair) load_u(head);
      __syncthreads();
      {
        f32x4 ks = ks_parts[0][wave][lane];
#pragma unroll
        for (int n = 1; n < 4; ++n) ks += ks_parts[n][wave][lane];
        Parts<3> rp;
#pragma unroll
        for (int r = 0; r < 4; r += 2) rp.set(r >> 1, to_float(vv[r]) - fk[r] * ks[r], to_float(vv[r + 1]) - fk[r + 1] * ks[r + 1]);
#pragma unroll
        for (int o = 0; o < 3; ++o) __builtin_memcpy(reinterpret_cast<char*>(&rest[wave >> 1][o][lane]) + 8 * (wave & 1), rp.w[o], 8);
      }
      values.to(b + 1, blocks, v_rows, a.v_stride, sq.len, v_col, value_row);
      load_values(head_then);
      __syncthreads();
      {
        // the three smallest products of a step, and the others
        f32x4 sums[2][2];
        Parts<3> rp[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          sums[n][0] = sums[n][1] = f32x4{0.f, 0.f, 0.f, 0.f};
          if (n > wave >> 1) break;
#pragma unroll
          for (int o = 0; o < 3; ++o) __builtin_memcpy(rp[n].w[o], &rest[n][o][lane], 16);
        }
        auto products = [&](int steps) {
#pragma unroll
          for (int o = 0; o < 3; ++o)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              if (n >= steps) break;
              sums[n][0] = mma_bf16(u[n][o], rp[n].part(2 - o), sums[n][0]);
              sums[n][1] = mma_bf16(u[n][o == 0], rp[n].part(o == 1), sums[n][1]);
            }
        };
        if (wave < 2)
          products(1);
        else
          products(2);
        const f32x4 nn = (sums[0][0] + sums[1][0]) + (sums[0][1] + sums[1][1]);
        news[wave][lane] = nn;
        Parts<3> np3;
#pragma unroll
        for (int r = 0; r < 4; r += 2) np3.set(r >> 1, fe[r] * nn[r], fe[r + 1] * nn[r + 1]);
#pragma unroll
        for (int o = 0; o < 3; ++o) __builtin_memcpy(reinterpret_cast<char*>(&wide[wave >> 1][o][lane]) + 8 * (wave & 1), np3.w[o], 8);
      }
      if (!kPair) load_u(head_then);
      if (kPair) load_kt(group, head);
      __syncthreads();
      {
        Parts<3> np3[2];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int o = 0; o < 3; ++o) __builtin_memcpy(np3[n].w[o], &wide[n][o][lane], 16);
#pragma unroll
        for (int t = 0; t < 2 * kW; ++t) st[t] *= fade;
#pragma unroll
        for (int p = 2; p >= 0; --p)
#pragma unroll
          for (int o = 0; o < kRaw; ++o)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int t = 0; t < 2 * kW; ++t)
                if (p - o >= 0) st[t] = mma_bf16(kt[t][n][o], np3[n].part(p - o), st[t]);
      }
      if (kAhead) load_kt(group_then, head_then);
      group = group_then;
      head = head_then;
    }

    if (slot < 0) return;
#pragma unroll
    for (int t = 0; t < 2 * kW; ++t) {
      const int more = 32 * (t >> 1) + 4 * (t & 1), have = mine ? N - key0 - more : 0;
      if (have <= 0) continue;
      float* const to = s.ssm_out + place + more;
      if (vec) {
        *reinterpret_cast<f32x4*>(to) = st[t];
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (r < have) to[r] = st[t][r];
      }
    }
    return;
  }

  const int strip = wave - 4;
  const T* const q_rows = static_cast<const T*>(a.q) + sq.first * a.q_stride + static_cast<int64_t>(g) * N;
  auto query_row = [&](int) { return 16 * strip + l16; };
  DeltaRows<T, 1> queries(q_rows, a.q_stride, sq.len, 8 * q, query_row);
  bf16x8 qf[kSteps][1][kRaw], p[2][3];
  f32x4 fq;
  auto load_queries = [&](const char* group, const char* head) {
    if (kDirect) {
#pragma unroll
      for (int n = 0; n < kSteps; ++n) __builtin_memcpy(&qf[n][0][0], queries.ptr[0] + 32 * n, 16);
    } else {
      const bf16x8* const from = reinterpret_cast<const bf16x8*>(group + 2 * Block::kKeys) + strip * kSteps * kRaw * 64;
#pragma unroll
      for (int n = 0; n < kSteps; ++n)
#pragma unroll
        for (int o = 0; o < kRaw; ++o) qf[n][0][o] = from[(n * kRaw + o) * 64 + lane];
    }
    fq = *reinterpret_cast<const f32x4*>(head + Block::kOffFactors + 256 + (16 * strip + 4 * q) * 4);
  };
  auto load_p = [&](const char* head) {
    const bf16x8* const from = reinterpret_cast<const bf16x8*>(head + Block::kOffP) + delta_pair(strip, 0) * 3 * 64;
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int o = 0; o < 3; ++o)
        if (n <= strip >> 1) p[n][o] = from[(n * 3 + o) * 64 + lane];
  };
  if (blocks > 0) {
    load_queries(group, head);
    load_p(head);
  }
  T* y_row = y + (16 * strip + 4 * q) * s.y_stride + l16;
  for (int b = 0; b < blocks; ++b) {
    if (b + 1 < blocks) {
      group += group_next;
      head += head_next;
    }
    __syncthreads();
    __syncthreads();
    f32x4 sums[2][1];
    sums[0][0] = sums[1][0] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int n = 0; n < kSteps; ++n) {
      Parts<3> sp;
#pragma unroll
      for (int o = 0; o < 3; ++o) __builtin_memcpy(sp.w[o], &state[n][o][lane], 16);
      mma_parts(qf[n], sp, sums[n & 1]);
    }
    f32x4 yy = (sums[0][0] + sums[1][0]) * fq;
    if (kDirect) queries.to(b + 1, blocks, q_rows, a.q_stride, sq.len, 8 * q, query_row);
    load_queries(group, head);
    __syncthreads();
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      if (n > strip >> 1) break;
      const f32x4 n0 = news[2 * n][lane], n1 = news[2 * n + 1][lane];
      Parts<3> np;
      np.set(0, n0[0], n0[1]);
      np.set(1, n0[2], n0[3]);
      np.set(2, n1[0], n1[1]);
      np.set(3, n1[2], n1[3]);
#pragma unroll
      for (int r = 2; r >= 0; --r)
#pragma unroll
        for (int o = 0; o <= r; ++o) yy = mma_bf16(p[n][o], np.part(r - o), yy);
    }
    load_p(head);
    const int left = sq.len - b * kScanBlock;
    if (left >= kScanBlock) {
      if (mine) {
#pragma unroll
        for (int r = 0; r < 4; ++r) y_row[r * s.y_stride] = from_float<T>(yy[r]);
      }
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (mine && 16 * strip + 4 * q + r < left) y_row[r * s.y_stride] = from_float<T>(yy[r]);
    }
    y_row += s.y_stride * kScanBlock;
  }
}

}  // namespace cdrge
