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
// k_delta_blocks forms U, P, the factors, and K and Q as operands, for all blocks at once; k_delta_heads walks a
// sequence's blocks for 16 values of one head, with S in the registers of four waves that share the keys. What a block's
// products leave is joined through LDS three times: the waves' parts of K S^T and Q S^T, V's rest, and N'.
//
// Operands of the matrix cores are bf16 (K, Q of bf16 tensors as they are), others the sum of three bf16 parts, which
// hold 24 bits whatever the magnitude; of two such operands the six products that reach 2^-24 are taken. For y in bf16 two
// parts (16 bits) do: they move it by 2e-5 of it.
//
// Along a reduction the order is free if both operands have it: entry e of lane group q stands for index
// 16 (e / 4) + 4 q + e % 4 of 32, so that a product's result is the next one's operand in the lane where it lies.
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ f32x4 mma_bf16(bf16x8 a, bf16x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }

// Entry e of the parts of v; v is pinned as one float (see split_half).
template <int kParts>
__device__ __forceinline__ void split_bf16(float v, bf16x8 (&to)[kParts], int e) {
  asm("" : "+v"(v));
#pragma unroll
  for (int p = 0; p < kParts; ++p) {
    const __bf16 part = static_cast<__bf16>(v);
    to[p][e] = part;
    v -= static_cast<float>(part);
  }
}

// c + a b, the products of parts that reach the last part's bits; small ones first.
template <int kA, int kB, int kReach>
__device__ __forceinline__ f32x4 mma_parts(const bf16x8 (&a)[kA], const bf16x8 (&b)[kB], f32x4 c) {
#pragma unroll
  for (int s = kReach - 1; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < kA; ++i)
      if (s - i >= 0 && s - i < kB) c = mma_bf16(a[i], b[s - i], c);
  return c;
}

template <class T>
struct DeltaParts;  // parts of K and Q, of y's operands
template <>
struct DeltaParts<float> {
  static constexpr int kRaw = 3, kOut = 3;
};
template <>
struct DeltaParts<uint16_t> {
  static constexpr int kRaw = 1, kOut = 2;
};

// What k_delta_blocks leaves, as operands of 1 KB (16 bytes a lane).
//   for a block and group  k, q   [step kN / 32][strip 4][part]: token 16 strip + l16, keys of the step
//                          kt     [tile kN / 16][step 2][part]: key 16 tile + l16, tokens of the step
//   for a block and head   u, p   [pair 6][part]: token 16 strip + l16, tokens of the step; pairs (strip, step) with
//                                 step <= strip / 2, in order
//                          factors: e^G r, e^G s and e^(G_last - G) of 64 tokens each, e^G_last
template <class T, int kN>
struct DeltaBlock {
  static constexpr int kRaw = DeltaParts<T>::kRaw, kOut = DeltaParts<T>::kOut;
  static constexpr int kKeys = 1024 * (kN / 32) * 4 * kRaw;  // of k, of q and of kt
  static constexpr int kGroupBytes = 3 * kKeys;
  static constexpr int kOffP = 6 * 3 * 1024, kOffFactors = kOffP + 6 * kOut * 1024, kHeadBytes = kOffFactors + 1024;
};
__host__ __device__ constexpr int delta_pair(int strip, int step) { return strip + (strip > 2) + step; }

struct DeltaWork {
  char* groups;  // [block][group]
  char* heads;   // [block][head]
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

// One block of a head: a wave takes 16 tokens. The first head of a group writes the group's operands.
template <class T, int kN>
__global__ __launch_bounds__(256) void k_delta_blocks(DeltaArgs a, ScanWork w, DeltaWork d) {
  using Block = DeltaBlock<T, kN>;
  constexpr int kRaw = Block::kRaw, kOut = Block::kOut, kSteps = kN / 32;
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
  if (L <= 0) return;  // a sequence without rows
  char* const group = d.groups + (static_cast<int64_t>(block) * s.G + g) * Block::kGroupBytes;
  char* const head = d.heads + (static_cast<int64_t>(block) * s.H + h) * Block::kHeadBytes;
  const bool first = h % rep == 0;

  // this wave's rows of K and Q
  const int i = 16 * wave + l16, N = s.N;
  bf16x8 kf[kSteps][kRaw], qf[kSteps][kRaw];
  float kk = 0.f, qq = 0.f;
  {
    const int64_t row = row0 + min(i, L - 1);
    const T* const kp = static_cast<const T*>(a.k) + row * a.k_stride + static_cast<int64_t>(g) * N;
    const T* const qp = static_cast<const T*>(a.q) + row * a.q_stride + static_cast<int64_t>(g) * N;
#pragma unroll
    for (int n = 0; n < kSteps; ++n)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int c = 32 * n + 16 * half + 4 * q, have = i < L ? N - c : 0;
        Four<T> kv, qv;
        kv.load(kp + c, have);
        qv.load(qp + c, have);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          kk += kv.at(e) * kv.at(e);
          qq += qv.at(e) * qv.at(e);
          split_bf16<kRaw>(kv.at(e), kf[n], 4 * half + e);
          split_bf16<kRaw>(qv.at(e), qf[n], 4 * half + e);
        }
      }
  }
#pragma unroll
  for (int n = 0; n < kSteps; ++n)
#pragma unroll
    for (int p = 0; p < kRaw; ++p) {
      kl[((wave * kSteps + n) * kRaw + p) * 64 + lane] = kf[n][p];
      if (first) {
        bf16x8* const to = reinterpret_cast<bf16x8*>(group) + ((n * 4 + wave) * kRaw + p) * 64 + lane;
        to[0] = kf[n][p];
        to[Block::kKeys / 16] = qf[n][p];
      }
    }
  kk += __shfl_xor(kk, 16);
  qq += __shfl_xor(qq, 16);
  kk += __shfl_xor(kk, 32);
  qq += __shfl_xor(qq, 32);
  const float rk = i < L ? delta_norm(kk, a.norm_eps) : 0.f, rq = i < L ? a.q_scale * delta_norm(qq, a.norm_eps) : 0.f;
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
#pragma unroll
        for (int n = 0; n < kSteps; ++n) {
          bf16x8 kj[kRaw];
#pragma unroll
          for (int p = 0; p < kRaw; ++p) kj[p] = kl[((strip * kSteps + n) * kRaw + p) * 64 + lane];
          kkt = mma_parts<kRaw, kRaw, kRaw>(kj, kf[n], kkt);
          qkt = mma_parts<kRaw, kRaw, kRaw>(kj, qf[n], qkt);
        }
      }
      f32x4 low;
      bf16x8 p[kOut];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int j = 16 * strip + 4 * q + r;
        const float fall = j <= i ? __builtin_amdgcn_exp2f((gi - sg[j]) + (gli - sgl[j])) : 0.f;
        low[r] = j < i ? bi * srk[j] * kkt[r] * fall : 0.f;
        split_bf16<kOut>(j <= i ? rq * qkt[r] * fall : 0.f, p, r);
      }
      if (strip <= wave) *reinterpret_cast<f32x4*>(lm + i * kDeltaRow + 16 * strip + 4 * q) = low;
#pragma unroll
      for (int o = 0; o < kOut; ++o)
        __builtin_memcpy(head + Block::kOffP + (delta_pair(wave, strip >> 1) * kOut + o) * 1024 + lane * 16 + 8 * (strip & 1), &p[o], 8);
    }
  }
  if (first) {  // K on its side
    const uint16_t* const kb = reinterpret_cast<const uint16_t*>(kl);
    for (int f = wave; f < kN / 8; f += 4) {
      const int n = 16 * (f >> 1) + l16;
#pragma unroll
      for (int p = 0; p < kRaw; ++p) {
        uint16_t v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int t = 32 * (f & 1) + 16 * (e >> 2) + 4 * q + (e & 3);
          v[e] = kb[((((t >> 4) * kSteps + (n >> 5)) * kRaw + p) * 64 + (t & 15) + 16 * ((n & 15) >> 2)) * 8 + 4 * (n >> 4 & 1) + (n & 3)];
        }
        __builtin_memcpy(group + 2 * Block::kKeys + (f * kRaw + p) * 1024 + lane * 16, v, 16);
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
    bf16x8 u[3];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int strip = 2 * step + half, j = 16 * strip + 4 * q;
      const f32x4 v = strip <= wave ? *reinterpret_cast<const f32x4*>(tm + i * kDeltaRow + j) : zero;
#pragma unroll
      for (int r = 0; r < 4; ++r) split_bf16<3>(rk * v[r] * sb[j + r], u, 4 * half + r);
    }
#pragma unroll
    for (int p = 0; p < 3; ++p) *reinterpret_cast<bf16x8*>(head + (delta_pair(wave, step) * 3 + p) * 1024 + lane * 16) = u[p];
  }
}

// The blocks of a sequence for 16 values of a head (see above). Wave n holds the state at keys 32 kW n + 16 tile + 4 q + r
// and value l16; of a block's tokens it takes 16 n + 4 q + r. Each operand is requested again, for the next block, when
// this block has used it.
template <class T, int kN>
__global__ __launch_bounds__(256, sizeof(T) == 2 && kN <= 128 ? 2 : 1) void k_delta_heads(DeltaArgs a, ScanWork w, DeltaWork d) {
  using Block = DeltaBlock<T, kN>;
  constexpr int kRaw = Block::kRaw, kOut = Block::kOut, kW = kN / 128;  // steps of 32 keys a wave has
  __shared__ f32x4 parts[2][4][4][64];                                   // of K S^T and Q S^T: [wave][strip]
  __shared__ bf16x8 rest[2][3][64], wide[2][3][64], out[2][kOut][64];    // V's rest, N' faded, N': [step][part]
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
  const int p0 = 16 * tile, np = min(16, s.P - p0), g = h / (s.H / s.G), N = s.N;
  const bool mine = l16 < np;
  T* const y = static_cast<T*>(s.y) + sq.first * s.y_stride + static_cast<int64_t>(h) * s.P + p0 + l16;
  int slot = -1, pos = 0;
  if (s.ssm_in) {
    slot = s.owned ? w.slots[i] : scan_slot(s, i);
    if (slot == -2) {
      for (int64_t t = tid >> 4; t < sq.len; t += 16)
        if (mine) y[t * s.y_stride] = from_float<T>(__builtin_nanf(""));
      return;
    }
    if (slot >= 0 && s.positions) pos = max(s.positions[i], 0);
  }

  f32x4 st[2 * kW];
  const int64_t place = ((static_cast<int64_t>(max(slot, 0)) * s.H + h) * s.P + p0 + l16) * N + 32 * kW * wave + 4 * q;
  const int have0 = N - 32 * kW * wave - 4 * q;
  const bool vec = N % 4 == 0;
#pragma unroll
  for (int t = 0; t < 2 * kW; ++t) {
    st[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int have = mine ? have0 - 16 * t : 0;
    if (slot >= 0 && pos > 0 && have > 0) {
      const float* const from = s.ssm_in + place + 16 * t;
      if (vec) {
        st[t] = *reinterpret_cast<const f32x4*>(from);
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (r < have) st[t][r] = from[r];
      }
    }
  }

  const int blocks = sq.len > 0 ? sq.blocks : 0;
  const char* const groups = d.groups + (static_cast<int64_t>(sq.block0) * s.G + g) * Block::kGroupBytes + lane * 16;
  const char* const heads = d.heads + (static_cast<int64_t>(sq.block0) * s.H + h) * Block::kHeadBytes;
  const int64_t group_next = static_cast<int64_t>(s.G) * Block::kGroupBytes, head_next = static_cast<int64_t>(s.H) * Block::kHeadBytes;
  // columns past the head's last value read that one's rows, and are dropped
  const T* const v = static_cast<const T*>(a.v) + sq.first * a.v_stride + static_cast<int64_t>(h) * s.P + p0 + min(l16, np - 1);
  bf16x8 kf[kW][4][kRaw], qf[kW][4][kRaw], kt[2 * kW][2][kRaw], u[2][3], p[2][kOut];
  T vv[4];
  f32x4 fk, fq, fe;
  float fade = 0.f;
  auto load_keys = [&](int b) {
    const bf16x8* const from = reinterpret_cast<const bf16x8*>(groups + b * group_next) + kW * wave * 4 * kRaw * 64;
#pragma unroll
    for (int n = 0; n < kW; ++n)
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int o = 0; o < kRaw; ++o) {
          kf[n][t][o] = from[((n * 4 + t) * kRaw + o) * 64];
          qf[n][t][o] = from[((n * 4 + t) * kRaw + o) * 64 + Block::kKeys / 16];
        }
  };
  auto load_kt = [&](int b) {
    const bf16x8* const from = reinterpret_cast<const bf16x8*>(groups + b * group_next + 2 * Block::kKeys) + 2 * kW * wave * 2 * kRaw * 64;
#pragma unroll
    for (int t = 0; t < 2 * kW; ++t)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int o = 0; o < kRaw; ++o) kt[t][n][o] = from[((t * 2 + n) * kRaw + o) * 64];
  };
  auto load_u = [&](int b) {
    const bf16x8* const from = reinterpret_cast<const bf16x8*>(heads + b * head_next) + delta_pair(wave, 0) * 3 * 64 + lane;
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int o = 0; o < 3; ++o)
        if (n <= wave >> 1) u[n][o] = from[(n * 3 + o) * 64];
  };
  auto load_p = [&](int b) {
    const bf16x8* const from = reinterpret_cast<const bf16x8*>(heads + b * head_next + Block::kOffP) + delta_pair(wave, 0) * kOut * 64 + lane;
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int o = 0; o < kOut; ++o)
        if (n <= wave >> 1) p[n][o] = from[(n * kOut + o) * 64];
  };
  auto load_rows = [&](int b) {
    const char* const f = heads + b * head_next + Block::kOffFactors + (16 * wave + 4 * q) * 4;
    fk = *reinterpret_cast<const f32x4*>(f);
    fq = *reinterpret_cast<const f32x4*>(f + 256);
    fe = *reinterpret_cast<const f32x4*>(f + 512);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t t = static_cast<int64_t>(b) * kScanBlock + 16 * wave + 4 * q + r;
      vv[r] = v[(t < sq.len ? t : sq.len - 1) * a.v_stride];
    }
  };
  auto load_fade = [&](int b) { fade = *reinterpret_cast<const float*>(heads + b * head_next + Block::kOffFactors + 768); };
  if (blocks > 0) {
    load_keys(0);
    load_rows(0);
    load_u(0);
    load_p(0);
    load_kt(0);
    load_fade(0);
  }
  for (int b = 0; b < blocks; ++b) {
    const int next = min(b + 1, blocks - 1);
    {
      f32x4 ks[4], qs[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) ks[t] = qs[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int n = 0; n < kW; ++n) {
        bf16x8 sp[3];
#pragma unroll
        for (int e = 0; e < 8; ++e) split_bf16<3>(st[2 * n + (e >> 2)][e & 3], sp, e);
        bf16x8 so[kOut];
#pragma unroll
        for (int o = 0; o < kOut; ++o) so[o] = sp[o];
#pragma unroll
        for (int t = 0; t < 4; ++t) ks[t] = mma_parts<kRaw, 3, 3>(kf[n][t], sp, ks[t]);
#pragma unroll
        for (int t = 0; t < 4; ++t) qs[t] = mma_parts<kRaw, kOut, kOut>(qf[n][t], so, qs[t]);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        parts[0][wave][t][lane] = ks[t];
        parts[1][wave][t][lane] = qs[t];
      }
    }
    load_keys(next);
    __syncthreads();
    f32x4 yy;
    {
      f32x4 ks = parts[0][0][wave][lane];
      yy = parts[1][0][wave][lane];
#pragma unroll
      for (int n = 1; n < 4; ++n) {
        ks += parts[0][n][wave][lane];
        yy += parts[1][n][wave][lane];
      }
      bf16x8 rp[3];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const bool ok = mine && b * kScanBlock + 16 * wave + 4 * q + r < sq.len;
        split_bf16<3>(ok ? to_float(vv[r]) - fk[r] * ks[r] : 0.f, rp, r);
        yy[r] *= fq[r];
      }
#pragma unroll
      for (int o = 0; o < 3; ++o) __builtin_memcpy(reinterpret_cast<char*>(&rest[wave >> 1][o][lane]) + 8 * (wave & 1), &rp[o], 8);
    }
    __syncthreads();
    {
      f32x4 nn = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        if (n > wave >> 1) break;
        bf16x8 rp[3];
#pragma unroll
        for (int o = 0; o < 3; ++o) rp[o] = rest[n][o][lane];
        nn = mma_parts<3, 3, 3>(u[n], rp, nn);
      }
      bf16x8 np3[3], npo[kOut];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        split_bf16<3>(fe[r] * nn[r], np3, r);
        split_bf16<kOut>(nn[r], npo, r);
      }
#pragma unroll
      for (int o = 0; o < 3; ++o) __builtin_memcpy(reinterpret_cast<char*>(&wide[wave >> 1][o][lane]) + 8 * (wave & 1), &np3[o], 8);
#pragma unroll
      for (int o = 0; o < kOut; ++o) __builtin_memcpy(reinterpret_cast<char*>(&out[wave >> 1][o][lane]) + 8 * (wave & 1), &npo[o], 8);
    }
    load_u(next);
    load_rows(next);
    __syncthreads();
#pragma unroll
    for (int t = 0; t < 2 * kW; ++t) st[t] *= fade;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      bf16x8 np3[3];
#pragma unroll
      for (int o = 0; o < 3; ++o) np3[o] = wide[n][o][lane];
#pragma unroll
      for (int t = 0; t < 2 * kW; ++t) st[t] = mma_parts<kRaw, 3, 3>(kt[t][n], np3, st[t]);
    }
    load_kt(next);
    load_fade(next);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      if (n > wave >> 1) break;
      bf16x8 npo[kOut];
#pragma unroll
      for (int o = 0; o < kOut; ++o) npo[o] = out[n][o][lane];
      yy = mma_parts<kOut, kOut, kOut>(p[n], npo, yy);
    }
    load_p(next);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t t = static_cast<int64_t>(b) * kScanBlock + 16 * wave + 4 * q + r;
      if (mine && t < sq.len) y[t * s.y_stride] = from_float<T>(yy[r]);
    }
  }

  if (slot < 0) return;
#pragma unroll
  for (int t = 0; t < 2 * kW; ++t) {
    const int have = mine ? have0 - 16 * t : 0;
    if (have <= 0) continue;
    float* const to = s.ssm_out + place + 16 * t;
    if (vec) {
      *reinterpret_cast<f32x4*>(to) = st[t];
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (r < have) to[r] = st[t][r];
    }
  }
}

}  // namespace cdrge
