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
  bool owned;            // whether k_scan_owners or k_scan_mark looks for slots that are named twice
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

// Slots that are named twice, in calls of many sequences, are looked for in a launch of its own; in others every
// workgroup reads the earlier slots for itself, beside its other loads: by scan_owned, from 2^28 pairs of a workgroup
// and a sequence on. 16 heads of 16 x 16, single tokens: 4,096 rows 182 us in two launches and 210 in one, 2,048 95 in
// one, 262,144 12.6 and 137 ms; one head of 4 x 4: 4,096 rows 26 and 18 us, 16,384 65 and 82; prompts of one token:
// 262,144 sequences 9.9 and 23.9 ms. Every pair is compared, 0.3 ms for 65,536 rows.
constexpr int kScanOwnerWaves = 16;
inline bool scan_owned(const int32_t* slots, int n_seqs, int64_t readers) {
  return slots && readers * n_seqs >= (int64_t(1) << 28);
}

// Of the 64 sequences from i0 on (a multiple of 64), those whose slots earlier ones of the call name, a bit each: lane =
// sequence, and the waves share the earlier slots, which are the same for all lanes and compared as scalars.
__device__ __forceinline__ uint64_t scan_taken(const ScanArgs& a, int i0, int slot) {
  __shared__ uint64_t found[kScanOwnerWaves];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint64_t taken = 0;
  for (int j = 16 * wave; j < i0; j += 16 * kScanOwnerWaves) {
#pragma unroll
    for (int e = 0; e < 16; ++e) taken |= __ballot(slot == a.slots[j + e]);
  }
#pragma unroll
  for (int e = 0; e < 64 / kScanOwnerWaves; ++e) {
    const int j = wave * (64 / kScanOwnerWaves) + e;
    taken |= __ballot(slot == __builtin_amdgcn_readlane(slot, j) && j < lane);
  }
  if (lane == 0) found[wave] = taken;
  __syncthreads();
#pragma unroll
  for (int v = 0; v < kScanOwnerWaves; ++v) taken |= found[v];
  return taken;
}

// Prompts: the sequences' slots as scan_slot has them.
static __global__ __launch_bounds__(64 * kScanOwnerWaves) void k_scan_owners(ScanArgs a, int32_t* slots) {
  const int i0 = blockIdx.x * 64, lane = threadIdx.x & 63, i = i0 + lane;
  const int slot = i < a.n_seqs ? a.slots[i] : -1;
  const uint64_t taken = scan_taken(a, i0, slot);
  if (threadIdx.x < 64 && i < a.n_seqs) slots[i] = slot < 0 ? -1 : (slot >= a.n_slots || (taken >> lane & 1) ? -2 : slot);
}

// Single tokens, which have no workspace: each workgroup of k_scan_step finds in its own first place of y, which it
// writes afterwards, NaN if an earlier row has the slot and zero if none has.
template <class T>
__global__ __launch_bounds__(64 * kScanOwnerWaves) void k_scan_mark(ScanArgs a, int tile) {
  const int i0 = blockIdx.x * 64, lane = threadIdx.x & 63, i = i0 + lane;
  const int slot = i < a.n_seqs ? a.slots[i] : -1;
  const uint64_t taken = scan_taken(a, i0, slot);
  if (slot < 0) return;
  T* const y = static_cast<T*>(a.y) + i * a.y_stride;
  for (int n = threadIdx.x >> 6; n < a.H * a.ptiles; n += kScanOwnerWaves)
    y[n / a.ptiles * a.P + n % a.ptiles * tile] = from_float<T>(taken >> lane & 1 ? __builtin_nanf("") : 0.f);
}

// ---------------------------------------------------------------------------------------------
// One token for each sequence. A workgroup owns kRpt * (256 / kLanes) channels of one head of one
// row: kLanes lanes side by side hold four columns of the state each, so a state row is read and
// written in whole lines. Bound by memory: the state is read and written once, past the caches (nobody
// reads it again before the next token). All loads of a workgroup are in flight together, the check for a
// repeated slot beside them. 256 rows, 64 heads of 64 x 128, bf16: 197 us, 5.4 TB/s (233 through the caches;
// 286 with the convolution's loads one after the other). One row of 16 heads: 7.1 us, the latency of a launch and
// two loads.
// ---------------------------------------------------------------------------------------------
template <class T, int kLanes, int kRpt>
__global__ __launch_bounds__(256) void k_scan_step(ScanArgs a) {
  constexpr int kRows = 256 / kLanes;
  constexpr int kTile = kRows * kRpt;
  constexpr int kConv = (kTile + 8 * kLanes + 255) / 256;  // channels of the convolution that a thread takes
  __shared__ float sb[kScanMaxState], sc[kScanMaxState], sx[kTile], sy[kTile];
  const int tid = threadIdx.x;
  const uint32_t id = static_cast<uint32_t>(block_number());
  const int tile = id % a.ptiles, h = id / a.ptiles % a.H, i = id / (a.ptiles * a.H);
  if (i >= a.n_seqs) return;
  const int slot = a.slots ? a.slots[i] : i, pos = max(a.positions[i], 0);
  if (slot < 0) return;
  const int p0 = tile * kTile, np = min(kTile, a.P - p0);
  const int64_t yp = static_cast<int64_t>(h) * a.P + p0;
  T* const y = static_cast<T*>(a.y) + i * a.y_stride + yp;
  if (slot >= a.n_slots) {
    if (tid < np) y[tid] = from_float<T>(__builtin_nanf(""));
    return;
  }
  // Everything that is read is requested at once; whether the slot is taken is known only further down.
  int taken = 0;
  if (a.owned)
    taken = !(to_float(y[0]) == 0.f);
  else if (a.slots)
    for (int j = tid; j < i; j += 256) taken |= a.slots[j] == slot;
  const int N = a.N, g = h / (a.H / a.G);
  const bool owns_bc = tile == 0 && h % (a.H / a.G) == 0;
  const T* const x = static_cast<const T*>(a.xbc) + i * a.xbc_stride;
  const T* const ring = static_cast<const T*>(a.conv_in) + static_cast<int64_t>(slot) * a.W * a.C;
  T now[kConv], past[kConv][kScanMaxConv - 1], cw[kConv][kScanMaxConv], cb[kConv];  // past[j - 1]: j tokens back
#pragma unroll
  for (int k = 0; k < kConv; ++k) {
    const int idx = tid + 256 * k;
    if (idx >= np + 2 * N) continue;
    const int c = idx < np ? h * a.P + p0 + idx : a.H * a.P + g * N + idx - np + (idx < np + N ? 0 : (a.G - 1) * N);
    now[k] = x[c];
    cb[k] = a.conv_bias ? static_cast<const T*>(a.conv_bias)[c] : T(0);
    const T* const w = static_cast<const T*>(a.conv_weight) + static_cast<int64_t>(c) * a.W;
#pragma unroll
    for (int j = 0; j < kScanMaxConv; ++j)
      if (j < a.W) {
        cw[k][j] = w[a.W - 1 - j];
        if (j > 0) past[k][j - 1] = pos >= j ? ring[static_cast<int64_t>((pos - j) % a.W) * a.C + c] : T(0);
      }
  }
  const T zv = (a.z && tid < np) ? (static_cast<const T*>(a.z) + i * a.z_stride + yp)[tid] : T(0);
  const float raw = to_float(static_cast<const T*>(a.dt)[i * a.dt_stride + h]);
  const int ln = tid % kLanes, n0 = ln * 4, pr = tid / kLanes;
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
        const f32x4 v = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(s));
        st[k][0] = v[0]; st[k][1] = v[1]; st[k][2] = v[2]; st[k][3] = v[3];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n0 + e < N) st[k][e] = s[e];
      }
    }
  }
  // convolution of this tile's x and of the group's B and C
#pragma unroll
  for (int k = 0; k < kConv; ++k) {
    const int idx = tid + 256 * k;
    if (idx >= np + 2 * N) continue;
    float u = to_float(cb[k]);
#pragma unroll
    for (int j = 1; j < kScanMaxConv; ++j)  // rows before the sequence's start are zeros
      if (j < a.W) u += to_float(cw[k][j]) * to_float(past[k][j - 1]);
    u = silu(u + to_float(cw[k][0]) * to_float(now[k]));
    (idx < np ? sx[idx] : (idx < np + N ? sb[idx - np] : sc[idx - np - N])) = u;
  }
  const float dt = softplus(raw + (a.dt_bias ? a.dt_bias[h] : 0.f));
  const float fade = expf(dt * a.decay[h]);
  if (__syncthreads_or(taken)) {  // an earlier row has the slot
    if (tid < np) y[tid] = from_float<T>(__builtin_nanf(""));
    return;
  }
  T* const ring_out = static_cast<T*>(a.conv_out) + static_cast<int64_t>(slot) * a.W * a.C;
#pragma unroll
  for (int k = 0; k < kConv; ++k) {
    const int idx = tid + 256 * k;
    if (idx >= np + 2 * N || !(idx < np || owns_bc)) continue;
    const int c = idx < np ? h * a.P + p0 + idx : a.H * a.P + g * N + idx - np + (idx < np + N ? 0 : (a.G - 1) * N);
    if (a.conv_in != a.conv_out)
      for (int e = 0; e < a.W; ++e) ring_out[static_cast<int64_t>(e) * a.C + c] = ring[static_cast<int64_t>(e) * a.C + c];
    ring_out[static_cast<int64_t>(pos % a.W) * a.C + c] = now[k];
  }
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
        __builtin_nontemporal_store(f32x4{st[k][0], st[k][1], st[k][2], st[k][3]}, reinterpret_cast<f32x4*>(s));
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
    if (a.z) v *= silu(to_float(zv));
    y[tid] = from_float<T>(v);
  }
}

// ---------------------------------------------------------------------------------------------
// Prompts. With a_q = step_q decay (in units of log 2), s_i the sum of a over a block's tokens up to i
// and S the state before the block, a block of up to 64 tokens is matrix products:
//
//   y_i = sum_{j <= i} (C_i B_j^T) 2^(s_i - s_j) step_j x_j  +  2^(s_i) S C_i  + skip x_i
//   S'  = 2^(s_last) S + sum_j 2^(s_last - s_j) step_j x_j B_j^T
//
// k_scan_blocks forms, once for all heads of a group, what they share: the convolved B and C, C B^T
// and, by head, the steps and sums s. k_scan_heads walks the blocks of a piece of a sequence for 64
// channels of one head, with S in its registers. Where sequences times heads leave compute units
// idle, sequences are cut into pieces: a first run of k_scan_heads forms each piece's own state from
// zero (without y), and in the second run a piece starts from its predecessors' states, each faded
// by the pieces behind it. This reads x twice but leaves no state in memory but one a piece.
// One sequence of 8,192 tokens, 64 heads of 64, state 128, bf16, takes 250 us: k_scan_blocks 23, the first run
// 62, the second 161, k_scan_ring 5 (37.7 ms by the step above, token after token; 44 us for the bytes); float32 296. It
// is bound by the vector unit's issue and by what two waves a SIMD leave uncovered: a block costs a wave 640 vector
// instructions beside 48 matrix products in the first run and 1,570 beside 114 in the second (convolution, gates, decays,
// splitting operands), 60% of the time in both.
// Pieces of at least four blocks: with at least 8, 1 x 2048 tokens and 16 heads takes 107 us instead of 73.
//
// Products run on the matrix cores in half precision (11 bits), operands scaled by a power of two of
// the block so that their largest magnitude is below 2^14, in two halves each (22 bits) and three
// products, for either type of tensor. With y's operands in one half, y in bf16 differs from the exact
// one's nearest by 1.2e-3 of y in the 2-norm, with two by 2e-5; the call above takes 221 us so, and 250.
// ---------------------------------------------------------------------------------------------
constexpr int kScanBlock = 64;

typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;
typedef __attribute__((ext_vector_type(4))) _Float16 f16x4;

__device__ __forceinline__ f32x4 mma16(f16x8 a, f16x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }

// The power of two that brings magnitudes of at most `most` below 2^14, as its exponent.
__device__ __forceinline__ int scan_scale(float most) {
  return 13 - min(max(static_cast<int>(__float_as_uint(most) >> 23) - 127, -100), 100);
}
__device__ __forceinline__ float two_to(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }  // |e| <= 126

// v in two halves. v is pinned as one float first: left to itself the compiler may convert a product to hi
// exactly in one place and from its rounded value in another, and near a tie the two differ.
__device__ __forceinline__ void split_half(float v, _Float16& hi, _Float16& lo) {
  asm("" : "+v"(v));
  hi = static_cast<_Float16>(v);
  lo = static_cast<_Float16>(v - static_cast<float>(hi));
}

// What k_scan_blocks leaves for a block and group: matrix-core operands, 16 bytes a lane.
//   cb     [strip 4][step 2][lane][8] float: C_i B_j^T, i = 16 strip + lane % 16, j = 32 step + 8 (lane / 16) + e
//   c      [strip 4][kN / 32][lane][8] half: C_i, columns 32 step + 8 (lane / 16) + e; then the low halves
//   b      [tile kN / 16][step 2][lane][8] half: B_j at column 16 tile + lane % 16; then the low halves
//   scale  float4: the scales of c and of b (exponents), the largest |cb|, the largest |B|
template <int kN>
struct ScanBlock {
  static constexpr int kCb = 4 * 2 * 64 * 8 * 4;
  static constexpr int kC = 4 * (kN / 32) * 64 * 16;
  static constexpr int kB = (kN / 16) * 2 * 64 * 16;
  static constexpr int kOffC = kCb, kOffB = kOffC + 2 * kC, kOffScale = kOffB + 2 * kB;
  static constexpr int kBytes = kOffScale + 256;
};

struct ScanWork {  // the workspace
  char* blocks;      // [block][group]
  float4* steps;     // [block][head][64]: s, r = s - log2(step), 2^(s_last - s) step, what s lacks below float32
  float* rests;      // [block][head][64]: what r lacks below float32
  float4* totals;    // [block][head]: s_last, largest step, largest and sum of 2^(s_last - s) step
  int32_t* slots;    // [sequence]: scan_slot
  int32_t* counts;   // blocks and pieces in all
  int2* start;       // [sequence]: its first block, its first piece
  int2* bounds;      // [sequence]: its first row, its rows
  int2* block_of;    // [block]: sequence, number in it
  int2* piece_of;    // [piece]: sequence, number in it
  float* states;     // [piece][head][tile]: a piece's own state (the last piece's place: the sequence's start)
  float* fades;      // [piece][head]: the sum of a over a piece
  int piece_blocks;  // blocks of a piece
  int max_blocks, max_pieces;
};

__host__ __device__ __forceinline__ int scan_blocks_of(int64_t len) { return len > kScanBlock ? static_cast<int>((len + kScanBlock - 1) / kScanBlock) : 1; }

// One sequence of a call: rows, blocks and pieces, and where the latter two start.
struct ScanSeq {
  int64_t first;
  int len, blocks, pieces, block0, piece0;
};

// Without offsets all sequences are equally long and everything follows by division; with offsets
// k_scan_map has worked it out.
__device__ __forceinline__ ScanSeq scan_seq(const ScanArgs& a, const ScanWork& w, int i) {
  ScanSeq q;
  int2 start;
  if (a.offsets) {
    const int2 b = w.bounds[i];
    start = w.start[i];
    q.first = b.x;
    q.len = b.y;
  } else {
    q.len = static_cast<int>(a.n_tokens / a.n_seqs);
    q.first = static_cast<int64_t>(i) * q.len;
  }
  q.blocks = scan_blocks_of(q.len);
  q.pieces = (q.blocks + w.piece_blocks - 1) / w.piece_blocks;
  q.block0 = a.offsets ? start.x : i * q.blocks;
  q.piece0 = a.offsets ? start.y : i * q.pieces;
  return q;
}

// Which sequence block (or piece) `id` belongs to, and which it is of it; x = -1 past the last.
__device__ __forceinline__ int2 scan_find(const ScanArgs& a, const ScanWork& w, int id, bool piece) {
  if (a.offsets) return id < w.counts[piece] ? (piece ? w.piece_of : w.block_of)[id] : make_int2(-1, 0);
  const int blocks = scan_blocks_of(a.n_tokens / a.n_seqs);
  const int each = piece ? (blocks + w.piece_blocks - 1) / w.piece_blocks : blocks;
  const int i = id / each;
  return i < a.n_seqs ? make_int2(i, id - i * each) : make_int2(-1, 0);
}

// Ragged sequences: bounds (offsets clamped into [0, n_tokens] and into a rising row), where blocks and
// pieces start, and whose each of them is. One workgroup; 1,024 sequences at a time. 5 us for 33 sequences, the
// latency of a launch.
static __global__ __launch_bounds__(1024) void k_scan_map(ScanArgs a, ScanWork w) {
  __shared__ int scan[3][16];
  __shared__ int seq_blocks[1024], seq_pieces[1024], seq_block0[1024], seq_piece0[1024];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  auto clamped = [&](int i) { return min(max(a.offsets[i], 0), static_cast<int>(a.n_tokens)); };
  int most = clamped(0), blocks = 0, pieces = 0;  // largest offset, blocks and pieces so far
  for (int i0 = 0; i0 < a.n_seqs; i0 += 1024) {
    const int i = i0 + tid;
    const bool ok = i < a.n_seqs;
    // running maximum of offsets[i + 1]
    int end = ok ? clamped(i + 1) : 0;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const int o = __shfl_up(end, m);
      if (lane >= m) end = max(end, o);
    }
    if (lane == 63) scan[0][wave] = end;
    __syncthreads();
    int before = most;  // the largest offset before this wave's
    for (int v = 0; v < wave; ++v) before = max(before, scan[0][v]);
    int first = __shfl_up(end, 1);
    first = lane == 0 ? before : max(before, first);
    end = max(before, end);
    for (int v = 0; v < 16; ++v) most = max(most, scan[0][v]);
    const int len = ok ? end - first : 0, nb = ok ? scan_blocks_of(len) : 0;
    const int np = (nb + w.piece_blocks - 1) / w.piece_blocks;
    int sb = nb, sp = np;  // running sums
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const int ob = __shfl_up(sb, m), op = __shfl_up(sp, m);
      if (lane >= m) {
        sb += ob;
        sp += op;
      }
    }
    if (lane == 63) {
      scan[1][wave] = sb;
      scan[2][wave] = sp;
    }
    __syncthreads();
    int b0 = blocks + sb - nb, p0 = pieces + sp - np;
    for (int v = 0; v < 16; ++v) {
      if (v < wave) {
        b0 += scan[1][v];
        p0 += scan[2][v];
      }
      blocks += scan[1][v];
      pieces += scan[2][v];
    }
    if (ok) {
      w.bounds[i] = make_int2(first, len);
      w.start[i] = make_int2(b0, p0);
    }
    seq_blocks[tid] = nb;
    seq_pieces[tid] = np;
    seq_block0[tid] = b0;
    seq_piece0[tid] = p0;
    __syncthreads();
    for (int t = wave; t < min(1024, a.n_seqs - i0); t += 16) {
      for (int n = lane; n < seq_blocks[t]; n += 64) w.block_of[seq_block0[t] + n] = make_int2(i0 + t, n);
      for (int n = lane; n < seq_pieces[t]; n += 64) w.piece_of[seq_piece0[t] + n] = make_int2(i0 + t, n);
    }
    __syncthreads();
  }
  if (tid == 0) {
    w.counts[0] = blocks;
    w.counts[1] = pieces;
  }
}

// Eight columns n0 .. n0 + 7 of a row of u as an operand, and its low half.
__device__ __forceinline__ void scan_operand(const float* row, float scale, f16x8& hi, f16x8& lo) {
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const float2 v = *reinterpret_cast<const float2*>(row + e);
    _Float16 h[2], l[2];
    split_half(v.x * scale, h[0], l[0]);
    split_half(v.y * scale, h[1], l[1]);
    hi[e] = h[0];
    hi[e + 1] = h[1];
    lo[e] = l[0];
    lo[e + 1] = l[1];
  }
}

// A token's decay in units of log 2. Past +-400 the state's factor is zero or infinite in float32 whatever it meets,
// so it stays there: the sums of a block's tokens are below 2^15 however long a step is, and the differences of two of
// them, each held as a float32 and what that lacks, are exact to 2^-33.
__device__ __forceinline__ double scan_log_decay(float step, float decay) {
  const double a = static_cast<double>(step) * static_cast<double>(decay) * 1.4426950408889634;
  return a < -400.0 ? -400.0 : (a > 400.0 ? 400.0 : a);
}

// Steps and decays of a block's heads: a wave takes kScanHeads heads, lane = token, with the loads of all
// of them in flight together.
constexpr int kScanHeads = 2;
template <class T>
__device__ __forceinline__ void scan_steps(const ScanArgs& a, const ScanWork& w, int block, int64_t row0, int L, int h0, int h1) {
  const int lane = threadIdx.x & 63;
  float raw[kScanHeads];
#pragma unroll
  for (int n = 0; n < kScanHeads; ++n)
    raw[n] = (lane < L && h0 + n < h1) ? to_float(static_cast<const T*>(a.dt)[(row0 + lane) * a.dt_stride + h0 + n]) : 0.f;
#pragma unroll
  for (int n = 0; n < kScanHeads; ++n) {
    const int h = h0 + n;
    if (h >= h1) break;
    const float step = lane < L ? softplus(raw[n] + (a.dt_bias ? a.dt_bias[h] : 0.f)) : 0.f;
    double sum = scan_log_decay(step, a.decay[h]);
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const double o = __shfl_up(sum, m);
      if (lane >= m) sum += o;
    }
    const double last = __shfl(sum, 63);
    // 2^(s_i - s_j) step_j is 2^(s_i - r_j), r = s - log2(step): infinite for a step of zero, which adds nothing
    const float s = static_cast<float>(sum);
    const double less = step > 0.f ? sum - log2(static_cast<double>(step)) : (step == step ? __builtin_inf() : static_cast<double>(step));
    const float r = static_cast<float>(less);
    const float rest_s = static_cast<float>(sum - static_cast<double>(s)), rest_r = fabsf(r) < 3e38f ? static_cast<float>(less - static_cast<double>(r)) : 0.f;
    const float left = lane < L ? step * __builtin_amdgcn_exp2f(static_cast<float>(last - sum)) : 0.f;
    const int64_t at_head = static_cast<int64_t>(block) * a.H + h;
    w.steps[at_head * 64 + lane] = make_float4(s, r, left, rest_s);
    w.rests[at_head * 64 + lane] = rest_r;
    const float most_step = wave_max(step), most_left = wave_max(left), all_left = wave_sum(left);
    if (lane == 0) w.totals[at_head] = make_float4(static_cast<float>(last), most_step, most_left, all_left);
  }
}

// What a block's heads share: one workgroup of eight waves a block and group for B and C, and further ones
// for the steps of kScanHeads * 8 heads each. kN: state_dim rounded up to 32, 64, 128 or 256. Bound by latency
// (convolution, products, store, one after the other): 128 blocks, state 128, 64 heads 23 us.
template <class T, int kN>
__global__ __launch_bounds__(512) void k_scan_blocks(ScanArgs a, ScanWork w, int parts) {
  using Block = ScanBlock<kN>;
  constexpr int kCols = 2 * kN, kRow = kCols + 2;  // a row's pad: eight rows on lies 16 banks on
  extern __shared__ float u[];                     // [64][kRow]: the convolved B, then C
  __shared__ float red[3][8];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l16 = lane & 15, q = lane >> 4;
  const uint32_t id = static_cast<uint32_t>(block_number());
  const int part = id % parts, g = id / parts % a.G, block = id / (parts * a.G);
  const int2 at = scan_find(a, w, block, false);
  if (at.x < 0) return;
  const ScanSeq sq = scan_seq(a, w, at.x);
  const int64_t row0 = sq.first + static_cast<int64_t>(at.y) * kScanBlock;
  const int L = min(kScanBlock, sq.len - at.y * kScanBlock);  // zero for a sequence without rows
  if (part > 0) {
    const int each = a.H / a.G, n = ((part - 1) * 8 + wave) * kScanHeads;
    if (n < each) scan_steps<T>(a, w, block, row0, L, g * each + n, min(g * each + n + kScanHeads, g * each + each));
    return;
  }
  int slot = -1, pos = 0;
  if (a.ssm_in) {
    slot = a.owned ? w.slots[at.x] : scan_slot(a, at.x);
    if (slot >= 0 && a.positions) pos = max(a.positions[at.x], 0);
    if (!a.owned && at.y == 0 && g == 0 && tid == 0) w.slots[at.x] = slot;
  }

  // convolution: a thread takes one column of B or C and an equal share of the block's tokens
  float most_b = 0.f, most_c = 0.f;
  {
    constexpr int kParts = 512 / kCols, kTokens = kScanBlock / kParts;
    const int col = tid % kCols, t0 = tid / kCols * kTokens;
    const T* const ring = (slot >= 0 && at.y == 0) ? static_cast<const T*>(a.conv_in) + static_cast<int64_t>(slot) * a.W * a.C : nullptr;
    const int n = col < kN ? col : col - kN;
    if (n >= a.N || L <= 0) {
      for (int t = t0; t < t0 + kTokens; ++t) u[t * kRow + col] = 0.f;
    } else {
      const int c = a.H * a.P + (col < kN ? 0 : a.G * a.N) + g * a.N + n;
      const T* const x = static_cast<const T*>(a.xbc) + row0 * a.xbc_stride + c;
      float cw[kScanMaxConv];  // the newest token's weight last
#pragma unroll
      for (int j = 0; j < kScanMaxConv; ++j)
        cw[j] = j >= kScanMaxConv - a.W ? to_float(static_cast<const T*>(a.conv_weight)[static_cast<int64_t>(c) * a.W + j - (kScanMaxConv - a.W)]) : 0.f;
      const float cb = a.conv_bias ? to_float(static_cast<const T*>(a.conv_bias)[c]) : 0.f;
      float past[3];  // tokens t - 3, t - 2, t - 1
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        const int t = t0 - 3 + j;
        past[j] = 0.f;
        if (3 - j < a.W) {
          if (t >= 0 || at.y > 0)
            past[j] = t < L ? to_float(x[static_cast<int64_t>(t) * a.xbc_stride]) : 0.f;
          else if (ring && pos + t >= 0)
            past[j] = to_float(ring[static_cast<int64_t>((pos + t) % a.W) * a.C + c]);
        }
      }
      for (int t = t0; t < t0 + kTokens; t += 8) {
        float now[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) now[e] = to_float(x[static_cast<int64_t>(min(t + e, L - 1)) * a.xbc_stride]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          // a tap past the width is left out, not multiplied by zero: its token may be anything
          float v = cb + cw[3] * now[e] + cw[2] * past[2];
          if (a.W > 2) v += cw[1] * past[1];
          if (a.W > 3) v += cw[0] * past[0];
          past[0] = past[1];
          past[1] = past[2];
          past[2] = now[e];
          v = t + e < L ? silu(v) : 0.f;
          u[(t + e) * kRow + col] = v;
          if (col < kN)
            most_b = fmaxf(most_b, fabsf(v));
          else
            most_c = fmaxf(most_c, fabsf(v));
        }
      }
    }
  }
  most_b = wave_max(most_b);
  most_c = wave_max(most_c);
  if (lane == 0) {
    red[0][wave] = most_b;
    red[1][wave] = most_c;
  }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < 8; ++v) {
    most_b = fmaxf(most_b, red[0][v]);
    most_c = fmaxf(most_c, red[1][v]);
  }
  const int eb = scan_scale(most_b), ec = scan_scale(most_c);
  const float fb = two_to(eb), fc = two_to(ec);
  char* const out = w.blocks + (static_cast<int64_t>(block) * a.G + g) * Block::kBytes;

  // C B^T: of the strips of tokens i (16 each) and steps of tokens j (32 each), the six that have j <= i
  float most_cb = 0.f;
  const int strip = wave < 2 ? wave : (wave < 4 ? 2 : 3), step = wave < 2 ? 0 : wave & 1;
  if (wave < 6 && 16 * strip < L) {
    f16x8 ch[kN / 32], cl[kN / 32];
#pragma unroll
    for (int k = 0; k < kN / 32; ++k) {
      scan_operand(u + (16 * strip + l16) * kRow + kN + 32 * k + 8 * q, fc, ch[k], cl[k]);
      if (step == 0 && (at.y > 0 || pos > 0)) {
        f16x8* const to = reinterpret_cast<f16x8*>(out + Block::kOffC) + (strip * (kN / 32) + k) * 64 + lane;
        to[0] = ch[k];
        to[4 * (kN / 32) * 64] = cl[k];
      }
    }
    f32x4 acc[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
      const int j = 32 * step + 8 * (l16 >> 2) + 4 * t + (l16 & 3);
#pragma unroll
      for (int k = 0; k < kN / 32; ++k) {
        f16x8 bh, bl;
        scan_operand(u + j * kRow + 32 * k + 8 * q, fb, bh, bl);
        acc[t] = mma16(bh, ch[k], acc[t]);
        acc[t] = mma16(bh, cl[k], acc[t]);
        acc[t] = mma16(bl, ch[k], acc[t]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc[t][e] = ldexpf(acc[t][e], -eb - ec);
        if (32 * step + 8 * q + 4 * t + e <= 16 * strip + l16) most_cb = fmaxf(most_cb, fabsf(acc[t][e]));
      }
    }
    f32x4* const to = reinterpret_cast<f32x4*>(out) + ((strip * 2 + step) * 64 + lane) * 2;
    to[0] = acc[0];
    to[1] = acc[1];
  }
  most_cb = wave_max(most_cb);
  if (lane == 0) red[2][wave] = most_cb;

  // B by column, for the state
  if (slot >= 0 || at.y < sq.blocks - 1) {
    for (int f = wave; f < (kN / 16) * 2; f += 8) {
      const int tile = f >> 1, step = f & 1;
      if (32 * step >= L) continue;
      f16x8 bh, bl;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = u[(32 * step + 8 * q + e) * kRow + 16 * tile + l16] * fb;
        _Float16 vh, vl;
        split_half(v, vh, vl);
        bh[e] = vh;
        bl[e] = vl;
      }
      f16x8* const to = reinterpret_cast<f16x8*>(out + Block::kOffB) + f * 64 + lane;
      to[0] = bh;
      to[(kN / 16) * 2 * 64] = bl;
    }
  }

  __syncthreads();
  if (tid == 0)
    *reinterpret_cast<float4*>(out + Block::kOffScale) =
        make_float4(__int_as_float(ec), __int_as_float(eb), fmaxf(fmaxf(fmaxf(red[2][0], red[2][1]), fmaxf(red[2][2], red[2][3])), fmaxf(red[2][4], red[2][5])), most_b);
}

// Four adjacent elements as they lie in memory.
template <class T>
struct Four;
template <>
struct Four<float> {
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  __device__ __forceinline__ void load(const float* from, int n) {  // n: how many there are
    if (n >= 4) {
      __builtin_memcpy(&v, from, 16);
    } else {
      if (n > 0) v.x = from[0];
      if (n > 1) v.y = from[1];
      if (n > 2) v.z = from[2];
    }
  }
  __device__ __forceinline__ void load_back(const float* from, int n) {  // two to four, the last in the last place
    v.w = from[n - 1];
    v.z = from[n - 2];
    if (n > 2) v.y = from[n - 3];
    if (n > 3) v.x = from[0];
  }
  __device__ __forceinline__ float at(int i) const { return i == 0 ? v.x : (i == 1 ? v.y : (i == 2 ? v.z : v.w)); }
};
template <>
struct Four<uint16_t> {
  uint2 v = make_uint2(0u, 0u);
  __device__ __forceinline__ void load(const uint16_t* from, int n) {
    if (n >= 4) {
      __builtin_memcpy(&v, from, 8);
    } else {
      if (n > 0) v.x = from[0];
      if (n > 1) v.x |= static_cast<uint32_t>(from[1]) << 16;
      if (n > 2) v.y = from[2];
    }
  }
  __device__ __forceinline__ void load_back(const uint16_t* from, int n) {
    v.y = from[n - 2] | static_cast<uint32_t>(from[n - 1]) << 16;
    if (n > 2) v.x = static_cast<uint32_t>(from[n - 3]) << 16;
    if (n > 3) v.x |= from[0];
  }
  __device__ __forceinline__ float at(int i) const {
    const uint32_t w = i < 2 ? v.x : v.y;
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
};

// LDS rows of 16-byte chunks, chunk c of row p at place c ^ f(p): the eight rows that a matrix-core read
// touches at a time (four neighbours, and those 16 on) take different places, and so do stores down the rows.
__device__ __forceinline__ int scan_place(int p) { return ((p ^ (p >> 2)) & 3) | ((p >> 2) & 4); }

// The blocks of a piece for 64 channels of a head (see above). kFirstRun: only the piece's own state, for
// pieces that have a successor. Lane (l16, q) of wave i holds the state at columns 16 tile + 4 q + e and
// channel 16 m + l16, the tiles shared among the waves, and y at token 16 i + l16 and channels 16 q + 4 m + e.
// Loads are issued a phase or more before their use: a block's time is otherwise theirs, one after the other.
// z and y, each met once, go past the caches, which keeps x there for the second run (1 x 8,192 tokens in bf16: 250 us, 262 through them).
template <class T, int kN, bool kFirstRun>
__global__ __launch_bounds__(256, 2) void k_scan_heads(ScanArgs a, ScanWork w) {
  constexpr bool first_run = kFirstRun;
  using Block = ScanBlock<kN>;
  constexpr int kTiles = kN / 16 >= 4 ? kN / 64 : 1;  // column tiles of a wave
  constexpr int kCh = kN / 16 >= 4 ? 4 : 2;           // channel tiles of a wave
  __shared__ _Float16 xt[2][64 * 64], xw[2][64 * 64], hs[2][64 * kN];  // by channel: x, faded x, state
  // by token, for this block and the next: s, r, faded step, and what s and r lack; totals and scales
  __shared__ float tokens[2][5][64], red[4];
  __shared__ float4 sums[2][2];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l16 = lane & 15, q = lane >> 4;
  const int tile0 = kN / 16 >= 4 ? wave * kTiles : wave & 1, ch0 = kN / 16 >= 4 ? 0 : (wave >> 1) * 2;

  // workgroups go round the eight XCDs: the heads of a piece, which share its blocks' operands, stay on one
  uint32_t id = static_cast<uint32_t>(block_number());
  {
    const uint32_t n = gridDim.x * gridDim.y, per = n >> 3, rest = n & 7, xcd = id & 7;
    id = xcd * per + min(xcd, rest) + (id >> 3);
  }
  const int tile = id % a.ptiles, h = id / a.ptiles % a.H, piece = id / (a.ptiles * a.H);
  const int2 at = scan_find(a, w, piece, true);
  if (at.x < 0) return;
  const ScanSeq sq = scan_seq(a, w, at.x);
  const bool last_piece = at.y == sq.pieces - 1;
  if (first_run && last_piece) return;
  const int slot = a.ssm_in ? w.slots[at.x] : -1;
  const int p0 = tile * 64, np = min(64, a.P - p0), g = h / (a.H / a.G);
  T* const y = static_cast<T*>(a.y) + static_cast<int64_t>(h) * a.P + p0;
  const int nb0 = at.y * w.piece_blocks, nb1 = min(sq.blocks, nb0 + w.piece_blocks);
  if (slot == -2) {
    if (!first_run)
      for (int64_t t = static_cast<int64_t>(nb0) * 64 + (tid >> 6); t < min(static_cast<int64_t>(nb1) * 64, static_cast<int64_t>(sq.len)); t += 4)
        if (lane < np) y[(sq.first + t) * a.y_stride + lane] = from_float<T>(__builtin_nanf(""));
    return;
  }
  const int pos = (slot >= 0 && a.positions) ? max(a.positions[at.x], 0) : 0;

  // the state before the piece
  f32x4 st[kTiles][kCh];
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int m = 0; m < kCh; ++m) st[t][m] = f32x4{0.f, 0.f, 0.f, 0.f};
  // a stored state of a piece, as the lanes hold it
  auto stored = [&](int which, int t, int m) {
    const int64_t tiles = static_cast<int64_t>(kTiles) * kCh;
    return reinterpret_cast<f32x4*>(w.states) +
           (((static_cast<int64_t>(which) * a.H + h) * a.ptiles + tile) * 4 + wave) * tiles * 64 + (t * kCh + m) * 64 + lane;
  };
  const int64_t sbase = ((static_cast<int64_t>(max(slot, 0)) * a.H + h) * a.P + p0) * a.N;
  bool has = false;
  if (at.y > 0) {
    if (!first_run) {
      has = true;
      for (int k = 0; k < at.y; ++k) {
        const float fade = k ? __builtin_amdgcn_exp2f(w.fades[static_cast<int64_t>(sq.piece0 + k) * a.H + h]) : 0.f;
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
          for (int m = 0; m < kCh; ++m) {
            const f32x4 v = *stored(sq.piece0 + k, t, m);
            st[t][m] = k ? st[t][m] * fade + v : v;
          }
      }
    }
  } else if (pos > 0) {
    has = true;
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int m = 0; m < kCh; ++m) {
        const int n = 16 * (tile0 + t) + 4 * q, p = 16 * (ch0 + m) + l16;
        if (!first_run && sq.pieces > 1) {
          // a later piece may have updated the slot in place already
          st[t][m] = *stored(sq.piece0 + sq.pieces - 1, t, m);
        } else if (p < np) {
          const float* const s = a.ssm_in + sbase + static_cast<int64_t>(p) * a.N + n;
          if (a.N % 4 == 0) {
            if (n < a.N) st[t][m] = *reinterpret_cast<const f32x4*>(s);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (n + e < a.N) st[t][m][e] = s[e];
          }
        }
        if (first_run) *stored(sq.piece0 + sq.pieces - 1, t, m) = st[t][m];
      }
  }
  float most_state = 0.f;  // bounds the state's magnitudes
  if (has) {
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int m = 0; m < kCh; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) most_state = fmaxf(most_state, fabsf(st[t][m][e]));
    most_state = wave_max(most_state);
    if (lane == 0) red[wave] = most_state;
    __syncthreads();
    most_state = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    __syncthreads();
  }

  // convolution of x: thread (tid / 16, tid % 16) takes four tokens of four channels
  const int pc = (tid & 15) * 4, tg = (tid >> 4) * 4;
  Four<T> cw[4], cb;  // by channel: the taps, as many as there are; the biases
  cb = Four<T>{};
  if (a.conv_bias) cb.load(static_cast<const T*>(a.conv_bias) + h * a.P + p0 + pc, np - pc);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    cw[c] = Four<T>{};
    if (pc + c < np) cw[c].load_back(static_cast<const T*>(a.conv_weight) + static_cast<int64_t>(h * a.P + p0 + pc + c) * a.W, a.W);
  }
  // Whole blocks of whole heads are loaded without conditions: 250 us instead of 261 at 1 x 8,192 tokens in bf16. Where
  // registers are short (float32, wide states) the second way costs more than it gives (state 256: 544 against 525 us).
  const bool whole = sizeof(T) == 2 && kN <= 128 && np == 64;
  Four<T> raw[7];  // tokens tg - 3 .. tg + 3 of the block
  auto load_raw = [&](int nth) {
    const int L = min(kScanBlock, sq.len - nth * kScanBlock);
    // the thread's place as new values: addresses made of them are not kept from one block to the next
    int t0 = tg - 3, c = pc;
    asm volatile("" : "+v"(t0), "+v"(c));
    const T* from = static_cast<const T*>(a.xbc) + (sq.first + static_cast<int64_t>(nth) * kScanBlock + t0) * a.xbc_stride + h * a.P + p0 + c;
    if (whole && nth > 0 && L == kScanBlock) {  // everything is there: no lane asks for itself
#pragma unroll
      for (int r = 0; r < 7; ++r, from += a.xbc_stride)
        if (r >= 4 - a.W) raw[r].load(from, 4);
      return;
    }
#pragma unroll
    for (int r = 0; r < 7; ++r, from += a.xbc_stride) {
      raw[r] = Four<T>{};
      if (r < 4 - a.W || t0 + r >= L) continue;
      const T* at_row = from;
      if (t0 + r < 0 && nth == 0) {
        if (slot < 0 || pos + t0 + r < 0) continue;
        at_row = static_cast<const T*>(a.conv_in) + (static_cast<int64_t>(slot) * a.W + (pos + t0 + r) % a.W) * a.C + h * a.P + p0 + c;
      }
      raw[r].load(at_row, np - c);
    }
  };

  const float skip = a.skip ? a.skip[h] : 0.f;
  double faded = 0.0;
  // a block's steps (wave 0, by token), totals and scales (wave 1)
  float4 early = make_float4(0.f, 0.f, 0.f, 0.f);
  float early_rest = 0.f;
  auto operands = [&](int nth) { return w.blocks + (static_cast<int64_t>(sq.block0 + nth) * a.G + g) * Block::kBytes; };
  auto load_steps = [&](int nth) {
    const int64_t at_head = static_cast<int64_t>(sq.block0 + nth) * a.H + h;
    if (wave == 0) {
      early = w.steps[at_head * 64 + lane];
      early_rest = w.rests[at_head * 64 + lane];
    }
    if (wave == 1) early = *(lane == 0 ? w.totals + at_head : reinterpret_cast<const float4*>(operands(nth) + Block::kOffScale));
  };
  load_raw(nb0);
  load_steps(nb0);
  for (int nth = nb0; nth < nb1; ++nth) {
    const int L = min(kScanBlock, sq.len - nth * kScanBlock);
    if (L <= 0) break;  // a sequence without rows
    const char* const in = operands(nth);
    // the lane's place as new values: addresses made of them are not kept in registers from block to block
    int lo16 = l16, lq = q, pcn = pc, tgn = tg;
    asm volatile("" : "+v"(lo16), "+v"(lq), "+v"(pcn), "+v"(tgn));
    const bool keep = slot >= 0 || nth < sq.blocks - 1;  // whether anybody wants the state behind the block
    float* const ts = tokens[nth & 1][0];
    float* const tr = tokens[nth & 1][1];
    float* const tw = tokens[nth & 1][2];
    float* const tl = tokens[nth & 1][3];
    float* const tq = tokens[nth & 1][4];
    if (wave == 0) {
      ts[lane] = early.x;
      tr[lane] = early.y;
      tw[lane] = early.z;
      tl[lane] = early.w;
      tq[lane] = early_rest;
    }
    if (wave == 1 && lane < 2) sums[nth & 1][lane] = early;
    // operands of the state; the first run has nothing else to do meanwhile, so it asks for them here
    f16x8 bhs[2][kTiles], bls[2][kTiles];
    auto load_b = [&]() {
      const f16x8* const bf = reinterpret_cast<const f16x8*>(in + Block::kOffB) + lane;
#pragma unroll
      for (int step = 0; step < 2; ++step)
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          bhs[step][t] = bf[((tile0 + t) * 2 + step) * 64];
          bls[step][t] = bf[((kN / 16 + tile0 + t) * 2 + step) * 64];
        }
    };
    if (first_run && keep) load_b();
    // z of the lane's token
    const int zi = min(16 * wave + lo16, L - 1);
    T zv[16];
    if (!first_run && a.z) {
      const T* const z = static_cast<const T*>(a.z) + (sq.first + static_cast<int64_t>(nth) * kScanBlock + zi) * a.z_stride +
                         static_cast<int64_t>(h) * a.P + p0 + 16 * lq;
      if (16 * lq + 16 <= np) {
        load_once(zv, z);
      } else {
#pragma unroll
        for (int k = 0; k < 16; ++k) zv[k] = 16 * lq + k < np ? z[k] : T(0);
      }
    }
    // operands of y: C B^T (of a strip's first 16 (wave 0: 16, 1: 32, 2: 48, 3: 64) tokens) and C
    f32x4 cbs[2][2];
    f16x8 chs[kN / 32], cls[kN / 32];
    if (!first_run) {
      const f32x4* const cbf = reinterpret_cast<const f32x4*>(in) + (wave * 2 * 64 + lane) * 2;
#pragma unroll
      for (int step = 0; step < 2; ++step)
#pragma unroll
        for (int half = 0; half < 2; ++half) cbs[step][half] = cbf[step * 128 + half];
      const f16x8* const cf = reinterpret_cast<const f16x8*>(in + Block::kOffC) + wave * (kN / 32) * 64 + lane;
#pragma unroll
      for (int k = 0; k < kN / 32; ++k) {
        chs[k] = cf[k * 64];
        cls[k] = cf[(4 * (kN / 32) + k) * 64];
      }
    }
    float u[4][4], most = 0.f;  // [token][channel]
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        // a tap past the width is left out, not multiplied by zero: its token may be anything
        float v = cb.at(c) + cw[c].at(3) * raw[t + 3].at(c) + cw[c].at(2) * raw[t + 2].at(c);
        if (a.W > 2) v += cw[c].at(1) * raw[t + 1].at(c);
        if (a.W > 3) v += cw[c].at(0) * raw[t].at(c);
        u[t][c] = tgn + t < L ? silu(v) : 0.f;  // zero past the head's channels: so are their taps
        most = fmaxf(most, fabsf(u[t][c]));
      }
    most = wave_max(most);
    if (lane == 0) red[wave] = most;
    __syncthreads();  // every wave is past the block before: its operands may be overwritten
    most = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float4 total = sums[nth & 1][0], scale = sums[nth & 1][1];
    const int ex = scan_scale(most), ew = scan_scale(most * total.z), eh = scan_scale(most_state);
    {
      const float fx = two_to(ex), fw = two_to(ew);
      const float4 left = *reinterpret_cast<const float4*>(tw + tgn);
      const float l4[4] = {left.x * fw, left.y * fw, left.z * fw, left.w * fw};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int p = pcn + c, to = p * 64 + (((tgn >> 3) ^ scan_place(p)) << 3) + (tgn & 7);
        f16x4 hi, lo, wh, wl;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          _Float16 vh, vl;
          split_half(u[t][c] * fx, vh, vl);
          hi[t] = vh;
          lo[t] = vl;
          split_half(u[t][c] * l4[t], vh, vl);
          wh[t] = vh;
          wl[t] = vl;
        }
        if (!first_run) {
          *reinterpret_cast<f16x4*>(&xt[0][to]) = hi;
          *reinterpret_cast<f16x4*>(&xt[1][to]) = lo;
        }
        if (keep) {
          *reinterpret_cast<f16x4*>(&xw[0][to]) = wh;
          *reinterpret_cast<f16x4*>(&xw[1][to]) = wl;
        }
      }
    }
    if (has && !first_run) {
      const float fh = two_to(eh);
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int m = 0; m < kCh; ++m) {
          const int p = 16 * (ch0 + m) + lo16, chunk = 2 * (tile0 + t) + (lq >> 1);
          const int to = p * kN + ((chunk ^ (scan_place(p) & (kN / 8 - 1))) << 3) + 4 * (lq & 1);
          f16x4 hi, lo;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            _Float16 vh, vl;
            split_half(st[t][m][e] * fh, vh, vl);
            hi[e] = vh;
            lo[e] = vl;
          }
          *reinterpret_cast<f16x4*>(&hs[0][to]) = hi;
          *reinterpret_cast<f16x4*>(&hs[1][to]) = lo;
        }
    }
    __syncthreads();
    if (nth + 1 < nb1) {
      load_raw(nth + 1);
      load_steps(nth + 1);
    }
    if (!first_run && keep) load_b();

    if (!first_run && 16 * wave < L) {
      const int i = 16 * wave + lo16;  // the lane's token
      // Where the operands of the lane's channels lie: chunk 4 k + lq of row p at place (4 k + lq) ^ f(p), for even k
      // the first of two places and for odd k the second, moved on by whole rows of eight chunks.
      int far_at[4][2], near_at[4][2];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int p = 16 * (lo16 >> 2) + 4 * m + (lo16 & 3), f = scan_place(p);
#pragma unroll
        for (int odd = 0; odd < 2; ++odd) {
          near_at[m][odd] = p * 64 + (((4 * odd + lq) ^ f) << 3);
          far_at[m][odd] = p * kN + (((4 * odd + lq) ^ (f & (kN / 8 - 1))) << 3);
        }
      }
      const float si = ts[i], li = tl[i];
      f32x4 far[4], near[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) far[m] = near[m] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (has) {
#pragma unroll
        for (int k = 0; k < kN / 32; ++k) {
          const f16x8 ch = chs[k], cl = cls[k];
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const int from = far_at[m][k & 1] + (k >> 1) * 64;
            const f16x8 hh = *reinterpret_cast<const f16x8*>(&hs[0][from]);
            far[m] = mma16(hh, ch, far[m]);
            far[m] = mma16(hh, cl, far[m]);
            far[m] = mma16(*reinterpret_cast<const f16x8*>(&hs[1][from]), ch, far[m]);
          }
        }
      }
      const float most_mix = fmaxf(scale.z * total.y * __builtin_amdgcn_exp2f(fmaxf(total.x, 0.f)), fabsf(skip));
      const int em = scan_scale(most_mix);
      const float fm = two_to(em), own = skip * fm;
#pragma unroll
      for (int step = 0; step < 2; ++step) {
        if (step > wave >> 1) continue;
        f16x8 mh, ml;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int j0 = 32 * step + 8 * lq + 4 * half;
          const f32x4 rj = *reinterpret_cast<const f32x4*>(tr + j0);
          const f32x4 qj = *reinterpret_cast<const f32x4*>(tq + j0);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float fall = (si - rj[e]) + (li - qj[e]);
            float v = cbs[step][half][e] * fm * __builtin_amdgcn_exp2f(fall);
            if (step == wave >> 1) v = j0 + e < i ? v : (j0 + e == i ? v + own : 0.f);  // tokens after i, and i itself
            _Float16 vh, vl;
            split_half(v, vh, vl);
            mh[4 * half + e] = vh;
            ml[4 * half + e] = vl;
          }
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const int from = near_at[m][step];
          const f16x8 xh = *reinterpret_cast<const f16x8*>(&xt[0][from]);
          near[m] = mma16(xh, mh, near[m]);
          near[m] = mma16(xh, ml, near[m]);
          near[m] = mma16(*reinterpret_cast<const f16x8*>(&xt[1][from]), mh, near[m]);
        }
      }
      if (i < L) {
        const float es = has ? ldexpf(__builtin_amdgcn_exp2f(si), -__float_as_int(scale.x) - eh) : 0.f;
        const int64_t row = sq.first + static_cast<int64_t>(nth) * kScanBlock + i;
        float v[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          v[k] = ldexpf(near[k >> 2][k & 3], -em - ex);
          if (has) v[k] += far[k >> 2][k & 3] * es;
        }
        const int p = 16 * lq;
        if (a.z) {
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] *= silu(to_float(zv[k]));
        }
        T o[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] = from_float<T>(v[k]);
        T* const to = y + row * a.y_stride + p;
        if (p + 16 <= np) {
          store_once(to, o);
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (p + k < np) to[k] = o[k];
        }
      }
    }

    if (keep) {
      const float fade = __builtin_amdgcn_exp2f(total.x);
      const int back = -ew - __float_as_int(scale.y);
      f32x4 add[kTiles][kCh];
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int m = 0; m < kCh; ++m) add[t][m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int step = 0; step < 2; ++step) {
        if (32 * step >= L) continue;
        f16x8 wh[kCh], wl[kCh];
#pragma unroll
        for (int m = 0; m < kCh; ++m) {
          const int p = 16 * (ch0 + m) + lo16, from = p * 64 + (((4 * step + lq) ^ scan_place(p)) << 3);
          wh[m] = *reinterpret_cast<const f16x8*>(&xw[0][from]);
          wl[m] = *reinterpret_cast<const f16x8*>(&xw[1][from]);
        }
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          const f16x8 bh = bhs[step][t], bl = bls[step][t];
#pragma unroll
          for (int m = 0; m < kCh; ++m) {
            add[t][m] = mma16(bh, wh[m], add[t][m]);
            add[t][m] = mma16(bh, wl[m], add[t][m]);
            add[t][m] = mma16(bl, wh[m], add[t][m]);
          }
        }
      }
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int m = 0; m < kCh; ++m)
#pragma unroll
          for (int e = 0; e < 4; ++e) st[t][m][e] = st[t][m][e] * fade + ldexpf(add[t][m][e], back);
      most_state = most_state * fade + scale.w * most * total.w;
      faded += static_cast<double>(total.x);
      has = true;
    }
  }

  if (first_run) {
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int m = 0; m < kCh; ++m) *stored(piece, t, m) = st[t][m];
    if (tid == 0) w.fades[static_cast<int64_t>(piece) * a.H + h] = static_cast<float>(faded);
  } else if (last_piece && slot >= 0) {
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int m = 0; m < kCh; ++m) {
        const int n = 16 * (tile0 + t) + 4 * q, p = 16 * (ch0 + m) + l16;
        if (p >= np) continue;
        float* const s = a.ssm_out + sbase + static_cast<int64_t>(p) * a.N + n;
        if (a.N % 4 == 0) {
          if (n < a.N) *reinterpret_cast<f32x4*>(s) = st[t][m];
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (n + e < a.N) s[e] = st[t][m][e];
        }
      }
  }
}

// ---------------------------------------------------------------------------------------------
// Sequences of up to 16 rows each, all equally long, that carry no state: one launch, everything in
// float32 on the matrix cores. A workgroup takes a sequence and group and up to kScanUnits (head, 64
// channels); its four waves convolve B and C together and then take the units in turn. Bound by
// latency and by the convolutions' and gates' exponentials: 1,024 sequences of 10 tokens, 16 heads of
// 64, state 64, bf16, take 50 us (1.3 TB/s), 291 by blocks of 64 tokens; in float32 66. Eight units a workgroup instead of 16: 55.
// ---------------------------------------------------------------------------------------------
constexpr int kScanShort = 16, kScanUnits = 16;

// bf16: four waves a SIMD, at the price of a few spilled registers (three without: 68 us instead of 50 at 1,024 x 10
// tokens, 16 heads of 64 x 64); float32's do not fit.
template <class T, int kN>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 4 : 3) void k_scan_short(ScanArgs a, int parts) {
  constexpr int kCols = 2 * kN, kRow = kCols + 4;
  __shared__ float u[kScanShort * kRow];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l16 = lane & 15, q = lane >> 4;
  const uint32_t id = static_cast<uint32_t>(block_number());
  const int part = id % parts, g = id / parts % a.G, i = id / (parts * a.G);
  if (i >= a.n_seqs) return;
  const int len = static_cast<int>(a.n_tokens / a.n_seqs), each = a.H / a.G;
  const int64_t first = static_cast<int64_t>(i) * len;
  const T* const xbc = static_cast<const T*>(a.xbc) + first * a.xbc_stride;

  // a unit's loads: x at tokens 4 q - 3 .. 4 q + 3 and channels 4 l16 .. + 3, the taps and biases, the step
  struct Unit {
    Four<T> raw[7], cw[4], cb;
    float dt, bias, decay, skip;
    int h, p0, np;
  };
  const int units = each * a.ptiles, last = min(units, (part + 1) * kScanUnits);
  auto load = [&](int n, Unit& v) {
    v.h = g * each + n / a.ptiles;
    v.p0 = n % a.ptiles * 64;
    v.np = min(64, a.P - v.p0);
    const int c0 = v.h * a.P + v.p0 + 4 * l16, ch = v.np - 4 * l16;
#pragma unroll
    for (int r = 0; r < 7; ++r) {
      const int t = 4 * q - 3 + r;
      v.raw[r] = Four<T>{};
      if (r >= 4 - a.W && t >= 0 && t < len) v.raw[r].load(xbc + static_cast<int64_t>(t) * a.xbc_stride + c0, ch);
    }
    v.cb = Four<T>{};
    if (a.conv_bias) v.cb.load(static_cast<const T*>(a.conv_bias) + c0, ch);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      v.cw[c] = Four<T>{};
      if (c < ch) v.cw[c].load_back(static_cast<const T*>(a.conv_weight) + static_cast<int64_t>(c0 + c) * a.W, a.W);
    }
    v.dt = l16 < len ? to_float(static_cast<const T*>(a.dt)[(first + l16) * a.dt_stride + v.h]) : 0.f;
    v.bias = a.dt_bias ? a.dt_bias[v.h] : 0.f;
    v.decay = a.decay[v.h];
    v.skip = a.skip ? a.skip[v.h] : 0.f;
  };
  Unit now;
  int n = part * kScanUnits + wave;
  if (n < last) load(n, now);

  {
    constexpr int kParts = kCols < 256 ? 256 / kCols : 1, kTokens = kScanShort / kParts;
    const int t0 = kCols < 256 ? tid / kCols * kTokens : 0;
    for (int col = kCols < 256 ? tid % kCols : tid; col < kCols; col += 256) {
      const int k = col < kN ? col : col - kN;
      const int c = a.H * a.P + (col < kN ? 0 : a.G * a.N) + g * a.N + k;
      float raw[kTokens + 3];
#pragma unroll
      for (int r = 0; r < kTokens + 3; ++r) {
        const int t = t0 - 3 + r;
        raw[r] = (k < a.N && r >= 4 - a.W && t >= 0 && t < len) ? to_float(xbc[static_cast<int64_t>(t) * a.xbc_stride + c]) : 0.f;
      }
      Four<T> cw;
      float cb = 0.f;
      if (k < a.N) {
        cw.load_back(static_cast<const T*>(a.conv_weight) + static_cast<int64_t>(c) * a.W, a.W);
        if (a.conv_bias) cb = to_float(static_cast<const T*>(a.conv_bias)[c]);
      }
#pragma unroll
      for (int t = 0; t < kTokens; ++t) {
        float v = cb + cw.at(3) * raw[t + 3] + cw.at(2) * raw[t + 2];
        if (a.W > 2) v += cw.at(1) * raw[t + 1];
        if (a.W > 3) v += cw.at(0) * raw[t];
        u[(t0 + t) * kRow + col] = (k < a.N && t0 + t < len) ? silu(v) : 0.f;
      }
    }
  }
  __syncthreads();
  // C_i B_j^T at i = l16 and j = 4 q + e; product t of four takes column 4 q + t of sixteen from each lane
  f32x4 cb = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int k = 0; k < kN; k += 16) {
    const f32x4 bj = *reinterpret_cast<const f32x4*>(u + l16 * kRow + k + 4 * q);
    const f32x4 ci = *reinterpret_cast<const f32x4*>(u + l16 * kRow + kN + k + 4 * q);
#pragma unroll
    for (int t = 0; t < 4; ++t) cb = __builtin_amdgcn_mfma_f32_16x16x4f32(bj[t], ci[t], cb, 0, 0, 0);
  }

  while (n < last) {
    const int h = now.h, p = now.p0 + 16 * q, np = now.np - 16 * q;  // the lane's channels of y: p .. p + 15
    const int64_t row = first + l16;
    T zv[16];
    if (a.z && l16 < len) {
      const T* const z = static_cast<const T*>(a.z) + row * a.z_stride + static_cast<int64_t>(h) * a.P + p;
      if (np >= 16) {
        load_once(zv, z);
      } else {
#pragma unroll
        for (int k = 0; k < 16; ++k) zv[k] = k < np ? z[k] : T(0);
      }
    }
    float x[4][4];  // [token 4 q + t][channel 4 l16 + c]
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float v = now.cb.at(c) + now.cw[c].at(3) * now.raw[t + 3].at(c) + now.cw[c].at(2) * now.raw[t + 2].at(c);
        if (a.W > 2) v += now.cw[c].at(1) * now.raw[t + 1].at(c);
        if (a.W > 3) v += now.cw[c].at(0) * now.raw[t].at(c);
        x[t][c] = (4 * q + t < len && 4 * l16 + c < now.np) ? silu(v) : 0.f;
      }
    const float step = l16 < len ? softplus(now.dt + now.bias) : 0.f, skip = now.skip;
    double s = scan_log_decay(step, now.decay);
#pragma unroll
    for (int m = 1; m < 16; m <<= 1) {
      const double o = __shfl_up(s, m, 16);
      if (l16 >= m) s += o;
    }
    n += 4;
    if (n < last) load(n, now);

    float mix[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = 4 * q + e;
      const float v = cb[e] * __shfl(step, j) * __builtin_amdgcn_exp2f(static_cast<float>(s - __shfl(s, j)));
      mix[e] = j < l16 ? v : (j == l16 ? v + skip : 0.f);
    }
    f32x4 y[4];  // y[c][e]: channel p + 4 e + c of token l16
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      y[c] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int e = 0; e < 4; ++e) y[c] = __builtin_amdgcn_mfma_f32_16x16x4f32(x[e][c], mix[e], y[c], 0, 0, 0);
    }
    if (l16 < len) {
      T o[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        float v = y[k & 3][k >> 2];
        if (a.z) v *= silu(to_float(zv[k]));
        o[k] = from_float<T>(v);
      }
      T* const to = static_cast<T*>(a.y) + row * a.y_stride + static_cast<int64_t>(h) * a.P + p;
      if (np >= 16) {
        store_once(to, o);
      } else {
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (k < np) to[k] = o[k];
      }
    }
  }
}

// The rings after a prompt call, a launch of its own: in place, every reader of the old rings is
// done. Workgroups go by sequence and 256 channels. 5 us for one sequence of 4,352 channels: the latency of a launch.
template <class T>
__global__ __launch_bounds__(256) void k_scan_ring(ScanArgs a, ScanWork w, int cblocks) {
  const uint32_t id = static_cast<uint32_t>(block_number());
  const int i = id / cblocks, c = (id % cblocks) * 256 + threadIdx.x;
  if (i >= a.n_seqs) return;
  const int slot = w.slots[i];
  if (slot < 0 || c >= a.C) return;
  const ScanSeq sq = scan_seq(a, w, i);
  const int pos = a.positions ? max(a.positions[i], 0) : 0;
  const T* ring = static_cast<const T*>(a.conv_in) + static_cast<int64_t>(slot) * a.W * a.C + c;
  T* out = static_cast<T*>(a.conv_out) + static_cast<int64_t>(slot) * a.W * a.C + c;
  for (int e = 0; e < a.W; ++e) {
    // the newest of this call's tokens whose place is e modulo W
    const int64_t last = static_cast<int64_t>(pos) + sq.len - 1;
    const int64_t q = last - (((last - e) % a.W) + a.W) % a.W;
    if (q >= pos)
      out[static_cast<int64_t>(e) * a.C] = static_cast<const T*>(a.xbc)[(sq.first + q - pos) * a.xbc_stride + c];
    else if (a.conv_in != a.conv_out)
      out[static_cast<int64_t>(e) * a.C] = ring[static_cast<int64_t>(e) * a.C];
  }
}

}  // namespace cdrge
