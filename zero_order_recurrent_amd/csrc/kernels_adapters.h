// A projection shared by all rows beside a low-rank adapter by row:
//   y_r = W x_r + b + s_r U_a (D_a x_r),  a = row_adapter[r].
//
// The parts:
//   down      vp[ks][r][j] = sum over the ks-th slice of K of D_a[j][k] x_r[k], by tiles of 64 rows.
//             Rows need no order: a tile runs once for each adapter that it meets and keeps, of each
//             run, the rows that name the adapter.
//   shared    W x, either in tiles that end with the epilogue, or in slices of K whose float32 sums
//             (P[s][r][o]) the epilogue's own launch adds up: with few rows the tiles alone would not
//             fill the chip.
//   epilogue  + bias + U_a v_r, v_r = s_r sum_ks vp, from the same matrix-core tiles, again once for
//             each adapter among 16 rows and kept by selection: what one adapter holds (NaN
//             included) cannot reach another's rows.
//
// Both element types run on the matrix cores with 16 bytes of a row in each lane: for bf16 that is
// one 16x16x32 product over 32 columns, for float32 four 16x16x4 products over 16 columns, in which
// product t takes element t of every lane - a permutation of the reduction index that both operands
// share. The operands are W (16 outputs) and x (16 rows), so that a lane ends with adjacent outputs
// of one row; tile t of four takes the outputs 16 (i / 4) + 4 t + i % 4 for its rows i, which makes a
// lane's outputs of all four tiles 16 adjacent ones.
#pragma once
#include "operators_common.h"

namespace cdrge {

struct AdapterArgs {
  const void* x;
  int64_t x_stride;
  const void* weight;
  int64_t weight_stride;
  const void* bias;
  const void* down;
  const void* up;
  const int32_t* ranks;
  const int32_t* row_adapter;
  const float* row_scale;
  void* y;
  int64_t y_stride;
  float* vp;        // [v_slices][n_rows][R]
  float* partial;   // [slices][n_rows][o_pad]
  int64_t n_rows;
  int K, O, A, R;
  int v_slices, v_cols;    // slices of K of the down product, columns of each (a multiple of 128)
  int v_slots;             // workgroups that share a row tile's adapters
  int slices, slice_cols;  // slices of K of the shared product (1: the tiles end with the epilogue)
  int o_pad;               // O rounded up to 64
  int tiles_r, tiles_o;    // tiles of the shared product
};

template <class T>
struct Frag;  // 16 bytes of a row per lane
template <>
struct Frag<uint16_t> {
  static constexpr int kCols = 32, kPer = 8;
  bf16x8 v;
};
template <>
struct Frag<float> {
  static constexpr int kCols = 16, kPer = 4;
  f32x4 v;
};

__device__ __forceinline__ f32x4 mma(const Frag<uint16_t>& a, const Frag<uint16_t>& b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(const Frag<float>& a, const Frag<float>& b, f32x4 c) {
#pragma unroll
  for (int t = 0; t < 4; ++t) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[t], b.v[t], c, 0, 0, 0);
  return c;
}

// Columns k .. k + kPer - 1 of a row that ends at column n: one 16-byte load where they lie inside (global
// memory takes it at any element's alignment), element by element at the end, zero past it.
template <class T>
__device__ __forceinline__ Frag<T> load_frag(const T* row, int k, int n) {
  Frag<T> f;
  if (k + Frag<T>::kPer <= n) {
    __builtin_memcpy(&f.v, row + k, 16);
    return f;
  }
  T e[Frag<T>::kPer];
#pragma unroll
  for (int i = 0; i < Frag<T>::kPer; ++i) e[i] = k + i < n ? row[k + i] : T(0);
  __builtin_memcpy(&f.v, e, 16);
  return f;
}

__device__ __forceinline__ int rank_of(const AdapterArgs& a, int ad) {
  return a.ranks ? min(max(a.ranks[ad], 0), a.R) : a.R;
}

// ---------------------------------------------------------------------------------------------
// down: one workgroup of four waves takes 64 rows (a lane knows the adapter of the row of its
// number), one slice of K, which its waves share step by step, and every v_slots-th of the adapters
// that the rows name.
// ---------------------------------------------------------------------------------------------
template <class T>
__device__ __forceinline__ void adapter_down(const AdapterArgs& a, int64_t tile, int slice, int slot, f32x4 (&lds)[4][4][64]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, q = lane >> 4;
  const int64_t r0 = tile * 64;
  const int ad = r0 + lane < a.n_rows ? a.row_adapter[r0 + lane] : -1;
  const T* x[4];
#pragma unroll
  for (int m = 0; m < 4; ++m) x[m] = static_cast<const T*>(a.x) + min(r0 + 16 * m + l16, a.n_rows - 1) * a.x_stride;
  const int k0 = slice * a.v_cols, k1 = min(a.K, k0 + a.v_cols);
  uint64_t todo = __ballot(ad >= 0 && ad < a.A);
  for (int n = 0; todo; ++n) {
    const int cur = __shfl(ad, __builtin_ctzll(todo));
    const uint64_t mine = __ballot(ad == cur);
    todo &= ~mine;
    if (n % a.v_slots != slot) continue;
    const int rank = rank_of(a, cur);
    for (int j0 = 0; j0 < rank; j0 += 16) {
      const T* d = static_cast<const T*>(a.down) + (static_cast<int64_t>(cur) * a.R + min(j0 + l16, rank - 1)) * a.K;
      f32x4 acc[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) acc[m] = f32x4{0.f, 0.f, 0.f, 0.f};
      for (int k = k0 + wave * Frag<T>::kCols; k < k1; k += 4 * Frag<T>::kCols) {
        const Frag<T> df = load_frag<T>(d, k + q * Frag<T>::kPer, k1);
#pragma unroll
        for (int m = 0; m < 4; ++m)
          if ((mine >> (16 * m)) & 0xffffu) acc[m] = mma(df, load_frag<T>(x[m], k + q * Frag<T>::kPer, k1), acc[m]);
      }
#pragma unroll
      for (int m = 0; m < 4; ++m) lds[wave][m][lane] = acc[m];
      __syncthreads();
      // wave m sums row tile m: rank indexes j0 + 4 q + e of row 16 m + l16
      f32x4 sum = lds[0][wave][lane];
#pragma unroll
      for (int w = 1; w < 4; ++w) sum += lds[w][wave][lane];
      __syncthreads();
      if ((mine >> (16 * wave + l16)) & 1) {
        float* v = a.vp + (static_cast<int64_t>(slice) * a.n_rows + r0 + 16 * wave + l16) * a.R + j0 + 4 * q;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (j0 + 4 * q + e < rank) v[e] = sum[e];
      }
    }
  }
}

template <class T>
__global__ __launch_bounds__(256) void k_adapter_down(AdapterArgs a) {
  __shared__ f32x4 lds[4][4][64];
  const int slot = blockIdx.x % a.v_slots, slice = (blockIdx.x / a.v_slots) % a.v_slices;
  adapter_down<T>(a, blockIdx.x / (a.v_slots * a.v_slices), slice, slot, lds);
}

// ---------------------------------------------------------------------------------------------
// epilogue: of the sums of kAll row tiles, the kMT from kFirst on; sums[kFirst + m][t][e] is output
// o0 + 16 q + 4 t + e of row r0 + 16 m + l16.
// ---------------------------------------------------------------------------------------------

// v_r from column j on: the sum over the slices of K, times the row's scale, zero from column n on.
template <int kPer>
__device__ __forceinline__ void v_values(const AdapterArgs& a, int64_t r, int j, int n, float scale, float (&f)[kPer]) {
#pragma unroll
  for (int i = 0; i < kPer; ++i) f[i] = 0.f;
  if (j >= n) return;
  const float* v = a.vp + r * a.R + j;
  if (j + kPer <= n) {
    for (int ks = 0; ks < a.v_slices; ++ks, v += a.n_rows * a.R) {
      float e[kPer];
      __builtin_memcpy(e, v, sizeof(e));
#pragma unroll
      for (int i = 0; i < kPer; ++i) f[i] += e[i];
    }
  } else {
    for (int ks = 0; ks < a.v_slices; ++ks, v += a.n_rows * a.R)
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (j + i < n) f[i] += v[i];
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) f[i] *= scale;
}

// v_r as an operand. bf16 takes it in two halves, which keeps 16 bits of it.
__device__ __forceinline__ void v_frag(const float (&f)[4], Frag<float>& hi, Frag<float>&) {
#pragma unroll
  for (int i = 0; i < 4; ++i) hi.v[i] = f[i];
}
__device__ __forceinline__ void v_frag(const float (&f)[8], Frag<uint16_t>& hi, Frag<uint16_t>& low) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    hi.v[i] = static_cast<__bf16>(f[i]);
    // an infinite v has no low half (inf - inf would turn it into NaN)
    low.v[i] = static_cast<__bf16>(fabsf(f[i]) <= 3.38953139e38f ? f[i] - static_cast<float>(hi.v[i]) : 0.f);
  }
}

// Columns from j on of the four output tiles of adapter cur's up matrix.
template <class T>
__device__ __forceinline__ void up_frags(const AdapterArgs& a, int cur, int rank, int o0, int j, Frag<T> (&u)[4]) {
  const int l16 = threadIdx.x & 15;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int o = min(o0 + 16 * (l16 >> 2) + 4 * t + (l16 & 3), a.O - 1);
    u[t] = load_frag<T>(static_cast<const T*>(a.up) + (static_cast<int64_t>(cur) * a.O + o) * a.R, j, rank);
  }
}

template <class T, int kFirst, int kMT, int kAll>
__device__ __forceinline__ void adapter_epilogue(const AdapterArgs& a, int64_t r0, int o0, f32x4 (&sums)[kAll][4]) {
  f32x4 acc[kMT][4];
#pragma unroll
  for (int m = 0; m < kMT; ++m)
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[m][t] = sums[kFirst + m][t];
  constexpr int kPer = Frag<T>::kPer, kCols = Frag<T>::kCols;
  const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
  int ad[kMT];
#pragma unroll
  for (int m = 0; m < kMT; ++m) {
    const int64_t r = r0 + 16 * m + l16;
    ad[m] = (a.row_adapter && r < a.n_rows) ? a.row_adapter[r] : -1;
  }
  if (a.row_adapter && a.A > 0) {
    const bool narrow = a.R <= kCols;  // one product a tile: all of v is fetched at once, and U once for equal neighbours
    Frag<T> vh[kMT], vl[kMT], u[4];
    int rank[kMT], u_of = -1;
    float scale[kMT];
#pragma unroll
    for (int m = 0; m < kMT; ++m) {
      const bool has = ad[m] >= 0 && ad[m] < a.A;
      rank[m] = has ? rank_of(a, ad[m]) : 0;
      scale[m] = has && a.row_scale ? a.row_scale[r0 + 16 * m + l16] : 1.f;
    }
    if (narrow) {
#pragma unroll
      for (int m = 0; m < kMT; ++m) {
        float f[kPer];
        v_values<kPer>(a, r0 + 16 * m + l16, q * kPer, rank[m], scale[m], f);
        v_frag(f, vh[m], vl[m]);
      }
    }
#pragma unroll
    for (int m = 0; m < kMT; ++m) {
      uint32_t todo = static_cast<uint32_t>(__ballot(rank[m] > 0)) & 0xffffu;
      while (todo) {
        const int first = __builtin_ctz(todo);
        const int cur = __builtin_amdgcn_readlane(ad[m], first), n = __builtin_amdgcn_readlane(rank[m], first);
        const bool mine = ad[m] == cur;
        todo &= ~static_cast<uint32_t>(__ballot(mine));
        f32x4 low[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) low[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (narrow) {
          if (cur != u_of) up_frags<T>(a, cur, n, o0, q * kPer, u);
          u_of = cur;
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            low[t] = mma(u[t], vh[m], low[t]);
            if (sizeof(T) == 2) low[t] = mma(u[t], vl[m], low[t]);
          }
        } else {
          for (int j = 0; j < n; j += kCols) {
            float f[kPer];
            Frag<T> hi, lo;
            v_values<kPer>(a, r0 + 16 * m + l16, j + q * kPer, mine ? n : 0, scale[m], f);
            v_frag(f, hi, lo);
            up_frags<T>(a, cur, n, o0, j + q * kPer, u);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              low[t] = mma(u[t], hi, low[t]);
              if (sizeof(T) == 2) low[t] = mma(u[t], lo, low[t]);
            }
          }
        }
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[m][t][e] = mine ? acc[m][t][e] + low[t][e] : acc[m][t][e];
      }
    }
  }
  const int o = o0 + 16 * q;
  float bias[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) bias[i] = a.bias && o + i < a.O ? to_float(static_cast<const T*>(a.bias)[o + i]) : 0.f;
#pragma unroll
  for (int m = 0; m < kMT; ++m) {
    const int64_t r = r0 + 16 * m + l16;
    if (r >= a.n_rows) continue;
    T* y = static_cast<T*>(a.y) + r * a.y_stride + o;
    T out[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) out[i] = from_float<T>(ad[m] >= a.A ? __builtin_nanf("") : acc[m][i >> 2][i & 3] + bias[i]);
    if (o + 16 <= a.O) {
      __builtin_memcpy(y, out, sizeof(out));
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (o + i < a.O) y[i] = out[i];
    }
  }
}

// The epilogue as a launch of its own, after a shared product in slices: 16 rows x 64 outputs a wave.
template <class T>
__global__ __launch_bounds__(64) void k_adapter_finish(AdapterArgs a) {
  const int lane = threadIdx.x, l16 = lane & 15, q = lane >> 4;
  const int64_t r = static_cast<int64_t>(blockIdx.y) * 16 + l16;
  const int o0 = blockIdx.x * 64;
  f32x4 acc[1][4];
#pragma unroll
  for (int t = 0; t < 4; ++t) acc[0][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (r < a.n_rows)
    for (int s = 0; s < a.slices; ++s) {
      const float* p = a.partial + (static_cast<int64_t>(s) * a.n_rows + r) * a.o_pad + o0 + 16 * q;
#pragma unroll
      for (int t = 0; t < 4; ++t) acc[0][t] += *reinterpret_cast<const f32x4*>(p + 4 * t);
    }
  adapter_epilogue<T, 0, 1>(a, static_cast<int64_t>(blockIdx.y) * 16, o0, acc);
}

// ---------------------------------------------------------------------------------------------
// Up to 64 rows (kTiles tiles of 16): bound by reading W once. A workgroup takes 64 outputs and one
// slice of K; its four waves take its steps in turn, each with all rows and outputs, straight from
// global memory into the matrix cores' registers, and add up through LDS. Workgroups past those run
// the down product, which needs nothing from them.
// ---------------------------------------------------------------------------------------------
template <class T, int kTiles>
__global__ __launch_bounds__(256) void k_adapter_rows(AdapterArgs a) {
  __shared__ f32x4 lds[4][4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, q = lane >> 4;
  const int main_blocks = a.tiles_o * a.slices;
  if (static_cast<int>(blockIdx.x) >= main_blocks) {
    const int i = blockIdx.x - main_blocks;
    adapter_down<T>(a, 0, i / a.v_slots, i % a.v_slots, lds);
    return;
  }
  const int o0 = (blockIdx.x / a.slices) * 64, slice = blockIdx.x % a.slices;
  const int k0 = slice * a.slice_cols, k1 = min(a.K, k0 + a.slice_cols);
  const T* w[4];
  const T* x[kTiles];
#pragma unroll
  for (int t = 0; t < 4; ++t)
    w[t] = static_cast<const T*>(a.weight) + min(o0 + 16 * (l16 >> 2) + 4 * t + (l16 & 3), a.O - 1) * a.weight_stride;
#pragma unroll
  for (int m = 0; m < kTiles; ++m) x[m] = static_cast<const T*>(a.x) + min(int64_t(16 * m + l16), a.n_rows - 1) * a.x_stride;
  f32x4 acc[kTiles][4];
#pragma unroll
  for (int m = 0; m < kTiles; ++m)
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[m][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  constexpr int kCols = Frag<T>::kCols, kPer = Frag<T>::kPer;
  int k = k0 + wave * kCols;
  constexpr int kDeep = kTiles > 2 ? 2 : 4;  // steps whose loads are in flight together
  for (; k + (4 * (kDeep - 1) + 1) * kCols <= k1; k += 4 * kDeep * kCols) {
    Frag<T> wf[kDeep][4], xf[kDeep][kTiles];
#pragma unroll
    for (int s = 0; s < kDeep; ++s) {
      const int at = k + 4 * s * kCols + q * kPer;
#pragma unroll
      for (int t = 0; t < 4; ++t) __builtin_memcpy(&wf[s][t].v, w[t] + at, 16);
#pragma unroll
      for (int m = 0; m < kTiles; ++m) __builtin_memcpy(&xf[s][m].v, x[m] + at, 16);
    }
#pragma unroll
    for (int s = 0; s < kDeep; ++s)
#pragma unroll
      for (int m = 0; m < kTiles; ++m)
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[m][t] = mma(wf[s][t], xf[s][m], acc[m][t]);
  }
  for (; k < k1; k += 4 * kCols) {
    const int at = k + q * kPer;
    Frag<T> wf[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) wf[t] = load_frag<T>(w[t], at, k1);
#pragma unroll
    for (int m = 0; m < kTiles; ++m) {
      const Frag<T> xf = load_frag<T>(x[m], at, k1);
#pragma unroll
      for (int t = 0; t < 4; ++t) acc[m][t] = mma(wf[t], xf, acc[m][t]);
    }
  }
#pragma unroll
  for (int m = 0; m < kTiles; ++m) {
    if (m) __syncthreads();
#pragma unroll
    for (int t = 0; t < 4; ++t) lds[wave][t][lane] = acc[m][t];
    __syncthreads();
    f32x4 sum = lds[0][wave][lane];
#pragma unroll
    for (int v = 1; v < 4; ++v) sum += lds[v][wave][lane];
    const int r = 16 * m + l16;
    if (r < a.n_rows)
      *reinterpret_cast<f32x4*>(a.partial + (static_cast<int64_t>(slice) * a.n_rows + r) * a.o_pad + o0 + 16 * q + 4 * wave) = sum;
  }
}

// ---------------------------------------------------------------------------------------------
// More rows: tiles of kRowsT rows x kOutsT outputs. K goes through LDS in steps of 128 bytes of each
// row, two buffers deep, so that one barrier a step does: the loads of a step are issued before the
// products of the one before. Rows lie in LDS as eight 16-byte chunks each, chunk c of row i at
// place c ^ f(i), f such that the eight rows that a matrix-core read touches at a time take all
// eight places: no bank conflicts. kDirect (rows of x and W 16-byte aligned, K a multiple of a step)
// loads straight into LDS; otherwise the chunks pass through registers and are cut at K.
// ---------------------------------------------------------------------------------------------
// s_waitcnt operand: no vector memory load in flight (vmcnt 0), the other counters not waited for
constexpr int kWaitLoads = 0x0f70;

// 16 bytes a lane from global memory into LDS, lane by lane behind `to` (the same for the whole wave). The
// load has no register result. It is written as an instruction because the compiler, which cannot tell
// the two buffers apart, would wait for every load of this kind before any read of LDS; the wait that
// is needed stands before the step's barrier.
__device__ __forceinline__ void load_to_lds(const char* from, uint4* to) {
  const uint32_t at = __builtin_amdgcn_readfirstlane(
      static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) void*)to)));
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(from), "s"(at) : "memory");
}

__device__ __forceinline__ int place_x(int row) { return row & 7; }
__device__ __forceinline__ int place_w(int row) { return (row & 3) | ((row >> 2) & 4); }

template <class T, int kRowsT, int kOutsT, int kWavesR, int kWavesO, bool kDirect>
__global__ __launch_bounds__(64 * kWavesR * kWavesO, 2) void k_adapter_tiles(AdapterArgs a) {
  constexpr int kThreads = 64 * kWavesR * kWavesO;
  constexpr int kStep = 128 / sizeof(T);  // columns of a step
  constexpr int kPer = Frag<T>::kPer;
  constexpr int kMT = kRowsT / kWavesR / 16, kOT = kOutsT / kWavesO / 64;  // 16-row tiles, 64-output tiles of a wave
  constexpr int kLoads = (kRowsT + kOutsT) * 8 / kThreads;                // chunks a thread loads a step
  static_assert((kRowsT * 8) % kThreads == 0 && (kOutsT * 8) % kThreads == 0, "a load step takes one operand");
  extern __shared__ uint4 stage[];  // [2][(kRowsT + kOutsT) * 8]
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l16 = lane & 15, q = lane >> 4;
  const int wr = wave / kWavesO, wo = wave % kWavesO;

  // Tiles by XCD: workgroups go round the eight XCDs, each of which has its own L2. XCD i gets the
  // i-th eighth of the tiles, walked in columns of up to four row tiles.
  const int n_tiles = a.tiles_r * a.tiles_o, slice = blockIdx.x / n_tiles;
  int id = blockIdx.x % n_tiles;
  {
    const int per = n_tiles >> 3, rest = n_tiles & 7, xcd = id & 7;
    id = xcd * per + min(xcd, rest) + (id >> 3);
  }
  const int band = id / (4 * a.tiles_o), in_band = id % (4 * a.tiles_o);
  const int band_rows = min(4, a.tiles_r - 4 * band);
  const int64_t r0 = static_cast<int64_t>(4 * band + in_band % band_rows) * kRowsT;
  const int o0 = in_band / band_rows * kOutsT;
  const int k_first = slice * a.slice_cols, k_end = min(a.K, k_first + a.slice_cols);

  // chunk i of a thread: row (tid + i kThreads) / 8 of the stage (x rows, then W rows), place tid % 8
  const char* src[kLoads];
  int chunk[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int at = tid + i * kThreads, row = at >> 3;
    if (i < kRowsT * 8 / kThreads) {
      chunk[i] = (at & 7) ^ place_x(row);
      src[i] = reinterpret_cast<const char*>(static_cast<const T*>(a.x) + min(r0 + row, a.n_rows - 1) * a.x_stride);
    } else {
      chunk[i] = (at & 7) ^ place_w(row - kRowsT);
      src[i] = reinterpret_cast<const char*>(static_cast<const T*>(a.weight) + static_cast<int64_t>(min(o0 + row - kRowsT, a.O - 1)) * a.weight_stride);
    }
    src[i] += chunk[i] * 16;
  }
  uint4 hold[kDirect ? 1 : kLoads];
  auto fetch = [&](int k, int buf) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      if (kDirect) {
        // a wave's 64 chunks are adjacent in LDS, lane by lane
        uint4* to = stage + buf * (kRowsT + kOutsT) * 8 + (tid & ~63) + i * kThreads;
        load_to_lds(src[i] + static_cast<int64_t>(k) * sizeof(T), to);
      } else {
        const Frag<T> f = load_frag<T>(reinterpret_cast<const T*>(src[i] - chunk[i] * 16), k + chunk[i] * kPer, k_end);
        __builtin_memcpy(&hold[i], &f.v, 16);
      }
    }
  };
  auto settle = [&](int buf) {
    if (!kDirect) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) stage[buf * (kRowsT + kOutsT) * 8 + tid + i * kThreads] = hold[i];
    }
  };

  f32x4 acc[kOT][kMT][4];
#pragma unroll
  for (int n = 0; n < kOT; ++n)
#pragma unroll
    for (int m = 0; m < kMT; ++m)
#pragma unroll
      for (int t = 0; t < 4; ++t) acc[n][m][t] = f32x4{0.f, 0.f, 0.f, 0.f};

  fetch(k_first, 0);
  settle(0);
  if (kDirect) __builtin_amdgcn_s_waitcnt(kWaitLoads);
  __syncthreads();
  int buf = 0;
  for (int k = k_first; k < k_end; k += kStep, buf ^= 1) {
    const bool more = k + kStep < k_end;
    if (more) fetch(k + kStep, buf ^ 1);
    const uint4* sx = stage + buf * (kRowsT + kOutsT) * 8;
    const uint4* sw = sx + kRowsT * 8;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      Frag<T> wf[kOT][4];
#pragma unroll
      for (int n = 0; n < kOT; ++n)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int row = (wo * kOT + n) * 64 + 16 * (l16 >> 2) + 4 * t + (l16 & 3);
          __builtin_memcpy(&wf[n][t].v, &sw[row * 8 + ((4 * half + q) ^ place_w(row))], 16);
        }
#pragma unroll
      for (int m = 0; m < kMT; ++m) {
        const int row = (wr * kMT + m) * 16 + l16;
        Frag<T> xf;
        __builtin_memcpy(&xf.v, &sx[row * 8 + ((4 * half + q) ^ place_x(row))], 16);
#pragma unroll
        for (int n = 0; n < kOT; ++n)
#pragma unroll
          for (int t = 0; t < 4; ++t) acc[n][m][t] = mma(wf[n][t], xf, acc[n][m][t]);
      }
    }
    if (more) settle(buf ^ 1);
    // loads into LDS are this wave's own until they have arrived: wait before the others may read them
    if (kDirect) __builtin_amdgcn_s_waitcnt(kWaitLoads);
    __syncthreads();
  }

  const int64_t rw = r0 + wr * kMT * 16;
#pragma unroll
  for (int n = 0; n < kOT; ++n) {
    const int o = o0 + (wo * kOT + n) * 64;
    if (o >= a.O) continue;
    if (a.slices > 1) {
#pragma unroll
      for (int m = 0; m < kMT; ++m) {
        const int64_t r = rw + 16 * m + l16;
        if (r >= a.n_rows) continue;
        float* p = a.partial + (static_cast<int64_t>(slice) * a.n_rows + r) * a.o_pad + o + 16 * q;
#pragma unroll
        for (int t = 0; t < 4; ++t) *reinterpret_cast<f32x4*>(p + 4 * t) = acc[n][m][t];
      }
    } else {
      adapter_epilogue<T, 0, 4>(a, rw, o, acc[n]);
      if constexpr (kMT > 4) adapter_epilogue<T, 4, 4>(a, rw + 64, o, acc[n]);
    }
  }
}

}  // namespace cdrge
