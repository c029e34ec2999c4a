// A projection shared by all rows beside a low-rank adapter by row:
//   y_r = W x_r + b + s_r U_a (D_a x_r),  a = row_adapter[r].
//
// The parts:
//   down      vp[ks][r][j] = sum over the ks-th slice of K of D_a[j][k] x_r[k], by tiles of 64 rows.
//             Rows need no order: a tile runs once for each adapter that it meets and keeps, of each
//             run, the rows that name the adapter.
//   shared    W x, either in tiles, or in slices of K whose float32 sums
//             (P[s][r][o]) a later launch adds up: with few rows the tiles alone would not
//             fill the chip.
//   up        + bias + U_a v_r, v_r = s_r sum_ks vp. A tile of the shared product takes it as further
//             steps of its own reduction, one adapter after the other, with zeros for the rows that name
//             another; after a product in slices it is a launch that adds the slices as well and keeps
//             each adapter's rows by selection. What one adapter holds (NaN included) cannot reach
//             another's rows: see there.
//
// Both element types run on the matrix cores with 16 bytes of a row in each lane: for bf16 that is
// one 16x16x32 product over 32 columns, for float32 four 16x16x4 products over 16 columns, in which
// product t takes element t of every lane - a permutation of the reduction index that both operands
// share. The operands are W (16 outputs) and x (16 rows), so that a lane ends with adjacent outputs
// of one row; tile t of four takes the outputs 16 (i / 4) + 4 t + i % 4 for its rows i, which makes a
// lane's outputs of all four tiles 16 adjacent ones.
#pragma once
#include <type_traits>

#include "operators_common.h"

namespace cdrge {

constexpr int kMostVSlices = 4;  // slices of K of the down product

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
  float* vp;        // v in slices of K, [v_slices][n_rows][R], without the rows' scales
  void* vq;         // or v as operand rows (see k_adapter_down), [n_rows][vq_row] of T
  int vq_row;
  float* partial;   // [slices][n_rows][o_pad]
  int64_t n_rows;
  int K, O, A, R;
  int v_slices, v_cols;    // slices of K of the down product, columns of each
  int v_slots;             // workgroups that share a row tile's adapters
  int slices, slice_cols;  // slices of K of the shared product (1: the tiles write y)
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

// The 16 bytes from element `at` of a matrix on (global memory takes them at any element's alignment).
template <class T>
__device__ __forceinline__ Frag<T> load_frag(const T* at) {
  Frag<T> f;
  __builtin_memcpy(&f.v, at, 16);
  return f;
}

// The same where a row may end inside: elements from n on are zero. The load is one for all lanes, with no
// branch between a wave's loads; it may pass into the next row, but never past the matrix's last element
// (`total` elements): there it starts earlier and is moved into place.
template <class T>
__device__ __forceinline__ Frag<T> load_cut(const T* base, int64_t at, int64_t total, int n) {
  constexpr int kPer = Frag<T>::kPer;
  T e[kPer];
  if (total >= kPer) {
    const int64_t from = min(at, total - kPer);
    __builtin_memcpy(e, base + from, 16);
    const int late = static_cast<int>(min(at - from, static_cast<int64_t>(kPer)));
    if (__any(late != 0)) {
#pragma unroll
      for (int step = 1; step <= kPer; step *= 2)
        if (late & step) {
#pragma unroll
          for (int i = 0; i < kPer; ++i) e[i] = i + step < kPer ? e[i + step] : T(0);
        }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) e[i] = at + i < total ? base[at + i] : T(0);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) e[i] = i < n ? e[i] : T(0);
  Frag<T> f;
  __builtin_memcpy(&f.v, e, 16);
  return f;
}

// Elements from the first of a matrix to its last.
__device__ __forceinline__ int64_t span_x(const AdapterArgs& a) { return (a.n_rows - 1) * a.x_stride + a.K; }
__device__ __forceinline__ int64_t span_w(const AdapterArgs& a) { return static_cast<int64_t>(a.O - 1) * a.weight_stride + a.K; }
__device__ __forceinline__ int64_t span_up(const AdapterArgs& a) { return static_cast<int64_t>(a.A) * a.O * a.R; }

__device__ __forceinline__ int rank_of(const AdapterArgs& a, int ad) {
  return a.ranks ? min(max(a.ranks[ad], 0), a.R) : a.R;
}

// ---------------------------------------------------------------------------------------------
// down: one workgroup takes 64 rows (a lane knows the adapter of the row of its number), one slice of
// K, which its waves share step by step, and every v_slots-th of the adapters that the rows name.
// An adapter's rows lie side by side, wherever they are among the 64, so that it costs its own number of rows; with all
// 64 multiplied for each adapter, 48 rows over 40 adapters took 59 us instead of 39 (K and O 5888, bf16).
// Bound by latency, then by reading x: 8,192 rows of 4,096 in bf16 take 28 us (2.4 TB/s).
// Beside up to 64 rows' shared product it runs in slices of K, four waves each, that leave float32
// sums (vp). As a launch of its own it takes all of K with 16 waves, and for tiles that end the call it
// leaves operand rows (vq): v_r times the row's scale, zero from the rank up to a multiple of 32 columns,
// in bf16 as its high halves followed by its low ones, which keeps 16 bits of it.
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ int vq_columns(int rank) { return (rank + 31) & ~31; }

// A wave's share of the columns k .. k1 - 1 of 16 rows of D times kTiles tiles of rows of x.
template <class T, int kWaves, int kTiles, int kDeep>
__device__ __forceinline__ void down_steps(const T* ds, int64_t d, int64_t total, const T* xs, const int64_t (&x)[4], int64_t span, int k, int k1, int q, f32x4 (&acc)[4]) {
  constexpr int kCols = Frag<T>::kCols, kPer = Frag<T>::kPer;
  for (; k + (kWaves * (kDeep - 1) + 1) * kCols <= k1; k += kWaves * kDeep * kCols) {  // kDeep steps' loads in flight together
    Frag<T> df[kDeep], xf[kDeep][kTiles];
#pragma unroll
    for (int s = 0; s < kDeep; ++s) {
      const int at = k + kWaves * s * kCols + q * kPer;
      df[s] = load_frag<T>(ds + d + at);
#pragma unroll
      for (int m = 0; m < kTiles; ++m) xf[s][m] = load_frag<T>(xs + x[m] + at);
    }
#pragma unroll
    for (int s = 0; s < kDeep; ++s)
#pragma unroll
      for (int m = 0; m < kTiles; ++m) acc[m] = mma(df[s], xf[s][m], acc[m]);
  }
  for (; k < k1; k += kWaves * kCols) {
    const int at = k + q * kPer;
    const Frag<T> df = load_cut<T>(ds, d + at, total, k1 - at);
#pragma unroll
    for (int m = 0; m < kTiles; ++m) acc[m] = mma(df, load_cut<T>(xs, x[m] + at, span, k1 - at), acc[m]);
  }
}

template <class T, int kWaves>
__device__ __forceinline__ void adapter_down(const AdapterArgs& a, int64_t tile, int slice, int slot, f32x4 (&lds)[kWaves][4][64]) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l16 = lane & 15, q = lane >> 4;
  const int64_t r0 = tile * 64;
  const int ad = r0 + lane < a.n_rows ? a.row_adapter[r0 + lane] : -1;
  const T* const xs = static_cast<const T*>(a.x);
  const int k0 = slice * a.v_cols, k1 = min(a.K, k0 + a.v_cols);
  uint64_t todo = __ballot(ad >= 0 && ad < a.A);
  const float scale = (a.vq && a.row_scale && r0 + lane < a.n_rows) ? a.row_scale[r0 + lane] : 1.f;
  for (int n = 0; todo; ++n) {
    const int cur = __shfl(ad, __builtin_ctzll(todo));
    const uint64_t mine = __ballot(ad == cur);
    todo &= ~mine;
    if (n % a.v_slots != slot) continue;
    // rows of D past the rank give values that are not kept, so with up to 16 of them nothing waits for the rank
    const int rank = rank_of(a, cur), most = a.R <= 16 ? a.R : rank;
    // the adapter's rows side by side: place i holds the i-th of them (of places past the last: the first)
    const int count = __popcll(mine);
    const uint64_t below = (uint64_t(1) << lane) - 1;
    const int place = mine >> lane & 1 ? __popcll(mine & below) : count + __popcll(~mine & below);
    int from = __builtin_amdgcn_ds_permute(4 * place, lane);  // every lane sends its number to its place
    if (lane >= count) from = __builtin_ctzll(mine);
    int64_t x[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) x[m] = (r0 + __shfl(from, 16 * m + l16)) * a.x_stride;
    for (int j0 = 0; j0 < (a.vq ? vq_columns(most) : most); j0 += 16) {
      const T* const ds = static_cast<const T*>(a.down);
      const int64_t d = (static_cast<int64_t>(cur) * a.R + min(j0 + l16, most - 1)) * a.K;
      f32x4 acc[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) acc[m] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (j0 < most) {  // past the rank: zeros
        const int64_t total = static_cast<int64_t>(a.A) * a.R * a.K;
        if (count > 32)
          down_steps<T, kWaves, 4, 4>(ds, d, total, xs, x, span_x(a), k0 + wave * Frag<T>::kCols, k1, q, acc);
        else if (count > 16)
          down_steps<T, kWaves, 2, 4>(ds, d, total, xs, x, span_x(a), k0 + wave * Frag<T>::kCols, k1, q, acc);
        else
          down_steps<T, kWaves, 1, kWaves == 4 ? 8 : 4>(ds, d, total, xs, x, span_x(a), k0 + wave * Frag<T>::kCols, k1, q, acc);
      }
#pragma unroll
      for (int m = 0; m < 4; ++m) lds[wave][m][lane] = acc[m];
      __syncthreads();
      if (wave < 4) {
        // wave m sums row tile m: rank indexes j0 + 4 q + e of the row at place 16 m + l16
        f32x4 sum = lds[0][wave][lane];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) sum += lds[w][wave][lane];
        const int at = 16 * wave + l16, row = __shfl(from, at), j = j0 + 4 * q;
        if (a.vq) {
          const float s = __shfl(scale, row);
          T hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float f = j + e < rank ? sum[e] * s : 0.f;
            hi[e] = from_float<T>(f);
            // an infinite v has no low half (inf - inf would turn it into NaN)
            lo[e] = from_float<T>(fabsf(f) <= 3.38953139e38f ? f - to_float(hi[e]) : 0.f);
          }
          if (at < count) {
            T* v = static_cast<T*>(a.vq) + (r0 + row) * a.vq_row + j;
            __builtin_memcpy(v, hi, sizeof(hi));
            if (sizeof(T) == 2) __builtin_memcpy(v + a.vq_row / 2, lo, sizeof(lo));
          }
        } else if (at < count) {
          float* v = a.vp + (static_cast<int64_t>(slice) * a.n_rows + r0 + row) * a.R + j;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (j + e < rank) v[e] = sum[e];
        }
      }
      __syncthreads();
    }
  }
}

template <class T>
__global__ __launch_bounds__(1024) void k_adapter_down(AdapterArgs a) {
  __shared__ f32x4 lds[16][4][64];
  const uint32_t block = static_cast<uint32_t>(block_number());
  adapter_down<T, 16>(a, block / a.v_slots, 0, block % a.v_slots, lds);
}

// v_r from column j on: the sum over the slices of K, without the row's scale; columns from R on are zero.
// A row without an adapter gives what lies there, not to be used.
template <int kPer>
__device__ __forceinline__ void v_sums(const AdapterArgs& a, int64_t r, int j, float (&f)[kPer]) {
#pragma unroll
  for (int i = 0; i < kPer; ++i) f[i] = 0.f;
  if (j >= a.R || r >= a.n_rows) return;
  const float* v = a.vp + r * a.R + j;
  if (j + kPer <= a.R) {
    // all slices' loads at once; a slice past the last reads the last again and is not added
#pragma unroll
    for (int ks = 0; ks < kMostVSlices; ++ks) {
      float e[kPer];
      __builtin_memcpy(e, v + min(ks, a.v_slices - 1) * a.n_rows * a.R, sizeof(e));
#pragma unroll
      for (int i = 0; i < kPer; ++i) f[i] += ks < a.v_slices ? e[i] : 0.f;
    }
  } else {
    for (int ks = 0; ks < a.v_slices; ++ks, v += a.n_rows * a.R)
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (j + i < a.R) f[i] += v[i];
  }
}

// Those columns from j on, times the scale, with zero from column n on.
template <int kPer>
__device__ __forceinline__ void v_scaled(float (&f)[kPer], int j, int n, float scale) {
#pragma unroll
  for (int i = 0; i < kPer; ++i) f[i] = j + i < n ? f[i] * scale : 0.f;
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

// Columns from j on of the four output tiles of adapter cur's up matrix; up_cut sets those from n on to zero. Where a
// row is whole pieces a lane's piece is inside or outside, and nothing has to be moved within it; those outside are
// somebody's, and up_cut has to follow.
template <class T>
__device__ __forceinline__ bool up_whole(const AdapterArgs& a) { return a.R % Frag<T>::kPer == 0; }
template <class T, bool kWhole>
__device__ __forceinline__ void up_frags(const AdapterArgs& a, int cur, int o0, int j, Frag<T> (&u)[4]) {
  const int l16 = threadIdx.x & 15;
  const T* const up = static_cast<const T*>(a.up);
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int64_t row = (static_cast<int64_t>(cur) * a.O + min(o0 + 16 * (l16 >> 2) + 4 * t + (l16 & 3), a.O - 1)) * a.R;
    u[t] = kWhole ? load_frag<T>(up + row + min(j, a.R - Frag<T>::kPer)) : load_cut<T>(up, row + j, span_up(a), a.R - j);
  }
}
template <class T>
__device__ __forceinline__ void up_cut(int j, int n, Frag<T> (&u)[4]) {
  constexpr int kEach = 4 / sizeof(T);  // elements of a word
  uint32_t keep[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int left = n - j - kEach * i;
    keep[i] = left >= kEach ? ~0u : (left > 0 ? 0xffffu : 0u);
  }
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    uint32_t v[4];
    __builtin_memcpy(v, &u[t].v, 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] &= keep[i];
    __builtin_memcpy(&u[t].v, v, 16);
  }
}

// ---------------------------------------------------------------------------------------------
// After a shared product in slices: 16 rows x 64 outputs by four waves, which share the slices and the
// adapters among the rows and add up through LDS. The time is the latency of a few loads, so each wave
// has those of up to four adapters in flight together (48 rows, 5888 outputs, 40 adapters of
// rank 16: 7.7 us, of rank 12 10.4; without adapters 4.6).
// sum[t][e] is output o0 + 16 q + 4 t + e of row l16.
// ---------------------------------------------------------------------------------------------
template <class T>
__global__ __launch_bounds__(256) void k_adapter_finish(AdapterArgs a) {
  constexpr int kPer = Frag<T>::kPer, kCols = Frag<T>::kCols;
  __shared__ f32x4 lds[4][4][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l16 = lane & 15, q = lane >> 4;
  const int64_t r = static_cast<int64_t>(blockIdx.y) * 16 + l16;
  const bool rok = r < a.n_rows;
  const int o0 = blockIdx.x * 64;
  const int ad = (a.row_adapter && rok) ? a.row_adapter[r] : -1;
  const bool narrow = a.R <= kCols;  // one product a tile
  // what no adapter decides is asked for first
  const int o = o0 + 16 * q + 4 * wave;
  float bias[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) bias[e] = a.bias && o + e < a.O ? to_float(static_cast<const T*>(a.bias)[o + e]) : 0.f;
  const float row_scale = a.row_scale && rok ? a.row_scale[r] : 1.f;
  float vs[kPer];
  if (narrow && a.row_adapter && a.A > 0) v_sums<kPer>(a, r, q * kPer, vs);
  f32x4 sum[4];
  auto add_slices = [&]() {
#pragma unroll
    for (int t = 0; t < 4; ++t) sum[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (!rok) return;
    const float* p = a.partial + r * a.o_pad + o0 + 16 * q;
#pragma unroll 2
    for (int s = wave; s < a.slices; s += 4)
#pragma unroll
      for (int t = 0; t < 4; ++t) sum[t] += *reinterpret_cast<const f32x4*>(p + s * a.n_rows * a.o_pad + 4 * t);
  };
  add_slices();
  const bool has = ad >= 0 && ad < a.A;
  uint32_t todo = static_cast<uint32_t>(__ballot(has)) & 0xffffu;
  if (todo) {
    bool here = false;  // whether this wave takes the row's adapter
    // two rounds of loads: the adapters of the rows, with the sums; then everything that an adapter names
    const int rank = has ? rank_of(a, ad) : 0;
    const float scale = has ? row_scale : 1.f;
    while (todo) {
      // the next four of this wave's adapters (every fourth); one that is missing repeats the first
      int cur[4], got = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        cur[i] = i ? cur[0] : 0;
        for (int step = 0; step < 4 && todo; ++step) {
          const int c = __builtin_amdgcn_readlane(ad, __builtin_ctz(todo));
          todo &= ~static_cast<uint32_t>(__ballot(ad == c));
          if (step == wave) {
            cur[i] = c;
            got = i + 1;
          }
        }
      }
      if (!got) break;
#pragma unroll
      for (int i = 0; i < 4; ++i) here |= i < got && ad == cur[i];
      if (narrow) {
        Frag<T> u[4][4];
        if (up_whole<T>(a)) {
#pragma unroll
          for (int i = 0; i < 4; ++i) up_frags<T, true>(a, cur[i], o0, q * kPer, u[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) up_frags<T, false>(a, cur[i], o0, q * kPer, u[i]);
        }
        Frag<T> vh, vl;
        float f[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) f[i] = vs[i];
        v_scaled<kPer>(f, q * kPer, rank, scale);
        v_frag(f, vh, vl);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (a.ranks || up_whole<T>(a)) up_cut<T>(q * kPer, rank_of(a, cur[i]), u[i]);
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            f32x4 low = mma(u[i][t], vh, f32x4{0.f, 0.f, 0.f, 0.f});
            if (sizeof(T) == 2) low = mma(u[i][t], vl, low);
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[t][e] = (i < got && ad == cur[i]) ? sum[t][e] + low[e] : sum[t][e];
          }
        }
      } else {
        for (int i = 0; i < got; ++i) {
          const int c = i == 0 ? cur[0] : (i == 1 ? cur[1] : (i == 2 ? cur[2] : cur[3]));
          const int rc = rank_of(a, c);
          f32x4 low[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) low[t] = f32x4{0.f, 0.f, 0.f, 0.f};
          for (int j = 0; j < rc; j += kCols) {
            float f[kPer];
            Frag<T> hi, lo, u[4];
            if (up_whole<T>(a))
              up_frags<T, true>(a, c, o0, j + q * kPer, u);
            else
              up_frags<T, false>(a, c, o0, j + q * kPer, u);
            v_sums<kPer>(a, r, j + q * kPer, f);
            v_scaled<kPer>(f, j + q * kPer, ad == c ? rc : 0, scale);
            v_frag(f, hi, lo);
            up_cut<T>(j + q * kPer, rc, u);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              low[t] = mma(u[t], hi, low[t]);
              if (sizeof(T) == 2) low[t] = mma(u[t], lo, low[t]);
            }
          }
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[t][e] = ad == c ? sum[t][e] + low[t][e] : sum[t][e];
        }
      }
    }
    if constexpr (sizeof(T) == 2) {
      // Where U holds an infinity, the two halves of v give infinities of either sign, or one of them is zero, and NaN comes
      // out: such sums are formed anew of the whole v.
      bool lost = false;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) lost |= !(sum[t][e] == sum[t][e]);
      if (__any(lost && here)) {
        f32x4 old[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) old[t] = sum[t];
        add_slices();
        for (int j = 0; j < (here ? rank : 0); ++j) {
          float v[1];
          v_sums<1>(a, r, j, v);
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int at = min(o0 + 16 * q + 4 * t + e, a.O - 1);
              sum[t][e] += v[0] * scale * to_float(static_cast<const T*>(a.up)[(static_cast<int64_t>(ad) * a.O + at) * a.R + j]);
            }
        }
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[t][e] = here && !(old[t][e] == old[t][e]) ? sum[t][e] : old[t][e];
      }
    }
  }
#pragma unroll
  for (int t = 0; t < 4; ++t) lds[wave][t][lane] = sum[t];
  __syncthreads();
  f32x4 out = lds[0][wave][lane];
#pragma unroll
  for (int w = 1; w < 4; ++w) out += lds[w][wave][lane];
  if (!rok) return;
  T v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = from_float<T>(ad >= a.A ? __builtin_nanf("") : out[e] + bias[e]);
  T* y = static_cast<T*>(a.y) + r * a.y_stride + o;
  if (o + 4 <= a.O) {
    __builtin_memcpy(y, v, sizeof(v));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (o + e < a.O) y[e] = v[e];
  }
}

// ---------------------------------------------------------------------------------------------
// A row or a few, in one launch: a workgroup takes 16 outputs over all of K, its eight waves the steps in turn,
// and beside W's rows it reads those of D that the rows' adapters name (kD tiles of 16: every workgroup repeats that
// product, out of the caches), so that the up product can follow from shared memory. The latter runs in float32 on
// the vector unit, a thread an output. Bound by latency: one row, 1024 -> 4096 with an adapter of rank 16 in bf16, 6.1
// us, of which 3.6 are a launch; in float32 9.5.
// ---------------------------------------------------------------------------------------------
constexpr int kFewTiles = 4;  // tiles of D at most

template <class T, int kD>
__global__ __launch_bounds__(512) void k_adapter_few(AdapterArgs a) {
  constexpr int kWaves = 8, kCols = Frag<T>::kCols, kPer = Frag<T>::kPer, kDeep = 4;
  __shared__ f32x4 lds[1 + kD][kWaves][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l16 = lane & 15, q = lane >> 4;
  const int o0 = blockIdx.x * 16, tiles = (a.R + 15) >> 4;  // tiles of a row's adapter
  const T* const ws = static_cast<const T*>(a.weight);
  const T* const xs = static_cast<const T*>(a.x);
  const T* const ds = static_cast<const T*>(a.down);
  const int64_t w = static_cast<int64_t>(min(o0 + l16, a.O - 1)) * a.weight_stride, x = min(static_cast<int64_t>(l16), a.n_rows - 1) * a.x_stride;
  int64_t d[kD > 0 ? kD : 1];
#pragma unroll
  for (int t = 0; t < kD; ++t) {
    // tile t % tiles of row t / tiles; where there is none, adapter 0's stands in and is not used
    const int r = t / tiles;
    const int ad = r < a.n_rows ? a.row_adapter[r] : 0;
    d[t] = (static_cast<int64_t>(ad >= 0 && ad < a.A ? ad : 0) * a.R + min(t % tiles * 16 + l16, a.R - 1)) * a.K;
  }
  // the thread's output at the end: everything that it needs but the sums
  const int c = tid & 15, o = o0 + c, r = tid >> 4;
  const bool mine = r < a.n_rows && o < a.O;
  const int ad = mine && a.row_adapter ? a.row_adapter[r] : -1;
  const bool has = kD > 0 && ad >= 0 && ad < a.A;
  const float bias = mine && a.bias ? to_float(static_cast<const T*>(a.bias)[o]) : 0.f;
  const float scale = has && a.row_scale ? a.row_scale[r] : 1.f;
  const int rank = has ? rank_of(a, ad) : 0;
  const int64_t up = has ? (static_cast<int64_t>(ad) * a.O + o) * a.R : 0;

  f32x4 acc[1 + kD];
#pragma unroll
  for (int t = 0; t <= kD; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  Frag<T> wf[kDeep], xf[kDeep], df[kDeep][kD > 0 ? kD : 1];
  const int first = wave * kCols, whole = max(0, (a.K - first + (kWaves - 1) * kCols) / (kWaves * kCols));
  auto load = [&](int s, int n) {
    const int at = first + n * kWaves * kCols + q * kPer;
    wf[s] = load_frag<T>(ws + w + at);
    xf[s] = load_frag<T>(xs + x + at);
#pragma unroll
    for (int t = 0; t < kD; ++t) df[s][t] = load_frag<T>(ds + d[t] + at);
  };
  auto multiply = [&](int s) {
    acc[0] = mma(wf[s], xf[s], acc[0]);
#pragma unroll
    for (int t = 0; t < kD; ++t) acc[1 + t] = mma(df[s][t], xf[s], acc[1 + t]);
  };
  if (whole > 0) {
#pragma unroll
    for (int s = 0; s < kDeep; ++s) load(s, min(s, whole - 1));
    int n = 0;
    for (; n + kDeep < whole; n += kDeep)
#pragma unroll
      for (int s = 0; s < kDeep; ++s) {
        multiply(s);
        load(s, min(n + s + kDeep, whole - 1));
      }
#pragma unroll
    for (int s = 0; s < kDeep; ++s)
      if (n + s < whole) multiply(s);
  }
  const int k = first + whole * kWaves * kCols;
  if (k < a.K) {  // the step that the rows end in
    const int at = k + q * kPer;
    wf[0] = load_cut<T>(ws, w + at, span_w(a), a.K - at);
    xf[0] = load_cut<T>(xs, x + at, span_x(a), a.K - at);
#pragma unroll
    for (int t = 0; t < kD; ++t) df[0][t] = load_cut<T>(ds, d[t] + at, static_cast<int64_t>(a.A) * a.R * a.K, a.K - at);
    multiply(0);
  }
#pragma unroll
  for (int t = 0; t <= kD; ++t) lds[t][wave][lane] = acc[t];
  __syncthreads();
  if (!mine) return;
  // a tile's value for its row j (output or rank index) and row r of x: element j % 4 of lane 16 (j / 4) + r
  float sum = bias;
#pragma unroll
  for (int v = 0; v < kWaves; ++v) sum += reinterpret_cast<const float*>(&lds[0][v][(c >> 2) * 16 + r])[c & 3];
  float low = 0.f;
  for (int j0 = 0; j0 < rank; j0 += kPer) {
    const Frag<T> f = load_cut<T>(static_cast<const T*>(a.up), up + j0, span_up(a), rank - j0);
    T u[kPer];
    __builtin_memcpy(u, &f.v, 16);
#pragma unroll
    for (int i = 0; i < kPer; i += 4) {
      const int j = j0 + i;
      if (j >= rank) break;
      f32x4 v = lds[1 + r * tiles + (j >> 4)][0][((j & 15) >> 2) * 16 + r];
#pragma unroll
      for (int n = 1; n < kWaves; ++n) v += lds[1 + r * tiles + (j >> 4)][n][((j & 15) >> 2) * 16 + r];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (j + e < rank) low += v[e] * to_float(u[i + e]);
    }
  }
  if (has) sum += scale * low;
  static_cast<T*>(a.y)[r * a.y_stride + o] = from_float<T>(ad >= a.A ? __builtin_nanf("") : sum);
}

// ---------------------------------------------------------------------------------------------
// Up to 64 rows (kTiles tiles of 16): bound by reading W once, and by x, which every workgroup reads from the caches.
// K and O 5888, bf16: 16 us for one row (4.3 TB/s of W), 17 for 16, 23 for 48; in float32 74 for 48. Reading W past the caches is slower (48 rows
// and joining 41 us instead of 35), two adjacent steps a wave are no faster. A workgroup takes 64 outputs and one
// slice of K; its four waves take its steps in turn, each with all rows and outputs, straight from
// global memory into the matrix cores' registers, and add up through LDS. Workgroups past those run
// the down product, which needs nothing from them.
// ---------------------------------------------------------------------------------------------
template <class T, int kTiles>
__global__ __launch_bounds__(256, 2) void k_adapter_rows(AdapterArgs a) {
  __shared__ f32x4 lds[4][4][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l16 = lane & 15, q = lane >> 4;
  const int main_blocks = a.tiles_o * a.slices;
  if (static_cast<int>(blockIdx.x) >= main_blocks) {
    const int i = blockIdx.x - main_blocks;
    adapter_down<T, 4>(a, 0, i / a.v_slots, i % a.v_slots, lds);
    return;
  }
  const int o0 = (blockIdx.x / a.slices) * 64, slice = blockIdx.x % a.slices;
  const int k0 = slice * a.slice_cols, k1 = min(a.K, k0 + a.slice_cols);
  const T* const ws = static_cast<const T*>(a.weight);
  const T* const xs = static_cast<const T*>(a.x);
  int64_t w[4], x[kTiles];
#pragma unroll
  for (int t = 0; t < 4; ++t) w[t] = min(o0 + 16 * (l16 >> 2) + 4 * t + (l16 & 3), a.O - 1) * a.weight_stride;
#pragma unroll
  for (int m = 0; m < kTiles; ++m) x[m] = min(int64_t(16 * m + l16), a.n_rows - 1) * a.x_stride;
  f32x4 acc[kTiles][4];
#pragma unroll
  for (int m = 0; m < kTiles; ++m)
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[m][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  constexpr int kCols = Frag<T>::kCols, kPer = Frag<T>::kPer;
  constexpr int kDeep = kTiles < 4 ? 4 : 3;  // steps whose loads are in flight together, the next ones' behind the products of these
  int k = k0 + wave * kCols;
  const int whole = max(0, (k1 - k + 3 * kCols) / (4 * kCols));  // steps within the row
  Frag<T> wf[kDeep][4], xf[kDeep][kTiles];
  auto load = [&](int s, int n) {
    const int at = k + 4 * n * kCols + q * kPer;
#pragma unroll
    for (int t = 0; t < 4; ++t) wf[s][t] = load_frag<T>(ws + w[t] + at);
#pragma unroll
    for (int m = 0; m < kTiles; ++m) xf[s][m] = load_frag<T>(xs + x[m] + at);
  };
  auto multiply = [&](int s) {
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
      for (int t = 0; t < 4; ++t) acc[m][t] = mma(wf[s][t], xf[s][m], acc[m][t]);
  };
  if (whole > 0) {
#pragma unroll
    for (int s = 0; s < kDeep; ++s) load(s, min(s, whole - 1));
    int n = 0;
    for (; n + kDeep < whole; n += kDeep)
#pragma unroll
      for (int s = 0; s < kDeep; ++s) {
        multiply(s);
        load(s, min(n + s + kDeep, whole - 1));
      }
#pragma unroll
    for (int s = 0; s < kDeep; ++s)
      if (n + s < whole) multiply(s);
  }
  k += 4 * whole * kCols;
  if (k < k1) {  // the step that the row ends in
    const int at = k + q * kPer;
#pragma unroll
    for (int t = 0; t < 4; ++t) wf[0][t] = load_cut<T>(ws, w[t] + at, span_w(a), k1 - at);
#pragma unroll
    for (int m = 0; m < kTiles; ++m) xf[0][m] = load_cut<T>(xs, x[m] + at, span_x(a), k1 - at);
    multiply(0);
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
// More rows: tiles of kRowsT rows x kOutsT outputs, a wave takes kMT * 16 rows x kOT * 64 outputs.
// K goes through LDS in steps of 128 bytes of each row, two buffers deep, in two halves:
//
//   read half 1 of step k | products of half 0      wait for the loads of step k + 1, barrier
//   issue the loads of step k + 2 into the buffer just read | read half 0 of step k + 1 | products of half 1
//
// so that a load has a whole step to arrive, and LDS is read beside the matrix cores' work, never
// before it. Rows lie in LDS as eight 16-byte chunks each, chunk c of row i at place c ^ f(i), f such
// that the eight rows that a matrix-core read touches at a time take all eight places: no bank
// conflicts. kDirect (rows of x and W 16-byte aligned, K a multiple of a step) loads straight into
// LDS; otherwise the chunks pass through registers and are cut at K.
//
// 8,192 rows of 4,096 to 4,096 outputs, bf16, four adapters of rank 8: 238 us with the up product, 1,155 TFLOP/s (a
// large library product reaches 1,500, and takes 183 us for the shared part alone). The matrix cores are busy in 57%
// of the cycles; the reads and writes of LDS of a step take as long as its products, with few cycles to hide either
// in. Waves of 128 x 128, which would read a third less, keep their sums in the second half of the register file and
// lost more to the moves there.
// ---------------------------------------------------------------------------------------------

__device__ __forceinline__ int place_x(int row) { return row & 7; }
__device__ __forceinline__ int place_w(int row) { return (row & 3) | ((row >> 2) & 4); }

template <class T, int kRowsT, int kOutsT, int kWavesR, int kWavesO, bool kDirect>
__global__ __launch_bounds__(64 * kWavesR * kWavesO, 2) void k_adapter_tiles(AdapterArgs a) {
  constexpr int kThreads = 64 * kWavesR * kWavesO;
  constexpr int kStep = 128 / sizeof(T);  // columns of a step
  constexpr int kPer = Frag<T>::kPer;
  constexpr int kMT = kRowsT / kWavesR / 16, kOT = kOutsT / kWavesO / 64;
  constexpr int kLoadsX = kRowsT * 8 / kThreads, kLoadsW = kOutsT * 8 / kThreads;  // chunks a thread loads a step
  constexpr int kBuf = (kRowsT + kOutsT) * 8;
  constexpr int kPerTile = (kLoadsX + kLoadsW) / kMT;  // loads of a step beside one row tile's products
  static_assert(kPerTile * kMT == kLoadsX + kLoadsW, "all loads of a step are issued");
  static_assert((kRowsT * 8) % kThreads == 0 && (kOutsT * 8) % kThreads == 0, "a load takes rows of one operand");
  extern __shared__ uint4 stage[];  // [2][kBuf]: x rows, then W rows
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l16 = lane & 15, q = lane >> 4;
  const int wr = wave / kWavesO, wo = wave % kWavesO;

  // Tiles by XCD: workgroups go round the eight XCDs, each of which has its own L2. XCD i gets the
  // i-th eighth of the tiles, walked in columns of up to four row tiles.
  const int n_tiles = a.tiles_r * a.tiles_o;
  const uint32_t block = static_cast<uint32_t>(block_number());
  if (block >= static_cast<uint32_t>(n_tiles * a.slices)) {
    // after a product in slices the up product has a launch of its own, and the down product runs beside it
    if constexpr (kThreads == 256) {
      const uint32_t past = block - n_tiles * a.slices;
      if (a.slices > 1)
        adapter_down<T, 4>(a, past / (a.v_slots * a.v_slices), past / a.v_slots % a.v_slices, past % a.v_slots,
                           *reinterpret_cast<f32x4(*)[4][4][64]>(stage));
    }
    return;
  }
  const int slice = block / n_tiles;
  int id = block % n_tiles;
  {
    const int per = n_tiles >> 3, rest = n_tiles & 7, xcd = id & 7;
    id = xcd * per + min(xcd, rest) + (id >> 3);
  }
  const int band = id / (4 * a.tiles_o), in_band = id % (4 * a.tiles_o);
  const int band_rows = min(4, a.tiles_r - 4 * band);
  const int64_t r0 = static_cast<int64_t>(4 * band + in_band % band_rows) * kRowsT;
  const int o0 = in_band / band_rows * kOutsT;
  const int k_first = slice * a.slice_cols, k_end = min(a.K, k_first + a.slice_cols);

  // load i of a thread: row (tid + i kThreads) / 8 of its operand, place tid % 8. Offsets in bytes from
  // the tile's first row fit 32 bits: the host sends strides past 2^23 bytes down the other way.
  const char* xb = reinterpret_cast<const char*>(static_cast<const T*>(a.x) + r0 * a.x_stride);
  const char* wb = reinterpret_cast<const char*>(static_cast<const T*>(a.weight) + static_cast<int64_t>(o0) * a.weight_stride);
  static_assert(kThreads % 256 == 0, "all loads of a thread have the same chunk");
  const int chunk_x = (tid & 7) ^ place_x(tid >> 3), chunk_w = (tid & 7) ^ place_w(tid >> 3);
  const int last_x = static_cast<int>(min(static_cast<int64_t>(kRowsT), a.n_rows - r0)) - 1, last_w = min(kOutsT, a.O - o0) - 1;
  auto row_x = [&](int t, int i) { return min((t + i * kThreads) >> 3, last_x); };
  auto row_w = [&](int t, int i) { return min((t + i * kThreads) >> 3, last_w); };
  // The thread's number, as a value that the compiler has to take for a new one each time: otherwise it
  // keeps every address that follows from it across the loop, and spills them for the products' registers.
  auto fresh_tid = [&]() {
    int t = tid;
    asm volatile("" : "+v"(t));
    return t;
  };
  const uint32_t stride_x = static_cast<uint32_t>(a.x_stride * sizeof(T)), stride_w = static_cast<uint32_t>(a.weight_stride * sizeof(T));
  uint4 hold[kDirect ? 1 : kLoadsX + kLoadsW];
  // Load n of a step (n counts x's, then W's), straight into LDS: a wave's 64 chunks are adjacent there.
  // Rows past the operand's last are read from the last.
  auto load = [&](int n, int k, int buf, int ft) {
    const bool of_x = n < kLoadsX;
    const int i = of_x ? n : n - kLoadsX;
    const uint32_t stride = of_x ? stride_x : stride_w, last = (of_x ? last_x : last_w) * stride;
    const uint32_t row = (ft >> 3) * stride + (i * kThreads / 8) * stride;
    load_to_lds((of_x ? xb : wb) + static_cast<int64_t>(k) * sizeof(T), min(row, last) + 16 * (of_x ? chunk_x : chunk_w),
                stage + buf * kBuf + (of_x ? 0 : kRowsT * 8) + (tid & ~63) + i * kThreads);
  };
  auto fetch = [&](int k, int buf) {
    const int ft = fresh_tid();
    if (kDirect) {
#pragma unroll
      for (int n = 0; n < kLoadsX + kLoadsW; ++n) load(n, k, buf, ft);
    } else {
      const bool whole = k + kStep <= k_end;
      auto one = [&](uint4& to, const void* base, int64_t row, int col, int64_t span) {
        const T* m = static_cast<const T*>(base);
        const Frag<T> f = whole ? load_frag<T>(m + row + col) : load_cut<T>(m, row + col, span, k_end - col);
        __builtin_memcpy(&to, &f.v, 16);
      };
#pragma unroll
      for (int i = 0; i < kLoadsX; ++i)
        one(hold[i], a.x, (r0 + row_x(ft, i)) * a.x_stride, k + chunk_x * kPer, span_x(a));
#pragma unroll
      for (int i = 0; i < kLoadsW; ++i)
        one(hold[kLoadsX + i], a.weight, (o0 + row_w(ft, i)) * a.weight_stride, k + chunk_w * kPer, span_w(a));
    }
  };
  // ends a fetch: its data is this wave's own until it has arrived in LDS
  auto settle = [&](int buf) {
    if (kDirect) {
      __builtin_amdgcn_s_waitcnt(kWaitLoads);
    } else {
#pragma unroll
      for (int i = 0; i < kLoadsX; ++i) stage[buf * kBuf + tid + i * kThreads] = hold[i];
#pragma unroll
      for (int i = 0; i < kLoadsW; ++i) stage[buf * kBuf + kRowsT * 8 + tid + i * kThreads] = hold[kLoadsX + i];
    }
  };
  // The operands of one half of a step: W's for all output tiles, x's by row tile.
  auto read_w = [&](int buf, int half, Frag<T> (&wf)[kOT][4]) {
    const uint4* sw = stage + buf * kBuf + kRowsT * 8;
#pragma unroll
    for (int n = 0; n < kOT; ++n)
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int row = (wo * kOT + n) * 64 + 16 * (l16 >> 2) + 4 * t + (l16 & 3);
        __builtin_memcpy(&wf[n][t].v, &sw[row * 8 + ((4 * half + q) ^ place_w(row))], 16);
      }
  };
  auto read_x = [&](int buf, int half, int m, Frag<T> (&xf)[kMT]) {
    const int row = (wr * kMT + m) * 16 + l16;
    __builtin_memcpy(&xf[m].v, &(stage + buf * kBuf)[row * 8 + ((4 * half + q) ^ place_x(row))], 16);
  };

  f32x4 acc[kOT][kMT][4];
#pragma unroll
  for (int n = 0; n < kOT; ++n)
#pragma unroll
    for (int m = 0; m < kMT; ++m)
#pragma unroll
      for (int t = 0; t < 4; ++t) acc[n][m][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto products = [&](int m, Frag<T> (&xf)[kMT], Frag<T> (&wf)[kOT][4]) {
#pragma unroll
    for (int n = 0; n < kOT; ++n)
#pragma unroll
      for (int t = 0; t < 4; ++t) acc[n][m][t] = mma(wf[n][t], xf[m], acc[n][m][t]);
  };

  // The up product: for each adapter among the tile's rows, steps of 32 rank columns at the end of the
  // reduction, x rows holding v (bf16: its high halves, then its low ones) or zero, W rows holding U
  // (bf16: twice). Zeros keep an adapter out of other rows unless it holds an infinity or NaN: such
  // entries are staged as zero, and the adapter's rows are noted and get those entries' products at the end.
  __shared__ uint32_t spoiled[kRowsT / 32];
  constexpr int kIds = (kRowsT + 63) / 64;
  constexpr int kSplit = sizeof(T) == 2 ? 4 : 8;  // chunks of a row before the columns repeat
  auto row_id = [&](int t, int i) {               // the adapter of tile row 64 i + t, t the lane
    const int64_t r = r0 + 64 * i + t;
    return (64 * i + t < kRowsT && r < a.n_rows) ? a.row_adapter[r] : -1;
  };
  uint64_t todo[kIds];  // tile rows whose adapter is still to come; the same in every wave
  int cur = -1, cur_rank = 0, cur_col = 0;
#pragma unroll
  for (int i = 0; i < kIds; ++i) todo[i] = 0;
  if (tid < kRowsT / 32) spoiled[tid] = 0u;
  if (a.vq) {
#pragma unroll
    for (int i = 0; i < kIds; ++i) {
      const int id = row_id(lane, i);
      todo[i] = __ballot(id >= 0 && id < a.A);
    }
  }
  auto next_up = [&]() {  // moves on by 32 columns or to the next adapter; false if none is left
    cur_col += 32;
    while (cur_col >= cur_rank) {
      int first = -1;
#pragma unroll
      for (int i = kIds - 1; i >= 0; --i)
        if (todo[i]) first = 64 * i + __builtin_ctzll(todo[i]);
      if (first < 0) return false;
      const int ft = fresh_tid() & 63;
      cur = __builtin_amdgcn_readfirstlane(a.row_adapter[r0 + first]);
#pragma unroll
      for (int i = 0; i < kIds; ++i) todo[i] &= ~__ballot(row_id(ft, i) == cur);
      cur_rank = __builtin_amdgcn_readfirstlane(rank_of(a, cur));
      cur_col = 0;
    }
    return true;
  };
  auto stage_up = [&](int buf) {
    const int ft = fresh_tid();
#pragma unroll
    for (int i = 0; i < kLoadsX; ++i) {
      const int64_t r = r0 + ((ft + i * kThreads) >> 3);
      uint4 v = make_uint4(0, 0, 0, 0);
      if (r < a.n_rows && a.row_adapter[r] == cur)
        v = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.vq) + r * a.vq_row + (chunk_x < kSplit ? 0 : a.vq_row / 2) + cur_col +
                                            (chunk_x & (kSplit - 1)) * kPer);
      stage[buf * kBuf + tid + i * kThreads] = v;
    }
    bool wild = false;
#pragma unroll
    for (int i = 0; i < kLoadsW; ++i) {
      const int col = cur_col + (chunk_w & (kSplit - 1)) * kPer;
      const Frag<T> u = load_cut<T>(static_cast<const T*>(a.up), (static_cast<int64_t>(cur) * a.O + o0 + row_w(ft, i)) * a.R + col,
                                    span_up(a), cur_rank - col);
      T e[kPer];
      __builtin_memcpy(e, &u.v, 16);
#pragma unroll
      for (int n = 0; n < kPer; ++n)
        if (!(fabsf(to_float(e[n])) <= 3.4028235e38f)) {
          wild = true;
          e[n] = T(0);
        }
      __builtin_memcpy(&stage[buf * kBuf + kRowsT * 8 + tid + i * kThreads], e, 16);
    }
    if (wild)
      for (int row = 0; row < kRowsT; ++row)
        if (r0 + row < a.n_rows && a.row_adapter[r0 + row] == cur) atomicOr(&spoiled[row >> 5], 1u << (row & 31));
  };

  Frag<T> x0[kMT], x1[kMT], w0[kOT][4], w1[kOT][4];
  fetch(k_first, 0);
  settle(0);
  __syncthreads();
  if (k_first + kStep < k_end) fetch(k_first + kStep, 1);
  read_w(0, 0, w0);
#pragma unroll
  for (int m = 0; m < kMT; ++m) read_x(0, 0, m, x0);
  // One step; kLoad: the step after next is loaded on the way, between two row tiles' products, so that a
  // full load queue does not keep the matrix cores waiting. Returns false after the last step.
  auto step = [&](auto load_too, int k, int buf) {
    constexpr bool kLoad = decltype(load_too)::value;
    read_w(buf, 1, w1);
#pragma unroll
    for (int m = 0; m < kMT; ++m) {
      read_x(buf, 1, m, x1);
      products(m, x0, w0);
      __builtin_amdgcn_sched_barrier(0);
    }
    bool more = true;
    if (kLoad || k + kStep < k_end)
      settle(buf ^ 1);
    else if ((more = next_up()))
      stage_up(buf ^ 1);
    __builtin_amdgcn_sched_barrier(0);
    __syncthreads();
    const int ft = fresh_tid();
    if (kLoad && !kDirect) fetch(k + 2 * kStep, buf);
    read_w(buf ^ 1, 0, w0);  // after the last step: what lies there, not used
#pragma unroll
    for (int m = 0; m < kMT; ++m) {
      if (kLoad && kDirect) {
#pragma unroll
        for (int n = m * kPerTile; n < (m + 1) * kPerTile; ++n) load(n, k + 2 * kStep, buf, ft);
      }
      read_x(buf ^ 1, 0, m, x0);
      products(m, x1, w1);
      __builtin_amdgcn_sched_barrier(0);
    }
    return more;
  };
  int k = k_first, buf = 0;
  for (; k + 2 * kStep < k_end; k += kStep, buf ^= 1) step(std::true_type{}, k, buf);
  for (; step(std::false_type{}, k, buf); k += kStep, buf ^= 1) {
  }

  const int64_t rw = r0 + wr * kMT * 16;
  if (a.slices > 1) {
#pragma unroll
    for (int n = 0; n < kOT; ++n) {
      const int o = o0 + (wo * kOT + n) * 64;
      if (o >= a.O) continue;
#pragma unroll
      for (int m = 0; m < kMT; ++m) {
        const int64_t r = rw + 16 * m + l16;
        if (r >= a.n_rows) continue;
        float* p = a.partial + (static_cast<int64_t>(slice) * a.n_rows + r) * a.o_pad + o + 16 * q;
#pragma unroll
        for (int t = 0; t < 4; ++t) *reinterpret_cast<f32x4*>(p + 4 * t) = acc[n][m][t];
      }
    }
    return;
  }

  uint32_t noted = 0;
#pragma unroll
  for (int i = 0; i < kRowsT / 32; ++i) noted |= spoiled[i];
#pragma unroll
  for (int n = 0; n < kOT; ++n) {
    const int o = o0 + (wo * kOT + n) * 64 + 16 * q;
    float bias[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) bias[i] = a.bias && o + i < a.O ? to_float(static_cast<const T*>(a.bias)[o + i]) : 0.f;
#pragma unroll
    for (int m = 0; m < kMT; ++m) {
      const int row = (wr * kMT + m) * 16 + l16;
      const int64_t r = r0 + row;
      if (r >= a.n_rows) continue;
      const bool out_of_range = a.row_adapter && a.row_adapter[r] >= a.A;
      T out[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) out[i] = from_float<T>(out_of_range ? __builtin_nanf("") : acc[n][m][i >> 2][i & 3] + bias[i]);
      T* y = static_cast<T*>(a.y) + r * a.y_stride + o;
      if (o + 16 <= a.O) {
        __builtin_memcpy(y, out, sizeof(out));
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (o + i < a.O) y[i] = out[i];
      }
    }
  }
  if (noted) {
    // A product with an infinity or NaN is one itself, so it may be added to what is stored already: outputs without
    // such an entry keep their value, the others become what they have to be. 8,192 x 4,096 x 4,096 with an infinity in
    // one up row 0.68 ms, in every one 1.2 (rows computed one by one: 150 and 347).
    __syncthreads();  // the rows are stored, by whichever wave
    for (int row = 0; row < kRowsT; ++row) {
      if (!(spoiled[row >> 5] >> (row & 31) & 1u)) continue;
      const int64_t r = r0 + row;
      const int ad = a.row_adapter[r], rank = rank_of(a, ad);
      const T* const v = static_cast<const T*>(a.vq) + r * a.vq_row;
      for (int o = o0 + tid; o < min(o0 + kOutsT, a.O); o += kThreads) {
        const T* const u = static_cast<const T*>(a.up) + (static_cast<int64_t>(ad) * a.O + o) * a.R;
        float s = 0.f;
        bool wild = false;
        for (int j = 0; j < rank; ++j) {
          const float e = to_float(u[j]);
          if (fabsf(e) <= 3.4028235e38f) continue;
          wild = true;
          s += (to_float(v[j]) + (sizeof(T) == 2 ? to_float(v[a.vq_row / 2 + j]) : 0.f)) * e;
        }
        T* const y = static_cast<T*>(a.y) + r * a.y_stride + o;
        if (wild) *y = from_float<T>(to_float(*y) + s);
      }
    }
  }
}

}  // namespace cdrge
