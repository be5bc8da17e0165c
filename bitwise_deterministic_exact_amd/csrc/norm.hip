// Layer norm and its gradients for MI355X (gfx950).
//
//   h = (x - mean) rstd,  y = h w + b
//   g = dy w,  dx = rstd (g - mean(g) - h mean(g h))
//   dw = sum over rows of dy h,  db = sum over rows of dy
//
// A row lives in the registers of T threads, so x (and dy) are read once.
// The reductions over a row are fp32 in a fixed tree that C alone decides.
//
// The weights' gradients are sums over rows (tokens).  A workgroup adds a
// chunk of 16, 32 or 64 consecutive rows in fp32 in a fixed order while it
// forms dx, and the chunks' sums are added as exact integers (the digits of
// the long accumulator) and rounded once: any split of the rows at multiples
// of 64, and any order of the chunks, gives the same bits.
#include <algorithm>
#include <type_traits>

#include "rowops.h"

// every fused multiply-add below is written as one: the compiler forms none
#pragma clang fp contract(off)

namespace {

using namespace rowops;

// ---------------------------------------------------------------- geometry
//
// T threads own a row, S vectors of W elements each: vector s of thread t
// starts at element (s T + t) W.  T is as few waves as hold C elements; for
// short rows a power of two of a wave's lanes (500000 x 128 bf16 forward 119 ->
// 52 us, 5.0 TB/s, backward 176 -> 89; 2000000 x 17 373 -> 44 and 646 -> 112;
// rows of 256 keep half a wave each: 75 -> 61 and 123 -> 97).  G rows at a time
// in a workgroup.  W is 8 when x and y are both bf16 (16 bytes), else 4; 1 for
// rows shorter than that.  All of it follows from C and the types, so the sums'
// order does.
//
// Every access is a whole vector: one that would pass the row's end starts at
// C - W instead.  Its first `own` elements are then the previous vector's too:
// they are left out of the sums and written a second time, with the same value
// (each operation below is spelled out, so every copy of it rounds alike).
// With the tail's loads element by element under a branch the loads of a
// ragged wave waited for each other (8000 x 5000 bf16 forward 52 us, 36 this
// way; backward 97 and 58); with the tail's stores element by element the
// backward took 120 us.

// Rows whose dw and db are added in fp32: each divides DET_NORM_SHARD_ROWS.
// Few rows mean many workgroups (16 rows: two per CU at 8192 tokens) but more
// chunk sums to write and add again (8 bytes per column and chunk against 6
// per element: 8 % at 16 rows, 4 % at 32).  Wide rows of 8193 and more fill a
// CU with one workgroup each: 16 again (3868 x 12995 bf16 132 -> 90 us).
constexpr int chunk_rows(int64_t C) { return C <= 512 ? 64 : C <= 4096 || C > 8192 ? 16 : 32; }

// Rows of at most this many columns (heads' norms, and all narrower ones): a
// wave holds several, each in 1, 2, .. 32 of its lanes.
constexpr int SHORT_C = 256;

// W elements of type DT as loaded, 16 or 8 bytes
template <int DT, int W>
struct Raw {
  static constexpr int U = (W * Elem<DT>::BYTES + 3) / 4;
  uint32_t u[U];
  // from element `at` of the row at p (a scalar address, a 32-bit offset)
  template <bool NT = false>
  __device__ __forceinline__ void load(const char* p, int at) {
    const char* const q = p + static_cast<uint32_t>(at * Elem<DT>::BYTES);
    if constexpr (W == 1) {
      if constexpr (DT == DET_F32) u[0] = *reinterpret_cast<const uint32_t*>(q);
      else u[0] = *reinterpret_cast<const uint16_t*>(q);
    } else if constexpr (U == 4 && DT == DET_F32) {
      const u32x4_a4 v = load_as<NT>(reinterpret_cast<const u32x4_a4*>(q));
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = v[i];
    } else if constexpr (U == 4) {
      const u32x4_a2 v = load_as<NT>(reinterpret_cast<const u32x4_a2*>(q));
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = v[i];
    } else {
      const u32x2_a2 v = load_as<NT>(reinterpret_cast<const u32x2_a2*>(q));
      u[0] = v[0];
      u[1] = v[1];
    }
  }
  __device__ __forceinline__ void floats(float (&v)[W]) const {
#pragma unroll
    for (int j = 0; j < W; ++j) {
      if constexpr (DT == DET_F32) v[j] = __uint_as_float(u[j]);
      else v[j] = __uint_as_float((j & 1) ? u[j / 2] & 0xFFFF0000u : u[j / 2] << 16);
    }
  }
};

template <int DT, int W>
__device__ __forceinline__ void store_row(char* p, int at, const float (&v)[W]) {
  char* const q = p + static_cast<uint32_t>(at * Elem<DT>::BYTES);
  if constexpr (W == 1) store_elem<DT>(q, 0, v[0]);
  else store_vec<DT, W>(q, 0, v);
}
template <int DT>
__device__ __forceinline__ const char* row_at(const void* p, int64_t i) {
  return static_cast<const char*>(p) + i * Elem<DT>::BYTES;
}
template <int DT>
__device__ __forceinline__ char* row_at(void* p, int64_t i) {
  return static_cast<char*>(p) + i * Elem<DT>::BYTES;
}
// w and b: their type is a run-time choice (they are read once per workgroup)
template <int W>
__device__ __forceinline__ void load_weights(int dt, const void* p, int at, float missing, float (&v)[W]) {
  if (p == nullptr) {
#pragma unroll
    for (int j = 0; j < W; ++j) v[j] = missing;
  } else if constexpr (W == 1) {
    v[0] = load_elem(dt, p, at);
  } else if (dt == DET_F32) {
    load_vec<DET_F32, W>(p, at, v);
  } else {
    load_vec<DET_BF16, W>(p, at, v);
  }
}

// where vector s of thread t starts, and its first element that no other
// vector has (W: none)
struct Place {
  int at, own;
};
template <int W>
__device__ __forceinline__ Place place(int s, int T, int t, int C) {
  const int at = (s * T + t) * W, from = min(at, C - W);
  return {from, min(at - from, W)};
}

// The sum of up to three values over a row's waves (wpr of them from wave `first`).
// One barrier: the buffers alternate, so one is rewritten only after every
// thread has passed the barrier that follows its last reads.
struct RowSum {
  float buf[2][16][3];
};
template <int NV>
__device__ __forceinline__ void row_sum(RowSum& m, int& turn, int wave, int first, int wpr, float (&v)[NV]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = wave_sum(v[i]);
  if (wpr == 1) return;                                       // uniform
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) m.buf[turn][wave][i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = 0.0f;
  for (int w = 0; w < wpr; ++w) {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] += m.buf[turn][first + w][i];
  }
  turn ^= 1;
}

// The same over the P lanes (1, 2, .. 32) that hold a short row: a butterfly,
// so every one of them has the sum, and the same bits.
template <int NV>
__device__ __forceinline__ void lanes_sum(int P, float (&v)[NV]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {          // all branches uniform
    if (P > 1) v[i] += dpp<0xB1>(0.0f, v[i]);                 // lane ^ 1
    if (P > 2) v[i] += dpp<0x4E>(0.0f, v[i]);                 // lane ^ 2
    if (P > 4) v[i] += dpp<0x141>(0.0f, v[i]);                // mirrored in 8 lanes
    if (P > 8) v[i] += dpp<0x140>(0.0f, v[i]);                // mirrored in 16
    if (P > 16) v[i] += __shfl_xor(v[i], 16);
  }
}

// ---------------------------------------------------------------- forward
struct NormArgs {
  const void* x; int64_t s_x;
  const void* w; const void* b;
  int64_t N;
  int C, T, G;
  float eps, inv_c;
  int w_dt;
  void* y;
  float* mean; float* rstd;
  int rows;                               // rows per workgroup, a multiple of G
};

// d = x - m0 with m0 the rounded mean; the sum of d corrects both the mean and
// the variance, so an offset that is large beside the spread costs no
// precision.  The next row's loads are in flight while this one is summed and
// written.  (Moments per wave joined behind one barrier instead of two: the
// same time on bf16 rows of 4096, 20 % more on 5120, for its 31 registers
// more.)  15 vector instructions per element are half of the issue slots at
// 16384 x 8192 bf16; the selections of ragged waves would make it 19, so waves
// that hold whole vectors go without (8000 x 5000: 41 -> 36 us).
// ONCE: no gradient will read x again, so it is read past the caches (16384 x
// 8192 bf16 95 -> 84 us; where the gradient follows, 282 us against 289).
template <int XT, int YT, int S, int W, int MAXT, bool ONCE, bool AHEAD, bool SHORT>
__global__ __launch_bounds__(MAXT, 4) void k_norm(NormArgs a) {
  __shared__ RowSum sm;
  int turn = 0;
  // a workgroup is T x G threads; where T is whole waves a wave's row, and its address, are scalars
  const int t = threadIdx.x, wpr = a.T >> 6;
  const int group = SHORT ? threadIdx.y : __builtin_amdgcn_readfirstlane(threadIdx.y);
  const int first = group * wpr, wave = first + __builtin_amdgcn_readfirstlane(t >> 6);
  Place at[S];
  float w[S][W], b[S][W];
  bool some = false;
#pragma unroll
  for (int s = 0; s < S; ++s) {
    at[s] = place<W>(s, a.T, t, a.C);
    load_weights<W>(a.w_dt, a.w, at[s].at, 1.0f, w[s]);
    load_weights<W>(a.w_dt, a.b, at[s].at, 0.0f, b[s]);
    some |= at[s].own > 0;
  }
  const bool ragged = __ballot(some) != 0;                    // uniform: the wave holds others' elements
  Raw<XT, W> next[S];
  auto fetch = [&](int64_t row) {         // past the last row: that row again, not used
    const char* const x = row_at<XT>(a.x, min(row, a.N - 1) * a.s_x);
#pragma unroll
    for (int s = 0; s < S; ++s) next[s].template load<ONCE>(x, at[s].at);
  };
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * a.rows;
  if constexpr (AHEAD) fetch(row0 + group);
  for (int r = group; r < a.rows; r += a.G) {
    const int64_t row = row0 + r;
    if constexpr (!AHEAD) fetch(row);
    float v[S][W];
    float sum[1] = {0.0f};
#pragma unroll
    for (int s = 0; s < S; ++s) {
      next[s].floats(v[s]);
      if (!ragged) {
#pragma unroll
        for (int j = 0; j < W; ++j) sum[0] += v[s][j];
      } else {
#pragma unroll
        for (int j = 0; j < W; ++j) sum[0] += j >= at[s].own ? v[s][j] : 0.0f;
      }
    }
    if (AHEAD && r + a.G < a.rows) fetch(row + a.G);
    if constexpr (SHORT) lanes_sum(a.T, sum);
    else row_sum(sm, turn, wave, first, wpr, sum);
    const float m0 = sum[0] * a.inv_c;
    float sq[2] = {0.0f, 0.0f};
#pragma unroll
    for (int s = 0; s < S; ++s) {
#pragma unroll
      for (int j = 0; j < W; ++j) v[s][j] -= m0;
      if (!ragged) {
#pragma unroll
        for (int j = 0; j < W; ++j) {
          sq[0] = fmaf(v[s][j], v[s][j], sq[0]);
          sq[1] += v[s][j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const float d = j >= at[s].own ? v[s][j] : 0.0f;
          sq[0] = fmaf(d, d, sq[0]);
          sq[1] += d;
        }
      }
    }
    if constexpr (SHORT) lanes_sum(a.T, sq);
    else row_sum(sm, turn, wave, first, wpr, sq);
    if (row >= a.N) continue;
    const float off = sq[1] * a.inv_c;
    const float var = fmaxf(fmaf(-off, off, sq[0] * a.inv_c), 0.0f);
    const float rstd = 1.0f / sqrtf((sq[0] != sq[0] ? sq[0] : var) + a.eps);
    const float shift = -off * rstd;
    char* const y = row_at<YT>(a.y, row * a.C);
#pragma unroll
    for (int s = 0; s < S; ++s) {
#pragma unroll
      for (int j = 0; j < W; ++j) v[s][j] = fmaf(fmaf(v[s][j], rstd, shift), w[s][j], b[s][j]);
      if (at[s].own < W) store_row<YT, W>(y, at[s].at, v[s]);
    }
    if (t == 0) {
      if (a.mean != nullptr) a.mean[row] = m0 + off;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
  }
}

// ---------------------------------------------------------------- backward
struct NormGradArgs {
  const void* x; int64_t s_x;
  const void* dy; int64_t s_dy;
  const void* w; int w_dt;
  const float* mean; const float* rstd;
  int64_t N;
  int C, T, G;
  float inv_c;
  void* dx;
  float* parts;                           // [chunks][2][C]: the chunks' dw and db; null: not needed
  int chunk;                              // rows per workgroup
};

// `mean` is the row's mean rounded to fp32, so h = (x - mean) rstd carries up to
// 2^-24 |mean| rstd, the same in the whole row.  A row further from 0 than 16 of
// its spreads, where that would pass 16 roundings of 1, gives it up again: it
// is the mean of h.  Whether a row does is a matter of that row alone; the sum
// is left out where no row needs it.  With it in every row 16384 x 8192 bf16
// took 205 us instead of 191, 500000 x 128 95 instead of 88.
__device__ __forceinline__ bool far_row(float mean, float rstd) { return fabsf(mean) * rstd > 16.0f; }

template <int P>
struct alignas(4 * P) RunOf {
  float v[P];
};

// x and dy are read once and dx written once: 16384 x 8192 bf16 take 170 us,
// 4.9 TB/s with the 34 MB of chunk sums, where a large copy moves 5.1; 158 us
// without the weights' sums.
// AHEAD: the next row's loads are in flight, where the registers allow it
template <int XT, int YT, int S, int W, int MAXT, bool AHEAD, bool SHORT>
__global__ __launch_bounds__(MAXT, 4) void k_norm_grad(NormGradArgs a) {
  __shared__ RowSum sm;
  extern __shared__ __align__(16) float4 fold_lds[];          // [G][2 S W / P][T] runs of P when G > 1
  int turn = 0;
  // a workgroup is T x G threads; where T is whole waves a wave's row, and its address, are scalars
  const int t = threadIdx.x, wpr = a.T >> 6;
  const int group = SHORT ? threadIdx.y : __builtin_amdgcn_readfirstlane(threadIdx.y);
  const int first = group * wpr, wave = first + __builtin_amdgcn_readfirstlane(t >> 6);
  Place at[S];
  float w[S][W], dw[S][W], db[S][W];
  bool some = false;
#pragma unroll
  for (int s = 0; s < S; ++s) {
    at[s] = place<W>(s, a.T, t, a.C);
    load_weights<W>(a.w_dt, a.w, at[s].at, 1.0f, w[s]);
#pragma unroll
    for (int j = 0; j < W; ++j) dw[s][j] = db[s][j] = 0.0f;
    some |= at[s].own > 0;
  }
  const bool ragged = __ballot(some) != 0;                    // uniform: the wave holds others' elements
  // the last rows first: they are what the forward pass left in the memory-side
  // cache (with it 16384 x 8192 bf16 282 us, the first rows first 289; 8192 x 4096
  // fp32 140 and 145)
  const int64_t chunk = gridDim.x - 1 - blockIdx.x;
  const int64_t row0 = chunk * a.chunk;
  const int rows = static_cast<int>(min(static_cast<int64_t>(a.chunk), a.N - row0));
  Raw<XT, W> nx[S];
  Raw<YT, W> ny[S];
  float nmean = 0.0f, nrstd = 0.0f;
  // rows side by side whose sums share barriers: the workgroup takes the third
  // sum together (each wave looks at all of its rows), else row by row
  const bool together = !SHORT && wpr > 1 && a.G > 1;
  bool far = false;
  if (together) {
    const int64_t row = row0 + min(t & 63, rows - 1);
    far = __ballot(far_row(a.mean[row], a.rstd[row])) != 0;
  }
  auto fetch = [&](int r) {               // past the last row: that row again, not used
    const int64_t row = row0 + min(r, rows - 1);
    const char* const x = row_at<XT>(a.x, row * a.s_x);
    const char* const dy = row_at<YT>(a.dy, row * a.s_dy);
#pragma unroll
    for (int s = 0; s < S; ++s) {
      nx[s].load(x, at[s].at);
      ny[s].load(dy, at[s].at);
    }
    nmean = a.mean[row];
    nrstd = a.rstd[row];
  };
  if constexpr (AHEAD) fetch(group);
  for (int r0 = 0; r0 < rows; r0 += a.G) {
    const int r = r0 + group;
    if constexpr (!AHEAD) fetch(r);
    float h[S][W], g[S][W];
    float sum[2] = {0.0f, 0.0f};
    const float mean = nmean, rstd = nrstd;
    const bool live = r < rows;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      nx[s].floats(h[s]);
      ny[s].floats(g[s]);
    }
    if (AHEAD && r0 + a.G < rows) fetch(r + a.G);
#pragma unroll
    for (int s = 0; s < S; ++s) {
#pragma unroll
      for (int j = 0; j < W; ++j) h[s][j] = (h[s][j] - mean) * rstd;
    }
    if (together ? far : __ballot(far_row(mean, rstd)) != 0) {                  // uniform: of the workgroup, row or wave
      float off[1] = {0.0f};
#pragma unroll
      for (int s = 0; s < S; ++s) {
#pragma unroll
        for (int j = 0; j < W; ++j) off[0] += j >= at[s].own ? h[s][j] : 0.0f;
      }
      if constexpr (SHORT) lanes_sum(a.T, off);
      else row_sum(sm, turn, wave, first, wpr, off);
      const float shift = far_row(mean, rstd) ? off[0] * a.inv_c : 0.0f;
#pragma unroll
      for (int s = 0; s < S; ++s) {
#pragma unroll
        for (int j = 0; j < W; ++j) h[s][j] -= shift;
      }
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
#pragma unroll
      for (int j = 0; j < W; ++j) {
        if (live) {                                           // of a wave, or of the short row's lanes
          dw[s][j] = fmaf(g[s][j], h[s][j], dw[s][j]);
          db[s][j] += g[s][j];
        }
        g[s][j] *= w[s][j];
      }
      if (!ragged) {
#pragma unroll
        for (int j = 0; j < W; ++j) {
          sum[0] += g[s][j];
          sum[1] = fmaf(g[s][j], h[s][j], sum[1]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const float u = j >= at[s].own ? g[s][j] : 0.0f;
          sum[0] += u;
          sum[1] = fmaf(u, h[s][j], sum[1]);
        }
      }
    }
    if (a.dx == nullptr) continue;                            // uniform
    if constexpr (SHORT) lanes_sum(a.T, sum);
    else row_sum(sm, turn, wave, first, wpr, sum);
    if (!live) continue;
    const float m1 = sum[0] * a.inv_c, m2 = sum[1] * a.inv_c;
    char* const dx = row_at<XT>(a.dx, (row0 + r) * a.C);
#pragma unroll
    for (int s = 0; s < S; ++s) {
#pragma unroll
      for (int j = 0; j < W; ++j) g[s][j] = rstd * fmaf(-h[s][j], m2, g[s][j] - m1);
      if (at[s].own < W) store_row<XT, W>(dx, at[s].at, g[s]);
    }
  }
  if (a.parts == nullptr) return;
  char* const pw = reinterpret_cast<char*>(a.parts + chunk * 2 * a.C);
  if (a.G == 1) {
#pragma unroll
    for (int s = 0; s < S; ++s) {
      if (at[s].own == W) continue;
      store_row<DET_F32, W>(pw, at[s].at, dw[s]);
      store_row<DET_F32, W>(row_at<DET_F32>(pw, a.C), at[s].at, db[s]);
    }
    return;
  }
  // the groups' sums, added in group order, eight by eight (short rows have up to
  // 64 groups): runs of P columns, dealt to the groups
  constexpr int P = W == 1 ? 1 : 4, Q = S * W / P;            // runs of dw; as many of db
  using run = RunOf<P>;
  run* const fold = reinterpret_cast<run*>(fold_lds);
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    constexpr int PER = W / P;
    const int s = q / PER, j = q % PER * P;
    run u, v;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      u.v[i] = dw[s][j + i];
      v.v[i] = db[s][j + i];
    }
    fold[(group * 2 * Q + q) * a.T + t] = u;
    fold[(group * 2 * Q + Q + q) * a.T + t] = v;
  }
  __syncthreads();
  for (int q = group; q < 2 * Q; q += a.G) {
    run v;
    for (int k0 = 0; k0 < a.G; k0 += 8) {
      run e = fold[(k0 * 2 * Q + q) * a.T + t];
      for (int k = k0 + 1; k < min(k0 + 8, a.G); ++k) {
        const run u = fold[(k * 2 * Q + q) * a.T + t];
#pragma unroll
        for (int i = 0; i < P; ++i) e.v[i] += u.v[i];
      }
#pragma unroll
      for (int i = 0; i < P; ++i) v.v[i] = k0 == 0 ? e.v[i] : v.v[i] + e.v[i];
    }
    const int qq = q < Q ? q : q - Q;
    const Place to = place<W>(qq / (W / P), a.T, t, a.C);
    if (to.own < W) store_row<DET_F32, P>(row_at<DET_F32>(pw, q < Q ? 0 : a.C), to.at + qq % (W / P) * P, v.v);
  }
}

// Rows of more than 16384 columns: dw and db of a whole row do not fit the
// registers, so the columns are taken in parts of T S W.  The chunk's row sums
// come first (one pass over all parts, kept in LDS), then each part's dx, dw
// and db: x and dy are read twice, the second time mostly from the caches.
template <int XT, int YT, int S, int W, int T>
__global__ __launch_bounds__(T, 4) void k_norm_grad_wide(NormGradArgs a) {
  __shared__ RowSum sm;
  __shared__ float row_m[3][DET_NORM_SHARD_ROWS];
  int turn = 0;
  const int t = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int64_t chunk = gridDim.x - 1 - blockIdx.x;
  const int64_t row0 = chunk * a.chunk;
  const int rows = static_cast<int>(min(static_cast<int64_t>(a.chunk), a.N - row0));
  auto spot = [&](int part, int s) {
    const int at = ((part * S + s) * T + t) * W, from = min(at, a.C - W);
    return Place{from, min(at - from, W)};
  };
  const int nparts = (a.C + T * S * W - 1) / (T * S * W);
  for (int r = 0; r < rows; ++r) {
    const char* const x = row_at<XT>(a.x, (row0 + r) * a.s_x);
    const char* const dy = row_at<YT>(a.dy, (row0 + r) * a.s_dy);
    const float mean = a.mean[row0 + r], rstd = a.rstd[row0 + r];
    if (a.dx == nullptr && !far_row(mean, rstd)) {            // uniform
      if (t == 0) row_m[2][r] = 0.0f;
      continue;
    }
    float sum[3] = {0.0f, 0.0f, 0.0f};
    for (int part = 0; part < nparts; ++part) {
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const Place at = spot(part, s);
        Raw<XT, W> rx;
        Raw<YT, W> ry;
        float h[W], g[W], w[W];
        rx.load(x, at.at);
        ry.load(dy, at.at);
        load_weights<W>(a.w_dt, a.w, at.at, 1.0f, w);
        rx.floats(h);
        ry.floats(g);
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const float u = j >= at.own ? g[j] * w[j] : 0.0f, hj = (h[j] - mean) * rstd;
          sum[0] += u;
          sum[1] = fmaf(u, hj, sum[1]);
          sum[2] += j >= at.own ? hj : 0.0f;
        }
      }
    }
    row_sum(sm, turn, wave, 0, T / 64, sum);
    if (t == 0) {
      const float shift = far_row(mean, rstd) ? sum[2] * a.inv_c : 0.0f, m1 = sum[0] * a.inv_c;
      row_m[0][r] = m1;
      row_m[1][r] = sum[1] * a.inv_c - shift * m1;
      row_m[2][r] = shift;
    }
  }
  __syncthreads();
  char* const pw = reinterpret_cast<char*>(a.parts + chunk * 2 * a.C);
  for (int part = 0; part < nparts; ++part) {
    Place at[S];
    float w[S][W], dw[S][W], db[S][W];
#pragma unroll
    for (int s = 0; s < S; ++s) {
      at[s] = spot(part, s);
      load_weights<W>(a.w_dt, a.w, at[s].at, 1.0f, w[s]);
#pragma unroll
      for (int j = 0; j < W; ++j) dw[s][j] = db[s][j] = 0.0f;
    }
    for (int r = 0; r < rows; ++r) {
      const char* const x = row_at<XT>(a.x, (row0 + r) * a.s_x);
      const char* const dy = row_at<YT>(a.dy, (row0 + r) * a.s_dy);
      const float mean = a.mean[row0 + r], rstd = a.rstd[row0 + r];
      const float m1 = row_m[0][r], m2 = row_m[1][r], shift = row_m[2][r];
      Raw<XT, W> rx[S];
      Raw<YT, W> ry[S];
#pragma unroll
      for (int s = 0; s < S; ++s) {
        rx[s].load(x, at[s].at);
        ry[s].load(dy, at[s].at);
      }
#pragma unroll
      for (int s = 0; s < S; ++s) {
        float h[W], g[W];
        rx[s].floats(h);
        ry[s].floats(g);
#pragma unroll
        for (int j = 0; j < W; ++j) {
          h[j] = (h[j] - mean) * rstd - shift;
          dw[s][j] = fmaf(g[j], h[j], dw[s][j]);
          db[s][j] += g[j];
          g[j] = rstd * fmaf(-h[j], m2, g[j] * w[s][j] - m1);
        }
        if (a.dx != nullptr && at[s].own < W)
          store_row<XT, W>(row_at<XT>(a.dx, (row0 + r) * a.C), at[s].at, g);
      }
    }
    if (a.parts == nullptr) continue;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      if (at[s].own == W) continue;
      store_row<DET_F32, W>(pw, at[s].at, dw[s]);
      store_row<DET_F32, W>(row_at<DET_F32>(pw, a.C), at[s].at, db[s]);
    }
  }
}

// ---------------------------------------------------------------- the exact sum of the chunks
//
// An fp32 value is sig 2^(e - 150) with e = max(exponent field, 1): it starts
// at bit o = e + 148 of the accumulator (digit 0 weighs 2^-298) and its 24
// bits touch digits o/32 and o/32 + 1, 4..13 of the 18.  A column's digits
// live in LDS; the waves of a workgroup add into them with 64-bit integer
// atomics, whose order cannot matter.  512 chunks of 8192 columns take 16 us
// (2.1 TB/s); sums kept in registers first took 3 us longer.
constexpr int DIG0 = 4, NDIG = 10, COL_WAVES = 16, SPLIT_MAX = 64;

struct ColArgs {
  const float* parts;                     // [chunks][2][C]
  int64_t chunks, C;
  int split;                              // workgroups per 64 columns, each a run of chunks
  int64_t per;                            // chunks per run
  int64_t* sums;                          // split > 1: [split][2 C][NDIG] in the workspace
  int32_t* bad;                           // split > 1: [split][2 C]
  void* dw; void* db; int w_dt;
  int64_t* digits;                        // [2][C][18] or null
  int32_t* status;
};

// digits to a value of the gradient's type, rounded once (nearest-even):
// carries first, then the top 24 bits (bf16: 8) with the rest as a sticky bit.
// By way of fp32 a bf16 gradient would be rounded twice: 1 + 2^-8 + 2^-30 to 1.
template <class D>
__device__ __forceinline__ float round_column(D digit, bool bf16) {
  uint32_t w[NDIG + 1];
  int64_t carry = 0;
#pragma unroll
  for (int j = 0; j < NDIG; ++j) {
    const int64_t v = digit(j) + carry;
    w[j] = static_cast<uint32_t>(v);
    carry = v >> 32;
  }
  const bool neg = carry < 0;
  w[NDIG] = static_cast<uint32_t>(carry);                     // |carry| < 2^31: the sums stay far below 2^62
  if (neg) {
    uint32_t c = 1u;
#pragma unroll
    for (int j = 0; j <= NDIG; ++j) {
      const uint32_t v = ~w[j] + c;
      c = (c != 0u && v == 0u) ? 1u : 0u;
      w[j] = v;
    }
  }
  int top = -1;
  uint32_t hi = 0u, lo = 0u;                                  // the highest nonzero word and the one below it
#pragma unroll
  for (int j = 0; j <= NDIG; ++j)
    if (w[j] != 0u) {
      top = j;
      hi = w[j];
      lo = j > 0 ? w[j > 0 ? j - 1 : 0] : 0u;
    }
  bool sticky = false;                                        // any bit below those two
#pragma unroll
  for (int j = 0; j <= NDIG; ++j)
    if (j < top - 1 && w[j] != 0u) sticky = true;
  if (top < 0) return 0.0f;
  uint64_t win = (static_cast<uint64_t>(hi) << 32) | lo;      // its bit 0 weighs 2^(32 (DIG0 + top - 1) - 298)
  int q = 32 * (DIG0 + top - 1) - 298;
  const int n = 64 - __builtin_clzll(win);                    // n >= 33
  // the bits below the kept ones; subnormal results keep 2^-149 (bf16: 2^-133)
  const int cut = bf16 ? max(n - 8, -133 - q) : max(n - 24, -149 - q);
  if (cut > 64) return neg ? -0.0f : 0.0f;                    // bf16, top = 0: 69, and less than 2^-138
  if (cut > 0) {
    const uint64_t rest = win & ((1ull << cut) - 1ull), half = 1ull << (cut - 1);
    win >>= cut;
    q += cut;
    if (rest > half || (rest == half && (sticky || (win & 1ull)))) win += 1ull;
  }
  const float mag = ldexpf(static_cast<float>(static_cast<uint32_t>(win)), q);
  return neg ? -mag : mag;
}

template <class D>
__device__ __forceinline__ void write_column(const ColArgs& a, int64_t col, D digit, bool bad) {
  void* const out = col < a.C ? a.dw : a.db;
  if (out != nullptr) {
    const float v = bad ? NAN : round_column(digit, a.w_dt == DET_BF16);
    store_elem(a.w_dt, out, col < a.C ? col : col - a.C, v);
  }
  if (a.digits != nullptr) {
#pragma unroll
    for (int j = 0; j < DET_NUM_DIGITS; ++j)
      a.digits[col * DET_NUM_DIGITS + j] = j >= DIG0 && j < DIG0 + NDIG ? digit(j - DIG0 < 0 || j - DIG0 >= NDIG ? 0 : j - DIG0) : 0;
  }
  if (bad) a.status[0] = 1;
}

// CB columns per workgroup: 64, or 32 or 16 (two or four chunks to a wave's
// load) where 64 would leave CUs without one.
template <int CB>
__global__ __launch_bounds__(64 * COL_WAVES) void k_norm_columns(ColArgs a) {
  constexpr int PER = 64 / CB, STEP = COL_WAVES * PER, AHEAD = 8;
  __shared__ unsigned long long dg[NDIG][CB];
  __shared__ int32_t bad[CB];
  const int lane = threadIdx.x & (CB - 1), lead = threadIdx.x / CB;
  const int64_t col = static_cast<int64_t>(blockIdx.x / a.split) * CB + lane;
  const int part = static_cast<int>(blockIdx.x % a.split);
  for (int i = threadIdx.x; i < NDIG * CB; i += 64 * COL_WAVES) dg[i / CB][i % CB] = 0ull;
  if (threadIdx.x < CB) bad[threadIdx.x] = 0;
  __syncthreads();
  const bool in = col < 2 * a.C;
  const int64_t end = min(a.chunks, (part + 1) * a.per);
  if (in) {
    const float* const src = a.parts + col;
    for (int64_t k0 = part * a.per + lead; k0 < end; k0 += AHEAD * STEP) {
      float v[AHEAD];                     // past the end: the last chunk again, not added
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) v[i] = src[min(k0 + i * STEP, end - 1) * 2 * a.C];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const uint32_t u = k0 + i * STEP < end ? __float_as_uint(v[i]) : 0u;
        const uint32_t ef = (u >> 23) & 0xFFu;
        if (ef == 0xFFu) {
          bad[lane] = 1;
        } else if (u << 1) {
          uint32_t sig = u & 0x7FFFFFu;
          if (ef != 0u) sig |= 0x800000u;
          const uint32_t o = max(ef, 1u) + 148u;
          const uint64_t wide = static_cast<uint64_t>(sig) << (o & 31u);
          int64_t lo = static_cast<int64_t>(wide & 0xFFFFFFFFull), hi = static_cast<int64_t>(wide >> 32);
          if (u >> 31) { lo = -lo; hi = -hi; }
          const int j = static_cast<int>(o >> 5) - DIG0;
          atomicAdd(&dg[j][lane], static_cast<unsigned long long>(lo));
          if (hi != 0) atomicAdd(&dg[j + 1][lane], static_cast<unsigned long long>(hi));
        }
      }
    }
  }
  __syncthreads();
  if (threadIdx.x >= CB || !in) return;
  auto digit = [&](int j) { return static_cast<int64_t>(dg[j][lane]); };
  if (a.split == 1) {
    write_column(a, col, digit, bad[lane] != 0);
    return;
  }
  int64_t* const out = a.sums + (part * 2 * a.C + col) * NDIG;
#pragma unroll
  for (int j = 0; j < NDIG; ++j) out[j] = digit(j);
  a.bad[part * 2 * a.C + col] = bad[lane];
}

__global__ __launch_bounds__(64) void k_norm_columns_join(ColArgs a) {
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x;
  if (col >= 2 * a.C) return;
  int64_t d[NDIG] = {};
  bool bad = false;
  for (int p = 0; p < a.split; ++p) {
    const int64_t* const in = a.sums + (p * 2 * a.C + col) * NDIG;
#pragma unroll
    for (int j = 0; j < NDIG; ++j) d[j] += in[j];
    bad |= a.bad[p * 2 * a.C + col] != 0;
  }
  write_column(a, col, [&](int j) { return d[j]; }, bad);
}

// ---------------------------------------------------------------- host side

int64_t chunks_of(int64_t N, int64_t C) { return ceil_div(N, chunk_rows(C)); }
// columns per workgroup of the exact sum
int columns_of(int64_t C) { return 2 * C >= 64 * 256 ? 64 : 2 * C >= 32 * 256 ? 32 : 16; }
// Runs of chunks per column: more than one only where a workgroup would have
// over 2048 chunks to add (a wave then waits for 128 / PER times 8 loads,
// longer than the join's launch), at most SPLIT_MAX, and no more than fill
// the chip twice.
int split_of(int64_t chunks, int64_t C) {
  const int64_t cols = ceil_div(2 * C, columns_of(C));
  return static_cast<int>(std::max<int64_t>(1, std::min({chunks / 1024, static_cast<int64_t>(SPLIT_MAX),
                                                         ceil_div(512, cols)})));
}
int64_t parts_bytes(int64_t N, int64_t C) { return (chunks_of(N, C) * 2 * C * 4 + 15) / 16 * 16; }
int64_t grad_ws_bytes(int64_t N, int64_t C) {
  const int split = split_of(chunks_of(N, C), C);
  return parts_bytes(N, C) + (split > 1 ? split * 2 * C * (NDIG * 8 + 4) : 0);
}

det_status check_rows(int x_dt, int w_dt, int y_dt, const void* x, int64_t s_x, int64_t N, int64_t C) {
  if (!known_dtype(x_dt) || !known_dtype(w_dt) || !known_dtype(y_dt))
    return fail(DET_EDTYPE, "unknown dtype (%d, %d, %d)", x_dt, w_dt, y_dt);
  if (N < 0 || C < 1 || s_x < 0) return fail(DET_EINVAL, "bad size or stride: N=%lld C=%lld stride=%lld", (long long)N,
                                             (long long)C, (long long)s_x);
  if (C > DET_NORM_C_MAX) return fail(DET_EINVAL, "C = %lld exceeds the limit 32768", (long long)C);
  if (N > DET_ROWS_MAX) return fail(DET_EINVAL, "N = %lld exceeds the limit 2^22 rows per call", (long long)N);
  if (N > 0 && x == nullptr) return fail(DET_EINVAL, "null x");
  if (!aligned_for(x, x_dt)) return fail(DET_EINVAL, "x must be aligned to its element size");
  return DET_OK;
}

// threads that hold a row of C elements, S W each
int threads_of(int64_t C, int S, int W) { return static_cast<int>(ceil_div(C, 64 * S * W)) * 64; }

// lanes that hold a short row: a power of two
int lanes_of(int64_t C, int S, int W) {
  int P = 1;
  while (P * S * W < C) P *= 2;
  return P;
}

template <int XT, int YT, int S, int W, int MAXT, bool SHORT = false>
void launch_norm(NormArgs a, hipStream_t s) {
  a.T = SHORT ? lanes_of(a.C, S, W) : threads_of(a.C, S, W);
  a.G = std::max(1, 256 / a.T);
  // enough workgroups for eight to a CU before rows share one (and its weights)
  a.rows = static_cast<int>(std::min<int64_t>(16, std::max<int64_t>(1, a.N / (2048 * a.G)))) * a.G;
  const dim3 grid(static_cast<unsigned>(ceil_div(a.N, a.rows))), block(a.T, a.G);
  if (a.rstd == nullptr) hipLaunchKernelGGL((k_norm<XT, YT, S, W, MAXT, true, (MAXT <= 512), SHORT>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_norm<XT, YT, S, W, MAXT, false, (MAXT <= 512), SHORT>), grid, block, 0, s, a);
}

template <int XT, int YT, int S, int W, int MAXT, bool SHORT = false>
void launch_norm_grad(NormGradArgs a, hipStream_t s) {
  a.T = SHORT ? lanes_of(a.C, S, W) : threads_of(a.C, S, W);
  // Rows at a time: 1024 threads' from 1025 columns on, 512 up to there; short
  // rows at most one chunk's.  The number of rows may not decide, for the order
  // of dw's sums follows.  With half of that from 1025 columns on, few rows
  // wait longer and many wait less: 1021 x 1537 fp32 15.6 -> 17.2 us, 100 x 3000
  // bf16 16.6 -> 23.1, 1021 x 4096 28.4 both ways, but 32768 x 1025 bf16 90.8 ->
  // 79.1, 8192 x 2048 30.6 -> 29.1, 32768 x 3000 146.7 -> 154.5.  With twice up to 1024
  // columns the same: 1021 x 768 fp32 11.8 -> 11.0, 32768 x 1024 bf16 53.3 -> 62.0.
  a.G = std::max(1, std::min(SHORT ? chunk_rows(SHORT_C) : 8, (a.C > 1024 ? 1024 : 512) / a.T));
  a.chunk = chunk_rows(a.C);
  const size_t lds = a.G > 1 && a.parts != nullptr ? static_cast<size_t>(a.G) * a.T * S * W * 2 * sizeof(float) : 0;
  hipLaunchKernelGGL((k_norm_grad<XT, YT, S, W, MAXT, (S * W <= 8), SHORT>), dim3(static_cast<unsigned>(ceil_div(a.N, a.chunk))),
                     dim3(a.T, a.G), lds, s, a);
}

template <int XT, int YT, int S, int W, int T>
void launch_norm_grad_wide(NormGradArgs a, hipStream_t s) {
  a.T = T;
  a.G = 1;
  a.chunk = chunk_rows(a.C);
  hipLaunchKernelGGL((k_norm_grad_wide<XT, YT, S, W, T>), dim3(static_cast<unsigned>(ceil_div(a.N, a.chunk))), dim3(T),
                     0, s, a);
}

// Elements a thread holds.  Forward: 8 up to 512 columns, 16 up to 16384 (more
// waves to a row wait longer at its barriers: 8 elements took 166 us on 16384 x
// 8192 bf16, 16 take 106; 32 cost 12 % more on 4096 columns for their
// registers).  Backward: 8 up to 8192 columns (dw, db and w take as much again
// three times: 16 spill).
template <int XT, int YT>
void forward(const NormArgs& a, hipStream_t s) {
  constexpr int W = XT == DET_BF16 && YT == DET_BF16 ? 8 : 4;
  if (a.C < W) launch_norm<XT, YT, 1, 1, 512, true>(a, s);
  else if (a.C <= SHORT_C) launch_norm<XT, YT, 8 / W, W, 512, true>(a, s);
  else if (a.C <= 512) launch_norm<XT, YT, 8 / W, W, 512>(a, s);
  else if (a.C <= 8192) launch_norm<XT, YT, 16 / W, W, 512>(a, s);
  else if (a.C <= 16384) launch_norm<XT, YT, 16 / W, W, 1024>(a, s);
  else launch_norm<XT, YT, 32 / W, W, 1024>(a, s);
}
template <int XT, int YT>
void backward(const NormGradArgs& a, hipStream_t s) {
  constexpr int W = XT == DET_BF16 && YT == DET_BF16 ? 8 : 4;
  if (a.C < W) launch_norm_grad<XT, YT, 1, 1, 512, true>(a, s);
  else if (a.C <= SHORT_C) launch_norm_grad<XT, YT, 8 / W, W, 512, true>(a, s);
  else if (a.C <= 512) launch_norm_grad<XT, YT, 8 / W, W, 512>(a, s);
  else if (a.C <= 8192) launch_norm_grad<XT, YT, 8 / W, W, 1024>(a, s);
  else if (a.C <= 16384) launch_norm_grad<XT, YT, 16 / W, W, 1024>(a, s);
  else launch_norm_grad_wide<XT, YT, 8 / W, W, 1024>(a, s);
}
template <class F>
void by_types(int x_dt, int y_dt, F f) {
  using std::integral_constant;
  const auto f32 = integral_constant<int, DET_F32>{};
  const auto bf16 = integral_constant<int, DET_BF16>{};
  if (x_dt == DET_F32 && y_dt == DET_F32) f(f32, f32);
  else if (x_dt == DET_F32) f(f32, bf16);
  else if (y_dt == DET_F32) f(bf16, f32);
  else f(bf16, bf16);
}

}  // namespace

extern "C" {

det_status det_layer_norm(det_dtype x_dt, const void* x, int64_t s_x, det_dtype w_dt, const void* w, const void* b,
                          int64_t N, int64_t C, double eps, det_dtype y_dt, void* y, float* mean, float* rstd,
                          void* stream) {
  det_status st = check_rows(x_dt, w_dt, y_dt, x, s_x, N, C);
  if (st != DET_OK) return st;
  if (!(eps >= 0.0) || !(eps < 1e30)) return fail(DET_EINVAL, "eps must be >= 0 and finite");
  if (N == 0) return DET_OK;
  if (y == nullptr) return fail(DET_EINVAL, "null output");
  if (!aligned_for(w, w_dt) || !aligned_for(b, w_dt) || !aligned_for(y, y_dt) || !aligned_for(mean, DET_F32) ||
      !aligned_for(rstd, DET_F32))
    return fail(DET_EINVAL, "operands must be aligned to their element size");
  NormArgs a{};
  a.x = x; a.s_x = s_x; a.w = w; a.b = b; a.N = N; a.C = static_cast<int>(C);
  a.eps = static_cast<float>(eps); a.inv_c = 1.0f / static_cast<float>(C);
  a.w_dt = w_dt; a.y = y; a.mean = mean; a.rstd = rstd;
  hipStream_t s = static_cast<hipStream_t>(stream);
  by_types(x_dt, y_dt, [&](auto xt, auto yt) { forward<decltype(xt)::value, decltype(yt)::value>(a, s); });
  return hip_check(hipGetLastError(), "layer norm launch");
}

int64_t det_layer_norm_grad_workspace_bytes(int64_t N, int64_t C) {
  if (N <= 0 || C <= 0 || N > DET_ROWS_MAX || C > DET_NORM_C_MAX) return 0;
  return grad_ws_bytes(N, C);
}

det_status det_layer_norm_grad(det_dtype x_dt, const void* x, int64_t s_x, det_dtype y_dt, const void* dy,
                               int64_t s_dy, det_dtype w_dt, const void* w, const float* mean, const float* rstd,
                               int64_t N, int64_t C, void* dx, void* dw, void* db, int64_t* digits,
                               void* workspace, size_t workspace_bytes, void* stream) {
  det_status st = check_rows(x_dt, w_dt, y_dt, x, s_x, N, C);
  if (st != DET_OK) return st;
  if (s_dy < 0) return fail(DET_EINVAL, "negative stride");
  const bool sums = dw != nullptr || db != nullptr || digits != nullptr;
  if (!aligned_for(dy, y_dt) || !aligned_for(w, w_dt) || !aligned_for(dx, x_dt) || !aligned_for(dw, w_dt) ||
      !aligned_for(db, w_dt) || !aligned_for(mean, DET_F32) || !aligned_for(rstd, DET_F32) || !aligned8(digits))
    return fail(DET_EINVAL, "operands must be aligned to their element size");
  if (N > 0 && (dy == nullptr || mean == nullptr || rstd == nullptr)) return fail(DET_EINVAL, "null pointer");
  if (!sums && (N == 0 || dx == nullptr)) return DET_OK;
  const int64_t need = N > 0 && sums ? grad_ws_bytes(N, C) : 0;
  if (need > 0 && (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 15u) ||
                   workspace_bytes < static_cast<size_t>(need)))
    return fail(DET_EINVAL, "workspace: %lld bytes, 16-byte aligned, are needed", (long long)need);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (N > 0) {
    NormGradArgs a{};
    a.x = x; a.s_x = s_x; a.dy = dy; a.s_dy = s_dy; a.w = w; a.w_dt = w_dt;
    a.mean = mean; a.rstd = rstd; a.N = N; a.C = static_cast<int>(C); a.inv_c = 1.0f / static_cast<float>(C);
    a.dx = dx; a.parts = sums ? static_cast<float*>(workspace) : nullptr;
    by_types(x_dt, y_dt, [&](auto xt, auto yt) { backward<decltype(xt)::value, decltype(yt)::value>(a, s); });
    st = hip_check(hipGetLastError(), "layer norm gradient launch");
    if (st != DET_OK) return st;
  }
  if (!sums) return DET_OK;
  ColArgs c{};
  c.chunks = N > 0 ? chunks_of(N, C) : 0;
  c.C = C;
  c.parts = static_cast<const float*>(workspace);
  c.split = split_of(c.chunks, C);
  c.per = ceil_div(c.chunks, c.split);
  c.dw = dw; c.db = db; c.w_dt = w_dt; c.digits = digits;
  c.status = det_device_status_word();
  if (c.status == nullptr) return DET_EHIP;
  if (c.split > 1) {
    c.sums = reinterpret_cast<int64_t*>(static_cast<char*>(workspace) + parts_bytes(N, C));
    c.bad = reinterpret_cast<int32_t*>(c.sums + c.split * 2 * C * NDIG);
  }
  const int cb = columns_of(C);
  const dim3 grid(static_cast<unsigned>(ceil_div(2 * C, cb) * c.split)), block(64 * COL_WAVES);
  if (cb == 64) hipLaunchKernelGGL(k_norm_columns<64>, grid, block, 0, s, c);
  else if (cb == 32) hipLaunchKernelGGL(k_norm_columns<32>, grid, block, 0, s, c);
  else hipLaunchKernelGGL(k_norm_columns<16>, grid, block, 0, s, c);
  st = hip_check(hipGetLastError(), "column sum launch");
  if (st != DET_OK || c.split == 1) return st;
  hipLaunchKernelGGL(k_norm_columns_join, dim3(static_cast<unsigned>(ceil_div(2 * C, 64))), dim3(64), 0, s, c);
  return hip_check(hipGetLastError(), "column join launch");
}

}  // extern "C"
