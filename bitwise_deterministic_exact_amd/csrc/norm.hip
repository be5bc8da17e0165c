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
// chunk of 16 or 32 consecutive rows in fp32 in a fixed order while it forms dx, and
// the chunks' sums are added as exact integers (the digits of the long
// accumulator) and rounded once: any split of the rows at multiples of 32,
// and any order of the chunks, gives the same bits.
#include <algorithm>

#include "rowops.h"

namespace {

using namespace rowops;

// ---------------------------------------------------------------- geometry
//
// T threads own a row, S vectors of W elements each (vector s of thread t
// starts at element (s T + t) W); G rows at a time in a workgroup.  W is 8
// when every 8 elements of the narrowest operand fill 16 bytes (all bf16), else 4.

constexpr int chunk_rows(int64_t C) { return C <= 2048 ? 16 : DET_NORM_SHARD_ROWS; }

// The sum over a row's T threads of N values at once.  One barrier: the
// buffers alternate, so a buffer is rewritten only after every thread has
// passed the barrier that follows its last reads.
template <int T, int G, int NV>
struct RowSum {
  static constexpr int WPR = T / 64;
  float buf[2][G][WPR][NV];
};
template <int T, int G, int NV>
__device__ __forceinline__ void row_sum(RowSum<T, G, NV>& m, int& turn, int group, int wave_in_row,
                                        float (&v)[NV]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = wave_sum(v[i]);
  if constexpr (T > 64) {
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) m.buf[turn][group][wave_in_row][i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < T / 64; ++w) s += m.buf[turn][group][w][i];
      v[i] = s;
    }
    turn ^= 1;
  }
}

template <int DT, int W>
__device__ __forceinline__ void load_part(const void* p, int64_t row0, int64_t at, int64_t C, float (&v)[W]) {
  if (at + W <= C) {
    load_vec<DT, W>(p, row0 + at, v);
  } else {
#pragma unroll
    for (int j = 0; j < W; ++j) v[j] = at + j < C ? load_elem<DT>(p, row0 + at + j) : 0.0f;
  }
}
template <int DT, int W>
__device__ __forceinline__ void store_part(void* p, int64_t row0, int64_t at, int64_t C, const float (&v)[W]) {
  if (at + W <= C) {
    store_vec<DT, W>(p, row0 + at, v);
  } else {
#pragma unroll
    for (int j = 0; j < W; ++j)
      if (at + j < C) store_elem<DT>(p, row0 + at + j, v[j]);
  }
}
// w and b: their type is a run-time choice (they are read once per workgroup)
template <int W>
__device__ __forceinline__ void load_weights(int dt, const void* p, int64_t at, int64_t C, float missing,
                                             float (&v)[W]) {
  if (p == nullptr) {
#pragma unroll
    for (int j = 0; j < W; ++j) v[j] = missing;
  } else if (dt == DET_F32) {
    load_part<DET_F32, W>(p, 0, at, C, v);
  } else {
    load_part<DET_BF16, W>(p, 0, at, C, v);
  }
}

// ---------------------------------------------------------------- forward
struct NormArgs {
  const void* x; int64_t s_x;
  const void* w; const void* b;
  int64_t N, C;
  float eps, inv_c;
  int w_dt;
  void* y;
  float* mean; float* rstd;
  int rows;                               // rows per workgroup, a multiple of G
};

template <int XT, int YT, int T, int S, int W, int G>
__global__ __launch_bounds__(T * G) void k_norm(NormArgs a) {
  __shared__ RowSum<T, G, 2> sm;
  int turn = 0;
  const int t = threadIdx.x % T, group = threadIdx.x / T, wr = t >> 6;
  float w[S][W], b[S][W];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int64_t at = static_cast<int64_t>(s * T + t) * W;
    load_weights<W>(a.w_dt, a.w, at, a.C, 1.0f, w[s]);
    load_weights<W>(a.w_dt, a.b, at, a.C, 0.0f, b[s]);
  }
  for (int r = group; r < a.rows; r += G) {
    const int64_t row = static_cast<int64_t>(blockIdx.x) * a.rows + r;
    const bool live = row < a.N;
    float v[S][W];
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int64_t at = static_cast<int64_t>(s * T + t) * W;
      if (live) load_part<XT, W>(a.x, row * a.s_x, at, a.C, v[s]);
      else {
#pragma unroll
        for (int j = 0; j < W; ++j) v[s][j] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < W; ++j) sum[0] += v[s][j];
    }
    row_sum<T, G, 2>(sm, turn, group, wr, sum);
    // d = x - m0 with m0 the rounded mean; the sum of d corrects m0
    const float m0 = sum[0] * a.inv_c;
    float sq[2] = {0.0f, 0.0f};
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int64_t at = static_cast<int64_t>(s * T + t) * W;
#pragma unroll
      for (int j = 0; j < W; ++j) {
        v[s][j] = at + j < a.C ? v[s][j] - m0 : 0.0f;
        sq[0] += v[s][j] * v[s][j];
        sq[1] += v[s][j];
      }
    }
    row_sum<T, G, 2>(sm, turn, group, wr, sq);
    const float off = sq[1] * a.inv_c;
    const float var = fmaxf(sq[0] * a.inv_c - off * off, 0.0f);
    const float rstd = 1.0f / sqrtf((sq[0] != sq[0] ? sq[0] : var) + a.eps);
    if (!live) continue;
    const float shift = -off * rstd;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int64_t at = static_cast<int64_t>(s * T + t) * W;
#pragma unroll
      for (int j = 0; j < W; ++j) v[s][j] = fmaf(fmaf(v[s][j], rstd, shift), w[s][j], b[s][j]);
      store_part<YT, W>(a.y, row * a.C, at, a.C, v[s]);
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
  int64_t N, C;
  float inv_c;
  void* dx;
  float* parts;                           // [chunks][2][C]: the chunks' dw and db; null: not needed
  int chunk;                              // rows per workgroup
};

template <int XT, int YT, int T, int S, int W, int G>
__global__ __launch_bounds__(T * G) void k_norm_grad(NormGradArgs a) {
  __shared__ RowSum<T, G, 2> sm;
  extern __shared__ __align__(16) float fold[];               // [T * S * W * 2] when G > 1
  int turn = 0;
  const int t = threadIdx.x % T, group = threadIdx.x / T, wr = t >> 6;
  float w[S][W], dw[S][W], db[S][W];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    load_weights<W>(a.w_dt, a.w, static_cast<int64_t>(s * T + t) * W, a.C, 1.0f, w[s]);
#pragma unroll
    for (int j = 0; j < W; ++j) dw[s][j] = db[s][j] = 0.0f;
  }
  const int64_t first = static_cast<int64_t>(blockIdx.x) * a.chunk;
  for (int r = group; r < a.chunk; r += G) {
    const int64_t row = first + r;
    if (first + (r - group) >= a.N) break;                    // no group has a row left: uniform
    const bool live = row < a.N;
    float h[S][W], g[S][W];
    float sum[2] = {0.0f, 0.0f};
    const float mean = live ? a.mean[row] : 0.0f, rstd = live ? a.rstd[row] : 0.0f;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int64_t at = static_cast<int64_t>(s * T + t) * W;
      if (live) {
        load_part<XT, W>(a.x, row * a.s_x, at, a.C, h[s]);
        load_part<YT, W>(a.dy, row * a.s_dy, at, a.C, g[s]);
      } else {
#pragma unroll
        for (int j = 0; j < W; ++j) h[s][j] = g[s][j] = 0.0f;
      }
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
#pragma unroll
      for (int j = 0; j < W; ++j) {
        h[s][j] = (h[s][j] - mean) * rstd;                    // past C: g = 0, so h counts nowhere
        dw[s][j] += g[s][j] * h[s][j];
        db[s][j] += g[s][j];
        g[s][j] *= w[s][j];
        sum[0] += g[s][j];
        sum[1] += g[s][j] * h[s][j];
      }
    }
    if (a.dx == nullptr) continue;                            // uniform
    row_sum<T, G, 2>(sm, turn, group, wr, sum);
    if (!live) continue;
    const float m1 = sum[0] * a.inv_c, m2 = sum[1] * a.inv_c;
#pragma unroll
    for (int s = 0; s < S; ++s) {
#pragma unroll
      for (int j = 0; j < W; ++j) g[s][j] = rstd * (g[s][j] - m1 - h[s][j] * m2);
      store_part<XT, W>(a.dx, row * a.C, static_cast<int64_t>(s * T + t) * W, a.C, g[s]);
    }
  }
  if (a.parts == nullptr) return;
  // the groups' sums, added in group order
  if constexpr (G > 1) {
    float* const mine = fold + t;
#pragma unroll 1
    for (int k = 1; k < G; ++k) {
      __syncthreads();
      if (group == k) {
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
          for (int j = 0; j < W; ++j) {
            mine[(2 * (s * W + j)) * T] = dw[s][j];
            mine[(2 * (s * W + j) + 1) * T] = db[s][j];
          }
      }
      __syncthreads();
      if (group == 0) {
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
          for (int j = 0; j < W; ++j) {
            dw[s][j] += mine[(2 * (s * W + j)) * T];
            db[s][j] += mine[(2 * (s * W + j) + 1) * T];
          }
      }
    }
  }
  if (group != 0) return;
  float* const pw = a.parts + static_cast<int64_t>(blockIdx.x) * 2 * a.C;
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int64_t at = static_cast<int64_t>(s * T + t) * W;
    store_part<DET_F32, W>(pw, 0, at, a.C, dw[s]);
    store_part<DET_F32, W>(pw, a.C, at, a.C, db[s]);
  }
}

// ---------------------------------------------------------------- the exact sum of the chunks
//
// An fp32 value is sig 2^(e - 150) with e = max(exponent field, 1): it starts
// at bit o = e + 148 of the accumulator (digit 0 weighs 2^-298) and its 24
// bits touch digits o/32 and o/32 + 1, 4..13 of the 18.  A column's digits
// live in LDS; the waves of a workgroup add into them with 64-bit integer
// atomics, whose order cannot matter.
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

// digits to fp32, rounded once (nearest-even): carries first, then the top
// 24 bits with the rest as a sticky bit
template <class D>
__device__ __forceinline__ float round_column(D digit) {
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
  int cut = n - 24;                                           // bits below the 24 kept ones
  cut = max(cut, -149 - q);                                   // subnormal results keep 2^-149
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
    const float v = bad ? NAN : round_column(digit);
    store_elem(a.w_dt, out, col < a.C ? col : col - a.C, v);
  }
  if (a.digits != nullptr) {
#pragma unroll
    for (int j = 0; j < DET_NUM_DIGITS; ++j)
      a.digits[col * DET_NUM_DIGITS + j] = j >= DIG0 && j < DIG0 + NDIG ? digit(j - DIG0 < 0 || j - DIG0 >= NDIG ? 0 : j - DIG0) : 0;
  }
  if (bad) a.status[0] = 1;
}

__global__ __launch_bounds__(64 * COL_WAVES) void k_norm_columns(ColArgs a) {
  __shared__ unsigned long long dg[NDIG][64];
  __shared__ int32_t bad[64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = static_cast<int64_t>(blockIdx.x / a.split) * 64 + lane;
  const int part = static_cast<int>(blockIdx.x % a.split);
  for (int i = threadIdx.x; i < NDIG * 64; i += 64 * COL_WAVES) dg[i / 64][i % 64] = 0ull;
  if (threadIdx.x < 64) bad[threadIdx.x] = 0;
  __syncthreads();
  const bool in = col < 2 * a.C;
  const int64_t end = min(a.chunks, (part + 1) * a.per);
  if (in) {
    for (int64_t k = part * a.per + wave; k < end; k += COL_WAVES) {
      const uint32_t u = __float_as_uint(a.parts[k * 2 * a.C + col]);
      const uint32_t ef = (u >> 23) & 0xFFu;
      if (ef == 0xFFu) { bad[lane] = 1; continue; }
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
  __syncthreads();
  if (threadIdx.x >= 64 || !in) return;
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
// column workgroups: at least 64 chunks (four per wave) to a run, at most SPLIT_MAX
// runs, and no more than fill the chip twice
int split_of(int64_t chunks, int64_t C) {
  const int64_t cols = ceil_div(2 * C, 64);
  return static_cast<int>(std::max<int64_t>(1, std::min({chunks / 64, static_cast<int64_t>(SPLIT_MAX),
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

// launches K<XT, YT, T, S, W, G> for the row width: T S W >= C
#define DET_NORM_WIDTHS(LAUNCH, XT, YT)                                                        \
  do {                                                                                         \
    if constexpr (XT == DET_BF16 && YT == DET_BF16) {                                          \
      if (C <= 512) LAUNCH(XT, YT, 64, 1, 8);                                                  \
      else if (C <= 1024) LAUNCH(XT, YT, 64, 2, 8);                                            \
      else if (C <= 2048) LAUNCH(XT, YT, 128, 2, 8);                                           \
      else if (C <= 4096) LAUNCH(XT, YT, 256, 2, 8);                                           \
      else if (C <= 8192) LAUNCH(XT, YT, 512, 2, 8);                                           \
      else if (C <= 16384) LAUNCH(XT, YT, 1024, 2, 8);                                         \
      else LAUNCH(XT, YT, 1024, 4, 8);                                                         \
    } else {                                                                                   \
      if (C <= 512) LAUNCH(XT, YT, 64, 2, 4);                                                  \
      else if (C <= 1024) LAUNCH(XT, YT, 64, 4, 4);                                            \
      else if (C <= 2048) LAUNCH(XT, YT, 128, 4, 4);                                           \
      else if (C <= 4096) LAUNCH(XT, YT, 256, 4, 4);                                           \
      else if (C <= 8192) LAUNCH(XT, YT, 512, 4, 4);                                           \
      else if (C <= 16384) LAUNCH(XT, YT, 1024, 4, 4);                                         \
      else LAUNCH(XT, YT, 1024, 8, 4);                                                         \
    }                                                                                          \
  } while (0)
#define DET_NORM_TYPES(LAUNCH)                                                                 \
  do {                                                                                         \
    if (x_dt == DET_F32 && y_dt == DET_F32) DET_NORM_WIDTHS(LAUNCH, DET_F32, DET_F32);         \
    else if (x_dt == DET_F32) DET_NORM_WIDTHS(LAUNCH, DET_F32, DET_BF16);                      \
    else if (y_dt == DET_F32) DET_NORM_WIDTHS(LAUNCH, DET_BF16, DET_F32);                      \
    else DET_NORM_WIDTHS(LAUNCH, DET_BF16, DET_BF16);                                          \
  } while (0)

template <int XT, int YT, int T, int S, int W>
void launch_norm(NormArgs a, hipStream_t s) {
  constexpr int G = T >= 256 ? 1 : 256 / T;
  // enough workgroups for eight to a CU before rows share one (and its weights)
  a.rows = static_cast<int>(std::min<int64_t>(16, std::max<int64_t>(1, a.N / (2048 * G)))) * G;
  hipLaunchKernelGGL((k_norm<XT, YT, T, S, W, G>), dim3(static_cast<unsigned>(ceil_div(a.N, a.rows))), dim3(T * G),
                     0, s, a);
}

template <int XT, int YT, int T, int S, int W>
void launch_norm_grad(NormGradArgs a, hipStream_t s) {
  constexpr int G = 1024 / T;
  a.chunk = chunk_rows(a.C);
  const size_t lds = G > 1 ? static_cast<size_t>(T) * S * W * 2 * sizeof(float) : 0;
  hipLaunchKernelGGL((k_norm_grad<XT, YT, T, S, W, G>), dim3(static_cast<unsigned>(chunks_of(a.N, a.C))),
                     dim3(T * G), lds, s, a);
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
  a.x = x; a.s_x = s_x; a.w = w; a.b = b; a.N = N; a.C = C;
  a.eps = static_cast<float>(eps); a.inv_c = 1.0f / static_cast<float>(C);
  a.w_dt = w_dt; a.y = y; a.mean = mean; a.rstd = rstd;
  hipStream_t s = static_cast<hipStream_t>(stream);
#define DET_LAUNCH(XT, YT, T, S, W) launch_norm<XT, YT, T, S, W>(a, s)
  DET_NORM_TYPES(DET_LAUNCH);
#undef DET_LAUNCH
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
    a.mean = mean; a.rstd = rstd; a.N = N; a.C = C; a.inv_c = 1.0f / static_cast<float>(C);
    a.dx = dx; a.parts = sums ? static_cast<float*>(workspace) : nullptr;
#define DET_LAUNCH(XT, YT, T, S, W) launch_norm_grad<XT, YT, T, S, W>(a, s)
    DET_NORM_TYPES(DET_LAUNCH);
#undef DET_LAUNCH
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
  const int64_t cols = ceil_div(2 * C, 64);
  hipLaunchKernelGGL(k_norm_columns, dim3(static_cast<unsigned>(cols * c.split)), dim3(64 * COL_WAVES), 0, s, c);
  st = hip_check(hipGetLastError(), "column sum launch");
  if (st != DET_OK || c.split == 1) return st;
  hipLaunchKernelGGL(k_norm_columns_join, dim3(static_cast<unsigned>(cols)), dim3(64), 0, s, c);
  return hip_check(hipGetLastError(), "column join launch");
}

}  // extern "C"
