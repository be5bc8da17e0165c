// Post-training losses on token log probabilities for MI355X (gfx950): the
// clipped policy loss with a KL term and the preference loss over pairs, each
// with its gradient.
//
// One pass over [rows][T] arrays each, bound by HBM on large batches and by the
// latency of a launch on small ones: 1024 x 8192 tokens with a reference 27 us and
// 8 to join the rows (143 MB, 5.2 TB/s; the exponentials, series and differences in
// 64 bits take 79 instructions a token), 29 for the gradient (176 MB, 6.1 TB/s);
// 2 x 2048 x 4096 preference 29 and 14 (5.2 and 6.0 TB/s).  A row's sums are formed
// in 64 bits, in an order that T alone decides; sums over rows are exact
// (exact_sum.h): any order of the rows gives the same bits.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "elementary.h"
#include "exact_sum.h"

// every fused multiply-add below is written as one: the compiler forms none
#pragma clang fp contract(off)

namespace {

using namespace rowops;

// A wave takes 512 tokens of a row at a time: two vectors of 4 per lane.  In the
// policy loss a workgroup of four takes a piece of 2048 tokens, or four rows of
// up to 512.
constexpr int PART = 512, VECS = 2, PIECE = 4 * PART;

struct __attribute__((packed, aligned(1))) MaskWord {
  uint32_t w;
};

// four tokens from element i on, n of them inside the row; those outside are 0
__device__ __forceinline__ void tokens(const float* p, int64_t i, int n, float (&v)[4]) {
  if (n >= 4) {
    load_vec<DET_F32, 4>(p, i, v);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = k < n ? p[i + k] : 0.0f;
  }
}
// which of them count, as four bytes of 0 or 1 (no mask: all that are inside)
__device__ __forceinline__ void counted(const uint8_t* p, int64_t i, int n, bool (&m)[4]) {
  uint32_t w = 0x01010101u;
  if (p != nullptr) {
    if (n >= 4) {
      w = reinterpret_cast<const MaskWord*>(p + i)->w;
    } else {
      w = 0u;
#pragma unroll
      for (int k = 0; k < 3; ++k)
        if (k < n) w |= static_cast<uint32_t>(p[i + k]) << (8 * k);
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) m[k] = k < n && ((w >> (8 * k)) & 0xFFu) != 0u;
}
__device__ __forceinline__ void store_tokens(float* p, int64_t i, int n, const float (&v)[4]) {
  if (n >= 4) {
    store_vec<DET_F32, 4>(p, i, v);
  } else {
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (k < n) p[i + k] = v[k];
  }
}

__device__ __forceinline__ int wave_count(int v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// ---------------------------------------------------------------- the policy loss
//
//   d = lp - old,  r = e^d,  l = -min(r A, clip(r) A) + kl_weight (e^q - 1 - q),  q = ref - lp
//
// d and q are differences in 64 bits: a token is clipped when d lies beyond the
// logarithms of the bounds, which no rounding moves.

struct PolicyArgs {
  const float* lp; int64_t s_lp;
  const float* old; int64_t s_old;
  const float* adv; int64_t s_adv; int adv_t;                 // adv_t: 1 per token, 0 one to a row
  const uint8_t* mask; int64_t s_mask;
  const float* ref; int64_t s_ref;        // null: no KL term
  int64_t B, T, pieces;
  double low, high;                       // ln(1 - clip_low), ln(1 + clip_high)
  float bound_low, bound_high, kl_weight;
  int reduction;
  // reduction none: per token; else one value each
  float* loss; float* kl; float* clipped;
  // what the pieces of rows leave, [pieces][B]: sums of loss and KL, tokens clipped and that count
  double2* piece_sums; int2* piece_counts;
  int64_t* count;                         // [B] tokens of a row that count, [B + 0] their divisor
  int64_t* joined; int groups;            // groups > 1: [groups][JOINED] of the workgroups that join rows
  int32_t* status;
  // the gradient
  const float* g; int64_t s_g, s_g_t;     // the incoming gradient: one value, or per token
  float* dlp;
};

struct Token {
  float loss, kl, slope;
  bool clipped;
};
// r A where r alone may leave fp32 and r A need not (no advantage: 0, however far
// the ratio is): in four factors.  Beyond e^+-350 every A that is not 0 is past
// fp32, or nothing.
__device__ __forceinline__ float far_ratio(double d, float adv) {
  if (!(fabs(d) < INFINITY)) return (d != d ? static_cast<float>(d) : exp_of(static_cast<float>(d))) * adv;
  const double quarter = 0.25 * fmin(fmax(d, -350.0), 350.0);
  const float near = static_cast<float>(quarter), rest = static_cast<float>(quarter - static_cast<double>(near));
  float part = exp_of(near);
  part = fmaf(part, rest, part);
  return adv * part * part * part * part;
}
// FAR: no bound is known for d; else |d| < 69, so that r lies within [2^-100, 2^100]
template <bool FAR>
__device__ __forceinline__ Token token_of(const PolicyArgs& a, float lp, float old, float adv, float ref) {
  const double d = static_cast<double>(lp) - static_cast<double>(old);
  const float hi = static_cast<float>(d), lo = static_cast<float>(d - static_cast<double>(hi));
  Token t;
  t.clipped = (adv > 0.0f && d > a.high) || (adv < 0.0f && d < a.low);
  const float e = exp_of(hi);
  const float whole = FAR && !(hi > -69.0f && hi < 88.5f) ? far_ratio(d, adv) : fmaf(e, lo, e) * adv;     // r A
  t.loss = t.clipped ? -(adv > 0.0f ? a.bound_high : a.bound_low) * adv : -whole;
  t.slope = t.clipped ? 0.0f : -whole;
  t.kl = 0.0f;
  if (a.ref != nullptr) {
    const double dq = static_cast<double>(ref) - static_cast<double>(lp);
    const float q = static_cast<float>(dq), rest = static_cast<float>(dq - static_cast<double>(q));
    float rise;                           // e^q - 1
    if (fabsf(q) <= 1.0f) {
      // e^q - 1 - q = q^2 (1/2 + q/6 + ...), to q^12: no difference of near values
      float s = 1.0f / 479001600.0f;
      const float f[10] = {1.0f / 39916800.0f, 1.0f / 3628800.0f, 1.0f / 362880.0f, 1.0f / 40320.0f, 1.0f / 5040.0f,
                           1.0f / 720.0f,      1.0f / 120.0f,     1.0f / 24.0f,     1.0f / 6.0f,     0.5f};
#pragma unroll
      for (int k = 0; k < 10; ++k) s = fmaf(s, q, f[k]);
      t.kl = q * q * s;
      rise = q + t.kl;
    } else {
      // the low part where it is one: without it e^q would be off by |q| half units
      const float e = exp_of(q);
      rise = (e < INFINITY && q > -INFINITY ? fmaf(e, rest, e) : e) - 1.0f;
      t.kl = q < INFINITY ? rise - q : q;
      if (q != q) t.kl = rise = q;
    }
    if (a.kl_weight != 0.0f) {            // without a weight it is reported only: 0 inf would be NaN
      t.loss = fmaf(a.kl_weight, t.kl, t.loss);
      t.slope = fmaf(-a.kl_weight, rise, t.slope);
    }
  }
  return t;
}

// whether a token that counts is FAR
__device__ __forceinline__ bool any_far(const float (&lp)[4], const float (&old)[4], const bool (&m)[4]) {
  bool far = false;
#pragma unroll
  for (int j = 0; j < 4; ++j) far |= m[j] && !(fabsf(lp[j] - old[j]) < 68.9f);
  return far;
}

// the row of a wave, its piece and the wave's first token
struct Place {
  int64_t b, piece, t;
};
__device__ __forceinline__ Place place_of(const PolicyArgs& a, int wave) {
  if (a.T <= PART) return {static_cast<int64_t>(blockIdx.x) * 4 + wave, 0, 0};
  const int64_t b = static_cast<int64_t>(blockIdx.x) / a.pieces, piece = static_cast<int64_t>(blockIdx.x) - b * a.pieces;
  return {b, piece, piece * PIECE + wave * PART};
}

// what a wave's tokens, or a row's, leave
struct Part {
  double loss, kl;
  int clipped, count;
};
// a wave's tokens from at.t on
__device__ __forceinline__ Part part_of(const PolicyArgs& a, const Place& at, int lane) {
  const int64_t b = at.b;
  const float adv_b = a.adv_t == 0 ? a.adv[b * a.s_adv] : 0.0f;
  double loss = 0.0, kl = 0.0;
  int clipped = 0, count = 0;
  bool bad = false;
#pragma unroll
  for (int v = 0; v < VECS; ++v) {
    const int64_t t = at.t + v * 256 + lane * 4;
    const int n = static_cast<int>(max<int64_t>(0, min<int64_t>(4, a.T - t)));
    float lp[4], old[4], adv[4], ref[4], l[4], k[4], c[4];
    bool m[4];
    tokens(a.lp, b * a.s_lp + t, n, lp);
    tokens(a.old, b * a.s_old + t, n, old);
    if (a.adv_t != 0) tokens(a.adv, b * a.s_adv + t, n, adv);
    if (a.ref != nullptr) tokens(a.ref, b * a.s_ref + t, n, ref);
    counted(a.mask, b * a.s_mask + t, n, m);
    // one branch for four tokens: 1024 x 8192 27.1 us, with one to each 31.9
    auto take = [&](auto far) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const Token x = token_of<decltype(far)::value>(a, lp[j], old[j], a.adv_t != 0 ? adv[j] : adv_b,
                                                       a.ref != nullptr ? ref[j] : 0.0f);
        // what a token that does not count holds is not looked at
        l[j] = m[j] ? x.loss : 0.0f;
        k[j] = m[j] ? x.kl : 0.0f;
        c[j] = m[j] && x.clipped ? 1.0f : 0.0f;
        bad |= !(fabsf(l[j]) < INFINITY);
        loss += static_cast<double>(l[j]);
        kl += static_cast<double>(k[j]);
        clipped += c[j] != 0.0f;
        count += m[j];
      }
    };
    if (any_far(lp, old, m)) take(std::true_type{});
    else take(std::false_type{});
    if (a.reduction == DET_REDUCE_NONE) {
      store_tokens(a.loss, b * a.T + t, n, l);
      store_tokens(a.kl, b * a.T + t, n, k);
      store_tokens(a.clipped, b * a.T + t, n, c);
    }
  }
  if (bad) a.status[0] = 1;
  if (a.reduction == DET_REDUCE_NONE) return {0.0, 0.0, 0, 0};
  return {wave_sum(loss), wave_sum(kl), wave_count(clipped), wave_count(count)};
}

__global__ __launch_bounds__(256) void k_policy(PolicyArgs a) {
  __shared__ double sums[4][2];
  __shared__ int counts[4][2];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Place at = place_of(a, wave);
  const int64_t b = at.b;
  if (b >= a.B) return;                   // short rows alone: no barrier follows there
  auto [loss, kl, clipped, count] = part_of(a, at, lane);
  if (a.reduction == DET_REDUCE_NONE) return;
  if (a.T > PART) {                       // the piece's four waves, in order
    if (lane == 0) {
      sums[wave][0] = loss;
      sums[wave][1] = kl;
      counts[wave][0] = clipped;
      counts[wave][1] = count;
    }
    __syncthreads();
    if (threadIdx.x != 0) return;
#pragma unroll
    for (int w = 1; w < 4; ++w) {
      loss += sums[w][0];
      kl += sums[w][1];
      clipped += counts[w][0];
      count += counts[w][1];
    }
  }
  if (lane == 0) {
    a.piece_sums[at.piece * a.B + b] = double2{loss, kl};
    a.piece_counts[at.piece * a.B + b] = int2{clipped, count};
  }
}

// Rows joined: a row's pieces are added in 64 bits, in ascending order (up to 16
// of them) or over the lanes of a wave; the rows' values are added exactly.  Three
// sums (loss, KL, clipped) of NDIG digits, their values that are not finite by
// kind, and two counts.
constexpr int SUMS = 3, JOINED = SUMS * NDIG + SUMS + 2, SERIAL = 16, AHEAD = 8, JOIN_THREADS = 1024;

struct JoinTotals {
  unsigned long long digits[SUMS][NDIG][64];                  // a lane's own, or all would wait for one address
  int32_t kinds[SUMS];                    // bit 0: NaN, 1: +inf, 2: -inf
  unsigned long long tokens, rows;
};

// the sum of `digits` and the kinds as a value
template <class D>
__device__ __forceinline__ double sum_value(D digit, int kinds) {
  if (kinds & 1 || kinds == 6) return NAN;
  if (kinds != 0) return kinds == 2 ? INFINITY : -INFINITY;
  return sum_of_digits(digit);
}
// the three results from the totals, divided in 64 bits (a sum may lie past fp32
// where its mean does not) and rounded to fp32 once
__device__ __forceinline__ void policy_results(const PolicyArgs& a, int k, double value, int64_t tokens, int64_t rows) {
  const int64_t n = max<int64_t>(1, a.reduction == DET_REDUCE_TOKENS ? tokens : rows);
  float* const to = k == 0 ? a.loss : k == 1 ? a.kl : a.clipped;
  *to = static_cast<float>(value / static_cast<double>(n));
  if (k == 0) a.count[a.B] = n;
}

__device__ __forceinline__ void clear(JoinTotals& s) {
  unsigned long long* const d = &s.digits[0][0][0];
  for (int i = threadIdx.x; i < SUMS * NDIG * 64; i += JOIN_THREADS) d[i] = 0ull;
  if (threadIdx.x < SUMS) s.kinds[threadIdx.x] = 0;
  if (threadIdx.x == 0) s.tokens = s.rows = 0ull;
}
// Joins the rows whose pieces' sums and counts `get` reads; the totals are cleared,
// and no wave writes what `get` reads any more.
template <class Get>
__device__ __forceinline__ void join_rows(const PolicyArgs& a, JoinTotals& s, Get get) {
  const int lane = threadIdx.x & 63;
  unsigned long long* const d = &s.digits[0][0][0];
  const bool serial = a.pieces <= SERIAL;
  const int64_t at_once = static_cast<int64_t>(a.groups) * (serial ? JOIN_THREADS : JOIN_THREADS / 64);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (serial ? JOIN_THREADS : JOIN_THREADS / 64) +
                        (serial ? threadIdx.x : threadIdx.x >> 6);
  unsigned long long tokens = 0, rows = 0;
  for (int64_t b = first; b < a.B; b += at_once) {
    double sum[SUMS] = {0.0, 0.0, 0.0};
    int64_t clipped = 0, count = 0;
    const int stride = serial ? 1 : 64;
    for (int64_t p0 = serial ? 0 : lane; p0 < a.pieces; p0 += AHEAD * stride) {
      // all in flight before the first is added; past the end: row b's first, not added
      double2 v[AHEAD];
      int2 n[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int64_t p = p0 + i * stride;
        get((p < a.pieces ? p : 0) * a.B + b, v[i], n[i]);
      }
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
        if (p0 + i * stride < a.pieces) {
          sum[0] += v[i].x;
          sum[1] += v[i].y;
          clipped += n[i].x;
          count += n[i].y;
        }
    }
    if (!serial) {
      sum[0] = wave_sum(sum[0]);
      sum[1] = wave_sum(sum[1]);
      clipped = wave_count(static_cast<int>(clipped));        // at most T <= 2^24
      count = wave_count(static_cast<int>(count));
      if (lane != 0) continue;
    }
    sum[2] = static_cast<double>(clipped);
    a.count[b] = count;
    tokens += count;
    rows += count > 0;
#pragma unroll
    for (int k = 0; k < SUMS; ++k) {
      if (a.reduction == DET_REDUCE_SEQUENCES) sum[k] /= static_cast<double>(max<int64_t>(count, 1));
      auto add = [&](int j, int64_t x) { atomicAdd(&s.digits[k][j][lane], static_cast<unsigned long long>(x)); };
      if (!(fabs(sum[k]) < INFINITY)) atomicOr(&s.kinds[k], sum[k] != sum[k] ? 1 : sum[k] > 0.0 ? 2 : 4);
      else add_digits(sum[k], add);
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {      // one address each: a thousand adds in a row would take 9 us
    tokens += __shfl_xor(tokens, o);
    rows += __shfl_xor(rows, o);
  }
  if (lane == 0 && rows != 0) {
    atomicAdd(&s.tokens, tokens);
    atomicAdd(&s.rows, rows);
  }
  __syncthreads();
  if (threadIdx.x < SUMS * NDIG) {
    unsigned long long t = 0;
    unsigned long long* const mine = d + threadIdx.x * 64;
    for (int i = 0; i < 64; ++i) t += mine[(i + threadIdx.x) & 63];       // all in one bank otherwise
    mine[0] = t;
  }
  __syncthreads();
  if (a.groups > 1) {
    int64_t* const out = a.joined + static_cast<int64_t>(blockIdx.x) * JOINED;
    if (threadIdx.x < SUMS * NDIG) out[threadIdx.x] = static_cast<int64_t>(d[threadIdx.x * 64]);
    if (threadIdx.x < SUMS) out[SUMS * NDIG + threadIdx.x] = s.kinds[threadIdx.x];
    if (threadIdx.x == 0) {
      out[SUMS * NDIG + SUMS] = static_cast<int64_t>(s.tokens);
      out[SUMS * NDIG + SUMS + 1] = static_cast<int64_t>(s.rows);
    }
    return;
  }
  if (threadIdx.x < SUMS) {
    const int k = threadIdx.x;
    policy_results(a, k, sum_value([&](int j) { return static_cast<int64_t>(s.digits[k][j][0]); }, s.kinds[k]),
                   static_cast<int64_t>(s.tokens), static_cast<int64_t>(s.rows));
  }
}

__global__ __launch_bounds__(JOIN_THREADS) void k_policy_join(PolicyArgs a) {
  __shared__ JoinTotals s;
  clear(s);
  __syncthreads();
  join_rows(a, s, [&](int64_t at, double2& v, int2& n) {
    v = a.piece_sums[at];
    n = a.piece_counts[at];
  });
}

// A few short rows in one launch, one to a wave: the same sums, read from the LDS.
// In a graph, us a call in one launch and in two: 8 x 300 9.1 and 9.9, 16 x 512 10.0
// and 9.4; two rows to a wave 32 x 64 15.8 and 10.2, 32 x 512 14.4 and 9.4.  A launch
// takes 3 us of the host, which bounds the call outside of graphs.
constexpr int FEW_ROWS = JOIN_THREADS / 64;
__global__ __launch_bounds__(JOIN_THREADS) void k_policy_few(PolicyArgs a) {
  __shared__ JoinTotals s;
  __shared__ double2 sums[FEW_ROWS];
  __shared__ int2 counts[FEW_ROWS];
  clear(s);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (wave < a.B) {
    const Part p = part_of(a, {wave, 0, 0}, lane);
    if (lane == 0) {
      sums[wave] = double2{p.loss, p.kl};
      counts[wave] = int2{p.clipped, p.count};
    }
  }
  __syncthreads();
  join_rows(a, s, [&](int64_t at, double2& v, int2& n) {
    v = sums[at];
    n = counts[at];
  });
}

// the totals of several workgroups
__global__ __launch_bounds__(64) void k_policy_total(PolicyArgs a) {
  __shared__ int64_t s[JOINED];
  if (threadIdx.x < JOINED) {
    const bool kinds = threadIdx.x >= SUMS * NDIG && threadIdx.x < SUMS * NDIG + SUMS;
    int64_t t = 0;
    for (int g = 0; g < a.groups; ++g) {
      const int64_t v = a.joined[static_cast<int64_t>(g) * JOINED + threadIdx.x];
      t = kinds ? t | v : t + v;
    }
    s[threadIdx.x] = t;
  }
  __syncthreads();
  if (threadIdx.x < SUMS) {
    const int k = threadIdx.x;
    policy_results(a, k, sum_value([&](int j) { return s[k * NDIG + j]; }, static_cast<int>(s[SUMS * NDIG + k])),
                   s[SUMS * NDIG + SUMS], s[SUMS * NDIG + SUMS + 1]);
  }
}

__global__ __launch_bounds__(256) void k_policy_grad(PolicyArgs a) {
  const int lane = threadIdx.x & 63;
  const Place at = place_of(a, __builtin_amdgcn_readfirstlane(threadIdx.x >> 6));
  const int64_t b = at.b;
  if (b >= a.B) return;
  const float adv_b = a.adv_t == 0 ? a.adv[b * a.s_adv] : 0.0f;
  float w_b = 0.0f;                       // this row's weight: g over the count it was divided by
  if (a.reduction != DET_REDUCE_NONE) {
    const double n = static_cast<double>(a.count[a.B]) *
                     (a.reduction == DET_REDUCE_SEQUENCES ? static_cast<double>(max<int64_t>(a.count[b], 1)) : 1.0);
    w_b = static_cast<float>(static_cast<double>(a.g[0]) / n);
  }
#pragma unroll
  for (int v = 0; v < VECS; ++v) {
    const int64_t t = at.t + v * 256 + lane * 4;
    const int n = static_cast<int>(max<int64_t>(0, min<int64_t>(4, a.T - t)));
    float lp[4], old[4], adv[4], ref[4], w[4], out[4];
    bool m[4];
    tokens(a.lp, b * a.s_lp + t, n, lp);
    tokens(a.old, b * a.s_old + t, n, old);
    if (a.adv_t != 0) tokens(a.adv, b * a.s_adv + t, n, adv);
    if (a.ref != nullptr) tokens(a.ref, b * a.s_ref + t, n, ref);
    counted(a.mask, b * a.s_mask + t, n, m);
    if (a.reduction == DET_REDUCE_NONE) {
      if (a.s_g_t == 1) {
        tokens(a.g, b * a.s_g + t, n, w);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = j < n ? a.g[b * a.s_g + (t + j) * a.s_g_t] : 0.0f;
      }
    }
    auto take = [&](auto far) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const Token x = token_of<decltype(far)::value>(a, lp[j], old[j], a.adv_t != 0 ? adv[j] : adv_b,
                                                       a.ref != nullptr ? ref[j] : 0.0f);
        out[j] = m[j] ? x.slope * (a.reduction == DET_REDUCE_NONE ? w[j] : w_b) : 0.0f;
      }
    };
    if (any_far(lp, old, m)) take(std::true_type{});
    else take(std::false_type{});
    store_tokens(a.dlp, b * a.T + t, n, out);
  }
}

// ---------------------------------------------------------------- the preference loss
//
//   s = sum over the tokens that count of lp - ref (or its mean), for both sides of a pair
//   z = beta (s_chosen - s_rejected) - margin
//
// One workgroup to a pair: half of its waves to each side, which take parts of
// 512 tokens in turn; two of them where the side has up to 2048 tokens, whatever
// the other one has: the order of a side's sum is its own length's.

struct Side {
  const float* lp; int64_t s_lp;
  const float* ref; int64_t s_ref;        // null: none
  const uint8_t* mask; int64_t s_mask;
  int64_t T;
  float* reward;                          // [P]
  float* dlp;                             // the gradient: [P][T]
};
struct PreferenceArgs {
  Side side[2];
  int64_t P;
  double beta, margin, smooth;
  int kind, by_length;
  float* loss;                            // [P]
  float* slope;                           // [P][2]: d loss / d lp of a token that counts
  const float* g; int64_t s_g;
  int32_t* status;
};

template <int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_preference(PreferenceArgs a) {
  __shared__ double sums[WAVES];
  __shared__ int counts[WAVES];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t p = blockIdx.x;
  const Side& s = a.side[wave < WAVES / 2 ? 0 : 1];
  const int turns = s.T <= 4 * PART ? 2 : WAVES / 2, turn = wave % (WAVES / 2);
  double sum = 0.0;
  int count = 0;
  for (int64_t t0 = turn < turns ? static_cast<int64_t>(turn) * PART : s.T; t0 < s.T; t0 += PART * turns) {
#pragma unroll
    for (int v = 0; v < VECS; ++v) {
      const int64_t t = t0 + v * 256 + lane * 4;
      const int n = static_cast<int>(max<int64_t>(0, min<int64_t>(4, s.T - t)));
      float lp[4], ref[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      bool m[4];
      tokens(s.lp, p * s.s_lp + t, n, lp);
      if (s.ref != nullptr) tokens(s.ref, p * s.s_ref + t, n, ref);
      counted(s.mask, p * s.s_mask + t, n, m);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sum += m[j] ? static_cast<double>(lp[j]) - static_cast<double>(ref[j]) : 0.0;
        count += m[j];
      }
    }
  }
  sum = wave_sum(sum);
  count = wave_count(count);
  if (lane == 0) {
    sums[wave] = sum;
    counts[wave] = count;
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
  double total[2] = {0.0, 0.0}, n[2] = {1.0, 1.0};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    int c = 0;
    for (int w = 0; w < WAVES / 2; ++w) {
      total[k] += sums[k * (WAVES / 2) + w];
      c += counts[k * (WAVES / 2) + w];
    }
    if (a.by_length) {
      n[k] = static_cast<double>(max(c, 1));
      total[k] /= n[k];
    }
    a.side[k].reward[p] = static_cast<float>(a.beta * total[k]);
  }
  const double ahead = total[0] - total[1], z = a.beta * ahead - a.margin;
  double loss, slope;                     // slope: d loss / d (s_chosen - s_rejected)
  if (a.kind == DET_PREFER_SIGMOID) {
    const double e = exp(-fabs(z)), soft = log1p(e), small = e / (1.0 + e), large = 1.0 / (1.0 + e);
    // -ln sigmoid(z), -ln sigmoid(-z)
    const double away = z > 0.0 ? soft : soft - z, toward = z > 0.0 ? soft + z : soft;
    loss = a.smooth == 0.0 ? away : (1.0 - a.smooth) * away + a.smooth * toward;
    slope = a.beta * (a.smooth - (z > 0.0 ? small : large));
    if (z != z) loss = slope = z;
  } else if (a.kind == DET_PREFER_HINGE) {
    loss = z < 1.0 ? 1.0 - z : z == z ? 0.0 : z;
    slope = z < 1.0 ? -a.beta : z == z ? 0.0 : z;
  } else {
    const double off = ahead - 0.5 / a.beta;
    loss = off * off;
    slope = 2.0 * off;
  }
  a.loss[p] = static_cast<float>(loss);
  a.slope[2 * p] = static_cast<float>(slope / n[0]);
  a.slope[2 * p + 1] = static_cast<float>(-slope / n[1]);
  if (!(fabs(loss) < INFINITY)) a.status[0] = 1;
}

// the gradient is one value over the tokens of a side that count
__global__ __launch_bounds__(256) void k_preference_grad(PreferenceArgs a, int64_t parts0, int64_t parts1) {
  const int lane = threadIdx.x & 63;
  int64_t id = static_cast<int64_t>(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (id >= a.P * (parts0 + parts1)) return;
  const int k = id < a.P * parts0 ? 0 : 1;
  if (k != 0) id -= a.P * parts0;
  const int64_t parts = k != 0 ? parts1 : parts0, p = id / parts;
  const Side& s = a.side[k];
  const float value = a.g[p * a.s_g] * a.slope[2 * p + k];
#pragma unroll
  for (int v = 0; v < VECS; ++v) {
    const int64_t t = id % parts * PART + v * 256 + lane * 4;
    const int n = static_cast<int>(max<int64_t>(0, min<int64_t>(4, s.T - t)));
    bool m[4];
    counted(s.mask, p * s.s_mask + t, n, m);
    const float out[4] = {m[0] ? value : 0.0f, m[1] ? value : 0.0f, m[2] ? value : 0.0f, m[3] ? value : 0.0f};
    store_tokens(s.dlp, p * s.T + t, n, out);
  }
}

// ---------------------------------------------------------------- host side

constexpr int64_t T_MAX = int64_t{1} << 24;

int64_t parts_of(int64_t T) { return ceil_div(T, PART); }
int64_t pieces_of(int64_t T) { return T <= PART ? std::min<int64_t>(T, 1) : ceil_div(T, PIECE); }
unsigned policy_blocks(int64_t B, int64_t T) {
  return static_cast<unsigned>(T <= PART ? ceil_div(B, 4) : B * pieces_of(T));
}
// workgroups that join rows: one up to 2^13 pieces of rows (up to 8 to a thread of its 1024)
int groups_of(int64_t B, int64_t pieces) {
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(64, ceil_div(B * pieces, 1 << 13))));
}
struct PolicyRoom {
  int64_t sums, joined, counts, total;
};
PolicyRoom policy_room(int64_t B, int64_t T) {
  const int64_t n = B * pieces_of(T);
  PolicyRoom r;
  r.sums = 0;
  r.joined = n * 16;
  r.counts = r.joined + groups_of(B, pieces_of(T)) * JOINED * 8;
  r.total = r.counts + n * 8;
  return r;
}

bool aligned4(const void* p) { return aligned_for(p, DET_F32); }

det_status check_tokens(int64_t B, int64_t T, std::initializer_list<int64_t> strides) {
  if (B < 0 || T < 0) return fail(DET_EINVAL, "bad size: %lld rows of %lld tokens", (long long)B, (long long)T);
  if (B > DET_ROWS_MAX || T > T_MAX) return fail(DET_EINVAL, "%lld rows of %lld tokens exceed the limits 2^22 and 2^24",
                                                 (long long)B, (long long)T);
  // a launch has fewer than 2^32 threads
  if (B * T > int64_t{1} << 32) return fail(DET_EINVAL, "more than 2^32 tokens in one call");
  for (int64_t s : strides)
    if (s < 0) return fail(DET_EINVAL, "negative stride");
  return DET_OK;
}

det_status check_policy(const PolicyArgs& a, double low, double high, double kl_weight) {
  det_status st = check_tokens(a.B, a.T, {a.s_lp, a.s_old, a.s_adv, a.s_mask, a.s_ref});
  if (st != DET_OK) return st;
  if (!(low >= 0.0) || !(low <= 1.0)) return fail(DET_EINVAL, "clip_low must lie in [0, 1]");
  if (!(high >= 0.0) || !(high < 1e6)) return fail(DET_EINVAL, "clip_high must lie in [0, 1e6)");
  if (!(kl_weight >= 0.0) || !(kl_weight < 1e6)) return fail(DET_EINVAL, "kl_weight must lie in [0, 1e6)");
  if (a.adv_t != 0 && a.adv_t != 1) return fail(DET_EINVAL, "the advantage's tokens are adjacent (1) or one value (0)");
  if (a.reduction != DET_REDUCE_NONE && a.reduction != DET_REDUCE_TOKENS && a.reduction != DET_REDUCE_SEQUENCES)
    return fail(DET_EINVAL, "unknown reduction %d", a.reduction);
  if (kl_weight > 0.0 && a.ref == nullptr && a.B * a.T > 0)
    return fail(DET_EINVAL, "a KL term needs the reference's log probabilities");
  if (a.B * a.T > 0 && (a.lp == nullptr || a.old == nullptr || a.adv == nullptr))
    return fail(DET_EINVAL, "null pointer");
  if (!aligned4(a.lp) || !aligned4(a.old) || !aligned4(a.adv) || !aligned4(a.ref))
    return fail(DET_EINVAL, "operands must be aligned to their element size");
  return DET_OK;
}

PolicyArgs policy_args(const float* lp, int64_t s_lp, const float* old, int64_t s_old, const float* adv, int64_t s_adv,
                       int adv_t, const uint8_t* mask, int64_t s_mask, const float* ref, int64_t s_ref, int64_t B, int64_t T,
                       double low, double high, double kl_weight, det_reduction reduction) {
  PolicyArgs a{};
  a.lp = lp; a.s_lp = s_lp; a.old = old; a.s_old = s_old; a.adv = adv; a.s_adv = s_adv; a.adv_t = adv_t;
  a.mask = mask; a.s_mask = s_mask; a.ref = ref; a.s_ref = s_ref;
  a.B = B; a.T = T; a.pieces = pieces_of(T);
  a.low = log1p(-low); a.high = log1p(high);
  a.bound_low = static_cast<float>(1.0 - low); a.bound_high = static_cast<float>(1.0 + high);
  a.kl_weight = static_cast<float>(kl_weight);
  a.reduction = reduction;
  return a;
}

bool known_kind(int k) { return k == DET_PREFER_SIGMOID || k == DET_PREFER_HINGE || k == DET_PREFER_IPO; }

}  // namespace

extern "C" {

int64_t det_policy_loss_workspace_bytes(int64_t B, int64_t T, det_reduction reduction) {
  if (B <= 0 || T <= 0 || B > DET_ROWS_MAX || T > T_MAX || reduction == DET_REDUCE_NONE) return 0;
  return policy_room(B, T).total;
}

det_status det_policy_loss(const float* logprob, int64_t s_logprob, const float* old_logprob, int64_t s_old,
                           const float* advantage, int64_t s_advantage, int advantage_t, const uint8_t* mask,
                           int64_t s_mask, const float* ref_logprob, int64_t s_ref, int64_t B, int64_t T,
                           double clip_low, double clip_high, double kl_weight, det_reduction reduction, float* loss,
                           float* kl, float* clipped, int64_t* count, void* workspace, size_t workspace_bytes,
                           void* stream) {
  PolicyArgs a = policy_args(logprob, s_logprob, old_logprob, s_old, advantage, s_advantage, advantage_t, mask, s_mask,
                             ref_logprob, s_ref, B, T, clip_low, clip_high, kl_weight, reduction);
  det_status st = check_policy(a, clip_low, clip_high, kl_weight);
  if (st != DET_OK) return st;
  const bool none = reduction == DET_REDUCE_NONE;
  if (none && B * T == 0) return DET_OK;
  if (loss == nullptr || kl == nullptr || clipped == nullptr || (!none && count == nullptr))
    return fail(DET_EINVAL, "null output");
  if (!aligned4(loss) || !aligned4(kl) || !aligned4(clipped) || !aligned8(count))
    return fail(DET_EINVAL, "outputs must be aligned to their element size");
  const int64_t need = det_policy_loss_workspace_bytes(B, T, reduction);
  if (need > 0 && (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 15u) ||
                   workspace_bytes < static_cast<size_t>(need)))
    return fail(DET_EINVAL, "workspace: %lld bytes, 16-byte aligned, are needed", (long long)need);
  a.loss = loss; a.kl = kl; a.clipped = clipped; a.count = count;
  a.status = det_device_status_word();
  if (a.status == nullptr) return DET_EHIP;
  hipStream_t s = static_cast<hipStream_t>(stream);
  a.groups = groups_of(B, a.pieces);
  if (need > 0) {
    const PolicyRoom r = policy_room(B, T);
    char* const ws = static_cast<char*>(workspace);
    a.piece_sums = reinterpret_cast<double2*>(ws + r.sums);
    a.joined = reinterpret_cast<int64_t*>(ws + r.joined);
    a.piece_counts = reinterpret_cast<int2*>(ws + r.counts);
  }
  if (!none && B * T > 0 && B <= FEW_ROWS && T <= PART) {
    hipLaunchKernelGGL(k_policy_few, dim3(1), dim3(JOIN_THREADS), 0, s, a);
    return hip_check(hipGetLastError(), "policy loss launch");
  }
  if (B * T > 0)
    hipLaunchKernelGGL(k_policy, dim3(policy_blocks(B, T)), dim3(256), 0, s, a);
  if (!none) {                            // without tokens: every sum is empty
    hipLaunchKernelGGL(k_policy_join, dim3(a.groups), dim3(JOIN_THREADS), 0, s, a);
    if (a.groups > 1) hipLaunchKernelGGL(k_policy_total, dim3(1), dim3(64), 0, s, a);
  }
  return hip_check(hipGetLastError(), "policy loss launch");
}

det_status det_policy_loss_grad(const float* logprob, int64_t s_logprob, const float* old_logprob, int64_t s_old,
                                const float* advantage, int64_t s_advantage, int advantage_t, const uint8_t* mask,
                                int64_t s_mask, const float* ref_logprob, int64_t s_ref, int64_t B, int64_t T,
                                double clip_low, double clip_high, double kl_weight, det_reduction reduction,
                                const int64_t* count, const float* g, int64_t s_g, int64_t s_g_t, float* dlogprob,
                                void* stream) {
  PolicyArgs a = policy_args(logprob, s_logprob, old_logprob, s_old, advantage, s_advantage, advantage_t, mask, s_mask,
                             ref_logprob, s_ref, B, T, clip_low, clip_high, kl_weight, reduction);
  det_status st = check_policy(a, clip_low, clip_high, kl_weight);
  if (st != DET_OK) return st;
  if (s_g < 0 || s_g_t < 0) return fail(DET_EINVAL, "negative stride");
  if (B * T == 0) return DET_OK;
  if (g == nullptr || dlogprob == nullptr || (reduction != DET_REDUCE_NONE && count == nullptr))
    return fail(DET_EINVAL, "null pointer");
  if (!aligned4(g) || !aligned4(dlogprob) || !aligned8(count))
    return fail(DET_EINVAL, "operands must be aligned to their element size");
  a.count = const_cast<int64_t*>(count);
  a.g = g; a.s_g = s_g; a.s_g_t = s_g_t; a.dlp = dlogprob;
  hipLaunchKernelGGL(k_policy_grad, dim3(policy_blocks(B, T)), dim3(256), 0,
                     static_cast<hipStream_t>(stream), a);
  return hip_check(hipGetLastError(), "policy loss gradient launch");
}

det_status det_preference_loss(const float* chosen, int64_t s_chosen, const float* ref_chosen, int64_t s_ref_chosen,
                               const uint8_t* chosen_mask, int64_t s_chosen_mask, int64_t T_chosen,
                               const float* rejected, int64_t s_rejected, const float* ref_rejected,
                               int64_t s_ref_rejected, const uint8_t* rejected_mask, int64_t s_rejected_mask,
                               int64_t T_rejected, int64_t P, det_preference kind, double beta, double margin,
                               double label_smoothing, int by_length, float* loss, float* chosen_reward,
                               float* rejected_reward, float* slope, void* stream) {
  det_status st = check_tokens(P, std::max(T_chosen, T_rejected),
                               {s_chosen, s_ref_chosen, s_chosen_mask, s_rejected, s_ref_rejected, s_rejected_mask});
  if (st != DET_OK) return st;
  if (T_chosen < 0 || T_rejected < 0) return fail(DET_EINVAL, "negative length");
  if (!known_kind(kind)) return fail(DET_EINVAL, "unknown kind of preference loss %d", kind);
  if (!(beta > 0.0) || !(beta < 1e6)) return fail(DET_EINVAL, "beta must lie in (0, 1e6)");
  if (!(fabs(margin) < INFINITY) || (margin != 0.0 && kind == DET_PREFER_IPO))
    return fail(DET_EINVAL, "margin must be finite, and 0 for ipo");
  if (!(label_smoothing >= 0.0) || !(label_smoothing <= 0.5) || (label_smoothing != 0.0 && kind != DET_PREFER_SIGMOID))
    return fail(DET_EINVAL, "label_smoothing must lie in [0, 0.5], and be 0 unless sigmoid");
  if ((ref_chosen == nullptr) != (ref_rejected == nullptr) && T_chosen > 0 && T_rejected > 0)
    return fail(DET_EINVAL, "reference log probabilities are given for both sides or for none");
  if (P == 0) return DET_OK;
  if ((T_chosen > 0 && chosen == nullptr) || (T_rejected > 0 && rejected == nullptr) || loss == nullptr ||
      chosen_reward == nullptr || rejected_reward == nullptr || slope == nullptr)
    return fail(DET_EINVAL, "null pointer");
  for (const void* p : {static_cast<const void*>(chosen), static_cast<const void*>(rejected),
                        static_cast<const void*>(ref_chosen), static_cast<const void*>(ref_rejected),
                        static_cast<const void*>(loss), static_cast<const void*>(chosen_reward),
                        static_cast<const void*>(rejected_reward), static_cast<const void*>(slope)})
    if (!aligned4(p)) return fail(DET_EINVAL, "operands must be aligned to their element size");
  PreferenceArgs a{};
  a.side[0] = {chosen, s_chosen, ref_chosen, s_ref_chosen, chosen_mask, s_chosen_mask, T_chosen, chosen_reward,
               nullptr};
  a.side[1] = {rejected, s_rejected, ref_rejected, s_ref_rejected, rejected_mask, s_rejected_mask, T_rejected,
               rejected_reward, nullptr};
  a.P = P; a.beta = beta; a.margin = margin; a.smooth = label_smoothing; a.kind = kind; a.by_length = by_length != 0;
  a.loss = loss; a.slope = slope;
  a.status = det_device_status_word();
  if (a.status == nullptr) return DET_EHIP;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (std::max(T_chosen, T_rejected) <= 4 * PART)
    hipLaunchKernelGGL(k_preference<4>, dim3(static_cast<unsigned>(P)), dim3(256), 0, s, a);
  else hipLaunchKernelGGL(k_preference<16>, dim3(static_cast<unsigned>(P)), dim3(1024), 0, s, a);
  return hip_check(hipGetLastError(), "preference loss launch");
}

det_status det_preference_loss_grad(const uint8_t* chosen_mask, int64_t s_chosen_mask, int64_t T_chosen,
                                    const uint8_t* rejected_mask, int64_t s_rejected_mask, int64_t T_rejected, int64_t P,
                                    const float* slope, const float* g, int64_t s_g, float* dchosen, float* drejected,
                                    void* stream) {
  det_status st = check_tokens(P, std::max(T_chosen, T_rejected), {s_chosen_mask, s_rejected_mask, s_g});
  if (st != DET_OK) return st;
  if (T_chosen < 0 || T_rejected < 0) return fail(DET_EINVAL, "negative length");
  // a side whose gradient is not needed has no parts
  const int64_t parts0 = dchosen == nullptr ? 0 : parts_of(T_chosen);
  const int64_t parts1 = drejected == nullptr ? 0 : parts_of(T_rejected);
  if (P * (parts0 + parts1) == 0) return DET_OK;
  if (slope == nullptr || g == nullptr) return fail(DET_EINVAL, "null pointer");
  if (!aligned4(slope) || !aligned4(g) || !aligned4(dchosen) || !aligned4(drejected))
    return fail(DET_EINVAL, "operands must be aligned to their element size");
  PreferenceArgs a{};
  a.side[0].mask = chosen_mask; a.side[0].s_mask = s_chosen_mask; a.side[0].T = T_chosen; a.side[0].dlp = dchosen;
  a.side[1].mask = rejected_mask; a.side[1].s_mask = s_rejected_mask; a.side[1].T = T_rejected; a.side[1].dlp = drejected;
  a.P = P; a.slope = const_cast<float*>(slope); a.g = g; a.s_g = s_g;
  hipLaunchKernelGGL(k_preference_grad, dim3(static_cast<unsigned>(ceil_div(P * (parts0 + parts1), 4))), dim3(256), 0,
                     static_cast<hipStream_t>(stream), a, parts0, parts1);
  return hip_check(hipGetLastError(), "preference loss gradient launch");
}

}  // extern "C"
