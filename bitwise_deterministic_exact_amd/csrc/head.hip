// The losses and scores of a language model's head for MI355X (gfx950): log
// probabilities of given tokens with entropy and top alternatives, and the
// distillation loss against a teacher's top logits, each with its gradient.
//
// For a row z of V logits and a scale s > 0 (1 / temperature):
//   l_j = s z_j - ln sum_i exp(s z_i),   p_j = exp(l_j)
//   logprob = l_t,   entropy H = -sum_j p_j l_j
//   loss = T^2 sum_k q_k (ln q_k - l_{i_k}),  q = softmax(teacher / T), s = 1/T
// and the gradients
//   dz_j = s (sum of the incoming gradients of j's own log probabilities
//             - p_j (G + gH (H + l_j))),  G = all of those gradients' sum
//   dz_j = g T (p_j - sum_{k: i_k = j} q_k)
//
// Everything is one pass over the logits: a wave takes a chunk of 2048
// consecutive logits into registers, finds its maximum m, and forms
// S = sum 2^(c (z - m)) and U = sum c (z - m) 2^(c (z - m)), c = s log2 e.
// The chunks' (m, S, U) are joined in 64 bits in a fixed order.  The chunks are
// cut by V alone, so a row's bits are a function of that row: not of the
// batch, of how many workgroups share a row, or of the alignment.
#include <algorithm>
#include <type_traits>

#include "rowops.h"

// every fused multiply-add below is written as one: the compiler forms none
#pragma clang fp contract(off)

namespace {

using namespace rowops;

constexpr int CHUNK_BITS = 11, CHUNK = 1 << CHUNK_BITS;       // logits per wave and step
constexpr int LANE_ELEMS = CHUNK / 64;    // 32 in registers per lane
constexpr int WAVES = 4;                  // per workgroup
constexpr int TOP_MAX = DET_HEAD_TOP_MAX;                     // alternatives per row: one per lane
static_assert(TOP_MAX == 64);
constexpr int LDS_PARTS = 512;            // chunks of a row whose (m, S, U) fit one workgroup's LDS
constexpr double LOG2E = 1.4426950408889634074, LN2 = 0.69314718055994530942;

constexpr int MODE_SCORE = 0, MODE_DISTILL = 1;

struct ScoreArgs {
  const void* z; int64_t s_row;
  int64_t N, V;
  float c;                                // s log2 e
  double scale;                           // s
  int dt, mode;
  int nchunk;                             // ceil(V / CHUNK)
  int wpr;                                // waves of a workgroup that share a row (1, 2, 4)
  int nblk;                               // workgroups that share a row (> 1 only with wpr = 4)
  int top;                                // alternatives
  // workspace of a row shared by several workgroups
  float* parts;                           // [N][nchunk][3]
  uint64_t* lists;                        // [N][nblk * WAVES][top]: the waves' lists, sorted, 0 at the end
  // score
  const int64_t* target; int64_t s_target;
  int64_t ignore;
  float* logprob; float* entropy;
  int64_t* top_index; float* top_value;
  // distill
  const void* teacher; int64_t s_teacher; int tdt;
  const int64_t* entry; int64_t s_entry;
  int K;
  float* q;                               // [N][K]
  float* loss;
  float4* stat;                           // [N]: m, 1/S, log2 S, H
  int32_t* status;
};

// ---------------------------------------------------------------- order keys
//
// (value, index) as one integer whose order is "larger value first, then lower
// index": the float's bits mapped to an order-preserving integer (-0 as +0)
// above the complement of the index.  Keys of a row are distinct, so the top
// k are one set whatever the order in which candidates are found.
__device__ __forceinline__ uint32_t order_bits(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t o) {
  return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ uint64_t key_of(uint32_t order, uint32_t index) {
  return (static_cast<uint64_t>(order) << 32) | (0xFFFFFFFFu - index);
}

// The largest `want` of the n keys in LDS at pool[0..n), sorted, into out (not
// overlapping the pool), by `lanes` threads numbered `t` (all of a wave, or of
// a workgroup): each key's rank is the number of larger keys, read two to an
// access and 16 in flight.  n^2 / lanes comparisons: n is close to `want`
// except for rows built against it.  pool is 16-byte aligned; the keys behind
// n up to a multiple of 16 are read and must be readable, their values unused.
__device__ __forceinline__ void rank_keys(const uint64_t* pool, int n, uint64_t* out, int want, int t, int lanes) {
  const ulonglong2* const two = reinterpret_cast<const ulonglong2*>(pool);
  for (int e = t; e < n; e += lanes) {
    const uint64_t mine = pool[e];
    int rank = 0;
    for (int i = 0; i < n; i += 16) {
      ulonglong2 k[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) k[j] = two[(i >> 1) + j];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        rank += i + 2 * j < n && k[j].x > mine ? 1 : 0;
        rank += i + 2 * j + 1 < n && k[j].y > mine ? 1 : 0;
      }
    }
    if (rank < want) out[rank] = mine;
  }
}

// how many lanes below this one are set in b
__device__ __forceinline__ int lanes_below(uint64_t b) {
  return __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(b >> 32), __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(b), 0));
}

// A bar that `want` of the lanes' keys reach (more only if keys are equal):
// the largest such one is sought bit by bit, but any that exactly `want` reach
// will do.  0 when fewer keys than that are not 0.
__device__ __forceinline__ uint64_t bar_of_lanes(uint64_t mine, int want) {
  uint64_t t = 0;
#pragma unroll 1
  for (uint64_t bit = 1ull << 63; bit != 0; bit >>= 1) {
    const int reach = __popcll(__ballot(mine >= (t | bit)));
    if (reach >= want) t |= bit;
    if (reach == want) break;
  }
  return t;
}

// ---------------------------------------------------------------- one chunk

// Vector i of a lane nominally starts at element base + (64 i + lane) VE; one
// that would pass the row's end starts at V - VE instead, so every load is a
// whole vector: its elements before the nominal start belong to the vector
// before it.  (With the row's last elements one by one under a branch, the
// loads of that wave waited for each other.)  A row shorter than a chunk leaves
// out the vectors that it does not reach: 400000 x 300 fp32 512 -> 320 us, its
// gradient 706 -> 322.  The last chunk of a longer row loads them all the same:
// with a branch per vector there, 50000 x 4000 bf16 took 120 us instead of 116.
template <int DT>
__device__ __forceinline__ int64_t vector_start(int64_t at, int64_t V) {
  return V >= Elem<DT>::VE ? min(at, V - Elem<DT>::VE) : at;
}

// a chunk's logits as they are loaded; MASK: -inf in the places of elements
// that are not the vector's own
template <int DT, bool MASK, bool NT>
__device__ __forceinline__ void load_chunk(const void* row, int64_t base, int64_t V, int lane,
                                           float (&v)[LANE_ELEMS]) {
  constexpr int VE = Elem<DT>::VE, NV = LANE_ELEMS / VE;
  if (base + CHUNK <= V) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      load_vec<DT, VE, NT>(row, base + (i * 64 + lane) * VE, reinterpret_cast<float (&)[VE]>(v[i * VE]));
  } else if (V >= VE) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (V > CHUNK || i * 64 * VE < V) {                     // uniform
        load_vec<DT, VE, NT>(row, vector_start<DT>(base + (i * 64 + lane) * VE, V),
                             reinterpret_cast<float (&)[VE]>(v[i * VE]));
      } else {
#pragma unroll
        for (int j = 0; j < VE; ++j) v[i * VE + j] = -INFINITY;
      }
    }
    if constexpr (MASK) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int64_t at = base + (i * 64 + lane) * VE;
        const int own = static_cast<int>(at - vector_start<DT>(at, V));
#pragma unroll
        for (int j = 0; j < VE; ++j) v[i * VE + j] = j >= own ? v[i * VE + j] : -INFINITY;
      }
    }
  } else {                               // fewer elements than a vector: lane 0, one by one
#pragma unroll
    for (int j = 0; j < LANE_ELEMS; ++j)
      v[j] = lane == 0 && j < V ? load_elem<DT>(row, j) : -INFINITY;
  }
}

// The largest keys of the logits a wave has seen, found without keeping the
// logits.  Every chunk leaves only its lanes' maxima in the LDS; after at most
// STEP_CHUNKS chunks the (lane, chunk) pairs whose best possible key passes
// the bar are listed, and only those pairs' logits are read again (from the
// caches), 64 vectors at a time.  On unordered rows that is little more than
// one pair per key.  The bar is the last key of a full list; before that, the
// top-th largest of the pairs' maxima, which at least `top` logits reach.
// Candidates collect in a pool, which is ranked down to `top` keys (and the
// bar raised) whenever 64 more might not fit, so ties, masks and rows built
// against it cost time but no correctness.
//   1024 x 131072 bf16, top 20: 75 us (50 without alternatives); 108 with the
//   logits of a chunk kept in registers for its candidates (123 registers, a
//   ranking per chunk).
template <int NW>                         // waves per workgroup: 16 of them share the LDS more sparingly
struct TopLds {
  static constexpr int STEP_CHUNKS = NW == WAVES ? 8 : 4, POOL = NW == WAVES ? 256 : 128;
  uint64_t pool[POOL];
  float lane_max[STEP_CHUNKS * 64];
  uint16_t pairs[STEP_CHUNKS * 64];
};

template <int DT, int NW>
struct TopList {
  static constexpr int VE = Elem<DT>::VE, NV = LANE_ELEMS / VE;
  static constexpr int STEP_CHUNKS = TopLds<NW>::STEP_CHUNKS, POOL = TopLds<NW>::POOL;
  TopLds<NW>& m;
  uint64_t* list;                        // the result: sorted
  const void* row;
  int64_t V;
  int top, n;                            // n keys in the pool
  uint64_t bar;                          // keys up to it are not wanted

  // down to `top` keys: 64 or fewer by rank, sorted; more by the largest value
  // that `top` of them reach, bit by bit (ranking 256 keys took 10 us)
  __device__ __forceinline__ void prune(int lane) {
    wave_sync();
    if (n > 64) {
      uint64_t k[POOL / 64], t = 0;
#pragma unroll
      for (int i = 0; i < POOL / 64; ++i) k[i] = i * 64 + lane < n ? m.pool[i * 64 + lane] : 0;
      // one value throughout (masked or constant logits): only the indices decide
      int same = 0;
#pragma unroll
      for (int i = 0; i < POOL / 64; ++i) same += __popcll(__ballot(k[i] != 0 && (k[i] >> 32) == (bar >> 32)));
      if (same == n) t = bar & 0xFFFFFFFF00000000ull;
#pragma unroll 1
      for (int bit = same == n ? 31 : 63; bit >= 0; --bit) {
        const uint64_t c = t | (1ull << bit);
        int reach = 0;
#pragma unroll
        for (int i = 0; i < POOL / 64; ++i) reach += __popcll(__ballot(k[i] >= c));
        if (reach >= top) t = c;
        if (reach == top) break;
      }
      wave_sync();
      n = 0;
#pragma unroll
      for (int i = 0; i < POOL / 64; ++i) {
        const uint64_t b = __ballot(k[i] >= t);
        if (k[i] >= t) m.pool[n + lanes_below(b)] = k[i];
        n += __popcll(b);
      }
      bar = max(bar, t);
      wave_sync();
      return;
    }
    rank_keys(m.pool, n, list, top, lane, 64);
    wave_sync();
    n = min(n, top);
    if (lane < n) m.pool[lane] = list[lane];
    wave_sync();
    if (n == top) bar = max(bar, list[top - 1]);
  }

  // the top-th largest of the pairs' maxima, bit by bit from the top; any value
  // that exactly `top` of them reach will do.  Of masked or constant logits
  // all are equal to the largest.
  template <int M>
  __device__ __forceinline__ uint32_t value_bar(int64_t first, int64_t step, int count, uint32_t most, int lane) const {
    uint32_t o[M], t = 0;
    int ties = 0;
#pragma unroll
    for (int i = 0; i < M; ++i) {
      o[i] = 0;
      if (i < count && (first + i * step) * CHUNK + lane * VE < V) o[i] = order_bits(m.lane_max[i * 64 + lane]);
      ties += __popcll(__ballot(o[i] == most));
    }
    if (ties >= top) return most;
#pragma unroll 1
    for (uint32_t bit = 0x80000000u; bit != 0; bit >>= 1) {
      if ((t | bit) > most) continue;
      int reach = 0;
#pragma unroll
      for (int i = 0; i < M; ++i) reach += __popcll(__ballot(o[i] >= (t | bit)));
      if (reach >= top) t |= bit;
      if (reach == top) break;
    }
    return t;
  }

  // chunks first, first + step, ..: `count` of them, their lane maxima in m.lane_max
  // and the largest of them
  __device__ __forceinline__ void take(int64_t first, int64_t step, int count, float largest, int lane) {
    wave_sync();
    if (n < top) {
      const uint32_t most = order_bits(largest);
      const uint32_t t = count == 1 ? value_bar<1>(first, step, count, most, lane)
                                    : value_bar<STEP_CHUNKS>(first, step, count, most, lane);
      bar = max(bar, static_cast<uint64_t>(t) << 32);         // below every logit of that value
    }
    int pairs = 0;
    for (int i = 0; i < count; ++i) {
      const bool hit = best_key(i, lane, first + i * step) > bar;
      const uint64_t b = __ballot(hit);
      if (hit) m.pairs[pairs + lanes_below(b)] = static_cast<uint16_t>(i * 64 + lane);
      pairs += __popcll(b);
    }
    wave_sync();
    // NV lanes to a pair, one for each of its vectors
    for (int p = lane / NV; p - lane / NV < pairs; p += 64 / NV) {
      const int e = p < pairs ? m.pairs[p] : 0;
      const int64_t ch = first + (e >> 6) * step;
      const bool on = p < pairs && best_key(e >> 6, e & 63, ch) > bar;
      if (__ballot(on) == 0) continue;
      const int64_t at = ch * CHUNK + ((lane & (NV - 1)) * 64 + (e & 63)) * VE;
      const int64_t from = vector_start<DT>(at, V);
      float v[VE];
#pragma unroll
      for (int j = 0; j < VE; ++j) v[j] = -INFINITY;
      if (on && at < V) {
        if (V >= VE) {
          load_vec<DT, VE>(row, from, v);
        } else {
#pragma unroll
          for (int j = 0; j < VE; ++j)
            if (j < V) v[j] = load_elem<DT>(row, j);
        }
      }
      // NaN is no candidate: its row's results are NaN
      uint64_t key[VE];
      int more = 0;
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        key[j] = on && from + j >= at && from + j < V && v[j] == v[j]
                     ? key_of(order_bits(v[j]), static_cast<uint32_t>(from + j)) : 0;
        more += __popcll(__ballot(key[j] > bar));
      }
      if (n + more <= POOL) {
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          const uint64_t b = __ballot(key[j] > bar);
          if (key[j] > bar) m.pool[n + lanes_below(b)] = key[j];
          n += __popcll(b);
        }
        continue;
      }
#pragma unroll 1
      for (int j = 0; j < VE; ++j) {     // 64 at a time, with a smaller pool before each
        const uint64_t k = key[0];
#pragma unroll
        for (int i = 0; i + 1 < VE; ++i) key[i] = key[i + 1];
        uint64_t b = __ballot(k > bar);
        if (b == 0) continue;
        if (n + 64 > POOL) {
          prune(lane);
          b = __ballot(k > bar);
          if (b == 0) continue;
        }
        if (k > bar) m.pool[n + lanes_below(b)] = k;
        n += __popcll(b);
      }
    }
    if (n > 64) prune(lane);             // a selection; then the list, sorted
    prune(lane);
  }

  // no logit of lane `l` in the i-th listed chunk has a larger key
  __device__ __forceinline__ uint64_t best_key(int i, int l, int64_t ch) const {
    const int64_t at = ch * CHUNK + l * VE;
    return at < V ? key_of(order_bits(m.lane_max[i * 64 + l]), static_cast<uint32_t>(at)) : 0;
  }
};

// ---------------------------------------------------------------- a row's end
//
// One wave joins a row's chunk sums in 64 bits and writes the row's results.
// Conventions: a row of nothing but -inf has log probabilities -inf, entropy
// 0 and probabilities 0; a NaN or +inf makes S NaN and with it every result.
struct RowSums {
  float m;                               // the maximum (0 for an empty row)
  double log2s;                          // log2 S (0 for an empty row)
  bool empty, bad;
};

__device__ __forceinline__ RowSums join(const ScoreArgs& a, const float* parts, int64_t row, int lane) {
  RowSums r;
  double S = 0.0, U = 0.0;
  if (a.nchunk == 1) {                   // uniform: nothing to join (the general way gives the same bits)
    const float m = parts[0];
    S = parts[1];
    U = parts[2];
    r.bad = S != S;
    r.empty = m == -INFINITY && !r.bad;
    r.m = m == -INFINITY ? 0.0f : m;
  } else {
    float m = -INFINITY;
    bool nan = false;
    for (int i = lane; i < a.nchunk; i += 64) {
      m = fmaxf(m, parts[3 * i]);
      nan |= parts[3 * i + 1] != parts[3 * i + 1];
    }
    m = wave_max(m);
    r.bad = __ballot(nan) != 0;
    r.empty = m == -INFINITY && !r.bad;
    r.m = m == -INFINITY ? 0.0f : m;
    const double c = a.scale * LOG2E;
    for (int i = lane; i < a.nchunk; i += 64) {
      const float mi = parts[3 * i];
      if (mi == -INFINITY) continue;
      const double d = (static_cast<double>(mi) - static_cast<double>(r.m)) * c;
      const double f = exp2(d), s = parts[3 * i + 1];
      if (f > 0.0) {
        S += s * f;
        U += f * (parts[3 * i + 2] + d * s);
      }
    }
    S = wave_sum(S);
    U = wave_sum(U);
  }
  r.log2s = r.empty ? 0.0 : log2(S);
  double H = r.empty ? 0.0 : LN2 * (r.log2s - U / S);
  if (H < 0.0) H = 0.0;                  // rounding of the 32-bit chunk sums
  if (r.bad) { r.log2s = NAN; H = NAN; }
  if (lane == 0) {
    a.stat[row] = make_float4(r.m, r.empty ? 0.0f : (r.bad ? NAN : static_cast<float>(1.0 / S)),
                              static_cast<float>(r.log2s), static_cast<float>(H));
    if (a.entropy != nullptr) a.entropy[row] = static_cast<float>(H);
    if (r.bad) a.status[0] = 1;
  }
  return r;
}

__device__ __forceinline__ double log_prob(const ScoreArgs& a, const RowSums& r, float z) {
  return (static_cast<double>(z) - static_cast<double>(r.m)) * a.scale - LN2 * r.log2s;
}

// the row's alternatives from its sorted keys (fewer than `top` only in a bad row)
__device__ __forceinline__ void write_top(const ScoreArgs& a, const RowSums& r, int64_t row, const uint64_t* list,
                                          int t) {
  if (t >= a.top) return;
  const uint64_t key = list[t];
  a.top_index[row * a.top + t] = r.bad ? -1 : static_cast<int64_t>(0xFFFFFFFFu - static_cast<uint32_t>(key));
  a.top_value[row * a.top + t] =
      r.bad ? NAN : static_cast<float>(log_prob(a, r, order_value(static_cast<uint32_t>(key >> 32))));
}

// What the end of a row reads besides the sums, read before the row's chunks:
// lane k's teacher entry (of the first 64) and its logit, or the target's.
struct Ahead {
  int64_t index;
  float teacher, z;
};

__device__ __forceinline__ float logit_at(const ScoreArgs& a, int64_t row, int64_t i) {
  return i >= 0 && i < a.V ? load_elem(a.dt, a.z, row * a.s_row + i) : 0.0f;
}

__device__ __forceinline__ Ahead read_ahead(const ScoreArgs& a, int64_t row, int lane) {
  Ahead h{-1, -INFINITY, 0.0f};
  if (a.mode == MODE_DISTILL) {
    if (lane < a.K) {
      h.index = a.entry[row * a.s_entry + lane];
      h.teacher = load_elem(a.tdt, a.teacher, row * a.s_teacher + lane);
      h.z = logit_at(a, row, h.index);
    }
  } else if (a.target != nullptr) {
    h.index = a.target[row * a.s_target];
    h.z = logit_at(a, row, h.index);
  }
  return h;
}

__device__ __forceinline__ void finish_score(const ScoreArgs& a, const RowSums& r, int64_t row, int lane,
                                             const Ahead& h) {
  if (lane != 0 || a.target == nullptr) return;
  float lp;
  if (h.index == a.ignore) lp = 0.0f;
  else if (h.index < 0 || h.index >= a.V || r.bad) lp = NAN;
  else lp = static_cast<float>(log_prob(a, r, h.z));
  a.logprob[row] = lp;
}

__device__ __forceinline__ void finish_distill(const ScoreArgs& a, const RowSums& r, int64_t row, int lane,
                                               const Ahead& h) {
  // q in 64 bits: K is small beside V
  const int64_t t0 = row * a.s_teacher, e0 = row * a.s_entry;
  auto teacher = [&](int k) { return k == lane ? h.teacher : load_elem(a.tdt, a.teacher, t0 + k); };
  float m = -INFINITY;
  bool nan = false;
  for (int k = lane; k < a.K; k += 64) {
    const float t = teacher(k);
    nan |= !(t < INFINITY);              // NaN or +inf
    m = fmaxf(m, t);
  }
  m = wave_max(m);
  const bool bad = __ballot(nan) != 0;
  const bool none = m == -INFINITY;      // no entry at all: loss and gradient 0
  double sum = 0.0;
  for (int k = lane; k < a.K; k += 64) {
    const float t = teacher(k);
    if (t > -INFINITY) sum += exp((static_cast<double>(t) - m) * a.scale);
  }
  sum = wave_sum(sum);
  const double lsum = none ? 0.0 : log(sum), inv = none ? 0.0 : 1.0 / sum;
  double loss = 0.0;
  bool invalid = false;
  for (int k = lane; k < a.K; k += 64) {
    const float t = teacher(k);
    float qk = 0.0f;
    if (t > -INFINITY) {
      const double d = (static_cast<double>(t) - m) * a.scale;
      const double q = exp(d) * inv;
      qk = static_cast<float>(q);
      if (q > 0.0) {
        const int64_t i = k == lane ? h.index : a.entry[e0 + k];
        if (i < 0 || i >= a.V) invalid = true;
        else loss += q * (d - lsum - log_prob(a, r, k == lane ? h.z : logit_at(a, row, i)));
      }
    }
    a.q[row * a.K + k] = bad ? NAN : qk;
  }
  loss = wave_sum(loss);
  // An entry outside the vocabulary leaves the row without a loss and, by q = 0
  // throughout, without a gradient: one without that entry's -q would push
  // probability out of the vocabulary.
  const bool lost = __ballot(invalid) != 0;
  if (lost && !bad)
    for (int k = lane; k < a.K; k += 64) a.q[row * a.K + k] = 0.0f;
  if (lane == 0) {
    a.loss[row] = (bad || lost || r.bad) ? NAN : static_cast<float>(loss / (a.scale * a.scale));
    if (bad) a.status[0] = 1;
  }
}

// The largest `top` keys of `lists` (up to 64) sorted lists of `top` keys, 0 at
// their ends, by a whole workgroup of `threads`; sorted, in LDS from `room` on
// (TOP_MAX + lists * top + 16 keys).  Only those keys can be among them that
// reach a bar: for any j, the ceil(top / j)-th largest of the lists' j-th keys,
// which at least `top` keys reach.  With j = ceil(2 top / lists), on unordered
// rows, about twice `top` keys reach it and are ranked.
template <class F>
__device__ __forceinline__ uint64_t* top_of_lists(F key, int lists, int top, uint64_t* room, int threads) {
  __shared__ int count;
  __shared__ uint64_t bar;
  uint64_t* const best = room;
  uint64_t* const pool = room + TOP_MAX;
  if (threadIdx.x < 64) {
    const int l = threadIdx.x;
    const bool some = l < lists && key(l, 0) != 0;
    const int held = max(__popcll(__ballot(some)), 1);        // lists with a key (none: a row of NaN)
    const int j = min((2 * top + held - 1) / held, top);
    uint64_t b = bar_of_lanes(some ? key(l, j - 1) : 0, (top + j - 1) / j);
    if (b == 0) b = bar_of_lanes(some ? key(l, top - 1) : 0, 1);          // short lists
    if (l == 0) {
      bar = b > 0 ? b : 1;
      count = 0;
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < lists * top; e += threads) {
    const uint64_t k = key(e / top, e % top);
    if (k >= bar) pool[atomicAdd(&count, 1)] = k;
  }
  __syncthreads();
  rank_keys(pool, count, best, top, threadIdx.x, threads);
  __syncthreads();
  return best;
}

// ---------------------------------------------------------------- the pass
//
// Wave w of a row (of nblk * wpr) takes chunks w, w + nblk * wpr, ...  With
// one workgroup per row (nblk = 1) one of its waves also finishes the row; rows
// of at most one or two chunks share a workgroup (wpr = 1, 2).  4096 x 131072
// bf16 take 167 us: 6.4 TB/s, more than a copy's reads and writes together.
// 8.8 vector instructions per logit, the exponential twice as long as the
// others, are 0.8 of the issue slots in that time.
template <int DT, bool TOP, int NW>
__global__ __launch_bounds__(64 * NW) void k_score(ScoreArgs a) {
  constexpr int VE = Elem<DT>::VE, NV = LANE_ELEMS / VE;
  extern __shared__ __align__(16) uint64_t lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rpb = NW / a.wpr;                                 // rows per workgroup
  const int64_t blk = blockIdx.x;
  const int64_t row = a.nblk > 1 ? blk / a.nblk : blk * rpb + wave / a.wpr;
  const int part = a.nblk > 1 ? static_cast<int>(blk % a.nblk) : 0;
  const int rw = wave % a.wpr;                                // this wave within the row and workgroup
  const bool live = row < a.N;
  const bool whole = a.nblk == 1;
  // LDS: the waves' room for their candidates and their lists, then the rows' chunk sums
  using Top = TopLds<NW>;
  Top* const tops = reinterpret_cast<Top*>(lds);
  uint64_t* const lists = reinterpret_cast<uint64_t*>(tops + (TOP ? NW : 0));
  float* const lparts = reinterpret_cast<float*>(lists + (TOP ? NW * TOP_MAX : 0));
  float* const parts = whole ? lparts + (wave / a.wpr) * a.nchunk * 3 : a.parts + row * a.nchunk * 3;
  Top& mine = tops[wave];                // these two are not touched without TOP
  uint64_t* const list = lists + wave * TOP_MAX;

  Ahead ahead{};
  if (live) {
    if (whole && rw == (NW > WAVES ? NW - 1 : 0)) ahead = read_ahead(a, row, lane);   // the wave that finishes
    const void* const zr = static_cast<const char*>(a.z) + row * a.s_row * Elem<DT>::BYTES;
    TopList<DT, NW> tl{mine, list, zr, a.V, a.top, 0, 0};
    const int step = a.nblk * a.wpr;
    bool masked = false;
    int waiting = 0;                     // chunks whose lane maxima wait for `take`
    float largest = -INFINITY;
    for (int ch = part * a.wpr + rw; ch < a.nchunk; ch += step) {
      const int64_t base = static_cast<int64_t>(ch) * CHUNK;
      float v[LANE_ELEMS];
      // Read past the caches (alternatives are read again from where the loads
      // left them): 4096 x 131072 bf16 181 us against 193, and with the gradient
      // that reads them again 577 against 603, 1024 x 32000 fp32 67 against 83;
      // only for logits that stay in a cache whole (4096 x 4096 bf16) 29.5 against 28.0.
      load_chunk<DT, true, !TOP>(zr, base, a.V, lane, v);
      float lane_max = -INFINITY;
#pragma unroll
      for (int j = 0; j < LANE_ELEMS; ++j) lane_max = fmaxf(lane_max, v[j]);
      const float m = wave_max(lane_max);
      const float ref = m == -INFINITY ? 0.0f : m;
      // e d is 0 -inf for a masked logit.  The bound on d that gives 0 there
      // instead changes no other bit (e is 0 long before d passes it), so it is
      // left out until a chunk needs it, and taken from then on.
      float s = 0.0f, u = 0.0f;
      if (!masked && base + CHUNK <= a.V) {
#pragma unroll
        for (int j = 0; j < LANE_ELEMS; ++j) {
          const float d = (v[j] - ref) * a.c;
          const float e = __builtin_amdgcn_exp2f(d);
          s += e;
          u = fmaf(e, d, u);
        }
        masked = __ballot(u != u && s == s) != 0;
      }
      if (masked || base + CHUNK > a.V) {                     // uniform
        s = u = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (base + i * 64 * VE >= a.V) break;               // uniform: nothing but the padding is left
#pragma unroll
          for (int j = i * VE; j < (i + 1) * VE; ++j) {
            const float d = (v[j] - ref) * a.c;
            const float e = __builtin_amdgcn_exp2f(d);
            s += e;
            u = fmaf(e, fmaxf(d, -2000.0f), u);
          }
        }
      }
      s = wave_sum(s);
      u = wave_sum(u);
      if (lane == 0) {
        parts[3 * ch] = m;
        parts[3 * ch + 1] = s;
        parts[3 * ch + 2] = u;
      }
      if constexpr (TOP) {
        mine.lane_max[waiting * 64 + lane] = lane_max;
        ++waiting;
        largest = fmaxf(largest, m);
        if (waiting == Top::STEP_CHUNKS || ch + step >= a.nchunk) {
          tl.take(ch - static_cast<int64_t>(waiting - 1) * step, step, waiting, largest, lane);
          waiting = 0;
          largest = -INFINITY;
        }
      }
    }
    if constexpr (TOP) {
      if (lane >= tl.n && lane < a.top) list[lane] = 0;       // a wave with few elements
      wave_sync();
    }
  }
  if (whole) __syncthreads();            // uniform: the other waves' sums and lists
  if constexpr (NW > WAVES) {            // one row, all waves here
    __shared__ RowSums sums;
    if (wave == NW - 1) {
      const RowSums r = join(a, parts, row, lane);
      if (lane == 0) sums = r;
      if (a.mode == MODE_DISTILL) finish_distill(a, r, row, lane, ahead);
      else finish_score(a, r, row, lane, ahead);
    }
    if constexpr (TOP) {
      // the waves' candidates are done with: their room holds the lists' keys
      uint64_t* const best = top_of_lists([&](int l, int j) { return lists[l * TOP_MAX + j]; }, NW, a.top, lds, 64 * NW);
      if (wave == 0) write_top(a, sums, row, best, lane);
    }
    return;
  } else {
    if (!live) return;
    if (!whole) {                        // k_score_join does the rest
      if (TOP && lane < a.top) a.lists[((row * a.nblk + part) * WAVES + wave) * a.top + lane] = list[lane];
      return;
    }
    if (rw != 0) return;
    const uint64_t* top = list;
    if (TOP && a.wpr > 1) {
      // the row's wave lists, gathered into this wave's pool, joined into the next one's
      for (int w = 0; w < a.wpr; ++w)
        if (lane < a.top) mine.pool[w * a.top + lane] = list[w * TOP_MAX + lane];
      uint64_t* const joined = tops[wave + 1].pool;
      if (lane < a.top) joined[lane] = 0;  // a row with a NaN may hold fewer than `top` keys
      wave_sync();
      rank_keys(mine.pool, a.wpr * a.top, joined, a.top, lane, 64);
      wave_sync();
      top = joined;
    }
    const RowSums r = join(a, parts, row, lane);
    if (a.mode == MODE_DISTILL) finish_distill(a, r, row, lane, ahead);
    else finish_score(a, r, row, lane, ahead);
    if constexpr (TOP) write_top(a, r, row, top, lane);
  }
}

// The end of rows that several workgroups shared: one workgroup per row, its
// last wave for everything but the alternatives.
__global__ __launch_bounds__(256) void k_score_join(ScoreArgs a) {
  extern __shared__ __align__(16) uint64_t lds[];
  __shared__ RowSums sums;
  const int64_t row = blockIdx.x;
  if (threadIdx.x >= 192) {
    const int l = threadIdx.x - 192;
    const Ahead ahead = read_ahead(a, row, l);
    const RowSums r = join(a, a.parts + row * a.nchunk * 3, row, l);
    if (l == 0) sums = r;
    if (a.mode == MODE_DISTILL) finish_distill(a, r, row, l, ahead);
    else finish_score(a, r, row, l, ahead);
  }
  if (a.top == 0) return;                 // uniform
  const int lists = a.nblk * WAVES;
  const uint64_t* const src = a.lists + row * lists * a.top;
  uint64_t* const best = top_of_lists([&](int l, int j) { return src[l * a.top + j]; }, lists, a.top, lds, 256);
  if (threadIdx.x < 64) write_top(a, sums, row, best, threadIdx.x);
}

// ---------------------------------------------------------------- gradients
//
// Reads the logits once and writes their gradient once; p_j = 2^(c (z_j - m))
// / S from the saved (m, 1/S).  The few elements with a gradient of their own
// (the target, the alternatives, the teacher's entries) are written again by
// the wave that has just written their chunk, while the lines are in the
// caches: at the end of the row instead, 64 entries a row cost 4096 x 131072
// bf16 8 % (450 us against 415).  Equal indices are added in list order first.
struct GradArgs {
  const void* z; int64_t s_row;
  int64_t N, V;
  float c, scale;
  int dt, mode;
  int nchunk, nblk;
  const float4* stat;
  void* dz; int64_t s_dz;
  // score: gradients of logprob, entropy (or null) and alternatives (or null)
  const int64_t* target; int64_t s_target; int64_t ignore;
  const float* glp; int64_t s_glp;
  const float* gent; int64_t s_gent;
  const float* gtop; int64_t s_gtop, s_gtop_k;
  const int64_t* top_index; int top;
  // distill: gradient of the loss
  const float* g; int64_t s_g;
  const float* q;
  const int64_t* entry; int64_t s_entry; int K;
};

struct GradRow {
  float c, m, inv, l2s;                  // p = 2^(c (z - m)) inv, ln p = ln2 (c (z - m) - l2s)
  float A, B;                            // dz = p (A + B log2 p)
};

template <bool ENT>
__device__ __forceinline__ float grad_elem(const GradRow& r, float z) {
  const float t = (z - r.m) * r.c;
  const float p = __builtin_amdgcn_exp2f(t) * r.inv;
  if constexpr (ENT) return p * fmaf(r.B, fmaxf(t - r.l2s, -2000.0f), r.A);
  else return p * r.A;
}

// A row of fewer than four chunks has a workgroup of as many waves: 1000000 x
// 64 bf16 685 us, with four waves 1813.
template <int DT, bool ENT>
__global__ __launch_bounds__(64 * WAVES) void k_score_grad(GradArgs a) {
  constexpr int VE = Elem<DT>::VE, NV = LANE_ELEMS / VE;
  // entries: index and gradient as given, then index (-1: none, or an equal
  // one before it) and gradient of all equal ones
  extern __shared__ __align__(16) int32_t lds_i[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // the first rows first: the forward pass reads past the caches and leaves no
  // rows there (the last first: 1024 x 32000 fp32 with its forward pass 67.4 us
  // against 65.9, 8192 x 32000 bf16 296 against 292)
  const int64_t row = blockIdx.x / a.nblk;
  const int part = static_cast<int>(blockIdx.x % a.nblk);
  const int n = a.mode == MODE_DISTILL ? a.K : 1 + a.top;
  float* const lds_w = reinterpret_cast<float*>(lds_i + n);
  int32_t* const own_i = lds_i + 2 * n;
  float* const own_w = reinterpret_cast<float*>(lds_i + 3 * n);

  const void* const zr = static_cast<const char*>(a.z) + row * a.s_row * Elem<DT>::BYTES;
  void* const dr = static_cast<char*>(a.dz) + row * a.s_dz * Elem<DT>::BYTES;
  const float4 st = a.stat[row];
  // the first chunk's loads are in flight while the entries are read
  const int waves = min(a.nchunk, WAVES), threads = 64 * waves, step = a.nblk * waves;
  float v[LANE_ELEMS];
  auto fetch = [&](int ch) {
    if (ch < a.nchunk) load_chunk<DT, false, false>(zr, static_cast<int64_t>(ch) * CHUNK, a.V, lane, v);
  };
  fetch(part * waves + wave);

  // an index outside [0, V) adds nothing
  constexpr int32_t LOST = -2;            // in the place of an index: q is NaN
  bool some = false;
  for (int e = threadIdx.x; e < n; e += threads) {
    int64_t i;
    float w;
    bool lost = false;
    if (a.mode == MODE_DISTILL) {
      i = a.entry[row * a.s_entry + e];
      w = a.q[row * a.K + e];
      lost = w != w;
      w = w > 0.0f ? -w * a.g[row * a.s_g] / a.scale : 0.0f;
    } else if (e == 0) {
      i = a.target != nullptr ? a.target[row * a.s_target] : -1;
      w = i == a.ignore || a.glp == nullptr ? 0.0f : a.glp[row * a.s_glp];
      if (i == a.ignore) i = -1;
    } else {
      i = a.top_index[row * a.top + e - 1];
      w = a.gtop != nullptr ? a.gtop[row * a.s_gtop + (e - 1) * a.s_gtop_k] : 0.0f;
    }
    const bool in = i >= 0 && i < a.V;
    lds_i[e] = lost ? LOST : in ? static_cast<int32_t>(i) : -1;
    lds_w[e] = in ? w : 0.0f;
    some |= in && w != 0.0f;
  }
  some = __syncthreads_or(some);
  const float ws = a.mode == MODE_DISTILL ? 1.0f : a.scale;
  // such a row has no gradient at all, whatever comes in (the log probability
  // -inf of its target easily makes that infinite or NaN)
  const bool empty = st.y == 0.0f;
  for (int e = threadIdx.x; e < n; e += threads) {
    const int i = lds_i[e];
    float w = 0.0f;
    bool first = i >= 0 && !empty;
    for (int k = 0; k < n; ++k) {
      if (lds_i[k] != i) continue;
      if (k < e) first = false;
      w += lds_w[k];
    }
    own_i[e] = first ? i : -1;
    own_w[e] = w * ws;
  }
  GradRow r;
  r.c = a.c;
  r.m = st.x; r.inv = st.y; r.l2s = st.z;
  if (a.mode == MODE_DISTILL) {
    // sum q = 1, or 0 for a row without entries, or all NaN (a teacher's NaN or
    // +inf): then so is the whole row's gradient, as its loss is
    r.A = lds_i[0] == LOST ? NAN : some && !empty ? a.g[row * a.s_g] / a.scale : 0.0f;
    r.B = 0.0f;
  } else {
    float G = 0.0f;
    for (int e = 0; e < n; ++e) G += lds_w[e];
    const float gent = a.gent != nullptr ? a.gent[row * a.s_gent] : 0.0f;
    r.A = empty ? 0.0f : -a.scale * (G + gent * st.w);
    r.B = empty ? 0.0f : -a.scale * gent * static_cast<float>(LN2);
  }
  __syncthreads();
  const int i_lane = lane < n ? own_i[lane] : -1;             // -1 is no chunk's
  const float w_lane = lane < n ? own_w[lane] : 0.0f;

  for (int ch = part * waves + wave; ch < a.nchunk; ch += step) {
    const int64_t base = static_cast<int64_t>(ch) * CHUNK;
#pragma unroll
    for (int j = 0; j < LANE_ELEMS; ++j) v[j] = grad_elem<ENT>(r, v[j]);
    if (base + CHUNK <= a.V) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        store_vec<DT, VE>(dr, base + (i * 64 + lane) * VE, reinterpret_cast<const float (&)[VE]>(v[i * VE]));
    } else {
      // a vector that was moved back from the row's end writes its first
      // elements a second time, with the same values; where they are the
      // chunk's before (another wave's, perhaps another workgroup's), only its own
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int64_t at = base + (i * 64 + lane) * VE, from = vector_start<DT>(at, a.V);
        if (at >= a.V) continue;
        if (from >= base && a.V >= VE) {
          store_vec<DT, VE>(dr, from, reinterpret_cast<const float (&)[VE]>(v[i * VE]));
        } else {
#pragma unroll
          for (int j = 0; j < VE; ++j)
            if (from + j >= at && from + j < a.V) store_elem<DT>(dr, from + j, v[i * VE + j]);
        }
      }
    }
    wave_sync();                          // the chunk's stores before its entries'
    auto again = [&](int i, float w) {
      if (i >> CHUNK_BITS == ch) store_elem<DT>(dr, i, grad_elem<ENT>(r, load_elem<DT>(zr, i)) + w);
    };
    again(i_lane, w_lane);
    for (int e = 64 + lane; e < n; e += 64) again(own_i[e], own_w[e]);
    fetch(ch + step);
  }
}

// ---------------------------------------------------------------- host side

// Four-wave workgroups per row.  One, which also finishes the row, when the
// rows alone give every CU about three workgroups, or when the row is so short
// that its four waves are through before a join would be.  Otherwise enough for
// four to a CU, at most one for every four chunks, and with alternatives at
// most 16 (64 lists to join).  Kernels alone, us, in one workgroup and shared:
//   rows   50257 fp32     131072 fp32    131072 bf16    50257 bf16, top 20
//   300    18.1  18.0     32.3  31.9     29.1  21.1     34.1  33.2
//   500    21.8  23.8     46.0  48.2     31.4  29.9     36.5  41.6
//   767    30.5  32.2     66.6  66.1     38.9  41.2     41.4  50.0
//   1000   37.2  39.7     83.9  83.8     48.2  52.4     46.0  55.9
// Of 1 .. 1000 rows of 5000 .. 131072 logits, fp32 and bf16, with 20
// alternatives and without, this rule and many_waves are within 11 % of the best of one,
// two or as many workgroups as here and of 16 waves, except at 1 and 16 x 50257
// fp32 (8.1 and 9.1 us, shared 6.6 and 7.3), 256 rows and less of 5000 with
// alternatives (14, 16 waves 12), 500 x 131072 bf16 top 20 (59, two workgroups
// 50), 300 x 50257 fp32 top 20 (35, two 31), 384 x 131072 fp32 top 20 (61, two
// 54) and 128 x 131072 bf16 (14.6, shared by 16 12.8).
constexpr int SHARED_MAX = 16;
int blocks_per_row(int64_t N, int64_t nchunk, int top) {
  const int64_t turns = ceil_div(nchunk, WAVES);              // chunks a wave of one workgroup takes
  int64_t b = 1;
  if (N < 768 && turns > (N >= 384 ? 8 : top > 0 ? 2 : 4)) b = std::min(turns, ceil_div(1024, N > 0 ? N : 1));
  if (top > 0) b = std::min<int64_t>(b, SHARED_MAX);
  if (nchunk > LDS_PARTS && b == 1) b = 2;                    // the sums go through the workspace
  return static_cast<int>(b);
}
// of the gradient, which has nothing to join
int grad_blocks_per_row(int64_t N, int64_t nchunk) {
  return static_cast<int>(N < 768 ? std::min(ceil_div(nchunk, WAVES), ceil_div(1024, N > 0 ? N : 1)) : 1);
}

// One workgroup of 16 waves to a row instead, in one launch, for rows of more
// than four chunks that they pass in at most two turns: 1 x 32000 fp32 6.7 us
// (one workgroup of four waves 9.0, several and a join 6.4), 200 x 17000 7.0
// (8.9, 9.5).  The second launch also costs the host: 1 x 50257, called and not
// replayed from a graph, 7.9 against 10.3.  With alternatives, whose search
// keeps a CU's four SIMDs busy, in one turn (64 x 17000 bf16 top 20 16.3, 21.3,
// 17.0; 64 x 50257 20.5 against 19.4 shared).  From 128 rows on, in up to eight
// turns: the other CUs have rows of their own (200 x 131072 fp32 22.5, 29.9,
// 24.2).
constexpr int MANY = 16;
bool many_waves(int64_t N, int64_t nchunk, int top) {
  return N <= 256 && nchunk > WAVES && nchunk <= (N >= 128 ? 8 * MANY : top > 0 ? MANY : 2 * MANY);
}

int64_t score_ws_bytes(int64_t N, int64_t V, int top) {
  const int64_t nchunk = ceil_div(V, CHUNK);
  if (many_waves(N, nchunk, top)) return 0;
  const int nblk = blocks_per_row(N, nchunk, top);
  if (nblk == 1) return 0;
  return N * (nblk * WAVES * static_cast<int64_t>(top) * 8 + nchunk * 12);
}

det_status check_logits(int dt, const void* z, int64_t N, int64_t V, int64_t s_row, double scale) {
  if (!known_dtype(dt)) return fail(DET_EDTYPE, "unknown dtype %d", dt);
  if (N < 0 || V < 1 || s_row < 0) return fail(DET_EINVAL, "bad size or stride: N=%lld V=%lld stride=%lld",
                                              (long long)N, (long long)V, (long long)s_row);
  if (V > DET_HEAD_V_MAX) return fail(DET_EINVAL, "V = %lld exceeds the limit 2^24", (long long)V);
  if (N > DET_ROWS_MAX) return fail(DET_EINVAL, "N = %lld exceeds the limit 2^22 rows per call", (long long)N);
  if (!(scale > 0.0) || !(scale < 1e6) || scale < 1e-6) return fail(DET_EINVAL, "the scale must lie in [1e-6, 1e6)");
  if (N == 0) return DET_OK;
  if (z == nullptr) return fail(DET_EINVAL, "null logits");
  if (!aligned_for(z, dt)) return fail(DET_EINVAL, "logits must be aligned to their element size");
  return DET_OK;
}

det_status launch_score(ScoreArgs a, void* ws, size_t ws_bytes, hipStream_t s) {
  a.nchunk = static_cast<int>(ceil_div(a.V, CHUNK));
  const bool many = many_waves(a.N, a.nchunk, a.top);
  a.nblk = many ? 1 : blocks_per_row(a.N, a.nchunk, a.top);
  a.wpr = many ? MANY : a.nchunk >= WAVES ? WAVES : a.nchunk;
  if (a.wpr == 3) a.wpr = 4;
  a.status = det_device_status_word();
  if (a.status == nullptr) return DET_EHIP;
  if (a.nblk > 1) {
    a.wpr = WAVES;
    const int64_t need = score_ws_bytes(a.N, a.V, a.top);
    if (ws == nullptr || !aligned8(ws) || ws_bytes < static_cast<size_t>(need))
      return fail(DET_EINVAL, "workspace: %lld bytes, 8-byte aligned, are needed", (long long)need);
    a.lists = static_cast<uint64_t*>(ws);
    a.parts = reinterpret_cast<float*>(a.lists + a.N * a.nblk * WAVES * a.top);
  }
  const int nw = many ? MANY : WAVES, rpb = nw / a.wpr;
  const int64_t blocks = a.nblk > 1 ? a.N * a.nblk : ceil_div(a.N, rpb);
  const size_t lds = (a.top > 0 ? nw * ((many ? sizeof(TopLds<MANY>) : sizeof(TopLds<WAVES>)) + TOP_MAX * 8) : 0) +
                     (a.nblk > 1 ? 0 : static_cast<size_t>(rpb) * a.nchunk * 12);
  const dim3 grid(static_cast<unsigned>(blocks)), block(64 * nw);
  auto launch = [&](auto dt, auto top) {
    constexpr int DT = decltype(dt)::value;
    constexpr bool TOP = decltype(top)::value;
    if (many) hipLaunchKernelGGL((k_score<DT, TOP, MANY>), grid, block, lds, s, a);
    else hipLaunchKernelGGL((k_score<DT, TOP, WAVES>), grid, block, lds, s, a);
  };
  auto by_top = [&](auto dt) {
    if (a.top > 0) launch(dt, std::true_type{});
    else launch(dt, std::false_type{});
  };
  if (a.dt == DET_F32) by_top(std::integral_constant<int, DET_F32>{});
  else by_top(std::integral_constant<int, DET_BF16>{});
  det_status st = hip_check(hipGetLastError(), "score launch");
  if (st != DET_OK || a.nblk == 1) return st;
  const size_t jl = a.top > 0 ? (TOP_MAX + static_cast<size_t>(a.nblk) * WAVES * a.top + 16) * 8 : 0;
  hipLaunchKernelGGL(k_score_join, dim3(static_cast<unsigned>(a.N)), dim3(256), jl, s, a);
  return hip_check(hipGetLastError(), "score join launch");
}

det_status launch_grad(GradArgs a, hipStream_t s) {
  a.nchunk = static_cast<int>(ceil_div(a.V, CHUNK));
  a.nblk = grad_blocks_per_row(a.N, a.nchunk);
  const int n = a.mode == MODE_DISTILL ? a.K : 1 + a.top;
  const dim3 grid(static_cast<unsigned>(a.N * a.nblk)), block(64 * std::min(a.nchunk, WAVES));
  const size_t lds = static_cast<size_t>(n) * 16;
  const bool ent = a.gent != nullptr;
  if (a.dt == DET_F32) {
    if (ent) hipLaunchKernelGGL((k_score_grad<DET_F32, true>), grid, block, lds, s, a);
    else hipLaunchKernelGGL((k_score_grad<DET_F32, false>), grid, block, lds, s, a);
  } else {
    if (ent) hipLaunchKernelGGL((k_score_grad<DET_BF16, true>), grid, block, lds, s, a);
    else hipLaunchKernelGGL((k_score_grad<DET_BF16, false>), grid, block, lds, s, a);
  }
  return hip_check(hipGetLastError(), "gradient launch");
}

}  // namespace

extern "C" {

int64_t det_head_workspace_bytes(int64_t N, int64_t V, int top) {
  if (N <= 0 || V <= 0 || top < 0 || N > DET_ROWS_MAX || V > DET_HEAD_V_MAX || top > TOP_MAX) return 0;
  return score_ws_bytes(N, V, top);
}

det_status det_token_logprobs(det_dtype dt, const void* z, int64_t s_row, int64_t N, int64_t V, double scale,
                              const int64_t* target, int64_t s_target, int64_t ignore, int top, float* logprob,
                              float* entropy, float* stat, int64_t* top_index, float* top_logprob, void* workspace,
                              size_t workspace_bytes, void* stream) {
  det_status st = check_logits(dt, z, N, V, s_row, scale);
  if (st != DET_OK) return st;
  if (top < 0 || top > TOP_MAX || top > V)
    return fail(DET_EINVAL, "top = %d must lie in 0..min(%d, V)", top, TOP_MAX);
  if (s_target < 0) return fail(DET_EINVAL, "negative target stride");
  if (N == 0) return DET_OK;
  if (stat == nullptr || (target != nullptr && logprob == nullptr) ||
      (top > 0 && (top_index == nullptr || top_logprob == nullptr)))
    return fail(DET_EINVAL, "null output");
  if (!aligned8(target) || !aligned8(top_index) || (reinterpret_cast<uintptr_t>(stat) & 15u) ||
      ((reinterpret_cast<uintptr_t>(logprob) | reinterpret_cast<uintptr_t>(entropy) |
        reinterpret_cast<uintptr_t>(top_logprob)) & 3u))
    return fail(DET_EINVAL, "misaligned target or output");
  ScoreArgs a{};
  a.z = z; a.s_row = s_row; a.N = N; a.V = V; a.dt = dt; a.mode = MODE_SCORE;
  a.scale = scale; a.c = static_cast<float>(scale * LOG2E);
  a.top = top;
  a.target = target; a.s_target = s_target; a.ignore = ignore;
  a.logprob = logprob; a.entropy = entropy; a.stat = reinterpret_cast<float4*>(stat);
  a.top_index = top_index; a.top_value = top_logprob;
  return launch_score(a, workspace, workspace_bytes, static_cast<hipStream_t>(stream));
}

det_status det_token_logprobs_grad(det_dtype dt, const void* z, int64_t s_row, int64_t N, int64_t V, double scale,
                                   const int64_t* target, int64_t s_target, int64_t ignore, int top,
                                   const int64_t* top_index, const float* stat, const float* g_logprob,
                                   int64_t s_g_logprob, const float* g_entropy, int64_t s_g_entropy,
                                   const float* g_top, int64_t s_g_top, int64_t s_g_top_k, void* dz, int64_t s_dz,
                                   void* stream) {
  det_status st = check_logits(dt, z, N, V, s_row, scale);
  if (st != DET_OK) return st;
  if (top < 0 || top > TOP_MAX || top > V)
    return fail(DET_EINVAL, "top = %d must lie in 0..min(%d, V)", top, TOP_MAX);
  if (s_target < 0 || s_g_logprob < 0 || s_g_entropy < 0 || s_g_top < 0 || s_g_top_k < 0 || s_dz < V)
    return fail(DET_EINVAL, "negative stride, or gradient rows that overlap");
  if (N == 0) return DET_OK;
  if (stat == nullptr || dz == nullptr || (g_logprob != nullptr && target == nullptr) ||
      (top > 0 && top_index == nullptr))
    return fail(DET_EINVAL, "null pointer");
  if (!aligned_for(dz, dt) || !aligned8(target) || !aligned8(top_index) || (reinterpret_cast<uintptr_t>(stat) & 15u) ||
      ((reinterpret_cast<uintptr_t>(g_logprob) | reinterpret_cast<uintptr_t>(g_entropy) |
        reinterpret_cast<uintptr_t>(g_top)) & 3u))
    return fail(DET_EINVAL, "misaligned pointer");
  GradArgs a{};
  a.z = z; a.s_row = s_row; a.N = N; a.V = V; a.dt = dt; a.mode = MODE_SCORE;
  a.scale = static_cast<float>(scale); a.c = static_cast<float>(scale * LOG2E);
  a.stat = reinterpret_cast<const float4*>(stat); a.dz = dz; a.s_dz = s_dz;
  a.target = target; a.s_target = s_target; a.ignore = ignore;
  a.glp = g_logprob; a.s_glp = s_g_logprob;
  a.gent = g_entropy; a.s_gent = s_g_entropy;
  a.gtop = g_top; a.s_gtop = s_g_top; a.s_gtop_k = s_g_top_k;
  a.top_index = top_index; a.top = g_top != nullptr ? top : 0;
  return launch_grad(a, static_cast<hipStream_t>(stream));
}

det_status det_distill(det_dtype dt, const void* z, int64_t s_row, int64_t N, int64_t V, double temperature,
                       det_dtype teacher_dt, const void* teacher, int64_t s_teacher, const int64_t* entry,
                       int64_t s_entry, int64_t K, float* loss, float* stat, float* q, void* workspace,
                       size_t workspace_bytes, void* stream) {
  if (!(temperature > 0.0)) return fail(DET_EINVAL, "the temperature must be positive");
  det_status st = check_logits(dt, z, N, V, s_row, 1.0 / temperature);
  if (st != DET_OK) return st;
  if (!known_dtype(teacher_dt)) return fail(DET_EDTYPE, "unknown teacher dtype %d", static_cast<int>(teacher_dt));
  if (K < 1 || K > DET_HEAD_ENTRIES_MAX) return fail(DET_EINVAL, "K = %lld must lie in 1..%d", (long long)K, DET_HEAD_ENTRIES_MAX);
  if (s_teacher < 0 || s_entry < 0) return fail(DET_EINVAL, "negative stride");
  if (N == 0) return DET_OK;
  if (teacher == nullptr || entry == nullptr || loss == nullptr || stat == nullptr || q == nullptr)
    return fail(DET_EINVAL, "null pointer");
  if (!aligned_for(teacher, teacher_dt) || !aligned8(entry) || (reinterpret_cast<uintptr_t>(stat) & 15u) ||
      ((reinterpret_cast<uintptr_t>(loss) | reinterpret_cast<uintptr_t>(q)) & 3u))
    return fail(DET_EINVAL, "misaligned pointer");
  ScoreArgs a{};
  a.z = z; a.s_row = s_row; a.N = N; a.V = V; a.dt = dt; a.mode = MODE_DISTILL;
  a.scale = 1.0 / temperature; a.c = static_cast<float>(a.scale * LOG2E);
  a.teacher = teacher; a.s_teacher = s_teacher; a.tdt = teacher_dt;
  a.entry = entry; a.s_entry = s_entry; a.K = static_cast<int>(K);
  a.loss = loss; a.stat = reinterpret_cast<float4*>(stat); a.q = q;
  return launch_score(a, workspace, workspace_bytes, static_cast<hipStream_t>(stream));
}

det_status det_distill_grad(det_dtype dt, const void* z, int64_t s_row, int64_t N, int64_t V, double temperature,
                            const int64_t* entry, int64_t s_entry, int64_t K, const float* stat, const float* q,
                            const float* g, int64_t s_g, void* dz, int64_t s_dz, void* stream) {
  if (!(temperature > 0.0)) return fail(DET_EINVAL, "the temperature must be positive");
  det_status st = check_logits(dt, z, N, V, s_row, 1.0 / temperature);
  if (st != DET_OK) return st;
  if (K < 1 || K > DET_HEAD_ENTRIES_MAX) return fail(DET_EINVAL, "K = %lld must lie in 1..%d", (long long)K, DET_HEAD_ENTRIES_MAX);
  if (s_entry < 0 || s_g < 0 || s_dz < V) return fail(DET_EINVAL, "negative stride, or gradient rows that overlap");
  if (N == 0) return DET_OK;
  if (entry == nullptr || stat == nullptr || q == nullptr || g == nullptr || dz == nullptr)
    return fail(DET_EINVAL, "null pointer");
  if (!aligned_for(dz, dt) || !aligned8(entry) || (reinterpret_cast<uintptr_t>(stat) & 15u) ||
      ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(g)) & 3u))
    return fail(DET_EINVAL, "misaligned pointer");
  GradArgs a{};
  a.z = z; a.s_row = s_row; a.N = N; a.V = V; a.dt = dt; a.mode = MODE_DISTILL;
  a.scale = static_cast<float>(1.0 / temperature); a.c = static_cast<float>(LOG2E / temperature);
  a.stat = reinterpret_cast<const float4*>(stat); a.dz = dz; a.s_dz = s_dz;
  a.entry = entry; a.s_entry = s_entry; a.K = static_cast<int>(K); a.q = q;
  a.g = g; a.s_g = s_g;
  return launch_grad(a, static_cast<hipStream_t>(stream));
}

}  // extern "C"
