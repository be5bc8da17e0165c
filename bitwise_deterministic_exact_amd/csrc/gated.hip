// The gated projection h = act(x Wg^T) * (x Wu^T) and its gradients for
// MI355X (gfx950).
//
//   g = x Wg^T,  u = x Wu^T,  h = act(g) u
//   dg = dh u act'(g),  du = dh act(g)
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x
//
// All products run on the matrix cores (v_mfma_f32_16x16x32_bf16).  Every
// output element is one chain of such instructions over its K in ascending
// steps of 32, whatever the tile, the launch or the number of rows: a token's
// h and dx have the same bits alone and in a batch of thousands.  K is never
// split between workgroups.
#include <algorithm>
#include <type_traits>

#include "elementary.h"
#include "int8_block.h"

// every fused multiply-add below is written as one: the compiler forms none
#pragma clang fp contract(off)

namespace {

using namespace rowops;

using bf16x8 = __bf16 __attribute__((ext_vector_type(8)));
using f32x4 = float __attribute__((ext_vector_type(4)));
using u32x4 = uint32_t __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------- activations

// s = 1 / (1 + e^-x) and 1 - s, neither from a difference
struct Sigmoid {
  float s, rest;
};
__device__ __forceinline__ Sigmoid sigmoid(float x) {
  const float e = exp_of(-fabsf(x)), r = __builtin_amdgcn_rcpf(1.0f + e), small = e * r;
  return x >= 0.0f ? Sigmoid{r, small} : Sigmoid{small, r};
}

// act(g) and act'(g); a NaN stays one by the factor g
struct Act {
  float a, d;
};
template <int ACT>
__device__ __forceinline__ Act act_of(float g) {
  if constexpr (ACT == DET_ACT_SILU) {
    const Sigmoid s = sigmoid(g);
    return {g * s.s, s.s * fmaf(g, s.rest, 1.0f)};
  } else if constexpr (ACT == DET_ACT_GELU_TANH) {
    // 0.5 g (1 + tanh t) = g sigmoid(2 t); from 1e4 on g^2 no longer matters, and inf would
    const float g2 = fminf(g * g, 1.0e4f), in = g * fmaf(0.0713548163f, g2, 1.59576912f);
    const Sigmoid s = sigmoid(in);
    const float slope = s.s * s.rest * fmaf(0.214064449f, g2, 1.59576912f);
    return {g * s.s, fmaf(g, slope, s.s)};
  } else {
    // Phi(-|g|) = e^(-g^2 / 2) E / 2 with E = erfcx(|g| / sqrt 2) = t p(t), t = 1 / (1 + |g| / sqrt 8):
    // p of degree 8 is fitted to E / t for |g| up to 14.7, off by 5.9e-8 of it at most; with the roundings
    // Phi is within 4 units.  The square is carried in two parts, as a rounded one costs g^2 / 2 half
    // units; from 20 on e^(-g^2 / 2) is 0.  (By erfcf, and e^(-g^2 / 2) beside it, 2048 x 1024 x 2816 forward
    // took 41 us, 35.5 so, and dx with dg and du 52.5, 46.5.)
    const float w = fminf(fabsf(g), 20.0f), s = w * w, e0 = exp_of(-0.5f * s);
    const float e = fmaf(e0, -0.5f * fmaf(w, w, -s), e0), t = __builtin_amdgcn_rcpf(fmaf(w, 0.353553391f, 1.0f));
    const float c[8] = {0.142540082f, -0.24412401f, 0.139634386f, -0.0137276426f,
                        0.101519361f, 0.121507309f, 0.141193792f, 0.141042858f};
    float p = -0.0295861568f;
#pragma unroll
    for (int k = 0; k < 8; ++k) p = fmaf(p, t, c[k]);
    const float q = t * p * e, cdf = g > 0.0f ? 1.0f - q : q;
    return {g * cdf, fmaf(g, 0.398942292f * e, cdf)};
  }
}

// h = act(g) u; the activation is a run-time choice, uniform over the launch
__device__ __forceinline__ void act_times(int act, const float (&g)[4], const float (&u)[4], float (&h)[4]) {
  if (act == DET_ACT_SILU) {
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = act_of<DET_ACT_SILU>(g[k]).a * u[k];
  } else if (act == DET_ACT_GELU_TANH) {
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = act_of<DET_ACT_GELU_TANH>(g[k]).a * u[k];
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = act_of<DET_ACT_GELU>(g[k]).a * u[k];
  }
}

// ---------------------------------------------------------------- the matrix product
//
// D[b][a] = sum_k A[k, a] B[k, b].  An operand lies with adjacent k (rows of A
// or B, "by row") or with adjacent a or b (rows of k, "by k"): the gradients read
// x, the weights, dg and du as they lie, with no transposed copy.
//
// A workgroup of WA x WB waves owns TA x TB outputs, a wave FA x FB blocks of 16
// x 16.  A ring of BUFS stages of KS k (32, 64 or 128) in LDS is filled with
// 16-byte copies that need no registers, BUFS - 1 stages ahead; while the MFMAs of
// 32 k run (128 where KS is; one per block and 32), the next ones' fragments are
// read.  One barrier per stage.
//
// By row: KS k per row, whose 16-byte pieces lie in the order piece ^ swap_row(row).
// A fragment is one 16-byte read; the 16 lanes that the LDS serves at once (0-3,
// 12-15, 20-23, 24-27 and so on) then hit every bank once: no conflicts are counted.
// By k: T elements per row of k; a fragment's 16 columns are 32 bytes of 8 rows
// per lane group, read by two transposing reads of 4 rows each (16 lanes give
// the addresses of 4 x 16 elements and get 4 of a column each).  The 32-byte
// pieces lie in the order piece ^ swap(k), again without conflicts.
//
// What bounds it is power.  8192 x 4096 x 11008 forward takes 1165-1190 us (1.25
// PFLOP/s), 917 where x and the weights are zeros; the clock is at 2.0 GHz forward
// and 1.8 in the gradients, whose matrix cores are busy 70 to 74 % of the time.
// torch's product of x and both weights takes 1144-1174 us alone.  Waves of 128 x
// 128 (four to a workgroup, a third fewer LDS reads) took 1.2 to 3 times as long.
struct Operand {
  const void* p; int64_t stride;          // elements between rows (of k, or of a or b)
  int64_t n;                              // its a or b
};
struct MmArgs {
  // a second operand A1 of the same size: the gate's rows are A's, the up
  // projection's A1's (gated); or k goes over A and then, from `turn` on, over A1
  Operand A, A1, B;
  int64_t K;                              // a multiple of 64 (dx: 256): what lies past the rows of k is 0
  int64_t ka, kb, turn;                   // by k: rows of k of A (and of A1), of B
  int64_t begin_a, begin_b, tiles_a, tiles_b;                // this launch's tiles
  // gated: h [n of B][n of A]; else D, rows [0, split0) in out, [split1, split1 + split0) in out1
  void* out; void* out1; int64_t split0, split1;
  // what the gradients read again
  void* gate; void* up; int64_t s_kept;
  int8_t* gate_exp; int8_t* up_exp;
  int32_t* status;                        // int8: noted where a block is not finite
  int dt, act, save;                      // type of out, activation, what gate and up hold
};

// s_waitcnt with vmcnt(n) and lgkmcnt(m) (gfx9 encoding)
constexpr int waitcnt(int vm, int lgkm) { return (vm & 15) | ((vm >> 4) << 14) | (7 << 4) | (lgkm << 8); }

// Workgroup barrier without the fence of __syncthreads, which would wait for
// every copy in flight: the callers wait for what they need.
__device__ __forceinline__ void step_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Tiles in ranges, one per XCD (workgroups go to the XCDs in turn), and in
// groups of 8 rows of tiles within: the 32 workgroups that are resident on an
// XCD cover about 8 x 4 tiles and share their operands in its L2.
__device__ __forceinline__ void tile_of(int64_t id, int64_t tiles_a, int64_t tiles_b, int64_t& ta, int64_t& tb) {
  const int64_t total = tiles_a * tiles_b, per = total >> 3, rem = total & 7, xcd = id & 7;
  const int64_t t = xcd * per + min(xcd, rem) + (id >> 3);
  const int64_t grp = t / (8 * tiles_a), rows = min<int64_t>(8, tiles_b - 8 * grp), in = t - grp * 8 * tiles_a;
  tb = 8 * grp + in % rows;
  ta = in / rows;
}

#ifdef __HIP_DEVICE_COMPILE__              // buffer descriptors are a type of the device's alone
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, static_cast<int>(bytes), 0x00020000);
}
using s16x4 = short __attribute__((ext_vector_type(4)));
using lds_s16x4 = __attribute__((address_space(3))) s16x4;

// One operand's share of a step: T of its a or b, copied by NW waves, read as
// fragments of 16.
template <bool BY_K, int T, int NW, int KS>
struct Tile {
  static_assert(T * KS % (512 * NW) == 0, "every wave copies as much");
  static constexpr int COPIES = T * KS / 512 / NW;            // of 1 KiB, per wave and stage
  static constexpr int BYTES = T * KS * 2;
  static constexpr int ROWS = 512 / KS, PIECES = KS / 8;      // by row: rows of a copy, pieces of 16 bytes in one
  static constexpr int LINE = T / 8;                          // by k: pieces of 16 bytes in a row of k
  // which 32-byte piece of a row of k lies where; 8 rows that are read at once differ in it
  static __device__ __forceinline__ int swap(int k) {
    const int s = (k & 3) | ((k >> 1) & 4);
    return T >= 128 ? s : ((k >> 1) & 1) | ((k >> 2) & 2);
  }
  // by row: what a row's pieces are swapped with
  static __device__ __forceinline__ int swap_row(int r) { return KS >= 64 ? r & (PIECES - 1) : -(r >> 2) & 3; }
  int64_t stride;                         // bytes
  const char* next;                       // by row: the tile; by k: the next stage's first row
  int at, end, bytes;                     // by row: bytes of k before the next stage, of a row, of the tile
  int left, cols;                         // by k: rows from `next` on, bytes of a row
  int from[COPIES];                       // by row: rows past the end are the last one again
  // `limit` of its a or b from `first` on are the tile's
  __device__ __forceinline__ void init(const Operand& o, int64_t first, int limit, int64_t K, int64_t rows, int wave,
                                       int lane) {
    stride = o.stride * 2;
    const int n = static_cast<int>(min<int64_t>(limit, o.n - first));
    if constexpr (BY_K) {
      next = static_cast<const char*>(o.p) + first * 2;
      left = static_cast<int>(rows);
      cols = (n * 2 + 15) & ~15;          // whole pieces: strides are multiples of 16 bytes
#pragma unroll
      for (int j = 0; j < COPIES; ++j) {
        const int at = (wave * COPIES + j) * 64 + lane, k = at / LINE, slot = at % LINE;
        const int piece = (((slot >> 1) ^ swap(k)) << 1) | (slot & 1);
        // columns past the end: the last ones
        from[j] = k * static_cast<int>(stride) + min(piece, cols / 16 - 1) * 16;
      }
    } else {
      next = static_cast<const char*>(o.p) + first * stride;
      at = 0;
      end = static_cast<int>(K * 2);
      bytes = (n - 1) * static_cast<int>(stride) + end;
#pragma unroll
      for (int j = 0; j < COPIES; ++j) {
        const int r = (wave * COPIES + j) * ROWS + lane / PIECES;
        from[j] = min(r, n - 1) * static_cast<int>(stride) + (((lane % PIECES) ^ swap_row(r)) * 16);
      }
    }
  }
  // The next stage into LDS at `to`; stages past the last one, which no MFMA
  // takes, read nothing and get 0.  By k: rows past the end lie past the end of the
  // buffer and come as 0.
  __device__ __forceinline__ void copy(char* to, int wave) {
    if constexpr (BY_K) {
      // No branch: one would keep the copies from going between the MFMAs.  Without
      // rows the bytes are at most cols - stride <= 0, and the product fits 32 bits: A is
      // at most 511 rows past its end (in dx 127 up to Fp and then (BUFS - 1) KS <= 384; in
      // dw it starts anew at K), of up to 2^22 bytes each; B, dg and du in dw, at most 255
      // + 384, of 4 Fp <= 2^18 bytes.
      const __amdgpu_buffer_rsrc_t b = buffer_of(next, max(0, (min(left, KS) - 1) * static_cast<int>(stride) + cols));
#pragma unroll
      for (int j = 0; j < COPIES; ++j)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(b, to + (wave * COPIES + j) * 1024, 16, from[j], 0, 0, 0);
      next += KS * stride;
      left -= KS;
    } else {
      const __amdgpu_buffer_rsrc_t b = buffer_of(next, at < end ? bytes : 0);
#pragma unroll
      for (int j = 0; j < COPIES; ++j)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(b, to + (wave * COPIES + j) * 1024, 16, from[j], at, 0, 0);
      at += KS * 2;
    }
  }
  // a lane's address of fragment 0, and the fragment that starts at a or b = 16 f
  static __device__ __forceinline__ int lane_at(int lane) {
    const int i = lane & 15, q = lane >> 4;
    if constexpr (BY_K) return (8 * q + (i >> 2)) * T * 2 + swap(8 * q + (i >> 2)) * 32 + (i & 3) * 8;
    else return i * KS * 2 + ((q ^ swap_row(i)) * 16);
  }
  static __device__ __forceinline__ bf16x8 fragment(const char* __restrict__ tile, int at, int f, int half) {
    if constexpr (BY_K) {
      // a row of k is a power of two: the bits do not meet
      const char* const p = tile + half * 32 * T * 2 + (at ^ (f * 32));
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * T * 2));
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      return *reinterpret_cast<const bf16x8*>(tile + (at ^ (half * 64)) + f * 16 * KS * 2);
    }
  }
};
#endif

template <bool GATED, bool A_BY_K, bool B_BY_K, int WA, int WB, int FA, int FB, int KS, int BUFS, bool SPREAD>
__global__ __launch_bounds__(64 * WA * WB, 2) void k_mm(MmArgs a) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int NW = WA * WB, TA = WA * FA * 16, TB = WB * FB * 16, TH = GATED ? TA / 2 : TA;
  using TileA = Tile<A_BY_K, TA, NW, KS>;
  using TileB = Tile<B_BY_K, TB, NW, KS>;
  static_assert((BUFS - 1) * KS <= 384, "stages past the last one: how far TileA and TileB run past their rows");
  constexpr int BUF = TileA::BYTES + TileB::BYTES, COPIES = TileA::COPIES + TileB::COPIES;
  __shared__ __attribute__((aligned(1024))) char lds[BUFS * BUF];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wa = wave / WB, wb = wave % WB;
  int64_t ta, tb;
  tile_of(blockIdx.x, a.tiles_a, a.tiles_b, ta, tb);
  const int64_t row_a = a.begin_a + ta * TH, row_b = a.begin_b + tb * TB;

  TileA A;
  TileB B;
  B.init(a.B, row_b, TB, a.K, a.kb, wave, lane);
  if constexpr (GATED) {
    // the tile's first half is the gate's, its second the up projection's: each wave copies rows of one of them
    static_assert(!A_BY_K && TH % (TileA::ROWS * TileA::COPIES) == 0, "a wave's copies lie in one half");
    constexpr int HALF = NW / 2;
    A.init(wave < HALF ? a.A : a.A1, row_a, TH, a.K, 0, wave % HALF, lane);
  } else {
    A.init(a.A, row_a, TA, a.K, a.ka, wave, lane);
  }
  const int stages = static_cast<int>(a.K / KS);
  int turn_at = static_cast<int>(a.turn / KS);                // stages until A1 follows
  const char* const second = static_cast<const char*>(a.A1.p) + row_a * 2;
  // the next stage of both operands
  auto copy = [&](int buf) {
    char* const to = lds + buf * BUF;
    if constexpr (A_BY_K) {
      const bool now = turn_at == 0;
      A.next = now ? second : A.next;
      A.left = now ? static_cast<int>(a.ka) : A.left;
      --turn_at;
    }
    A.copy(to, wave);
    B.copy(to + TileA::BYTES, wave);
  };
  // the first row of A's tile of fragment i of this wave
  auto frag_row = [&](int i) {
    if constexpr (GATED) return (i < FA / 2 ? 0 : TH) + wa * FA * 8 + (i % (FA / 2)) * 16;
    else return (wa * FA + i) * 16;
  };
  const int at_a = TileA::lane_at(lane), at_b = TileB::lane_at(lane);
  // fragments of SET x 32 k: of a whole stage, or of one of its halves
  constexpr int SET = KS == 64 ? 1 : KS / 32;
  struct Frags {
    bf16x8 fa[SET][FA], fb[SET][FB];
  };
  auto read = [&](Frags& f, int buf, int half) {
    const char* const tile = lds + buf * BUF;
#pragma unroll
    for (int h = 0; h < SET; ++h) {
#pragma unroll
      for (int j = 0; j < FB; ++j) f.fb[h][j] = TileB::fragment(tile + TileA::BYTES, at_b, wb * FB + j, half + h);
#pragma unroll
      for (int i = 0; i < FA; ++i) f.fa[h][i] = TileA::fragment(tile, at_a, frag_row(i) / 16, half + h);
    }
  };
  f32x4 acc[FA][FB];
#pragma unroll
  for (int i = 0; i < FA; ++i)
#pragma unroll
    for (int j = 0; j < FB; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  auto multiply = [&](const Frags& f) {
#pragma unroll
    for (int h = 0; h < SET; ++h)
#pragma unroll
      for (int i = 0; i < FA; ++i)
#pragma unroll
        for (int j = 0; j < FB; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.fa[h][i], f.fb[h][j], acc[i][j], 0, 0, 0);
  };

  Frags f0, f1;
#pragma unroll
  for (int s = 0; s < BUFS; ++s) copy(s);
  __builtin_amdgcn_s_waitcnt(waitcnt((BUFS - 1) * COPIES, 15));
  step_barrier();
  read(f0, 0, 0);
  // SPREAD: the reads and copies go between the MFMAs.  Else they go before them:
  // then one of a SIMD's two waves reads while the other multiplies.
  constexpr int MFMAS = SET * FA * FB, READS = SET * (FA * (A_BY_K ? 2 : 1) + FB * (B_BY_K ? 2 : 1));
  auto run = [&](const Frags& now, auto copies) {
    if constexpr (SPREAD) {
      constexpr int C = decltype(copies)::value, PER = MFMAS - C > READS ? (MFMAS - C) / READS : 1;
      multiply(now);
#pragma unroll
      for (int r = 0; r < READS; ++r) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);    // a read of the LDS
        __builtin_amdgcn_sched_group_barrier(0x008, PER, 0);  // MFMAs
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);    // a copy, behind the reads: both are LDS accesses
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      }
    } else {
      __builtin_amdgcn_sched_barrier(0);
      multiply(now);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  int buf = 0;                            // of the stage whose last MFMAs run
  // the last MFMAs of a stage, while the next one's first fragments are read
  auto turn = [&](const Frags& now, Frags& then) {
    // this wave's reads of the stage are done and its copies of the next one have landed; then every wave's
    __builtin_amdgcn_s_waitcnt(waitcnt((BUFS - 2) * COPIES, 0));
    step_barrier();
    const int next = buf + 1 == BUFS ? 0 : buf + 1;
    __builtin_amdgcn_sched_barrier(0);
    read(then, next, 0);                  // after the last stage: not used
    copy(buf);
    run(now, std::integral_constant<int, COPIES>{});
    buf = next;
  };
  if constexpr (SET == KS / 32) {
    for (int s = 0; s < stages; s += 2) { // K is a multiple of two stages
      turn(f0, f1);
      turn(f1, f0);
    }
  } else {
    for (int s = 0; s < stages; ++s) {
      __builtin_amdgcn_sched_barrier(0);
      read(f1, buf, 1);
      run(f0, std::integral_constant<int, 0>{});
      turn(f1, f0);
    }
  }
  __builtin_amdgcn_s_waitcnt(waitcnt(0, 0));                  // no copy or read of these buffers is left
  step_barrier();

  // The sums go through LDS, 16 rows of the output at a time and each wave
  // by itself, so that a row is written in whole lines.  Lane l holds features
  // 4 (l / 16) .. + 3 of a block, of row l % 16.
  constexpr int ROW = FA * 16 + 4;        // floats; 4 more, or all rows would start in one bank
  static_assert(NW * 16 * ROW * 4 <= BUFS * BUF, "the rows lie in the ring's room");
  float* const own = reinterpret_cast<float*>(lds) + wave * 16 * ROW;
  bool noted = false;                     // a block of codes that is not finite
#pragma unroll
  for (int j = 0; j < FB; ++j) {
    wave_sync();
#pragma unroll
    for (int i = 0; i < FA; ++i)
      *reinterpret_cast<f32x4*>(own + (lane & 15) * ROW + i * 16 + 4 * (lane >> 4)) = acc[i][j];
    wave_sync();
    constexpr int LANES = (GATED ? FA / 2 : FA) * 4;           // lanes to a row
    const int64_t c = row_a + wa * (LANES * 4) + (lane % LANES) * 4;
    const int64_t na = a.A.n;
    const int n = static_cast<int>(min<int64_t>(4, na - c));
#pragma unroll 1
    for (int r0 = 0; r0 < 16; r0 += 64 / LANES) {
      const int r = r0 + lane / LANES;
      const int64_t b = row_b + (wb * FB + j) * 16 + r;
      const int in = b < a.B.n ? n : 0;
      const float* const from = own + r * ROW + (lane % LANES) * 4;
      const f32x4 first = *reinterpret_cast<const f32x4*>(from);
      if constexpr (!GATED) {
        const float v[4] = {first[0], first[1], first[2], first[3]};
        const bool hi = b >= a.split1;
        const int64_t row = hi ? b - a.split1 : b;
        store4(a.dt, hi ? a.out1 : a.out, row * na + c, v, row < a.split0 ? in : 0);
      } else {
        const f32x4 upper = *reinterpret_cast<const f32x4*>(from + FA * 8);
        const float g[4] = {first[0], first[1], first[2], first[3]}, u[4] = {upper[0], upper[1], upper[2], upper[3]};
        float h[4];
        act_times(a.act, g, u, h);
        store4(a.dt, a.out, b * na + c, h, in);
        if (a.save != DET_SAVE_NONE) {
          // 8 lanes hold a block of 32 features; those past the end count as 0
          const bool int8 = a.save == DET_SAVE_INT8;
          uint32_t tg = 0u, tu = 0u;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k < n) {
              tg = max(tg, int8 ? magnitude(g[k]) : finite_magnitude(g[k]));
              tu = max(tu, int8 ? magnitude(u[k]) : finite_magnitude(u[k]));
            }
          tg = top_of_8(tg);
          tu = top_of_8(tu);
          const bool bad_g = not_finite(tg), bad_u = not_finite(tu);        // int8 alone
          noted |= in > 0 && (bad_g || bad_u);
          const int eg = int8 ? block_exponent(tg) : half_exponent(tg), eu = int8 ? block_exponent(tu) : half_exponent(tu);
          const int64_t blocks = (na + 31) / 32, at = b * a.s_kept + c;
          if ((lane & 7) == 0 && in > 0) {
            a.gate_exp[b * blocks + c / 32] = static_cast<int8_t>(bad_g ? DET_INT8_NAN : eg);
            a.up_exp[b * blocks + c / 32] = static_cast<int8_t>(bad_u ? DET_INT8_NAN : eu);
          }
          const float ig = power_of_two(-eg), iu = power_of_two(-eu);
          if (int8) {
            store_codes(static_cast<int8_t*>(a.gate) + at, codes_of(g, ig, bad_g), in);
            store_codes(static_cast<int8_t*>(a.up) + at, codes_of(u, iu, bad_u), in);
          } else {
            store_halves(static_cast<uint16_t*>(a.gate) + at, g, ig, in);
            store_halves(static_cast<uint16_t*>(a.up) + at, u, iu, in);
          }
        }
      }
    }
  }
  if constexpr (GATED)
    if (noted) a.status[0] = 1;
#endif
}

// ---------------------------------------------------------------- few tokens
//
// The weights' bytes bound it.  A wave owns 16 features, reads their gate and up
// rows straight into fragments (16 bytes to a lane, UN steps of 32 k at a time
// and the next UN ahead, at any alignment) and multiplies them with up to four
// blocks of 16 tokens: the same chain of MFMAs per output as above.  (Four waves
// to the same features, taking the batches of a chain in turn, had more in
// flight but waited for each other: 1 x 2048 x 5461 11.9 -> 16.1 us.)  One token
// x 4096 x 11008: 34 us, 5.3 TB/s of the weights.

struct FewArgs {
  const void* x; int64_t s_x;
  const void* w[2]; int64_t s_w[2];
  int64_t N, F;
  int C;
  void* h;
  int dt, act;
};

// 8 elements from element i of a row, those past C zero
__device__ __forceinline__ bf16x8 fragment(const char* row, int i, int C) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (i + 8 <= C) {
    v = *reinterpret_cast<const u32x4_a2*>(row + i * 2);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (i + e < C)
        v[e / 2] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(row + (i + e) * 2)) << (16 * (e & 1));
  }
  return __builtin_bit_cast(bf16x8, v);
}

template <int NT, int UN>
__global__ __launch_bounds__(64, 2) void k_few(FewArgs a) {
  const int lane = threadIdx.x, q = lane >> 4;
  const int64_t f0 = static_cast<int64_t>(blockIdx.x) * 16, f = min(f0 + (lane & 15), a.F - 1);
  const char* const pg = static_cast<const char*>(a.w[0]) + f * a.s_w[0] * 2;
  const char* const pu = static_cast<const char*>(a.w[1]) + f * a.s_w[1] * 2;
  const char* px[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
    px[j] = static_cast<const char*>(a.x) + min<int64_t>(16 * j + (lane & 15), a.N - 1) * a.s_x * 2;
  f32x4 acc[2][NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[0][j] = acc[1][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  struct Batch {
    u32x4 g[UN], u[UN], x[NT][UN];
  };
  const int whole = a.C / 32;             // steps of 32 that lie inside the row
  auto load = [&](Batch& b, int s0) {
#pragma unroll
    for (int s = 0; s < UN; ++s) {
      const int at = min(s0 + s, whole - 1) * 64 + q * 16;    // past the last one: that one again, not used
      b.g[s] = *reinterpret_cast<const u32x4_a2*>(pg + at);
      b.u[s] = *reinterpret_cast<const u32x4_a2*>(pu + at);
#pragma unroll
      for (int j = 0; j < NT; ++j) b.x[j][s] = *reinterpret_cast<const u32x4_a2*>(px[j] + at);
    }
  };
  auto step = [&](bf16x8 g, bf16x8 u, int j, bf16x8 x) {
    acc[0][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(g, x, acc[0][j], 0, 0, 0);
    acc[1][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(u, x, acc[1][j], 0, 0, 0);
  };
  auto multiply = [&](const Batch& b, int s0) {
#pragma unroll
    for (int s = 0; s < UN; ++s)
      if (s0 + s < whole) {               // uniform
#pragma unroll
        for (int j = 0; j < NT; ++j)
          step(__builtin_bit_cast(bf16x8, b.g[s]), __builtin_bit_cast(bf16x8, b.u[s]), j,
               __builtin_bit_cast(bf16x8, b.x[j][s]));
      }
  };
  if (whole > 0) {
    Batch b0, b1;
    load(b0, 0);
    for (int s = 0; s < whole; s += 2 * UN) {
      load(b1, s + UN);
      multiply(b0, s);
      load(b0, s + 2 * UN);
      multiply(b1, s + UN);
    }
  }
  if (a.C % 32 != 0) {
    const int i = whole * 32 + q * 8;
#pragma unroll
    for (int j = 0; j < NT; ++j) step(fragment(pg, i, a.C), fragment(pu, i, a.C), j, fragment(px[j], i, a.C));
  }
  const int64_t c = f0 + 4 * q;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int64_t b = 16 * j + (lane & 15);
    const float g[4] = {acc[0][j][0], acc[0][j][1], acc[0][j][2], acc[0][j][3]};
    const float u[4] = {acc[1][j][0], acc[1][j][1], acc[1][j][2], acc[1][j][3]};
    float h[4];
    act_times(a.act, g, u, h);
    store4(a.dt, a.h, b * a.F + c, h, b < a.N ? static_cast<int>(min<int64_t>(4, a.F - c)) : 0);
  }
}

// ---------------------------------------------------------------- the gradients' operands

// i / per where both fit 32 bits (a division in 64 costs tens of instructions)
__device__ __forceinline__ int64_t row_of(int64_t i, int64_t per) {
  return i <= 0xFFFFFFFFll ? static_cast<uint32_t>(i) / static_cast<uint32_t>(per) : i / per;
}

struct GateGradArgs {
  const void* dh; int64_t s_dh; int dh_dt;
  const void* gate; const void* up;       // [N] rows of F halves or codes
  int64_t s_kept;
  const int8_t* gate_exp; const int8_t* up_exp;
  int64_t N, F, Fp;
  int act, save;
  uint16_t* rows;                         // [N][2 Fp]: dg and du, zeros from F to Fp
};

// dg and du, rounded to bf16 for the matrix cores (each off by at most half a
// unit; the sums they enter are fp32).  A thread takes 8 adjacent features.  Bound
// by HBM: 8192 x 11008 bf16, 912 MB in 165 to 176 us.
template <int ACT>
__global__ __launch_bounds__(256) void k_gate_grad(GateGradArgs a) {
  const int64_t per = a.Fp / 8, i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= a.N * per) return;
  const int64_t b = row_of(i, per), f0 = (i - b * per) * 8, blocks = (a.F + 31) / 32;
  const float ug = f0 < a.F ? unit_of(a.gate_exp[b * blocks + f0 / 32]) : 0.0f;
  const float uu = f0 < a.F ? unit_of(a.up_exp[b * blocks + f0 / 32]) : 0.0f;
  float dh[2][4], g[2][4], u[2][4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t f = f0 + 4 * h, at = b * a.s_kept + f;
    const int in = static_cast<int>(min<int64_t>(4, a.F - f));
    load4(a.dh_dt, a.dh, b * a.s_dh + f, dh[h], in);
    if (a.save == DET_SAVE_INT8) {
      values_of(load_codes(static_cast<const int8_t*>(a.gate) + at, in), ug, g[h]);
      values_of(load_codes(static_cast<const int8_t*>(a.up) + at, in), uu, u[h]);
    } else {
      load_halves(static_cast<const uint16_t*>(a.gate) + at, ug, g[h], in);
      load_halves(static_cast<const uint16_t*>(a.up) + at, uu, u[h], in);
    }
  }
  float dg[8], du[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const Act t = act_of<ACT>(g[c / 4][c % 4]);
    const bool inside = f0 + c < a.F;
    dg[c] = inside ? dh[c / 4][c % 4] * u[c / 4][c % 4] * t.d : 0.0f;
    du[c] = inside ? dh[c / 4][c % 4] * t.a : 0.0f;
  }
  store_vec<DET_BF16, 8>(a.rows, b * 2 * a.Fp + f0, dg);
  store_vec<DET_BF16, 8>(a.rows, b * 2 * a.Fp + a.Fp + f0, du);
}

// rows of C elements as rows of Cp, the rest zeros: up to three operands at once
struct PadArgs {
  const void* src[3]; int64_t stride[3], R[3];
  void* dst[3];
  unsigned first[3];                      // blocks of the operands before
  int n;
  int64_t C, Cp;
};
__global__ __launch_bounds__(256) void k_pad(PadArgs a) {
  int o = 0;                              // uniform
  while (o + 1 < a.n && blockIdx.x >= a.first[o + 1]) ++o;
  const int64_t per = a.Cp / 8, i = static_cast<int64_t>(blockIdx.x - a.first[o]) * 256 + threadIdx.x;
  if (i >= a.R[o] * per) return;
  const int64_t r = row_of(i, per);
  const int c = static_cast<int>(i - r * per) * 8;
  const bf16x8 v = fragment(static_cast<const char*>(a.src[o]) + r * a.stride[o] * 2, c, static_cast<int>(a.C));
  *reinterpret_cast<bf16x8*>(static_cast<char*>(a.dst[o]) + i * 16) = v;
}

// the same from codes
__global__ __launch_bounds__(256) void k_unpack_pad(const int8_t* src, int64_t s_src, const int8_t* exps, int64_t R,
                                                    int64_t C, int64_t Cp, void* dst) {
  const int64_t per = Cp / 8, i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= R * per) return;
  const int64_t r = row_of(i, per);
  const int c = static_cast<int>(i - r * per) * 8;
  const float unit = c < C ? unit_of(exps[r * ((C + 31) / 32) + c / 32]) : 0.0f;
  float v[8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int in = static_cast<int>(min<int64_t>(4, C - c - 4 * h));
    float q[4];
    values_of(load_codes(src + r * s_src + c + 4 * h, in), unit, q);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[4 * h + e] = e < in ? q[e] : 0.0f;
  }
  store_vec<DET_BF16, 8>(dst, i * 8, v);
}

__global__ __launch_bounds__(256) void k_clear(uint16_t* p, int64_t n) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += step) p[i] = 0;
}

// ---------------------------------------------------------------- host side

// Tokens that go without tiles: up to 16, or 64 where the operands would have to
// be copied first.  64 x 4096 x 11008: 94 us against 45 with tiles, 48 x 2048 x
// 5461 22 against 10.5, with rows of 2047 22 against 30; one token 34 us.
constexpr int64_t FEW = 16, FEW_COPIED = 64;
constexpr int64_t STRIDE_MAX = 1 << 21;   // elements: 512 rows of x or of the weights lie within 2^31 bytes

int64_t up_to(int64_t v, int64_t m) { return ceil_div(v, m) * m; }
int64_t room(int64_t bytes) { return up_to(bytes, 256); }

// whether the copies of the matrix product can take rows of K elements as they lie
bool direct(const void* p, int64_t stride, int64_t K) {
  return K % 64 == 0 && stride % 8 == 0 && stride >= K && stride <= STRIDE_MAX &&
         (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

// Tiles (A x B): large ones move fewer bytes per product, small ones fill the
// chip.  The rule takes the least of what each would take, rounds (stages t +
// end), from what was measured: us per stage of 64 k where up to half the slots
// have a tile, where a few more have and where all have, and for a round's start
// and end.  The forward pass, 4096 features of gate and up together, k 4096, by
// tokens, with 64 x 64 (which fits twice on a CU), 128 x 128, 128 x 256 and 256 x
// 256: 256: 17 us 28 52 87, 512: 28 28 52 87, 1024: 53 35 52 88, 2048: 103 69 65 89,
// 4096: 202 135 124 106.
// "Twice" has a ring short enough for two workgroups on a CU: one's start and end
// go beside the other's products, where many tiles have few stages (forward with
// projections kept, 2000 x 512 x 2816: 35 -> 26 us, 2000 x 1024 x 2816 43 -> 38; dw
// of 500 x 2048 x 5632 54 -> 45).  It waits for its copies where it is alone (512 x
// 4096 x 2048 forward 45, 29 with the long ring) or they come from HBM for long
// (362 x 5824 x 8192 100, 91), so it is left to short k (dw of 2426 x 832 x 3520 57,
// 54).
// The gradients have small tiles with 128 k to a stage, alone on their CU, where
// the chain of stages bounds them: fewer barriers and waits for the LDS (dw of 8192
// x 64 x 64 45 -> 33 us, dx of 200 x 4096 x 4096 40 -> 31; the forward pass gains
// nothing, 16.2 -> 15.6 at best).  A CU gets at most 55 to 90 GB/s into its LDS, so
// dx has 64 x 32 for few tokens (64 x 4160 x 11008: 110 -> 86) and 128 x 64 (1021 x
// 1537 x 4099: 73 -> 58).  The result's bits are the same for all.
enum TileKind { T64_TWICE, T128, T128_TWICE, T128x256, T256, T64, T128x64, T64x32 };
struct TileCost {
  TileKind kind;
  int a, b, slots;
  double half, more, full, end;           // `more`: just past half
  int64_t longest = int64_t{1} << 32;     // k that it is taken for
};
struct Tiles {
  const TileCost* of;
  int n;
};
constexpr TileCost FORWARD[5] = {{T64_TWICE, 64, 64, 512, 0.21, 0.30, 0.40, 2.0},
                                 {T128, 128, 128, 256, 0.44, 0.48, 0.52, 4.0},
                                 {T128_TWICE, 128, 128, 512, 0.64, 0.70, 0.88, 5.0, 2048},
                                 {T128x256, 128, 256, 256, 0.72, 0.76, 0.93, 6.3},
                                 {T256, 256, 256, 256, 1.16, 1.2, 1.52, 12.5}};
constexpr TileCost DX[6] = {{T64x32, 64, 32, 256, 0.15, 0.17, 0.20, 1.5},
                            {T64, 64, 64, 256, 0.21, 0.21, 0.21, 2.0},
                            {T128x64, 128, 64, 256, 0.35, 0.36, 0.38, 2.0},
                            {T128, 128, 128, 256, 0.50, 0.50, 0.55, 2.0},
                            {T128x256, 128, 256, 256, 0.82, 0.82, 0.95, 4.0},
                            {T256, 256, 256, 256, 1.3, 1.3, 1.6, 8.0}};
constexpr TileCost DW[6] = {{T64, 64, 64, 256, 0.25, 0.36, 0.38, 2.0},
                            {T64_TWICE, 64, 64, 512, 0.37, 0.42, 0.50, 2.0},
                            {T128, 128, 128, 256, 0.53, 0.55, 0.55, 3.5},
                            {T128_TWICE, 128, 128, 512, 0.68, 0.80, 0.99, 6.4, 1024},
                            {T128x256, 128, 256, 256, 0.75, 0.80, 1.1, 7.3},
                            {T256, 256, 256, 256, 1.1, 1.3, 1.62, 13.0}};
double tile_time(const TileCost& t, int64_t na, int64_t nb, int64_t K) {
  if (K > t.longest) return INFINITY;
  const int64_t tiles = ceil_div(na, t.a) * ceil_div(nb, t.b), whole = tiles / t.slots, last = tiles % t.slots;
  const double stages = static_cast<double>(K) / 64.0, share = static_cast<double>(last) / t.slots;
  const double partly = share <= 0.5 ? t.half : t.more + (t.full - t.more) * (2.0 * share - 1.0);
  return static_cast<double>(whole) * (stages * t.full + t.end) + (last > 0 ? stages * partly + t.end : 0.0);
}
struct Part {
  TileKind tile;
  int64_t a0, a1, b0, b1;                 // of A (gated: of both halves together) and B
};
double best_tile(const Tiles& tiles, int64_t a0, int64_t a1, int64_t b0, int64_t b1, int64_t K, Part& p) {
  double least = 0.0;
  for (int i = 0; i < tiles.n; ++i) {
    const double time = tile_time(tiles.of[i], a1 - a0, b1 - b0, K);
    if (i == 0 || time < least) {
      p = {tiles.of[i].kind, a0, a1, b0, b1};
      least = time;
    }
  }
  return least;
}
// One launch, or two where a last round would leave most CUs idle: whole rounds
// of one tile first, then the rest with the tile that suits it.  5000 x 5000 x
// 5000 forward 547 -> 483 us, dw of 8000 x 1000 x 10000 512 -> 429, of 1030 x 1024
// x 4100, where the estimate misses, 42 -> 45.
constexpr double LAUNCH = 4.0;            // us
int plan(const Tiles& tiles, int64_t na, int64_t nb, int64_t K, Part (&parts)[2]) {
  double least = best_tile(tiles, 0, na, 0, nb, K, parts[0]);
  int n = 1;
  for (int i = 0; i < tiles.n; ++i) {
    const TileCost& t = tiles.of[i];
    const int64_t ta = ceil_div(na, t.a), tb = ceil_div(nb, t.b), whole = ta * tb / t.slots * t.slots;
    for (int by_b = 0; by_b < 2; ++by_b) {
      const int64_t cut = whole / (by_b ? ta : tb);           // columns (rows) of tiles in whole rounds
      if (cut < 1 || cut >= (by_b ? tb : ta)) continue;
      const int64_t a1 = by_b ? na : cut * t.a, b1 = by_b ? cut * t.b : nb;
      Part rest{};
      const double time =
          LAUNCH + tile_time(t, a1, b1, K) + best_tile(tiles, by_b ? 0 : a1, na, by_b ? b1 : 0, nb, K, rest);
      if (time < least) {
        least = time;
        parts[0] = {t.kind, 0, a1, 0, b1};
        parts[1] = rest;
        n = 2;
      }
    }
  }
  return n;
}

template <bool GATED, bool A_BY_K, bool B_BY_K, int WA, int WB, int FA, int FB, int KS, int BUFS, bool SPREAD>
void launch_tiles(MmArgs a, const Part& p, hipStream_t s) {
  constexpr int halves = GATED ? 2 : 1;
  a.begin_a = p.a0 / halves;
  a.begin_b = p.b0;
  a.tiles_a = ceil_div(p.a1 - p.a0, WA * FA * 16);
  a.tiles_b = ceil_div(p.b1 - p.b0, WB * FB * 16);
  if constexpr (B_BY_K && KS == 128) a.K = a.turn = up_to(a.K, 2 * KS);      // rows past the end are 0
  hipLaunchKernelGGL((k_mm<GATED, A_BY_K, B_BY_K, WA, WB, FA, FB, KS, BUFS, SPREAD>),
                     dim3(static_cast<unsigned>(a.tiles_a * a.tiles_b)), dim3(64 * WA * WB), 0, s, a);
}

// Large tiles: by row 64 k to a stage (whole lines of memory), its reads before
// its MFMAs; by k 32 and 64, spread: 8192 x 4096 x 11008 forward 1187 us so, 1204
// spread, 1306 with 32; dx and its dg and du 1287 against 1387 and 1362, dw 1349
// against 1500.
template <bool GATED, bool A_BY_K, bool B_BY_K>
void launch_part(const MmArgs& a, const Part& p, hipStream_t s) {
  switch (p.tile) {
    case T64_TWICE:
      if constexpr (GATED) launch_tiles<GATED, A_BY_K, B_BY_K, 1, 4, 4, 1, 64, 5, false>(a, p, s);
      else if constexpr (B_BY_K) launch_tiles<GATED, A_BY_K, B_BY_K, 1, 4, 4, 1, 32, 5, true>(a, p, s);
      break;
    case T128:
      if constexpr (!B_BY_K) launch_tiles<GATED, A_BY_K, B_BY_K, 2, 4, 4, 2, 64, 5, true>(a, p, s);
      else launch_tiles<GATED, A_BY_K, B_BY_K, 2, 2, 4, 4, 32, 5, true>(a, p, s);
      break;
    case T128_TWICE:
      if constexpr (GATED) launch_tiles<GATED, A_BY_K, B_BY_K, 2, 4, 4, 2, 64, 2, true>(a, p, s);
      else if constexpr (B_BY_K) launch_tiles<GATED, A_BY_K, B_BY_K, 2, 2, 4, 4, 32, 3, true>(a, p, s);
      break;
    case T128x256:
      if constexpr (!B_BY_K) launch_tiles<GATED, A_BY_K, B_BY_K, 2, 4, 4, 4, 64, 3, !GATED>(a, p, s);
      else launch_tiles<GATED, A_BY_K, B_BY_K, 2, 4, 4, 4, 32, 5, true>(a, p, s);
      break;
    case T256:
      if constexpr (GATED) launch_tiles<GATED, A_BY_K, B_BY_K, 2, 4, 8, 4, 64, 2, false>(a, p, s);
      else launch_tiles<GATED, A_BY_K, B_BY_K, 2, 4, 8, 4, 32, 5, true>(a, p, s);
      break;
    case T64:
      if constexpr (!GATED) launch_tiles<GATED, A_BY_K, B_BY_K, 4, 2, 1, 2, 128, 4, true>(a, p, s);
      break;
    case T128x64:
      if constexpr (!GATED && !B_BY_K) launch_tiles<GATED, A_BY_K, B_BY_K, 8, 2, 1, 2, 128, 3, true>(a, p, s);
      break;
    case T64x32:
      if constexpr (!GATED && !B_BY_K) launch_tiles<GATED, A_BY_K, B_BY_K, 4, 2, 1, 1, 128, 4, true>(a, p, s);
      break;
  }
}
template <bool GATED, bool A_BY_K, bool B_BY_K>
void launch_mm(const MmArgs& a, hipStream_t s) {
  Part parts[2];
  const Tiles tiles = GATED ? Tiles{FORWARD, 5} : B_BY_K ? Tiles{DW, 6} : Tiles{DX, 6};
  const int n = plan(tiles, a.A.n * (GATED ? 2 : 1), a.B.n, a.K, parts);
  for (int i = 0; i < n; ++i) launch_part<GATED, A_BY_K, B_BY_K>(a, parts[i], s);
}

unsigned blocks_for(int64_t threads) { return static_cast<unsigned>(ceil_div(threads, 256)); }

// padded copies of operands, made by one launch
struct Pads {
  PadArgs a{};
  unsigned blocks = 0;
  char* ws;
  Pads(int64_t C, void* workspace) : ws(static_cast<char*>(workspace)) {
    a.C = C;
    a.Cp = up_to(C, 64);
  }
  void copy(const void*& p, int64_t& stride, int64_t R) {
    a.src[a.n] = p;
    a.stride[a.n] = stride;
    a.R[a.n] = R;
    a.dst[a.n] = ws;
    a.first[a.n++] = blocks;
    blocks += blocks_for(R * (a.Cp / 8));
    p = ws;
    stride = a.Cp;
    ws += room(R * a.Cp * 2);
  }
  void launch(hipStream_t s) const {
    if (a.n > 0) hipLaunchKernelGGL(k_pad, dim3(blocks), dim3(256), 0, s, a);
  }
};

bool known_act(int act) { return act == DET_ACT_SILU || act == DET_ACT_GELU || act == DET_ACT_GELU_TANH; }
bool known_save(int save) { return save == DET_SAVE_NONE || save == DET_SAVE_HALF || save == DET_SAVE_INT8; }

det_status check_sizes(int64_t N, int64_t C, int64_t F, int act, int save) {
  if (!known_act(act)) return fail(DET_EINVAL, "unknown activation %d", act);
  if (!known_save(save)) return fail(DET_EINVAL, "unknown kind of checkpoint %d", save);
  if (N < 0 || C < 1 || F < 1)
    return fail(DET_EINVAL, "bad size: N=%lld C=%lld F=%lld", (long long)N, (long long)C, (long long)F);
  if (N > DET_ROWS_MAX) return fail(DET_EINVAL, "N = %lld exceeds the limit 2^22 rows per call", (long long)N);
  if (C > DET_GATED_MAX || F > DET_GATED_MAX)
    return fail(DET_EINVAL, "C = %lld and F = %lld must not exceed 65536", (long long)C, (long long)F);
  // a thread takes 8 elements where rows are copied, and a launch has fewer than 2^32
  if (N * std::max(C, F) > int64_t{1} << 34)
    return fail(DET_EINVAL, "more than 2^34 elements of x or h in one call: N=%lld C=%lld F=%lld", (long long)N,
                (long long)C, (long long)F);
  return DET_OK;
}
det_status check_operand(const void* p, int64_t stride, const char* name) {
  if (p == nullptr) return fail(DET_EINVAL, "null %s", name);
  if (stride < 0) return fail(DET_EINVAL, "negative stride of %s", name);
  if (!aligned_for(p, DET_BF16)) return fail(DET_EINVAL, "%s must be aligned to its element size", name);
  return DET_OK;
}
det_status check_workspace(const void* ws, size_t bytes, int64_t need) {
  if (need > 0 && (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) || bytes < static_cast<size_t>(need)))
    return fail(DET_EINVAL, "workspace: %lld bytes, 256-byte aligned, are needed", (long long)need);
  return DET_OK;
}

}  // namespace

extern "C" {

int64_t det_gated_linear_workspace_bytes(int64_t N, int64_t C, int64_t F, det_save save, int aligned) {
  if (N <= 0 || C <= 0 || F <= 0 || N > DET_ROWS_MAX || C > DET_GATED_MAX || F > DET_GATED_MAX) return 0;
  if ((save == DET_SAVE_NONE && N <= FEW_COPIED) || (C % 64 == 0 && aligned)) return 0;
  const int64_t Cp = up_to(C, 64);
  return room(N * Cp * 2) + 2 * room(F * Cp * 2);
}

det_status det_gated_linear(const void* x, int64_t s_x, const void* w_gate, int64_t s_gate, const void* w_up,
                            int64_t s_up, int64_t N, int64_t C, int64_t F, det_activation act, det_dtype h_dt, void* h,
                            det_save save, void* gate, void* up, int64_t s_kept, int8_t* gate_exp, int8_t* up_exp, void* workspace,
                            size_t workspace_bytes, void* stream) {
  if (!known_dtype(h_dt)) return fail(DET_EDTYPE, "unknown dtype %d", h_dt);
  det_status st = check_sizes(N, C, F, act, save);
  if (st != DET_OK || N == 0) return st;
  if ((st = check_operand(x, s_x, "x")) != DET_OK || (st = check_operand(w_gate, s_gate, "w_gate")) != DET_OK ||
      (st = check_operand(w_up, s_up, "w_up")) != DET_OK)
    return st;
  if (h == nullptr ||
      (save != DET_SAVE_NONE && (gate == nullptr || up == nullptr || gate_exp == nullptr || up_exp == nullptr)))
    return fail(DET_EINVAL, "null output");
  if (save != DET_SAVE_NONE && s_kept < F)
    return fail(DET_EINVAL, "rows of gate and up overlap: stride %lld", (long long)s_kept);
  if (!aligned_for(h, h_dt) || (save == DET_SAVE_HALF && (!aligned_for(gate, DET_BF16) || !aligned_for(up, DET_BF16))))
    return fail(DET_EINVAL, "outputs must be aligned to their element size");
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool copies = !direct(x, s_x, C) || !direct(w_gate, s_gate, C) || !direct(w_up, s_up, C);
  if (save == DET_SAVE_NONE && N <= (copies ? FEW_COPIED : FEW)) {
    FewArgs a{x, s_x, {w_gate, w_up}, {s_gate, s_up}, N, F, static_cast<int>(C), h, h_dt, act};
    const dim3 grid(static_cast<unsigned>(ceil_div(F, 16)));
    if (N <= 16) hipLaunchKernelGGL((k_few<1, 8>), grid, dim3(64), 0, s, a);
    else if (N <= 32) hipLaunchKernelGGL((k_few<2, 4>), grid, dim3(64), 0, s, a);
    else hipLaunchKernelGGL((k_few<4, 4>), grid, dim3(64), 0, s, a);
    return hip_check(hipGetLastError(), "gated projection launch");
  }
  const int64_t Cp = up_to(C, 64);
  const int64_t need = (direct(x, s_x, C) ? 0 : room(N * Cp * 2)) + (direct(w_gate, s_gate, C) ? 0 : room(F * Cp * 2)) +
                       (direct(w_up, s_up, C) ? 0 : room(F * Cp * 2));
  if ((st = check_workspace(workspace, workspace_bytes, need)) != DET_OK) return st;
  MmArgs a{};
  a.A = {w_gate, s_gate, F};
  a.A1 = {w_up, s_up, F};
  a.B = {x, s_x, N};
  Pads pads(C, workspace);
  for (Operand* o : {&a.A, &a.A1, &a.B})
    if (!direct(o->p, o->stride, C)) pads.copy(o->p, o->stride, o->n);
  pads.launch(s);
  a.K = Cp;
  a.out = h; a.dt = h_dt; a.act = act; a.save = save;
  a.gate = gate; a.up = up; a.s_kept = s_kept; a.gate_exp = gate_exp; a.up_exp = up_exp;
  if (save == DET_SAVE_INT8 && (a.status = det_device_status_word()) == nullptr) return DET_EHIP;
  launch_mm<true, false, false>(a, s);
  return hip_check(hipGetLastError(), "gated projection launch");
}

int64_t det_gated_linear_grad_workspace_bytes(int64_t N, int64_t C, int64_t F, int need_dx, int need_dw, int aligned,
                                              int packed) {
  if (N <= 0 || C <= 0 || F <= 0 || N > DET_ROWS_MAX || C > DET_GATED_MAX || F > DET_GATED_MAX ||
      (!need_dx && !need_dw))
    return 0;
  const int64_t Cp = up_to(C, 64);
  const bool as_is = C % 64 == 0 && aligned;
  return room(N * 2 * up_to(F, 128) * 2) + (need_dx && !as_is ? 2 * room(F * Cp * 2) : 0) +
         (need_dw && (packed || !as_is) ? room(N * Cp * 2) : 0);
}

det_status det_gated_linear_grad(det_dtype dh_dt, const void* dh, int64_t s_dh, const void* x, int64_t s_x,
                                 const int8_t* x_exp, const void* w_gate, int64_t s_gate, const void* w_up,
                                 int64_t s_up, det_save save, const void* gate, const void* up, int64_t s_kept,
                                 const int8_t* gate_exp,
                                 const int8_t* up_exp, int64_t N, int64_t C, int64_t F, det_activation act, void* dx,
                                 void* dw_gate, void* dw_up, void* workspace, size_t workspace_bytes, void* stream) {
  if (!known_dtype(dh_dt)) return fail(DET_EDTYPE, "unknown dtype %d", dh_dt);
  det_status st = check_sizes(N, C, F, act, save);
  if (st != DET_OK) return st;
  if (save == DET_SAVE_NONE)
    return fail(DET_EINVAL, "the gradient needs both projections: save them in the forward call");
  const bool need_dx = dx != nullptr, need_dw = dw_gate != nullptr || dw_up != nullptr;
  if (need_dw && (dw_gate == nullptr || dw_up == nullptr))
    return fail(DET_EINVAL, "dw_gate and dw_up are formed together");
  if (!aligned_for(dx, DET_BF16) || !aligned_for(dw_gate, DET_BF16) || !aligned_for(dw_up, DET_BF16))
    return fail(DET_EINVAL, "outputs must be aligned to their element size");
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (N == 0) {
    if (need_dw)
      for (void* p : {dw_gate, dw_up})
        hipLaunchKernelGGL(k_clear, dim3(static_cast<unsigned>(std::min<int64_t>(ceil_div(F * C, 256), 1 << 16))),
                           dim3(256), 0, s, static_cast<uint16_t*>(p), F * C);
    return need_dw ? hip_check(hipGetLastError(), "clearing launch") : DET_OK;
  }
  if (!need_dx && !need_dw) return DET_OK;
  if (dh == nullptr || gate == nullptr || up == nullptr || gate_exp == nullptr || up_exp == nullptr)
    return fail(DET_EINVAL, "null pointer");
  if (s_dh < 0 || s_kept < 0) return fail(DET_EINVAL, "negative stride");
  if (!aligned_for(dh, dh_dt) ||
      (save == DET_SAVE_HALF && (!aligned_for(gate, DET_BF16) || !aligned_for(up, DET_BF16))))
    return fail(DET_EINVAL, "operands must be aligned to their element size");
  if (need_dx && ((st = check_operand(w_gate, s_gate, "w_gate")) != DET_OK ||
                  (st = check_operand(w_up, s_up, "w_up")) != DET_OK))
    return st;
  if (need_dw) {
    if (x == nullptr || s_x < 0) return fail(DET_EINVAL, "null x or negative stride");
    if (x_exp == nullptr && !aligned_for(x, DET_BF16)) return fail(DET_EINVAL, "x must be aligned to its element size");
  }
  const int64_t Cp = up_to(C, 64), Fp = up_to(F, 128), rows = room(N * 2 * Fp * 2);
  const bool codes = need_dw && x_exp != nullptr;
  // k runs over both weights with one stride
  const bool copy_w = !direct(w_gate, s_gate, C) || !direct(w_up, s_up, C) || s_gate != s_up;
  const int64_t need = rows + (need_dx && copy_w ? 2 * room(F * Cp * 2) : 0) +
                       (need_dw && (codes || !direct(x, s_x, C)) ? room(N * Cp * 2) : 0);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != DET_OK) return st;
  GateGradArgs g{};
  g.dh = dh; g.s_dh = s_dh; g.dh_dt = dh_dt;
  g.gate = gate; g.up = up; g.s_kept = s_kept; g.gate_exp = gate_exp; g.up_exp = up_exp;
  g.N = N; g.F = F; g.Fp = Fp; g.save = save;
  g.rows = static_cast<uint16_t*>(workspace);
  const dim3 grid(blocks_for(N * (Fp / 8)));
  if (act == DET_ACT_SILU) hipLaunchKernelGGL(k_gate_grad<DET_ACT_SILU>, grid, dim3(256), 0, s, g);
  else if (act == DET_ACT_GELU_TANH) hipLaunchKernelGGL(k_gate_grad<DET_ACT_GELU_TANH>, grid, dim3(256), 0, s, g);
  else hipLaunchKernelGGL(k_gate_grad<DET_ACT_GELU>, grid, dim3(256), 0, s, g);
  Operand gates{w_gate, s_gate, C}, ups{w_up, s_up, C}, xs{x, s_x, C};
  Pads pads(C, static_cast<char*>(workspace) + rows);
  if (need_dx && copy_w) {
    pads.copy(gates.p, gates.stride, F);
    pads.copy(ups.p, ups.stride, F);
  }
  if (need_dw && codes) {
    hipLaunchKernelGGL(k_unpack_pad, dim3(blocks_for(N * (Cp / 8))), dim3(256), 0, s, static_cast<const int8_t*>(x),
                       s_x, x_exp, N, C, Cp, static_cast<void*>(pads.ws));
    xs = {pads.ws, Cp, C};
  } else if (need_dw && !direct(x, s_x, C)) {
    pads.copy(xs.p, xs.stride, N);
  }
  pads.launch(s);
  if (need_dx) {                          // dx [N][C]: k over the gate's features, then over the up projection's
    MmArgs a{};
    a.A = gates;
    a.A1 = ups;
    a.B = {workspace, 2 * Fp, N};
    a.K = 2 * Fp; a.ka = F; a.turn = Fp;
    a.out = dx; a.split0 = a.split1 = N; a.dt = DET_BF16;
    launch_mm<false, true, false>(a, s);
  }
  if (need_dw) {                          // dw [2 F][C]: k over the rows
    MmArgs a{};
    a.A = a.A1 = xs;
    a.B = {workspace, 2 * Fp, 2 * Fp};
    a.K = a.turn = up_to(N, 64); a.ka = a.kb = N;
    a.out = dw_gate; a.out1 = dw_up; a.split0 = F; a.split1 = Fp; a.dt = DET_BF16;
    launch_mm<false, true, true>(a, s);
  }
  return hip_check(hipGetLastError(), "gated projection gradient launch");
}

}  // extern "C"
