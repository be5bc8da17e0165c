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
using u32x2 = uint32_t __attribute__((ext_vector_type(2)));

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
    // 0.5 g (1 + tanh t) = g sigmoid(2 t)
    const float g2 = g * g, in = g * fmaf(0.0713548163f, g2, 1.59576912f);
    const Sigmoid s = sigmoid(in);
    const float slope = s.s * s.rest * fmaf(0.214064449f, g2, 1.59576912f);
    return {g * s.s, fmaf(g, slope, s.s)};
  } else {
    const float p = 0.5f * erfcf(g * -0.707106769f);
    return {g * p, fmaf(g, 0.398942292f * exp_of(-0.5f * g * g), p)};
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
// D[b][a] = sum_k A[a][k] B[b][k], both operands with adjacent k and K a
// multiple of 64.  A workgroup of WA x WB waves owns TA x TB outputs, a wave
// FA x FB blocks of 16 x 16.  Per step of 64 k the TA + TB rows (128 bytes
// each) are copied into one of two LDS buffers with 16-byte copies that need
// no registers, while the other buffer is read.  A row's eight 16-byte pieces
// lie in its LDS row in the order piece ^ (row & 7), so that the 8 lanes that
// read a piece of 8 rows at a time hit different banks.
//
// A step is two halves of one MFMA per block: while a half's MFMAs run, the
// next half's fragments are read.

enum { MM_GATED, MM_ROWS };

struct MmArgs {
  const void* A; int64_t s_a;             // MM_GATED: the gate's weights
  const void* A1; int64_t s_a1;           // MM_GATED: the up projection's
  const void* B; int64_t s_b;
  int64_t na, nb;                         // rows of A (MM_GATED: of each half) and of B
  int K;
  int64_t tiles_a, tiles_b;
  // MM_GATED: out is h [nb][na]; MM_ROWS: D itself, rows from `split` on in out1
  void* out; void* out1; int64_t split;
  // what the gradients read again (null: nothing)
  void* gate; void* up;
  int8_t* gate_exp; int8_t* up_exp;
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

#ifdef __HIP_DEVICE_COMPILE__              // buffer descriptors are a type of the device's alone
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, static_cast<int>(bytes), 0x00020000);
}
#endif

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

template <int MODE, int WA, int WB, int FA, int FB>
__global__ __launch_bounds__(64 * WA * WB, 2) void k_mm(MmArgs a) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int NW = WA * WB, TA = WA * FA * 16, TB = WB * FB * 16, TH = MODE == MM_GATED ? TA / 2 : TA;
  constexpr int CA = TA / 8 / NW, CB = TB / 8 / NW;           // copies (8 rows each) of a wave and step
  constexpr int BUF = (TA + TB) * 128;
  __shared__ __attribute__((aligned(1024))) char lds[2 * BUF];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wa = wave / WB, wb = wave % WB;
  int64_t ta, tb;
  tile_of(blockIdx.x, a.tiles_a, a.tiles_b, ta, tb);
  const int64_t row_a = ta * TH, row_b = tb * TB;

  // where this wave's copies come from: rows past the end are the last one again
  const bool second = MODE == MM_GATED && wave * CA * 8 >= TH;            // uniform: the up projection's rows
  const int64_t s_a = second ? a.s_a1 : a.s_a;
  const char* const pa = static_cast<const char*>(second ? a.A1 : a.A) + row_a * s_a * 2;
  const char* const pb = static_cast<const char*>(a.B) + row_b * a.s_b * 2;
  const int rows_a = static_cast<int>(min<int64_t>(TH, a.na - row_a)), rows_b = static_cast<int>(min<int64_t>(TB, a.nb - row_b));
  const __amdgpu_buffer_rsrc_t ra = buffer_of(pa, (rows_a - 1) * s_a * 2 + static_cast<int64_t>(a.K) * 2);
  const __amdgpu_buffer_rsrc_t rb = buffer_of(pb, (rows_b - 1) * a.s_b * 2 + static_cast<int64_t>(a.K) * 2);
  const int piece = ((lane & 7) ^ (lane >> 3)) * 16;
  int from_a[CA], from_b[CB];
#pragma unroll
  for (int j = 0; j < CA; ++j) {
    const int r = (wave * CA + j) * 8 + (lane >> 3) - (second ? TH : 0);
    from_a[j] = min(r, rows_a - 1) * static_cast<int>(s_a * 2) + piece;
  }
#pragma unroll
  for (int j = 0; j < CB; ++j) {
    const int r = (wave * CB + j) * 8 + (lane >> 3);
    from_b[j] = min(r, rows_b - 1) * static_cast<int>(a.s_b * 2) + piece;
  }
  auto copy = [&](int k, int buf) {
    char* const to = lds + buf * BUF;
#pragma unroll
    for (int j = 0; j < CA; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, to + (wave * CA + j) * 1024, 16, from_a[j], k * 2, 0, 0);
#pragma unroll
    for (int j = 0; j < CB; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, to + TA * 128 + (wave * CB + j) * 1024, 16, from_b[j], k * 2, 0, 0);
  };

  // the first LDS row of fragment i of A (of this wave)
  auto frag_row = [&](int i) {
    if constexpr (MODE == MM_GATED) return (i < FA / 2 ? 0 : TH) + wa * FA * 8 + (i % (FA / 2)) * 16;
    else return (wa * FA + i) * 16;
  };
  const int in_row = (lane & 15) * 128 + (((lane >> 4) ^ (lane & 7)) * 16);   // the second half: ^ 64
  struct Frags {
    bf16x8 fa[FA], fb[FB];
  };
  auto read = [&](Frags& f, int buf, int half) {
    const char* const at = lds + buf * BUF + (in_row ^ (half * 64));
#pragma unroll
    for (int j = 0; j < FB; ++j) f.fb[j] = *reinterpret_cast<const bf16x8*>(at + TA * 128 + (wb * FB + j) * 2048);
#pragma unroll
    for (int i = 0; i < FA; ++i) f.fa[i] = *reinterpret_cast<const bf16x8*>(at + frag_row(i) * 128);
  };
  f32x4 acc[FA][FB];
#pragma unroll
  for (int i = 0; i < FA; ++i)
#pragma unroll
    for (int j = 0; j < FB; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  auto multiply = [&](const Frags& f) {
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
      for (int j = 0; j < FB; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.fa[i], f.fb[j], acc[i][j], 0, 0, 0);
  };

  const int steps = a.K / 64;
  Frags f0, f1;
  copy(0, 0);
  __builtin_amdgcn_s_waitcnt(waitcnt(0, 15));
  step_barrier();
  read(f0, 0, 0);
  copy(min(1, steps - 1) * 64, 1);
  __builtin_amdgcn_sched_barrier(0);
  for (int s = 0; s < steps; ++s) {
    const int buf = s & 1;
    read(f1, buf, 1);
    __builtin_amdgcn_sched_barrier(0);
    multiply(f0);
    __builtin_amdgcn_sched_barrier(0);
    // this buffer's reads are done and the other buffer's copies have landed, for every wave
    __builtin_amdgcn_s_waitcnt(waitcnt(0, 0));
    step_barrier();
    read(f0, buf ^ 1, 0);                 // after the last step: read again, not used
    __builtin_amdgcn_sched_barrier(0);
    copy(min(s + 2, steps - 1) * 64, buf);
    __builtin_amdgcn_sched_barrier(0);
    multiply(f1);
    __builtin_amdgcn_sched_barrier(0);
  }
  __builtin_amdgcn_s_waitcnt(waitcnt(0, 0));                  // no copy or read of these buffers is left
  step_barrier();

  // The sums go through LDS, 16 rows of the output at a time and each wave
  // by itself, so that a row is written in whole lines.  Lane l holds features
  // 4 (l / 16) .. + 3 of a block, of row l % 16.
  constexpr int ROW = FA * 16 + 4;        // floats; 4 more, or all rows would start in one bank
  float* const own = reinterpret_cast<float*>(lds) + wave * 16 * ROW;
#pragma unroll
  for (int j = 0; j < FB; ++j) {
    wave_sync();
#pragma unroll
    for (int i = 0; i < FA; ++i)
      *reinterpret_cast<f32x4*>(own + (lane & 15) * ROW + i * 16 + 4 * (lane >> 4)) = acc[i][j];
    wave_sync();
    constexpr int LANES = (MODE == MM_GATED ? FA / 2 : FA) * 4;           // lanes to a row
    const int64_t c = row_a + wa * (LANES * 4) + (lane % LANES) * 4;
    const int n = static_cast<int>(min<int64_t>(4, a.na - c));
#pragma unroll 1
    for (int r0 = 0; r0 < 16; r0 += 64 / LANES) {
      const int r = r0 + lane / LANES;
      const int64_t b = row_b + (wb * FB + j) * 16 + r;
      const int in = b < a.nb ? n : 0;
      const float* const from = own + r * ROW + (lane % LANES) * 4;
      const f32x4 first = *reinterpret_cast<const f32x4*>(from);
      if constexpr (MODE == MM_ROWS) {
        const float v[4] = {first[0], first[1], first[2], first[3]};
        const bool hi = b >= a.split;
        store4(a.dt, hi ? a.out1 : a.out, (hi ? b - a.split : b) * a.na + c, v, in);
      } else {
        const f32x4 upper = *reinterpret_cast<const f32x4*>(from + FA * 8);
        const float g[4] = {first[0], first[1], first[2], first[3]}, u[4] = {upper[0], upper[1], upper[2], upper[3]};
        float h[4];
        act_times(a.act, g, u, h);
        store4(a.dt, a.out, b * a.na + c, h, in);
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
          const int eg = int8 ? block_exponent(tg) : half_exponent(tg), eu = int8 ? block_exponent(tu) : half_exponent(tu);
          const int64_t blocks = (a.na + 31) / 32, at = b * a.na + c;
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
#endif
}

// ---------------------------------------------------------------- few tokens
//
// Up to 64 tokens: the weights' bytes bound it.  A wave owns 16 features, reads
// their gate and up rows straight into fragments (16 bytes to a lane, UN steps
// of 32 k ahead) and multiplies them with up to four blocks of 16 tokens: the
// same chain of MFMAs per output as above.

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
      if (i + e < C) v[e / 2] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(row + (i + e) * 2)) << (16 * (e & 1));
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
          step(__builtin_bit_cast(bf16x8, b.g[s]), __builtin_bit_cast(bf16x8, b.u[s]), j, __builtin_bit_cast(bf16x8, b.x[j][s]));
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
//
// Tiles of 64 x 64, 4 x 4 elements to a thread; what is needed with the other
// index adjacent goes through LDS (68 elements to a row: 8-byte accesses of 16
// rows fall in different banks).

constexpr int TILE = 64, TILE_ROW = 68;

struct Tile {
  uint16_t v[TILE][TILE_ROW];
};
// element (r, c) of the thread's 4 x 4, from (4 tr, 4 tc) of the tile, into row c, column r
__device__ __forceinline__ void turn(Tile& t, int tr, int tc, const float (&v)[4][4]) {
#pragma unroll
  for (int c = 0; c < 4; ++c)
    *reinterpret_cast<u32x2*>(&t.v[4 * tc + c][4 * tr]) = u32x2{pack_bf16(v[0][c], v[1][c]), pack_bf16(v[2][c], v[3][c])};
}
// the turned tile's rows [0, rows) at dst (element (0, 0)), `cols` of each
__device__ __forceinline__ void write_turned(const Tile& t, char* dst, int64_t stride, int rows, int cols) {
  const int c = (threadIdx.x & 15) * 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 16 + (threadIdx.x >> 4);
    if (r < rows && c < cols)             // cols is a multiple of 4
      *reinterpret_cast<u32x2_a2*>(dst + (r * stride + c) * 2) = *reinterpret_cast<const u32x2*>(&t.v[r][c]);
  }
}

struct GateGradArgs {
  const void* dh; int64_t s_dh; int dh_dt;
  const void* gate; const void* up;       // [N][F] halves or codes
  const int8_t* gate_exp; const int8_t* up_exp;
  int64_t N, F, Fp, Np;
  int act, save;
  char* rows;                             // [N][2 Fp]: dg and du, zeros from F to Fp; null: not needed
  char* turned;                           // [2 F][Np]: the same by feature, zeros from N to Np
};

// dg and du, rounded to bf16 for the matrix cores (each off by at most half a
// unit; the sums they enter are fp32)
__global__ __launch_bounds__(256) void k_gate_grad(GateGradArgs a) {
  __shared__ Tile tg, tu;
  const int64_t f0 = static_cast<int64_t>(blockIdx.y) * TILE, b0 = static_cast<int64_t>(blockIdx.x) * TILE;
  const int tr = threadIdx.x >> 4, tc = threadIdx.x & 15;
  const int64_t f = f0 + 4 * tc;
  const int n = static_cast<int>(min<int64_t>(4, a.F - f));
  const int64_t blocks = (a.F + 31) / 32;
  float dg[4][4], du[4][4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int64_t b = b0 + 4 * tr + r;
    const int in = b < a.N ? n : 0;
    float dh[4], g[4], u[4];
    load4(a.dh_dt, a.dh, b * a.s_dh + f, dh, in);
    const float ug = in > 0 ? unit_of(a.gate_exp[b * blocks + f / 32]) : 0.0f;
    const float uu = in > 0 ? unit_of(a.up_exp[b * blocks + f / 32]) : 0.0f;
    if (a.save == DET_SAVE_INT8) {
      values_of(load_codes(static_cast<const int8_t*>(a.gate) + b * a.F + f, in), ug, g);
      values_of(load_codes(static_cast<const int8_t*>(a.up) + b * a.F + f, in), uu, u);
    } else {
      load_halves(static_cast<const uint16_t*>(a.gate) + b * a.F + f, ug, g, in);
      load_halves(static_cast<const uint16_t*>(a.up) + b * a.F + f, uu, u, in);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      Act t;
      if (a.act == DET_ACT_SILU) t = act_of<DET_ACT_SILU>(g[c]);
      else if (a.act == DET_ACT_GELU_TANH) t = act_of<DET_ACT_GELU_TANH>(g[c]);
      else t = act_of<DET_ACT_GELU>(g[c]);
      const bool inside = c < in;
      dg[r][c] = inside ? dh[c] * u[c] * t.d : 0.0f;
      du[r][c] = inside ? dh[c] * t.a : 0.0f;
    }
    if (a.rows != nullptr && b < a.N && f < a.Fp) {           // Fp is a multiple of 4
      store_vec<DET_BF16, 4>(a.rows, b * 2 * a.Fp + f, dg[r]);
      store_vec<DET_BF16, 4>(a.rows, b * 2 * a.Fp + a.Fp + f, du[r]);
    }
  }
  if (a.turned == nullptr) return;        // uniform
  turn(tg, tr, tc, dg);
  turn(tu, tr, tc, du);
  __syncthreads();
  const int rows = static_cast<int>(min<int64_t>(TILE, a.F - f0)), cols = static_cast<int>(min<int64_t>(TILE, a.Np - b0));
  write_turned(tg, a.turned + (f0 * a.Np + b0) * 2, a.Np, rows, cols);
  write_turned(tu, a.turned + ((a.F + f0) * a.Np + b0) * 2, a.Np, rows, cols);
}

struct TurnArgs {
  const void* src; int64_t s_src;         // [R][C], bf16 or codes with exponents
  const int8_t* exps;
  int64_t R, C, Rp;
  char* dst; int64_t s_dst;               // [C][Rp]: zeros from R to Rp, a multiple of 4
};
__global__ __launch_bounds__(256) void k_turn(TurnArgs a) {
  __shared__ Tile t;
  const int64_t c0 = static_cast<int64_t>(blockIdx.y) * TILE, r0 = static_cast<int64_t>(blockIdx.x) * TILE;
  const int tr = threadIdx.x >> 4, tc = threadIdx.x & 15;
  const int64_t c = c0 + 4 * tc;
  const int n = static_cast<int>(min<int64_t>(4, a.C - c));
  float v[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + 4 * tr + i;
    const int in = r < a.R ? n : 0;
    if (a.exps != nullptr) {
      const float unit = in > 0 ? unit_of(a.exps[r * ((a.C + 31) / 32) + c / 32]) : 0.0f;
      values_of(load_codes(static_cast<const int8_t*>(a.src) + r * a.s_src + c, in), unit, v[i]);
    } else {
      load4(DET_BF16, a.src, r * a.s_src + c, v[i], in);
    }
  }
  turn(t, tr, tc, v);
  __syncthreads();
  write_turned(t, a.dst + (c0 * a.s_dst + r0) * 2, a.s_dst, static_cast<int>(min<int64_t>(TILE, a.C - c0)),
               static_cast<int>(min<int64_t>(TILE, a.Rp - r0)));
}

// rows of C elements as rows of Cp, the rest zeros
__global__ __launch_bounds__(256) void k_pad(const void* src, int64_t s_src, int64_t R, int64_t C, int64_t Cp, void* dst) {
  const int64_t per = Cp / 8, i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= R * per) return;
  const int64_t r = i / per;
  const int c = static_cast<int>(i % per) * 8;
  const bf16x8 v = fragment(static_cast<const char*>(src) + r * s_src * 2, c, static_cast<int>(C));
  *reinterpret_cast<bf16x8*>(static_cast<char*>(dst) + i * 16) = v;
}

__global__ __launch_bounds__(256) void k_clear(uint16_t* p, int64_t n) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i < n) p[i] = 0;
}

// ---------------------------------------------------------------- host side

constexpr int64_t FEW = 64;               // tokens
constexpr int64_t STRIDE_MAX = 1 << 22;   // 256 rows lie within 2^31 bytes: offsets fit a buffer's 32 bits

int64_t up_to(int64_t v, int64_t m) { return ceil_div(v, m) * m; }
int64_t room(int64_t bytes) { return up_to(bytes, 256); }

// whether the copies of the matrix product can take this operand as it lies
bool direct(const void* p, int64_t stride, int64_t K) {
  return K % 64 == 0 && stride % 8 == 0 && stride >= K && stride <= STRIDE_MAX && (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

template <int MODE>
void launch_mm(MmArgs a, hipStream_t s) {
  constexpr int half = MODE == MM_GATED ? 2 : 1;
  // tiles of 256 x 256 (one workgroup per CU) where they fill the chip, else of 128 x 128
  const int64_t large = ceil_div(a.na * half, 256) * ceil_div(a.nb, 256);
  if (large >= 256) {
    a.tiles_a = ceil_div(a.na * half, 256);
    a.tiles_b = ceil_div(a.nb, 256);
    hipLaunchKernelGGL((k_mm<MODE, 2, 4, 8, 4>), dim3(static_cast<unsigned>(a.tiles_a * a.tiles_b)), dim3(512), 0, s, a);
  } else {
    a.tiles_a = ceil_div(a.na * half, 128);
    a.tiles_b = ceil_div(a.nb, 128);
    hipLaunchKernelGGL((k_mm<MODE, 2, 2, 4, 4>), dim3(static_cast<unsigned>(a.tiles_a * a.tiles_b)), dim3(256), 0, s, a);
  }
}

// p as an operand of the matrix product: itself, or a padded copy at ws (which advances)
const void* operand(const void* p, int64_t& stride, int64_t R, int64_t K, char*& ws, hipStream_t s) {
  if (direct(p, stride, K)) return p;
  const int64_t Kp = up_to(K, 64);
  void* const to = ws;
  ws += room(R * Kp * 2);
  hipLaunchKernelGGL(k_pad, dim3(static_cast<unsigned>(ceil_div(R * (Kp / 8), 256))), dim3(256), 0, s, p, stride, R, K, Kp, to);
  stride = Kp;
  return to;
}

struct GradRoom {
  int64_t rows, turned, x, w, total;
};
GradRoom grad_room(int64_t N, int64_t C, int64_t F, bool need_dx, bool need_dw) {
  const int64_t Fp = up_to(F, 32), Np = up_to(N, 64);
  GradRoom r{};
  if (need_dx) {
    r.rows = room(N * 2 * Fp * 2);
    r.w = room(C * 2 * Fp * 2);
  }
  if (need_dw) {
    r.turned = room(2 * F * Np * 2);
    r.x = room(C * Np * 2);
  }
  r.total = r.rows + r.turned + r.x + r.w;
  return r;
}

void turn_rows(const void* src, int64_t s_src, const int8_t* exps, int64_t R, int64_t C, int64_t Rp, char* dst,
               int64_t s_dst, hipStream_t s) {
  TurnArgs a{src, s_src, exps, R, C, Rp, dst, s_dst};
  hipLaunchKernelGGL(k_turn, dim3(static_cast<unsigned>(ceil_div(Rp, TILE)), static_cast<unsigned>(ceil_div(C, TILE))),
                     dim3(256), 0, s, a);
}

bool known_act(int act) { return act == DET_ACT_SILU || act == DET_ACT_GELU || act == DET_ACT_GELU_TANH; }
bool known_save(int save) { return save == DET_SAVE_NONE || save == DET_SAVE_HALF || save == DET_SAVE_INT8; }

det_status check_sizes(int64_t N, int64_t C, int64_t F, int act, int save) {
  if (!known_act(act)) return fail(DET_EINVAL, "unknown activation %d", act);
  if (!known_save(save)) return fail(DET_EINVAL, "unknown kind of checkpoint %d", save);
  if (N < 0 || C < 1 || F < 1) return fail(DET_EINVAL, "bad size: N=%lld C=%lld F=%lld", (long long)N, (long long)C, (long long)F);
  if (N > DET_ROWS_MAX) return fail(DET_EINVAL, "N = %lld exceeds the limit 2^22 rows per call", (long long)N);
  if (C > DET_GATED_MAX || F > DET_GATED_MAX)
    return fail(DET_EINVAL, "C = %lld and F = %lld must not exceed 65536", (long long)C, (long long)F);
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
  if ((save == DET_SAVE_NONE && N <= FEW) || (C % 64 == 0 && aligned)) return 0;
  const int64_t Cp = up_to(C, 64);
  return room(N * Cp * 2) + 2 * room(F * Cp * 2);
}

det_status det_gated_linear(const void* x, int64_t s_x, const void* w_gate, int64_t s_gate, const void* w_up,
                            int64_t s_up, int64_t N, int64_t C, int64_t F, det_activation act, det_dtype h_dt, void* h,
                            det_save save, void* gate, void* up, int8_t* gate_exp, int8_t* up_exp, void* workspace,
                            size_t workspace_bytes, void* stream) {
  if (!known_dtype(h_dt)) return fail(DET_EDTYPE, "unknown dtype %d", h_dt);
  det_status st = check_sizes(N, C, F, act, save);
  if (st != DET_OK || N == 0) return st;
  if ((st = check_operand(x, s_x, "x")) != DET_OK || (st = check_operand(w_gate, s_gate, "w_gate")) != DET_OK ||
      (st = check_operand(w_up, s_up, "w_up")) != DET_OK)
    return st;
  if (h == nullptr || (save != DET_SAVE_NONE && (gate == nullptr || up == nullptr || gate_exp == nullptr || up_exp == nullptr)))
    return fail(DET_EINVAL, "null output");
  if (!aligned_for(h, h_dt) || (save == DET_SAVE_HALF && (!aligned_for(gate, DET_BF16) || !aligned_for(up, DET_BF16))))
    return fail(DET_EINVAL, "outputs must be aligned to their element size");
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (save == DET_SAVE_NONE && N <= FEW) {
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
  char* ws = static_cast<char*>(workspace);
  MmArgs a{};
  a.s_a = s_gate; a.s_a1 = s_up; a.s_b = s_x;
  a.A = operand(w_gate, a.s_a, F, C, ws, s);
  a.A1 = operand(w_up, a.s_a1, F, C, ws, s);
  a.B = operand(x, a.s_b, N, C, ws, s);
  a.na = F; a.nb = N; a.K = static_cast<int>(Cp);
  a.out = h; a.dt = h_dt; a.act = act; a.save = save;
  a.gate = gate; a.up = up; a.gate_exp = gate_exp; a.up_exp = up_exp;
  launch_mm<MM_GATED>(a, s);
  return hip_check(hipGetLastError(), "gated projection launch");
}

int64_t det_gated_linear_grad_workspace_bytes(int64_t N, int64_t C, int64_t F, int need_dx, int need_dw) {
  if (N <= 0 || C <= 0 || F <= 0 || N > DET_ROWS_MAX || C > DET_GATED_MAX || F > DET_GATED_MAX) return 0;
  return grad_room(N, C, F, need_dx != 0, need_dw != 0).total;
}

det_status det_gated_linear_grad(det_dtype dh_dt, const void* dh, int64_t s_dh, const void* x, int64_t s_x,
                                 const int8_t* x_exp, const void* w_gate, int64_t s_gate, const void* w_up,
                                 int64_t s_up, det_save save, const void* gate, const void* up, const int8_t* gate_exp,
                                 const int8_t* up_exp, int64_t N, int64_t C, int64_t F, det_activation act, void* dx,
                                 void* dw_gate, void* dw_up, void* workspace, size_t workspace_bytes, void* stream) {
  if (!known_dtype(dh_dt)) return fail(DET_EDTYPE, "unknown dtype %d", dh_dt);
  det_status st = check_sizes(N, C, F, act, save);
  if (st != DET_OK) return st;
  if (save == DET_SAVE_NONE) return fail(DET_EINVAL, "the gradient needs both projections: save them in the forward call");
  const bool need_dx = dx != nullptr, need_dw = dw_gate != nullptr || dw_up != nullptr;
  if (need_dw && (dw_gate == nullptr || dw_up == nullptr)) return fail(DET_EINVAL, "dw_gate and dw_up are formed together");
  if (!aligned_for(dx, DET_BF16) || !aligned_for(dw_gate, DET_BF16) || !aligned_for(dw_up, DET_BF16))
    return fail(DET_EINVAL, "outputs must be aligned to their element size");
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (N == 0) {
    if (need_dw)
      for (void* p : {dw_gate, dw_up})
        hipLaunchKernelGGL(k_clear, dim3(static_cast<unsigned>(ceil_div(F * C, 256))), dim3(256), 0, s, static_cast<uint16_t*>(p), F * C);
    return need_dw ? hip_check(hipGetLastError(), "clearing launch") : DET_OK;
  }
  if (!need_dx && !need_dw) return DET_OK;
  if (dh == nullptr || gate == nullptr || up == nullptr || gate_exp == nullptr || up_exp == nullptr)
    return fail(DET_EINVAL, "null pointer");
  if (s_dh < 0) return fail(DET_EINVAL, "negative stride");
  if (!aligned_for(dh, dh_dt) || (save == DET_SAVE_HALF && (!aligned_for(gate, DET_BF16) || !aligned_for(up, DET_BF16))))
    return fail(DET_EINVAL, "operands must be aligned to their element size");
  if (need_dx && ((st = check_operand(w_gate, s_gate, "w_gate")) != DET_OK || (st = check_operand(w_up, s_up, "w_up")) != DET_OK))
    return st;
  if (need_dw) {
    if (x == nullptr || s_x < 0) return fail(DET_EINVAL, "null x or negative stride");
    if (x_exp == nullptr && !aligned_for(x, DET_BF16)) return fail(DET_EINVAL, "x must be aligned to its element size");
  }
  const GradRoom r = grad_room(N, C, F, need_dx, need_dw);
  if ((st = check_workspace(workspace, workspace_bytes, r.total)) != DET_OK) return st;
  char* const ws = static_cast<char*>(workspace);
  const int64_t Fp = up_to(F, 32), Np = up_to(N, 64);
  GateGradArgs g{};
  g.dh = dh; g.s_dh = s_dh; g.dh_dt = dh_dt;
  g.gate = gate; g.up = up; g.gate_exp = gate_exp; g.up_exp = up_exp;
  g.N = N; g.F = F; g.Fp = Fp; g.Np = Np; g.act = act; g.save = save;
  g.rows = need_dx ? ws : nullptr;
  g.turned = need_dw ? ws + r.rows : nullptr;
  hipLaunchKernelGGL(k_gate_grad, dim3(static_cast<unsigned>(ceil_div(Np, TILE)), static_cast<unsigned>(ceil_div(Fp, TILE))),
                     dim3(256), 0, s, g);
  if (need_dx) {
    char* const wt = ws + r.rows + r.turned + r.x;
    turn_rows(w_gate, s_gate, nullptr, F, C, Fp, wt, 2 * Fp, s);
    turn_rows(w_up, s_up, nullptr, F, C, Fp, wt + Fp * 2, 2 * Fp, s);
    MmArgs a{};
    a.A = wt; a.s_a = 2 * Fp; a.na = C;
    a.B = ws; a.s_b = 2 * Fp; a.nb = N;
    a.K = static_cast<int>(2 * Fp);
    a.out = dx; a.split = N; a.dt = DET_BF16;
    launch_mm<MM_ROWS>(a, s);
  }
  if (need_dw) {
    char* const xt = ws + r.rows + r.turned;
    turn_rows(x, s_x, x_exp, N, C, Np, xt, Np, s);
    MmArgs a{};
    a.A = xt; a.s_a = Np; a.na = C;
    a.B = ws + r.rows; a.s_b = Np; a.nb = 2 * F;
    a.K = static_cast<int>(Np);
    a.out = dw_gate; a.out1 = dw_up; a.split = F; a.dt = DET_BF16;
    launch_mm<MM_ROWS>(a, s);
  }
  return hip_check(hipGetLastError(), "gated projection gradient launch");
}

}  // extern "C"
