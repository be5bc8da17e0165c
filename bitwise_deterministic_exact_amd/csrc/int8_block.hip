// 8-bit checkpoints (int8_block.h) for MI355X (gfx950): rows written and read
// back.  One pass each, bound by HBM: 16384 x 8192 bf16 in 76 us either way, 407
// MB at 5.3 TB/s.
#include <algorithm>

#include "int8_block.h"

#pragma clang fp contract(off)

namespace {

using namespace rowops;

// Eight elements to a thread (16 bytes of bf16, 8 of codes), four threads to a
// block.  Rows that follow each other without a gap and hold whole blocks are
// one long row: no division per thread.
constexpr int PER = 8, UNITS = 4;         // of a thread, blocks of 256 threads apart

struct PackArgs {
  const void* x; int64_t s_x;             // pack: x; unpack: the codes
  int64_t N, C;
  int64_t per_row, total;                 // units of PER elements, a multiple of 4 to a row
  int8_t* codes; int8_t* exps;
  void* y;
  int32_t* status;
};

struct Unit {
  int64_t row, c;
  int n;                                  // elements of it that are inside
};
__device__ __forceinline__ Unit unit_at(const PackArgs& a, int64_t i) {
  Unit u;
  u.row = a.N == 1 ? 0 : a.total <= 0xFFFFFFFFll ? static_cast<uint32_t>(i) / static_cast<uint32_t>(a.per_row) : i / a.per_row;
  u.c = (i - u.row * a.per_row) * PER;
  u.n = i < a.total ? static_cast<int>(max<int64_t>(0, min<int64_t>(PER, a.C - u.c))) : 0;
  return u;
}

template <int DT>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&v)[PER], int n) {
  if (n == PER) {
    load_vec<DT, PER>(p, i, v);
  } else {
#pragma unroll
    for (int k = 0; k < PER; ++k) v[k] = k < n ? load_elem<DT>(p, i + k) : 0.0f;
  }
}

struct __attribute__((packed, aligned(1))) CodePair {
  uint32_t w[2];
};

template <int DT>
__global__ __launch_bounds__(256) void k_int8_pack(PackArgs a) {
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * 256 * UNITS + threadIdx.x;
  Unit u[UNITS];
  float v[UNITS][PER];
#pragma unroll
  for (int k = 0; k < UNITS; ++k) {
    u[k] = unit_at(a, i0 + 256 * k);
    load8<DT>(a.x, u[k].row * a.s_x + u[k].c, v[k], u[k].n);
  }
#pragma unroll
  for (int k = 0; k < UNITS; ++k) {
    uint32_t top = 0u;
#pragma unroll
    for (int e = 0; e < PER; ++e) top = max(top, magnitude(v[k][e]));
    top = max(top, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(top), 0xB1, 0xF, 0xF, false)));
    top = max(top, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(top), 0x4E, 0xF, 0xF, false)));
    const bool bad = not_finite(top);
    const int e = block_exponent(top);
    const float inv = power_of_two(-e);
    if (u[k].n <= 0) continue;
    const int64_t at = u[k].row * a.C + u[k].c;
    if ((threadIdx.x & 3) == 0) {
      a.exps[u[k].row * (a.per_row / 4) + u[k].c / INT8_BLOCK] = static_cast<int8_t>(bad ? DET_INT8_NAN : e);
      if (bad) a.status[0] = 1;
    }
    const float lo[4] = {v[k][0], v[k][1], v[k][2], v[k][3]}, hi[4] = {v[k][4], v[k][5], v[k][6], v[k][7]};
    const CodePair w = {{codes_of(lo, inv, bad), codes_of(hi, inv, bad)}};
    if (u[k].n == PER) {
      *reinterpret_cast<CodePair*>(a.codes + at) = w;
    } else {
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if (j < u[k].n) a.codes[at + j] = static_cast<int8_t>(w.w[j / 4] >> (8 * (j & 3)));
    }
  }
}

template <int DT>
__global__ __launch_bounds__(256) void k_int8_unpack(PackArgs a) {
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * 256 * UNITS + threadIdx.x;
  Unit u[UNITS];
  CodePair w[UNITS];
  int8_t e[UNITS];
#pragma unroll
  for (int k = 0; k < UNITS; ++k) {
    u[k] = unit_at(a, i0 + 256 * k);
    w[k] = {{0u, 0u}};
    e[k] = 0;
    if (u[k].n <= 0) continue;
    const int8_t* const from = static_cast<const int8_t*>(a.x) + u[k].row * a.s_x + u[k].c;
    if (u[k].n == PER) {
      w[k] = *reinterpret_cast<const CodePair*>(from);
    } else {
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if (j < u[k].n) w[k].w[j / 4] |= static_cast<uint32_t>(static_cast<uint8_t>(from[j])) << (8 * (j & 3));
    }
    e[k] = a.exps[u[k].row * (a.per_row / 4) + u[k].c / INT8_BLOCK];
  }
#pragma unroll
  for (int k = 0; k < UNITS; ++k) {
    if (u[k].n <= 0) continue;
    const float unit = unit_of(e[k]);
    float lo[4], hi[4];
    values_of(w[k].w[0], unit, lo);
    values_of(w[k].w[1], unit, hi);
    const float v[PER] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    const int64_t at = u[k].row * a.C + u[k].c;
    if (u[k].n == PER) {
      store_vec<DT, PER>(a.y, at, v);
    } else {
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if (j < u[k].n) store_elem<DT>(a.y, at + j, v[j]);
    }
  }
}

constexpr int64_t ROWS_MAX = int64_t{1} << 31, COLS_MAX = int64_t{1} << 24;

det_status check_block_rows(int dt, int64_t s, int64_t N, int64_t C) {
  if (!known_dtype(dt)) return fail(DET_EDTYPE, "unknown dtype %d", dt);
  if (N < 0 || C < 1 || s < 0) return fail(DET_EINVAL, "bad size or stride: N=%lld C=%lld stride=%lld", (long long)N,
                                           (long long)C, (long long)s);
  if (N > ROWS_MAX || C > COLS_MAX) return fail(DET_EINVAL, "N = %lld and C = %lld exceed the limits 2^31 and 2^24",
                                                (long long)N, (long long)C);
  return DET_OK;
}

// one long row where there is no gap and no ragged block; false: more threads than one launch takes (2^32)
bool lay_out(PackArgs& a) {
  if (a.s_x == a.C && a.C % INT8_BLOCK == 0) {
    a.C *= a.N;
    a.s_x = a.C;
    a.N = 1;
  }
  a.per_row = ceil_div(a.C, INT8_BLOCK) * (INT8_BLOCK / PER);
  a.total = a.N * a.per_row;
  return a.total <= int64_t{1} << 33;
}

}  // namespace

extern "C" {

det_status det_int8_pack(det_dtype dt, const void* x, int64_t s_x, int64_t N, int64_t C, int8_t* codes, int8_t* exps,
                         void* stream) {
  det_status st = check_block_rows(dt, s_x, N, C);
  if (st != DET_OK || N == 0) return st;
  if (x == nullptr || codes == nullptr || exps == nullptr) return fail(DET_EINVAL, "null pointer");
  if (!aligned_for(x, dt)) return fail(DET_EINVAL, "x must be aligned to its element size");
  PackArgs a{};
  a.x = x; a.s_x = s_x; a.N = N; a.C = C; a.codes = codes; a.exps = exps;
  if (!lay_out(a)) return fail(DET_EINVAL, "more than 2^36 elements in one call");
  a.status = det_device_status_word();
  if (a.status == nullptr) return DET_EHIP;
  const dim3 grid(static_cast<unsigned>(ceil_div(a.total, 256 * UNITS)));
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dt == DET_F32) hipLaunchKernelGGL(k_int8_pack<DET_F32>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(k_int8_pack<DET_BF16>, grid, dim3(256), 0, s, a);
  return hip_check(hipGetLastError(), "8-bit pack launch");
}

det_status det_int8_unpack(const int8_t* codes, int64_t s_codes, const int8_t* exps, int64_t N, int64_t C,
                           det_dtype dt, void* y, void* stream) {
  det_status st = check_block_rows(dt, s_codes, N, C);
  if (st != DET_OK || N == 0) return st;
  if (codes == nullptr || exps == nullptr || y == nullptr) return fail(DET_EINVAL, "null pointer");
  if (!aligned_for(y, dt)) return fail(DET_EINVAL, "y must be aligned to its element size");
  PackArgs a{};
  a.x = codes; a.s_x = s_codes; a.N = N; a.C = C; a.exps = const_cast<int8_t*>(exps); a.y = y;
  if (!lay_out(a)) return fail(DET_EINVAL, "more than 2^36 elements in one call");
  const dim3 grid(static_cast<unsigned>(ceil_div(a.total, 256 * UNITS)));
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dt == DET_F32) hipLaunchKernelGGL(k_int8_unpack<DET_F32>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(k_int8_unpack<DET_BF16>, grid, dim3(256), 0, s, a);
  return hip_check(hipGetLastError(), "8-bit unpack launch");
}

}  // extern "C"
