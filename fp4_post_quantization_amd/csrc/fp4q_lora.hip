// Low-rank adapters of many requests beside a shared projection
// (include/fp4q_grouped.h): out = y + s (x A^T) B^T, A and B by the row's
// adapter, in two kernels on the bf16 matrix cores (v_mfma_f32_16x16x32_bf16;
// lane l takes row l % 16 and the 8 elements of K at 8 (l / 16), and register
// v of its accumulator holds row 4 (l / 16) + v, column l % 16).
//
//   shrink  u = x A^T in float32, into the workspace; K split over waves and
//           workgroups where there are few rows.
//   expand  y + s u B^T: u s as three bfloat16 parts, each the 8 leading bits
//           of what the ones before leave, which hold float32's 24 bits
//           exactly.  B's rows are the first operand and u's the second, so a
//           lane ends with 16 consecutive columns of one row (tile i of a
//           wave's four takes columns 16 (m / 4) + 4 i + m % 4), which it
//           adds to y and stores without any exchange.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "fp4q.h"
#include "fp4q_device.h"
#include "fp4q_grouped.h"
#include "fp4q_grouped_device.h"
#include "fp4q_grouped_host.h"
#include "fp4q_mfma.h"

namespace fp4q {
namespace {

using fp4q_gemm::bf16x8;

struct LoraArgs {
  const void *y;
  const uint16_t *x, *a, *b;
  const float *scales;
  void *out;
  int64_t ld_y, ld_x, ld_out;
  Groups groups;
  int n, k, rank, splits, tiles_n;
  bool in_place, wide;
  float *u;  // [splits][entries][rank]
  uint32_t *status;
};

__device__ __forceinline__ bf16x8 load_bf16x8(const uint16_t *p) {
  return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4 *>(p));
}
__device__ __forceinline__ bf16x8 zero_bf16x8() { return __builtin_bit_cast(bf16x8, u32x4{0, 0, 0, 0}); }

constexpr int kLoraWaves = 4, kLoraThreads = 64 * kLoraWaves;

// RT tiles of 16 ranks.  SPLIT: a workgroup's waves share 16 rows, each a part of K; else each has 16 rows of 64.
template <int RT, bool SPLIT>
__global__ __launch_bounds__(kLoraThreads) void shrink_kernel(LoraArgs a) {
  constexpr int ROWS = SPLIT ? 16 : 16 * kLoraWaves;
  __shared__ f32x4 part[SPLIT ? kLoraWaves : 1][SPLIT ? RT : 1][64];
  const int lane = threadIdx.x & 63, wave = wave_index(), r16 = lane & 15, h = lane >> 4;
  uint32_t err = 0;
  const RowTile t = find_tile(a.groups, ROWS, (int)blockIdx.x);
  if (blockIdx.x == 0 && blockIdx.y == 0 && wave == 0 && offsets_bad(a.groups)) err = FP4Q_DATA_BAD_GROUP;
  if (t.group >= 0) {
    const int row = t.lo + r16 + (SPLIT ? 0 : 16 * wave);
    const int p = row < t.hi ? row : t.hi - 1;
    int e = entry_at(a.groups, p);
    if (e < 0) {
      err = FP4Q_DATA_BAD_GROUP;
      e = 0;
    }
    const uint16_t *x = a.x + e * a.ld_x + 8 * h;
    const uint16_t *w = a.a + (int64_t)t.group * a.rank * a.k + 8 * h;
    int64_t at[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int r = 16 * i + r16;
      at[i] = (int64_t)(r < a.rank ? r : a.rank - 1) * a.k;
    }
    const int steps = (a.k + 31) / 32, shares = a.splits * (SPLIT ? kLoraWaves : 1);
    const int share = (int)blockIdx.y * (SPLIT ? kLoraWaves : 1) + (SPLIT ? wave : 0);
    const int per = (steps + shares - 1) / shares;
    const int s0 = share * per, s1 = s0 + per < steps ? s0 + per : steps;
    f32x4 acc[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[i] = f32x4{0, 0, 0, 0};
    for (int s = s0; s < s1; ++s) {
      const bool in = 32 * s + 8 * h < a.k;
      const bf16x8 xv = in ? load_bf16x8(x + 32 * s) : zero_bf16x8();
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const bf16x8 wv = in ? load_bf16x8(w + at[i] + 32 * s) : zero_bf16x8();
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv, wv, acc[i], 0, 0, 0);
      }
    }
    float *u = a.u + (int64_t)blockIdx.y * a.groups.entries * a.rank;
    if constexpr (SPLIT) {
#pragma unroll
      for (int i = 0; i < RT; ++i) part[wave][i][lane] = acc[i];
      __syncthreads();
      for (int i = wave; i < RT; i += kLoraWaves) {
        f32x4 sum = part[0][i][lane];
#pragma unroll
        for (int q = 1; q < kLoraWaves; ++q) sum += part[q][i][lane];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int to = t.lo + 4 * h + v;
          if (to < t.hi && 16 * i + r16 < a.rank) u[(int64_t)to * a.rank + 16 * i + r16] = sum[v];
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int to = t.lo + 16 * wave + 4 * h + v;
          if (to < t.hi && 16 * i + r16 < a.rank) u[(int64_t)to * a.rank + 16 * i + r16] = acc[i][v];
        }
    }
  }
  if (__builtin_expect(err != 0u, 0) || (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0))
    Status{a.status, true}.report(err);
}

// The three bfloat16 parts of 8 float32 values: leading bits, cut off, so that every part and what it leaves is exact
// and nothing overflows.
struct Parts {
  bf16x8 p[3];
};
__device__ __forceinline__ Parts parts_of(const float v[8]) {
  uint32_t w[3][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t half[3][2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      float z = v[2 * j + q];
      const bool finite = __builtin_fabsf(z) < __builtin_inff();
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        // infinities and NaN (whose first bit stays set) go into the first part alone
        const uint32_t top = as_u(z) & 0xFFFF0000u;
        half[i][q] = finite || i == 0 ? (finite ? top : top | (z != z ? 0x400000u : 0u)) : 0u;
        z -= as_f(top);
      }
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) w[i][j] = half[i][0] >> 16 | half[i][1];
  }
  Parts r;
#pragma unroll
  for (int i = 0; i < 3; ++i) r.p[i] = __builtin_bit_cast(bf16x8, u32x4{w[i][0], w[i][1], w[i][2], w[i][3]});
  return r;
}

__device__ __forceinline__ void load16_row(const uint16_t *p, float z[16]) {
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const u32x4 w = reinterpret_cast<const u32x4 *>(p)[q];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      z[8 * q + 2 * i] = as_f(w[i] << 16);
      z[8 * q + 2 * i + 1] = as_f(w[i] & 0xFFFF0000u);
    }
  }
}
__device__ __forceinline__ void load16_row(const float *p, float z[16]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const f32x4 w = reinterpret_cast<const f32x4 *>(p)[q];
#pragma unroll
    for (int i = 0; i < 4; ++i) z[4 * q + i] = w[i];
  }
}
__device__ __forceinline__ void store16_row(uint16_t *p, const float z[16]) {
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = fp4q_gemm::f32x2_to_bf16x2(z[8 * q + 2 * i], z[8 * q + 2 * i + 1]);
    reinterpret_cast<u32x4 *>(p)[q] = w;
  }
}
__device__ __forceinline__ void store16_row(float *p, const float z[16]) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    reinterpret_cast<f32x4 *>(p)[q] = f32x4{z[4 * q], z[4 * q + 1], z[4 * q + 2], z[4 * q + 3]};
}
__device__ __forceinline__ float load1(const uint16_t *p) { return as_f((uint32_t)*p << 16); }
__device__ __forceinline__ float load1(const float *p) { return *p; }

// RK steps of 32 ranks; ROWS rows (a multiple of 16) times 256 columns a workgroup, 64 a wave.
template <int RK, int ROWS, typename O>
__global__ __launch_bounds__(kLoraThreads) void expand_kernel(LoraArgs a) {
  const int lane = threadIdx.x & 63, wave = wave_index(), r16 = lane & 15, h = lane >> 4;
  const int tile = (int)(blockIdx.x / a.tiles_n);
  RowTile t = find_tile(a.groups, ROWS, tile);
  const bool rest = t.group < 0;  // rows of no group
  if (rest) {
    if (a.in_place) return;
    const int last = a.groups.offsets[a.groups.groups];
    const int64_t first = (last < 0 ? 0 : (int64_t)last) + (int64_t)t.lo * ROWS;
    if (first >= a.groups.entries) return;
    t.lo = (int)first;
    t.hi = a.groups.entries - t.lo > ROWS ? t.lo + ROWS : a.groups.entries;
  }
  const int n0 = (int)(blockIdx.x % a.tiles_n) * 64 * kLoraWaves + 64 * wave;
  if (n0 >= a.n) return;
  bf16x8 b[4][RK];
  float scale = 1.0f;
  if (!rest) {
    if (a.scales) scale = a.scales[t.group];
    const uint16_t *w = a.b + (int64_t)t.group * a.n * a.rank;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int col = n0 + 16 * (r16 >> 2) + 4 * i + (r16 & 3);
      const uint16_t *row = w + (int64_t)(col < a.n ? col : a.n - 1) * a.rank + 8 * h;
#pragma unroll
      for (int s = 0; s < RK; ++s) b[i][s] = 32 * s + 8 * h < a.rank ? load_bf16x8(row + 32 * s) : zero_bf16x8();
    }
  }
  const int c0 = n0 + 16 * h;  // this lane's 16 columns
  const bool whole = a.wide && c0 + 16 <= a.n;
  const O *y = (const O *)a.y;
  O *out = (O *)a.out;
#pragma unroll 1
  for (int m = 0; m < ROWS && t.lo + m < t.hi; m += 16) {
    const int row = t.lo + m + r16, p = row < t.hi ? row : t.hi - 1;
    const int e = entry_at(a.groups, p);
    float z[16];
    const O *from = y + (int64_t)(e < 0 ? 0 : e) * a.ld_y + c0;
    if (whole) {
      load16_row(from, z);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) z[i] = c0 + i < a.n ? load1(from + i) : 0.0f;
    }
    f32x4 acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = f32x4{0, 0, 0, 0};
    if (!rest) {
#pragma unroll
      for (int s = 0; s < RK; ++s) {
        const bool in = 32 * s + 8 * h < a.rank;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
        if (in)
          for (int q = 0; q < a.splits; ++q) {
            const f32x4 *u = reinterpret_cast<const f32x4 *>(
                a.u + ((int64_t)q * a.groups.entries + p) * a.rank + 32 * s + 8 * h);
            const f32x4 u0 = u[0], u1 = u[1];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              v[j] += u0[j];
              v[4 + j] += u1[j];
            }
          }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= scale;
        const Parts w = parts_of(v);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int q = 2; q >= 0; --q)
            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[i][s], w.p[q], acc[i], 0, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) z[4 * i + v] += acc[i][v];
    if (row < t.hi && e >= 0) {
      O *to = out + (int64_t)e * a.ld_out + c0;
      if (whole) {
        store16_row(to, z);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (c0 + i < a.n) fp4q_gemm::store_out(to + i, z[i]);
      }
    }
  }
}

__global__ __launch_bounds__(64) void lora_status_kernel(uint32_t *status) {
  if (threadIdx.x == 0) Status{status, true}.merge(0u);
}

fp4q_status_t hip_status() { return hipGetLastError() == hipSuccess ? FP4Q_OK : FP4Q_ERR_HIP; }

}  // namespace
}  // namespace fp4q

using namespace fp4q;

extern "C" size_t fp4q_lora_add_workspace_bytes(int64_t entries, int64_t groups, int64_t n, int64_t k, int64_t rank) {
  if (lora_check_sizes(entries, groups, n, k, rank) != FP4Q_OK) return 0;
  const LoraPlan p = lora_plan(entries, groups, k);
  return 256 + (size_t)(p.splits * entries * rank * 4);
}

extern "C" fp4q_status_t fp4q_lora_add(const void *y, fp4q_dtype_t dtype, int64_t ld_y, const void *x, int64_t ld_x,
                                       const void *a, const void *b, const float *scales,
                                       const fp4q_row_groups_t *groups, int64_t n, int64_t k, int64_t rank, void *out,
                                       int64_t ld_out, void *workspace, size_t workspace_bytes, void *stream) {
  if (!groups) return FP4Q_ERR_NULL;
  if (dtype != FP4Q_F32 && dtype != FP4Q_BF16) return FP4Q_ERR_ARG;
  fp4q_status_t st = grouped_check(*groups);
  if (st != FP4Q_OK) return st;
  const int64_t entries = groups->entries, size = dtype == FP4Q_F32 ? 4 : 2;
  if ((st = lora_check_sizes(entries, groups->groups, n, k, rank)) != FP4Q_OK) return st;
  if (!grouped_rows_ok(entries, n, ld_y, size) || !grouped_rows_ok(entries, n, ld_out, size) ||
      !grouped_rows_ok(entries, k, ld_x, 2))
    return FP4Q_ERR_SHAPE;
  if (!grouped_ws_ok(workspace, workspace_bytes, fp4q_lora_add_workspace_bytes(entries, groups->groups, n, k, rank)))
    return FP4Q_ERR_WORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  uint32_t *status = (uint32_t *)workspace;
  if (entries == 0 || n == 0) {
    hipLaunchKernelGGL(lora_status_kernel, dim3(1), dim3(64), 0, s, status);
    return hip_status();
  }
  if (!y || !x || !a || !b || !out) return FP4Q_ERR_NULL;
  if (!kv_aligned(x, 16) || !kv_aligned(a, 16) || !kv_aligned(b, 16) || ld_x % 8 || !kv_aligned(scales, 4) ||
      !kv_aligned(y, size) || !kv_aligned(out, size))
    return FP4Q_ERR_ALIGN;
  if (out == y && ld_out != ld_y) return FP4Q_ERR_ARG;
  const LoraPlan p = lora_plan(entries, groups->groups, k);
  const bool wide = kv_aligned(y, 16) && kv_aligned(out, 16) && ld_y * size % 16 == 0 && ld_out * size % 16 == 0;
  const LoraArgs l{y, (const uint16_t *)x, (const uint16_t *)a, (const uint16_t *)b, scales, out, ld_y, ld_x, ld_out,
                   groups_of(*groups), (int)n, (int)k, (int)rank, (int)p.splits, (int)ceil_div(n, 64 * kLoraWaves),
                   out == y, wide, (float *)((char *)workspace + 256), status};
  const int64_t tiles = l.tiles_n * (most_tiles(entries, groups->groups, p.few ? 16 : 64) + 1);
  if (tiles > kMaxTiles) return FP4Q_ERR_SHAPE;
  const dim3 shrink_grid((unsigned)most_tiles(entries, groups->groups, p.few ? 16 : 64), (unsigned)p.splits);
  auto shrink = [&](auto rt) {
    constexpr int RT = decltype(rt)::value;
    if (p.few) hipLaunchKernelGGL((shrink_kernel<RT, true>), shrink_grid, dim3(kLoraThreads), 0, s, l);
    else hipLaunchKernelGGL((shrink_kernel<RT, false>), shrink_grid, dim3(kLoraThreads), 0, s, l);
  };
  if (rank <= 16) shrink(std::integral_constant<int, 1>{});
  else if (rank <= 32) shrink(std::integral_constant<int, 2>{});
  else if (rank <= 64) shrink(std::integral_constant<int, 4>{});
  else if (rank <= 128) shrink(std::integral_constant<int, 8>{});
  else shrink(std::integral_constant<int, 16>{});
  auto expand = [&](auto rk) {
    constexpr int RK = decltype(rk)::value;
    auto go = [&](auto op) {
      using O = std::remove_pointer_t<decltype(op)>;
      if (p.few) hipLaunchKernelGGL((expand_kernel<RK, 16, O>), dim3((unsigned)tiles), dim3(kLoraThreads), 0, s, l);
      else hipLaunchKernelGGL((expand_kernel<RK, 64, O>), dim3((unsigned)tiles), dim3(kLoraThreads), 0, s, l);
    };
    if (dtype == FP4Q_F32) go((float *)nullptr);
    else go((uint16_t *)nullptr);
  };
  if (rank <= 32) expand(std::integral_constant<int, 1>{});
  else if (rank <= 64) expand(std::integral_constant<int, 2>{});
  else if (rank <= 128) expand(std::integral_constant<int, 4>{});
  else expand(std::integral_constant<int, 8>{});
  return hip_status();
}
