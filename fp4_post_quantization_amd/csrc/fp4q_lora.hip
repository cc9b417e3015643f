// Low-rank adapters of many requests beside a shared projection
// (include/fp4q_grouped.h): out = y + s (x A^T) B^T, A and B by the row's
// adapter, in two kernels on the bf16 matrix cores (v_mfma_f32_16x16x32_bf16;
// lane l takes row l % 16 and the 8 elements of K at 8 (l / 16), and register
// v of its accumulator holds row 4 (l / 16) + v, column l % 16).
//
//   shrink  u = s x A^T: 16 rows a workgroup, K shared by its four waves, and
//           where there are few rows by several workgroups.  Their sums meet
//           in LDS.  A row's u is taken on as bfloat16 parts, each the leading
//           bits of what the ones before leave: three hold float32's 24 bits
//           exactly.  For a bfloat16 result two do, the second rounded: they
//           are off by 2^-17 of u, 2^-9 of the result's own half step.
//           Workgroups that share K write float32 sums instead.
//   expand  y + u B^T, 256 columns a workgroup, 64 a wave, which keeps its part
//           of B in registers for up to 64 rows.  B's rows are the first
//           operand and u's the second, so a lane ends with several consecutive
//           columns of one row, which it adds to y and stores without any
//           exchange.
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
  void *u;  // one split: bfloat16 [parts][entries][rank]; else float32 [splits][entries][rank], without the scale
  uint32_t *status;
};

__device__ __forceinline__ bf16x8 load_bf16x8(const uint16_t *p) {
  return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4 *>(p));
}
__device__ __forceinline__ bf16x8 zero_bf16x8() { return __builtin_bit_cast(bf16x8, u32x4{0, 0, 0, 0}); }

constexpr int kLoraWaves = 4, kLoraThreads = 64 * kLoraWaves;

// The leading bits of z that bfloat16 holds (cut off, so that nothing overflows and the rest is exact); infinities and
// NaN, whose first bit is set, go into the first part alone.
template <int PARTS>
__device__ __forceinline__ void parts_of(float z, uint16_t p[PARTS]) {
  const bool finite = __builtin_fabsf(z) < __builtin_inff();
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    const uint32_t top = as_u(z) & 0xFFFF0000u;
    const uint32_t part = PARTS == 2 && i == 1 ? (uint32_t)fp4q_gemm::f32_to_bf16_rne(z) << 16 : top;
    p[i] = (uint16_t)((finite ? part : (i ? 0u : top | (z != z ? 0x400000u : 0u))) >> 16);
    z -= as_f(top);
  }
}

// Elements of a row of u's parts: padded, so that 16 rows read from LDS at once fall on different banks.
__host__ __device__ __forceinline__ int part_stride(int rank) { return rank + 8; }
// Elements of one part: room for the rows that a copy of 64 reads past the last one.
__host__ __device__ __forceinline__ int64_t part_size(int64_t entries, int rank) {
  return (entries + 64) * part_stride(rank);
}

// RT tiles of 16 ranks, MR of 16 rows, WAVES that share K; PARTS bfloat16 parts, or 0: float32 sums of a share of K.
// All workgroups of a group read the same A at about the same time, which is what bounds this kernel for many rows
// (A's rows lie a power of two apart and meet in few channels of the L2): two row tiles halve it.
template <int RT, int MR, int WAVES, int PARTS>
__global__ __launch_bounds__(64 * WAVES) void shrink_kernel(LoraArgs a) {
  constexpr int STEPS = RT <= 4 ? 4 : (RT == 8 ? 2 : 1);  // steps of K whose loads are in flight together
  __shared__ f32x4 part[WAVES][RT * MR][64];
  const int lane = threadIdx.x & 63, wave = wave_index(), r16 = lane & 15, h = lane >> 4;
  uint32_t err = 0;
  const RowTile t = find_tile(a.groups, 16 * MR, (int)blockIdx.x);
  if (blockIdx.x == 0 && blockIdx.y == 0 && wave == 0 && offsets_bad(a.groups)) err = FP4Q_DATA_BAD_GROUP;
  if (t.group >= 0) {
    const uint16_t *x[MR];
#pragma unroll
    for (int m = 0; m < MR; ++m) {
      const int row = t.lo + 16 * m + r16;
      int e = entry_at(a.groups, row < t.hi ? row : t.hi - 1);
      if (e < 0) {
        err = FP4Q_DATA_BAD_GROUP;
        e = 0;
      }
      x[m] = a.x + e * a.ld_x + 8 * h;
    }
    const uint16_t *w = a.a + (int64_t)t.group * a.rank * a.k + 8 * h;
    int64_t at[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int r = 16 * i + r16;
      at[i] = (int64_t)(r < a.rank ? r : a.rank - 1) * a.k;
    }
    const int steps = (a.k + 31) / 32, shares = a.splits * WAVES;
    const int share = (int)blockIdx.y * WAVES + wave, per = (steps + shares - 1) / shares;
    const int s0 = share * per, s1 = s0 + per < steps ? s0 + per : steps;
    f32x4 acc[RT][MR];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int m = 0; m < MR; ++m) acc[i][m] = f32x4{0, 0, 0, 0};
    for (int s = s0; s < s1; s += STEPS) {
      bf16x8 xv[STEPS][MR], wv[STEPS][RT];
#pragma unroll
      for (int q = 0; q < STEPS; ++q) {
        // past the wave's share or the end of K: an earlier piece of the row, which then meets zeros
        const int k0 = 32 * (s + q < s1 ? s + q : s1 - 1), off = k0 + 8 * h < a.k ? k0 : -8 * h;
#pragma unroll
        for (int m = 0; m < MR; ++m) xv[q][m] = load_bf16x8(x[m] + off);
#pragma unroll
        for (int i = 0; i < RT; ++i) wv[q][i] = load_bf16x8(w + at[i] + off);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int q = 0; q < STEPS; ++q) {
        const bool in = s + q < s1 && 32 * (s + q) + 8 * h < a.k;
        const bf16x8 z = zero_bf16x8();
        bf16x8 xq[MR];
#pragma unroll
        for (int m = 0; m < MR; ++m) xq[m] = in ? xv[q][m] : z;
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const bf16x8 wq = in ? wv[q][i] : z;
#pragma unroll
          for (int m = 0; m < MR; ++m)
            acc[i][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xq[m], wq, acc[i][m], 0, 0, 0);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int m = 0; m < MR; ++m) part[wave][i * MR + m][lane] = acc[i][m];
    __syncthreads();
    const float scale = PARTS && a.scales ? a.scales[t.group] : 1.0f;
    for (int i = wave; i < RT * MR; i += WAVES) {
      f32x4 sum = part[0][i][lane];
#pragma unroll
      for (int q = 1; q < WAVES; ++q) sum += part[q][i][lane];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int to = t.lo + 16 * (i % MR) + 4 * h + v, r = 16 * (i / MR) + r16;
        if (to >= t.hi || r >= a.rank) continue;
        if constexpr (PARTS == 0) {
          ((float *)a.u)[((int64_t)blockIdx.y * a.groups.entries + to) * a.rank + r] = sum[v];
        } else {
          uint16_t q[PARTS];
          parts_of<PARTS>(sum[v] * scale, q);
#pragma unroll
          for (int j = 0; j < PARTS; ++j)
            ((uint16_t *)a.u)[j * part_size(a.groups.entries, a.rank) + (int64_t)to * part_stride(a.rank) + r] = q[j];
        }
      }
    }
  }
  if (__builtin_expect(err != 0u, 0) || (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0))
    Status{a.status, true}.report(err);
}

// A lane's 16 columns of a wave's 64, in runs of 16 bytes whose neighbours the lanes of the same row have: register v
// of tile i of lane quarter h holds column 16 i + 4 h + v in float32, 32 (i / 2) + 8 h + 4 (i % 2) + v in bfloat16.
template <typename O>
__device__ __forceinline__ int column_of(int i, int h) {
  return sizeof(O) == 4 ? 16 * i + 4 * h : 32 * (i >> 1) + 8 * h + 4 * (i & 1);
}
struct LaneRow {
  u32x4 q[4];  // 16 float32, or in the first two 16 bfloat16
};
template <typename O>
__device__ __forceinline__ LaneRow load_lane(const O *p, int h) {
  LaneRow r;
#pragma unroll
  for (int i = 0; i < 16 / (16 / (int)sizeof(O)); ++i)
    r.q[i] = *reinterpret_cast<const u32x4 *>(p + column_of<O>(sizeof(O) == 4 ? i : 2 * i, h));
  return r;
}
__device__ __forceinline__ float lane_item(const LaneRow &r, float *, int k) { return as_f(r.q[k / 4][k % 4]); }
__device__ __forceinline__ float lane_item(const LaneRow &r, uint16_t *, int k) {
  const uint32_t w = r.q[k / 8][k / 2 % 4];
  return k % 2 ? as_f(w & 0xFFFF0000u) : as_f(w << 16);
}
__device__ __forceinline__ void store_lane(float *p, int h, const float z[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<f32x4 *>(p + column_of<float>(i, h)) = f32x4{z[4 * i], z[4 * i + 1], z[4 * i + 2], z[4 * i + 3]};
}
__device__ __forceinline__ void store_lane(uint16_t *p, int h, const float z[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    u32x4 w;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = fp4q_gemm::f32x2_to_bf16x2(z[8 * i + 2 * j], z[8 * i + 2 * j + 1]);
    *reinterpret_cast<u32x4 *>(p + column_of<uint16_t>(2 * i, h)) = w;
  }
}
__device__ __forceinline__ float load1(const uint16_t *p) { return as_f((uint32_t)*p << 16); }
__device__ __forceinline__ float load1(const float *p) { return *p; }

// RK steps of 32 ranks; ROWS rows (a multiple of 16) a workgroup.  SUMS: u is float32 sums of several workgroups, added
// and split here; else its parts, one run of memory, go straight to LDS.  Everything that a wave reads is asked for at
// once: its rows of y, u, and its columns of B.
template <int RK, int ROWS, bool SUMS, typename O>
__global__ __launch_bounds__(kLoraThreads) void expand_kernel(LoraArgs a) {
  constexpr int PARTS = sizeof(O) == 4 ? 3 : 2, TILES = ROWS / 16;
  constexpr int PART_BYTES = (ROWS * (32 * RK + 8) * 2 + 1023) / 1024 * 1024;  // LDS of a part, at most
  __shared__ __attribute__((aligned(1024))) uint8_t u_lds[SUMS ? 16 : PARTS * PART_BYTES];
  const int lane = threadIdx.x & 63, wave = wave_index(), r16 = lane & 15, h = lane >> 4;
  RowTile t = find_tile(a.groups, ROWS, (int)(blockIdx.x / a.tiles_n));
  const bool rest = t.group < 0;  // rows of no group
  if (rest) {
    if (a.in_place) return;
    const int last = a.groups.offsets[a.groups.groups];
    const int64_t first = (last < 0 ? 0 : (int64_t)last) + (int64_t)t.lo * ROWS;
    if (first >= a.groups.entries) return;
    t.lo = (int)first;
    t.hi = a.groups.entries - t.lo > ROWS ? t.lo + ROWS : a.groups.entries;
  }
  const int stride = part_stride(a.rank);
  if (!SUMS && !rest) {
    const int pieces = (ROWS * stride * 2 + 1023) / 1024;  // of 1 KB
#pragma unroll
    for (int q = 0; q < PARTS; ++q) {
      const uint8_t *src = (const uint8_t *)a.u + 2 * (q * part_size(a.groups.entries, a.rank) + (int64_t)t.lo * stride);
      for (int c = wave; c < pieces; c += kLoraWaves) {
        // the last piece ends with the tile's rows: lanes past them load its first bytes again
        const int at = 1024 * c + 16 * lane;
        fp4q_gemm::load_lds16(src + (at < ROWS * stride * 2 ? at : 0), u_lds + q * PART_BYTES + 1024 * c);
      }
    }
  }
  const int n0 = (int)(blockIdx.x % a.tiles_n) * 64 * kLoraWaves + 64 * wave;
  const bool live = n0 < a.n, whole = a.wide && n0 + 64 <= a.n;
  int entry[TILES];  // of this lane's row in each 16; -1: none
#pragma unroll
  for (int i = 0; i < TILES; ++i) {
    const int row = t.lo + 16 * i + r16;
    entry[i] = entry_at(a.groups, row < t.hi ? row : t.hi - 1);
    if (row >= t.hi) entry[i] |= -2147483647 - 1;  // read again, not stored
  }
  const O *y = (const O *)a.y + n0;
  O *out = (O *)a.out + n0;
  auto row_of = [&](int i) { return entry[i] == -1 ? 0 : entry[i] & 2147483647; };
  LaneRow old[TILES];
  if (whole) {
#pragma unroll
    for (int i = 0; i < TILES; ++i) old[i] = load_lane(y + (int64_t)row_of(i) * a.ld_y, h);
  }
  bf16x8 b[4][RK];
  float scale = 1.0f;
  bool in[RK];  // whether this lane's piece of a step lies within the rank
#pragma unroll
  for (int s = 0; s < RK; ++s) in[s] = 32 * s + 8 * h < a.rank;
  if (!rest) {
    if (SUMS && a.scales) scale = a.scales[t.group];
    const uint16_t *w = a.b + (int64_t)t.group * a.n * a.rank;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int col = n0 + column_of<O>(i, r16 >> 2) + (r16 & 3);
      const uint16_t *row = w + (int64_t)(col < a.n ? col : a.n - 1) * a.rank + 8 * h;
#pragma unroll
      for (int s = 0; s < RK; ++s) b[i][s] = in[s] ? load_bf16x8(row + 32 * s) : zero_bf16x8();
    }
  }
  if constexpr (!SUMS) __syncthreads();  // u has landed
  if (!live) return;
#pragma unroll
  for (int m = 0; m < TILES; ++m) {
    if (t.lo + 16 * m >= t.hi) break;
    f32x4 acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = f32x4{0, 0, 0, 0};
    if (!rest) {
#pragma unroll
      for (int s = 0; s < RK; ++s) {
        bf16x8 u[PARTS];
        if constexpr (SUMS) {
          const int row = t.lo + 16 * m + r16, p = row < t.hi ? row : t.hi - 1;
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = 0.0f;
          if (in[s])
            for (int q = 0; q < a.splits; ++q) {
              const f32x4 *at = reinterpret_cast<const f32x4 *>(
                  (const float *)a.u + ((int64_t)q * a.groups.entries + p) * a.rank + 32 * s + 8 * h);
              const f32x4 u0 = at[0], u1 = at[1];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                v[j] += u0[j];
                v[4 + j] += u1[j];
              }
            }
          uint32_t w[PARTS][4];
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            uint16_t q0[PARTS], q1[PARTS];
            parts_of<PARTS>(v[j] * scale, q0);
            parts_of<PARTS>(v[j + 1] * scale, q1);
#pragma unroll
            for (int i = 0; i < PARTS; ++i) w[i][j / 2] = q0[i] | (uint32_t)q1[i] << 16;
          }
#pragma unroll
          for (int i = 0; i < PARTS; ++i) u[i] = __builtin_bit_cast(bf16x8, u32x4{w[i][0], w[i][1], w[i][2], w[i][3]});
        } else {
          // past the rank: the next row's numbers or the padding, which are no numbers of this row
          const uint8_t *at = u_lds + ((16 * m + r16) * stride + 32 * s + 8 * h) * 2;
#pragma unroll
          for (int i = 0; i < PARTS; ++i)
            u[i] = in[s] ? *reinterpret_cast<const bf16x8 *>(at + i * PART_BYTES) : zero_bf16x8();
        }
#pragma unroll
        for (int q = PARTS - 1; q >= 0; --q)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[i][s], u[q], acc[i], 0, 0, 0);
      }
    }
    O *to = out + (int64_t)row_of(m) * a.ld_out;
    if (whole) {
      float z[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) z[k] = lane_item(old[m], (O *)nullptr, k) + acc[k / 4][k % 4];
      if (entry[m] >= 0) store_lane(to, h, z);
    } else {
      const O *from = y + (int64_t)row_of(m) * a.ld_y;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const int c = column_of<O>(k / 4, h) + k % 4;
        if (entry[m] >= 0 && n0 + c < a.n) fp4q_gemm::store_out(to + c, load1(from + c) + acc[k / 4][k % 4]);
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
  if (p.splits > 1) return 256 + (size_t)(p.splits * entries * rank * 4);
  return 256 + (size_t)(3 * part_size(entries, (int)rank) * 2);
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
                   out == y, wide, (char *)workspace + 256, status};
  const int64_t rows = lora_rows(p, rank, size);
  const int64_t tiles = l.tiles_n * (most_tiles(entries, groups->groups, rows) + 1);
  const int64_t mr = p.splits == 1 && rank <= 64 ? 2 : 1;
  const int64_t shrink_tiles = most_tiles(entries, groups->groups, 16 * mr);
  if (tiles > kMaxTiles || shrink_tiles > kMaxTiles) return FP4Q_ERR_SHAPE;
  auto shrink = [&](auto rt) {
    constexpr int RT = decltype(rt)::value, W = RT == 16 ? 4 : 8, MR = RT <= 4 ? 2 : 1;
    auto kernel = p.splits > 1 ? shrink_kernel<RT, 1, W, 0>
                               : (dtype == FP4Q_F32 ? shrink_kernel<RT, MR, W, 3> : shrink_kernel<RT, MR, W, 2>);
    hipLaunchKernelGGL(kernel, dim3((unsigned)shrink_tiles, (unsigned)p.splits), dim3(64 * W), 0, s, l);
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
      constexpr int MOST = sizeof(O) == 4 || RK == 8 ? 32 : 64;
      auto kernel = p.splits > 1 ? (rows == 16 ? expand_kernel<RK, 16, true, O> : expand_kernel<RK, MOST, true, O>)
                                 : (rows == 16 ? expand_kernel<RK, 16, false, O> : expand_kernel<RK, MOST, false, O>);
      hipLaunchKernelGGL(kernel, dim3((unsigned)tiles), dim3(kLoraThreads), 0, s, l);
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
