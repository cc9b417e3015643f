// Low-rank adapters of many requests beside a shared projection
// (include/fp4q_grouped.h): out = y + s (x A^T) B^T, A and B by the row's
// adapter, in two kernels on the bf16 matrix cores (v_mfma_f32_16x16x32_bf16;
// lane l takes row l % 16 and the 8 elements of K at 8 (l / 16), and register
// v of its accumulator holds row 4 (l / 16) + v, column l % 16).
//
//   shrink  u = s x A^T: 16 or 32 rows a workgroup, K shared by its four waves,
//           and where there are few rows by several workgroups.  Their sums
//           meet in LDS.  A row's u is taken on as three bfloat16 parts, each
//           the leading bits of what the ones before leave, which hold float32's
//           24 bits exactly, whatever the result's type: where terms of u B^T,
//           or y and u B^T, cancel, a bfloat16 result shows them too.  (Two
//           parts, off by up to 2^-16 of u: 120 us instead of 130 for 8191 rows,
//           rank 64, K 4096, 14336 columns.)
//           Workgroups that share K write float32 sums instead.
//   expand  y + u B^T, 256 columns a workgroup, 64 a wave, which keeps its part
//           of B in registers for up to 64 rows.  Column 4 q + i of the wave's
//           64 is column q of tile i, so that a lane ends with four consecutive
//           columns of a row and 16 lanes with all 64, which they add to y and
//           store without any exchange.
//
// Both read through LDS what the matrix core wants by rows: a load of 16 bytes a
// lane takes 16 cycles where its first 16 lanes read one run of memory, and 64
// where they read 16 rows (8191 rows, rank 64, K 4096: shrink 31 us so, 21 by
// LDS; expand to 14336 columns, with two parts of u, 115 with y and out in the
// operand's layout too, and 90; with all three parts 95; 64 requests on 32
// adapters, rank 64, N 4096: 9.6 -> 5.0).  Then y and out bound it for many rows
// (5.0 TB/s), B and two launches for few.
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
  void *u;  // one split: bfloat16 [kParts][entries][rank]; else float32 [splits][entries][rank], without the scale
  uint32_t *status;
};

__device__ __forceinline__ bf16x8 zero_bf16x8() { return __builtin_bit_cast(bf16x8, u32x4{0, 0, 0, 0}); }

constexpr int kLoraWaves = 4, kLoraThreads = 64 * kLoraWaves;

constexpr int kParts = 3;

// The leading bits of z that bfloat16 holds (cut off, so that nothing overflows and the rest is exact); infinities and
// NaN, whose first bit is set, go into the first part alone.
__device__ __forceinline__ void parts_of(float z, uint16_t p[kParts]) {
  const bool finite = __builtin_fabsf(z) < __builtin_inff();
#pragma unroll
  for (int i = 0; i < kParts; ++i) {
    const uint32_t top = as_u(z) & 0xFFFF0000u;
    p[i] = (uint16_t)((finite ? top : (i ? 0u : top | (z != z ? 0x400000u : 0u))) >> 16);
    z -= as_f(top);
  }
}

// Elements of a row of u's parts: padded, so that 16 rows read from LDS at once fall on different banks.
__host__ __device__ __forceinline__ int part_stride(int rank) { return rank + 8; }
// Elements of one part: room for the rows that a copy of 64 reads past the last one.
__host__ __device__ __forceinline__ int64_t part_size(int64_t entries, int rank) {
  return (entries + 64) * part_stride(rank);
}

// RT tiles of 16 ranks, MR of 16 rows, WAVES that share K; SUMS: float32 sums of a share of K, else u's parts.
//
// A wave copies 64 elements of K of its rows of x and of A at a time to its own part of the LDS, NS such stages in
// flight, and reads its operands there: a load of 16 bytes a lane straight into the operand's layout has 16 rows in its
// first 16 lanes, and such a load takes the 64 cycles of 64 lines.  16-byte piece p of row r lies at p ^ (r / 2 % 8) of
// its 128 bytes, so that 16 rows read at once fall on all banks.
template <int RT, int MR, int WAVES, int NS, bool SUMS>
__global__ __launch_bounds__(64 * WAVES) void shrink_kernel(LoraArgs a) {
  constexpr int LOADS = 2 * (MR + RT), STAGE = 1024 * LOADS;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[WAVES * NS * STAGE];
  static_assert(RT * MR <= NS * LOADS, "the waves' sums lie where their stages were");
  const int lane = threadIdx.x & 63, wave = wave_index(), r16 = lane & 15, h = lane >> 4;
  uint32_t err = 0;
  const RowTile t = find_tile(a.groups, 16 * MR, (int)blockIdx.x);
  if (blockIdx.x == 0 && blockIdx.y == 0 && wave == 0 && offsets_bad(a.groups)) err = FP4Q_DATA_BAD_GROUP;
  if (t.group >= 0) {
    const int row8 = lane >> 3;  // of the eight rows of a load
    int64_t x[2 * MR];
#pragma unroll
    for (int j = 0; j < 2 * MR; ++j) {
      const int row = t.lo + 8 * j + row8;
      int e = entry_at(a.groups, row < t.hi ? row : t.hi - 1);
      if (e < 0) {
        err = FP4Q_DATA_BAD_GROUP;
        e = 0;
      }
      x[j] = e * a.ld_x;
    }
    const uint16_t *w = a.a + ((int64_t)t.group * a.rank + row8) * a.k;
    const int eights = a.rank / 8, piece = 8 * ((lane & 7) ^ (row8 >> 1));
    const int stages = (a.k + 63) / 64, shares = a.splits * WAVES;
    const int share = (int)blockIdx.y * WAVES + wave, per = (stages + shares - 1) / shares;
    const int s0 = share * per, s1 = s0 + per < stages ? s0 + per : stages;
    uint8_t *mine = lds + wave * NS * STAGE;
    auto load = [&](int s, int slot) {
      int at[2];  // elements past the end of K: the row's first ones
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int k = 64 * s + (piece ^ (32 * i));
        at[i] = k < a.k ? k : 0;
      }
#pragma unroll
      for (int j = 0; j < 2 * MR; ++j) fp4q_gemm::load_lds16(a.x + x[j] + at[j & 1], mine + slot * STAGE + 1024 * j);
#pragma unroll
      for (int j = 0; j < 2 * RT; ++j)  // past the rank: its last rows, whose columns are not stored
        fp4q_gemm::load_lds16(w + (int64_t)(8 * (j < eights ? j : eights - 1)) * a.k + at[j & 1],
                              mine + slot * STAGE + 1024 * (2 * MR + j));
    };
    f32x4 acc[RT][MR];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int m = 0; m < MR; ++m) acc[i][m] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < NS; ++s)
      if (s0 + s < s1) load(s0 + s, s);
    int slot = 0;
    for (int s = s0; s < s1; ++s) {
      if (NS > 1 && s + NS <= s1) fp4q_gemm::wait_vmcnt<(NS - 1) * LOADS>();
      else fp4q_gemm::wait_vmcnt<0>();
      __atomic_signal_fence(__ATOMIC_SEQ_CST);
      __builtin_amdgcn_sched_barrier(0);
      bf16x8 xv[2][MR], wv[2][RT];
      const uint8_t *from = mine + slot * STAGE + r16 * 128;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint8_t *at = from + 16 * ((4 * q + h) ^ (r16 >> 1));
#pragma unroll
        for (int m = 0; m < MR; ++m) xv[q][m] = *reinterpret_cast<const bf16x8 *>(at + 2048 * m);
#pragma unroll
        for (int i = 0; i < RT; ++i) wv[q][i] = *reinterpret_cast<const bf16x8 *>(at + 2048 * (MR + i));
      }
      if (64 * s + 64 > a.k) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const bool in = 64 * s + 32 * q + 8 * h < a.k;
          const bf16x8 z = zero_bf16x8();
#pragma unroll
          for (int m = 0; m < MR; ++m) xv[q][m] = in ? xv[q][m] : z;
#pragma unroll
          for (int i = 0; i < RT; ++i) wv[q][i] = in ? wv[q][i] : z;
        }
      }
      fp4q_gemm::wait_lgkmcnt0();
      __atomic_signal_fence(__ATOMIC_SEQ_CST);
      __builtin_amdgcn_sched_barrier(0);
      if (s + NS < s1) load(s + NS, slot);
      slot = slot == NS - 1 ? 0 : slot + 1;
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int m = 0; m < MR; ++m)
            acc[i][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv[q][m], wv[q][i], acc[i][m], 0, 0, 0);
    }
    // the waves' sums [wave][tile][lane], in the part of the LDS that the wave itself used
    f32x4 *part = reinterpret_cast<f32x4 *>(lds);
    constexpr int WAVE_PART = NS * STAGE / 16;
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int m = 0; m < MR; ++m) part[wave * WAVE_PART + (i * MR + m) * 64 + lane] = acc[i][m];
    __syncthreads();
    const float scale = !SUMS && a.scales ? a.scales[t.group] : 1.0f;
    for (int i = wave; i < RT * MR; i += WAVES) {
      f32x4 sum = part[i * 64 + lane];
#pragma unroll
      for (int q = 1; q < WAVES; ++q) sum += part[q * WAVE_PART + i * 64 + lane];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int to = t.lo + 16 * (i % MR) + 4 * h + v, r = 16 * (i / MR) + r16;
        if (to >= t.hi || r >= a.rank) continue;
        if constexpr (SUMS) {
          ((float *)a.u)[((int64_t)blockIdx.y * a.groups.entries + to) * a.rank + r] = sum[v];
        } else {
          uint16_t q[kParts];
          parts_of(sum[v] * scale, q);
#pragma unroll
          for (int j = 0; j < kParts; ++j)
            ((uint16_t *)a.u)[j * part_size(a.groups.entries, a.rank) + (int64_t)to * part_stride(a.rank) + r] = q[j];
        }
      }
    }
  }
  if (__builtin_expect(err != 0u, 0) || (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0))
    Status{a.status, true}.report(err);
}

// Four consecutive values of a row.
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
template <typename O>
struct Four;
template <>
struct Four<float> {
  f32x4 v;
  __device__ __forceinline__ float at(int i) const { return v[i]; }
};
template <>
struct Four<uint16_t> {
  u32x2 v;
  __device__ __forceinline__ float at(int i) const { return as_f(i % 2 ? v[i / 2] & 0xFFFF0000u : v[i / 2] << 16); }
};
__device__ __forceinline__ void store_four(float *p, const float z[4]) {
  *reinterpret_cast<f32x4 *>(p) = f32x4{z[0], z[1], z[2], z[3]};
}
__device__ __forceinline__ void store_four(uint16_t *p, const float z[4]) {
  *reinterpret_cast<u32x2 *>(p) = u32x2{fp4q_gemm::f32x2_to_bf16x2(z[0], z[1]), fp4q_gemm::f32x2_to_bf16x2(z[2], z[3])};
}
__device__ __forceinline__ float load1(const uint16_t *p) { return as_f((uint32_t)*p << 16); }
__device__ __forceinline__ float load1(const float *p) { return *p; }

// RK steps of 32 ranks; ROWS rows (a multiple of 16) a workgroup.  SUMS: u is float32 sums of several workgroups,
// added and split here; else its parts, one run of memory, go straight to LDS.  So do a wave's 64 columns of B, up to
// 128 ranks (64 beside many rows, whose u takes the room) at a time, on their way to its registers; but for TURNS
// everything that a wave reads is asked for at once.
template <int RK, int ROWS, bool SUMS, typename O>
__global__ __launch_bounds__(kLoraThreads) void expand_kernel(LoraArgs a) {
  constexpr int TILES = ROWS / 16;
  constexpr int PART_BYTES = (ROWS * (32 * RK + 8) * 2 + 1023) / 1024 * 1024;  // LDS of a part, at most
  constexpr int MOST_B = ROWS == 16 ? 4 : 2, BK = RK < MOST_B ? RK : MOST_B;  // steps of B a round
  constexpr int B_BYTES = 4096 * BK;                                          // LDS of a wave's
  constexpr int U_BYTES = kParts * PART_BYTES, ALL_B = kLoraWaves * B_BYTES;
  // Where three workgroups would not fit a CU's LDS with both, u takes B's place once B is in registers: 8191 rows of
  // rank 64 on 14336 columns 139 -> 130 us, 2000 of rank 256 on 4096 64 -> 54.  For few rows, which a second trip to
  // memory would cost more, and where they fit (rank 16: 36.6 us, in turns 37.7) both are asked for at once.
  constexpr bool TURNS = ROWS > 16 && U_BYTES + ALL_B > 53 * 1024;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[!TURNS ? U_BYTES + ALL_B : (U_BYTES > ALL_B ? U_BYTES : ALL_B)];
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
  const int n0 = (int)(blockIdx.x % a.tiles_n) * 64 * kLoraWaves + 64 * wave;
  const bool live = n0 < a.n;
  // Slot c / (4 BK) of a wave's part of LDS holds column 4 q + i of tile i, q = slot % 16, whose 16-byte pieces lie so
  // that the 16 columns read at once fall on all banks; pieces past the rank are its last one again, and not used.
  auto shuffle = [](int q) { return BK == 1 ? q >> 2 & 3 : (BK == 2 ? q >> 1 & 7 : q); };
  uint8_t *b_lds = lds + (TURNS ? 0 : U_BYTES) + wave * B_BYTES;
  const uint16_t *w = a.b + ((int64_t)t.group * a.n + n0) * a.rank;
  auto load_b = [&](int round) {
    const int most = a.n - 1 - n0, pieces = a.rank / 8;
#pragma unroll
    for (int j = 0; j < 4 * BK; ++j) {
      const int slot = 16 / BK * j + lane / (4 * BK), q = slot & 15, col = 4 * q + (slot >> 4);
      const int piece = 4 * BK * round + ((lane & (4 * BK - 1)) ^ shuffle(q));
      fp4q_gemm::load_lds16(w + (col < most ? col : most) * a.rank + 8 * (piece < pieces ? piece : pieces - 1),
                            b_lds + 1024 * j);
    }
  };
  bool in[RK];  // whether this lane's piece of a step lies within the rank
#pragma unroll
  for (int s = 0; s < RK; ++s) in[s] = 32 * s + 8 * h < a.rank;
  bf16x8 b[4][RK];
  auto read_b = [&]() {
#pragma unroll
    for (int round = 0; round < RK / BK; ++round) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int s = 0; s < BK; ++s) {
          const bf16x8 z = *reinterpret_cast<const bf16x8 *>(b_lds + (16 * i + r16) * 64 * BK +
                                                             16 * ((4 * s + h) ^ shuffle(r16)));
          b[i][BK * round + s] = in[BK * round + s] ? z : zero_bf16x8();
        }
      if (round + 1 < RK / BK) {
        fp4q_gemm::wait_lgkmcnt0();
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        __builtin_amdgcn_sched_barrier(0);
        load_b(round + 1);
        fp4q_gemm::wait_vmcnt<0>();
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  // this lane's rows of tile m, 4 h + v of its 16, and its columns, 4 r16 + i of the wave's 64; the rows' numbers are
  // waited for before B is asked for, whose loads they would else wait for too
  const int row0 = t.lo + lane, here = entry_at(a.groups, row0 < t.hi ? row0 : t.hi - 1);
  int entry[TILES][4];
#pragma unroll
  for (int m = 0; m < TILES; ++m)
#pragma unroll
    for (int v = 0; v < 4; ++v) entry[m][v] = __shfl(here, 16 * m + 4 * h + v);
  __builtin_amdgcn_sched_barrier(0);
  if (live && !rest) load_b(0);
  const int stride = part_stride(a.rank);
  if constexpr (TURNS) {
    if (live && !rest) {
      fp4q_gemm::wait_vmcnt<0>();
      __atomic_signal_fence(__ATOMIC_SEQ_CST);
      __builtin_amdgcn_sched_barrier(0);
      read_b();
      fp4q_gemm::wait_lgkmcnt0();
    }
    __syncthreads();
  }
  if (!rest) {
    if constexpr (SUMS) {
      const float scale = a.scales ? a.scales[t.group] : 1.0f;
      const int fours = (t.hi - t.lo) * a.rank / 4;
      for (int c = threadIdx.x; c < fours; c += kLoraThreads) {
        const float *at = (const float *)a.u + (int64_t)t.lo * a.rank + 4 * c;
        f32x4 v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (q < a.splits) v[q] = *reinterpret_cast<const f32x4 *>(at + (int64_t)q * a.groups.entries * a.rank);
        f32x4 sum = v[0];
#pragma unroll
        for (int q = 1; q < 8; ++q)
          if (q < a.splits) sum += v[q];
        uint16_t z[4][kParts];
#pragma unroll
        for (int i = 0; i < 4; ++i) parts_of(sum[i] * scale, z[i]);
        const int row = (int)((uint32_t)(4 * c) / (uint32_t)a.rank), to = 2 * (4 * c + 8 * row);
#pragma unroll
        for (int i = 0; i < kParts; ++i)
          *reinterpret_cast<u32x2 *>(lds + i * PART_BYTES + to) =
              u32x2{z[0][i] | (uint32_t)z[1][i] << 16, z[2][i] | (uint32_t)z[3][i] << 16};
      }
    } else {
      const int pieces = (ROWS * stride * 2 + 1023) / 1024;  // of 1 KB
#pragma unroll
      for (int q = 0; q < kParts; ++q) {
        const uint8_t *src =
            (const uint8_t *)a.u + 2 * (q * part_size(a.groups.entries, a.rank) + (int64_t)t.lo * stride);
        for (int c = wave; c < pieces; c += kLoraWaves) {
          // the last piece ends with the tile's rows: lanes past them load its first bytes again
          const int at = 1024 * c + 16 * lane;
          fp4q_gemm::load_lds16(src + (at < ROWS * stride * 2 ? at : 0), lds + q * PART_BYTES + 1024 * c);
        }
      }
    }
  }
  const int c0 = n0 + 4 * r16;
  const bool whole = a.wide && c0 + 4 <= a.n;
  const O *y = (const O *)a.y + c0;
  O *out = (O *)a.out + c0;
  Four<O> old[TILES][4];
  if (whole) {
#pragma unroll
    for (int m = 0; m < TILES; ++m)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        old[m][v].v = *reinterpret_cast<const decltype(Four<O>::v) *>(y + (entry[m][v] < 0 ? 0 : entry[m][v]) * a.ld_y);
  }
  __syncthreads();  // u and B have landed
  if (!live) return;
  if constexpr (!TURNS) {
    if (!rest) read_b();
  }
#pragma unroll
  for (int m = 0; m < TILES; ++m) {
    if (t.lo + 16 * m >= t.hi) break;
    f32x4 acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = f32x4{0, 0, 0, 0};
    if (!rest) {
#pragma unroll
      for (int s = 0; s < RK; ++s) {
        bf16x8 u[kParts];
        // past the rank: the next row's numbers or the padding, which are no numbers of this row
        const uint8_t *at = lds + ((16 * m + r16) * stride + 32 * s + 8 * h) * 2;
#pragma unroll
        for (int i = 0; i < kParts; ++i)
          u[i] = in[s] ? *reinterpret_cast<const bf16x8 *>(at + i * PART_BYTES) : zero_bf16x8();
#pragma unroll
        for (int q = kParts - 1; q >= 0; --q)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(u[q], b[i][s], acc[i], 0, 0, 0);
      }
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int e = entry[m][v];
      if (e < 0 || t.lo + 16 * m + 4 * h + v >= t.hi) continue;
      O *to = out + e * a.ld_out;
      if (whole) {
        float z[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = old[m][v].at(i) + acc[i][v];
        store_four(to, z);
      } else {
        const O *from = y + e * a.ld_y;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c0 + i < a.n) fp4q_gemm::store_out(to + i, load1(from + i) + acc[i][v]);
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
  return 256 + (size_t)(kParts * part_size(entries, (int)rank) * 2);
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
  const bool wide = kv_aligned(y, 4 * size) && kv_aligned(out, 4 * size) && ld_y % 4 == 0 && ld_out % 4 == 0;
  const LoraArgs l{y, (const uint16_t *)x, (const uint16_t *)a, (const uint16_t *)b, scales, out, ld_y, ld_x, ld_out,
                   groups_of(*groups), (int)n, (int)k, (int)rank, (int)p.splits, (int)ceil_div(n, 64 * kLoraWaves),
                   out == y, wide, (char *)workspace + 256, status};
  const int64_t rows = lora_rows(p, rank, size);
  const int64_t tiles = l.tiles_n * (most_tiles(entries, groups->groups, rows) + 1);
  const int64_t mr = p.splits == 1 && rank <= 64 ? 2 : 1;
  const int64_t shrink_tiles = most_tiles(entries, groups->groups, 16 * mr);
  if (tiles > kMaxTiles || shrink_tiles > kMaxTiles) return FP4Q_ERR_SHAPE;
  auto shrink = [&](auto rt) {
    constexpr int RT = decltype(rt)::value, MR = RT <= 4 ? 2 : 1;
    constexpr int W = 4, NS = RT <= 2 ? 4 : (RT == 4 ? 3 : (RT == 8 ? 2 : 1)), SPLIT_NS = RT <= 4 ? 2 : 1;
    auto kernel = p.splits > 1 ? shrink_kernel<RT, 1, W, SPLIT_NS, true> : shrink_kernel<RT, MR, W, NS, false>;
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
      constexpr int MOST = sizeof(O) == 4 || RK >= 4 ? 32 : 64;
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
