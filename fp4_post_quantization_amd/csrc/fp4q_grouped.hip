// Grouped MXFP4 products: every entry's row times its group's matrix
// (include/fp4q_grouped.h), on gfx950's scaled FP4 matrix cores.
//
// A tile is rows of one group times columns of its matrix.
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

using fp4q_gemm::i32x4;
using fp4q_gemm::i32x8;
using fp4q_gemm::f32x16;
using fp4q_gemm::store_out;

struct GroupedArgs {
  const uint8_t *a, *as, *b, *bs;
  Groups groups;
  int a_rows, gather, scatter;
  int n, k, n_out, tiles_n;  // n_out: columns of C
  float alpha;
  void *c;
  int64_t ldc;
  uint32_t *status;
};

// The row of A of position p, whose entry is e.
__device__ __forceinline__ int a_row(const GroupedArgs &a, int p, int e) {
  return a.gather ? (e < 0 ? 0 : e / a.gather) : p;
}

__device__ __forceinline__ float silu(float z) { return z / (1.0f + __expf(-z)); }

// Any k that is a multiple of 32: 64 rows times 128 rows of B (gated: 64 gates and their 64 ups), registers to a
// padded LDS double buffer, 128 elements of K a stage, the tail filled with zeros.
constexpr int kAnyRows = 64, kAnyCols = 128, kAnyThreads = 256, kAnyRowBytes = 80;

template <typename OutT, bool GATED>
__global__ __launch_bounds__(kAnyThreads) void grouped_any_kernel(GroupedArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t lA[2][kAnyRows * kAnyRowBytes], lB[2][kAnyCols * kAnyRowBytes];
  __shared__ uint32_t sA[2][kAnyRows], sB[2][kAnyCols];
  __shared__ int row_of[kAnyRows];  // row of C, -1: not stored
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_index();
  const int wm = wave & 1, wn = wave >> 1, l32 = lane & 31, h = lane >> 5;
  uint32_t err = 0;
  if (blockIdx.x == 0 && wave == 0 && offsets_bad(a.groups)) err = FP4Q_DATA_BAD_GROUP;
  const RowTile t = find_tile(a.groups, kAnyRows, (int)(blockIdx.x / a.tiles_n));
  if (t.group < 0) {
    Status{a.status, true}.finish(err);
    return;
  }
  const int n0 = (int)(blockIdx.x % a.tiles_n) * (GATED ? kAnyCols / 2 : kAnyCols);  // first column of C
  const int kb = a.k / 2, ksc = a.k / 32, nst = (a.k + 127) / 128;
  const uint8_t *b = a.b + (int64_t)t.group * a.n * kb, *bs = a.bs + (int64_t)t.group * a.n * ksc;
  // tile row r of B: the matrix's row, -1 past the last
  auto b_row = [&](int r) {
    const int col = GATED ? n0 + (r >> 6) * 32 + (r & 31) : n0 + r;
    return col < a.n_out ? col + (GATED && (r & 32) ? a.n_out : 0) : -1;
  };
  int64_t a_at;
  int ar;
  i32x4 ra, rb[2];
  uint32_t rsa = 0x7F7F7F7Fu, rsb = 0x7F7F7F7Fu;
  {  // piece tid of A: row tid / 4, 16-byte chunk tid % 4 of the stage
    const int p = t.lo + (tid >> 2);
    const int e = p < t.hi ? entry_at(a.groups, p) : -1;
    if (p < t.hi && e < 0) err = FP4Q_DATA_BAD_GROUP;
    ar = p < t.hi && (e >= 0 || !a.gather) ? a_row(a, p, e) : -1;
    a_at = (int64_t)ar * kb;
    if ((tid & 3) == 0) row_of[tid >> 2] = p < t.hi && e >= 0 ? (a.scatter ? e : p) : -1;
  }
  auto scales = [&](const uint8_t *row, int st) {
    uint32_t v = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) v |= (uint32_t)(4 * st + j < ksc ? row[4 * st + j] : 0x7F) << (8 * j);
    return v;
  };
  auto gload = [&](int st) {
    const int pc = tid & 3;
    ra = ar >= 0 && st * 128 + 32 * pc < a.k
                ? *reinterpret_cast<const i32x4 *>(a.a + a_at + st * 64 + 16 * pc) : i32x4{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = b_row((tid >> 2) + 64 * j);
      rb[j] = r >= 0 && st * 128 + 32 * pc < a.k
                  ? *reinterpret_cast<const i32x4 *>(b + (int64_t)r * kb + st * 64 + 16 * pc) : i32x4{0, 0, 0, 0};
    }
    if (pc == 0) rsa = ar >= 0 ? scales(a.as + (int64_t)ar * ksc, st) : 0x7F7F7F7Fu;
    if (tid < kAnyCols) {
      const int r = b_row(tid);
      rsb = r >= 0 ? scales(bs + (int64_t)r * ksc, st) : 0x7F7F7F7Fu;
    }
  };
  auto lstore = [&](int buf) {
    const int r = tid >> 2, pc = tid & 3;
    *reinterpret_cast<i32x4 *>(&lA[buf][r * kAnyRowBytes + 16 * pc]) = ra;
#pragma unroll
    for (int j = 0; j < 2; ++j) *reinterpret_cast<i32x4 *>(&lB[buf][(r + 64 * j) * kAnyRowBytes + 16 * pc]) = rb[j];
    if (pc == 0) sA[buf][r] = rsa;
    if (tid < kAnyCols) sB[buf][tid] = rsb;
  };
  f32x16 acc[2] = {f32x16{0}, f32x16{0}};
  gload(0);
  lstore(0);
  __syncthreads();
  for (int st = 0; st < nst; ++st) {
    const int buf = st & 1;
    if (st + 1 < nst) gload(st + 1);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const int r = wm * 32 + l32;
      const i32x4 va = *reinterpret_cast<const i32x4 *>(&lA[buf][r * kAnyRowBytes + 32 * ks + 16 * h]);
      const int sa = (int)((sA[buf][r] >> (8 * (2 * ks + h))) & 0xFFu);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int q = wn * 64 + j * 32 + l32;
        const i32x4 vb = *reinterpret_cast<const i32x4 *>(&lB[buf][q * kAnyRowBytes + 32 * ks + 16 * h]);
        const int sb = (int)((sB[buf][q] >> (8 * (2 * ks + h))) & 0xFFu);
        acc[j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(i32x8{va.x, va.y, va.z, va.w, 0, 0, 0, 0},
                                                                 i32x8{vb.x, vb.y, vb.z, vb.w, 0, 0, 0, 0}, acc[j], 4,
                                                                 4, 0, sa, 0, sb);
      }
    }
    if (st + 1 < nst) {
      lstore(buf ^ 1);
      __syncthreads();
    }
  }
  OutT *c = (OutT *)a.c;
#pragma unroll
  for (int v = 0; v < 16; ++v) {
    const int row = row_of[wm * 32 + 8 * (v >> 2) + 4 * h + (v & 3)];
    if (row < 0) continue;
    if constexpr (GATED) {
      const int col = n0 + wn * 32 + l32;
      if (col < a.n_out) store_out(c + (int64_t)row * a.ldc + col, silu(a.alpha * acc[0][v]) * (a.alpha * acc[1][v]));
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int col = n0 + wn * 64 + j * 32 + l32;
        if (col < a.n_out) store_out(c + (int64_t)row * a.ldc + col, a.alpha * acc[j][v]);
      }
    }
  }
  Status{a.status, true}.finish(err);
}

__global__ __launch_bounds__(64) void grouped_status_kernel(uint32_t *status) {
  if (threadIdx.x == 0) Status{status, true}.merge(0u);
}

template <typename F>
void with_type(fp4q_dtype_t t, F &&f) {
  if (t == FP4Q_BF16) f((uint16_t *)nullptr);
  else f((float *)nullptr);
}

fp4q_status_t hip_status() { return hipGetLastError() == hipSuccess ? FP4Q_OK : FP4Q_ERR_HIP; }

}  // namespace
}  // namespace fp4q

using namespace fp4q;

extern "C" fp4q_status_t fp4q_gemm_mxfp4_grouped(const uint8_t *a_codes, const uint8_t *a_scales, int64_t a_rows,
                                                 const uint8_t *b_codes, const uint8_t *b_scales,
                                                 const fp4q_row_groups_t *groups, int64_t n, int64_t k,
                                                 int64_t gather, int scatter, int gated, float alpha,
                                                 fp4q_dtype_t out_dtype, void *c, int64_t ldc, void *workspace,
                                                 size_t workspace_bytes, void *stream) {
  if (!groups) return FP4Q_ERR_NULL;
  if ((out_dtype != FP4Q_F32 && out_dtype != FP4Q_BF16) || (scatter != 0 && scatter != 1) || (gated != 0 && gated != 1))
    return FP4Q_ERR_ARG;
  fp4q_status_t st = grouped_check(*groups);
  if (st != FP4Q_OK) return st;
  if ((st = grouped_product_check(*groups, a_rows, n, k, gather, gated, ldc, out_dtype == FP4Q_F32 ? 4 : 2)) != FP4Q_OK)
    return st;
  if (!grouped_ws_ok(workspace, workspace_bytes, kWorkspaceBytes)) return FP4Q_ERR_WORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  uint32_t *status = (uint32_t *)workspace;
  if (groups->entries == 0 || n == 0) {
    hipLaunchKernelGGL(grouped_status_kernel, dim3(1), dim3(64), 0, s, status);
    return hip_status();
  }
  if (!a_codes || !a_scales || !b_codes || !b_scales || !c) return FP4Q_ERR_NULL;
  if (!kv_aligned(a_codes, 16) || !kv_aligned(b_codes, 16) || !kv_aligned(c, out_dtype == FP4Q_F32 ? 4 : 2))
    return FP4Q_ERR_ALIGN;
  if (k % 128 == 0 && (!kv_aligned(a_scales, 4) || !kv_aligned(b_scales, 4))) return FP4Q_ERR_ALIGN;
  GroupedArgs a{a_codes, a_scales, b_codes, b_scales, groups_of(*groups), (int)a_rows, (int)gather, scatter, (int)n, (int)k, (int)(gated ? n / 2 : n), 0,
                alpha, c, ldc, status};
  a.tiles_n = (int)ceil_div(n, kAnyCols);
  const int64_t tiles = a.tiles_n * most_tiles(groups->entries, groups->groups, kAnyRows);
  if (tiles > kMaxTiles) return FP4Q_ERR_SHAPE;
  with_type(out_dtype, [&](auto op) {
    using O = std::remove_pointer_t<decltype(op)>;
    if (gated)
      hipLaunchKernelGGL((grouped_any_kernel<O, true>), dim3((unsigned)tiles), dim3(kAnyThreads), 0, s, a);
    else
      hipLaunchKernelGGL((grouped_any_kernel<O, false>), dim3((unsigned)tiles), dim3(kAnyThreads), 0, s, a);
  });
  return hip_status();
}
