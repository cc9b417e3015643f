// Grouped MXFP4 products: every entry's row times its group's matrix
// (include/fp4q_grouped.h), on gfx950's scaled FP4 matrix cores.
//
// A tile is rows of one group times columns of its matrix.  Few rows a group are
// bound by the matrices' bytes: 16 tokens of 128 experts, 8 each, gate and up
// rows of 4096 x 1536 read 276 MB in 54 us (5.1 TB/s, the rate of a large copy)
// where eight layers' matrices follow each other, and in 43 where the same ones
// are read again, a sixth of them from the last level cache.  Many are bound by
// the steps of the LDS ring, as in the plain product, and by rows that fill no
// tile: 4096 tokens (256 rows a group on average, 1.5 tiles of 256) 203 to 218
// us, 2.0 PFLOP/s of the entries' products and 3 of the tiles'; 8192 tokens of 8
// experts, two each, on 4096 x 4096 181 to 199 us, 2.8 PFLOP/s.  product_tiles()
// chooses the kernel.
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
  int run;                   // tiles in a row that go to one XCD
  float alpha;
  void *c;
  int64_t ldc;
  uint32_t *status;
  bool zeroed;  // rows of C of entries of no group become zeros
};

// The row of A of position p, whose entry is e.
__device__ __forceinline__ int a_row(const GroupedArgs &a, int p, int e) {
  return a.gather ? (e < 0 ? 0 : e / a.gather) : p;
}

// Zeros in the rows of C of entries of no group, a row a workgroup of whatever kernel at a time: they are read like any
// other by what quantizes or sums C next.  (A call with none of them: one load a workgroup, 11.9 us instead of 11.7 for
// one token of 8 experts; 333 tokens of which every seventh is padding 18.8 instead of 18.1.)
template <typename OutT>
__device__ __forceinline__ void zero_rest(const GroupedArgs &a) {
  constexpr int VEC = 16 / (int)sizeof(OutT);
  const int last = a.groups.offsets[a.groups.groups], from = last < 0 ? 0 : last;
  const bool wide = ((uintptr_t)a.c % 16 == 0) && ((a.ldc * (int64_t)sizeof(OutT)) % 16 == 0);
  const int whole = wide ? a.n_out / VEC * VEC : 0;
  for (int64_t p = (int64_t)from + blockIdx.x; p < a.groups.entries; p += gridDim.x) {
    const int row = a.scatter ? entry_at(a.groups, (int)p) : (int)p;
    if (row < 0) continue;
    OutT *c = (OutT *)a.c + (int64_t)row * a.ldc;
    for (int i = threadIdx.x * VEC; i < whole; i += blockDim.x * VEC)
      *reinterpret_cast<u32x4 *>(c + i) = u32x4{0, 0, 0, 0};
    for (int i = whole + threadIdx.x; i < a.n_out; i += blockDim.x) c[i] = OutT(0);
  }
}

// z / (1 + exp(-z)) to 7 units of 2^-24, for z < 0 as z exp(z) / (1 + exp(z)), so that nothing leaves float32's range
// before the result does.  exp(-|z|) is 2^(i + f) with i = round(-|z| log2 e) and f from two parts of log2 e, so that
// the error of the product does not grow with |z| (from 200 on it is 0 all the same); 1 / (1 + exp(-|z|)) is the
// hardware's, off by one unit, after one Newton step.  -inf gives NaN, as the quotient does.  (The hardware's exponential
// and reciprocal of 1 + exp(-z) alone: off by |z| units, and 0 from z = -87 on where float32 reaches to -92; 4096 tokens of
// 128 experts, gates and ups of 4096 x 1536, 212 us instead of 221.)
__device__ __forceinline__ float silu(float z) {
  constexpr float kLog2e = 1.44269502f, kLog2eRest = 1.92596299e-8f;
  const float a = __builtin_fminf(__builtin_fabsf(z), 200.0f);
  const float i = __builtin_rintf(-a * kLog2e);
  const float f = __builtin_fmaf(-a, kLog2eRest, __builtin_fmaf(-a, kLog2e, -i));
  const float e = __builtin_ldexpf(__builtin_amdgcn_exp2f(f), (int)i), d = 1.0f + e;
  float r = __builtin_amdgcn_rcpf(d);
  r = __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r);
  return (z < 0.0f ? z * e : z) * r;
}

// Any k that is a multiple of 32: 64 rows times 128 rows of B (gated: 64 gates and their 64 ups), registers to a
// padded LDS double buffer, 128 elements of K a stage, the tail filled with zeros.  For K below 256, which the ring's
// stages do not fit, and for matrices or rows of A past 4 GiB, whose offsets it does not hold (2^21 rows of K 4096 on
// N 32: reading A bounds it there as well).
constexpr int kAnyThreads = 256, kAnyRowBytes = 80;

template <typename OutT, bool GATED>
__global__ __launch_bounds__(kAnyThreads) void grouped_any_kernel(GroupedArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t lA[2][kAnyRows * kAnyRowBytes], lB[2][kAnyCols * kAnyRowBytes];
  __shared__ uint32_t sA[2][kAnyRows], sB[2][kAnyCols];
  __shared__ int row_of[kAnyRows];  // row of C, -1: not stored
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_index();
  const int wm = wave & 1, wn = wave >> 1, l32 = lane & 31, h = lane >> 5;
  if (a.zeroed) zero_rest<OutT>(a);
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

// ---------------------------------------------------------------------------
// K of 256 or more: operands move from global memory straight into an LDS ring of NS stages of 128 code bytes of
// every row, as in the plain product (fp4q_gemm.hip): one wave computes TM x TN blocks of 32 x 32, WGM x WGN waves a
// tile; rows are unpadded and swizzled; K step ks takes, in lane half h, the 32-element block h KS + ks of the stage,
// so that a lane's scale bytes of a stage are one word, of which the instruction selects byte ks.  What differs is
// where rows come from: a lane loads the entry numbers of the rows that it stages once, before the loop.
// TAIL, where K is no multiple of 256: chunks past a row's end are loaded from zeros, and scales, whose rows need not
// be aligned, come through registers, where they are put in place as they arrive: the next stage's products begin only
// when the loads of the one after it, just issued, have landed, so that every stage shows a trip to memory.
//
// Gated: block column j of a wave is gates for even j and the ups of the same columns for odd j, so that both meet in
// a lane's registers.
//
// Tiles of one group are taken together, up to kTileGroup row tiles column by column, and runs of `run` tiles go to
// one XCD (workgroups are dealt round robin over the eight), so that what shares rows or a matrix shares an L2.
constexpr int kTileGroup = 8;

__device__ __forceinline__ int tile_number(const GroupedArgs &a) {
  const int local = (int)blockIdx.x / kXcdCount;
  return (local / a.run * kXcdCount + (int)blockIdx.x % kXcdCount) * a.run + local % a.run;
}
// Positions [lo, hi) and column tile of tile number lin, one of group g.
struct GroupTile {
  int lo, hi, col;
};
__device__ __forceinline__ GroupTile group_tile(const GroupedArgs &a, const TileGroup &g, int rows, int lin) {
  const int within = lin - g.first * a.tiles_n, chunk = within / (kTileGroup * a.tiles_n);
  const int left = span_tiles(g.lo, g.hi, rows) - chunk * kTileGroup, deep = left < kTileGroup ? left : kTileGroup;
  const int r = within - chunk * kTileGroup * a.tiles_n;
  const int lo = g.lo + (chunk * kTileGroup + r % deep) * rows;
  return GroupTile{lo, g.hi - lo > rows ? lo + rows : g.hi, r / deep};
}

constexpr int kRowBytes = 128;  // code bytes of a row and stage: 256 elements of K

template <bool GATED, int WGM, int WGN, int TM, int TN>
struct RingShape {
  static constexpr int ROWB = kRowBytes;
  static constexpr int WAVES = WGM * WGN, THREADS = 64 * WAVES;
  static constexpr int BM = WGM * TM * 32, BN = WGN * TN * 32;   // rows of A and of B
  static constexpr int COLS = GATED ? BN / 2 : BN;               // columns of C
  static constexpr int CPR = ROWB / 16, KS = ROWB / 32, SPR = ROWB / 16;
  static constexpr int A_BYTES = BM * ROWB, B_BYTES = BN * ROWB;
  static constexpr int SA_OFF = A_BYTES + B_BYTES, SB_OFF = SA_OFF + BM * SPR;
  static constexpr int STAGE = SB_OFF + BN * SPR;
};

// The accumulators' registers v .. v + 3 (four columns of one row, B's rows being the first operand) to the staging.
template <typename OutT, bool GATED>
__device__ __forceinline__ void stage_four(const f32x16 &x, const f32x16 &up, int v, float alpha, OutT *to) {
  float z[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    z[k] = alpha * x[v + k];
    if constexpr (GATED) z[k] = silu(z[k]) * (alpha * up[v + k]);
  }
  if constexpr (sizeof(OutT) == 4)
    *reinterpret_cast<f32x4 *>(to) = f32x4{z[0], z[1], z[2], z[3]};
  else
    *reinterpret_cast<uint2 *>(to) =
        uint2{fp4q_gemm::f32x2_to_bf16x2(z[0], z[1]), fp4q_gemm::f32x2_to_bf16x2(z[2], z[3])};
}

// The E8M0 bytes of blocks 8 st .. 8 st + 7 of a row that has ksc >= 8 of them, at any alignment; 127 past the last.
__device__ __forceinline__ uint64_t scale_bytes(const uint8_t *row, int ksc, int st) {
  const int want = 8 * st, at = want + 8 <= ksc ? want : ksc - 8, skip = want - at;  // skip < 8
  uint64_t v;
  __builtin_memcpy(&v, row + at, 8);
  return skip ? v >> (8 * skip) | 0x7F7F7F7F7F7F7F7Full << (64 - 8 * skip) : v;
}

__device__ const u32x4 kZeroCodes = {0, 0, 0, 0};

template <typename OutT, bool GATED, bool TAIL, int NS, int WGM, int WGN, int TM, int TN>
__global__ __launch_bounds__(64 * WGM * WGN) void grouped_ring_kernel(GroupedArgs a) {
  using S = RingShape<GATED, WGM, WGN, TM, TN>;
  static_assert(!TAIL || NS == 2, "scales that come through registers are a stage ahead");
  constexpr int ROWB = kRowBytes, WAVES = S::WAVES, BM = S::BM, BN = S::BN;
  constexpr int CPR = S::CPR, KS = S::KS, SPR = S::SPR, STAGE = S::STAGE;
  constexpr int RPL = 1024 / ROWB;  // rows of a 1 KB load
  constexpr int A_INSTR = BM / RPL / WAVES, B_INSTR = BN / RPL / WAVES;
  constexpr int SA_INSTR = BM * SPR / 256, SB_INSTR = BN * SPR / 256;
  constexpr int SQ = TAIL ? 0 : (SA_INSTR + SB_INSTR + WAVES - 1) / WAVES;
  constexpr int SROWS = (BM + BN + S::THREADS - 1) / S::THREADS;  // TAIL: rows whose scales a thread brings
  constexpr int DPR = SPR / 4, RPS = 256 / SPR;  // scale words of a row, rows of a scale load
  static_assert(A_INSTR * WAVES * RPL == BM && B_INSTR * WAVES * RPL == BN, "code loads must divide evenly");
  static_assert(SA_INSTR * 256 == BM * SPR && SB_INSTR * 256 == BN * SPR, "scale loads cover whole rows");
  static_assert(!GATED || TN % 2 == 0, "gates and ups in pairs of block columns");
  constexpr int LOADS = A_INSTR + B_INSTR + SQ + (TAIL ? SROWS : 0);  // of a wave and stage; one without a scale load
                                                                     // fills a spare slot
  constexpr int SPARE = NS * STAGE;
  // One array: with two, the compiler tells them apart and then waits for every load into LDS before it reads any.
  __shared__ __attribute__((aligned(1024))) uint8_t smem[NS * STAGE + 256 + 4 * BM];
  int *row_of = reinterpret_cast<int *>(smem + NS * STAGE + 256);  // row of C, -1: not stored

  const int tid = threadIdx.x, lane = tid & 63, wave = wave_index();
  const int wm = wave / WGN, wn = wave % WGN, l32 = lane & 31, h = lane >> 5;
  if (a.zeroed) zero_rest<OutT>(a);
  uint32_t err = 0;
  if (blockIdx.x == 0 && wave == 0 && offsets_bad(a.groups)) err = FP4Q_DATA_BAD_GROUP;
  const int lin = tile_number(a);
  const TileGroup g = find_group(a.groups, BM, lin / a.tiles_n);
  if (g.group < 0) {
    Status{a.status, true}.finish(err);
    return;
  }
  const GroupTile t = group_tile(a, g, BM, lin);
  const int lo = t.lo, hi = t.hi, n0 = t.col * S::COLS;  // first column of C

  const uint32_t kb = a.k / 2, ksc = a.k / 32;
  const int nst = (a.k + 2 * ROWB - 1) / (2 * ROWB);
  const uint8_t *B = a.b + (int64_t)g.group * a.n * kb, *Bs = a.bs + (int64_t)g.group * a.n * ksc;
  // row of A of tile row i (those past the tile repeat its last one: computed, never stored)
  auto a_of = [&](int i) {
    const int p = lo + i < hi ? lo + i : hi - 1;
    return (uint32_t)(a.gather ? a_row(a, p, entry_at(a.groups, p)) : p);
  };
  auto b_of = [&](int i) {
    const int col = GATED ? (i / 64) * 32 + (i & 31) : i;
    return (uint32_t)((n0 + col < a.n_out ? n0 + col : a.n_out - 1) + (GATED && (i & 32) ? a.n_out : 0));
  };
  for (int i = tid; i < BM; i += S::THREADS) {
    const int e = lo + i < hi ? entry_at(a.groups, lo + i) : -1;
    if (lo + i < hi && e < 0) err = FP4Q_DATA_BAD_GROUP;
    row_of[i] = e < 0 ? -1 : (a.scatter ? e : lo + i);
  }
  // sources as 32-bit offsets from scalar bases: A and a group's matrix are below 4 GiB
  uint32_t srcA[A_INSTR], srcB[B_INSTR], srcS[SQ > 0 ? SQ : 1];
  const uint8_t *baseS[SQ > 0 ? SQ : 1];
  int dstS[SQ > 0 ? SQ : 1];
  // TAIL: the 16-byte chunks that the last stage has of a row, and which of them this lane brings
  const int last_chunks = (a.k - 2 * ROWB * (nst - 1)) / 32;
  int chunkA[A_INSTR], chunkB[B_INSTR];
#pragma unroll
  for (int i = 0; i < A_INSTR; ++i) {
    const int row = (wave * A_INSTR + i) * RPL + lane / CPR;
    chunkA[i] = (lane % CPR) ^ fp4q_gemm::swz<ROWB>(row);
    srcA[i] = a_of(row) * kb + 16 * chunkA[i];
  }
#pragma unroll
  for (int i = 0; i < B_INSTR; ++i) {
    const int row = (wave * B_INSTR + i) * RPL + lane / CPR;
    chunkB[i] = (lane % CPR) ^ fp4q_gemm::swz<ROWB>(row);
    srcB[i] = b_of(row) * kb + 16 * chunkB[i];
  }
  // TAIL: scales of rows that need not be aligned come through registers, a row a thread
  const uint8_t *rowS[SROWS];
  uint64_t nextS[SROWS];
#pragma unroll
  for (int i = 0; i < SROWS; ++i) {
    const int r = tid + i * S::THREADS;
    rowS[i] = r < BM ? a.as + (uint64_t)a_of(r) * ksc : Bs + (uint64_t)b_of(r - BM < BN ? r - BM : BN - 1) * ksc;
    nextS[i] = 0;
  }
#pragma unroll
  for (int j = 0; j < SQ; ++j) {
    const int q = wave + WAVES * j, rl = lane / DPR, dw = lane % DPR;
    if (q < SA_INSTR) {
      baseS[j] = a.as;
      srcS[j] = a_of(RPS * q + rl) * ksc + 4 * dw;
      dstS[j] = S::SA_OFF + 256 * q;
    } else if (q < SA_INSTR + SB_INSTR) {
      baseS[j] = Bs;
      srcS[j] = b_of(RPS * (q - SA_INSTR) + rl) * ksc + 4 * dw;
      dstS[j] = S::SB_OFF + 256 * (q - SA_INSTR);
    } else {
      baseS[j] = Bs;
      srcS[j] = 4 * dw;
      dstS[j] = -1;
    }
  }
  auto issue = [&](int st, int slot) {
    uint8_t *base = smem + slot * STAGE;
    const int chunks = TAIL && st == nst - 1 ? last_chunks : CPR;
    const uint8_t *a_st = a.a + (int64_t)st * ROWB, *b_st = B + (int64_t)st * ROWB;
    auto source = [&](const uint8_t *p, uint32_t off, int chunk) {
      return TAIL && chunk >= chunks ? reinterpret_cast<const uint8_t *>(&kZeroCodes) : p + off;
    };
#pragma unroll
    for (int i = 0; i < A_INSTR; ++i)
      fp4q_gemm::load_lds16(source(a_st, srcA[i], chunkA[i]), base + (wave * A_INSTR + i) * 1024);
#pragma unroll
    for (int i = 0; i < B_INSTR; ++i)
      fp4q_gemm::load_lds16(source(b_st, srcB[i], chunkB[i]), base + S::A_BYTES + (wave * B_INSTR + i) * 1024);
    if constexpr (TAIL) {
#pragma unroll
      for (int i = 0; i < SROWS; ++i) nextS[i] = scale_bytes(rowS[i], (int)ksc, st);
    }
#pragma unroll
    for (int j = 0; j < SQ; ++j)
      fp4q_gemm::load_lds4(baseS[j] + (int64_t)st * SPR + srcS[j], dstS[j] >= 0 ? base + dstS[j] : smem + SPARE);
  };
  auto put_scales = [&](int slot) {  // TAIL: of the stage last issued, into its slot
    if constexpr (TAIL) {
#pragma unroll
      for (int i = 0; i < SROWS; ++i) {
        const int r = tid + i * S::THREADS;
        if (r < BM + BN) *reinterpret_cast<uint64_t *>(smem + slot * STAGE + S::SA_OFF + 8 * r) = nextS[i];
      }
    }
  };
  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x16{0};
  struct Ops {
    i32x8 a[TM], b[TN];
    int sa[TM], sb[TN];
  };
  auto scale_word = [&](const uint8_t *p) { return (int)*reinterpret_cast<const uint32_t *>(p + 4 * h); };
  const int lane_sw = fp4q_gemm::swz<ROWB>(l32);  // of every row a lane reads: they differ by multiples of 32
  auto read_ops = [&](int slot, auto ks_c, Ops &o, const Ops &prev) {
    constexpr int ks = decltype(ks_c)::value;
    const uint8_t *base = smem + slot * STAGE;
    const uint8_t *at = base + l32 * ROWB + 16 * ((h * KS + ks) ^ lane_sw);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const i32x4 v = *reinterpret_cast<const i32x4 *>(at + (wm * TM + i) * 32 * ROWB);
      o.a[i] = i32x8{v.x, v.y, v.z, v.w, 0, 0, 0, 0};
      o.sa[i] = ks == 0 ? scale_word(base + S::SA_OFF + SPR * ((wm * TM + i) * 32 + l32)) : prev.sa[i];
    }
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const i32x4 v = *reinterpret_cast<const i32x4 *>(at + S::A_BYTES + (wn * TN + j) * 32 * ROWB);
      o.b[j] = i32x8{v.x, v.y, v.z, v.w, 0, 0, 0, 0};
      o.sb[j] = ks == 0 ? scale_word(base + S::SB_OFF + SPR * ((wn * TN + j) * 32 + l32)) : prev.sb[j];
    }
  };
  auto mfmas = [&](const Ops &o, auto ks_c) {
    constexpr int ks = decltype(ks_c)::value;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(o.b[j], o.a[i], acc[i][j], 4, 4, ks, o.sb[j], ks,
                                                                    o.sa[i]);
  };
  const bool live = lo + wm * TM * 32 < hi;  // whether any of this wave's rows is there
  auto stage_barrier = [&]() {  // keeps LDS accesses on their side, without draining the loads in flight
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
  };

  // Stage s sits in slot s % NS; once every wave has read all of it, stage s + NS is issued into its slot (past the
  // last one the last is loaded again, so that every wait is one constant).
  issue(0, 0);
  put_scales(0);
#pragma unroll
  for (int s = 1; s < NS; ++s) issue(s < nst ? s : nst - 1, s);
  fp4q_gemm::wait_lgkmcnt0();  // row_of and the scales are written
  fp4q_gemm::wait_vmcnt<(NS - 1) * LOADS>();
  stage_barrier();
  Ops o0, o1;
  int slot = 0;
  if (live) read_ops(0, std::integral_constant<int, 0>{}, o0, o1);
  for (int st = 0; st < nst; ++st) {
    if (live) {
      fp4q_gemm::unroll(std::make_integer_sequence<int, KS - 1>{}, [&](auto ks_c) {
        constexpr int ks = decltype(ks_c)::value;
        if constexpr (ks % 2 == 0) {
          read_ops(slot, std::integral_constant<int, ks + 1>{}, o1, o0);
          __builtin_amdgcn_sched_barrier(0);
          mfmas(o0, ks_c);
        } else {
          read_ops(slot, std::integral_constant<int, ks + 1>{}, o0, o1);
          __builtin_amdgcn_sched_barrier(0);
          mfmas(o1, ks_c);
        }
      });
    }
    __builtin_amdgcn_sched_barrier(0);
    const int next = slot == NS - 1 ? 0 : slot + 1;
    put_scales(next);
    fp4q_gemm::wait_lgkmcnt0();  // this wave's reads of stage st are complete, and its scales of st + 1 written
    fp4q_gemm::wait_vmcnt<(NS - 2) * LOADS>();  // stage st + 1 has landed
    stage_barrier();                            // ... for every wave, and nobody reads stage st any more
    issue(st + NS < nst ? st + NS : nst - 1, slot);
    if (live) {
      read_ops(next, std::integral_constant<int, 0>{}, o0, o1);
      __builtin_amdgcn_sched_barrier(0);
      mfmas(o1, std::integral_constant<int, KS - 1>{});
    }
    slot = next;
  }
  __syncthreads();  // every load has landed, every wave is done reading the ring

  // Each wave writes 32 rows of its columns at a time into its own area (padded by 16 bytes a row) and stores them in
  // pieces of 16 bytes along the rows of C.
  constexpr int WCOLS = S::COLS / WGN, VEC = 16 / (int)sizeof(OutT), EROW = WCOLS + VEC;
  constexpr int LPR = WCOLS / VEC, RPI = 64 / LPR;
  static_assert(WAVES * 32 * EROW * (int)sizeof(OutT) <= NS * STAGE, "epilogue staging must fit in the ring");
  OutT *area = reinterpret_cast<OutT *>(smem) + wave * 32 * EROW;
  OutT *C = (OutT *)a.c;
  const bool wide = ((uintptr_t)C % 16 == 0) && ((a.ldc * (int64_t)sizeof(OutT)) % 16 == 0);
  const float alpha = a.alpha;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    constexpr int JS = GATED ? 2 : 1;
#pragma unroll
    for (int j = 0; j < TN; j += JS)
#pragma unroll
      for (int v = 0; v < 16; v += 4)
        stage_four<OutT, GATED>(acc[i][j], acc[i][j + JS - 1], v, alpha,
                                area + l32 * EROW + j / JS * 32 + 2 * v + 4 * h);
#pragma unroll
    for (int q = 0; q < 32 / RPI; ++q) {
      const int rr = q * RPI + lane / LPR, c = lane % LPR * VEC;
      const int row = row_of[(wm * TM + i) * 32 + rr], col = n0 + wn * WCOLS + c;
      const i32x4 v = *reinterpret_cast<const i32x4 *>(area + rr * EROW + c);
      if (row >= 0) {
        OutT *dst = C + (int64_t)row * a.ldc + col;
        if (wide && col + VEC <= a.n_out) {
          *reinterpret_cast<i32x4 *>(dst) = v;
        } else {
          const OutT *e = reinterpret_cast<const OutT *>(&v);
#pragma unroll
          for (int t = 0; t < VEC; ++t)
            if (col + t < a.n_out) dst[t] = e[t];
        }
      }
    }
  }
  Status{a.status, true}.finish(err);
}

// ---------------------------------------------------------------------------
// Few rows a group (K a multiple of 128): 16 rows times 32 rows of B (gated: 16 gates and their 16 ups) a workgroup,
// whose waves share K.  v_mfma_scale_f32_16x16x128_f8f6f4 takes from lane l row l % 16 and the 32 elements at
// 32 (l / 16) of a step; register v of its accumulator holds row 4 (l / 16) + v, column l % 16.  A wave's codes come
// straight to registers, kFewSteps steps of 128 elements at a time, all of them asked for before the first is used;
// the matrix is known before the rows are, so its loads go first.  The waves' sums meet in LDS and are added in order.
constexpr int kFewSteps = 4, kFewWaves = 8;
typedef float f32x4v __attribute__((ext_vector_type(4)));

template <typename OutT, bool GATED>
__global__ __launch_bounds__(64 * kFewWaves) void grouped_few_kernel(GroupedArgs a) {
  __shared__ f32x4v part[kFewWaves][2][64];
  const int lane = threadIdx.x & 63, wave = wave_index(), r16 = lane & 15, h = lane >> 4;
  if (a.zeroed) zero_rest<OutT>(a);
  uint32_t err = 0;
  if (blockIdx.x == 0 && wave == 0 && offsets_bad(a.groups)) err = FP4Q_DATA_BAD_GROUP;
  const int lin = tile_number(a);
  const TileGroup g = find_group(a.groups, kFewRows16, lin / a.tiles_n);
  if (g.group < 0) {
    Status{a.status, true}.finish(err);
    return;
  }
  const GroupTile t = group_tile(a, g, kFewRows16, lin);
  const int n0 = t.col * (GATED ? kFewCols / 2 : kFewCols);
  const int64_t kb = a.k / 2, ksc = a.k / 32;
  const int p = t.lo + r16 < t.hi ? t.lo + r16 : t.hi - 1;
  const uint8_t *b[2], *bs[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int col = GATED ? n0 + r16 : n0 + 16 * j + r16;
    const int64_t row = (int64_t)g.group * a.n + (col < a.n_out ? col : a.n_out - 1) + (GATED && j ? a.n_out : 0);
    b[j] = a.b + row * kb + 16 * h;
    bs[j] = a.bs + row * ksc;
  }
  const int nst = a.k / 128, per = (nst + kFewWaves - 1) / kFewWaves;
  const int s0 = wave * per, s1 = s0 + per < nst ? s0 + per : nst;
  f32x4v acc[2] = {f32x4v{0, 0, 0, 0}, f32x4v{0, 0, 0, 0}};
  const int e = entry_at(a.groups, p);
  const int64_t ar = a.gather ? a_row(a, p, e) : p;
  const uint8_t *A = a.a + ar * kb + 16 * h, *As = a.as + ar * ksc;
  for (int s = s0; s < s1; s += kFewSteps) {
    i32x4 bc[2][kFewSteps], ac[kFewSteps];
    uint32_t bw[2][kFewSteps], aw[kFewSteps];
#pragma unroll
    for (int q = 0; q < kFewSteps; ++q) {
      const int st = s + q < s1 ? s + q : s1 - 1;  // past the wave's last step: loaded, and multiplied by zeros
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        bc[j][q] = *reinterpret_cast<const i32x4 *>(b[j] + 64 * (int64_t)st);
        bw[j][q] = *reinterpret_cast<const uint32_t *>(bs[j] + 4 * (int64_t)st);
      }
    }
#pragma unroll
    for (int q = 0; q < kFewSteps; ++q) {
      const int st = s + q < s1 ? s + q : s1 - 1;
      ac[q] = *reinterpret_cast<const i32x4 *>(A + 64 * (int64_t)st);
      aw[q] = *reinterpret_cast<const uint32_t *>(As + 4 * (int64_t)st);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int q = 0; q < kFewSteps; ++q) {
      const bool in = s + q < s1;
      const i32x8 av = {in ? ac[q][0] : 0, in ? ac[q][1] : 0, in ? ac[q][2] : 0, in ? ac[q][3] : 0, 0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const i32x8 bv = {bc[j][q][0], bc[j][q][1], bc[j][q][2], bc[j][q][3], 0, 0, 0, 0};
        acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, acc[j], 4, 4, 0, (int)(aw[q] >> (8 * h)), 0,
                                                                  (int)(bw[j][q] >> (8 * h)));
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) part[wave][j][lane] = acc[j];
  __syncthreads();
  if (wave < (GATED ? 1 : 2)) {
    f32x4v sum[2];
#pragma unroll
    for (int j = 0; j < (GATED ? 2 : 1); ++j) {
      sum[j] = part[0][GATED ? j : wave][lane];
#pragma unroll
      for (int w = 1; w < kFewWaves; ++w) sum[j] += part[w][GATED ? j : wave][lane];
    }
    const int col = GATED ? n0 + r16 : n0 + 16 * wave + r16;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int q = t.lo + 4 * h + v;
      const int eq = q < t.hi ? entry_at(a.groups, q) : -1;
      if (q < t.hi && eq < 0) err = FP4Q_DATA_BAD_GROUP;
      float z = a.alpha * sum[0][v];
      if constexpr (GATED) z = silu(z) * (a.alpha * sum[1][v]);
      if (eq >= 0 && col < a.n_out) store_out((OutT *)a.c + (int64_t)(a.scatter ? eq : q) * a.ldc + col, z);
    }
  }
  Status{a.status, true}.finish(err);
}

// ---------------------------------------------------------------------------
// The ring in tiles of 256 x 256 for many of them (K a multiple of 256, from 512 on; up to kPersistGroups groups): one
// workgroup a CU walks tiles gridDim apart, and loads the next tile's first stages while it finishes the one before.
// Started anew, a tile costs 8 us beside its stages (2.4 us for 256 elements of K): the search for its
// group, its rows' numbers, the first loads, the stores.  Here the groups' tiles are summed once into LDS, and the next
// tile's loads follow the last ones of the tile without a gap.  Its rows are looked up when a tile begins; where they are
// gathered, that is up to six trips to memory one after the other, each number being checked before the next is asked for.
template <typename OutT, bool GATED>
__global__ __launch_bounds__(512) void grouped_persist_kernel(GroupedArgs a) {
  constexpr int WGN = 4, TM = 4, TN = 2;
  using S = RingShape<GATED, 2, WGN, TM, TN>;
  constexpr int ROWB = kRowBytes, WAVES = S::WAVES, BM = S::BM, CPR = S::CPR, KS = S::KS, SPR = S::SPR;
  constexpr int STAGE = S::STAGE, RPL = 1024 / ROWB, LOADS = BM / RPL / WAVES;  // 1 KB loads of A, and of B, a wave
  constexpr int RPS = 256 / SPR;  // rows of a scale load: a wave's first is A's, its second B's
  static_assert(BM == S::BN && BM == RPS * WAVES, "a wave brings the scales of 32 rows of A and of B");
  constexpr int ROWS_OFF = 2 * STAGE, SUMS_OFF = ROWS_OFF + 2 * 4 * BM, SPANS_OFF = SUMS_OFF + 4 * (kPersistGroups + 2);
  __shared__ __attribute__((aligned(1024))) uint8_t smem[SPANS_OFF + 8 * kPersistGroups];
  int *row_of = reinterpret_cast<int *>(smem + ROWS_OFF);  // rows of C of this tile and of the next, -1: not stored
  int *sums = reinterpret_cast<int *>(smem + SUMS_OFF);    // row tiles of the groups before
  int2 *spans = reinterpret_cast<int2 *>(smem + SPANS_OFF);

  const int tid = threadIdx.x, lane = tid & 63, wave = wave_index();
  const int wm = wave / WGN, wn = wave % WGN, l32 = lane & 31, h = lane >> 5;
  if (a.zeroed) zero_rest<OutT>(a);
  uint32_t err = 0;
  if (wave == 0) {
    int run = 0;
    bool bad = a.groups.offsets[0] != 0;
    for (int g0 = 0; g0 < a.groups.groups; g0 += 64) {
      const int g = g0 + lane;
      const bool in = g < a.groups.groups;
      const GroupSpan s = group_span(in ? a.groups.offsets[g] : 0, in ? a.groups.offsets[g + 1] : 0, a.groups.entries);
      const int mine = in ? span_tiles(s.lo, s.hi, BM) : 0, upto = wave_scan(mine);
      if (in) {
        sums[g] = run + upto - mine;
        spans[g] = int2{s.lo, s.hi};
      }
      bad |= s.bad;
      run += __builtin_amdgcn_readlane(upto, 63);
    }
    if (lane == 0) sums[a.groups.groups] = run;
    if (blockIdx.x == 0 && __ballot(bad)) err = FP4Q_DATA_BAD_GROUP;
  }
  __syncthreads();
  const int total = __builtin_amdgcn_readfirstlane(sums[a.groups.groups]) * a.tiles_n;

  struct Tile {
    int lin, group, lo, hi, n0;  // n0: first column of C
  };
  auto find = [&](int v) {  // tile of workgroup number v
    Tile t;
    const int local = v / kXcdCount;
    t.lin = __builtin_amdgcn_readfirstlane((local / a.run * kXcdCount + v % kXcdCount) * a.run + local % a.run);
    t.group = -1;
    if (t.lin >= total) return t;
    const int want = t.lin / a.tiles_n;
    for (int g0 = 0; g0 < a.groups.groups; g0 += 64) {
      const int g = g0 + lane;
      const uint64_t hit = __ballot(g < a.groups.groups && sums[g < a.groups.groups ? g + 1 : 0] > want);
      if (hit) {
        t.group = g0 + __ffsll((unsigned long long)hit) - 1;
        break;
      }
    }
    const int2 s = spans[t.group];
    const TileGroup g{t.group, __builtin_amdgcn_readfirstlane(s.x), __builtin_amdgcn_readfirstlane(s.y),
                      __builtin_amdgcn_readfirstlane(sums[t.group])};
    const GroupTile w = group_tile(a, g, BM, t.lin);
    t.group = __builtin_amdgcn_readfirstlane(t.group);
    t.lo = __builtin_amdgcn_readfirstlane(w.lo);
    t.hi = __builtin_amdgcn_readfirstlane(w.hi);
    t.n0 = __builtin_amdgcn_readfirstlane(w.col * S::COLS);
    return t;
  };

  // Rows of A that this lane's loads of a tile take, and (threads below BM) the entry of a tile row.
  struct Numbers {
    int a[LOADS], s, entry;
  };
  auto numbers = [&](const Tile &t) {
    Numbers r;
    auto of = [&](int i) {
      const int p = t.lo + i < t.hi ? t.lo + i : t.hi - 1;
      return a.gather ? entry_at(a.groups, p) : p;
    };
#pragma unroll
    for (int i = 0; i < LOADS; ++i) r.a[i] = of((wave * LOADS + i) * RPL + lane / CPR);
    r.s = of(RPS * wave + lane / 2);
    const int p = t.lo + tid;
    r.entry = tid < BM && p < t.hi ? entry_at(a.groups, p) : -1;
    return r;
  };
  const uint32_t kb = a.k / 2, ksc = a.k / 32;
  const int nst = a.k / (2 * ROWB);
  uint32_t offA[LOADS], offB[LOADS], offAs, offBs;  // of the tile whose stages are being issued
  const uint8_t *B = nullptr, *Bs = nullptr;
  auto set_sources = [&](const Tile &t, const Numbers &r, int which) {
    const int lane = fp4q_gemm::opaque_lane();
    auto a_of = [&](int n) { return (uint32_t)(a.gather ? (n < 0 ? 0 : n / a.gather) : n); };
    auto b_of = [&](int i) {
      const int col = t.n0 + (GATED ? (i / 64) * 32 + (i & 31) : i);
      return (uint32_t)((col < a.n_out ? col : a.n_out - 1) + (GATED && (i & 32) ? a.n_out : 0));
    };
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int row = (wave * LOADS + i) * RPL + lane / CPR, chunk = (lane % CPR) ^ fp4q_gemm::swz<ROWB>(row);
      offA[i] = a_of(r.a[i]) * kb + 16 * chunk;
      offB[i] = b_of(row) * kb + 16 * chunk;
    }
    offAs = a_of(r.s) * ksc + 4 * (lane % 2);
    offBs = b_of(RPS * wave + lane / 2) * ksc + 4 * (lane % 2);
    B = a.b + (int64_t)t.group * a.n * kb;
    Bs = a.bs + (int64_t)t.group * a.n * ksc;
    if (tid < BM) {
      const int p = t.lo + tid;
      if (p < t.hi && r.entry < 0) err = FP4Q_DATA_BAD_GROUP;
      row_of[which * BM + tid] = r.entry < 0 ? -1 : (a.scatter ? r.entry : p);
    }
  };
  auto issue = [&](int st, int slot) {
    uint8_t *base = smem + slot * STAGE;
    const uint8_t *a_st = a.a + (int64_t)st * ROWB, *b_st = B + (int64_t)st * ROWB;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) fp4q_gemm::load_lds16(a_st + offA[i], base + (wave * LOADS + i) * 1024);
#pragma unroll
    for (int i = 0; i < LOADS; ++i)
      fp4q_gemm::load_lds16(b_st + offB[i], base + S::A_BYTES + (wave * LOADS + i) * 1024);
    fp4q_gemm::load_lds4(a.as + (int64_t)st * SPR + offAs, base + S::SA_OFF + 256 * wave);
    fp4q_gemm::load_lds4(Bs + (int64_t)st * SPR + offBs, base + S::SB_OFF + 256 * wave);
  };

  f32x16 acc[TM][TN];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = f32x16{0};
  };
  struct Ops {
    i32x8 a[TM], b[TN];
    int sa[TM], sb[TN];
  };
  const int lane_sw = fp4q_gemm::swz<ROWB>(l32);
  auto read_ops = [&](int slot, auto ks_c, Ops &o, const Ops &prev) {
    constexpr int ks = decltype(ks_c)::value;
    const uint8_t *base = smem + slot * STAGE;
    const uint8_t *at = base + l32 * ROWB + 16 * ((h * KS + ks) ^ lane_sw);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const i32x4 v = *reinterpret_cast<const i32x4 *>(at + (wm * TM + i) * 32 * ROWB);
      o.a[i] = i32x8{v.x, v.y, v.z, v.w, 0, 0, 0, 0};
      const uint8_t *scales = base + S::SA_OFF + SPR * ((wm * TM + i) * 32 + l32) + 4 * h;
      o.sa[i] = ks == 0 ? (int)*reinterpret_cast<const uint32_t *>(scales) : prev.sa[i];
    }
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const i32x4 v = *reinterpret_cast<const i32x4 *>(at + S::A_BYTES + (wn * TN + j) * 32 * ROWB);
      o.b[j] = i32x8{v.x, v.y, v.z, v.w, 0, 0, 0, 0};
      const uint8_t *scales = base + S::SB_OFF + SPR * ((wn * TN + j) * 32 + l32) + 4 * h;
      o.sb[j] = ks == 0 ? (int)*reinterpret_cast<const uint32_t *>(scales) : prev.sb[j];
    }
  };
  auto mfmas = [&](const Ops &o, auto ks_c) {
    constexpr int ks = decltype(ks_c)::value;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(o.b[j], o.a[i], acc[i][j], 4, 4, ks, o.sb[j], ks,
                                                                    o.sa[i]);
  };
  auto pin = [&]() {  // the MFMAs issued so far are placed here
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) __asm__ volatile("" : "+v"(acc[i][j]));
  };
  auto stage_barrier = [&]() {
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
  };

  constexpr int WCOLS = S::COLS / WGN, VEC = 16 / (int)sizeof(OutT), EROW = WCOLS + VEC;
  constexpr int LPR = WCOLS / VEC, RPI = 64 / LPR;
  static_assert(WAVES * 32 * EROW * (int)sizeof(OutT) <= STAGE, "epilogue staging must fit in a stage");
  const bool wide = ((uintptr_t)a.c % 16 == 0) && ((a.ldc * (int64_t)sizeof(OutT)) % 16 == 0);
  auto epilogue = [&](const Tile &t, int which, uint8_t *room) {
    const int ln = fp4q_gemm::opaque_lane(), l32 = ln & 31, h = ln >> 5;
    OutT *area = reinterpret_cast<OutT *>(room) + wave * 32 * EROW;
    OutT *C = (OutT *)a.c;
    const float alpha = a.alpha;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      constexpr int JS = GATED ? 2 : 1;
#pragma unroll
      for (int j = 0; j < TN; j += JS)
#pragma unroll
        for (int v = 0; v < 16; v += 4)
          stage_four<OutT, GATED>(acc[i][j], acc[i][j + JS - 1], v, alpha,
                                  area + l32 * EROW + j / JS * 32 + 2 * v + 4 * h);
#pragma unroll
      for (int q = 0; q < 32 / RPI; ++q) {
        const int rr = q * RPI + ln / LPR, c = ln % LPR * VEC;
        const int row = row_of[which * BM + (wm * TM + i) * 32 + rr], col = t.n0 + wn * WCOLS + c;
        const i32x4 v = *reinterpret_cast<const i32x4 *>(area + rr * EROW + c);
        if (row >= 0) {
          OutT *dst = C + (int64_t)row * a.ldc + col;
          if (wide && col + VEC <= a.n_out) {
            *reinterpret_cast<i32x4 *>(dst) = v;
          } else {
            const OutT *e = reinterpret_cast<const OutT *>(&v);
#pragma unroll
            for (int x = 0; x < VEC; ++x)
              if (col + x < a.n_out) dst[x] = e[x];
          }
        }
      }
    }
  };

  // The issue stream runs over the stages of all this workgroup's tiles, two ahead of the MFMAs; a tile's stage g sits
  // in the slot that follows the one before.  Every wait is for all of a wave's loads (and the epilogue's stores).
  // A workgroup moves on by one within its XCD from one of its tiles to the next: where groups have two row tiles, a whole
  // one and a remainder (which takes half as long), it would else get the same kind every time (272 rows a group 248 us,
  // so 227; 256 on average 210 and 207).
  int walked = 0;
  auto number = [&](int i) {
    const int b = (int)blockIdx.x, eighth = (int)gridDim.x / kXcdCount;
    return i * (int)gridDim.x + (b / kXcdCount + i) % eighth * kXcdCount + b % kXcdCount;
  };
  Tile cur = find(number(0)), nxt;
  if (cur.group >= 0) {
    set_sources(cur, numbers(cur), 0);
    issue(0, 0);
    issue(1, 1);
    fp4q_gemm::wait_lgkmcnt0();
    fp4q_gemm::wait_vmcnt<2 * LOADS + 2>();
    stage_barrier();
    int slot = 0, which = 0;
    Numbers ahead;
    auto stage_end = [&]() {
      __builtin_amdgcn_sched_barrier(0);
      fp4q_gemm::wait_lgkmcnt0();  // this wave's reads of the stage are complete
      fp4q_gemm::wait_vmcnt<0>();  // the next one has landed
      stage_barrier();             // ... for every wave, and nobody reads this one any more
    };
    // The stages of a tile, by waves that have rows of it and by those that only load.
    auto walk = [&](auto live_c) {
      constexpr bool LIVE = decltype(live_c)::value;
      Ops o0, o1;
      if constexpr (LIVE) {
        clear();
        read_ops(slot, std::integral_constant<int, 0>{}, o0, o1);
      }
      auto body = [&]() {
        if constexpr (LIVE) {
          fp4q_gemm::unroll(std::make_integer_sequence<int, KS - 1>{}, [&](auto ks_c) {
            constexpr int ks = decltype(ks_c)::value;
            if constexpr (ks % 2 == 0) {
              read_ops(slot, std::integral_constant<int, ks + 1>{}, o1, o0);
              __builtin_amdgcn_sched_barrier(0);
              mfmas(o0, ks_c);
            } else {
              read_ops(slot, std::integral_constant<int, ks + 1>{}, o0, o1);
              __builtin_amdgcn_sched_barrier(0);
              mfmas(o1, ks_c);
            }
          });
          pin();
        }
        stage_end();
      };
#pragma nounroll
      for (int st = 0; st + 1 < nst; ++st) {
        body();
        if (st + 2 < nst) {
          issue(st + 2, slot);
        } else if (nxt.group >= 0) {  // the next tile's first stage
          set_sources(nxt, ahead, which ^ 1);
          issue(0, slot);
        }
        slot ^= 1;
        if constexpr (LIVE) {
          read_ops(slot, std::integral_constant<int, 0>{}, o0, o1);
          __builtin_amdgcn_sched_barrier(0);
          mfmas(o1, std::integral_constant<int, KS - 1>{});
        }
      }
      body();  // the last stage: its slot takes the epilogue's staging before the next tile's second stage
      if constexpr (LIVE) {
        mfmas(o1, std::integral_constant<int, KS - 1>{});
        pin();
        epilogue(cur, which, smem + slot * STAGE);
      }
    };
#pragma nounroll
    for (;;) {
      nxt = find(number(++walked));
      if (nxt.group >= 0) ahead = numbers(nxt);
      if (cur.lo + wm * TM * 32 < cur.hi) walk(std::true_type{});
      else walk(std::false_type{});
      if (nxt.group < 0) break;
      fp4q_gemm::wait_lgkmcnt0();  // this wave's reads of the staging are complete
      stage_barrier();             // ... for every wave: the slot may be filled
      issue(1, slot);
      slot ^= 1;
      which ^= 1;
      cur = nxt;
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

// Launches a kernel; false where it has too many tiles.
template <typename K>
bool launch_tiles(K kernel, GroupedArgs &a, const ProductTiles &t, int threads, hipStream_t s) {
  if (t.workgroups > kMaxTiles) return false;
  a.tiles_n = (int)ceil_div(a.n, t.cols);
  a.run = t.run;
  hipLaunchKernelGGL(kernel, dim3((unsigned)t.workgroups), dim3(threads), 0, s, a);
  return true;
}

template <typename O, bool GATED>
bool launch(GroupedArgs &a, hipStream_t s) {
  const ProductTiles t = product_tiles(a.groups.entries, a.groups.groups, a.n, a.k, a.a_rows);
  auto go = [&](auto kernel, int threads) { return launch_tiles(kernel, a, t, threads, s); };
  if (t.kind == kPersistTiles) return go(grouped_persist_kernel<O, GATED>, 512);
  if (t.kind == kAnyTiles) return go(grouped_any_kernel<O, GATED>, kAnyThreads);
  if (t.kind == kFewTiles) return go(grouped_few_kernel<O, GATED>, 64 * kFewWaves);
  if (t.kind == kDeepTiles) return go(grouped_ring_kernel<O, GATED, false, 3, 2, 2, 1, 2>, 256);
  auto ring = [&](auto tail) {
    constexpr bool TAIL = decltype(tail)::value;
    if (t.rows == 128) return go(grouped_ring_kernel<O, GATED, TAIL, 2, 2, 2, 2, 2>, 256);
    return go(grouped_ring_kernel<O, GATED, TAIL, 2, 2, 2, 1, 2>, 256);
  };
  return a.k % 256 ? ring(std::true_type{}) : ring(std::false_type{});
}

fp4q_status_t hip_status() { return hipGetLastError() == hipSuccess ? FP4Q_OK : FP4Q_ERR_HIP; }

// The calls of the header; zeroed: rows of C of entries of no group become zeros.
fp4q_status_t grouped_call(const uint8_t *a_codes, const uint8_t *a_scales, int64_t a_rows, const uint8_t *b_codes,
                           const uint8_t *b_scales, const fp4q_row_groups_t *groups, int64_t n, int64_t k,
                           int64_t gather, int scatter, int gated, float alpha, fp4q_dtype_t out_dtype, void *c,
                           int64_t ldc, void *workspace, size_t workspace_bytes, void *stream, bool zeroed) {
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
  GroupedArgs a{a_codes, a_scales, b_codes, b_scales, groups_of(*groups), (int)a_rows, (int)gather, scatter, (int)n,
                (int)k, (int)(gated ? n / 2 : n), 0, 1, alpha, c, ldc, status, zeroed};
  bool fits = true;
  with_type(out_dtype, [&](auto op) {
    using O = std::remove_pointer_t<decltype(op)>;
    if (gated) fits = launch<O, true>(a, s);
    else fits = launch<O, false>(a, s);
  });
  if (!fits) return FP4Q_ERR_SHAPE;
  return hip_status();
}

}  // namespace
}  // namespace fp4q

using namespace fp4q;

extern "C" fp4q_status_t fp4q_gemm_mxfp4_grouped(const uint8_t *a_codes, const uint8_t *a_scales, int64_t a_rows,
                                                 const uint8_t *b_codes, const uint8_t *b_scales,
                                                 const fp4q_row_groups_t *groups, int64_t n, int64_t k,
                                                 int64_t gather, int scatter, int gated, float alpha,
                                                 fp4q_dtype_t out_dtype, void *c, int64_t ldc, void *workspace,
                                                 size_t workspace_bytes, void *stream) {
  return grouped_call(a_codes, a_scales, a_rows, b_codes, b_scales, groups, n, k, gather, scatter, gated, alpha, out_dtype,
                      c, ldc, workspace, workspace_bytes, stream, false);
}

extern "C" fp4q_status_t fp4q_gemm_mxfp4_grouped_zeroed(const uint8_t *a_codes, const uint8_t *a_scales, int64_t a_rows,
                                                        const uint8_t *b_codes, const uint8_t *b_scales,
                                                        const fp4q_row_groups_t *groups, int64_t n, int64_t k,
                                                        int64_t gather, int scatter, int gated, float alpha,
                                                        fp4q_dtype_t out_dtype, void *c, int64_t ldc,
                                                        void *workspace, size_t workspace_bytes, void *stream) {
  return grouped_call(a_codes, a_scales, a_rows, b_codes, b_scales, groups, n, k, gather, scatter, gated, alpha, out_dtype,
                      c, ldc, workspace, workspace_bytes, stream, true);
}
