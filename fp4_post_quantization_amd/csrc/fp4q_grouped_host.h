// Argument checks, sizes and index arithmetic of the grouped calls
// (include/fp4q_grouped.h): plain C++ without HIP, so that a host program can
// exercise them; the functions marked FP4Q_HD are the ones the kernels run.
#pragma once

#include <math.h>
#include <stdint.h>

#include "fp4q.h"
#include "fp4q_grouped.h"
#include "fp4q_kv_host.h"

namespace fp4q {

constexpr int64_t kMaxRowGroups = 2048;
constexpr int64_t kMaxEntries = (int64_t)1 << 30;
constexpr int64_t kMaxExperts = 1024;
constexpr int64_t kMaxTopK = 64;
constexpr int64_t kMaxTiles = (int64_t)1 << 22;  // workgroups of a launch: with 1024 threads each below 2^32 threads

inline bool grouped_ws_ok(const void *ws, size_t bytes, size_t need) {
  return ws && bytes >= need && kv_aligned(ws, 16);
}

inline fp4q_status_t grouped_check(const fp4q_row_groups_t &g) {
  if (g.groups < 1 || g.groups > kMaxRowGroups || g.entries < 0 || g.entries > kMaxEntries) return FP4Q_ERR_SHAPE;
  if (!g.offsets || (g.entries && !g.rows)) return FP4Q_ERR_NULL;
  if (!kv_aligned(g.offsets, 4) || !kv_aligned(g.rows, 4)) return FP4Q_ERR_ALIGN;
  return FP4Q_OK;
}

// Rows of n elements of `size` bytes, ld apart: the last one ends before 2^62
// bytes from the first.
inline bool grouped_rows_ok(int64_t rows, int64_t n, int64_t ld, int64_t size) {
  return n >= 0 && ld >= n && ((__int128)(rows > 0 ? rows - 1 : 0) * ld + n) * size < ((__int128)1 << 62);
}

// ---------------------------------------------------------------- tiles ----

// Entries lo .. hi - 1 of a group as the kernels see them: its offsets cut to
// the entries there are.
struct GroupSpan {
  int lo, hi;
  bool bad;
};
FP4Q_HD GroupSpan group_span(int o0, int o1, int entries) {
  GroupSpan s;
  s.bad = o0 < 0 || o1 < o0 || o1 > entries;
  s.lo = o0 < 0 ? 0 : (o0 > entries ? entries : o0);
  s.hi = o1 > entries ? entries : o1;
  if (s.hi < s.lo) s.hi = s.lo;
  return s;
}
FP4Q_HD int span_tiles(int lo, int hi, int rows) { return (int)(((int64_t)hi - lo + rows - 1) / rows); }

// Row tiles of that many rows that all groups have, at most: each has its
// whole ones and one that is not full.
inline int64_t most_tiles(int64_t entries, int64_t groups, int64_t rows) {
  return entries / rows + (groups < entries ? groups : entries);
}

inline fp4q_status_t grouped_product_check(const fp4q_row_groups_t &g, int64_t a_rows, int64_t n, int64_t k,
                                           int64_t gather, int gated, int64_t ldc, int64_t size) {
  const int64_t most = (int64_t)1 << 31;
  if (n < 0 || n >= most || k <= 0 || k % 32 || k >= most || (gated && n % 2)) return FP4Q_ERR_SHAPE;
  if (a_rows < 0 || a_rows >= most || gather < 0 || gather >= most) return FP4Q_ERR_SHAPE;
  if (gather ? a_rows < (g.entries + gather - 1) / gather : a_rows < g.entries) return FP4Q_ERR_SHAPE;
  if (!grouped_rows_ok(g.entries, gated ? n / 2 : n, ldc, size)) return FP4Q_ERR_SHAPE;
  if ((__int128)g.groups * n * (k / 2) >= ((__int128)1 << 62)) return FP4Q_ERR_SHAPE;
  return FP4Q_OK;
}

constexpr int kXcdCount = 8;
constexpr int kPersistGroups = 512;
constexpr int kAnyRows = 64, kAnyCols = 128;
constexpr int kFewRows16 = 16, kFewCols = 32;
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The kernel of a grouped product, its tiles (rows of A times rows of B), and the tiles in a row that go to one XCD.
enum ProductKind { kAnyTiles, kFewTiles, kRingTiles, kDeepTiles, kPersistTiles };
struct ProductTiles {
  ProductKind kind;
  int rows, cols, run;
  int64_t workgroups;
};
inline ProductTiles product_tiles(int64_t entries, int64_t groups, int64_t n, int64_t k, int64_t a_rows) {
  ProductTiles t;
  const int64_t far = (int64_t)UINT32_MAX - 4096;  // the ring's kernels take 32-bit offsets into A and into a matrix
  auto tiles = [&](int rows, int cols) { return most_tiles(entries, groups, rows) * ceil_div(n, cols); };
  // Tiles in a row to one XCD: 16 where there are many (2000 tokens of 64 experts, 704 x 2048, in runs of 4 49 us, of
  // 16 45; 16 tokens of 128 experts 44.5 and 43.8), 4 where long runs would leave XCDs without any (one token, in runs
  // of 64: 25 us instead of 18).
  auto run = [&](int rows) { return tiles(rows, 128) >= 512 ? 16 : 4; };
  if (k < 256 || a_rows * (k / 2) > far || n * (k / 2) > far) {
    t = ProductTiles{kAnyTiles, kAnyRows, kAnyCols, 1, tiles(kAnyRows, kAnyCols)};
    return t;
  }
  const int64_t rows = entries / (groups < entries ? groups : (entries ? entries : 1));  // of a group, on average
  // Measured, us, gate and up products of 4096 x 1536 unless said:
  // few rows (16 x 32) where a call has at most one tile a CU: 2 rows on 4096 x 4096 7.2, in tiles of 64 x 128 10.0; on
  // 14336 x 4096 19.6 and 25.6; 4 rows on 1408 x 2048 5.1 and 7.3.  With more the tiles of 64 rows are faster: 8 rows of 8
  // experts (384 tiles) 11.6 and 11.3, on 2048 x 2048 (512) 11.8 and 7.6, of 16 tokens (3600) 70 and 43.
  if (k % 128 == 0 && tiles(kFewRows16, kFewCols) <= kCus) {
    t = ProductTiles{kFewTiles, kFewRows16, kFewCols, 4, 0};
  } else if (rows <= 64) {
    // 64 rows up to 64 a group: 16 tokens of 128 experts 47, with 128 50; 64 tokens 92 and 100; 512 (32 rows) 115 and
    // 116; 1000 (62 rows) 130 and 130; 1500 (94 rows) 157 and 145.  A third stage in flight where K has many, at two
    // workgroups a CU instead of three: 43, 89, 105 and 126; 64 tokens of 8 experts on 14336 x 4096 44 and 40; 1000
    // tokens on 768 x 4096 74 and 85.
    t = ProductTiles{k % 256 == 0 && k >= 4096 ? kDeepTiles : kRingTiles, 64, 128, run(64), 0};
  } else {
    const int64_t live = groups < entries ? groups : entries;
    auto rounds = [&](int64_t r, int64_t c, int64_t at_once) {  // every group's last tile half full
      return ceil_div((entries / r + live / 2) * ceil_div(n, c), at_once);
    };
    // 256 x 256, one a CU, where it takes fewer rounds of 1.55 times the length than 128 x 128, two a CU: 2500 tokens
    // of 128 experts (156 rows) 173 and 187; 4096 tokens (256) 215 and 253; 768 x 4096 151 and 192; 2048 rows on 4096 x
    // 4096 192 and 244; 512 rows on 4096 x 4096 (two rounds, the second a quarter full) 74 and 68; 94 rows 149 and 145.
    // All of it goes by the average, entries of no group included: the offsets are on the device.  2048 tokens of 128
    // experts, 8 each, take 167; with nine of ten on the same 8 experts 198.
    if (k % 256 == 0 && k >= 512 && groups <= kPersistGroups &&
        155 * rounds(256, 256, 256) <= 100 * rounds(128, 128, 512))
      t = ProductTiles{kPersistTiles, 256, 256, 16, 0};
    else
      t = ProductTiles{kRingTiles, 128, 128, run(128), 0};
  }
  t.workgroups = ceil_div(tiles(t.rows, t.cols), t.run * kXcdCount) * t.run * kXcdCount;
  if (t.kind == kPersistTiles && t.workgroups > kCus && t.workgroups <= kMaxTiles) t.workgroups = kCus;
  return t;
}

// --------------------------------------------------------------- routing ----

inline fp4q_status_t router_check(const fp4q_router_t &r, int64_t experts) {
  if (r.score != FP4Q_SOFTMAX && r.score != FP4Q_SIGMOID) return FP4Q_ERR_ARG;
  if (r.renormalize != 0 && r.renormalize != 1) return FP4Q_ERR_ARG;
  if (r.group_best != 1 && r.group_best != 2) return FP4Q_ERR_ARG;
  if (!(fabsf(r.scale) <= 3.4028234e38f)) return FP4Q_ERR_ARG;
  if (experts < 1 || experts > kMaxExperts) return FP4Q_ERR_SHAPE;
  if (r.top_k < 1 || r.top_k > kMaxTopK || r.top_k > experts) return FP4Q_ERR_SHAPE;
  if (r.n_groups < 1 || r.n_groups > 64 || experts % r.n_groups || r.top_groups < 1 || r.top_groups > r.n_groups)
    return FP4Q_ERR_SHAPE;
  if (!kv_aligned(r.bias, 4)) return FP4Q_ERR_ALIGN;
  return FP4Q_OK;
}

constexpr int kSortChunk = 1024;  // entries that a workgroup places at a time

// Tokens up to which one workgroup routes and sorts (one launch, which from Python saves 4 us of a call): 24 of 64 experts
// 8.4 us on the GPU, in two launches 9.9, and where scores are compared (with a bias, in groups) 12.6 and 11.5; of 128
// 10.2 and 10.4, scores 17.0 and 13.1; of 256 11.7 and 11.4.  16 of 128 with scores 12.8 and 13.1, of 256 16.4 and 15.2.
inline int64_t solo_tokens(int64_t experts, bool scored) {
  return experts <= 64 || (!scored && experts <= 256) ? 24 : 16;
}

// How entries are counted and placed.  Counting block b holds the units
// (tokens, or entries of ids) [b per, (b + 1) per); placing block p holds
// `join` counting blocks.
struct SortPlan {
  int64_t per, blocks;   // units of a counting block, counting blocks
  int64_t join, places;  // counting blocks of a placing block, placing blocks
};
inline SortPlan sort_plan(int64_t units, int64_t per_unit, int64_t least) {
  SortPlan p;
  p.per = ceil_div(units, 512);
  if (p.per < least) p.per = least;
  if (p.per > 65535 / per_unit) p.per = 65535 / per_unit;  // counts are 16 bits
  p.blocks = ceil_div(units, p.per);
  p.join = kSortChunk / (p.per * per_unit);
  if (p.join < 1) p.join = 1;
  p.places = ceil_div(p.blocks, p.join);
  return p;
}
// 16-bit counts of a counting block: of the groups, then of the entries of no group, padded to 16 bytes.
FP4Q_HD int sort_stride(int groups) { return (groups + 8) & ~7; }
inline size_t sort_bytes(const SortPlan &p, int64_t groups) {
  return 256 + (size_t)(p.blocks * sort_stride((int)groups) * 2);
}

// -------------------------------------------------------------- adapters ----

inline fp4q_status_t lora_check_sizes(int64_t entries, int64_t groups, int64_t n, int64_t k, int64_t rank) {
  const int64_t most = (int64_t)1 << 31;
  if (entries < 0 || entries > kMaxEntries || groups < 1 || groups > kMaxRowGroups) return FP4Q_ERR_SHAPE;
  if (n < 0 || n >= most || k < 8 || k >= most || k % 8 || rank < 8 || rank > 256 || rank % 8) return FP4Q_ERR_SHAPE;
  return FP4Q_OK;
}

// few: B meets 16 rows at a time, else 64 (8191 rows, rank 64, N 14336: 131 us, with 32 145), but 32 in float32 and for
// ranks beyond 64, which take twice the registers and LDS (4000 rows, rank 128, N 4096: 42 us, with 64 the same; rank 256
// does not fit a CU's LDS twice).
// splits: of K, over workgroups.
struct LoraPlan {
  bool few;
  int64_t splits;
};
inline LoraPlan lora_plan(int64_t entries, int64_t groups, int64_t k) {
  LoraPlan p;
  p.few = entries < 64 * groups || entries <= 256;
  const int64_t tiles = most_tiles(entries, groups, 16);
  const int64_t steps = ceil_div(k, 32) / 16;  // at least two stages of 64 a wave
  p.splits = tiles ? 256 / tiles : 1;
  if (p.splits > steps) p.splits = steps;
  if (p.splits > 8) p.splits = 8;
  if (p.splits < 1) p.splits = 1;
  return p;
}
inline int64_t lora_rows(const LoraPlan &p, int64_t rank, int64_t size) {
  return p.few ? 16 : (size == 4 || rank > 64 ? 32 : 64);
}

}  // namespace fp4q
