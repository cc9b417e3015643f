// Argument checks and index arithmetic of the key/value cache calls: plain
// C++ without HIP, so that a host program can exercise them; the functions
// marked FP4Q_HD are the ones the kernels run.
#pragma once

#include <math.h>
#include <stdint.h>

#include "fp4q.h"
#include "fp4q_kv.h"

#ifdef __HIPCC__
#define FP4Q_HD __host__ __device__ __forceinline__
#else
#define FP4Q_HD inline
#endif

namespace fp4q {


inline bool kv_aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

inline int kv_log2(int64_t n) {
  int k = 0;
  while (((int64_t)1 << k) < n) ++k;
  return k;
}

inline bool kv_head_dim_ok(int64_t d) { return d == 64 || d == 128 || d == 256; }

// Elements of a tensor of heads: below 2^33, so that a grid of one thread for
// every 8 of them has fewer than the 2^32 threads that a launch may have.
inline bool kv_size_ok(int64_t tokens, int64_t heads, int64_t head_dim) {
  return tokens >= 0 && (heads == 0 || tokens < ((int64_t)1 << 33) / (heads * head_dim));
}

inline fp4q_status_t kv_check_heads(fp4q_dtype_t dtype, int64_t tokens, int64_t heads, int64_t head_dim,
                                    int64_t token_stride, int64_t head_stride, const void *x) {
  if (dtype != FP4Q_F32 && dtype != FP4Q_BF16) return FP4Q_ERR_ARG;
  if (tokens < 0 || heads < 0 || heads > 65536 || !kv_head_dim_ok(head_dim)) return FP4Q_ERR_SHAPE;
  if (tokens == 0 || heads == 0) return FP4Q_OK;
  if (!kv_size_ok(tokens, heads, head_dim)) return FP4Q_ERR_SHAPE;
  // the last element, below 2^60: no byte offset passes 63 bits
  if (token_stride < 0 || head_stride < 0 ||
      (__int128)token_stride * (tokens - 1) + (__int128)head_stride * (heads - 1) >= ((__int128)1 << 60) - head_dim)
    return FP4Q_ERR_SHAPE;
  const int64_t chunk = dtype == FP4Q_BF16 ? 8 : 4;  // elements of 16 bytes
  if (!kv_aligned(x, 16) || token_stride % chunk || head_stride % chunk) return FP4Q_ERR_ALIGN;
  return FP4Q_OK;
}

inline fp4q_status_t kv_check_map(const fp4q_head_map_t &m, int64_t head_dim, bool empty) {
  if (m.hadamard_n != 0 && m.hadamard_n != 16 && m.hadamard_n != 32 && m.hadamard_n != 64 && m.hadamard_n != 128)
    return FP4Q_ERR_ARG;
  if (m.hadamard_n > head_dim) return FP4Q_ERR_SHAPE;
  if (m.interleaved != 0 && m.interleaved != 1) return FP4Q_ERR_ARG;
  if (m.norm_weight && !(m.eps >= 0.0 && m.eps <= 1.7e308)) return FP4Q_ERR_ARG;
  if (m.norm_weight && !kv_aligned(m.norm_weight, 16)) return FP4Q_ERR_ALIGN;
  if (m.rotary_dim < 0 || m.rotary_dim > head_dim || m.rotary_dim % 16) return FP4Q_ERR_SHAPE;
  if (m.rotary_dim) {
    if (!m.table || (!m.positions && !empty)) return FP4Q_ERR_NULL;
    if (m.table_positions < 1 || m.table_positions > ((int64_t)1 << 40)) return FP4Q_ERR_SHAPE;
    if (!kv_aligned(m.table, 16) || !kv_aligned(m.positions, 8)) return FP4Q_ERR_ALIGN;
  } else if (m.table) {
    return FP4Q_ERR_SHAPE;
  }
  return FP4Q_OK;
}

// Rows of row_bytes bytes at the three strides do not overlap: taken from
// the smallest stride up, each is at least the extent of what it repeats.
inline bool kv_rows_apart(int64_t row_bytes, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2, int64_t s2) {
  int64_t n[3] = {n0, n1, n2}, s[3] = {s0, s1, s2};
  __int128 extent = row_bytes;
  for (int k = 0; k < 3; ++k) {
    int at = -1;
    for (int i = 0; i < 3; ++i)
      if (n[i] > 1 && (at < 0 || s[i] < s[at])) at = i;
    if (at < 0) break;
    if ((__int128)s[at] < extent) return false;
    extent += (__int128)s[at] * (n[at] - 1);
    n[at] = 1;
  }
  return extent < ((__int128)1 << 62);
}

inline fp4q_status_t kv_check_cache(const fp4q_kv_cache_t &c) {
  if (!c.k_codes || !c.k_scales || !c.v_codes || !c.v_scales) return FP4Q_ERR_NULL;
  if (!kv_head_dim_ok(c.head_dim) || c.heads < 1 || (int64_t)c.heads * c.head_dim > 65536) return FP4Q_ERR_SHAPE;
  if (c.page_size < 16 || c.page_size > 1024 || (c.page_size & (c.page_size - 1))) return FP4Q_ERR_SHAPE;
  if (c.pages < 1 || c.pages > 0x7FFFFFFF) return FP4Q_ERR_SHAPE;
  if (c.pages * c.page_size >= ((int64_t)1 << 40) / c.heads) return FP4Q_ERR_SHAPE;
  if (c.page_stride < 0 || c.head_stride < 0 || c.token_stride < 0 || c.token_stride > ((int64_t)1 << 26))
    return FP4Q_ERR_SHAPE;
  if (!kv_rows_apart(c.head_dim / 2, c.pages, c.page_stride, c.heads, c.head_stride, c.page_size, c.token_stride))
    return FP4Q_ERR_SHAPE;
  if (!kv_aligned(c.k_codes, 16) || !kv_aligned(c.v_codes, 16) || c.page_stride % 16 || c.head_stride % 16 ||
      c.token_stride % 16)
    return FP4Q_ERR_ALIGN;
  return FP4Q_OK;
}

// Division of numbers below 2^31 by a fixed d (1 .. 65536): with l the least
// power of two 2^l >= d and m = ceil(2^(31 + l) / d), m d exceeds 2^(31 + l)
// by less than d <= 2^l, so n m / 2^(31 + l) exceeds n / d by less than
// 1 / d and has the same whole part.
struct Divider {
  uint32_t d, m, shift;
};
inline Divider make_divider(uint32_t d) {
  uint32_t l = 0;
  while ((1u << l) < d) ++l;
  return Divider{d, (uint32_t)((((uint64_t)1 << (31 + l)) + d - 1) / d), 31 + l};
}
FP4Q_HD uint32_t divide(uint32_t n, const Divider &v) { return (uint32_t)(((uint64_t)n * v.m) >> v.shift); }

// ------------------------------------------------- attention's work list ----

struct AttnShape {
  int64_t tokens;       // rows of q
  int batch, groups;    // sequences; query heads per cache head
  int heads;            // cache heads
  int max_new, max_len; // host bounds on a sequence's new tokens and length
  int causal, window;
  int min_rows = 0, max_rows = INT32_MAX;  // (token, head of the group) rows of the sequences that are served
};

// One sequence as the kernels see it: its values cut to what the call's
// bounds allow, so that nothing derived from it leaves the given tensors.
struct AttnSeq {
  int64_t first;  // its first row of q
  int fresh;      // its rows of q
  int len;        // cached tokens
  bool bad;       // a value had to be cut
};

FP4Q_HD AttnSeq attn_seq(const AttnShape &a, int len, int64_t begin, int64_t end) {
  AttnSeq s;
  s.bad = false;
  if (len < 0 || len > a.max_len) {
    s.bad = true;
    len = len < 0 ? 0 : a.max_len;
  }
  if (begin < 0 || begin > a.tokens || end < begin || end > a.tokens || end - begin > a.max_new) {
    s.bad = true;
    begin = begin < 0 ? 0 : (begin > a.tokens ? a.tokens : begin);
    end = end > a.tokens ? a.tokens : end;
    end = end < begin ? begin : (end - begin > a.max_new ? begin + a.max_new : end);
  }
  s.first = begin;
  s.fresh = (int)(end - begin);
  s.len = len;
  return s;
}

// Keys [lo, hi) that row token i of a sequence sees (empty where hi <= lo).
FP4Q_HD int attn_hi(const AttnShape &a, const AttnSeq &s, int i) {
  const int64_t p = (int64_t)s.len - s.fresh + i + 1;
  return a.causal && p < s.len ? (p < 0 ? 0 : (int)p) : s.len;
}
FP4Q_HD int attn_lo(const AttnShape &a, const AttnSeq &s, int i) {
  if (!a.window) return 0;
  const int64_t p = (int64_t)s.len - s.fresh + i + 1 - a.window;
  return p < 0 ? 0 : (p > s.len ? s.len : (int)p);
}

// Row tiles of a sequence (rows_per_tile of its fresh * groups rows each; none
// where another pass serves it) and the key tiles of tile_len tokens that any
// of its rows can see: key tiles lo .. lo + n - 1, at least one, so that every
// row tile is somebody's work.
struct AttnWork {
  int64_t row_tiles;
  int lo, n;
};
FP4Q_HD AttnWork attn_work(const AttnShape &a, const AttnSeq &s, int rows_per_tile, int tile_len) {
  AttnWork w;
  const int rows = s.fresh * a.groups;  // below 2^27
  w.row_tiles = rows < a.min_rows || rows > a.max_rows ? 0 : (rows + rows_per_tile - 1) / rows_per_tile;
  w.lo = attn_lo(a, s, 0) / tile_len;
  const int hi = s.fresh ? attn_hi(a, s, s.fresh - 1) : 0;
  w.n = (int)(((int64_t)hi + tile_len - 1) / tile_len) - w.lo;
  if (w.n < 1) w.n = 1;
  return w;
}

// A unit of n key tiles takes n + kUnitCost of the work: besides its tiles it
// costs a chain of dependent loads and a merge, about as long as that many
// tiles take a workgroup.  Measured on 64 sequences of 0 to 8192 tokens (64
// heads on 8, 128 wide): none 93 us, 5 72, 8 66, 12 64, 16 64.  Its first kUnitCost positions stand for them, so
// the part of the unit within positions [from, to) is the tiles t0 .. t1 - 1.
constexpr int kUnitCost = 12;
struct AttnPart {
  int t0, t1;
};
FP4Q_HD AttnPart attn_part(int64_t from, int64_t to, int n) {
  AttnPart p;
  from -= kUnitCost;
  to -= kUnitCost;
  p.t0 = from < 0 ? 0 : (from < n ? (int)from : n);
  p.t1 = to < 0 ? 0 : (to < n ? (int)to : n);
  return p;
}

// Quotient of non-negative numbers, by the shorter division where both fit.
FP4Q_HD int64_t attn_div(int64_t a, int64_t b) {
  if ((((uint64_t)a | (uint64_t)b) >> 32) == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
  return a / b;
}
// Work of all sequences laid end to end is cut into `spans` equal spans; span i is [attn_cut(i), attn_cut(i + 1)).
FP4Q_HD int64_t attn_cut(int64_t total, int64_t spans, int64_t i) {
  const int64_t q = attn_div(total, spans), r = total - q * spans;
  return q * i + (i < r ? i : r);
}
// The spans that `total` positions of work are worth: none has fewer than a
// unit's cost and four key tiles, one for each wave.
FP4Q_HD int attn_spans(int64_t total, int spans) {
  const int64_t most = attn_div(total, kUnitCost + 4);
  return most < 1 ? 1 : (most < spans ? (int)most : spans);
}
// The span that position pos (0 .. total - 1) lies in.
FP4Q_HD int64_t attn_span_of(int64_t total, int64_t spans, int64_t pos) {
  const int64_t q = attn_div(total, spans), r = total - q * spans;
  const int64_t wide = r * (q + 1);
  return pos < wide ? attn_div(pos, q + 1) : r + attn_div(pos - wide, q);
}

// --------------------------------------------------- attention's kernels ----

constexpr int kCus = 256;
constexpr int64_t kMaxGroups = 1 << 22;  // with 512 threads each, half of what a launch may have

constexpr int kFewRows = 96;  // of a sequence and cache head, up to which tiles of 16 serve it

// One kernel's part of a call: the sequences that have min_rows to max_rows rows (of one head).
struct Pass {
  int rows;       // of a row tile: 16 (attn_rows_kernel), 128 or 256 (attn_prompt_kernel)
  int waves;      // of attn_rows_kernel
  int64_t units;  // upper bound of (sequence, row tile, head) units
  int spans;
  int64_t part_floats;
  int min_rows, max_rows;
};
struct Plan {
  int passes;  // 1 or 2, one after the other in the same workspace
  Pass pass[2];
};

inline Pass make_pass(int rows, int64_t units, int64_t keys, int64_t head_dim, int min_rows, int max_rows) {
  const int64_t fit = kCus * (head_dim == 256 || rows == 256 ? 1 : 2);  // workgroups on the chip at once
  // Not split: one workgroup a unit, no second kernel (5 us).  For short units, and for middling ones where there
  // are enough to fill the chip: 64 sequences of up to 2000 keys (512 units of up to 63 tiles) 25.0 us, split 27.3.
  // Short is up to 1024 keys of 16 rows and 2048 of more.  Whole and split: 512 keys 9.3 us and 12.2; 1000 keys 12.9
  // and 12.4, of 16 sequences 13.4 and 15.9, heads of 256 (16 on 2) 19.3 and 17.1; 2000 keys 19.8 and 12.9; a prompt
  // of 2000 tokens 61 and 91, two chunks of 600 on 1500 keys 49 and 76.
  const int64_t tiles = keys / (rows == 16 ? 32 : 64) + 2;
  // More units than a launch may have workgroups are taken in spans too.  Tiles of 256 rows never are: there are 512
  // units at least, and with 512 rows a sequence on average and fewer than 2^27 rows in all fewer than 2^20.
  // No units (max_new 0): nothing to split, and a second kernel without rows would be no launch at all.
  const bool direct =
      units <= kMaxGroups && (tiles <= 34 || units == 0 || (units >= fit && (rows != 16 || tiles <= 66)));
  Pass p;
  p.rows = rows;
  p.units = units;
  p.spans = direct ? 0 : (int)fit - 1;  // one workgroup serves the status
  // Waves that share a unit of attn_rows_kernel: four, and one for many short units, each of which costs its waves
  // about six key tiles' time whatever their number.  256 sequences of up to 100 keys (2048 units) 12 us with one, 26
  // with four; 200 of up to 500, 25 and 32; 128 of up to 1000, 34 and 29.
  p.waves = direct && units > 512 && tiles <= 18 ? 1 : 4;
  p.part_floats = direct ? 0 : 2 * (int64_t)p.spans * rows * (head_dim + 2);
  p.min_rows = min_rows;
  p.max_rows = max_rows;
  return p;
}

inline Plan make_plan(int64_t tokens, int64_t batch, int64_t q_heads, int64_t heads, int64_t head_dim, int64_t max_new,
                      int64_t max_len, int64_t window) {
  const int64_t groups = q_heads / heads, seq_rows = max_new * groups, all_rows = tokens * groups;
  const int64_t live = batch < tokens ? batch : tokens;  // sequences that have rows, at most
  const int64_t keys = window && window + max_new < max_len ? window + max_new : max_len;  // of a row tile, at most
  // units of so many sequences of so many rows, at most: a sequence's rows fill its row tiles except the last one
  auto units_of = [&](int64_t rows, int64_t seqs, int64_t most_rows) {
    const int64_t tiles = all_rows / rows + seqs, most = seqs * ((most_rows + rows - 1) / rows);
    return (tiles < most ? tiles : most) * heads;
  };
  // The average sequence has half of the longest one's rows or more: one kernel for all.  Else there can be a few long
  // ones among short or empty ones (a chunk of a prompt beside decoding tokens, a padded batch, no bound on the new
  // tokens), and a row tile costs the same however few of its rows are live: each kernel serves its own.
  // Measured, us (32 heads on 8, 128 wide): two passes, one of tiles of 128, one of 16: 63 tokens and a chunk of 512 on
  // 8192 keys 232, 409, 289; 60 and four of 512 on 4096 228, 296, 426; 31 and 2048 on 4096 160, 201, 405; 127 and 128
  // on 2048 113, 174, 74; 512 alone in a batch of 64 on 8192 116, 190, 169; 64 tokens without a bound (64 heads) 78,
  // 234, 71.  Units that run at once, most of them full, need no second pass: three tokens and 1000 on 2048 keys 70
  // and 57.
  const bool even =
      2 * all_rows >= seq_rows * live ||
      (all_rows >= 128 * live && units_of(128, live, seq_rows) <= kCus * (head_dim == 256 ? 1 : 2));
  int64_t long_ones = all_rows / (kFewRows + 1);
  if (even || live < long_ones) long_ones = live;
  // A row tile of 128 costs a fifth of eight of 16 for each key, but it has to be filled, and there have to be
  // enough of them for half the CUs, or keys enough to be split.  Measured (32 heads on 8, 128 wide; one sequence
  // unless said): 80 rows a head on 8192 keys, two sequences: 37 us with 16, 52 with 128; 512 rows on 16384 keys
  // 103 and 85; 2048 rows on 512 keys 34 (with 32) and 25; five sequences of up to 951 rows behind a window of 1000
  // (12 heads on 4 of 64) 20 and 37.
  Plan p;
  p.passes = 1;
  if (seq_rows <= kFewRows || (units_of(128, long_ones, seq_rows) < kCus / 2 && keys <= 4096)) {
    p.pass[0] = make_pass(16, units_of(16, live, seq_rows), keys, head_dim, 0, INT32_MAX);
    return p;
  }
  // 256 rows share the staging of a key tile among twice the waves where there are still two workgroups for each CU:
  // 16384 rows a head on 8192 keys 505 us with 128, 470 with 256; 8192 rows on 2048 keys 65 and 71; 64 sequences of
  // 512 rows on 2048 keys 320 and 297.  Sequences with fewer rows leave much of them empty: 64 of 128 rows on 4096
  // keys 177 and 274.
  const int64_t most = units_of(256, long_ones, seq_rows);
  const int rows = head_dim != 256 && all_rows >= 512 * long_ones && most >= 2 * kCus ? 256 : 128;
  p.pass[0] = make_pass(rows, units_of(rows, long_ones, seq_rows), keys, head_dim, even ? 0 : kFewRows + 1, INT32_MAX);
  if (!even) {
    p.passes = 2;
    p.pass[1] = make_pass(16, units_of(16, live, kFewRows), keys, head_dim, 0, kFewRows);
  }
  return p;
}

}  // namespace fp4q
