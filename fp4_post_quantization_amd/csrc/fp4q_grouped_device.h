// What the grouped kernels share: which group a row tile belongs to, found by
// every wave from the groups' offsets, 64 groups at a time, their tiles summed
// by DPP.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp4q_device.h"
#include "fp4q_grouped.h"
#include "fp4q_grouped_host.h"

namespace fp4q {

struct Groups {
  const int32_t *offsets, *rows;
  int groups, entries;
};
inline Groups groups_of(const fp4q_row_groups_t &g) { return Groups{g.offsets, g.rows, (int)g.groups, (int)g.entries}; }

template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_add_step(int v) {
  return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, true);
}
// Sum of v over the lanes up to the caller's, its own included.
__device__ __forceinline__ int wave_scan(int v) {
  v = dpp_add_step<0x111, 0xF>(v);  // row_shr:1, 2, 4, 8
  v = dpp_add_step<0x112, 0xF>(v);
  v = dpp_add_step<0x114, 0xF>(v);
  v = dpp_add_step<0x118, 0xF>(v);
  v = dpp_add_step<0x142, 0xA>(v);  // row_bcast:15 into rows 1 and 3
  v = dpp_add_step<0x143, 0xC>(v);  // row_bcast:31 into rows 2 and 3
  return v;
}

// The group that row tile number `tile` (of `rows` rows, group after group) belongs to: its positions [lo, hi) in the
// groups' order, and the number of its first tile.  Past the last one group is -1 and first the number of all tiles.
struct TileGroup {
  int group, lo, hi, first;
};
__device__ __forceinline__ TileGroup find_group(const Groups &a, int rows, int tile) {
  const int lane = threadIdx.x & 63;
  int run = 0;
  for (int g0 = 0; g0 < a.groups; g0 += 64) {
    const int g = g0 + lane;
    const bool in = g < a.groups;
    const GroupSpan s = group_span(in ? a.offsets[g] : 0, in ? a.offsets[g + 1] : 0, a.entries);
    const int mine = in ? span_tiles(s.lo, s.hi, rows) : 0;
    const int upto = wave_scan(mine);
    const int all = __builtin_amdgcn_readlane(upto, 63);
    if (tile < run + all) {
      const int at = __ffsll((unsigned long long)__ballot(run + upto > tile)) - 1;
      return TileGroup{g0 + at, __builtin_amdgcn_readlane(s.lo, at), __builtin_amdgcn_readlane(s.hi, at),
                       run + __builtin_amdgcn_readlane(upto - mine, at)};
    }
    run += all;
  }
  return TileGroup{-1, 0, 0, run};
}

// The tile itself: positions [lo, hi).  Past the last one: group -1, and its number among those that follow in lo.
struct RowTile {
  int group, lo, hi;
};
__device__ __forceinline__ RowTile find_tile(const Groups &a, int rows, int tile) {
  const TileGroup g = find_group(a, rows, tile);
  if (g.group < 0) return RowTile{-1, tile - g.first, 0};
  const int lo = g.lo + (tile - g.first) * rows;
  return RowTile{g.group, lo, g.hi - lo > rows ? lo + rows : g.hi};
}

// Whether the groups' offsets are not what they should be (one wave).
__device__ __forceinline__ bool offsets_bad(const Groups &a) {
  bool bad = a.offsets[0] != 0;
  for (int g = threadIdx.x & 63; g < a.groups; g += 64)
    bad |= group_span(a.offsets[g], a.offsets[g + 1], a.entries).bad;
  return __ballot(bad) != 0;
}

// Entry at position p, -1 for a number that is none.
__device__ __forceinline__ int entry_at(const Groups &a, int p) {
  const int e = a.rows[p];
  return (uint32_t)e < (uint32_t)a.entries ? e : -1;
}

}  // namespace fp4q
