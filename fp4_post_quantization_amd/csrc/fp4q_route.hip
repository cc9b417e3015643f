// Routing of tokens to experts, entries sorted by group, and the weighted sum
// of the experts' results (include/fp4q_grouped.h).
//
// Routing: a wave takes a token, lane l its experts l J .. l J + J - 1.  The
// best of what is left is found top_k times by a wave maximum over 32-bit keys
// that order as the values do (one DPP instruction a step): exact for logits,
// and for float64 scores with a bias their float32 roundings, whose rare ties
// are settled in float64.  (With the lane's experts sorted first: 1 us less for
// 256 of them, 12 more for 1024.)  8192 tokens of 256 experts in 8 groups,
// sigmoid and bias: 32 us, of which 15 are there for 32 tokens too (two
// launches, a token's chain of dependent steps); the rest is the issue of some
// 1000 vector instructions a token, a third of them the float64 exponentials.
// By softmax without a bias and without groups 21.
//
// Sorting is a counting sort in two launches: every workgroup counts its
// entries by group; then every placing workgroup sums the counts before its
// own and those of all (they come from the cache), and places its entries,
// 1024 at a time, one a thread: its rank among the equal ones of the wave from
// ballots over the bits of the group number, plus the equal ones of the waves
// before.  No atomic decides an order.  A call of few tokens is one workgroup's.
// Placing takes 6 us for 4084 entries and 10 for 65536, most of it in rounds of
// loads of the counts; nothing near a rate of the card bounds it.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "fp4q.h"
#include "fp4q_device.h"
#include "fp4q_grouped.h"
#include "fp4q_grouped_device.h"
#include "fp4q_grouped_host.h"

namespace fp4q {
namespace {

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;

// ----------------------------------------------------------------- sorting ----
struct SortArgs {
  const int32_t *ids;
  int64_t entries;
  int groups;
  const uint16_t *counts;  // [blocks][sort_stride(groups)]
  int blocks, join;
  int64_t per;             // entries of a counting block
  int32_t *offsets, *rows;
};

// LDS of a placing workgroup: two bases and a 16-bit count for each wave, of every column.
size_t sort_lds(int64_t groups, int waves) { return (size_t)(sort_stride((int)groups) * (8 + 2 * waves)); }

__device__ __forceinline__ int group_of(int32_t id, int groups) {
  return (uint32_t)id < (uint32_t)groups ? id : groups;
}

// Places the entries [begin, end).  SOLO: they are all there are, and are counted here.
template <bool SOLO, int WAVES>
__device__ void place_entries(const SortArgs &a, int64_t begin, int64_t end, int first_block, uint8_t *lds) {
  constexpr int THREADS = 64 * WAVES;
  const int cols = a.groups + 1, stride = sort_stride(a.groups), tid = threadIdx.x, lane = tid & 63;
  const int wave = wave_index();
  int *base0 = reinterpret_cast<int *>(lds), *base1 = base0 + stride;
  uint16_t *cnt = reinterpret_cast<uint16_t *>(base1 + stride);  // [wave][stride]
  // base0: entries of the group in the blocks before; base1: in all
  for (int e = tid; e < stride; e += THREADS) base0[e] = base1[e] = 0;
  __syncthreads();
  if constexpr (SOLO) {
    for (int64_t i = begin + tid; i < end; i += THREADS) atomicAdd(&base1[group_of(a.ids[i], a.groups)], 1);
  } else {  // eight columns a thread, as many blocks side by side as there are threads for, four of them in flight
    const int eights = stride / 8, side = THREADS / eights > 0 ? THREADS / eights : 1;
    for (int q = tid; q < side * eights; q += THREADS) {
      const int c = q % eights;
      int before[8] = {}, all[8] = {};
      for (int b0 = q / eights; b0 < a.blocks; b0 += 4 * side) {
        u32x4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int b = b0 + i * side < a.blocks ? b0 + i * side : b0;
          v[i] = *reinterpret_cast<const u32x4 *>(a.counts + (int64_t)b * stride + 8 * c);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int b = b0 + i * side;
          const int in = b < a.blocks, early = b < first_block;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int n = (int)(v[i][j / 2] >> (16 * (j % 2)) & 0xFFFFu);
            all[j] += in ? n : 0;
            before[j] += early ? n : 0;
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        atomicAdd(&base0[8 * c + j], before[j]);
        atomicAdd(&base1[8 * c + j], all[j]);
      }
    }
  }
  __syncthreads();
  if (wave == 0) {  // exclusive sum of the totals over the groups
    int run = 0;
    for (int e0 = 0; e0 < cols; e0 += 64) {
      const int e = e0 + lane;
      const int mine = e < cols ? base1[e] : 0;
      const int v = wave_scan(mine);
      if (e < cols) {
        const int at = run + v - mine;
        base0[e] += at;
        if (first_block == 0) a.offsets[e] = at;
      }
      run += __builtin_amdgcn_readlane(v, 63);
    }
  }
  const int bits = 32 - __clz(a.groups);
  int *from = base0, *to = base1;
  for (int64_t i0 = begin; i0 < end; i0 += THREADS) {
    for (int q = tid; q < WAVES * stride / 8; q += THREADS) reinterpret_cast<u32x4 *>(cnt)[q] = u32x4{0, 0, 0, 0};
    __syncthreads();
    const int64_t i = i0 + tid;
    const bool in = i < end;
    const int g = in ? group_of(a.ids[i], a.groups) : 0;
    uint64_t same = __ballot(in);
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot((g >> b) & 1);
      same &= (g >> b) & 1 ? set : ~set;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    if (in && rank == 0) cnt[wave * stride + g] = (uint16_t)__popcll(same);
    __syncthreads();
    for (int e = tid; e < cols; e += THREADS) {
      int run = 0;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        const int v = cnt[w * stride + e];
        cnt[w * stride + e] = (uint16_t)run;
        run += v;
      }
      to[e] = from[e] + run;
    }
    __syncthreads();
    if (in) {
      const int64_t at = (int64_t)from[g] + cnt[wave * stride + g] + rank;
      if (at >= 0 && at < a.entries) a.rows[at] = (int32_t)i;
    }
    __syncthreads();
    int *t = from;
    from = to;
    to = t;
  }
}

__global__ __launch_bounds__(kSortThreads) void place_kernel(SortArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int first = (int)blockIdx.x * a.join;
  const int64_t begin = first * a.per, want = begin + a.join * a.per;
  place_entries<false, kSortWaves>(a, begin, want < a.entries ? want : a.entries, first, lds);
}

// Counts of the ids of a block; reports those past the last group.
__global__ __launch_bounds__(kSortThreads) void count_kernel(SortArgs a, uint16_t *counts, uint32_t *status) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  int *sum = reinterpret_cast<int *>(lds);
  const int cols = a.groups + 1;
  for (int e = threadIdx.x; e < cols; e += kSortThreads) sum[e] = 0;
  __syncthreads();
  const int64_t begin = blockIdx.x * a.per, want = begin + a.per, end = want < a.entries ? want : a.entries;
  uint32_t err = 0;
  for (int64_t i = begin + threadIdx.x; i < end; i += kSortThreads) {
    const int32_t id = a.ids[i];
    if (id >= a.groups) err = FP4Q_DATA_BAD_GROUP;
    atomicAdd(&sum[group_of(id, a.groups)], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < sort_stride(a.groups); e += kSortThreads)
    counts[(int64_t)blockIdx.x * sort_stride(a.groups) + e] = e < cols ? (uint16_t)sum[e] : 0;
  Status{status, true}.finish(err);
}

__global__ __launch_bounds__(kSortThreads) void group_solo_kernel(SortArgs a, uint32_t *status) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  uint32_t err = 0;
  for (int64_t i = threadIdx.x; i < a.entries; i += kSortThreads)
    if (a.ids[i] >= a.groups) err = FP4Q_DATA_BAD_GROUP;
  if (err || threadIdx.x == kSortThreads - 1) Status{status, true}.merge(err);
  place_entries<true, kSortWaves>(a, 0, a.entries, 0, lds);
}

// ----------------------------------------------------------------- routing ----
struct RouteArgs {
  const void *logits;
  int64_t ld, tokens, per;  // per: tokens of a workgroup
  int experts, k, score, n_groups, run, top_groups, group_best, renormalize;  // run: experts of a group
  const float *bias;
  float scale;
  float *weights;
  int32_t *chosen;
  uint16_t *counts;
  uint32_t *status;
};

__device__ __forceinline__ float widen1(uint16_t v) { return as_f((uint32_t)v << 16); }
__device__ __forceinline__ float widen1(float v) { return v; }

// Orders as the float32 values do (both zeros alike); above 0 for finite ones.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = as_u(v + 0.0f);
  return (b >> 31) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t key) { return as_f((key >> 31) ? key & 0x7FFFFFFFu : ~key); }

// The value of a lane that is the same in all lanes' view (a scalar).
__device__ __forceinline__ double lane_value(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ float lane_value(float v, int lane) {
  return as_f((uint32_t)__builtin_amdgcn_readlane((int)as_u(v), lane));
}

// Sum over the wave, in every lane: rows of 16 by shifts, then across rows (lanes shifted in from outside read 0).
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_sum_step(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xF, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xF, true);
  return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_sum(double v) {
  v = dpp_sum_step<0x111, 0xF>(v);
  v = dpp_sum_step<0x112, 0xF>(v);
  v = dpp_sum_step<0x114, 0xF>(v);
  v = dpp_sum_step<0x118, 0xF>(v);
  v = dpp_sum_step<0x142, 0xA>(v);
  v = dpp_sum_step<0x143, 0xC>(v);
  return lane_value(v, 63);
}

__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Which of the groups of experts are kept: bit g * (64 >> log) of the result, log = log2 of the groups, rounded up.
// pick: the wave's values in LDS.
template <typename V>
__device__ uint64_t kept_groups(const RouteArgs &a, const V *pick, int log, int lane) {
  const int lanes = 64 >> log, g = lane >> (6 - log), part = lane & (lanes - 1);
  const V none = (V)-__builtin_inff();
  V b1 = none, b2 = none;
  if (g < a.n_groups)
    for (int i = part; i < a.run; i += lanes) {
      const V v = pick[g * a.run + i];
      b2 = v > b1 ? b1 : (v > b2 ? v : b2);
      b1 = v > b1 ? v : b1;
    }
  for (int d = 1; d < lanes; d <<= 1) {
    const V o1 = __shfl_xor(b1, d), o2 = __shfl_xor(b2, d);
    const V low = b1 < o1 ? b1 : o1, next = b2 > o2 ? b2 : o2;
    b1 = b1 < o1 ? o1 : b1;
    b2 = low > next ? low : next;
  }
  const V mine = a.group_best == 2 && b2 > none ? b1 + b2 : b1;
  int rank = 0;
  for (int h = 0; h < a.n_groups; ++h) {
    const V v = lane_value(mine, h * lanes);
    rank += v > mine || (v == mine && h < g);
  }
  return __ballot(part == 0 && g < a.n_groups && rank < a.top_groups);
}

// A lane's experts, what does not change from token to token.
template <int J>
struct LaneExperts {
  float bias[J];
  int bit[J];  // of the expert's group in kept_groups' result
  bool there[J];
  int log;     // log2 of the groups, rounded up
};

// Routes token t by the wave.  SCORED: scores matter for the choice (with a bias, or for the sum of a group's two
// best); else the logits order the experts.
template <int J, typename T, bool SCORED>
__device__ __forceinline__ void route_token(const RouteArgs &a, int64_t t, const float x[J], const LaneExperts<J> &my,
                                            int lane, void *lds, int *sum, uint32_t &err) {
  using V = std::conditional_t<SCORED, double, float>;
  const float minus_inf = -__builtin_inff();
  const int e0 = lane * J;
  const bool biased = SCORED && a.bias;  // choices compare scores, not logits
  bool bad = false;
  uint32_t key[J], top = 0;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    bad |= !(x[j] < __builtin_inff());
    key[j] = x[j] > minus_inf ? order_key(x[j]) : 0u;
    top = key[j] > top ? key[j] : top;
  }
  top = wave_max_u32(top);
  const float most = order_value(top);
  double total = 0.0;
  V pick[J];
  if constexpr (!SCORED) {
#pragma unroll
    for (int j = 0; j < J; ++j) pick[j] = x[j];
    if (a.score == FP4Q_SOFTMAX && !a.renormalize) {
#pragma unroll
      for (int j = 0; j < J; ++j) total += exp(key[j] ? (double)x[j] - (double)most : (double)minus_inf);
      total = wave_sum(total);
    }
  } else {
    if (a.score == FP4Q_SOFTMAX) {
#pragma unroll
      for (int j = 0; j < J; ++j) {  // an expert that is off has exp(-inf), without a branch around it
        pick[j] = exp(key[j] ? (double)x[j] - (double)most : (double)minus_inf);
        total += pick[j];
      }
      total = wave_sum(total);
      const double one = total > 0.0 ? 1.0 / total : 0.0;
#pragma unroll
      for (int j = 0; j < J; ++j) pick[j] *= one;
    } else {
#pragma unroll
      for (int j = 0; j < J; ++j) pick[j] = 1.0 / (1.0 + exp(-(double)x[j]));
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      pick[j] += (V)my.bias[j];
      const bool on = key[j] != 0u;
      bad |= on & !(pick[j] < (V)__builtin_inff());
      const bool off = !on | !(pick[j] > (V)minus_inf);
      pick[j] = off ? (V)minus_inf : pick[j];
      const uint32_t rounded = order_key((float)pick[j]);
      key[j] = biased ? rounded : key[j];
      key[j] = off ? 0u : key[j];
    }
  }
  const bool dropped = __ballot(bad) != 0;
  if (dropped) err = FP4Q_DATA_NONFINITE_INPUT;
  if (a.n_groups > 1) {
    V *room = reinterpret_cast<V *>(lds);
    wave_fence();
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (my.there[j]) room[e0 + j] = pick[j];
    wave_fence();
    const uint64_t kept = kept_groups<V>(a, room, my.log, lane);
#pragma unroll
    for (int j = 0; j < J; ++j) key[j] = (kept >> my.bit[j]) & 1 ? key[j] : 0u;
  }
  int mine = -1;        // lane i: the token's i-th choice
  uint32_t my_key = 0;  // and its key
  for (int i = 0; i < a.k && !dropped; ++i) {
    uint32_t best = key[0];
    int at = 0;
#pragma unroll
    for (int j = 1; j < J; ++j)
      if (key[j] > best) {
        best = key[j];
        at = j;
      }
    const uint32_t m = wave_max_u32(best);
    if (m == 0) break;
    const uint64_t ties = __ballot(best == m);
    int from = __ffsll((unsigned long long)ties) - 1;
    if constexpr (SCORED) {
      if (biased) {
        bool twice = false;
#pragma unroll
        for (int j = 0; j < J; ++j) twice |= key[j] == m && at != j;
        // float32 rounds some alike: float64 decides, then the lowest index
        if ((ties & (ties - 1)) || __ballot(twice)) {
          double high = (double)minus_inf;
#pragma unroll
          for (int j = 0; j < J; ++j)
            if (key[j] == m && pick[j] > high) {
              high = pick[j];
              at = j;
            }
          double highest = (double)minus_inf;
          for (uint64_t rest = ties; rest; rest &= rest - 1) {
            const int l = __ffsll((unsigned long long)rest) - 1;
            const double v = lane_value(high, l);
            if (v > highest) {
              highest = v;
              from = l;
            }
          }
        }
      }
    }
    const int e = __builtin_amdgcn_readlane(e0 + at, from);
    mine = lane == i ? e : mine;
    my_key = lane == i ? m : my_key;
#pragma unroll
    for (int j = 0; j < J; ++j) key[j] = lane == from && at == j ? 0u : key[j];
  }
  double w = 0.0;
  if (mine >= 0) {
    const double v = biased ? (double)widen1(((const T *)a.logits)[t * a.ld + mine]) : (double)order_value(my_key);
    if (a.score == FP4Q_SIGMOID) w = 1.0 / (1.0 + exp(-v));
    else w = exp(v - (double)most) / (a.renormalize ? 1.0 : total);
  }
  if (a.renormalize) {
    const double all = wave_sum(w);
    w = all > 0.0 ? w / all : 0.0;
  }
  if (lane < a.k) {
    a.weights[t * a.k + lane] = (float)(w * (double)a.scale);
    a.chosen[t * a.k + lane] = mine;
    if (sum) atomicAdd(&sum[mine < 0 ? a.experts : mine], 1);
  }
}

// Routes the tokens [begin, end), one a wave at a time.
template <int J, typename T, bool SCORED, int WAVES>
__device__ void route_tokens(const RouteArgs &a, int64_t begin, int64_t end, int *sum, uint8_t *lds_pick,
                             uint32_t &err) {
  const int lane = threadIdx.x & 63, wave = wave_index();
  const T *logits = (const T *)a.logits;
  const int e0 = lane * J;
  void *room = lds_pick + (size_t)wave * a.experts * (SCORED ? 8 : 4);
  LaneExperts<J> my;
  my.log = 32 - __clz(a.n_groups - 1);
#pragma unroll
  for (int j = 0; j < J; ++j) {
    my.there[j] = e0 + j < a.experts;
    my.bias[j] = SCORED && a.bias && my.there[j] ? a.bias[e0 + j] : 0.0f;
    my.bit[j] = a.n_groups > 1 && my.there[j] ? (e0 + j) / a.run << (6 - my.log) : 0;
  }
  for (int64_t t = begin + wave; t < end; t += WAVES) {
    float x[J];
#pragma unroll
    for (int j = 0; j < J; ++j) x[j] = my.there[j] ? widen1(logits[t * a.ld + e0 + j]) : -__builtin_inff();
    route_token<J, T, SCORED>(a, t, x, my, lane, room, sum, err);
  }
}

constexpr int kRouteWaves = 8;

template <int J, typename T, bool SCORED>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(RouteArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  int *sum = reinterpret_cast<int *>(lds);
  const int cols = a.experts + 1;
  for (int e = threadIdx.x; e < cols; e += 64 * kRouteWaves) sum[e] = 0;
  __syncthreads();
  uint32_t err = 0;
  const int64_t begin = blockIdx.x * a.per, want = begin + a.per;
  route_tokens<J, T, SCORED, kRouteWaves>(a, begin, want < a.tokens ? want : a.tokens, sum, lds + (cols + 3) / 4 * 16,
                                          err);
  __syncthreads();
  if (a.counts)
    for (int e = threadIdx.x; e < sort_stride(a.experts); e += 64 * kRouteWaves)
      a.counts[(int64_t)blockIdx.x * sort_stride(a.experts) + e] = e < cols ? (uint16_t)sum[e] : 0;
  Status{a.status, true}.finish(err);
}

// One workgroup for all tokens, and their entries sorted behind.
template <int J, typename T, bool SCORED>
__global__ __launch_bounds__(64 * kRouteWaves) void route_solo_kernel(RouteArgs a, SortArgs s) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  uint32_t err = 0;
  // by the last wave, which has the fewest tokens: at the kernel's end these two trips to memory would be waited for
  if (threadIdx.x == 64 * kRouteWaves - 1) Status{a.status, true}.merge(0u);
  route_tokens<J, T, SCORED, kRouteWaves>(a, 0, a.tokens, nullptr, lds, err);
  if (err) Status{a.status, true}.merge(err);
  if (!s.offsets) return;
  __syncthreads();
  place_entries<true, kRouteWaves>(s, 0, s.entries, 0, lds);
}

// ------------------------------------------------------------- weighted sum ----
struct CombineArgs {
  const void *y, *add;
  void *out;
  int64_t ld_y, ld_add, ld_out;
  const float *weights;
  const int32_t *chosen;
  int k, n, slices;  // slices of a row
};

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
template <int N>
__device__ __forceinline__ void load_row(const uint16_t *p, float z[N]) {
  if constexpr (N == 8) {
    const u32x4 w = *reinterpret_cast<const u32x4 *>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      z[2 * i] = as_f(w[i] << 16);
      z[2 * i + 1] = as_f(w[i] & 0xFFFF0000u);
    }
  } else {
    z[0] = widen1(*p);
  }
}
template <int N>
__device__ __forceinline__ void load_row(const float *p, float z[N]) {
  if constexpr (N == 8) {
    const f32x4 a = reinterpret_cast<const f32x4 *>(p)[0], b = reinterpret_cast<const f32x4 *>(p)[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      z[i] = a[i];
      z[4 + i] = b[i];
    }
  } else {
    z[0] = *p;
  }
}
template <int N>
__device__ __forceinline__ void store_row(uint16_t *p, const float z[N]) {
  if constexpr (N == 8) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)z[2 * i], (__bf16)z[2 * i + 1]});
    *reinterpret_cast<u32x4 *>(p) = w;
  } else {
    *p = __builtin_bit_cast(uint16_t, (__bf16)z[0]);
  }
}
template <int N>
__device__ __forceinline__ void store_row(float *p, const float z[N]) {
  if constexpr (N == 8) {
    reinterpret_cast<f32x4 *>(p)[0] = f32x4{z[0], z[1], z[2], z[3]};
    reinterpret_cast<f32x4 *>(p)[1] = f32x4{z[4], z[5], z[6], z[7]};
  } else {
    *p = z[0];
  }
}

// N elements of a token's row a thread: 8, or 1 where a row or its start is not aligned for 16 bytes.  Bound by HBM:
// 8192 tokens of eight bfloat16 rows of 4096, 605 MB, 114 us (5.3 TB/s; a large copy runs at 5.1).
template <typename T, typename O, int N>
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs a) {
  const int64_t t = blockIdx.x / a.slices;
  const int c = ((int)(blockIdx.x % a.slices) * 256 + (int)threadIdx.x) * N;
  if (c >= a.n) return;
  float acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.0f;
  const T *y = (const T *)a.y + t * a.k * a.ld_y + c;
#pragma unroll 4
  for (int j = 0; j < a.k; ++j) {
    if (a.chosen && a.chosen[t * a.k + j] < 0) continue;
    const float w = a.weights[t * a.k + j];
    float z[N];
    load_row<N>(y + j * a.ld_y, z);
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = __builtin_fmaf(w, z[i], acc[i]);
  }
  if (a.add) {
    float z[N];
    load_row<N>((const O *)a.add + t * a.ld_add + c, z);
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] += z[i];
  }
  store_row<N>((O *)a.out + t * a.ld_out + c, acc);
}

// The only kernel of a call without entries.
__global__ __launch_bounds__(kSortThreads) void no_entries_kernel(int32_t *offsets, int groups, uint32_t *status) {
  if (offsets)
    for (int e = threadIdx.x; e <= groups; e += kSortThreads) offsets[e] = 0;
  if (threadIdx.x == 0) Status{status, true}.merge(0u);
}

template <typename F>
void with_type(fp4q_dtype_t t, F &&f) {
  if (t == FP4Q_BF16) f((uint16_t *)nullptr);
  else f((float *)nullptr);
}
template <typename F>
void with_lanes(int64_t experts, F &&f) {
  if (experts <= 64) f(std::integral_constant<int, 1>{});
  else if (experts <= 128) f(std::integral_constant<int, 2>{});
  else if (experts <= 256) f(std::integral_constant<int, 4>{});
  else if (experts <= 512) f(std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 16>{});
}

fp4q_status_t hip_status() { return hipGetLastError() == hipSuccess ? FP4Q_OK : FP4Q_ERR_HIP; }

bool solo_route(int64_t tokens, int64_t experts, int64_t top_k, bool scored) {
  return tokens <= solo_tokens(experts, scored) && tokens * top_k <= kSortChunk;
}
bool solo_group(int64_t entries) { return entries <= 2 * kSortChunk; }

}  // namespace
}  // namespace fp4q

using namespace fp4q;

extern "C" size_t fp4q_group_rows_workspace_bytes(int64_t entries, int64_t groups) {
  if (entries < 0 || entries > kMaxEntries || groups < 1 || groups > kMaxRowGroups) return 0;
  return entries == 0 || solo_group(entries) ? 256 : sort_bytes(sort_plan(entries, 1, kSortChunk), groups);
}

extern "C" fp4q_status_t fp4q_group_rows(const int32_t *ids, int64_t entries, int64_t groups, int32_t *offsets,
                                         int32_t *rows, void *workspace, size_t workspace_bytes, void *stream) {
  if (entries < 0 || entries > kMaxEntries || groups < 1 || groups > kMaxRowGroups) return FP4Q_ERR_SHAPE;
  if (!offsets || (entries && (!ids || !rows))) return FP4Q_ERR_NULL;
  if (!grouped_ws_ok(workspace, workspace_bytes, fp4q_group_rows_workspace_bytes(entries, groups)))
    return FP4Q_ERR_WORKSPACE;
  if (!kv_aligned(ids, 4) || !kv_aligned(offsets, 4) || !kv_aligned(rows, 4)) return FP4Q_ERR_ALIGN;
  hipStream_t s = (hipStream_t)stream;
  uint32_t *status = (uint32_t *)workspace;
  if (entries == 0) {
    hipLaunchKernelGGL(no_entries_kernel, dim3(1), dim3(kSortThreads), 0, s, offsets, (int)groups, status);
    return hip_status();
  }
  uint16_t *counts = (uint16_t *)((char *)workspace + 256);
  const SortPlan p = sort_plan(entries, 1, kSortChunk);
  const SortArgs a{ids, entries, (int)groups, counts, (int)p.blocks, (int)p.join, p.per, offsets, rows};
  if (solo_group(entries)) {
    hipLaunchKernelGGL(group_solo_kernel, dim3(1), dim3(kSortThreads), sort_lds(groups, kSortWaves), s, a, status);
    return hip_status();
  }
  hipLaunchKernelGGL(count_kernel, dim3((unsigned)p.blocks), dim3(kSortThreads), (size_t)(groups + 1) * 4, s, a, counts,
                     status);
  hipLaunchKernelGGL(place_kernel, dim3((unsigned)p.places), dim3(kSortThreads), sort_lds(groups, kSortWaves), s, a);
  return hip_status();
}

extern "C" size_t fp4q_route_experts_workspace_bytes(int64_t tokens, int64_t experts, int64_t top_k) {
  if (tokens < 0 || experts < 1 || experts > kMaxExperts || top_k < 1 || top_k > kMaxTopK ||
      tokens > kMaxEntries / top_k)
    return 0;
  return tokens == 0 || solo_route(tokens, experts, top_k, true)
             ? 256
             : sort_bytes(sort_plan(tokens, top_k, kRouteWaves), experts);
}

extern "C" fp4q_status_t fp4q_route_experts(const void *logits, fp4q_dtype_t dtype, int64_t tokens, int64_t experts,
                                            int64_t ld, const fp4q_router_t *router, float *weights, int32_t *chosen,
                                            int32_t *offsets, int32_t *rows, void *workspace, size_t workspace_bytes,
                                            void *stream) {
  if (!router) return FP4Q_ERR_NULL;
  if (dtype != FP4Q_F32 && dtype != FP4Q_BF16) return FP4Q_ERR_ARG;
  const fp4q_status_t st = router_check(*router, experts);
  if (st != FP4Q_OK) return st;
  const int64_t k = router->top_k, size = dtype == FP4Q_F32 ? 4 : 2;
  if (tokens < 0 || tokens > kMaxEntries / k || !grouped_rows_ok(tokens, experts, ld, size)) return FP4Q_ERR_SHAPE;
  if (tokens && (!logits || !weights || !chosen)) return FP4Q_ERR_NULL;
  if (!offsets != !rows && tokens) return FP4Q_ERR_NULL;
  if (!grouped_ws_ok(workspace, workspace_bytes, fp4q_route_experts_workspace_bytes(tokens, experts, k)))
    return FP4Q_ERR_WORKSPACE;
  if (!kv_aligned(logits, size) || !kv_aligned(weights, 4) || !kv_aligned(chosen, 4) || !kv_aligned(offsets, 4) ||
      !kv_aligned(rows, 4))
    return FP4Q_ERR_ALIGN;
  hipStream_t s = (hipStream_t)stream;
  uint32_t *status = (uint32_t *)workspace;
  if (tokens == 0) {
    hipLaunchKernelGGL(no_entries_kernel, dim3(1), dim3(kSortThreads), 0, s, offsets, (int)experts, status);
    return hip_status();
  }
  const bool scored = router->bias || (router->n_groups > 1 && router->group_best == 2);
  const bool solo = solo_route(tokens, experts, k, scored);
  const SortPlan p = sort_plan(tokens, k, kRouteWaves);
  uint16_t *counts = solo || !offsets ? nullptr : (uint16_t *)((char *)workspace + 256);
  const RouteArgs a{logits, ld, tokens, p.per, (int)experts, (int)k, (int)router->score, router->n_groups,
                    (int)(experts / router->n_groups), router->top_groups, router->group_best, router->renormalize,
                    router->bias, router->scale, weights, chosen, counts, status};
  const SortArgs e{chosen, tokens * k, (int)experts, counts, (int)p.blocks, (int)p.join, p.per * k, offsets, rows};
  const size_t pick = router->n_groups > 1 ? (size_t)experts * (scored ? 8 : 4) : 0;  // LDS of a wave
  with_lanes(experts, [&](auto jc) {
    constexpr int J = decltype(jc)::value;
    with_type(dtype, [&](auto tp) {
      using T = std::remove_pointer_t<decltype(tp)>;
      auto go = [&](auto sc) {
        constexpr bool SCORED = decltype(sc)::value;
        if (solo) {
          const size_t need = sort_lds(experts, kRouteWaves);
          const size_t lds = pick * kRouteWaves > need ? pick * kRouteWaves : need;
          hipLaunchKernelGGL((route_solo_kernel<J, T, SCORED>), dim3(1), dim3(64 * kRouteWaves), lds, s, a, e);
        } else {
          const size_t lds = (size_t)(experts + 4) / 4 * 16 + pick * kRouteWaves;
          hipLaunchKernelGGL((route_kernel<J, T, SCORED>), dim3((unsigned)p.blocks), dim3(64 * kRouteWaves), lds, s, a);
        }
      };
      if (scored) go(std::true_type{});
      else go(std::false_type{});
    });
  });
  if (counts)
    hipLaunchKernelGGL(place_kernel, dim3((unsigned)p.places), dim3(kSortThreads), sort_lds(experts, kSortWaves), s, e);
  return hip_status();
}

extern "C" fp4q_status_t fp4q_combine_experts(const void *y, fp4q_dtype_t dtype, int64_t tokens, int64_t top_k,
                                              int64_t n, int64_t ld_y, const float *weights, const int32_t *chosen,
                                              const void *add, int64_t ld_add, fp4q_dtype_t out_dtype, void *out,
                                              int64_t ld_out, void *stream) {
  if ((dtype != FP4Q_F32 && dtype != FP4Q_BF16) || (out_dtype != FP4Q_F32 && out_dtype != FP4Q_BF16))
    return FP4Q_ERR_ARG;
  const int64_t size = dtype == FP4Q_F32 ? 4 : 2, out_size = out_dtype == FP4Q_F32 ? 4 : 2;
  if (tokens < 0 || top_k < 1 || top_k > kMaxTopK || tokens > kMaxEntries / top_k || n >= ((int64_t)1 << 31))
    return FP4Q_ERR_SHAPE;
  if (!grouped_rows_ok(tokens * top_k, n, ld_y, size) || !grouped_rows_ok(tokens, n, ld_out, out_size) ||
      (add && !grouped_rows_ok(tokens, n, ld_add, out_size)))
    return FP4Q_ERR_SHAPE;
  if (tokens == 0 || n == 0) return FP4Q_OK;
  if (!y || !weights || !out) return FP4Q_ERR_NULL;
  if (!kv_aligned(y, size) || !kv_aligned(weights, 4) || !kv_aligned(chosen, 4) || !kv_aligned(add, out_size) ||
      !kv_aligned(out, out_size))
    return FP4Q_ERR_ALIGN;
  const bool wide = n % 8 == 0 && kv_aligned(y, 16) && ld_y * size % 16 == 0 && kv_aligned(out, 16) &&
                    ld_out * out_size % 16 == 0 && (!add || (kv_aligned(add, 16) && ld_add * out_size % 16 == 0));
  const int64_t slices = ceil_div(n, wide ? 2048 : 256);
  if (tokens * slices >= ((int64_t)1 << 24)) return FP4Q_ERR_SHAPE;  // 2^32 threads
  const CombineArgs a{y, add, out, ld_y, ld_add, ld_out, weights, chosen, (int)top_k, (int)n, (int)slices};
  const dim3 grid((unsigned)(tokens * slices));
  hipStream_t s = (hipStream_t)stream;
  with_type(dtype, [&](auto tp) {
    using T = std::remove_pointer_t<decltype(tp)>;
    with_type(out_dtype, [&](auto op) {
      using O = std::remove_pointer_t<decltype(op)>;
      if (wide) hipLaunchKernelGGL((combine_kernel<T, O, 8>), grid, dim3(256), 0, s, a);
      else hipLaunchKernelGGL((combine_kernel<T, O, 1>), grid, dim3(256), 0, s, a);
    });
  });
  return hip_status();
}
