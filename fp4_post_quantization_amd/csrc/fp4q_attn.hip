// Attention over an MXFP4 key/value cache (include/fp4q_kv.h) on gfx950.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "fp4q.h"
#include "fp4q_device.h"
#include "fp4q_kv.h"
#include "fp4q_kv_host.h"

namespace fp4q {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr float kNegInf = -__builtin_inff();
constexpr float kLn2 = 0.6931471805599453f;
constexpr size_t kAttnHeader = 256;  // workspace: status word; then the spans' Joins, then partial results

// What a span leaves for the joining kernel: the unit that begins in it and
// ends in a later one (rows 0: there is none).
struct Join {
  int64_t first;  // the sequence's first row of q
  int64_t row0;   // the row tile's first (token, head) row
  int last, rows, head, pad;
};

struct AttnArgs {
  AttnShape sh;
  const uint16_t *q;
  int64_t q_st, q_sh;
  const uint8_t *kc, *ks, *vc, *vs;
  int64_t pages, page_stride, head_stride, token_stride;
  int log_page;
  const int32_t *table, *lens, *cu;
  int64_t table_stride;
  float scale_log2;  // scale * log2(e): scores are kept in units of log 2
  uint16_t *out;
  float *lse;
  uint32_t *status;
  float *parts;
  Join *joins;  // [spans]
  int spans;  // work items of the split form; 0: one workgroup per (sequence, row tile, head)
};

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform64(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(v >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

// v, without the compiler knowing that it does not change: what is derived
// from it is computed where it is used instead of being kept in registers
// throughout a loop.
__device__ __forceinline__ int opaque(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// In a block that few iterations enter: keeps the compiler from running it
// in all of them and selecting afterwards.
__device__ __forceinline__ void not_speculated() { asm volatile(""); }

__device__ __forceinline__ AttnSeq seq_of(const AttnArgs &a, int b) {
  const int64_t begin = a.cu ? a.cu[b] : b, end = a.cu ? a.cu[b + 1] : b + 1;
  return attn_seq(a.sh, a.lens[b], begin, end);
}

// The same for a sequence that is the same in every lane.
__device__ __forceinline__ AttnSeq seq_of_uniform(const AttnArgs &a, int b) {
  const int begin = a.cu ? uniform(a.cu[b]) : b, end = a.cu ? uniform(a.cu[b + 1]) : b + 1;
  return attn_seq(a.sh, uniform(a.lens[b]), begin, end);
}

// Work of sequence b: (row tile, head) units times its key tiles (split
// form), or the units alone.
template <int ROWS, int TT>
__device__ __forceinline__ int64_t work_of(const AttnArgs &a, int b, bool split) {
  if (b >= a.sh.batch) return 0;
  const AttnWork w = attn_work(a.sh, seq_of(a, b), ROWS, TT);
  return w.row_tiles * a.sh.heads * (split ? w.n + kUnitCost : 1);
}

__device__ __forceinline__ int64_t shfl_up64(int64_t v, int d) {
  const int lo = __shfl_up((int)(uint32_t)v, d), hi = __shfl_up((int)(v >> 32), d);
  return (int64_t)(((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo);
}

// The sequences' work, scanned by one wave 64 sequences at a time; the first
// 64 are scanned once.
template <int ROWS, int TT>
struct WorkScan {
  const AttnArgs &a;
  int lane;
  bool split;
  int64_t mine0, sum0;
  __device__ WorkScan(const AttnArgs &args, int l, bool sp) : a(args), lane(l), split(sp) { sum0 = scan(0, mine0); }
  __device__ int64_t scan(int base, int64_t &mine) const {  // inclusive prefix of this group
    mine = work_of<ROWS, TT>(a, base + lane, split);
    int64_t s = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t o = shfl_up64(s, d);
      if (lane >= d) s += o;
    }
    return s;
  }
  static __device__ int64_t lane_value(int64_t v, int l) {
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)v, l), hi = __builtin_amdgcn_readlane((int)(v >> 32), l);
    return (int64_t)(((uint64_t)hi << 32) | lo);
  }
  __device__ int64_t total() const {
    int64_t t = lane_value(sum0, 63), mine;
    for (int base = 64; base < a.sh.batch; base += 64) t += lane_value(scan(base, mine), 63);
    return t;
  }
  // The sequence that position pos of the work falls in, and the position
  // within it; false past the end.
  __device__ bool find(int64_t pos, int &b, int64_t &off) const {
    int64_t run = 0, mine = mine0, s = sum0;
    for (int base = 0;;) {
      const uint64_t hit = __ballot(pos < run + s);
      if (hit) {
        const int l = __builtin_ctzll(hit);
        b = base + l;
        off = pos - run - lane_value(s - mine, l);
        return true;
      }
      run += lane_value(s, 63);
      base += 64;
      if (base >= a.sh.batch) return false;
      s = scan(base, mine);
    }
  }
};

template <int D>
struct Geo {
  static constexpr int KP = D == 256 ? 2 : 1;    // pieces of a key row that a lane loads
  static constexpr int KW = D == 64 ? 2 : 4;     // dwords (8 elements) of a piece
  static constexpr int QS = KP * KW;             // 32-element steps of a score
  static constexpr int DT = D / 16;              // output tiles; lane c of 16 owns elements c DT .. c DT + DT - 1
  static constexpr int TT = 32;                  // tokens of a key tile
  static constexpr int TG = TT / 16;
  using KT = std::conditional_t<D == 64, u32x2, u32x4>;
  using VT = std::conditional_t<D == 64, uint16_t, std::conditional_t<D == 128, uint32_t, u32x2>>;
  // first element of lane group g's 8 in step (p, w) of a score: any order of the row will do, as long as queries
  // and keys agree, so a lane takes whole loaded dwords
  static __device__ constexpr int step_at(int p, int w, int g) { return p * 128 + g * (8 * KW) + w * 8; }
};

// A wave's registers of one key tile, as loaded.
template <int D>
struct KvTile {
  using G = Geo<D>;
  typename G::KT k[G::TG][G::KP];
  uint32_t ks[G::TG][G::KP];
  typename G::VT v[G::TG][4];
  uint32_t vs[G::TG][4];
};

// Offsets of a lane within the 16 tokens of a group (bytes of codes).  Keys:
// lane (m = lane % 16, g = lane / 16) takes part g of token (m % 4) 4 + m / 4,
// so that register i of the score tile is token 4 i + g.  Values: lane
// (c, g) takes the elements it owns of token 4 j + g in load j: a wave's load
// covers 4 whole rows.
template <int D>
struct LaneAt {
  uint32_t k, ks, v, vs;
  __device__ LaneAt(int lane, int64_t token_stride) {
    const uint32_t m = lane & 15, g = lane >> 4, ts = (uint32_t)token_stride;
    const uint32_t kt = (m & 3) * 4 + (m >> 2);
    k = kt * ts + g * 4 * Geo<D>::KW;
    ks = kt * (ts / 16) + (D == 64 ? g / 2 : g);
    v = g * ts + m * (D / 32);
    vs = g * (ts / 16) + m * Geo<D>::DT / 32;
  }
};

template <int D>
__device__ __forceinline__ void load_tile(const AttnArgs &a, const LaneAt<D> &at, int64_t head_off, int token0,
                                          const int (&page)[Geo<D>::TG], KvTile<D> &t) {
  using G = Geo<D>;
  // 32-bit offsets from uniform bases, opaque so that they are not widened to 64-bit registers outside the loop
  const uint32_t k_at = opaque(at.k), ks_at = opaque(at.ks), v_at = opaque(at.v), vs_at = opaque(at.vs);
#pragma unroll
  for (int tg = 0; tg < G::TG; ++tg) {
    const int r = (token0 + 16 * tg) & ((1 << a.log_page) - 1);
    const int64_t off = head_off + (int64_t)page[tg] * a.page_stride + r * a.token_stride;
    const uint8_t *kc = a.kc + off, *vc = a.vc + off, *ks = a.ks + (off >> 4), *vs = a.vs + (off >> 4);
#pragma unroll
    for (int p = 0; p < G::KP; ++p) {
      t.k[tg][p] = *reinterpret_cast<const typename G::KT *>(kc + (k_at + p * 64u));
      t.ks[tg][p] = ks[ks_at + p * 4u];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      t.v[tg][j] = *reinterpret_cast<const typename G::VT *>((vc + 4 * j * a.token_stride) + v_at);
      t.vs[tg][j] = (vs + j * (a.token_stride >> 2))[vs_at];
    }
  }
}

__device__ __forceinline__ float xor16(float v) { return __shfl_xor(v, 16); }
__device__ __forceinline__ float xor32(float v) { return __shfl_xor(v, 32); }

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const bf16x2 v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}

// Query operand of the score product for 16 rows: lane (row n, g) holds the
// elements step_at(p, w, g) .. + 7 of its row for every step.
template <int D>
struct QFrag {
  u32x4 x[Geo<D>::QS];
};

template <int D>
__device__ __forceinline__ void load_query(const uint16_t *q, bool on, int g, QFrag<D> &f) {
  using G = Geo<D>;
#pragma unroll
  for (int p = 0; p < G::KP; ++p)
#pragma unroll
    for (int w = 0; w < G::KW; ++w)
      f.x[p * G::KW + w] =
          on ? *reinterpret_cast<const u32x4 *>(q + G::step_at(p, w, g)) : u32x4{0u, 0u, 0u, 0u};
}

// The two bfloat16 values q 2^(b - 127) of byte BYTE of w; scale holds b in
// its exponent bits (all 256 values of b were checked to decode as E8M0).
template <int BYTE>
__device__ __forceinline__ uint32_t fp4x2_to_bf16(uint32_t w, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, BYTE));
}
__device__ __forceinline__ bf16x8 fp4x8_to_bf16(uint32_t w, float scale) {
  const u32x4 v = {fp4x2_to_bf16<0>(w, scale), fp4x2_to_bf16<1>(w, scale), fp4x2_to_bf16<2>(w, scale),
                   fp4x2_to_bf16<3>(w, scale)};
  return __builtin_bit_cast(bf16x8, v);
}

// Online softmax state and outputs of 16 query rows (row n = lane % 16):
// o[dt][i] is element (4 g + i) DT + dt, l the lane's own share of the sum.
template <int D>
struct RowState {
  f32x4 o[Geo<D>::DT];
  float m, l;
};

// One key tile: scores, softmax, and the tile's part of the output.
template <int D, int NR>
__device__ __forceinline__ void consume_tile(const AttnArgs &a, const KvTile<D> &t, const QFrag<D> (&q)[NR],
                                             const int (&lo)[NR], const int (&hi)[NR], int token0, bool full,
                                             uint32_t groups_ok, int keys_lo, int keys_hi, int lane,
                                             RowState<D> (&st)[NR]) {
  using G = Geo<D>;
  const int g = lane >> 4;
  f32x4 s[NR][G::TG];
#pragma unroll
  for (int tg = 0; tg < G::TG; ++tg) {
#pragma unroll
    for (int r = 0; r < NR; ++r) s[r][tg] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < G::KP; ++k) {
      const float ks = as_f(t.ks[tg][k] << 23);
#pragma unroll
      for (int w = 0; w < G::KW; ++w) {
        const bf16x8 kv = fp4x8_to_bf16(t.k[tg][k][w], ks);
#pragma unroll
        for (int r = 0; r < NR; ++r)
          s[r][tg] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              kv, __builtin_bit_cast(bf16x8, q[r].x[k * G::KW + w]), s[r][tg], 0, 0, 0);
      }
    }
  }
  uint32_t p[NR][G::TG / 2][4];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    float mx = kNegInf;
#pragma unroll
    for (int tg = 0; tg < G::TG; ++tg) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[r][tg][i] *= a.scale_log2;
      }
    }
    if (!full) {
      not_speculated();
#pragma unroll
      for (int tg = 0; tg < G::TG; ++tg) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = token0 + 16 * tg + 4 * i + g;
          s[r][tg][i] = (tok >= lo[r]) & (tok < hi[r]) & ((groups_ok >> tg) & 1u) ? s[r][tg][i] : kNegInf;
        }
      }
    }
#pragma unroll
    for (int tg = 0; tg < G::TG; ++tg)
#pragma unroll
      for (int i = 0; i < 4; ++i) mx = fmaxf(mx, s[r][tg][i]);
    // the running maximum moves only when a score passes it by more than 2^8: until then the exponentials stay
    // below 2^8, and neither the sum nor the outputs need rescaling
    if (__ballot(mx > st[r].m + 8.0f)) {
      mx = fmaxf(mx, xor16(mx));
      mx = fmaxf(mx, xor32(mx));
      const float m = fmaxf(st[r].m, mx);
      const float shrink = st[r].m == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(st[r].m - m);
      st[r].m = m;
      st[r].l *= shrink;
#pragma unroll
      for (int dt = 0; dt < G::DT; ++dt)
#pragma unroll
        for (int i = 0; i < 4; ++i) st[r].o[dt][i] *= shrink;
    }
    const float ref = st[r].m == kNegInf ? 0.0f : st[r].m;
#pragma unroll
    for (int tg = 0; tg < G::TG; ++tg) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[r][tg][i] = __builtin_amdgcn_exp2f(s[r][tg][i] - ref);
        st[r].l += s[r][tg][i];
      }
      p[r][tg / 2][2 * (tg & 1)] = pack_bf16(s[r][tg][0], s[r][tg][1]);
      p[r][tg / 2][2 * (tg & 1) + 1] = pack_bf16(s[r][tg][2], s[r][tg][3]);
    }
  }
#pragma unroll
  for (int h = 0; h < G::TG / 2; ++h) {
    typename G::VT v[8];
    float vs[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int tg = 2 * h + j / 4;
      v[j] = t.v[tg][j & 3];
      vs[j] = as_f(t.vs[tg][j & 3] << 23);
    }
    if (!full) {  // what lies outside every row's keys must not reach a product, where 0 * NaN is NaN
      not_speculated();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int tg = 2 * h + j / 4;
        const int tok = token0 + 16 * tg + 4 * (j & 3) + g;
        if (!((tok >= keys_lo) & (tok < keys_hi) & ((groups_ok >> tg) & 1u))) {
          v[j] = typename G::VT{};
          vs[j] = 1.0f;
        }
      }
    }
    bf16x8 pv[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const u32x4 w = {p[r][h][0], p[r][h][1], p[r][h][2], p[r][h][3]};
      pv[r] = __builtin_bit_cast(bf16x8, w);
    }
#pragma unroll
    for (int d2 = 0; d2 < G::DT / 2; ++d2) {  // elements 2 d2 and 2 d2 + 1 of the lane
      uint32_t x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t w;
        if constexpr (D == 256) w = v[j][d2 / 4];
        else w = v[j];
        x[j] = (d2 & 3) == 0   ? fp4x2_to_bf16<0>(w, vs[j])
               : (d2 & 3) == 1 ? fp4x2_to_bf16<1>(w, vs[j])
               : (d2 & 3) == 2 ? fp4x2_to_bf16<2>(w, vs[j])
                               : fp4x2_to_bf16<3>(w, vs[j]);
      }
      u32x4 e0, e1;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        e0[k] = __builtin_amdgcn_perm(x[2 * k + 1], x[2 * k], 0x05040100u);
        e1[k] = __builtin_amdgcn_perm(x[2 * k + 1], x[2 * k], 0x07060302u);
      }
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        st[r].o[2 * d2] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, e0), pv[r],
                                                                  st[r].o[2 * d2], 0, 0, 0);
        st[r].o[2 * d2 + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, e1), pv[r],
                                                                      st[r].o[2 * d2 + 1], 0, 0, 0);
      }
    }
  }
}

// A partial result: ROWS x D float32 outputs (unnormalised, relative to m),
// then the rows' maxima m and sums l.
template <int D, int ROWS>
struct Part {
  static constexpr int64_t kFloats = (int64_t)ROWS * (D + 2);
  static __device__ float *o(float *parts, int64_t slot) { return parts + slot * kFloats; }
  static __device__ float *m(float *parts, int64_t slot) { return parts + slot * kFloats + ROWS * D; }
  static __device__ float *l(float *parts, int64_t slot) { return parts + slot * kFloats + ROWS * (D + 1); }
};

__device__ __forceinline__ float part_weight(float m, float top) {
  return m == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m - top);
}

// Waves of a SIMD that the registers of a variant leave room for.
constexpr int waves_per_simd(int dim, int nr) { return nr == 1 && dim <= 128 ? 2 : 1; }

// Row r of a sequence's row tile: token i = r / groups, query head of group r % groups.
template <int D, int NR, int NW>
__global__ __launch_bounds__(64 * NW, waves_per_simd(D, NR)) void attn_rows_kernel(AttnArgs a) {
  using G = Geo<D>;
  constexpr int ROWS = 16 * NR, TT = G::TT, TG = G::TG;
  constexpr int LD = D + 4;  // padded row of the merge buffer
  __shared__ __align__(16) float mo[NW][16][LD];
  __shared__ float mm[NW][16], ml[NW][16];
  const int lane = threadIdx.x & 63, wave = wave_index();
  const Status status{a.status, true};
  if (blockIdx.x == 0 && wave == 0) {  // takes the status slot, and checks every sequence's length and rows
    bool bad = false;
    for (int i = lane; i < a.sh.batch; i += 64) bad |= seq_of(a, i).bad;
    const uint32_t bits = __ballot(bad) ? FP4Q_DATA_BAD_TABLE : 0u;
    if (lane == 0) status.merge(bits);
  }
  uint32_t err = 0u;
  const LaneAt<D> at(lane, a.token_stride);
  const WorkScan<ROWS, TT> scan{a, lane, a.spans != 0};

  int64_t pos, end, total = 0;
  int64_t span = blockIdx.x;
  bool joined = false;  // this span's Join is written
  if (a.spans) {
    total = uniform64(scan.total());
    pos = attn_cut(total, a.spans, span);
    end = attn_cut(total, a.spans, span + 1);
  } else {
    pos = span;
    end = span + 1;
  }
  int b = 0;
  int64_t off = 0;
  if (pos >= end || !scan.find(pos, b, off)) {
    if (a.spans && threadIdx.x == 0) a.joins[span] = Join{0, 0, 0, 0, 0, 0};
    return;
  }
  b = uniform(b);
  off = uniform64(off);

  while (pos < end) {
    const AttnSeq sq = seq_of_uniform(a, b);
    const AttnWork wk = attn_work(a.sh, sq, ROWS, TT);
    const int64_t size = a.spans ? wk.n + kUnitCost : 1;  // of a unit
    const int64_t units = wk.row_tiles * a.sh.heads;
    if (off >= units * size) {  // on to the next sequence that has rows
      off = 0;
      if (++b >= a.sh.batch) break;
      continue;
    }
    const int64_t unit = attn_div(off, size);
    const int rt = uniform((int)attn_div(unit, a.sh.heads)), h = uniform((int)(unit - (int64_t)rt * a.sh.heads));
    const int64_t from = off - unit * size, here = end - pos < size - from ? end - pos : size - from;
    AttnPart part{0, wk.n};  // this workgroup's key tiles of the unit
    if (a.spans) part = attn_part(from, from + here, wk.n);
    pos += here;
    off += here;
    const int t0 = uniform(part.t0), t1 = uniform(part.t1);
    if (t0 == t1) continue;
    const bool whole = t0 == 0 && t1 == wk.n;
    const int64_t r0 = (int64_t)rt * ROWS, rows = (int64_t)sq.fresh * a.sh.groups;
    const int live = uniform((int)(rows - r0 < ROWS ? rows - r0 : ROWS));
    if (!whole && t0 == 0) {
      joined = true;
      if (threadIdx.x == 0)
        a.joins[span] = Join{sq.first, r0, (int)attn_span_of(total, a.spans, pos - here - from + size - 1), live, h, 0};
    }
    const int i0 = uniform((int)attn_div(r0, a.sh.groups)), i1 = uniform((int)attn_div(r0 + live - 1, a.sh.groups));
    // keys that all rows of the tile see
    const int all_lo = uniform(attn_lo(a.sh, sq, i1)), all_hi = uniform(attn_hi(a.sh, sq, i0));
    // keys that any row of the sequence sees
    const int keys_lo = uniform(attn_lo(a.sh, sq, 0)), keys_hi = uniform(attn_hi(a.sh, sq, sq.fresh - 1));

    const int ln = opaque(lane), ng = ln >> 4, nn = ln & 15;
    QFrag<D> q[NR];
    RowState<D> st[NR];
    int lo[NR], hi[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int64_t row = r0 + 16 * r + nn;
      const bool on = row < rows;
      const int i = on ? (int)attn_div(row, a.sh.groups) : i0;
      const int qh = h * a.sh.groups + (on ? (int)(row - (int64_t)i * a.sh.groups) : 0);
      load_query<D>(a.q + (sq.first + i) * a.q_st + qh * a.q_sh, on, ng, q[r]);
      lo[r] = attn_lo(a.sh, sq, i);
      hi[r] = attn_hi(a.sh, sq, i);
#pragma unroll
      for (int dt = 0; dt < G::DT; ++dt) st[r].o[dt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      st[r].m = kNegInf;
      st[r].l = 0.0f;
    }

    // the workgroup's tiles, a contiguous part for each wave
    const int nt = t1 - t0;
    const int w0 = t0 + (int)((int64_t)nt * wave / NW), w1 = t0 + (int)((int64_t)nt * (wave + 1) / NW);
    const int64_t head_off = h * a.head_stride;
    const int32_t *row_table = a.table + b * a.table_stride;
    // lane i holds the page of the i-th group of 16 tokens of a block of 64 groups; -1: none
    constexpr int BLOCK = 64 / TG;  // key tiles of it
    auto pages_of = [&](int tile) {
      const int tok = (wk.lo + tile) * TT + 16 * lane;  // below 2^30 + 64 * 16
      int id = -1;
      if (tile < w1 && tok < keys_hi && tok + 15 >= keys_lo) {
        id = row_table[(uint32_t)(tok >> a.log_page)];
        if (id < 0 || id >= a.pages) {
          err |= FP4Q_DATA_BAD_TABLE;
          id = -1;
        }
      }
      return id;
    };
    auto fetch = [&](int tile, int ids, int first, KvTile<D> &t, uint32_t &ok) {
      int page[TG];
      ok = 0u;
#pragma unroll
      for (int tg = 0; tg < TG; ++tg) {
        const int id = __builtin_amdgcn_readlane(ids, (tile - first) * TG + tg);
        ok |= id >= 0 ? 1u << tg : 0u;
        page[tg] = id < 0 ? 0 : id;
      }
      load_tile<D>(a, at, head_off, (wk.lo + tile) * TT, page, t);
    };
    if (w0 < w1) {
      int first = w0;
      int ids = pages_of(first), ids_next = pages_of(first + BLOCK);
      KvTile<D> even, odd;
      uint32_t ok_even, ok_odd = 0u;
      fetch(w0, ids, first, even, ok_even);
      auto step = [&](int tile, const KvTile<D> &cur, uint32_t ok, KvTile<D> &nxt, uint32_t &ok_next) {
        if (tile + 1 < w1) {
          if (tile + 1 == first + BLOCK) {
            first += BLOCK;
            ids = ids_next;
            ids_next = pages_of(first + BLOCK);
          }
          fetch(tile + 1, ids, first, nxt, ok_next);
        }
        const int token0 = (wk.lo + tile) * TT;
        const bool full = ok == (1u << TG) - 1u && token0 >= all_lo && token0 + TT <= all_hi;
        consume_tile<D, NR>(a, cur, q, lo, hi, token0, full, ok, keys_lo, keys_hi, lane, st);
      };
      for (int tile = w0; tile < w1; tile += 2) {
        step(tile, even, ok_even, odd, ok_odd);
        if (tile + 1 < w1) step(tile + 1, odd, ok_odd, even, ok_even);
      }
    }

    // merge the waves, 16 rows at a time
    const int mt = opaque((int)threadIdx.x), mn = mt & 15, mg = (mt >> 4) & 3;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      float l = st[r].l;
      l += xor16(l);
      l += xor32(l);
      if (mg == 0) {
        mm[wave][mn] = st[r].m;
        ml[wave][mn] = l;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int dt = 0; dt < G::DT; dt += 4)
          *reinterpret_cast<f32x4 *>(&mo[wave][mn][(4 * mg + i) * G::DT + dt]) =
              f32x4{st[r].o[dt][i], st[r].o[dt + 1][i], st[r].o[dt + 2][i], st[r].o[dt + 3][i]};
      __syncthreads();
      // 8 elements of a row a thread
      for (int e = mt; e < 16 * D / 8; e += 64 * NW) {
        const int row = e / (D / 8), d = e % (D / 8) * 8;
        if (16 * r + row >= live) continue;
        float top = mm[0][row];
#pragma unroll
        for (int w = 1; w < NW; ++w) top = fmaxf(top, mm[w][row]);
        float sum = 0.0f, o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const float f = part_weight(mm[w][row], top);
          sum = fmaf(ml[w][row], f, sum);
#pragma unroll
          for (int k = 0; k < 8; ++k) o[k] = fmaf(mo[w][row][d + k], f, o[k]);
        }
        if (whole) {
          const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
          const int64_t gr = r0 + 16 * r + row;
          const int64_t i = attn_div(gr, a.sh.groups);
          const int64_t head = (sq.first + i) * (a.sh.heads * a.sh.groups) + h * a.sh.groups + (gr - i * a.sh.groups);
          u32x4 w;
#pragma unroll
          for (int k = 0; k < 4; ++k) w[k] = pack_bf16(o[2 * k] * inv, o[2 * k + 1] * inv);
          *reinterpret_cast<u32x4 *>(a.out + head * D + d) = w;
          if (a.lse && d == 0) a.lse[head] = sum > 0.0f ? (top + log2f(sum)) * kLn2 : (sum == 0.0f ? kNegInf : sum);
        } else {
          using P = Part<D, ROWS>;
          const int64_t slot = 2 * span + (t0 == 0 ? 1 : 0);
          float *po = P::o(a.parts, slot) + (16 * r + row) * D + d;
          *reinterpret_cast<f32x4 *>(po) = f32x4{o[0], o[1], o[2], o[3]};
          *reinterpret_cast<f32x4 *>(po + 4) = f32x4{o[4], o[5], o[6], o[7]};
          if (d == 0) {
            P::m(a.parts, slot)[16 * r + row] = top;
            P::l(a.parts, slot)[16 * r + row] = sum;
          }
        }
      }
      __syncthreads();
    }
  }
  if (a.spans && !joined && threadIdx.x == 0) a.joins[span] = Join{0, 0, 0, 0, 0, 0};
  if (__builtin_expect(err != 0u, 0)) status.report(err);
}

// Joins the partial results of units that several spans share: workgroup
// (w, row) joins a row of the unit that begins in span w and ends in a later
// one, from span w's second slot and the first slots of the spans after it.
template <int D, int ROWS>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
  constexpr int PER = D / 64;  // elements of a lane
  __shared__ float so[4][D];
  __shared__ float sm[4], sl[4];
  const int lane = threadIdx.x & 63, wave = wave_index();
  const int64_t span = blockIdx.x;
  const int row = blockIdx.y;
  const Join j = a.joins[span];
  if (row >= j.rows) return;
  const int64_t last = j.last, gr = j.row0 + row;
  using P = Part<D, ROWS>;
  float m = kNegInf, l = 0.0f, o[PER];
#pragma unroll
  for (int k = 0; k < PER; ++k) o[k] = 0.0f;
  for (int64_t s = span + wave; s <= last; s += 4) {
    const int64_t slot = 2 * s + (s == span ? 1 : 0);
    const float pm = P::m(a.parts, slot)[row], pl = P::l(a.parts, slot)[row];
    const float *po = P::o(a.parts, slot) + row * D + lane * PER;
    float v[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) v[k] = po[k];
    const float top = fmaxf(m, pm);
    const float f0 = part_weight(m, top), f1 = part_weight(pm, top);
    m = top;
    l = l * f0 + pl * f1;
#pragma unroll
    for (int k = 0; k < PER; ++k) o[k] = o[k] * f0 + v[k] * f1;
  }
  if (lane == 0) {
    sm[wave] = m;
    sl[wave] = l;
  }
#pragma unroll
  for (int k = 0; k < PER; ++k) so[wave][lane * PER + k] = o[k];
  __syncthreads();
  if (threadIdx.x >= D / 2) return;
  float top = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  float sum = 0.0f, x = 0.0f, y = 0.0f;
  const int d = 2 * threadIdx.x;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float f = part_weight(sm[w], top);
    sum = fmaf(sl[w], f, sum);
    x = fmaf(so[w][d], f, x);
    y = fmaf(so[w][d + 1], f, y);
  }
  const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
  const int64_t i = attn_div(gr, a.sh.groups);
  const int64_t head = (j.first + i) * (a.sh.heads * a.sh.groups) + j.head * a.sh.groups + (gr - i * a.sh.groups);
  reinterpret_cast<uint32_t *>(a.out)[(head * D + d) / 2] = pack_bf16(x * inv, y * inv);
  if (a.lse && d == 0) a.lse[head] = sum > 0.0f ? (top + log2f(sum)) * kLn2 : (sum == 0.0f ? kNegInf : sum);
}

__global__ __launch_bounds__(64) void attn_status_kernel(uint32_t *status) {
  if (threadIdx.x == 0) Status{status, true}.merge(0u);
}

// ------------------------------------------------------------ dispatch ----
constexpr int kCus = 256;
constexpr int kDirectTiles = 32; // units of at most this many key tiles are not split

struct Plan {
  int nr;         // row tiles of 16 a workgroup
  int64_t units;  // upper bound of (sequence, row tile, head) units
  int spans;
  int64_t part_floats;
};

Plan make_plan(int64_t tokens, int64_t batch, int64_t q_heads, int64_t heads, int64_t head_dim, int64_t max_new,
               int64_t max_len) {
  Plan p;
  const int64_t groups = q_heads / heads;
  p.nr = max_new * groups <= 16 || head_dim == 256 ? 1 : 2;
  const int rows = 16 * p.nr;
  const int64_t tile = 32;
  // a sequence's rows fill its tiles except the last one
  int64_t row_tiles = tokens * groups / rows + batch;
  const int64_t per_seq = (max_new * groups + rows - 1) / rows;
  if (row_tiles > batch * per_seq) row_tiles = batch * per_seq;
  p.units = row_tiles * heads;
  const bool direct = (max_len + tile - 1) / tile + 1 <= kDirectTiles;
  p.spans = direct ? 0 : kCus * waves_per_simd((int)head_dim, p.nr);  // as many workgroups as fit the chip at once
  p.part_floats = direct ? 0 : 2 * (int64_t)p.spans * rows * (head_dim + 2);
  return p;
}

bool sizes_ok(int64_t tokens, int64_t batch, int64_t q_heads, int64_t heads, int64_t head_dim, int64_t max_new,
              int64_t max_len) {
  return kv_head_dim_ok(head_dim) && heads >= 1 && heads * head_dim <= 65536 && q_heads >= heads &&
         q_heads <= 65536 && q_heads % heads == 0 && tokens >= 0 && tokens < kKvMaxUnits / q_heads && batch >= 0 &&
         batch < ((int64_t)1 << 24) && max_new >= 0 && max_new <= tokens && max_len >= 0 &&
         max_len <= ((int64_t)1 << 30);
}

fp4q_status_t hip_status() { return hipGetLastError() == hipSuccess ? FP4Q_OK : FP4Q_ERR_HIP; }

template <int D, int NR>
void launch_rows(const AttnArgs &a, const Plan &p, hipStream_t s) {
  constexpr int NW = 4;
  if (p.spans) {
    hipLaunchKernelGGL((attn_rows_kernel<D, NR, NW>), dim3((unsigned)p.spans), dim3(64 * NW), 0, s, a);
    // no unit has more rows than a sequence
    const int64_t rows = (int64_t)a.sh.max_new * a.sh.groups;
    hipLaunchKernelGGL((attn_join_kernel<D, 16 * NR>), dim3((unsigned)p.spans, (unsigned)(rows < 16 * NR ? rows : 16 * NR)),
                       dim3(256), 0, s, a);
  } else {
    hipLaunchKernelGGL((attn_rows_kernel<D, NR, NW>), dim3((unsigned)p.units), dim3(64 * NW), 0, s, a);
  }
}

}  // namespace
}  // namespace fp4q

using namespace fp4q;

extern "C" size_t fp4q_attention_mxfp4_workspace_bytes(int64_t tokens, int64_t batch, int64_t q_heads, int64_t heads,
                                                       int64_t head_dim, int64_t max_new, int64_t max_len) {
  if (!sizes_ok(tokens, batch, q_heads, heads, head_dim, max_new, max_len)) return 0;
  const Plan p = make_plan(tokens, batch, q_heads, heads, head_dim, max_new, max_len);
  return kAttnHeader + p.spans * sizeof(Join) + 4 * (size_t)p.part_floats;
}

extern "C" fp4q_status_t fp4q_attention_mxfp4(const fp4q_kv_cache_t *cache, const void *q, int64_t q_token_stride,
                                              int64_t q_head_stride, int64_t tokens, int64_t q_heads,
                                              const int32_t *block_table, int64_t table_stride, int64_t table_width,
                                              int64_t batch, const int32_t *seq_lens, const int32_t *cu_q,
                                              int64_t max_new, int64_t max_len, float scale, int causal,
                                              int64_t window, void *out, float *lse, void *workspace,
                                              size_t workspace_bytes, void *stream) {
  const bool empty = tokens == 0 || batch == 0;
  if (!cache || (!empty && (!q || !block_table || !seq_lens || !out))) return FP4Q_ERR_NULL;
  fp4q_status_t st = kv_check_cache(*cache);
  if (st != FP4Q_OK) return st;
  if (!sizes_ok(tokens, batch, q_heads, cache->heads, cache->head_dim, max_new, max_len)) return FP4Q_ERR_SHAPE;
  if (table_width < 0 || table_width > 0x7FFFFFFF || table_stride < table_width ||
      max_len > table_width * cache->page_size || (!cu_q && !empty && tokens != batch))
    return FP4Q_ERR_SHAPE;
  if (!cu_q && !empty && max_new < 1) return FP4Q_ERR_SHAPE;
  if ((causal != 0 && causal != 1) || window < 0 || window > 0x7FFFFFFF || !(scale >= -3e38f && scale <= 3e38f))
    return FP4Q_ERR_ARG;
  if ((st = kv_check_heads(FP4Q_BF16, tokens, q_heads, cache->head_dim, q_token_stride, q_head_stride, q)) != FP4Q_OK)
    return st;
  if (!empty && (!kv_aligned(out, 16) || !kv_aligned(lse, 4) || !kv_aligned(block_table, 4) ||
                 !kv_aligned(seq_lens, 4) || !kv_aligned(cu_q, 4)))
    return FP4Q_ERR_ALIGN;
  const size_t need =
      fp4q_attention_mxfp4_workspace_bytes(tokens, batch, q_heads, cache->heads, cache->head_dim, max_new, max_len);
  if (!workspace || workspace_bytes < need || !kv_aligned(workspace, 16)) return FP4Q_ERR_WORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  uint32_t *status = (uint32_t *)workspace;
  if (empty) {
    hipLaunchKernelGGL(attn_status_kernel, dim3(1), dim3(64), 0, s, status);
    return hip_status();
  }
  const Plan p = make_plan(tokens, batch, q_heads, cache->heads, cache->head_dim, max_new, max_len);
  if (p.units == 0) {  // no sequence has a row
    hipLaunchKernelGGL(attn_status_kernel, dim3(1), dim3(64), 0, s, status);
    return hip_status();
  }
  AttnArgs a;
  a.sh = AttnShape{tokens, (int)batch, (int)(q_heads / cache->heads), cache->heads, (int)max_new, (int)max_len,
                   causal, (int)window};
  a.q = (const uint16_t *)q;
  a.q_st = q_token_stride;
  a.q_sh = q_head_stride;
  a.kc = cache->k_codes;
  a.ks = cache->k_scales;
  a.vc = cache->v_codes;
  a.vs = cache->v_scales;
  a.pages = cache->pages;
  a.page_stride = cache->page_stride;
  a.head_stride = cache->head_stride;
  a.token_stride = cache->token_stride;
  a.log_page = kv_log2(cache->page_size);
  a.table = block_table;
  a.table_stride = table_stride;
  a.lens = seq_lens;
  a.cu = cu_q;
  a.scale_log2 = (float)((double)scale * 1.4426950408889634);
  a.out = (uint16_t *)out;
  a.lse = lse;
  a.status = status;
  a.joins = (Join *)((char *)workspace + kAttnHeader);
  a.parts = (float *)(a.joins + p.spans);
  a.spans = p.spans;
  auto go = [&](auto dc) {
    constexpr int D = decltype(dc)::value;
    if constexpr (D == 256) launch_rows<D, 1>(a, p, s);
    else if (p.nr == 1) launch_rows<D, 1>(a, p, s);
    else launch_rows<D, 2>(a, p, s);
  };
  if (cache->head_dim == 64) go(std::integral_constant<int, 64>{});
  else if (cache->head_dim == 128) go(std::integral_constant<int, 128>{});
  else go(std::integral_constant<int, 256>{});
  return hip_status();
}
