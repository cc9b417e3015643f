// Attention over an MXFP4 key/value cache (include/fp4q_kv.h) on gfx950.
//
// For a row of queries (a token's query head) and the keys t that it sees,
//   s_t = scale q.k_t,  O = sum_t 2^(s_t' - m) v_t / l,  l = sum_t 2^(s_t' - m),
// with s' = s log2(e) and m a running maximum, in one pass over the cache.
// Every query head of a group reads the same keys, so the rows of a unit of
// work are (token, query head of the group) pairs of one key/value head: the
// cache is read once for all of them.
//  * Both products run on the bfloat16 matrix cores.  Keys and values become
//    bfloat16 by one conversion for 2 elements, exactly (a code times a power
//    of two).  The scaled FP4 x FP8 instruction would take the codes as they
//    are, but it cuts a product 13 bits below the largest of its step, which
//    cost the scores 2e-5, and queries would have to be split in two.
//  * Both are computed transposed, S^T = K Q^T and O^T += V^T P^T: a lane's
//    score registers belong to one query row, and after exponentiation they
//    are P^T's operand as they lie, so that no score passes through LDS.
//    P is rounded to bfloat16 there (2^-8 of each term at most); the sum l
//    adds the exponentials before that, in float32, as are m, S and O.  The
//    result, bfloat16 itself, is then off by 0.0017 to 0.0024 (relative, root
//    mean square) where its own rounding alone gives 0.0016.  P in two parts
//    gave that 0.0016 for few rows, at 3 to 8% of the time (64 sequences 63.9
//    -> 68.7 us), and would take half as many matrix instructions again in a
//    prompt, which they bound beside the vector pipe.
//  * Few rows (attn_rows_kernel) are bound by the cache's bytes and, where
//    there are few of those, by a chain of dependent loads: lengths, page
//    number, codes.  Many rows (attn_prompt_kernel) are bound by the vector
//    and matrix pipes.  A call whose sequences differ much runs both, each on
//    its own sequences, one after the other (make_plan).
//  * A long cache with few units is cut into equal spans of work, one for
//    each workgroup that the chip holds, whatever sequence they fall in; a
//    span keeps what it has of a unit in float32 and attn_join_kernel joins
//    it.  The order of the joins is fixed, so results repeat bit for bit.
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
typedef float f32x16 __attribute__((ext_vector_type(16)));
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
  Divider by_groups, by_heads;
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
  bool first;  // the call's first kernel, which takes the status slot
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

// Work of a sequence: (row tile, head) units times what each costs (split
// form), or the units alone.
template <int ROWS, int TT>
__device__ __forceinline__ int64_t work_of(const AttnArgs &a, const AttnSeq &sq) {
  const AttnWork w = attn_work(a.sh, sq, ROWS, TT);
  return w.row_tiles * a.sh.heads * (a.spans ? w.n + kUnitCost : 1);
}

__device__ __forceinline__ int64_t lane_value(int64_t v, int l) {
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)v, l), hi = __builtin_amdgcn_readlane((int)(v >> 32), l);
  return (int64_t)(((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ int64_t shfl_up64(int64_t v, int d) {
  const int lo = __shfl_up((int)(uint32_t)v, d), hi = __shfl_up((int)(v >> 32), d);
  return (int64_t)(((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo);
}

// Inclusive prefix sums over the lanes of a wave: within the rows of 16 by
// shifts of 1, 2, 4 and 8 (lanes from outside a row count as 0), then row 0's
// and row 2's last lanes into rows 1 and 3, and lane 31 into rows 2 and 3.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_add(uint32_t v) {
  return v + (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, true);
}
__device__ __forceinline__ uint32_t dpp_prefix(uint32_t v) {
  v = dpp_add<0x111, 0xF>(v);
  v = dpp_add<0x112, 0xF>(v);
  v = dpp_add<0x114, 0xF>(v);
  v = dpp_add<0x118, 0xF>(v);
  v = dpp_add<0x142, 0xA>(v);
  return dpp_add<0x143, 0xC>(v);
}

// The sequences' work, scanned by one wave 64 sequences at a time; the first
// 64 are loaded and scanned once, lane i keeping sequence i.
template <int ROWS, int TT>
struct WorkScan {
  const AttnArgs &a;
  int lane;
  AttnSeq seq0;
  int64_t mine0, sum0;
  __device__ WorkScan(const AttnArgs &args, int l) : a(args), lane(l), seq0{0, 0, 0, false} {
    if (lane < a.sh.batch) seq0 = seq_of(a, lane);
    mine0 = lane < a.sh.batch ? work_of<ROWS, TT>(a, seq0) : 0;
    sum0 = prefix(mine0);
  }
  __device__ int64_t prefix(int64_t s) const {  // inclusive
    if (__ballot((uint64_t)s >> 25) == 0) return dpp_prefix((uint32_t)s);  // their sum fits 31 bits
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t o = shfl_up64(s, d);
      if (lane >= d) s += o;
    }
    return s;
  }
  __device__ int64_t scan(int base, int64_t &mine) const {
    mine = base + lane < a.sh.batch ? work_of<ROWS, TT>(a, seq_of(a, base + lane)) : 0;
    return prefix(mine);
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
  __device__ __forceinline__ AttnSeq seq(int b) const {  // of a sequence that is the same in every lane
    if (b >= 64) return seq_of_uniform(a, b);
    AttnSeq s;
    s.first = __builtin_amdgcn_readlane((int)seq0.first, b);  // below 2^30
    s.fresh = __builtin_amdgcn_readlane(seq0.fresh, b);
    s.len = __builtin_amdgcn_readlane(seq0.len, b);
    s.bad = false;
    return s;
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
  static constexpr int VS = D == 256 ? 4 : 1;    // value scales of 16 tokens that a lane loads
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
  uint32_t vs[G::TG][G::VS];
};

// Offsets of a lane within the 16 tokens of a group (bytes of codes).  Keys:
// lane (m = lane % 16, g = lane / 16) takes part g of token (m % 4) 4 + m / 4,
// so that register i of the score tile is token 4 i + g.  Values: lane
// (c, g) takes the elements it owns of token 4 j + g in load j: a wave's load
// covers 4 whole rows.  Up to heads of 128 a lane's values are of the same
// block as its quad's, so it loads the scale of token 4 (m % 4) + g and takes
// the others from its neighbours (value_scale): 2 loads in place of 8 of a
// tile's 20.  131072 keys 35.7 -> 34.8 us, 128 sequences of up to 1000 30.0 ->
// 29.2; for heads of 256, by pairs, it was slower (19.8 -> 20.5).
template <int D>
struct LaneAt {
  uint32_t k, ks, v, vs;
  __device__ LaneAt(int lane, int64_t token_stride) {
    const uint32_t m = lane & 15, g = lane >> 4, ts = (uint32_t)token_stride;
    const uint32_t kt = (m & 3) * 4 + (m >> 2);
    k = kt * ts + g * 4 * Geo<D>::KW;
    ks = kt * (ts / 16) + (D == 64 ? g / 2 : g);
    v = g * ts + m * (D / 32);
    vs = (D == 256 ? g : 4 * (m & 3) + g) * (ts / 16) + m * Geo<D>::DT / 32;
  }
};

// The scale of the lane's values of token 4 j + g, in a float32's exponent bits.
template <int D, int J>
__device__ __forceinline__ float value_scale(const uint32_t (&vs)[Geo<D>::VS]) {
  if constexpr (D == 256) return as_f(vs[J] << 23);
  else return as_f((uint32_t)__builtin_amdgcn_mov_dpp((int)(vs[0] << 23), J * 0x55, 0xF, 0xF, true));  // quad_perm
}

// off[tg]: byte offset of the first code row of the tile's 16-token group tg.
template <int D>
__device__ __forceinline__ void load_tile(const AttnArgs &a, const LaneAt<D> &at, const int64_t (&off)[Geo<D>::TG],
                                          KvTile<D> &t) {
  using G = Geo<D>;
  // 32-bit offsets from uniform bases, opaque so that they are not widened to 64-bit registers outside the loop
  const uint32_t k_at = opaque(at.k), ks_at = opaque(at.ks), v_at = opaque(at.v), vs_at = opaque(at.vs);
  const uint32_t v_step = 4 * (uint32_t)a.token_stride, vs_step = v_step >> 4;
#pragma unroll
  for (int tg = 0; tg < G::TG; ++tg) {
    const uint8_t *kc = a.kc + off[tg], *vc = a.vc + off[tg];
    const uint8_t *ks = a.ks + (off[tg] >> 4), *vs = a.vs + (off[tg] >> 4);
#pragma unroll
    for (int p = 0; p < G::KP; ++p) {
      t.k[tg][p] = *reinterpret_cast<const typename G::KT *>(kc + (k_at + p * 64u));
      t.ks[tg][p] = ks[ks_at + p * 4u];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      t.v[tg][j] = *reinterpret_cast<const typename G::VT *>(vc + (v_at + j * v_step));
    }
#pragma unroll
    for (int y = 0; y < G::VS; ++y) t.vs[tg][y] = vs[vs_at + y * vs_step];
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
template <int D>
__device__ __forceinline__ void consume_tile(const AttnArgs &a, const KvTile<D> &t, const QFrag<D> &q, int lo,
                                             int hi, int token0, bool full,
                                             uint32_t groups_ok, int keys_lo, int keys_hi, int lane,
                                             RowState<D> &st) {
  using G = Geo<D>;
  const int g = lane >> 4;
  f32x4 s[G::TG];
#pragma unroll
  for (int tg = 0; tg < G::TG; ++tg) {
    s[tg] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < G::KP; ++k) {
      const float ks = as_f(t.ks[tg][k] << 23);
#pragma unroll
      for (int w = 0; w < G::KW; ++w) {
        const bf16x8 kv = fp4x8_to_bf16(t.k[tg][k][w], ks);
        s[tg] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              kv, __builtin_bit_cast(bf16x8, q.x[k * G::KW + w]), s[tg], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int tg = 0; tg < G::TG; ++tg)
#pragma unroll
    for (int i = 0; i < 4; ++i) s[tg][i] *= a.scale_log2;
  if (!full) {
    not_speculated();
#pragma unroll
    for (int tg = 0; tg < G::TG; ++tg) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tok = token0 + 16 * tg + 4 * i + g;
        s[tg][i] = (tok >= lo) & (tok < hi) & ((groups_ok >> tg) & 1u) ? s[tg][i] : kNegInf;
      }
    }
  }
  float mx = kNegInf;
#pragma unroll
  for (int tg = 0; tg < G::TG; ++tg)
#pragma unroll
    for (int i = 0; i < 4; ++i) mx = fmaxf(mx, s[tg][i]);
  // the running maximum moves only when a score passes it by more than 2^8: until then the exponentials stay
  // below 2^8, and neither the sum nor the outputs need rescaling
  if (__ballot(mx > st.m + 8.0f)) {
    mx = fmaxf(mx, xor16(mx));
    mx = fmaxf(mx, xor32(mx));
    const float m = fmaxf(st.m, mx);
    const float shrink = st.m == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(st.m - m);
    st.m = m;
    st.l *= shrink;
#pragma unroll
    for (int dt = 0; dt < G::DT; ++dt)
#pragma unroll
      for (int i = 0; i < 4; ++i) st.o[dt][i] *= shrink;
  }
  const float ref = st.m == kNegInf ? 0.0f : st.m;
  uint32_t p[G::TG / 2][4];
#pragma unroll
  for (int tg = 0; tg < G::TG; ++tg) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[tg][i] = __builtin_amdgcn_exp2f(s[tg][i] - ref);
      st.l += s[tg][i];
    }
    p[tg / 2][2 * (tg & 1)] = pack_bf16(s[tg][0], s[tg][1]);
    p[tg / 2][2 * (tg & 1) + 1] = pack_bf16(s[tg][2], s[tg][3]);
  }
#pragma unroll
  for (int h = 0; h < G::TG / 2; ++h) {
    typename G::VT v[8];
    float vs[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int tg = 2 * h + j / 4;
      v[j] = t.v[tg][j & 3];
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t(&b)[G::VS] = t.vs[2 * h + k];
      vs[4 * k] = value_scale<D, 0>(b);
      vs[4 * k + 1] = value_scale<D, 1>(b);
      vs[4 * k + 2] = value_scale<D, 2>(b);
      vs[4 * k + 3] = value_scale<D, 3>(b);
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
    const bf16x8 pv = __builtin_bit_cast(bf16x8, u32x4{p[h][0], p[h][1], p[h][2], p[h][3]});
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
      st.o[2 * d2] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, e0), pv,
                                                             st.o[2 * d2], 0, 0, 0);
      st.o[2 * d2 + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, e1), pv,
                                                                 st.o[2 * d2 + 1], 0, 0, 0);
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

// A workgroup's part of a unit: key tiles lo + t0 .. lo + t1 - 1 of one
// (sequence, row tile, head).
struct Unit {
  AttnSeq sq;
  int64_t r0;            // first of the row tile's rows; row r is token r / groups, query head r % groups of the group
  int b, h, live;        // sequence, head, rows
  int lo, t0, t1;
  int i0, i1;            // first and last token of the rows
  int keys_lo, keys_hi;  // keys that any row of the sequence sees
  bool whole;            // these are all key tiles of the unit
};

// The units of a workgroup, one after another: with a.spans those of its span
// of the work, else the one with its number.
template <int ROWS, int TT>
struct Walk {
  const AttnArgs &a;
  WorkScan<ROWS, TT> scan;
  int64_t pos, end, off, total;
  int b, spans;
  bool joined;  // this span's Join is written

  __device__ __forceinline__ Walk(const AttnArgs &args, int lane, int index)
      : a(args), scan(args, lane), off(0), total(0), b(0), spans(0), joined(false) {
    pos = index;
    end = pos + 1;
    if (a.spans) {
      total = uniform64(scan.total());
      spans = attn_spans(total, a.spans);
      end = index < spans ? attn_cut(total, spans, pos + 1) : 0;
      pos = index < spans ? attn_cut(total, spans, pos) : 0;
    }
    if (!a.spans && !a.cu) {
      // One row each: all sequences have the same units, and no workgroup scans a large batch for its own (4096
      // sequences of up to 200 keys 437 -> 161 us, 256 of up to 100 11.9 -> 11).
      const uint32_t per = (uint32_t)((a.sh.groups + ROWS - 1) / ROWS) * (uint32_t)a.sh.heads;
      b = (int)((uint32_t)pos / per);
      off = pos - (int64_t)b * per;
      if (b >= a.sh.batch) end = pos;
    } else if (pos < end && !scan.find(pos, b, off)) {
      end = pos;
    }
    b = uniform(b);
    off = uniform64(off);
  }

  __device__ __forceinline__ bool next(Unit &u) {
    while (pos < end) {
      const AttnSeq sq = scan.seq(b);
      const AttnWork wk = attn_work(a.sh, sq, ROWS, TT);
      const int64_t size = a.spans ? wk.n + kUnitCost : 1;  // of a unit
      if (off >= wk.row_tiles * a.sh.heads * size) {        // on to the next sequence that has rows
        off = 0;
        if (++b >= a.sh.batch) return false;
        continue;
      }
      const int64_t unit = a.spans ? attn_div(off, size) : off;  // below 2^30 rows of 2^16 heads / 16
      int rt = uniform((int)divide((uint32_t)unit, a.by_heads));
      const int h = uniform((int)unit - rt * a.sh.heads);
      // causal: the last rows see the most keys; their workgroups start first
      if (!a.spans) rt = (int)wk.row_tiles - 1 - rt;
      const int64_t from = off - unit * size, here = end - pos < size - from ? end - pos : size - from;
      AttnPart part{0, wk.n};
      if (a.spans) part = attn_part(from, from + here, wk.n);
      pos += here;
      off += here;
      u.t0 = uniform(part.t0);
      u.t1 = uniform(part.t1);
      if (u.t0 == u.t1) continue;
      u.sq = sq;
      u.b = b;
      u.h = h;
      u.lo = wk.lo;
      u.whole = u.t0 == 0 && u.t1 == wk.n;
      u.r0 = (int64_t)rt * ROWS;
      const int64_t rows = (int64_t)sq.fresh * a.sh.groups;
      u.live = uniform((int)(rows - u.r0 < ROWS ? rows - u.r0 : ROWS));
      u.i0 = uniform((int)divide((uint32_t)u.r0, a.by_groups));
      u.i1 = uniform((int)divide((uint32_t)(u.r0 + u.live - 1), a.by_groups));
      u.keys_lo = uniform(attn_lo(a.sh, sq, 0));
      u.keys_hi = uniform(attn_hi(a.sh, sq, sq.fresh - 1));
      if (!u.whole && u.t0 == 0) {
        joined = true;
        if (threadIdx.x == 0)
          a.joins[blockIdx.x - 1] =
              Join{sq.first, u.r0, (int)attn_span_of(total, spans, pos - here - from + size - 1), u.live, u.h, 0};
      }
      return true;
    }
    return false;
  }
  __device__ __forceinline__ void finish() const {
    if (a.spans && !joined && threadIdx.x == 0) a.joins[blockIdx.x - 1] = Join{0, 0, 0, 0, 0, 0};
  }
};

// Position of row r of a unit among the rows of out and lse.
__device__ __forceinline__ int64_t out_row(const AttnArgs &a, int64_t first, int h, int64_t r) {
  const int64_t i = divide((uint32_t)r, a.by_groups);
  return (first + i) * (a.sh.heads * a.sh.groups) + h * a.sh.groups + (r - i * a.sh.groups);
}
__device__ __forceinline__ float row_factor(float sum) { return sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum); }
__device__ __forceinline__ float row_lse(float m, float sum) {
  return sum > 0.0f ? (m + log2f(sum)) * kLn2 : (sum == 0.0f ? kNegInf : sum);
}

// The first workgroup of a call takes the status slot and checks every
// sequence's length and rows; it has no other work, so that nobody's work
// waits for the slot's atomics.  In a second pass it has none at all.
__device__ __forceinline__ bool is_status_group(const AttnArgs &a, int lane, int wave) {
  if (blockIdx.x != 0) return false;
  if (wave == 0 && a.first) {
    bool bad = false;
    for (int i = lane; i < a.sh.batch; i += 64) bad |= seq_of(a, i).bad;
    const uint32_t bits = __ballot(bad) ? FP4Q_DATA_BAD_TABLE : 0u;
    if (lane == 0) Status{a.status, true}.merge(bits);
  }
  return true;
}

// The page of token tok of a sequence, -1 where it is outside the cache.
__device__ __forceinline__ int page_of(const AttnArgs &a, const int32_t *row_table, int tok, uint32_t &err) {
  const int id = row_table[(uint32_t)(tok >> a.log_page)];
  if (id >= 0 && id < a.pages) return id;
  err |= FP4Q_DATA_BAD_TABLE;
  return -1;
}

// Few rows: a unit is 16 rows (r is token r / groups, query head r % groups
// of the group) and one key/value head; the NW waves of its workgroup take
// equal parts of its key tiles (32 tokens, on v_mfma_f32_16x16x32_bf16), each
// with its own running maximum, and merge them through LDS at the end.  There
// is no LDS in the loop: a lane loads its operands' codes from memory (whole
// rows for each 16 lanes), the next tile's while it computes this one's.
// Bound by the cache's bytes: 64 sequences of 0 to 8192 tokens (64 query
// heads on 8, 128 wide; 292 MB) 61 us, 4.8 TB/s; 131072 tokens of one
// sequence (64 on 8, 143 MB) 30 us, 4.7 TB/s; the join takes 5 us more.  HBM
// traffic is 1.00 of the bytes.  Short ones are bound by latency: 100 tokens
// take 6 us (launch, length, page, codes, merge), and each further tile of a
// wave 0.8 us, with one wave on a SIMD: 1024 tokens 12.5 us.  A third register
// set, two tiles ahead, was no faster, so it is the tile's own chain (decode,
// scores, maximum, exponentials, decode, outputs).
// Measured and not kept: tiles of 64 tokens (short units wait longer for their
// first), eight waves (0.5 us less for one short sequence, more for the rest),
// 32 rows for each wave (the registers leave one wave on a SIMD), codes to LDS
// by direct loads (the compiler waits for all of them before each read).
template <int D, int NW>
__global__ __launch_bounds__(64 * NW, D == 256 ? 1 : 2) void attn_rows_kernel(AttnArgs a) {
  using G = Geo<D>;
  constexpr int ROWS = 16, TT = G::TT, TG = G::TG;
  constexpr int LD = D + 4;  // padded row of the merge buffer
  __shared__ __align__(16) float mo[NW][16][LD];
  __shared__ float mm[NW][16], ml[NW][16];
  const int lane = threadIdx.x & 63, wave = wave_index();
  if (is_status_group(a, lane, wave)) return;
  uint32_t err = 0u;
  const LaneAt<D> at(lane, a.token_stride);
  Walk<ROWS, TT> walk(a, lane, (int)blockIdx.x - 1);
  Unit u;
  while (walk.next(u)) {
    const int t0 = u.t0, t1 = u.t1;
    // keys that all rows of the tile see
    const int all_lo = uniform(attn_lo(a.sh, u.sq, u.i1)), all_hi = uniform(attn_hi(a.sh, u.sq, u.i0));
    const int ln = opaque(lane), ng = ln >> 4, nn = ln & 15;
    QFrag<D> q;
    RowState<D> st;
    const bool on = nn < u.live;
    const int64_t row = u.r0 + (on ? nn : 0);
    const int i = (int)divide((uint32_t)row, a.by_groups);
    const int qh = u.h * a.sh.groups + (int)(row - (int64_t)i * a.sh.groups);
    load_query<D>(a.q + (u.sq.first + i) * a.q_st + qh * a.q_sh, on, ng, q);
    const int lo = attn_lo(a.sh, u.sq, i), hi = attn_hi(a.sh, u.sq, i);
#pragma unroll
    for (int dt = 0; dt < G::DT; ++dt) st.o[dt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    st.m = kNegInf;
    st.l = 0.0f;

    // the workgroup's tiles, a contiguous part for each wave
    const int nt = t1 - t0;
    const int w0 = t0 + (int)((int64_t)nt * wave / NW), w1 = t0 + (int)((int64_t)nt * (wave + 1) / NW);
    const int64_t head_off = u.h * a.head_stride;
    const int32_t *row_table = a.table + u.b * a.table_stride;
    // lane i holds the offset of the i-th group of 16 tokens of a block of 64 groups, and valid its bit: whether
    // the group has a page (else the offset is that of page 0, whose bytes are masked)
    constexpr int BLOCK = 64 / TG;  // key tiles of it
    auto groups_of = [&](int tile, uint64_t &valid) {
      const int tok = (u.lo + tile) * TT + 16 * lane;  // below 2^30 + 64 * 16
      int id = -1;
      if (tile < w1 && tok < u.keys_hi && tok + 15 >= u.keys_lo) id = page_of(a, row_table, tok, err);
      valid = __ballot(id >= 0);
      return head_off + (int64_t)max(id, 0) * a.page_stride +
             (int64_t)(tok & ((1 << a.log_page) - 1)) * a.token_stride;
    };
    auto fetch = [&](int i, int64_t offs, uint64_t valid, KvTile<D> &t, uint32_t &ok) {  // tile i of a block
      int64_t off[TG];
#pragma unroll
      for (int tg = 0; tg < TG; ++tg) off[tg] = lane_value(offs, i * TG + tg);
      ok = (uint32_t)(valid >> (i * TG)) & ((1u << TG) - 1u);
      load_tile<D>(a, at, off, t);
    };
    if (w0 < w1) {
      int first = w0;
      uint64_t valid, valid_next;
      int64_t offs = groups_of(first, valid), offs_next = groups_of(first + BLOCK, valid_next);
      KvTile<D> even, odd;
      uint32_t ok_even, ok_odd = 0u;
      fetch(0, offs, valid, even, ok_even);
      auto step = [&](int tile, const KvTile<D> &cur, uint32_t ok, KvTile<D> &nxt, uint32_t &ok_next) {
        if (tile + 1 < w1) {
          if (tile + 1 == first + BLOCK) {
            first += BLOCK;
            offs = offs_next;
            valid = valid_next;
            offs_next = groups_of(first + BLOCK, valid_next);
          }
          fetch(tile + 1 - first, offs, valid, nxt, ok_next);
        }
        const int token0 = (u.lo + tile) * TT;
        const bool full = ok == (1u << TG) - 1u && token0 >= all_lo && token0 + TT <= all_hi;
        consume_tile<D>(a, cur, q, lo, hi, token0, full, ok, u.keys_lo, u.keys_hi, lane, st);
      };
      for (int tile = w0; tile < w1; tile += 2) {
        step(tile, even, ok_even, odd, ok_odd);
        if (tile + 1 < w1) step(tile + 1, odd, ok_odd, even, ok_even);
      }
    }

    // merge the waves, 16 rows at a time
    const int mt = opaque((int)threadIdx.x), mn = mt & 15, mg = (mt >> 4) & 3;
    float l = st.l;
    l += xor16(l);
    l += xor32(l);
    if (mg == 0) {
      mm[wave][mn] = st.m;
      ml[wave][mn] = l;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int dt = 0; dt < G::DT; dt += 4)
        *reinterpret_cast<f32x4 *>(&mo[wave][mn][(4 * mg + i) * G::DT + dt]) =
            f32x4{st.o[dt][i], st.o[dt + 1][i], st.o[dt + 2][i], st.o[dt + 3][i]};
    __syncthreads();
    // 8 elements of a row a thread
    for (int e = mt; e < 16 * D / 8; e += 64 * NW) {
      const int row = e / (D / 8), d = e % (D / 8) * 8;
      if (row >= u.live) continue;
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
      if (u.whole) {
        const float inv = row_factor(sum);
        const int64_t head = out_row(a, u.sq.first, u.h, u.r0 + row);
        u32x4 w;
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = pack_bf16(o[2 * k] * inv, o[2 * k + 1] * inv);
        *reinterpret_cast<u32x4 *>(a.out + head * D + d) = w;
        if (a.lse && d == 0) a.lse[head] = row_lse(top, sum);
      } else {
        using P = Part<D, ROWS>;
        const int64_t slot = 2 * (int64_t)(blockIdx.x - 1) + (t0 == 0 ? 1 : 0);
        float *po = P::o(a.parts, slot) + row * D + d;
        *reinterpret_cast<f32x4 *>(po) = f32x4{o[0], o[1], o[2], o[3]};
        *reinterpret_cast<f32x4 *>(po + 4) = f32x4{o[4], o[5], o[6], o[7]};
        if (d == 0) {
          P::m(a.parts, slot)[row] = top;
          P::l(a.parts, slot)[row] = sum;
        }
      }
    }
    __syncthreads();
  }
  walk.finish();
  if (__builtin_expect(err != 0u, 0)) Status{a.status, a.first}.report(err);
}

// ------------------------------------------------------------ prompts ----
// Many rows: a workgroup of NW waves takes 32 NW rows, a wave 32 of them, and
// the workgroup's waves share the key tiles (64 tokens) through LDS.  Scores
// and outputs run on v_mfma_f32_32x32x16_bf16 in the transposed form, S^T =
// K Q^T and O^T += V^T P^T: a lane's score registers are one query row's, so
// the softmax needs one exchange, and they are P^T's operand as they lie.
//  * Keys stay FP4 in LDS (a quarter of the reads); a lane decodes its own
//    operand.  Key tile row m is token 16 (m / 16) + 8 (m / 4 % 2) + 4 (m / 8
//    % 2) + m % 4, so that score register i of lane half h is token 16 (i / 8)
//    + 8 h + i % 8: eight consecutive tokens for each step of the second
//    product.
//  * Values are decoded once for all waves and written transposed, [element]
//    [token] bfloat16, 8 tokens (16 bytes) an operand.  Operand row m is
//    element 16 (m / 4 % 2) + 4 (m / 8) + m % 4 of 32, so that a lane ends with
//    16 consecutive elements of its row.
// 16-byte pieces of both are swizzled so that 16 lanes that read or write
// together fall on different banks.
// 4096 new tokens on 8192 keys (32 query heads on 8, 128 wide; 412 GFLOP)
// take 385 to 430 us, as the clock allows: 0.96 to 1.07 PFLOP/s, 69 to 77% of
// what a large bfloat16 matrix product of the vendor's library reaches (1.38).  The vector pipe (key
// decoding, exponentials) is busy 70% of the cycles and the matrix cores 48%,
// at a clock that the load lowers to 1.7 - 2.1 GHz.  Measured and not kept:
// 64 rows for each wave (620 us against 505: one wave on a SIMD), a fixed
// interleaving of the two pipes' instructions (4% slower), wave priorities
// (slower), a SIMD's two waves held in opposite phases, vector work of one
// beside matrix work of the other, by four barriers a tile (525 us against
// 418), values staged by all eight waves in pieces of half the size (461).
template <int D>
struct PromptGeo {
  static constexpr int TT = 64;
  static constexpr int RB = D / 2;    // code bytes of a row
  static constexpr int GR = D / 32;   // its pieces of 16 bytes, one scale block each
  static constexpr int HG = GR / 2;   // pieces of a lane half
  static constexpr int DT = D / 32;   // output tiles
  static constexpr int ITEMS = 2 * D; // staging work: (row, piece) of keys, and (4 tokens, 8 elements) of values
  // bytes of a buffer: keys, key scales, values
  static constexpr int KS = TT * RB, V = KS + TT * GR, BUF = V + D * TT * 2;
  static __device__ int key_piece(int row, int piece) { return piece ^ ((row / (8 / HG)) & (GR - 1)); }
  static __device__ int value_swizzle(int d) {
    return (((d >> 1) & 3) ^ (((d >> 3) & 1) | ((d >> 4) & 2))) | ((d >> 2) & 4);
  }
};

// Where a thread's staging items lie: offsets from their group of 16 tokens
// in memory, and in a buffer.  Item x of thread t is number t + x threads:
// piece item % GR of key row item / GR, and elements 8 (item % (D / 8)) .. of
// the four tokens from 4 (item / (D / 8)) on.
template <int D>
struct StageAt {
  using G = PromptGeo<D>;
  uint32_t k, ks, v, vs;
  uint32_t to_k, to_ks, to_v, v_piece;
  __device__ StageAt(int tid, int64_t token_stride) {
    const uint32_t ts = (uint32_t)token_stride;
    // within the wave's rows, or the lane's group of 16 where the wave has two
    const int in = tid % (64 < 16 * G::GR ? 64 : 16 * G::GR);
    k = in / G::GR * ts + in % G::GR * 16;
    ks = in / G::GR * (ts / 16) + in % G::GR;
    const int e8 = tid % (D / 8), t4 = tid / (D / 8), iv = tid % (64 < 4 * (D / 8) ? 64 : 4 * (D / 8));
    v = 4 * (iv / (D / 8)) * ts + e8 * 4;
    vs = 4 * (iv / (D / 8)) * (ts / 16) + e8 / 4;
    const int row = tid / G::GR;
    to_k = row * G::RB + G::key_piece(row, tid % G::GR) * 16;
    to_ks = G::KS + tid;
    to_v = G::V + e8 * 8 * (G::TT * 2) + (t4 & 1) * 8;
    v_piece = (t4 >> 1) ^ G::value_swizzle(e8 * 8);  // of the item's first element; (e / 2) flips its low bits
  }
};

template <int D, int NW>
__global__ __launch_bounds__(64 * NW, D == 256 ? 1 : 2) void attn_prompt_kernel(AttnArgs a) {
  using G = PromptGeo<D>;
  constexpr int TT = G::TT, M = 32 * NW, THREADS = 64 * NW;
  constexpr int PT = (G::ITEMS + THREADS - 1) / THREADS;  // staging items of a thread
  __shared__ __align__(16) uint8_t smem[3 * G::BUF];
  const int lane = threadIdx.x & 63, wave = wave_index(), n = lane & 31, hh = lane >> 5;
  if (is_status_group(a, lane, wave)) return;
  uint32_t err = 0u;
  // the sign of the scale goes into the queries; never zero, since a masked score times zero would be NaN: the least
  // float32 moves no finite score by 2^-20
  const float c = fmaxf(fabsf(a.scale_log2), as_f(1u));
  const uint32_t flip = a.scale_log2 < 0.0f ? 0x80008000u : 0u;
  const float slack = 8.0f / fmaxf(c, 1e-30f);  // finite; a tiny scale moves the maximum at less than 2^8
  // the lane's places in a buffer
  const int kt = 16 * (n >> 4) + 8 * ((n >> 2) & 1) + 4 * ((n >> 3) & 1) + (n & 3);
  const int vd = 16 * ((n >> 2) & 1) + 4 * (n >> 3) + (n & 3);
  const int v_piece = hh ^ G::value_swizzle(vd);
  const StageAt<D> at(threadIdx.x, a.token_stride);

  Walk<M, TT> walk(a, lane, (int)blockIdx.x - 1);
  Unit u;
  while (walk.next(u)) {
    // key tiles that the row tile's own rows see
    const int see_lo = attn_lo(a.sh, u.sq, u.i0) / TT, see_hi = (attn_hi(a.sh, u.sq, u.i1) + TT - 1) / TT;
    const int tb = uniform(max(u.lo + u.t0, see_lo)), te = uniform(min(u.lo + u.t1, see_hi));
    const int w_rows = u.live - 32 * wave;  // of the wave: 32 or fewer, none where it is not positive
    const int j0 = uniform((int)divide((uint32_t)(u.r0 + (w_rows > 0 ? 32 * wave : 0)), a.by_groups));
    const int j1 = uniform(
        (int)divide((uint32_t)(u.r0 + (w_rows > 0 ? 32 * wave + min(w_rows, 32) - 1 : 0)), a.by_groups));
    const int all_lo = uniform(attn_lo(a.sh, u.sq, j1)), all_hi = uniform(attn_hi(a.sh, u.sq, j0));

    u32x4 q[G::HG * 4];
    f32x16 o[G::DT];
    float m, l;
    const bool on = n < w_rows;
    const int64_t row = u.r0 + (on ? 32 * wave + n : 0);
    const int i = (int)divide((uint32_t)row, a.by_groups);
    const int lo = attn_lo(a.sh, u.sq, i), hi = attn_hi(a.sh, u.sq, i);
    const uint16_t *qp =
        a.q + (u.sq.first + i) * a.q_st + (u.h * a.sh.groups + (row - (int64_t)i * a.sh.groups)) * a.q_sh;
#pragma unroll
    for (int x = 0; x < G::HG * 4; ++x) {
      q[x] = u32x4{0u, 0u, 0u, 0u};
      if (on) q[x] = *reinterpret_cast<const u32x4 *>(qp + hh * (D / 2) + 8 * x);
      q[x] ^= flip;
    }
#pragma unroll
    for (int dt = 0; dt < G::DT; ++dt)
#pragma unroll
      for (int x = 0; x < 16; ++x) o[dt][x] = 0.0f;
    m = kNegInf;
    l = 0.0f;

    const int64_t head_off = u.h * a.head_stride;
    const int32_t *row_table = a.table + u.b * a.table_stride;
    auto pages_of = [&](int tile) {  // lane i: the page of the i-th group of 16 tokens from the tile on; -1: none
      const int tok = tile * TT + 16 * lane;
      int id = -1;
      if (tile < te && tok < u.keys_hi && tok + 15 >= u.keys_lo) id = page_of(a, row_table, tok, err);
      return id;
    };

    // a tile's bytes on their way from memory to LDS
    u32x4 kr[PT];
    uint32_t kb[PT], vr[PT][4], vb[PT][4], ok_next = 0u;
    auto fetch = [&](int tile, int ids, int first) {
      const uint64_t bad = __ballot(ids < 0);
      ok_next = ~(uint32_t)(bad >> (4 * (tile - first))) & 15u;
      if (G::ITEMS < THREADS && 64 * wave >= G::ITEMS) return;
#pragma unroll
      for (int x = 0; x < PT; ++x) {
        // the wave's 64 items of keys are 64 / GR rows, those of values as many tokens: part of one group of 16
        // tokens, or (head_dim 64) two groups
        auto group_off = [&](int g) {
          const int id = __builtin_amdgcn_readlane(ids, 4 * (tile - first) + g);
          return head_off + (int64_t)max(id, 0) * a.page_stride +
                 ((tile * TT + 16 * g) & ((1 << a.log_page) - 1)) * a.token_stride;
        };
        const int row0 = (x * THREADS + 64 * wave) / G::GR;
        int64_t off = group_off(row0 / 16) + (row0 % 16) * a.token_stride;
        if constexpr (D == 64) {
          const int64_t other = group_off(row0 / 16 + 1);
          off = lane < 32 ? off : other;
        }
        const uint8_t *kc = a.kc + off, *ks = a.ks + (off >> 4), *vc = a.vc + off, *vs = a.vs + (off >> 4);
        const uint32_t k_at = opaque(at.k), ks_at = opaque(at.ks), v_at = opaque(at.v), vs_at = opaque(at.vs);
        kr[x] = *reinterpret_cast<const u32x4 *>(kc + k_at);
        kb[x] = ks[ks_at];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          vr[x][j] = *reinterpret_cast<const uint32_t *>((vc + j * a.token_stride) + v_at);
          vb[x][j] = (vs + j * (a.token_stride >> 4))[vs_at];
        }
      }
    };
    auto store = [&](int tile, uint8_t *buf, uint32_t ok) {
      if (G::ITEMS < THREADS && 64 * wave >= G::ITEMS) return;
      const bool inside = ok == 15u && tile * TT >= u.keys_lo && tile * TT + TT <= u.keys_hi;
#pragma unroll
      for (int x = 0; x < PT; ++x) {
        *reinterpret_cast<u32x4 *>(buf + at.to_k + x * (THREADS * 16)) = kr[x];
        buf[at.to_ks + x * THREADS] = (uint8_t)kb[x];
        float sc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[j] = as_f(vb[x][j] << 23);
        constexpr int T4X = THREADS / (D / 8);  // groups of 4 tokens from one x to the next
        if (!inside) {  // what lies outside every row's keys must not reach a product, where 0 * NaN is NaN
          not_speculated();
          const int t4 = x * T4X + threadIdx.x / (D / 8);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int tok = tile * TT + 4 * t4 + j;
            if (!((tok >= u.keys_lo) & (tok < u.keys_hi) & ((ok >> (t4 / 4)) & 1u))) {
              vr[x][j] = 0u;
              sc[j] = 1.0f;
            }
          }
        }
#pragma unroll
        for (int e2 = 0; e2 < 4; ++e2) {  // elements 2 e2 and 2 e2 + 1 of the item's 8
          uint32_t y[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            y[j] = e2 == 0   ? fp4x2_to_bf16<0>(vr[x][j], sc[j])
                   : e2 == 1 ? fp4x2_to_bf16<1>(vr[x][j], sc[j])
                   : e2 == 2 ? fp4x2_to_bf16<2>(vr[x][j], sc[j])
                             : fp4x2_to_bf16<3>(vr[x][j], sc[j]);
          // pieces of 8 tokens; from one x to the next the piece moves by a power of two that the swizzle leaves
          // alone when it is added by an exclusive or
          const uint32_t piece = at.v_piece ^ (uint32_t)((x * T4X / 2) ^ e2);
          uint8_t *vp = buf + at.to_v + piece * 16;
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const uint32_t sel = p ? 0x07060302u : 0x05040100u;
            *reinterpret_cast<u32x2 *>(vp + (2 * e2 + p) * (TT * 2)) =
                u32x2{__builtin_amdgcn_perm(y[1], y[0], sel), __builtin_amdgcn_perm(y[3], y[2], sel)};
          }
        }
      }
    };

    // key operands of 32 tokens of a tile, still FP4
    u32x4 kc[G::HG];
    float ks[G::HG];
    auto load_keys = [&](const uint8_t *buf, int sub) {
      const int kr_row = 32 * sub + kt;
#pragma unroll
      for (int p = 0; p < G::HG; ++p) {
        const int piece = hh * G::HG + p;
        kc[p] = *reinterpret_cast<const u32x4 *>(buf + kr_row * G::RB + G::key_piece(kr_row, piece) * 16);
        ks[p] = as_f((uint32_t)buf[G::KS + kr_row * G::GR + piece] << 23);
      }
    };
    // their scores
    auto scores = [&](f32x16 &s) {
      #pragma unroll
        for (int x = 0; x < 16; ++x) s[x] = 0.0f;
#pragma unroll
      for (int p = 0; p < G::HG; ++p)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const bf16x8 kv = fp4x8_to_bf16(kc[p][w], ks[p]);
          s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kv, __builtin_bit_cast(bf16x8, q[4 * p + w]), s, 0, 0, 0);
        }
    };
    // value operands of 16 tokens of a tile
    u32x4 vv[G::DT];
    auto load_values = [&](const uint8_t *buf, int st) {
#pragma unroll
      for (int dt = 0; dt < G::DT; ++dt) {
        // the swizzle of element vd + 32 dt is vd's with bit 1 flipped where dt is odd
        const int piece = v_piece ^ (2 * st) ^ (2 * (dt & 1));
        vv[dt] = *reinterpret_cast<const u32x4 *>(buf + G::V + (vd + 32 * dt) * (TT * 2) + piece * 16);
      }
    };
    // masks them and keeps the running maximum
    auto settle = [&](int token0, uint32_t ok, f32x16 &s) {
      if (!(ok == 3u && token0 >= all_lo && token0 + 32 <= all_hi)) {
        not_speculated();
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const int tok = token0 + 16 * (x / 8) + 8 * hh + x % 8;
          s[x] = (tok >= lo) & (tok < hi) & ((ok >> (x / 8)) & 1u) ? s[x] : kNegInf;
        }
      }
      float mx = s[0];
#pragma unroll
      for (int x = 1; x < 16; ++x) mx = fmaxf(mx, s[x]);
      // the running maximum moves only when a score passes it by more than 2^8 (see consume_tile)
      if (__ballot(mx > m + slack)) {
        const float top = fmaxf(m, fmaxf(mx, xor32(mx)));
        const float shrink = m == kNegInf ? 0.0f : __builtin_amdgcn_exp2f((m - top) * c);
        m = top;
        l *= shrink;
#pragma unroll
        for (int dt = 0; dt < G::DT; ++dt)
#pragma unroll
          for (int x = 0; x < 16; ++x) o[dt][x] *= shrink;
      }
    };
    // their part of the output; the first 16 tokens' value operands are loaded
    auto outputs = [&](const uint8_t *buf, int sub, f32x16 &s) {
      const float ref = m == kNegInf ? 0.0f : m * c;
#pragma unroll
      for (int st = 0; st < 2; ++st) {  // 16 tokens each
        u32x4 pw;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          s[8 * st + x] = __builtin_amdgcn_exp2f(fmaf(s[8 * st + x], c, -ref));
          l += s[8 * st + x];
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) pw[x] = pack_bf16(s[8 * st + 2 * x], s[8 * st + 2 * x + 1]);
        const bf16x8 pv = __builtin_bit_cast(bf16x8, pw);
        if (st == 1) load_values(buf, 2 * sub + 1);
#pragma unroll
        for (int dt = 0; dt < G::DT; ++dt)
          o[dt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, vv[dt]), pv, o[dt], 0, 0, 0);
      }
    };

    if (tb < te) {
      int first = tb;
      int ids = pages_of(first), ids_next = pages_of(first + 16);
      auto fetch_next = [&](int tile) {
        if (tile == first + 16) {
          first += 16;
          ids = ids_next;
          ids_next = pages_of(first + 16);
        }
        fetch(tile, ids, first);
      };
      // Three buffers: while a tile's scores of 32 tokens turn into probabilities and outputs, the matrix cores run
      // the scores of the next 32, which for a tile's second half are the next tile's first.
      fetch(tb, ids, first);
      uint32_t ok_cur = ok_next;
      store(tb, smem, ok_cur);
      if (tb + 1 < te) fetch_next(tb + 1);
      __syncthreads();
      f32x16 s0, s1;
      load_keys(smem, 0);
      scores(s0);
      int at_cur = 0, at_nxt = G::BUF;
      for (int tile = tb; tile < te; ++tile) {
        const uint32_t ok_tile = ok_next;
        if (tile + 1 < te) store(tile + 1, smem + at_nxt, ok_tile);
        if (tile + 2 < te) fetch_next(tile + 2);
        load_keys(smem + at_cur, 1);
        load_values(smem + at_cur, 0);
        settle(tile * TT, ok_cur & 3u, s0);
        scores(s1);
        outputs(smem + at_cur, 0, s0);
        __syncthreads();
        load_keys(smem + at_nxt, 0);  // past the last tile: whatever is there, not used
        load_values(smem + at_cur, 2);
        settle(tile * TT + 32, ok_cur >> 2, s1);
        scores(s0);
        outputs(smem + at_cur, 1, s1);
        ok_cur = ok_tile;
        at_cur = at_nxt;
        at_nxt = at_nxt == 2 * G::BUF ? 0 : at_nxt + G::BUF;
      }
      __syncthreads();  // the buffers are free for the next unit
    }

    const float sum = l + xor32(l);
    const float top = m == kNegInf ? kNegInf : m * c;
    const int pr = 32 * wave + n;  // row of the tile
    if (pr < u.live && u.whole) {
      const float inv = row_factor(sum);
      const int64_t head = out_row(a, u.sq.first, u.h, u.r0 + pr);
#pragma unroll
      for (int dt = 0; dt < G::DT; ++dt) {
        u32x4 w[2];
#pragma unroll
        for (int x = 0; x < 8; ++x) w[x >> 2][x & 3] = pack_bf16(o[dt][2 * x] * inv, o[dt][2 * x + 1] * inv);
        u32x4 *p = reinterpret_cast<u32x4 *>(a.out + head * D + dt * 32 + hh * 16);
        p[0] = w[0];
        p[1] = w[1];
      }
      if (a.lse && hh == 0) a.lse[head] = row_lse(top, sum);
    } else if (pr < u.live) {
      using P = Part<D, M>;
      const int64_t slot = 2 * (int64_t)(blockIdx.x - 1) + (u.t0 == 0 ? 1 : 0);
#pragma unroll
      for (int dt = 0; dt < G::DT; ++dt)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          *reinterpret_cast<f32x4 *>(P::o(a.parts, slot) + pr * D + dt * 32 + hh * 16 + 4 * x) =
              f32x4{o[dt][4 * x], o[dt][4 * x + 1], o[dt][4 * x + 2], o[dt][4 * x + 3]};
      if (hh == 0) {
        P::m(a.parts, slot)[pr] = top;
        P::l(a.parts, slot)[pr] = sum;
      }
    }
  }
  walk.finish();
  if (__builtin_expect(err != 0u, 0)) Status{a.status, a.first}.report(err);
}

// Joins the partial results of units that several spans share: workgroups
// (w, y) join the rows y, y + gridDim.y, ... of the unit that begins in span w
// and ends in a later one, from span w's second slot and the first slots of
// the spans after it; each wave takes every fourth part, up to eight at a time
// with their loads together.  Bound by latency: 255 spans of rows of 128
// elements (16 rows, 2 MB) take 4.8 us, where a launch alone takes 2.
template <int D, int ROWS>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
  using P = Part<D, ROWS>;
  constexpr int PER = D / 64;  // elements of a lane
  __shared__ float so[4][D];
  __shared__ float sm[4], sl[4];
  const int lane = threadIdx.x & 63, wave = wave_index();
  const int span = blockIdx.x;
  const Join j = a.joins[span];
  const int n = j.last - span + 1;
  for (int row = blockIdx.y; row < j.rows; row += gridDim.y) {
    float m = kNegInf, l = 0.0f, o[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) o[k] = 0.0f;
    auto take = [&](auto count, int base) {
      constexpr int CH = decltype(count)::value;
      float pm[CH], pl[CH], v[CH][PER];
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int part = min(base + 4 * k, n - 1);
        const int64_t slot = 2 * (int64_t)(span + part) + (part == 0 ? 1 : 0);
        pm[k] = base + 4 * k < n ? P::m(a.parts, slot)[row] : kNegInf;
        pl[k] = P::l(a.parts, slot)[row];
        const float *po = P::o(a.parts, slot) + row * D + lane * PER;
#pragma unroll
        for (int e = 0; e < PER; ++e) v[k][e] = po[e];
      }
      float top = m;
#pragma unroll
      for (int k = 0; k < CH; ++k) top = fmaxf(top, pm[k]);
      const float f = part_weight(m, top);
      m = top;
      l *= f;
#pragma unroll
      for (int e = 0; e < PER; ++e) o[e] *= f;
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const float w = part_weight(pm[k], top);
        l = fmaf(pl[k], w, l);
#pragma unroll
        for (int e = 0; e < PER; ++e) o[e] = fmaf(v[k][e], w, o[e]);
      }
    };
    if (n <= 4) {
      if (wave < n) take(std::integral_constant<int, 1>{}, wave);
    } else if (n <= 8) {
      take(std::integral_constant<int, 2>{}, wave);
    } else {
      for (int base = wave; base < n; base += 32) take(std::integral_constant<int, 8>{}, base);
    }
    if (lane == 0) {
      sm[wave] = m;
      sl[wave] = l;
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) so[wave][lane * PER + k] = o[k];
    __syncthreads();
    if (threadIdx.x < D / 2) {
      const float top = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
      float sum = 0.0f, x = 0.0f, y = 0.0f;
      const int d = 2 * threadIdx.x;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = part_weight(sm[w], top);
        sum = fmaf(sl[w], f, sum);
        x = fmaf(so[w][d], f, x);
        y = fmaf(so[w][d + 1], f, y);
      }
      const float inv = row_factor(sum);
      const int64_t head = out_row(a, j.first, j.head, j.row0 + row);
      reinterpret_cast<uint32_t *>(a.out)[(head * D + d) / 2] = pack_bf16(x * inv, y * inv);
      if (a.lse && d == 0) a.lse[head] = row_lse(top, sum);
    }
    __syncthreads();
  }
}

__global__ __launch_bounds__(64) void attn_status_kernel(uint32_t *status) {
  if (threadIdx.x == 0) Status{status, true}.merge(0u);
}

// ------------------------------------------------------------ dispatch ----
bool sizes_ok(int64_t tokens, int64_t batch, int64_t q_heads, int64_t heads, int64_t head_dim, int64_t max_new,
              int64_t max_len) {
  return kv_head_dim_ok(head_dim) && heads >= 1 && heads * head_dim <= 65536 && q_heads >= heads &&
         q_heads <= 65536 && q_heads % heads == 0 && kv_size_ok(tokens, q_heads, head_dim) && batch >= 0 &&
         batch < ((int64_t)1 << 24) && max_new >= 0 && max_new <= tokens && max_len >= 0 &&
         max_len <= ((int64_t)1 << 30);
}

fp4q_status_t hip_status() { return hipGetLastError() == hipSuccess ? FP4Q_OK : FP4Q_ERR_HIP; }

template <int D, int ROWS>
void launch(const AttnArgs &a, const Pass &p, hipStream_t s) {
  const dim3 grid((unsigned)(p.spans ? p.spans : p.units) + 1);
  if constexpr (ROWS >= 128)
    hipLaunchKernelGGL((attn_prompt_kernel<D, ROWS / 32>), grid, dim3(2 * ROWS), 0, s, a);
  else if (p.waves == 4)
    hipLaunchKernelGGL((attn_rows_kernel<D, 4>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((attn_rows_kernel<D, 1>), grid, dim3(64), 0, s, a);
  if constexpr (ROWS < 256) {  // tiles of 256 rows are never split (make_pass)
    if (!p.spans) return;
    const int64_t rows = (int64_t)a.sh.max_new * a.sh.groups;  // no unit has more than its sequence
    hipLaunchKernelGGL((attn_join_kernel<D, ROWS>), dim3((unsigned)p.spans, (unsigned)(rows < 16 ? rows : 16)),
                       dim3(256), 0, s, a);
  }
}

// Bytes that a pass leaves for its joining kernel.
size_t shared_bytes(const Pass &p) { return p.spans * sizeof(Join) + 4 * (size_t)p.part_floats; }

}  // namespace
}  // namespace fp4q

using namespace fp4q;

extern "C" size_t fp4q_attention_mxfp4_workspace_bytes(int64_t tokens, int64_t batch, int64_t q_heads, int64_t heads,
                                                       int64_t head_dim, int64_t max_new, int64_t max_len,
                                                       int64_t window) {
  if (window < 0 || window > 0x7FFFFFFF) return 0;
  if (!sizes_ok(tokens, batch, q_heads, heads, head_dim, max_new, max_len)) return 0;
  const Plan p = make_plan(tokens, batch, q_heads, heads, head_dim, max_new, max_len, window);
  size_t most = 0;  // the passes run one after the other
  for (int i = 0; i < p.passes; ++i) most = shared_bytes(p.pass[i]) > most ? shared_bytes(p.pass[i]) : most;
  return kAttnHeader + most;
}

extern "C" fp4q_status_t fp4q_attention_mxfp4(const fp4q_kv_cache_t *cache, const void *q, int64_t q_token_stride,
                                              int64_t q_head_stride, int64_t tokens, int64_t q_heads,
                                              const int32_t *block_table, int64_t table_stride, int64_t table_width,
                                              int64_t batch, const int32_t *seq_lens, const int32_t *cu_q,
                                              int64_t max_new, int64_t max_len, float scale, int causal,
                                              int64_t window, void *out, float *lse, void *workspace,
                                              size_t workspace_bytes, void *stream) {
  const bool empty = tokens == 0 || batch == 0;
  if (!cache || (!empty && (!q || (!block_table && max_len > 0) || !seq_lens || !out))) return FP4Q_ERR_NULL;
  fp4q_status_t st = kv_check_cache(*cache);
  if (st != FP4Q_OK) return st;
  if (!sizes_ok(tokens, batch, q_heads, cache->heads, cache->head_dim, max_new, max_len)) return FP4Q_ERR_SHAPE;
  if (table_width < 0 || table_width > 0x7FFFFFFF || table_stride < table_width ||
      max_len > table_width * cache->page_size || (!cu_q && !empty && tokens != batch))
    return FP4Q_ERR_SHAPE;
  if (!cu_q && !empty && max_new < 1) return FP4Q_ERR_SHAPE;
  // the table's last entry, below 2^60: no byte offset passes 63 bits
  if (!empty && (__int128)table_stride * (batch - 1) + table_width >= ((__int128)1 << 60)) return FP4Q_ERR_SHAPE;
  if ((causal != 0 && causal != 1) || window < 0 || window > 0x7FFFFFFF || !(fabsf(scale) <= 0x1p127f))
    return FP4Q_ERR_ARG;
  if ((st = kv_check_heads(FP4Q_BF16, tokens, q_heads, cache->head_dim, q_token_stride, q_head_stride, q)) != FP4Q_OK)
    return st;
  if (!empty && (!kv_aligned(out, 16) || !kv_aligned(lse, 4) || !kv_aligned(block_table, 4) ||
                 !kv_aligned(seq_lens, 4) || !kv_aligned(cu_q, 4)))
    return FP4Q_ERR_ALIGN;
  const size_t need = fp4q_attention_mxfp4_workspace_bytes(tokens, batch, q_heads, cache->heads, cache->head_dim,
                                                           max_new, max_len, window);
  if (!workspace || workspace_bytes < need || !kv_aligned(workspace, 16)) return FP4Q_ERR_WORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  uint32_t *status = (uint32_t *)workspace;
  if (empty) {
    hipLaunchKernelGGL(attn_status_kernel, dim3(1), dim3(64), 0, s, status);
    return hip_status();
  }
  const Plan p = make_plan(tokens, batch, q_heads, cache->heads, cache->head_dim, max_new, max_len, window);
  AttnArgs a;
  a.sh = AttnShape{tokens, (int)batch, (int)(q_heads / cache->heads), cache->heads, (int)max_new, (int)max_len,
                   causal, (int)window};
  a.by_groups = make_divider((uint32_t)a.sh.groups);
  a.by_heads = make_divider((uint32_t)a.sh.heads);
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
  a.first = true;
  a.joins = (Join *)((char *)workspace + kAttnHeader);
  for (int i = 0; i < p.passes; ++i) {
    const Pass &pass = p.pass[i];
    // without cu_q every sequence has the rows of one token, and one pass serves them all
    if (!cu_q && (a.sh.groups < pass.min_rows || a.sh.groups > pass.max_rows)) continue;
    a.sh.min_rows = pass.min_rows;
    a.sh.max_rows = pass.max_rows;
    a.spans = pass.spans;
    a.parts = (float *)(a.joins + pass.spans);
    auto go = [&](auto dc) {
      constexpr int D = decltype(dc)::value;
      if (pass.rows == 16) launch<D, 16>(a, pass, s);
      else if (pass.rows == 128) launch<D, 128>(a, pass, s);
      else if constexpr (D != 256) launch<D, 256>(a, pass, s);
    };
    if (cache->head_dim == 64) go(std::integral_constant<int, 64>{});
    else if (cache->head_dim == 128) go(std::integral_constant<int, 128>{});
    else go(std::integral_constant<int, 256>{});
    a.first = false;
  }
  return hip_status();
}
