// Heads of queries, keys and values on their way to and from an MXFP4
// key/value cache (include/fp4q_kv.h): norm and rotation of heads, append
// into page slots, and the decoded rows of slots.
//
// Work decomposition: a lane owns 8 contiguous elements of a head, a head
// is head_dim / 8 adjacent lanes, so every load and store of a wave is
// contiguous over its heads (16 bytes a lane for bfloat16) and one token of
// one head is already work for 16 lanes.  Nothing is read twice from memory:
// the element a rotation pairs with comes from the same cache lines, loaded
// again by the lane that needs it.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "fp4q.h"
#include "fp4q_device.h"
#include "fp4q_kv.h"
#include "fp4q_kv_host.h"

namespace fp4q {
namespace {

constexpr int kChunk = 8;  // elements of a lane

struct HeadMap {
  const float *weight;
  double eps;
  const int64_t *positions;
  const float *table;
  int64_t n_positions;
  int rotary, interleaved, hadamard;
};

// n * stride for a non-negative 32-bit n: a product of 32 by 64 bits.
__device__ __forceinline__ int64_t times(int n, int64_t stride) {
  return (int64_t)((uint64_t)(uint32_t)n * (uint64_t)stride);
}

__device__ __forceinline__ void load8(const uint16_t *p, float z[8]) {
  const u32x4 w = *reinterpret_cast<const u32x4 *>(p);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    z[2 * k] = as_f(w[k] << 16);
    z[2 * k + 1] = as_f(w[k] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const float *p, float z[8]) {
  const f32x4 *q = reinterpret_cast<const f32x4 *>(p);
  const f32x4 a = q[0], b = q[1];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    z[k] = a[k];
    z[4 + k] = b[k];
  }
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void store8(uint16_t *p, const float z[8]) {  // to nearest, ties to even
  u32x4 w;
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)z[2 * k], (__bf16)z[2 * k + 1]});
  __builtin_nontemporal_store(w, reinterpret_cast<u32x4 *>(p));
}
__device__ __forceinline__ void store8(float *p, const float z[8]) {
  f32x4 *q = reinterpret_cast<f32x4 *>(p);
  q[0] = f32x4{z[0], z[1], z[2], z[3]};
  q[1] = f32x4{z[4], z[5], z[6], z[7]};
}

// Value of lane l ^ M of the wave, M a power of two up to 16.
template <int M>
__device__ __forceinline__ float lane_xor(float v) {
  if constexpr (M <= 4) return xor_lane<M>(v);
  else if constexpr (M == 8)  // 8 places round within the row of 16
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x128, 0xF, 0xF, true));
  else return __int_as_float(__builtin_amdgcn_ds_swizzle(__float_as_int(v), 0x401F));  // and 0x1F, xor 16
}
template <int M>
__device__ __forceinline__ double lane_xor(double v) {
  const uint64_t b = __double_as_longlong(v);
  const uint32_t lo = as_u(lane_xor<M>(as_f((uint32_t)b))), hi = as_u(lane_xor<M>(as_f((uint32_t)(b >> 32))));
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}

// One stage of the block Hadamard over lanes l and l ^ M.
template <int M>
__device__ __forceinline__ void hadamard_lanes(float z[8], int lane) {
  const uint32_t flip = lane & M ? 0x80000000u : 0u;  // the upper lane takes o - z, which is o + -z
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = lane_xor<M>(z[i]) + as_f(as_u(z[i]) ^ flip);
}

// fp4q_block_hadamard's stages on a lane's 8 elements: h = 1, 2, 4 inside
// the lane, then lanes 1, 2, 4 and 8 apart.  n is the same in every lane.
__device__ __forceinline__ void hadamard8(float z[8], int n, int lane) {
#pragma unroll
  for (int h = 1; h < 8; h <<= 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if ((i & h) == 0) {
        const float a = z[i], b = z[i + h];
        z[i] = a + b;
        z[i + h] = a - b;
      }
    }
  }
  hadamard_lanes<1>(z, lane);
  if (n >= 32) hadamard_lanes<2>(z, lane);
  if (n >= 64) hadamard_lanes<4>(z, lane);
  if (n >= 128) hadamard_lanes<8>(z, lane);
  const float c = n == 16 ? hadamard_scale<16>()
                          : (n == 32 ? hadamard_scale<32>() : (n == 64 ? hadamard_scale<64>() : hadamard_scale<128>()));
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = z[i] * c;
}

// What a lane loads of a head: its 8 elements (chunk c) and, where the head
// is rotated in halves, the 8 that they are paired with; and where its angles
// are.
struct HeadLoad {
  float z[8], p[8];
  int64_t pos;
};

// x is a row of the input in every lane: a lane without a head of its own
// loads the first row, which nobody uses.
template <typename T>
__device__ __forceinline__ void load_head(const T *x, int c, int64_t token, const HeadMap &m, HeadLoad &h) {
  const int half = m.rotary / 2, at = c * kChunk;
  if (m.table) {
    h.pos = m.positions[token];
    // lanes beyond the rotated elements load their own again
    if (!m.interleaved) load8(x + (at >= m.rotary ? at : (at < half ? at + half : at - half)), h.p);
  }
  load8(x + at, h.z);
}

// 1 / sqrt(v) in float64: the hardware's estimate (to 2^-23 at least) and two
// Newton steps, each of which squares the error.
__device__ __forceinline__ double rsqrt64(double v) {
  double y = __builtin_amdgcn_rsq(v);
  const double half = 0.5 * v;
#pragma unroll
  for (int k = 0; k < 2; ++k) y = fma(y, fma(-half * y, y, 0.5), y);
  return v < __builtin_inf() ? y : 1.0 / sqrt(v);
}

// The lane's 8 elements of a loaded head after the map.  Every lane of a head
// calls this together; counts: whether a bad position is an error.  The sum of
// squares is kept in float64, where the square of a float32 is exact and 256
// of them lose at most 2^-45 of the sum, so r does not depend on the order
// in which lanes add.
template <int D>
__device__ __forceinline__ void map_head(HeadLoad &h, int c, int lane, bool counts, const HeadMap &m, uint32_t &err) {
  const int half = m.rotary / 2, at = c * kChunk;
  const bool turned = m.table != nullptr && at < m.rotary;
  const bool first = at < half, paired = turned && !m.interleaved;
  float(&z)[8] = h.z;
  float(&p)[8] = h.p;
  float cs[8], sn[8];
  if (turned) {
    int64_t pos = h.pos;
    if (pos < 0 || pos >= m.n_positions) {
      if (counts) err |= FP4Q_DATA_BAD_POSITION;
      pos = 0;
    }
    const float *row = m.table + pos * m.rotary;
    if (m.interleaved) {
      const f32x4 a = *reinterpret_cast<const f32x4 *>(row + at / 2);
      const f32x4 b = *reinterpret_cast<const f32x4 *>(row + half + at / 2);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        cs[i] = a[i];
        sn[i] = b[i];
      }
    } else {
      const int k = first ? at : at - half;
      load8(row + k, cs);
      load8(row + half + k, sn);
    }
  }
  if (m.weight) {
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += (double)z[i] * (double)z[i];
    s += lane_xor<1>(s);
    s += lane_xor<2>(s);
    s += lane_xor<4>(s);
    if constexpr (D >= 128) s += lane_xor<8>(s);
    if constexpr (D >= 256) s += lane_xor<16>(s);
    const float r = (float)rsqrt64(s * (1.0 / D) + m.eps);
    float w[8];
    load8(m.weight + at, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = (z[i] * r) * w[i];
    if (paired) {
      load8(m.weight + (first ? at + half : at - half), w);
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = (p[i] * r) * w[i];
    }
  }
  if (turned) {
    if (m.interleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = z[2 * i], b = z[2 * i + 1];
        z[2 * i] = a * cs[i] - b * sn[i];
        z[2 * i + 1] = b * cs[i] + a * sn[i];
      }
    } else {
      const uint32_t flip = first ? 0x80000000u : 0u;  // a c - b s is a c + -b s
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = z[i] * cs[i] + as_f(as_u(p[i]) ^ flip) * sn[i];
    }
  }
  if (m.hadamard) hadamard8(z, m.hadamard, lane);
}

// -------------------------------------------------------- rotate_heads ----
// Per head: z = x r w with r = 1 / sqrt(mean x^2 + eps), pairs (a, b) turned
// to (a c - b s, b c + a s), groups of n multiplied by H_n / sqrt(n).  Bound by
// the bytes for long inputs: 8192 tokens of 32 heads of 128 in float32 (268 MB)
// take 45 us, 6.0 TB/s (part of it from the last level cache), bfloat16 26 us;
// one token takes 2.7 us, a launch.
// float32 results are stored through the cache: a lane's 32 bytes are two
// stores, and streamed past it they were written 16% more than once (48.5 us
// with two heads a thread, 54 with one).
template <typename T, typename OutT, int D>
__global__ __launch_bounds__(kThreads) void rotate_heads_kernel(const T *x, int units, Divider heads, int64_t st,
                                                                 int64_t sh, HeadMap m, OutT *out,
                                                                 uint32_t *status) {
  constexpr int LPH = D / kChunk;
  const int lane = threadIdx.x & 63, c = threadIdx.x % LPH;
  const int64_t u = (int64_t)blockIdx.x * (kThreads / LPH) + threadIdx.x / LPH;
  const bool active = u < units;
  const int token = active ? (int)divide((uint32_t)u, heads) : 0;
  const int h = active ? (int)u - token * (int)heads.d : 0;
  uint32_t err = 0u;
  HeadLoad l;
  load_head(x + times(token, st) + times(h, sh), c, token, m, l);
  map_head<D>(l, c, lane, active, m, err);
  if (active) store8(out + u * D + c * kChunk, l.z);
  Status{status, true}.finish(err);
}

// ----------------------------------------------------------- kv_append ----
struct CacheView {
  uint8_t *codes[2], *scales[2];  // keys, values
  int64_t rows;                   // pages * page_size: slot numbers below it are in the cache
  int log_page;
  int64_t page_stride, head_stride, token_stride;
  // byte offset of a row's codes; its scales are at a sixteenth of it
  __device__ __forceinline__ int64_t at(int64_t slot, int h) const {
    const int page = (int)(slot >> log_page), r = (int)slot & ((1 << log_page) - 1);
    return times(page, page_stride) + times(h, head_stride) + times(r, token_stride);
  }
};

// Value of lane S of the caller's quad.
template <int S>
__device__ __forceinline__ float quad_bcast(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), S * 0x55, 0xF, 0xF, true));
}

// This lane's part of a block's loss chain, continued from acc.
__device__ __forceinline__ float chain8(const float z[8], const float q[8], float V, float acc) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float e = fmaf(-q[i], V, z[i]);
    acc = fmaf(e, e, acc);
  }
  return acc;
}

// fp4q_quantize_mxfp4 of a block of 32 spread over a quad: the base
// exponent from the block's maximum, then the window's exponents in
// ascending order with the loss as one chain in element order, handed from
// lane to lane.  Returns the lane's 8 codes; E is the block's exponent.  Codes
// and E of a block that is not finite mean nothing.
__device__ __forceinline__ uint32_t quantize_quad(const float z[8], int lo, int hi, int &E, bool &finite) {
  uint32_t a = 0u;  // the order of |z|'s bits is the order of |z|, infinities and NaN above
#pragma unroll
  for (int i = 0; i < 8; ++i) a = max(a, as_u(z[i]) & 0x7FFFFFFFu);
  a = max(a, as_u(xor_lane<1>(as_f(a))));
  a = max(a, as_u(xor_lane<2>(as_f(a))));
  finite = a < 0x7F800000u;
  const int eb = mx_base_exponent(as_f(a));
  E = max(-127, eb + lo);
  auto codes_at = [&](int e) {
    const float down = pow2f(-e);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = z[i] * down;
    return cvt_fp4x8(y);
  };
  uint32_t codes = codes_at(E);
  if (lo < hi) {
    float best = __builtin_inff();
    const int top = min(127, eb + hi);
    uint32_t w = codes;
    for (int e = E;;) {
      const float V = pow2f(e);
      float q[8];
      fp4x8_to_f32(w, q);
      float L = quad_bcast<0>(chain8(z, q, V, 0.0f));
      L = quad_bcast<1>(chain8(z, q, V, L));
      L = quad_bcast<2>(chain8(z, q, V, L));
      L = quad_bcast<3>(chain8(z, q, V, L));
      if (L < best) {
        best = L;
        E = e;
        codes = w;
      }
      if (++e > top) break;
      w = codes_at(e);
    }
  }
  return codes;
}

struct AppendArgs {
  const void *src[2];  // keys, values
  int64_t st[2], sh[2];
  const int64_t *slots;
  int units;  // tokens * heads of each
  Divider heads;
  HeadMap m;
  int lo, hi;
  CacheView cache;
  uint32_t *status;
};

// blockIdx.y: keys or values.  8192 tokens of 8 heads of 128, bfloat16, keys
// rotated and put through H_128 (34 + 9 MB and 4 MB of the rotation table), in
// a graph: 15.5 us with one exponent (window 0, 0), 19.3 with two searched (-1, 0),
// 25.1 with four; the bytes alone would take 9.0.  Bound by the vector pipe: 226
// instructions a wave (the mean of keys and values) without a search and 364
// with two exponents, since a loss is a sum in element order and so passes from
// lane to lane.  Of the 226, a lane whose keys are rotated in halves spends some
// on its partner's 8 elements, which it loads (and norms) a second time; without a
// map two exponents take 13.9 us.
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(AppendArgs a) {
  constexpr int LPH = D / kChunk;
  const int kv = blockIdx.y;
  const int lane = threadIdx.x & 63, c = threadIdx.x % LPH;
  const int64_t u = (int64_t)blockIdx.x * (kThreads / LPH) + threadIdx.x / LPH;
  uint32_t err = 0u;
  const bool here = u < a.units;
  const int token = here ? (int)divide((uint32_t)u, a.heads) : 0;
  const int h = here ? (int)u - token * (int)a.heads.d : 0;
  // a skipped token's row is loaded all the same, so that nothing waits for its slot
  const T *x = static_cast<const T *>(a.src[kv]) + times(token, a.st[kv]) + times(h, a.sh[kv]);
  int64_t slot = here ? a.slots[token] : -1;
  HeadLoad l;
  if (kv == 0) load_head(x, c, token, a.m, l);
  else load8(x + c * kChunk, l.z);
  if (slot >= a.cache.rows) {
    err |= FP4Q_DATA_BAD_SLOT;
    slot = -1;
  }
  const bool active = slot >= 0;
  if (kv == 0) map_head<D>(l, c, lane, active, a.m, err);
  const float(&z)[8] = l.z;
  int E;
  bool finite;
  const uint32_t codes = quantize_quad(z, a.lo, a.hi, E, finite);
  if (!finite && active) err |= FP4Q_DATA_NONFINITE_INPUT;
  if (active) {
    const int64_t row = a.cache.at(slot, h);
    *reinterpret_cast<uint32_t *>(a.cache.codes[kv] + row + c * 4) = codes;
    if ((c & 3) == 0) a.cache.scales[kv][row / 16 + c / 4] = (uint8_t)(E + 127);
  }
  const Status st{a.status, true};
  if (__builtin_expect(err != 0u, 0)) st.report(err);
  else if (blockIdx.x == 0 && kv == 0 && threadIdx.x == 0) st.merge(0u);
}

// ------------------------------------------------------------- kv_read ----
// 8192 tokens of 8 heads of 128 to bfloat16 (9 MB read, 34 written): 7.4 us in a
// graph, 8.8 among other kernels (4.9 TB/s; 10.6 with multiplications in place of
// the conversion to bfloat16); to float32 (67 MB written) 17 us, 4.5 TB/s.
template <typename OutT, int D>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(CacheView cache, const int64_t *__restrict__ slots,
                                                            int units, Divider heads, OutT *k_out, OutT *v_out,
                                                            uint32_t *status) {
  constexpr int LPH = D / kChunk;
  const int kv = blockIdx.y;
  OutT *out = kv ? v_out : k_out;
  const int c = threadIdx.x % LPH;
  const int64_t u = (int64_t)blockIdx.x * (kThreads / LPH) + threadIdx.x / LPH;
  uint32_t err = 0u;
  if (u < units) {
    const int token = (int)divide((uint32_t)u, heads), h = (int)u - token * (int)heads.d;
    int64_t slot = slots[token];
    if (slot >= cache.rows) {
      err |= FP4Q_DATA_BAD_SLOT;
      slot = -1;
    }
    if (out) {
      float z[8];
      u32x4 raw = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = 0.0f;
      if (slot >= 0) {
        const int64_t row = cache.at(slot, h);
        const uint32_t w = *reinterpret_cast<const uint32_t *>(cache.codes[kv] + row + c * 4);
        const uint32_t b = cache.scales[kv][row / 16 + c / 4];
        const float s = b == 255u ? __builtin_nanf("") : pow2f((int)b - 127);
        if constexpr (sizeof(OutT) == 2) {  // the conversion takes b in the exponent bits of its scale
          const float e = as_f(b << 23);
          raw = u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, e, 0)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, e, 1)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, e, 2)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, e, 3))};
        } else {
          fp4x8_to_f32(w, z);
#pragma unroll
          for (int i = 0; i < 8; ++i) z[i] = z[i] * s;
        }
      }
      OutT *to = out + u * D + c * kChunk;
      if constexpr (sizeof(OutT) == 2) __builtin_nontemporal_store(raw, reinterpret_cast<u32x4 *>(to));
      else store8(to, z);
    }
  }
  const Status st{status, true};
  if (__builtin_expect(err != 0u, 0)) st.report(err);
  else if (blockIdx.x == 0 && kv == 0 && threadIdx.x == 0) st.merge(0u);
}

// The only kernel of a call without tokens: takes the status slot.
__global__ __launch_bounds__(64) void kv_status_kernel(uint32_t *status) {
  if (threadIdx.x == 0) Status{status, true}.merge(0u);
}

// ------------------------------------------------------------ dispatch ----
template <typename F>
void with_dim(int64_t d, F &&f) {
  if (d == 64) f(std::integral_constant<int, 64>{});
  else if (d == 128) f(std::integral_constant<int, 128>{});
  else f(std::integral_constant<int, 256>{});
}
template <typename F>
void with_type(fp4q_dtype_t t, F &&f) {
  if (t == FP4Q_BF16) f((uint16_t *)nullptr);
  else f((float *)nullptr);
}

fp4q_status_t hip_status() { return hipGetLastError() == hipSuccess ? FP4Q_OK : FP4Q_ERR_HIP; }

HeadMap head_map(const fp4q_head_map_t &m) {
  return HeadMap{m.norm_weight, m.eps, m.positions, m.rotary_dim ? m.table : nullptr, m.table_positions,
                 m.rotary_dim, m.interleaved, m.hadamard_n};
}

CacheView view(const fp4q_kv_cache_t &c) {
  return CacheView{{c.k_codes, c.v_codes}, {c.k_scales, c.v_scales}, c.pages * c.page_size, kv_log2(c.page_size),
                   c.page_stride, c.head_stride, c.token_stride};
}

bool ws_ok(const void *ws, size_t bytes) { return ws && bytes >= kWorkspaceBytes && kv_aligned(ws, 8); }

}  // namespace
}  // namespace fp4q

using namespace fp4q;

extern "C" fp4q_status_t fp4q_rotate_heads(const void *x, fp4q_dtype_t dtype, int64_t tokens, int64_t heads,
                                           int64_t head_dim, int64_t token_stride, int64_t head_stride,
                                           const fp4q_head_map_t *map, fp4q_dtype_t out_dtype, void *out,
                                           void *workspace, size_t workspace_bytes, void *stream) {
  const bool empty = tokens == 0 || heads == 0;
  if (!map || (!empty && (!x || !out))) return FP4Q_ERR_NULL;
  if (!ws_ok(workspace, workspace_bytes)) return FP4Q_ERR_WORKSPACE;
  fp4q_status_t st = kv_check_heads(dtype, tokens, heads, head_dim, token_stride, head_stride, x);
  if (st != FP4Q_OK) return st;
  if (out_dtype != FP4Q_F32 && out_dtype != FP4Q_BF16) return FP4Q_ERR_ARG;
  if ((st = kv_check_map(*map, head_dim, empty)) != FP4Q_OK) return st;
  hipStream_t s = (hipStream_t)stream;
  uint32_t *status = (uint32_t *)((char *)workspace + kWsStatus);
  if (empty) {
    hipLaunchKernelGGL(kv_status_kernel, dim3(1), dim3(64), 0, s, status);
    return hip_status();
  }
  if (!kv_aligned(out, 16)) return FP4Q_ERR_ALIGN;
  const int units = (int)(tokens * heads);
  const HeadMap m = head_map(*map);
  with_dim(head_dim, [&](auto dc) {
    constexpr int D = decltype(dc)::value;
    constexpr int U = kThreads / (D / kChunk);
    with_type(dtype, [&](auto tp) {
      using T = std::remove_pointer_t<decltype(tp)>;
      with_type(out_dtype, [&](auto op) {
        using O = std::remove_pointer_t<decltype(op)>;
        const int64_t groups = ((int64_t)units + U - 1) / U;
        hipLaunchKernelGGL((rotate_heads_kernel<T, O, D>), dim3((unsigned)groups), dim3(kThreads), 0, s, (const T *)x,
                           units, make_divider((uint32_t)heads), token_stride, head_stride, m, (O *)out, status);
      });
    });
  });
  return hip_status();
}

extern "C" fp4q_status_t fp4q_kv_append_mxfp4(const fp4q_kv_cache_t *cache, const void *k, int64_t k_token_stride,
                                              int64_t k_head_stride, const void *v, int64_t v_token_stride,
                                              int64_t v_head_stride, fp4q_dtype_t dtype, int64_t tokens,
                                              const int64_t *slots, const fp4q_head_map_t *map, int off_lo,
                                              int off_hi, void *workspace, size_t workspace_bytes, void *stream) {
  if (!cache || !map || (tokens != 0 && (!k || !v || !slots))) return FP4Q_ERR_NULL;
  if (!ws_ok(workspace, workspace_bytes)) return FP4Q_ERR_WORKSPACE;
  if (off_lo > 0 || off_hi < 0 || off_lo < -16 || off_hi > 16) return FP4Q_ERR_ARG;
  fp4q_status_t st = kv_check_cache(*cache);
  if (st != FP4Q_OK) return st;
  if ((st = kv_check_heads(dtype, tokens, cache->heads, cache->head_dim, k_token_stride, k_head_stride, k)) != FP4Q_OK)
    return st;
  if ((st = kv_check_heads(dtype, tokens, cache->heads, cache->head_dim, v_token_stride, v_head_stride, v)) != FP4Q_OK)
    return st;
  if ((st = kv_check_map(*map, cache->head_dim, tokens == 0)) != FP4Q_OK) return st;
  if (tokens && !kv_aligned(slots, 8)) return FP4Q_ERR_ALIGN;
  hipStream_t s = (hipStream_t)stream;
  uint32_t *status = (uint32_t *)((char *)workspace + kWsStatus);
  if (tokens == 0) {
    hipLaunchKernelGGL(kv_status_kernel, dim3(1), dim3(64), 0, s, status);
    return hip_status();
  }
  const AppendArgs a{{k, v}, {k_token_stride, v_token_stride}, {k_head_stride, v_head_stride}, slots,
                     (int)(tokens * cache->heads), make_divider((uint32_t)cache->heads), head_map(*map), off_lo,
                     off_hi, view(*cache), status};
  with_dim(cache->head_dim, [&](auto dc) {
    constexpr int D = decltype(dc)::value;
    constexpr int U = kThreads / (D / kChunk);
    const dim3 grid((unsigned)(((int64_t)a.units + U - 1) / U), 2);
    with_type(dtype, [&](auto tp) {
      using T = std::remove_pointer_t<decltype(tp)>;
      hipLaunchKernelGGL((kv_append_kernel<T, D>), grid, dim3(kThreads), 0, s, a);
    });
  });
  return hip_status();
}

extern "C" fp4q_status_t fp4q_kv_read_mxfp4(const fp4q_kv_cache_t *cache, const int64_t *slots, int64_t tokens,
                                            fp4q_dtype_t out_dtype, void *k_out, void *v_out, void *workspace,
                                            size_t workspace_bytes, void *stream) {
  if (!cache || (tokens != 0 && (!slots || (!k_out && !v_out)))) return FP4Q_ERR_NULL;
  if (!ws_ok(workspace, workspace_bytes)) return FP4Q_ERR_WORKSPACE;
  if (out_dtype != FP4Q_F32 && out_dtype != FP4Q_BF16) return FP4Q_ERR_ARG;
  fp4q_status_t st = kv_check_cache(*cache);
  if (st != FP4Q_OK) return st;
  if (!kv_size_ok(tokens, cache->heads, cache->head_dim)) return FP4Q_ERR_SHAPE;
  if (tokens && (!kv_aligned(slots, 8) || !kv_aligned(k_out, 16) || !kv_aligned(v_out, 16))) return FP4Q_ERR_ALIGN;
  hipStream_t s = (hipStream_t)stream;
  uint32_t *status = (uint32_t *)((char *)workspace + kWsStatus);
  if (tokens == 0) {
    hipLaunchKernelGGL(kv_status_kernel, dim3(1), dim3(64), 0, s, status);
    return hip_status();
  }
  const int units = (int)(tokens * cache->heads);
  const CacheView c = view(*cache);
  with_dim(cache->head_dim, [&](auto dc) {
    constexpr int D = decltype(dc)::value;
    constexpr int U = kThreads / (D / kChunk);
    const dim3 grid((unsigned)(((int64_t)units + U - 1) / U), 2);
    with_type(out_dtype, [&](auto op) {
      using O = std::remove_pointer_t<decltype(op)>;
      hipLaunchKernelGGL((kv_read_kernel<O, D>), grid, dim3(kThreads), 0, s, c, slots, units,
                         make_divider((uint32_t)cache->heads), (O *)k_out, (O *)v_out, status);
    });
  });
  return hip_status();
}
