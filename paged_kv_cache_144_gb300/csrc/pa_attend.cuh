// pa_attend.cuh - device code shared by the kernels of pa_attend: a sequence's
// query range, which positions a query sees, and one query row computed by a
// warp from the definition.
#pragma once

#include <type_traits>

#include "pa_common.cuh"
#include "pa_ops.h"

namespace pa {

struct SeqView {
  int T;     // cached tokens, clamped to the table's capacity
  int row0;  // first query row
  int L;     // queries (0 when the range is invalid)
};

__device__ __forceinline__ SeqView seq_view(const AttendParams& p, int s, bool report) {
  SeqView v;
  int T = __ldg(p.seq_lens + s);
  const int cap = p.max_blocks_per_seq << p.block_shift;
  if (T < 0 || T > cap) {
    if (report) raise_error(p.err, PA_DEVERR_SEQ_LEN);
    T = T < 0 ? 0 : cap;
  }
  v.T = T;
  if (p.q_starts) {
    const int a = __ldg(p.q_starts + s), b = __ldg(p.q_starts + s + 1);
    const bool ok = a >= 0 && b >= a && b <= p.num_tokens && b - a <= p.max_q_len;
    if (!ok && report) raise_error(p.err, PA_DEVERR_QUERY);
    v.row0 = ok ? a : 0;
    v.L = ok ? b - a : 0;
  } else {
    v.row0 = s;
    v.L = 1;
  }
  return v;
}

// Bounds [lo, hi) of what query i sees; with a tree, positions from `first` on
// also need their bit.
struct RowBounds {
  int pos, lo, hi;
};
__device__ __forceinline__ RowBounds row_bounds(const AttendParams& p, const SeqView& v, int prefix, int i) {
  RowBounds b;
  b.pos = v.T - v.L + i;
  if (b.pos < 0) {  // more queries than tokens: nothing
    b.lo = b.hi = 0;
  } else if (p.tree_mask) {
    b.lo = 0;
    b.hi = v.T;
  } else {
    b.lo = p.window > 0 ? max(0, b.pos + 1 - p.window) : 0;
    b.hi = max(b.pos + 1, prefix);
  }
  return b;
}
__device__ __forceinline__ int seq_prefix(const AttendParams& p, int s, int T) {
  return p.prefix_lens ? max(0, min(__ldg(p.prefix_lens + s), T)) : 0;
}

// softcap * tanh(x / softcap) with an absolute error of a few 1e-7 softcap:
// tanh(y) = 1 - 2 / (1 + e^2y) (the exponential overflows to infinity for a
// large y, which gives 1, and underflows to 0, which gives -1).
__device__ __forceinline__ float cap_score(float x, float cap, float two_log2e_over_cap) {
  return cap - __fdividef(2.f * cap, 1.f + fast_exp2(x * two_log2e_over_cap));
}

// One cache element, widened and (INT8) with its zero point subtracted; scales stay outside.
template <typename KVT>
__device__ __forceinline__ float cache_elem(const uint8_t* row, int c, int zp) {
  if constexpr (std::is_same<KVT, e4m3_t>::value) {
    return widen2_e4m3(row[c]).x;
  } else if constexpr (std::is_same<KVT, i8_t>::value) {
    return static_cast<float>(static_cast<int>(reinterpret_cast<const int8_t*>(row)[c]) - zp);
  } else {
    return load_scalar<KVT>(row, c);
  }
}

// One (query row, head) by one warp: the running maximum and sum in log2
// domain over 32 positions at a time, one per lane; then each visible
// position's V row, one column per lane and step.  Positions that are not
// visible are never read from V.  The query sits in registers, D / 32 columns
// per lane.  A row whose columns have all become NaN stays so: it ends early.
template <typename KVT, int D>
__device__ __forceinline__ void attend_row(const AttendParams& p, int s, const SeqView& v, int i, int h) {
  const int lane = threadIdx.x & 31;
  const int kvh = h / p.group;
  const int64_t n = static_cast<int64_t>(v.row0) + i;
  const RowBounds rb = row_bounds(p, v, seq_prefix(p, s, v.T), i);
  const float kLog2e = 1.4426950408889634f;
  float ks = 1.f, vs = 1.f;
  int kz = 0, vz = 0;
  if constexpr (elem<KVT>::bytes == 1) {
    ks = __ldg(p.k_scale + kvh);
    vs = __ldg(p.v_scale + kvh);
  }
  if constexpr (std::is_same<KVT, i8_t>::value) {
    kz = __ldg(p.k_zero_point + kvh);
    vz = __ldg(p.v_zero_point + kvh);
  }
  float q[D / 32];
#pragma unroll
  for (int j = 0; j < D / 32; ++j) {
    const int64_t e = n * p.q_stride + static_cast<int64_t>(h) * D + lane + 32 * j;
    q[j] = p.q_dtype == PA_BF16 ? load_scalar<bf16_t>(p.q, e) : load_scalar<f16_t>(p.q, e);
  }
  __syncwarp();  // what other lanes stored to this row before is overwritten below
  const float slope = p.slopes ? __ldg(p.slopes + h) : 0.f;
  const float capk = p.softcap > 0.f ? 2.f * kLog2e / p.softcap : 0.f;
  const int32_t* table = p.block_tables + static_cast<int64_t>(s) * p.max_blocks_per_seq;
  const int first = v.T - v.L;
  auto row_of = [&](const void* cache, int t) -> const uint8_t* {
    int pb = __ldg(table + (t >> p.block_shift));
    if (pb < 0 || pb >= p.num_blocks) {
      raise_error(p.err, PA_DEVERR_BLOCK_ID);
      pb = 0;
    }
    return static_cast<const uint8_t*>(cache) +
           ((static_cast<int64_t>(pb) * p.num_kv_heads + kvh) * p.block_size + (t & (p.block_size - 1))) *
               (D * elem<KVT>::bytes);
  };
  float m = -INFINITY, l = 0.f, acc[D / 32];
#pragma unroll
  for (int j = 0; j < D / 32; ++j) acc[j] = 0.f;
  for (int t0 = rb.lo & ~31; t0 < rb.hi; t0 += 32) {
    const int t = t0 + lane;
    bool see = t >= rb.lo && t < rb.hi;
    if (see && p.tree_mask && t >= first) {
      const int j = t - first;
      see = (p.tree_mask[n * p.tree_words + (j >> 6)] >> (j & 63)) & 1ull;
    }
    float z = -INFINITY;
    const uint8_t* kr = see ? row_of(p.k_cache, t) : static_cast<const uint8_t*>(p.k_cache);
    float x = 0.f;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
#pragma unroll 1
      for (int c = 0; c < 32; ++c) x = fmaf(__shfl_sync(0xffffffffu, q[j], c), cache_elem<KVT>(kr, c + 32 * j, kz), x);
    }
    if (see) {
      x *= p.scale * ks;
      if (p.softcap > 0.f) x = cap_score(x, p.softcap, capk);
      if (p.slopes) x -= slope * static_cast<float>(abs(rb.pos - t));
      z = x * kLog2e;
    }
    if (__any_sync(0xffffffffu, z != z || z == INFINITY)) {  // no maximum to subtract: every weight is NaN, and so is the row
      m = INFINITY;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) acc[j] = nanf("");
      break;
    }
    float mx = z;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float mn = fmaxf(m, mx);
    if (mn == -INFINITY) continue;
    const float a = exp2f(m - mn), e = exp2f(z - mn);
    m = mn;
    l = l * a + e;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) acc[j] *= a;
    unsigned left = __ballot_sync(0xffffffffu, see);
    while (left) {
      const int k = __ffs(left) - 1;
      left &= left - 1;
      const float w = __shfl_sync(0xffffffffu, e, k);
      const uint8_t* vr = row_of(p.v_cache, t0 + k);
#pragma unroll
      for (int j = 0; j < D / 32; ++j) acc[j] = fmaf(w, cache_elem<KVT>(vr, lane + 32 * j, vz), acc[j]);
    }
    bool lost = true;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) lost = lost && acc[j] != acc[j];
    if (__all_sync(0xffffffffu, lost)) break;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const float inv = l > 0.f ? vs / l : 0.f;
#pragma unroll
  for (int j = 0; j < D / 32; ++j) {
    const float o = m == -INFINITY ? 0.f : acc[j] * inv;
    store_out(p.out, p.out_dtype, (n * p.num_heads + h) * D + lane + 32 * j, o);
  }
}

// Whether row n (query * heads + head) of out, as stored, holds NaN or infinity (all lanes of a warp call it).
template <int D>
__device__ __forceinline__ bool row_not_finite(const AttendParams& p, int64_t n) {
  bool bad = false;
#pragma unroll
  for (int j = 0; j < D / 32; ++j) {
    const int64_t e = n * D + (threadIdx.x & 31) + 32 * j;
    if (p.out_dtype == PA_F32) {
      bad |= (__ldcg(static_cast<const unsigned int*>(p.out) + e) & 0x7f800000u) == 0x7f800000u;
    } else {
      const unsigned int most = p.out_dtype == PA_BF16 ? 0x7f80u : 0x7c00u;  // an exponent of ones
      bad |= (__ldcg(static_cast<const unsigned short*>(p.out) + e) & most) == most;
    }
  }
  return __any_sync(0xffffffffu, bad);
}

// Out of line, for the decode kernel's variants, which call it in two places.  It runs only for rows whose result is not finite,
// and only when no wait of a pipeline depends on the warp any more: a row takes about a microsecond per position (96 queries
// x heads of a KV head over 12000 positions, one V row NaN: 130 ms, against 0.2 ms).
template <typename KVT, int D>
__device__ __noinline__ void attend_row_again(const AttendParams& p, int s, const SeqView& v, int i, int h) {
  attend_row<KVT, D>(p, s, v, i, h);
}

// The 32 visibility bits of positions b0 .. b0 + 31 in a drafted tree's mask row (words tree[0 .. words)): bit
// position - first from position `first` on, ones before it.
__device__ __forceinline__ uint32_t tree_bits(const uint64_t* tree, int words, int first, int b0) {
  const int k0 = b0 - first;  // node of the first position (may be negative)
  if (k0 <= -32) return 0xffffffffu;
  const int kk = max(k0, 0), w = kk >> 6, sh = kk & 63;
  uint64_t x = w < words ? tree[w] >> sh : 0ull;
  if (sh > 32 && w + 1 < words) x |= tree[w + 1] << (64 - sh);
  return k0 >= 0 ? static_cast<uint32_t>(x) : (static_cast<uint32_t>(x) << (-k0)) | ((1u << (-k0)) - 1u);
}

}  // namespace pa
