// pa_attend_tc.cuh - attention of ragged query rows over the paged cache on
// the 5th-generation tensor cores (tcgen05), sm_103a.
//
// Mathematics.  The queries of one sequence and the G heads that share a KV
// head form R = L * G rows; S = Q K^T over 128 cached positions at a time, the
// modifiers and masks of include/pa.h on each score, the running maximum m and
// sum l of the softmax per row in base 2, O = O + P V.  m only follows the
// maximum once it is kSlack above it (weights up to 2^kSlack are exact in
// float32), so O is rarely rescaled.
//
// CTAs work alone (CG = 1) or in clusters of two (CG = 2, head size 128 with
// more than 128 rows, and 8-bit caches): a pair's tcgen05.mma takes 128 rows
// from each CTA against a K or V tile of which each loaded half, so the pair
// reads a tile from L2 once for up to 512 rows.
//
// Layout on the SM.  One persistent CTA per SM, 12 warps:
//   warp 0     TMA producer of the K tiles (128 positions, one box per cache
//              block) into a ring of stages
//   warps 1-2  issue the tcgen05.mma of streams 0 and 1 (TMEM, 512 columns: S0,
//              S1, O0, O1 of 128 lanes x 128 columns; the weights P overwrite S)
//   warp 3     the same for the V tiles and both streams' query rows; zeroes V
//              rows where it must (V apart from K: with the streams taking turns
//              a V stage comes free long after the K stage needed next)
//   warps 4-7, 8-11   softmax of streams 0 and 1, one row per thread: the row
//              maximum and sum need no exchange between threads
// The streams' turns, and the two halves (64 positions) of each stream's tile,
// keep the tensor cores and the softmax busy at once: while the weights of one
// half are computed, the other half's are multiplied and the next tile's scores
// take their columns.  With more than 128 rows per (sequence, KV head) the streams
// are two row tiles over the same K/V tiles ("paired": every K/V byte read
// from L2 serves 256 rows); with up to 128 rows they take the positions' tiles
// in turn ("alternating") and their results are joined like any other split.
//
// Shared-memory tiles are stored as 8-row groups of [128-byte half][8 rows][128
// bytes] with the 128-byte swizzle, which one 4-D TMA box per block writes for
// any block size; it is the K-major operand layout of S = Q K^T (row groups
// NH * 1024 bytes apart) and the MN-major one of P V as it is.
//
// 8-bit caches (pairs of CTAs only): the producer brings the codes as they are
// and four more warps (12-15) widen them to f16 in the operands' layout, exactly
// (the K scale multiplies the scores, the V scale the output), zero V rows on
// the way and bring bf16 queries into f16's range: each row is multiplied by the
// power of two that puts its largest element at 2^14 .. 2^15, its scores by the
// inverse, as in the decode kernel.
//
// Work split.  A segment is (sequence, KV head, row tile).  All segments'
// position tiles in order, each segment charged kFragCost tiles more for what
// a fragment costs besides them, are cut into equal contiguous ranges, one per
// CTA.  A fragment that is not its whole segment leaves (m, l, O) in the
// workspace and counts itself in; the one that arrives last joins them in
// order, so the result does not depend on who that is.
//
// Rounding.  P enters P V as 16 bits (bf16 with a bf16 cache, else f16 with
// weights scaled by 2^7, so that small ones stay above its smallest value):
// half a step of the type, below the rounding of a 16-bit output.  In the SPLIT
// form (float32 outputs; also with few rows, where memory traffic bounds the
// call and the second product is free) P is two such values, hi + lo, and its
// rounding that of as many bits more.
//
// A position's V row is multiplied by P = 0 in rows that do not see it, which
// is not enough when it holds NaN or infinity: rows past the sequence's end (or
// before the window) are zeroed in shared memory, and a result row that is
// not finite is computed again by one warp from the definition (attend_row):
// once all of the CTA's fragments are done, so that no wait of the pipeline
// depends on it.
//
// Every wait on a barrier ends after a limit (2 s) with PA_DEVERR_TIMEOUT.
//
// What bounds it.  Prompt chunks of 4 x 1-2K queries over 4-8K tokens (32 heads
// on 8, head size 128): 555 us, 62 % of the measured bf16 matrix rate; 64-node
// trees over 8 x 32K (64 heads on 8): 435 us, 65 %.  Without the softmax's work
// the same loop takes 357 and 277 us, without its loads either 324 and 252: the
// tensor cores wait for weights.  Half a tile costs a softmax warp about 1490
// cycles, 760 of them arithmetic (two warps share each scheduler's exponential
// unit), the rest the way to and from TMEM and the barriers; the products of
// both streams' halves need 1024.  Taken: whole tiles to half tiles 697 -> 571
// us, single CTAs to pairs 571 -> 555.  Tried and slower: fetching the next
// half's scores before handing this one over (604 us, registers), computing on
// the first 32 columns while the rest arrive (559), the two streams set half a
// tile apart (550 to 555), their warps on a scheduler taking turns (630).
#pragma once

#include "pa_attend.cuh"

namespace pa {

constexpr int kTile = 128;      // positions per tile, rows per stream
constexpr int kHalfTile = kTile / 2;
constexpr int kFragCost = 1;    // tiles charged per fragment
constexpr float kSlack = 8.f;   // log2 by which the maximum may lag

// ----------------------------------------------------------------- tcgen05 wrappers

// CG: CTAs that share a tensor-core operation (1, or the 2 of a cluster).
template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t smem_addr, uint32_t cols) {
  if constexpr (CG == 1)
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr), "r"(cols) : "memory");
  else
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr), "r"(cols) : "memory");
}
template <int CG>
__device__ __forceinline__ void tmem_dealloc(uint32_t addr, uint32_t cols) {
  if constexpr (CG == 1) {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
  } else {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
  }
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Arrives on `bar` (in both CTAs of a pair, at the same offset) when this thread's tensor-core operations so far are done.
template <int CG>
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  if constexpr (CG == 1)
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}
// Barriers between the CTAs of a pair: arrive on the pair's first CTA, wait with the cluster's scope.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void arrive_first_cta(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %0, 0;\n\t"
      "mbarrier.arrive.shared::cluster.b64 _, [r];\n\t}" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mbar_wait_bounded_cluster(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (true) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    if (global_timer_ns() - t0 > limit_ns) return false;
  }
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// One lane of the warp, always the same one, chosen in a way that leaves the branch on it warp-uniform to the compiler.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}" : "=r"(p));
  return p != 0;
}
// Operand descriptors are passed as their two words: the high word holds no address and is a constant.
template <int CG>
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                          bool accumulate) {
#define PA_MMA_SS(CGS)                                                                                                   \
  asm volatile(                                                                                                          \
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, %6, 0;\n\tmov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t" \
      "tcgen05.mma.cta_group::" CGS ".kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),                                       \
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))                     \
      : "memory")
  if constexpr (CG == 1) PA_MMA_SS("1"); else PA_MMA_SS("2");
#undef PA_MMA_SS
}
template <int CG>
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi, uint32_t idesc, bool accumulate) {
#define PA_MMA_TS(CGS)                                                                                            \
  asm volatile(                                                                                                   \
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.u32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\t"                       \
      "tcgen05.mma.cta_group::" CGS ".kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),                             \
      "r"(a), "r"(b_lo), "r"(hi), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))                              \
      : "memory")
  if constexpr (CG == 1) PA_MMA_TS("1"); else PA_MMA_TS("2");
#undef PA_MMA_TS
}
// 32 columns of this warp's 32 lanes
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
// 16 columns
__device__ __forceinline__ void tmem_ld16(uint32_t addr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}
// 32 consecutive outputs from element i (a multiple of 32) of one row by one thread: whole 32-byte sectors (`wide`: the
// buffer is 32-byte aligned), or 16 bytes at a time.
__device__ __forceinline__ void store32(void* dst, const uint32_t* w, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
__device__ __forceinline__ void store_row32(void* out, int dtype, int64_t i, const float* v, bool wide) {
  if (dtype == PA_F32) {
#pragma unroll
    for (int k = 0; k < 32; k += 8) store32(static_cast<float*>(out) + i + k, reinterpret_cast<const uint32_t*>(v + k), wide);
  } else {
    uint32_t w[16];
    if (dtype == PA_BF16) {
#pragma unroll
      for (int k = 0; k < 16; ++k) w[k] = pack2<true>(v[2 * k], v[2 * k + 1]);
    } else {
#pragma unroll
      for (int k = 0; k < 16; ++k) w[k] = pack2<false>(v[2 * k], v[2 * k + 1]);
    }
    store32(static_cast<uint16_t*>(out) + i, w, wide);
    store32(static_cast<uint16_t*>(out) + i + 16, w + 8, wide);
  }
}
// V = 2 or 4 consecutive floats of a record, and the same columns of an output row
template <int V>
__device__ __forceinline__ void load_columns(const float* src, float* v) {
  if constexpr (V == 4) {
    const float4 x = __ldcg(reinterpret_cast<const float4*>(src));
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
  } else {
    const float2 x = __ldcg(reinterpret_cast<const float2*>(src));
    v[0] = x.x, v[1] = x.y;
  }
}
template <int V>
__device__ __forceinline__ void store_columns(void* out, int dtype, int64_t i, const float* v) {
  if constexpr (V == 4) {
    store_out4(out, dtype, i, make_float4(v[0], v[1], v[2], v[3]), true);
  } else {
    store_out(out, dtype, i, v[0]);
    store_out(out, dtype, i + 1, v[1]);
  }
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// 4-D tiled TMA load global -> shared, completion counted on `bar`.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// Shared-memory operand descriptor, 128-byte swizzle: start address and leading byte offset (between 128-byte halves; used
// by the MN-major operand) in 16-byte units in the low word; stride byte offset (between 8-row groups), descriptor
// version 1 and the swizzle in the high word.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr) { return ((addr & 0x3ffffu) >> 4) | ((1024u >> 4) << 16); }
constexpr uint32_t desc_hi(uint32_t sbo) { return (sbo >> 4) | (1u << 14) | (2u << 29); }

// Instruction descriptor: float32 accumulators, 16-bit operands, M = 128 per CTA.
constexpr uint32_t mma_idesc(bool bf16, bool b_mn_major, int n, int cg) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((b_mn_major ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(8 * cg) << 24);
}

// ----------------------------------------------------------------- geometry

struct TcParams {
  AttendParams a;
  int paired;        // the streams are two row tiles (else: one, its position tiles in turn)
  int seg_rows;      // rows of a segment: stream_rows x CTAs of a group x (paired: 2)
  float max_segments;  // an upper bound
  int rec_rows;      // rows of a record
  int slots;         // records of one stream per CTA: paired 2, alternating 4
  int* counters;     // arrivals: paired: by the segment's first CTA; alternating: by s * H_kv + kvh
  float* records;
};

// Rows of one stream's tile: whole queries, as one TMA box of 128 / G queries by G heads brings them.
__host__ __device__ __forceinline__ int stream_rows(int group) { return kTile / group * group; }

// Position tiles [lo, hi) of row tile m of a sequence.
struct TileRange {
  int lo, hi;
};
__device__ __forceinline__ TileRange tile_range(const AttendParams& p, const SeqView& v, int prefix, int rows_per_tile, int m) {
  TileRange r;
  const int i0 = m * rows_per_tile / p.group;                       // first query with a row in the tile
  const int i1 = min(v.L, (m * rows_per_tile + rows_per_tile - 1) / p.group + 1) - 1;  // last one
  const int last = v.T - v.L + i1;
  if (v.L <= 0 || last < 0) {
    r.lo = r.hi = 0;
    return r;
  }
  const int first = max(0, v.T - v.L + i0);
  const int lo = p.window > 0 ? max(0, first + 1 - p.window) : 0;
  const int hi = p.tree_mask ? v.T : max(last + 1, prefix);
  r.lo = lo / kTile;
  r.hi = (hi + kTile - 1) / kTile;
  return r;
}

struct Frag {
  int s, kvh, m;      // segment
  SeqView v;
  int prefix;         // visible prefix length
  int t0, t1;         // its position tiles
  int lo;             // first position any row of the segment sees
  int seg_start;      // cost position of the segment
  int seg_tiles;
  bool whole;
  int idx;            // ordinal in the CTA
};

// Walks the fragments of one CTA's range of cost positions.
struct FragIter {
  int u, u1, U, nw;
  int s, seg_cost_sum;  // sequence, its cost per KV head
  int m, m_pos;         // row tile being looked at and its position within the head (scan state)
  int kvh;
  int s_state;          // sequence the scan state belongs to (-1: none)
  int idx;
};

__device__ __forceinline__ int seg_cost(int tiles) { return tiles > 0 ? tiles + kFragCost : 0; }

// A warp's iterator and its current fragment live in shared memory, not in its registers.
struct WarpFrag {
  FragIter it;
  Frag f;
};

__device__ __forceinline__ bool advance_frag(FragIter& it, Frag& f, const int* prefix, const TcParams& p) {
  const AttendParams& a = p.a;
  const int rpt = p.seg_rows;
  while (it.u < it.u1) {
    while (prefix[it.s + 1] <= it.u) ++it.s;  // last sequence starting at or before u (u < U: one exists)
    const int per = (prefix[it.s + 1] - prefix[it.s]) / a.num_kv_heads;
    const int r = it.u - prefix[it.s];
    const int kvh = r / per;
    const int off = r - kvh * per;
    const SeqView v = seq_view(a, it.s, false);
    const int pre = seq_prefix(a, it.s, v.T);
    if (it.s_state != it.s || it.kvh != kvh || off < it.m_pos) {
      it.m = 0;
      it.m_pos = 0;
      it.s_state = it.s;
      it.kvh = kvh;
    }
    TileRange tr = tile_range(a, v, pre, rpt, it.m);
    while (off >= it.m_pos + seg_cost(tr.hi - tr.lo)) {
      it.m_pos += seg_cost(tr.hi - tr.lo);
      ++it.m;
      tr = tile_range(a, v, pre, rpt, it.m);
    }
    const int n = tr.hi - tr.lo;
    const int seg_start = prefix[it.s] + kvh * per + it.m_pos;
    const int fend = min(it.u1, seg_start + n + kFragCost);
    const int ja = max(0, it.u - seg_start - kFragCost), jb = fend - seg_start - kFragCost;
    it.u = fend;
    if (jb <= ja) continue;  // the range ends inside the segment's overhead
    f.s = it.s;
    f.kvh = kvh;
    f.m = it.m;
    f.v = v;
    f.prefix = pre;
    f.t0 = tr.lo + ja;
    f.t1 = tr.lo + jb;
    f.lo = a.window > 0 ? max(0, max(0, v.T - v.L + it.m * rpt / a.group) + 1 - a.window) : 0;
    f.seg_start = seg_start;
    f.seg_tiles = n;
    f.whole = ja == 0 && jb == n;
    f.idx = it.idx++;
    return true;
  }
  return false;
}

// The warp's next fragment (all lanes call it); false at the end of the CTA's range.
__device__ __forceinline__ bool next_frag(WarpFrag* w, const int* prefix, const TcParams& p) {
  FragIter it = w->it;
  Frag f;
  const bool more = advance_frag(it, f, prefix, p);
  __syncwarp();  // every lane has read the old state
  if ((threadIdx.x & 31) == 0) {
    w->it = it;
    if (more) w->f = f;
  }
  __syncwarp();
  return more;
}

// CTA whose range holds cost position x.
__device__ __forceinline__ int cta_of(int x, int U, int nw) {
  return static_cast<int>((static_cast<long long>(x + 1) * nw - 1) / U);
}
__device__ __forceinline__ int range_start(int c, int U, int nw) {
  return static_cast<int>(static_cast<long long>(c) * U / nw);
}
// Tiles of a segment (its cost position, its tiles) in CTA c's range.
__device__ __forceinline__ int tiles_in(int c, int U, int nw, int seg_start, int seg_tiles) {
  const int b = max(0, range_start(c, U, nw) - seg_start - kFragCost);
  return min(seg_tiles, range_start(c + 1, U, nw) - seg_start - kFragCost) - b;
}
// Which of a CTA's records its fragment of a segment fills: 0: the CTA's first fragment, 1: a later one (both cut), 2 and
// 3: whole segments in turn (alternating streams: two contributions of one CTA).  Whole segments of a CTA may be many: a slot is
// written again only when its records have been joined (barriers JD), since a stream that need not join can be several
// fragments ahead of the one that does.
__device__ __forceinline__ int slot_kind_of(bool whole, int idx) { return whole ? 2 + (idx & 1) : (idx == 0 ? 0 : 1); }
// The same for CTA c of a cut segment, seen from outside: a range that starts before the segment holds a fragment before it.
__device__ __forceinline__ int cut_slot_kind(int c, int c0, int U, int nw, int seg_start) {
  return c > c0 || range_start(c, U, nw) >= seg_start ? 0 : 1;
}

template <typename KVT, int D, int CG>
struct TcTraits {
  static constexpr bool BF16 = std::is_same<KVT, bf16_t>::value;
  static constexpr bool B8 = elem<KVT>::bytes == 1;
  static_assert(!B8 || (CG == 2 && D == 128), "8-bit caches: pairs of CTAs, head_dim 128");
  static constexpr int THREADS = B8 ? 512 : 384;
  // The softmax threads hold 64 scores each: registers move to their warps from the others (at launch 65536 / THREADS,
  // rounded down to a multiple of 8, each).
  static constexpr int REGS_LOW = B8 ? 72 : 88, REGS_HIGH = B8 ? 184 : 208;
  static_assert((THREADS - 256) * REGS_LOW + 256 * REGS_HIGH <= THREADS * (65536 / THREADS / 8 * 8), "register split");
  static constexpr int NH = D * 2 / 128;           // 128-byte halves per 16-bit row
  static constexpr int TILE_BYTES = kTile * D * 2;  // a tile of K, V or Q
  // A pair of CTAs halves every K and V tile: each holds 64 of a K tile's positions, and one 128-byte half of all of a
  // V tile's rows.
  static_assert(CG == 1 || NH == 2, "a pair of CTAs shares tiles of 256-byte rows");
  static constexpr int KROWS = kTile / CG;         // rows of a K stage
  static constexpr int VH = NH / CG;               // halves of a V stage
  static constexpr int KGROUP = NH * 1024, VGROUP = VH * 1024;  // bytes of 8 rows
  static constexpr int STAGE = TILE_BYTES / CG;    // bytes of a K or V stage
  static constexpr int NST = B8 ? 3 : (D == 128 ? 2 : 4) * CG;  // stages of K and of V
  // 8-bit caches: stages of codes as they come, [rows][128 / CG bytes] for V
  static constexpr int NR = B8 ? 2 : 0, RAW = B8 ? STAGE / 2 : 0;
  static constexpr int OFF_Q = 0;                  // two tiles
  static constexpr int OFF_K = 2 * TILE_BYTES;
  static constexpr int OFF_V = OFF_K + NST * STAGE;
  static constexpr int OFF_RK = OFF_V + NST * STAGE;
  static constexpr int OFF_RV = OFF_RK + NR * RAW;
  static constexpr int OFF_QX = OFF_RV + NR * RAW;  // bf16 queries: 2^-exponent per row, [stream][use & 1][128]
  static constexpr int OFF_BAR = OFF_QX + (B8 ? 4 * kTile * 4 : 0);
  // barriers (8 bytes each)
  static constexpr int KF = 0, KE = KF + NST, VF = KE + NST, VE = VF + NST, QF = VE + NST, QE = QF + 2, SF = QE + 2,
                       PF = SF + 4, OH = PF + 4, OD = OH + 2, RB = OD + 2,  // SF, PF: per half of a tile; OH, OD: its halves
                       KP = RB + 2, VP = KP + NST, QP = VP + NST,  // the peer's has arrived
                       VL = QP + 2,                                // a V tile with rows to be zeroed has arrived
                       RKF = VL + NST, RKE = RKF + NR, RVF = RKE + NR, RVE = RVF + NR, QL = RVE + NR,  // 8-bit caches
                       JD = QL + 2,  // a whole segment's records have been joined, per slot
                       NBAR = JD + 2;
  static constexpr int OFF_MISC = OFF_BAR + ((NBAR * 8 + 15) / 16) * 16;  // tmem address, flags, scan scratch
  static constexpr int OFF_FRAG = OFF_MISC + 256;                         // WarpFrag per warp
  static constexpr int OFF_PREFIX = OFF_FRAG + (THREADS / 32 * static_cast<int>(sizeof(WarpFrag)) + 15) / 16 * 16;
  static size_t smem_bytes(int num_seqs) { return 1024 + OFF_PREFIX + static_cast<size_t>(num_seqs + 1) * 4; }
};

// Word of the shared scratch that notes where rows of the CTA are not finite, and a fragment's bits in it: one for all whole
// segments, one for each stream's rows of a cut one (slot kind 0 or 1) that this CTA has joined.
constexpr int kRedo = 40;
__device__ __forceinline__ int redo_bits(bool whole, int slot_kind, int stream) {
  return whole ? 16 : 1 << (2 * slot_kind + stream);
}

// Where contribution c of a fragment with this slot kind lies.
template <int D>
__device__ __forceinline__ float* record_at(const TcParams& p, int cta, int kind, int c) {
  return p.records + (static_cast<int64_t>(cta) * p.slots * 2 + kind * 2 + c) * (p.rec_rows * (D + 2));
}

// Joins the contributions of CTA groups c0 .. c1 to rows 32 wq .. 32 wq + 31 of a stream's row tile, in order, and writes the
// rows out; run by one warp of the contribution that arrived last.  Each lane takes one row's maximum, sum and weights; then
// kJoin rows at a time, D / 32 columns per lane.  This runs at the end of most CTAs, where nothing hides the latency of its
// loads (one row and record after the other they took 100 us at the end of a 600 us call): those of kJoin rows of kRecs
// records are under way at once, which the registers of the softmax warps allow.
constexpr int kJoin = 4, kRecs = 3;
// True: a row is not finite.
template <typename KVT, int D, int CG>
__device__ __forceinline__ bool join_rows(const TcParams& p, const Frag& f, int U, int nw, int c0, int c1, int rank, int t, int wq,
                                          int row0, int rows, int slot_kind) {
  const AttendParams& a = p.a;
  const int lane = threadIdx.x & 31;
  constexpr int V = D / 32;  // columns per lane
  // contribution k: CTA group c0 + k (paired), or c0 + k / 2, stream k % 2 (alternating: the second may be missing)
  const int total = (c1 - c0 + 1) * (p.paired ? 1 : 2);
  auto record_of = [&](int k) -> const float* {
    const int c = c0 + (p.paired ? k : k >> 1);
    if (k >= total || (!p.paired && (k & 1) >= tiles_in(c, U, nw, f.seg_start, f.seg_tiles))) return nullptr;
    const int kind = f.whole ? slot_kind : cut_slot_kind(c, c0, U, nw, f.seg_start);
    return record_at<D>(p, c * CG + rank, kind, p.paired ? t : k & 1);
  };
  const int lr = min(wq * 32 + lane, rows - 1);
  auto stats_of = [&](const float* rec) {
    return rec ? __ldcg(reinterpret_cast<const float2*>(rec + p.rec_rows * D + 2 * lr)) : make_float2(-INFINITY, 0.f);
  };
  float M = -INFINITY, L = 0.f;
#pragma unroll 4
  for (int k = 0; k < total; ++k) M = fmaxf(M, stats_of(record_of(k)).x);
#pragma unroll 4
  for (int k = 0; k < total; ++k) {
    const float2 ml = stats_of(record_of(k));
    L = fmaf(ml.x == -INFINITY ? 0.f : exp2f(ml.x - M), ml.y, L);
  }
  float inv = L > 0.f ? 1.f / L : 0.f;
  if constexpr (elem<KVT>::bytes == 1) inv *= __ldg(a.v_scale + f.kvh);
  bool bad = false;
  for (int g = 0; g < total; g += kRecs) {
    // (more than kRecs records: the rows are gone through again, from the sums so far)
    const float* rec[kRecs];
    float w[kRecs];
#pragma unroll
    for (int x = 0; x < kRecs; ++x) {
      rec[x] = record_of(g + x);
      const float m = stats_of(rec[x]).x;
      w[x] = m == -INFINITY ? 0.f : exp2f(m - M);
    }
    float* const sums = record_at<D>(p, c0 * CG + rank, f.whole ? slot_kind : cut_slot_kind(c0, c0, U, nw, f.seg_start),
                                     p.paired ? t : 0);  // of this warp's rows, in place of the first record's
    const bool last = g + kRecs >= total;
#pragma unroll 1
    for (int r0 = 0; r0 < 32 && wq * 32 + r0 < rows; r0 += kJoin) {
      float o[kRecs][kJoin][V], acc[kJoin][V];
#pragma unroll
      for (int x = 0; x < kRecs; ++x) {
#pragma unroll
        for (int k = 0; k < kJoin; ++k) {
          if (rec[x] && wq * 32 + r0 + k < rows) {
            load_columns<V>(rec[x] + static_cast<int64_t>(wq * 32 + r0 + k) * D + lane * V, o[x][k]);
          } else {
#pragma unroll
            for (int q = 0; q < V; ++q) o[x][k][q] = 0.f;
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kJoin; ++k) {
        const int row = wq * 32 + r0 + k;
#pragma unroll
        for (int q = 0; q < V; ++q) acc[k][q] = 0.f;
        if (g > 0 && row < rows) load_columns<V>(sums + static_cast<int64_t>(row) * D + lane * V, acc[k]);
#pragma unroll
        for (int x = 0; x < kRecs; ++x) {
          const float wk = __shfl_sync(0xffffffffu, w[x], r0 + k);
#pragma unroll
          for (int q = 0; q < V; ++q) acc[k][q] = fmaf(wk, o[x][k][q], acc[k][q]);
        }
        const float ik = __shfl_sync(0xffffffffu, inv, r0 + k), Lk = __shfl_sync(0xffffffffu, L, r0 + k);
        if (row >= rows) continue;
        if (!last) {
#pragma unroll
          for (int q = 0; q < V; ++q) sums[static_cast<int64_t>(row) * D + lane * V + q] = acc[k][q];
          continue;
        }
        const int i = (row0 + row) / a.group, h = f.kvh * a.group + (row0 + row) - i * a.group;
        const int64_t o0 = ((static_cast<int64_t>(f.v.row0) + i) * a.num_heads + h) * D + lane * V;
        bad |= Lk != Lk;
#pragma unroll
        for (int q = 0; q < V; ++q) {
          acc[k][q] *= ik;
          bad |= !(fabsf(acc[k][q]) < INFINITY);
        }
        store_columns<V>(a.out, a.out_dtype, o0, acc[k]);
      }
    }
  }
  return __any_sync(0xffffffffu, bad);
}

// ----------------------------------------------------------------- kernel

template <typename KVT, int D, int CG, bool SPLIT>
__global__ void __launch_bounds__(TcTraits<KVT, D, CG>::THREADS, 1)
attend_tc_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                 const __grid_constant__ CUtensorMap tmap_q,
                 const __grid_constant__ TcParams p) {
  using Tr = TcTraits<KVT, D, CG>;
  constexpr int NST = Tr::NST;
  const AttendParams& a = p.a;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const sm = smem_raw + (base - raw);
  const uint32_t bars = base + Tr::OFF_BAR;
  int* const misc = reinterpret_cast<int*>(sm + Tr::OFF_MISC);
  int* const prefix = reinterpret_cast<int*>(sm + Tr::OFF_PREFIX);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = a.num_seqs;
  const int rank = CG == 1 ? 0 : static_cast<int>(cluster_rank());  // CTA of its group; the first issues the products
  const bool q_widen = Tr::B8 && a.q_dtype == PA_BF16;  // bf16 queries become f16
  const int group_id = static_cast<int>(blockIdx.x) / CG, groups = static_cast<int>(gridDim.x) / CG;
  auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };
  auto wait = [&](int i, uint32_t parity, bool full = false) -> bool {  // full: the whole limit, whatever the call's
    if (mbar_wait_bounded(bar(i), parity, full ? kDefaultWaitLimitNs : a.wait_limit_ns)) return true;
    raise_error(a.err, PA_DEVERR_TIMEOUT);
    return false;
  };
  // the same for what the other CTA of a pair arrives on
  auto wait_pair = [&](int i, uint32_t parity) -> bool {
    if (mbar_wait_bounded_cluster(bar(i), parity, a.wait_limit_ns)) return true;
    raise_error(a.err, PA_DEVERR_TIMEOUT);
    return false;
  };

  if (threadIdx.x == 0) {
    prefetch_tensormap(&tmap_k);
    prefetch_tensormap(&tmap_v);
    prefetch_tensormap(&tmap_q);
    for (int i = 0; i < NST; ++i) {
      mbar_init(bar(Tr::KF + i), Tr::B8 ? 4 : 1);  // (8-bit caches: the widening warps)
      mbar_init(bar(Tr::KE + i), p.paired ? 2 : 1);  // paired: both streams read every tile
      mbar_init(bar(Tr::VF + i), Tr::B8 ? 4 : 1);
      mbar_init(bar(Tr::VE + i), p.paired ? 2 : 1);
      mbar_init(bar(Tr::VL + i), 1);
      mbar_init(bar(Tr::KP + i), 1);
      mbar_init(bar(Tr::VP + i), 1);
    }
    for (int i = 0; i < Tr::NR; ++i) {
      mbar_init(bar(Tr::RKF + i), 1);
      mbar_init(bar(Tr::RKE + i), 4);
      mbar_init(bar(Tr::RVF + i), 1);
      mbar_init(bar(Tr::RVE + i), 4);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(Tr::QF + t), q_widen ? 4 : 1);
      mbar_init(bar(Tr::QL + t), 1);
      mbar_init(bar(Tr::QE + t), 1);
      mbar_init(bar(Tr::SF + t), 1);
      mbar_init(bar(Tr::SF + 2 + t), 1);
      mbar_init(bar(Tr::PF + t), 4 * CG);
      mbar_init(bar(Tr::PF + 2 + t), 4 * CG);
      mbar_init(bar(Tr::OH + t), 1);
      mbar_init(bar(Tr::QP + t), 1);
      mbar_init(bar(Tr::OD + t), 1);
      mbar_init(bar(Tr::RB + t), 4);
      mbar_init(bar(Tr::JD + t), 4);
    }
    misc[kRedo] = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc<CG>(base + Tr::OFF_MISC, 512);
  griddep_wait();

  // ---- cost positions before each sequence (every CTA computes the same)
  {
    const int rpt = p.seg_rows;
    int carry = 0;
    constexpr int NW = Tr::THREADS / 32;
    int* const wsum = misc + 8;
    for (int s0 = 0; s0 < S; s0 += p.paired ? NW : Tr::THREADS) {
      int cost = 0, s;
      if (p.paired) {  // a warp per sequence, its lanes over the row tiles
        s = s0 + warp;
        if (s < S) {
          const SeqView v = seq_view(a, s, blockIdx.x == 0 && lane == 0);
          const int pre = seq_prefix(a, s, v.T);
          const int nm = (v.L * a.group + rpt - 1) / rpt;
          for (int m = lane; m < nm; m += 32) {
            const TileRange tr = tile_range(a, v, pre, rpt, m);
            cost += seg_cost(tr.hi - tr.lo);
          }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) cost += __shfl_xor_sync(0xffffffffu, cost, o);
        cost *= a.num_kv_heads;
        if (lane == 0) wsum[warp] = cost;
        __syncthreads();
        int before = carry, all = 0;
        for (int w = 0; w < NW; ++w) {
          before += w < warp ? wsum[w] : 0;
          all += wsum[w];
        }
        if (lane == 0 && s < S) prefix[s] = before;
        carry += all;
      } else {
        s = s0 + threadIdx.x;
        if (s < S) {
          const SeqView v = seq_view(a, s, blockIdx.x == 0);
          const TileRange tr = tile_range(a, v, seq_prefix(a, s, v.T), rpt, 0);
          cost = seg_cost(tr.hi - tr.lo) * a.num_kv_heads;
        }
        int x = cost;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        if (lane == 31) wsum[warp] = x;
        __syncthreads();
        int before = carry, all = 0;
        for (int w = 0; w < NW; ++w) {
          before += w < warp ? wsum[w] : 0;
          all += wsum[w];
        }
        if (s < S) prefix[s] = before + x - cost;
        carry += all;
      }
      __syncthreads();
    }
    if (threadIdx.x == 0) prefix[S] = carry;
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync_all();  // the peer's barriers exist
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(misc[0]);
  const int U = prefix[S];
  const int want = (U + kFragCost) / (kFragCost + 1);  // at least one tile per CTA
  // A segment cut n ways costs its tiles / n and its join n records of about 1.6 tiles' time: with few segments, fewer CTAs
  // than there are (n near the root of 0.6 tiles).
  const int balanced = static_cast<int>(sqrtf(0.6f * static_cast<float>(U) * p.max_segments));
  const int nw = min(groups, max(min(want, balanced), 1));
  WarpFrag* const wf = reinterpret_cast<WarpFrag*>(sm + Tr::OFF_FRAG) + warp;
  const Frag& f = wf->f;
  auto start_frags = [&] {  // the warp's iterator at the start of the CTA's range
    FragIter it;
    it.U = U;
    it.nw = nw;
    it.idx = 0;
    it.s = 0;
    it.s_state = -1;
    it.m = it.m_pos = it.kvh = 0;
    it.u = it.u1 = 0;
    if (group_id < nw && U > 0) {
      it.u = range_start(group_id, U, nw);
      it.u1 = range_start(group_id + 1, U, nw);
      int lo = 0, hi = S - 1;
      while (lo < hi) {  // last sequence with prefix <= u
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= it.u) lo = mid; else hi = mid - 1;
      }
      it.s = lo;
    }
    __syncwarp();
    if (lane == 0) wf->it = it;
    __syncwarp();
  };
  start_frags();

  // row tile of stream t in this CTA within its sequence
  auto row_tile = [&](int m, int t) { return p.paired ? (m * 2 + t) * CG + rank : m * CG + rank; };

  // V rows of a stage outside the sequence (or before the window) may hold anything, or were not loaded: zero for the
  // products (one warp; n_hi, n_lo: the first row past the end, the first visible one)
  auto partial = [&](int j) { return f.v.T - j * kTile < kTile || f.lo > j * kTile; };
  auto clear_v = [&](int st, int n_hi, int n_lo) {
    const uint32_t vt = base + Tr::OFF_V + st * Tr::STAGE;
    for (int x = lane; x < kTile * Tr::VH * 8; x += 32) {
      const int r = x / (Tr::VH * 8), c = x % (Tr::VH * 8);
      if (r >= n_hi || r < n_lo) sts128_zero(vt + (r >> 3) * Tr::VGROUP + (c >> 3) * 1024 + (r & 7) * 128 + (c & 7) * 16);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
  };

  // Boxes of this CTA's part of a K or V tile, and its first position.
  auto tile_rows = [&](bool is_v) { return is_v ? kTile : Tr::KROWS; };
  auto tile_start = [&](bool is_v, int j) { return j * kTile + (is_v ? 0 : rank * Tr::KROWS); };
  // This lane's block of tile j (its table entry), or -1.
  auto tile_block = [&](bool is_v, int j) -> int {
    const int boxes = tile_rows(is_v) / min(a.block_size, tile_rows(is_v));
    const int blk = (tile_start(is_v, j) >> a.block_shift) + (boxes > 1 ? lane : 0);
    const int nblk = (f.v.T + a.block_size - 1) >> a.block_shift;
    if (lane >= boxes || blk < (f.lo >> a.block_shift) || blk >= nblk) return -1;
    const int pb = __ldg(a.block_tables + static_cast<int64_t>(f.s) * a.max_blocks_per_seq + blk);
    if (pb >= 0 && pb < a.num_blocks) return pb;
    raise_error(a.err, PA_DEVERR_BLOCK_ID);
    return 0;
  };
  // One tile of K or V: its boxes, one lane each (block pb), into the next stage of the ring (8-bit caches: of codes).
  auto issue_tile = [&](bool is_v, int count, int j, int pb) -> bool {
    constexpr int RING = Tr::B8 ? Tr::NR : NST;
    const int box_rows = min(a.block_size, tile_rows(is_v)), boxes = tile_rows(is_v) / box_rows;
    const uint32_t box = static_cast<uint32_t>(box_rows / 8) * (is_v ? Tr::VGROUP : Tr::KGROUP) / (Tr::B8 ? 2 : 1);
    const int t0 = tile_start(is_v, j);
    const int st = count % RING;
    const uint32_t ph = static_cast<uint32_t>(count / RING) & 1u;
    const int empty = Tr::B8 ? (is_v ? Tr::RVE : Tr::RKE) : (is_v ? Tr::VE : Tr::KE);
    if (!__all_sync(0xffffffffu, wait(empty + st, ph ^ 1u))) return false;
    const uint32_t bytes = box * static_cast<uint32_t>(__popc(__ballot_sync(0xffffffffu, pb >= 0)));
    // a V tile with rows to be zeroed is announced once that is done
    const uint32_t full = bar((Tr::B8 ? (is_v ? Tr::RVF : Tr::RKF) : is_v ? (partial(j) ? Tr::VL : Tr::VF) : Tr::KF) + st);
    if (lane == 0) mbar_arrive_expect_tx(full, bytes);
    __syncwarp();
    const int row = boxes > 1 ? 0 : (t0 & (a.block_size - 1));
    if (pb >= 0) {
      if constexpr (Tr::B8)
        tma_load_2d(base + (is_v ? Tr::OFF_RV : Tr::OFF_RK) + st * Tr::RAW + lane * box, is_v ? &tmap_v : &tmap_k,
                    is_v ? rank * (D / CG) : 0, (pb * a.num_kv_heads + f.kvh) * a.block_size + row, full);
      else
        tma_load_4d(base + (is_v ? Tr::OFF_V : Tr::OFF_K) + st * Tr::STAGE + lane * box, is_v ? &tmap_v : &tmap_k, 0, 0,
                    is_v && CG == 2 ? rank : 0, (pb * a.num_kv_heads + f.kvh) * (a.block_size >> 3) + (row >> 3), full);
    }
    return true;
  };
  // Nothing of ours, and no arrival of the tensor cores, may land after the CTA has left: wait until each stage's last tile
  // has been used (after a wait that ran out, at least until it has arrived).
  auto drain = [&](bool is_v, int count) {
    for (int i = 0; i < NST; ++i) {
      const int n = count / NST + (i < count % NST ? 1 : 0);
      const uint32_t ph = static_cast<uint32_t>(n - 1) & 1u;
      if (n > 0 && !wait((is_v ? Tr::VE : Tr::KE) + i, ph, true)) wait((is_v ? Tr::VF : Tr::KF) + i, ph, true);
    }
    for (int i = 0; i < Tr::NR; ++i) {
      const int n = count / (Tr::B8 ? Tr::NR : 1) + (i < count % (Tr::B8 ? Tr::NR : 1) ? 1 : 0);
      if (n > 0) wait((is_v ? Tr::RVF : Tr::RKF) + i, static_cast<uint32_t>(n - 1) & 1u, true);
    }
  };

  if (warp < 4) {
    regs_dec<Tr::REGS_LOW>();
    if (warp == 0) {
      // ================================================================= K tiles (TMA)
      int kt = 0;
      bool ok = true;
      while (ok && next_frag(wf, prefix, p)) {
        const int t1 = f.t1;
        int pb = tile_block(false, f.t0);
        for (int j = f.t0; ok && j < t1; ++j) {
          ok = issue_tile(false, kt, j, pb);
          kt += ok ? 1 : 0;
          if (j + 1 < t1) pb = tile_block(false, j + 1);  // read while the next stage is waited for
        }
      }
      drain(false, kt);
    } else if (warp == 3) {
      // ================================================================= query rows and V tiles (TMA), V rows to be zeroed
      // (query rows past the sequence's last are another sequence's, or zero past the last token: their results are not stored)
      int uses[2] = {0, 0}, parity = 0, kt = 0;
      uint32_t vl = 0u;  // phases of VL used, per stage (a bit each)
      const int per_box = kTile / a.group;
      const uint32_t bytes = static_cast<uint32_t>(per_box * a.group) * D * 2;
      bool ok = true;
      while (ok && next_frag(wf, prefix, p)) {
        const int t1 = f.t1, n = t1 - f.t0;
        for (int e = 0; ok && e < 2; ++e) {
          const int t = p.paired ? e : e ^ parity;  // in the order in which the streams need them
          if (!p.paired && n <= e) continue;
          if (uses[t] > 0 && !wait(Tr::QE + t, static_cast<uint32_t>(uses[t] - 1) & 1u)) {
            ok = false;
            break;
          }
          ++uses[t];
          if (lane == 0) {
            const uint32_t full = bar((q_widen ? Tr::QL : Tr::QF) + t);
            mbar_arrive_expect_tx(full, bytes);
            tma_load_4d(base + Tr::OFF_Q + t * Tr::TILE_BYTES, &tmap_q, 0, f.kvh * a.group,
                        f.v.row0 + row_tile(f.m, t) * per_box, 0, full);
          }
          __syncwarp();
        }
        // the first V tile is under way before the queries are waited for
        int j = f.t0, pb = -1;
        if (ok) {
          ok = issue_tile(true, kt, j, tile_block(true, j));
          kt += ok ? 1 : 0;
          if (j + 1 < t1) pb = tile_block(true, j + 1);
        }
        for (int e = 0; ok && CG == 2 && rank != 0 && e < 2; ++e) {
          const int t = p.paired ? e : e ^ parity;
          if (!p.paired && n <= e) continue;
          if (!(ok = wait(Tr::QF + t, static_cast<uint32_t>(uses[t] - 1) & 1u))) break;
          if (lane == 0) arrive_first_cta(bar(Tr::QP + t));
        }
        if (!p.paired) parity ^= n & 1;
        while (ok) {
          if (!Tr::B8 && partial(j)) {
            const int st = (kt - 1) % NST;
            if (!(ok = wait(Tr::VL + st, (vl >> st) & 1u))) break;
            vl ^= 1u << st;
            clear_v(st, f.v.T - j * kTile, f.lo - j * kTile);
            if (lane == 0) mbar_arrive(bar(Tr::VF + st));
          }
          if (++j >= t1) break;
          ok = issue_tile(true, kt, j, pb);
          kt += ok ? 1 : 0;
          if (j + 1 < t1) pb = tile_block(true, j + 1);
        }
      }
      drain(true, kt);
      for (int t = 0; t < 2; ++t)
        if (uses[t] > 0 && !wait(Tr::QE + t, static_cast<uint32_t>(uses[t] - 1) & 1u, true))
          wait((q_widen ? Tr::QL : Tr::QF) + t, static_cast<uint32_t>(uses[t] - 1) & 1u, true);
    } else if (rank != 0) {
      // ================================================================= the second CTA of a pair: says what has arrived
      // (warp 1: K, warp 2: V)
      const bool is_v = warp == 2;
      int kt = 0;
      bool ok = true;
      while (ok && next_frag(wf, prefix, p)) {
        for (int j = f.t0; ok && j < f.t1; ++j, ++kt) {
          const int st = kt % NST;
          if (!(ok = wait((is_v ? Tr::VF : Tr::KF) + st, static_cast<uint32_t>(kt / NST) & 1u))) break;
          if (lane == 0) arrive_first_cta(bar((is_v ? Tr::VP : Tr::KP) + st));
        }
      }
    } else {
      // ================================================================= MMA issuers, one per stream
      // (issuing, and committing to a barrier, keeps a thread as long as the products before it: two threads keep the
      // tensor cores fed from both streams)
      const int t = warp - 1;
      constexpr uint32_t kIdQK = mma_idesc(Tr::BF16, false, kHalfTile, CG);
      constexpr uint32_t kIdPV = mma_idesc(Tr::BF16, true, D, CG);
      constexpr uint32_t kKDescHi = desc_hi(Tr::KGROUP), kVDescHi = desc_hi(Tr::VGROUP), kQDescHi = desc_hi(1024);
      const uint32_t q_half = static_cast<uint32_t>(stream_rows(a.group)) * 128;  // the query tile is [half][row][128 bytes]
      const uint32_t s_tm = tmem + t * 128, o_tm = tmem + 256 + t * 128;
      int uses = 0, parity = 0, kt = 0;  // query tiles used; tiles before this fragment
      uint32_t pf = 0u;
      bool ok = true;
      while (ok && next_frag(wf, prefix, p)) {
        const int t0 = f.t0, t1 = f.t1;
        const int step = p.paired ? 1 : 2;
        const int j0 = t0 + (p.paired ? 0 : t ^ parity);
        if (!p.paired) parity ^= (t1 - t0) & 1;
        const int kt0 = kt - t0;  // tile j has count kt0 + j
        kt += t1 - t0;
        if (j0 >= t1) continue;
        // S = Q K^T of half a tile, into its half of the stream's columns (a pair of CTAs: 32 positions of each CTA's 64)
        auto issue_qk = [&](int j, int half) -> bool {
          const int st = (kt0 + j) % NST;
          const uint32_t ph = static_cast<uint32_t>((kt0 + j) / NST) & 1u;
          if (half == 0) {
            if (!wait(Tr::KF + st, ph)) return false;
            if (CG == 2 && !wait_pair(Tr::KP + st, ph)) return false;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint32_t qa = desc_lo(base + Tr::OFF_Q + t * Tr::TILE_BYTES);
            const uint32_t kb = desc_lo(base + Tr::OFF_K + st * Tr::STAGE) + half * (kHalfTile / CG / 8 * Tr::KGROUP >> 4);
  #pragma unroll
            for (int s = 0; s < D / 16; ++s) {
              const uint32_t oq = ((s >> 2) * q_half + (s & 3) * 32) >> 4, ok = ((s >> 2) * 1024 + (s & 3) * 32) >> 4;
              tc_mma_ss<CG>(s_tm + half * kHalfTile, qa + oq, kQDescHi, kb + ok, kKDescHi, kIdQK, s > 0);
            }
            tc_commit<CG>(bar(Tr::SF + 2 * half + t));
            if (half) {
              tc_commit<CG>(bar(Tr::KE + st));
              if (j + step >= t1) tc_commit<CG>(bar(Tr::QE + t));
            }
          }
          __syncwarp();
          return true;
        };
        const uint32_t qph = static_cast<uint32_t>(uses++) & 1u;
        if (!(ok = wait(Tr::QF + t, qph))) break;
        if (CG == 2 && !(ok = wait_pair(Tr::QP + t, qph))) break;
        if (!(ok = issue_qk(j0, 0) && issue_qk(j0, 1))) break;
        for (int j = j0; ok && j < t1; j += step, ++pf) {
          const int st = (kt0 + j) % NST;
          const uint32_t ph = static_cast<uint32_t>((kt0 + j) / NST) & 1u;
          if (!(ok = wait(Tr::VF + st, ph))) break;
          if (CG == 2 && !(ok = wait_pair(Tr::VP + st, ph))) break;
  #pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (!(ok = CG == 2 ? wait_pair(Tr::PF + 2 * half + t, pf & 1u) : wait(Tr::PF + 2 * half + t, pf & 1u))) break;
            tc_fence_after();
            if (elect_one()) {
              const uint32_t vb = desc_lo(base + Tr::OFF_V + st * Tr::STAGE);
              const uint32_t pa = s_tm + half * kHalfTile;
  #pragma unroll
              for (int x = 0; x < (SPLIT ? 2 : 1) * (kHalfTile / 16); ++x) {
                const int s = x % (kHalfTile / 16), lo = x / (kHalfTile / 16);
                // 16 positions of the half: in a pair of CTAs its columns are positions 32 half .. and 64 + 32 half ..
                const int row = CG == 1 ? half * kHalfTile + s * 16 : (s >> 1) * kHalfTile + half * 32 + (s & 1) * 16;
                tc_mma_ts<CG>(o_tm, pa + lo * (kHalfTile / 2) + s * 8, vb + (row / 8 * Tr::VGROUP >> 4), kVDescHi, kIdPV,
                              x > 0 || half != 0 || j != j0);
              }
              tc_commit<CG>(bar((half ? Tr::OD : Tr::OH) + t));
              if (half) tc_commit<CG>(bar(Tr::VE + st));
            }
            __syncwarp();
            if (j + step < t1 && !(ok = issue_qk(j + step, half))) break;
          }
        }
      }
    }
  } else if (Tr::B8 && warp >= 12) {
    regs_dec<Tr::REGS_LOW>();
    // ================================================================= 8-bit caches: codes to f16
    if constexpr (Tr::B8) {
      const int tid = static_cast<int>(threadIdx.x) - 384;
      int kt = 0, parity = 0, uses[2] = {0, 0};
      bool ok = true;
      // 16 codes to two 16-byte chunks of f16
      auto widen16 = [&](const uint4& w, uint32_t zp2, uint4& lo, uint4& hi) {
        widen4<KVT>(w.x, zp2, lo.x, lo.y);
        widen4<KVT>(w.y, zp2, lo.z, lo.w);
        widen4<KVT>(w.z, zp2, hi.x, hi.y);
        widen4<KVT>(w.w, zp2, hi.z, hi.w);
      };
      auto done = [&](int full, int raw_empty) {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(full));
          if (raw_empty >= 0) mbar_arrive(bar(raw_empty));
        }
      };
      const int rps = stream_rows(a.group);
      while (ok && next_frag(wf, prefix, p)) {
        uint32_t zk2 = 0u, zv2 = 0u;
        if constexpr (std::is_same<KVT, i8_t>::value) {
          const uint32_t zk = __half_as_ushort(__float2half_rn(1152.f + static_cast<float>(__ldg(a.k_zero_point + f.kvh))));
          const uint32_t zv = __half_as_ushort(__float2half_rn(1152.f + static_cast<float>(__ldg(a.v_zero_point + f.kvh))));
          zk2 = zk | (zk << 16);
          zv2 = zv | (zv << 16);
        }
        const int n = f.t1 - f.t0;
        for (int e = 0; ok && q_widen && e < 2; ++e) {
          const int t = p.paired ? e : e ^ parity;
          if (!p.paired && n <= e) continue;
          if (!(ok = wait(Tr::QL + t, static_cast<uint32_t>(uses[t]) & 1u))) break;
          // one query row per thread: its largest element decides the power of two
          float* const qx = reinterpret_cast<float*>(sm + Tr::OFF_QX) + (t * 2 + (uses[t] & 1)) * kTile;
          ++uses[t];
          if (tid < rps) {
            auto chunk = [&](int c) -> uint4* {
              const uint32_t row = static_cast<uint32_t>(c >> 3) * rps * 128 + tid * 128;  // (tiles are 1024-byte aligned)
              return reinterpret_cast<uint4*>(sm + Tr::OFF_Q + t * Tr::TILE_BYTES + row + (((c & 7) ^ ((row >> 7) & 7)) << 4));
            };
            float top = 0.f;
#pragma unroll 4
            for (int c = 0; c < D / 8; ++c) {
              const uint4 w = *chunk(c);
              const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int i = 0; i < 4; ++i)
                top = fmaxf(top, fmaxf(__uint_as_float((r[i] << 16) & 0x7fffffffu), __uint_as_float(r[i] & 0x7fff0000u)));
            }
            const int ebits = (__float_as_int(top) >> 23) & 0xff;
            const int e2 = top > 0.f ? min(100, max(-100, 141 - ebits)) : 0;
            const float mul = __int_as_float((127 + e2) << 23);
#pragma unroll 4
            for (int c = 0; c < D / 8; ++c) {
              uint4* const at = chunk(c);
              const uint4 w = *at;
              const uint32_t r[4] = {w.x, w.y, w.z, w.w};
              uint32_t h[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float2 x = widen2<bf16_t>(r[i]);
                h[i] = pack2<false>(x.x * mul, x.y * mul);
              }
              *at = make_uint4(h[0], h[1], h[2], h[3]);
            }
            qx[tid] = __int_as_float((127 - e2) << 23);
          }
          done(Tr::QF + t, -1);
        }
        if (!p.paired) parity ^= n & 1;
        for (int j = f.t0; ok && j < f.t1; ++j, ++kt) {
          const int st = kt % NST, r = kt % Tr::NR;
          const uint32_t eph = (static_cast<uint32_t>(kt / NST) & 1u) ^ 1u, rph = static_cast<uint32_t>(kt / Tr::NR) & 1u;
          constexpr int PER = Tr::RAW / 16 / 128;  // 16-byte chunks of codes per thread
          {
            if (!(ok = wait(Tr::RKF + r, rph) && wait(Tr::KE + st, eph))) break;
            uint4 w[PER];
#pragma unroll
            for (int k = 0; k < PER; ++k) w[k] = lds128(base + Tr::OFF_RK + r * Tr::RAW + (k * 128 + tid) * 16);
#pragma unroll
            for (int k = 0; k < PER; ++k) {
              const int x = k * 128 + tid, row = x >> 3, c = 2 * (x & 7);
              uint4 lo, hi;
              widen16(w[k], zk2, lo, hi);
              uint8_t* const to = sm + Tr::OFF_K + st * Tr::STAGE + (row >> 3) * Tr::KGROUP + (c >> 3) * 1024 + (row & 7) * 128;
              *reinterpret_cast<uint4*>(to + (((c & 7) ^ (row & 7)) << 4)) = lo;
              *reinterpret_cast<uint4*>(to + ((((c & 7) + 1) ^ (row & 7)) << 4)) = hi;
            }
            done(Tr::KF + st, Tr::RKE + r);
          }
          {
            if (!(ok = wait(Tr::RVF + r, rph) && wait(Tr::VE + st, eph))) break;
            const int n_hi = f.v.T - j * kTile, n_lo = f.lo - j * kTile;
            uint4 w[PER];
#pragma unroll
            for (int k = 0; k < PER; ++k) w[k] = lds128(base + Tr::OFF_RV + r * Tr::RAW + (k * 128 + tid) * 16);
#pragma unroll
            for (int k = 0; k < PER; ++k) {
              const int x = k * 128 + tid, row = x >> 2, c = 2 * (x & 3);
              uint4 lo, hi;
              widen16(w[k], zv2, lo, hi);
              if (row >= n_hi || row < n_lo) lo = hi = make_uint4(0u, 0u, 0u, 0u);  // outside the sequence or the window
              uint8_t* const to = sm + Tr::OFF_V + st * Tr::STAGE + (row >> 3) * Tr::VGROUP + (row & 7) * 128;
              *reinterpret_cast<uint4*>(to + ((c ^ (row & 7)) << 4)) = lo;
              *reinterpret_cast<uint4*>(to + (((c + 1) ^ (row & 7)) << 4)) = hi;
            }
            done(Tr::VF + st, Tr::RVE + r);
          }
        }
      }
    }
  } else {
    regs_inc<Tr::REGS_HIGH>();
    // ================================================================= softmax, one row per thread
    const int t = (warp - 4) >> 2;
    const int wq = warp & 3;                       // TMEM lanes 32 wq ..
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t ts = tmem + t * 128 + lanes, to = tmem + 256 + t * 128 + lanes;
    constexpr float kLog2e = 1.4426950408889634f;
    // f16 weights carry a factor 2^7 (m is lowered by it), so that weights down to 2^-21 of the largest are normal and none
    // above 2^-32 becomes zero
    constexpr float kLift = Tr::BF16 ? 0.f : 7.f;
    constexpr float kMost = Tr::BF16 ? 256.f : 32768.f;  // 2^(kLift + kSlack): 64 weights of at most 2^kLift stay below it
    int jobs = 0, parity = 0, q_uses = 0;
    uint32_t slot_uses = 0u;  // parity of the uses of the whole segments' record slots, a bit each

    // queries at negative positions (more queries than tokens) see nothing
    for (int s = blockIdx.x; s < S; s += gridDim.x) {
      const SeqView v = seq_view(a, s, false);
      const int64_t n = static_cast<int64_t>(min(v.L, max(0, v.L - v.T))) * a.num_heads * D;
      for (int64_t x = threadIdx.x - 128; x < n; x += 256)
        store_out(a.out, a.out_dtype, static_cast<int64_t>(v.row0) * a.num_heads * D + x, 0.f);
    }

    // the four warps of the stream wait for one another (bounded, unlike a named barrier)
    uint32_t syncs = 0u;
    auto stream_sync = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(Tr::RB + t));
      return wait(Tr::RB + t, syncs++ & 1u);
    };
    bool ok = true;
    while (ok && next_frag(wf, prefix, p)) {
      const int n = f.t1 - f.t0;
      const int e = p.paired ? t : (t ^ parity);    // which of the fragment's contributions this stream makes
      const int step = p.paired ? 1 : 2;
      const int j0 = f.t0 + (p.paired ? 0 : e);
      if (!p.paired) parity ^= n & 1;
      if (j0 >= f.t1) continue;
      const int rps = stream_rows(a.group);
      const int row0 = row_tile(f.m, t) * rps;
      const int rows = min(rps, f.v.L * a.group - row0);  // of this stream (none: the segment's last rows are the other's)
      const int r = row0 + wq * 32 + lane;
      const bool valid = wq * 32 + lane < rows;
      const bool warp_on = wq * 32 < rows;
      const int qi = valid ? r / a.group : 0;
      const int h = f.kvh * a.group + (valid ? r - qi * a.group : 0);
      RowBounds rb = row_bounds(a, f.v, f.prefix, qi);
      if (!valid) rb.lo = rb.hi = 0;
      const int first = f.v.T - f.v.L;              // tree: position of node 0
      const uint64_t* tree = a.tree_mask ? a.tree_mask + (static_cast<int64_t>(f.v.row0) + qi) * a.tree_words : nullptr;
      const float slope2 = a.slopes ? __ldg(a.slopes + h) * kLog2e : 0.f;
      float sc2 = a.scale * kLog2e;
      if constexpr (Tr::B8) sc2 *= __ldg(a.k_scale + f.kvh);
      float capk = a.softcap > 0.f ? 2.f * sc2 / a.softcap : 0.f;
      const float cap2 = a.softcap * kLog2e;
      // (a negative scale would turn the maximum of raw products into a minimum)
      const bool modified = a.softcap > 0.f || a.slopes || !(sc2 >= 0.f);
      float m = -INFINITY, l = 0.f;

      for (int j = j0; ok && j < f.t1; j += step, ++jobs) {
        // Half a tile at a time: while one half's weights are computed, the tensor cores multiply the other's and compute the
        // next tile's scores in its place.
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          if (!wait(Tr::SF + 2 * half + t, static_cast<uint32_t>(jobs) & 1u)) { ok = false; break; }
          tc_fence_after();
          if (q_widen && j == j0 && half == 0) {  // the row's power of two (written before its first scores were computed)
            const float x = reinterpret_cast<const float*>(sm + Tr::OFF_QX)[(t * 2 + (q_uses & 1)) * kTile + wq * 32 + lane];
            sc2 *= x;
            capk *= x;
            ++q_uses;
          }
          if (warp_on) {
            // positions of the half: 32 from tb, 32 from tb + gap on
            const int tb = j * kTile + half * (CG == 1 ? kHalfTile : 32);
            constexpr int kGap = CG == 1 ? 32 : kHalfTile;
            const uint32_t ps = ts + half * kHalfTile;  // the half's scores; its weights replace them (hi, then lo)
            float z[kHalfTile];
#pragma unroll
            for (int c = 0; c < kHalfTile; c += 32) tmem_ld32(ps + c, z + c);
            tmem_wait_ld();
            const bool full = rb.lo <= tb && rb.hi >= tb + kGap + 32 && (!tree || tb + kGap + 32 <= first);
            const bool masked = !__all_sync(0xffffffffu, full || !valid);
            // z: scores in the log2 domain, or (the plain case) raw products that the exponent's FMA scales by mul
            float mul = sc2;
            if (masked || modified) {
              mul = 1.f;
              if (a.softcap > 0.f) {
#pragma unroll
                for (int c = 0; c < kHalfTile; ++c) z[c] = cap2 - __fdividef(2.f * cap2, 1.f + fast_exp2(z[c] * capk));
              } else {
#pragma unroll
                for (int c = 0; c < kHalfTile; c += 2) {
                  const float2 x = fmul2(make_float2(z[c], z[c + 1]), make_float2(sc2, sc2));
                  z[c] = x.x;
                  z[c + 1] = x.y;
                }
              }
              if (a.slopes) {
                const float d0 = static_cast<float>(tb - rb.pos);
#pragma unroll
                for (int c = 0; c < kHalfTile; ++c)
                  z[c] = fmaf(-slope2, fabsf(d0 + static_cast<float>((c >> 5) * kGap + (c & 31))), z[c]);
              }
            }
            if (masked) {
#pragma unroll
              for (int c = 0; c < kHalfTile / 32; ++c) {
                const int b0 = tb + kGap * c;
                // bits [lo, hi) of this 32-position chunk
                const int lo = max(0, min(32, rb.lo - b0)), hi = max(0, min(32, rb.hi - b0));
                uint32_t see = (hi >= 32 ? 0xffffffffu : (1u << hi) - 1u) & (lo >= 32 ? 0u : 0xffffffffu << lo);
                if (tree && valid) see &= tree_bits(tree, a.tree_words, first, b0);
#pragma unroll
                for (int k = 0; k < 32; ++k) z[32 * c + k] = (see >> k) & 1u ? z[32 * c + k] : -INFINITY;
              }
            }
            // Weights against the maximum so far first: after a row's first positions it seldom moves by kSlack (a sum of
            // weights above kMost tells; one below it means no weight is large).  Only then, and for a row that has seen
            // nothing yet, is this half's maximum found, O rescaled and the weights computed again.
            const bool fresh = j == j0 && half == 0;  // nothing multiplied for this fragment yet
            float lt;
#pragma unroll 1
            for (bool again = fresh;; again = true) {
              if (again) {
                float x = fmaxf(z[0], z[1]);
#pragma unroll
                for (int c = 2; c < kHalfTile; c += 2) x = fmax3(x, z[c], z[c + 1]);
                const float mn = fmaxf(m, x * mul);
                const float alpha = mn != -INFINITY ? fast_exp2(m - mn) : 1.f;   // nothing seen before: 2^-inf = 0
                m = mn;
                l *= alpha;
                if (!fresh) {
                  // the products before this half must have left O
                  if (!wait((half ? Tr::OH : Tr::OD) + t, static_cast<uint32_t>(half ? jobs : jobs - 1) & 1u)) ok = false;
                  tc_fence_after();
#pragma unroll 1
                  for (int c = 0; c < D; c += 16) {
                    float o[16];
                    tmem_ld16(to + c, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 16; ++k) o[k] *= alpha;
                    tmem_st16(to + c, reinterpret_cast<const uint32_t*>(o));
                  }
                }
              }
              const float ms = m == -INFINITY ? 0.f : m - kLift;
              const float2 mul2 = make_float2(mul, mul), neg = make_float2(-ms, -ms);
              float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
#pragma unroll
              for (int c = 0; c < kHalfTile / 32; ++c) {
                float2 w[16];
                uint32_t hi[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) w[k] = ffma2(make_float2(z[32 * c + 2 * k], z[32 * c + 2 * k + 1]), mul2, neg);
#pragma unroll
                for (int k = 0; k < 16; ++k) w[k] = make_float2(fast_exp2(w[k].x), fast_exp2(w[k].y));
#pragma unroll
                for (int k = 0; k < 16; k += 2) {
                  sum0 = fadd2(sum0, w[k]);
                  sum1 = fadd2(sum1, w[k + 1]);
                }
#pragma unroll
                for (int k = 0; k < 16; ++k) hi[k] = pack2<Tr::BF16>(w[k].x, w[k].y);
                tmem_st16(ps + 16 * c, hi);
                if constexpr (SPLIT) {
                  uint32_t lo[16];
#pragma unroll
                  for (int k = 0; k < 16; ++k) {
                    const float2 q = unpack2<Tr::BF16>(hi[k]);
                    lo[k] = pack2<Tr::BF16>(w[k].x - q.x, w[k].y - q.y);
                  }
                  tmem_st16(ps + kHalfTile / 2 + 16 * c, lo);
                }
              }
              sum0 = fadd2(sum0, sum1);
              lt = sum0.x + sum0.y;
              if (again || !__any_sync(0xffffffffu, valid && (lt > kMost || m == -INFINITY))) break;
            }
            l += lt;
            tmem_wait_st();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            const uint32_t pf = bar(Tr::PF + 2 * half + t);
            if constexpr (CG == 2) arrive_first_cta(pf); else mbar_arrive(pf);
          }
        }
      }
      if (!ok) break;

      // ---- the stream's part of the fragment is done
      if (!wait(Tr::OD + t, static_cast<uint32_t>(jobs - 1) & 1u)) { ok = false; break; }
      tc_fence_after();
      const float me = m == -INFINITY ? m : m - kLift;  // O and l are relative to 2^me
      const int contributions = p.paired ? 1 : min(2, n);
      if (f.whole && contributions == 1) {
        if (warp_on) {
          float inv = l > 0.f ? 1.f / l : 0.f;
          if constexpr (Tr::B8) inv *= __ldg(a.v_scale + f.kvh);
          bool bad = l != l;
          const int64_t o0 = ((static_cast<int64_t>(f.v.row0) + qi) * a.num_heads + h) * D;
          const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            float o[32];
            tmem_ld32(to + c, o);
            tmem_wait_ld();
            if (valid) {
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                o[k] *= inv;
                bad |= !(fabsf(o[k]) < INFINITY);
              }
              store_row32(a.out, a.out_dtype, o0 + c, o, wide);
            }
          }
          if (__any_sync(0xffffffffu, bad && valid) && lane == 0) atomicOr(misc + kRedo, redo_bits(true, 0, t));
        }
        continue;
      }
      // ---- record, then count in; the last contribution joins them all
      const int slot_kind = slot_kind_of(f.whole, f.idx), slot = slot_kind & 1;
      if (f.whole) {  // the slot's last segment has been joined (by either stream; at once for the slot's first)
        if (!(ok = wait(Tr::JD + slot, ((slot_uses >> slot) & 1u) ^ 1u))) break;
        slot_uses ^= 1u << slot;
      }
      {
        float* const rec = record_at<D>(p, blockIdx.x, slot_kind, e);
        const int lr = wq * 32 + lane;
        if (warp_on) {
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            float o[32];
            tmem_ld32(to + c, o);
            tmem_wait_ld();
            if (valid) {
#pragma unroll
              for (int k = 0; k < 32; k += 8) store32(rec + lr * D + c + k, reinterpret_cast<const uint32_t*>(o + k), true);
            }
          }
          if (valid) *reinterpret_cast<float2*>(rec + p.rec_rows * D + 2 * lr) = make_float2(me, l);
        }
      }
      __threadfence();
      if (!(ok = stream_sync())) break;
      const int c0 = cta_of(f.seg_start + kFragCost, U, nw), c1 = cta_of(f.seg_start + kFragCost + f.seg_tiles - 1, U, nw);
      int total = 0;  // contributions to this stream's rows (paired: its own row tile; alternating: both streams)
      for (int c = c0; c <= c1; ++c) total += p.paired ? 1 : min(2, tiles_in(c, U, nw, f.seg_start, f.seg_tiles));
      // paired: the streams' rows are joined apart (the segment that leaves a CTA unfinished is its last one); alternating:
      // the segment's only rows
      int* const counter = p.paired ? p.counters + (2 * c0 + t) * CG + rank
                                    : p.counters + (f.s * a.num_kv_heads + f.kvh) * CG + rank;
      // (two words in turn: a warp still reading one is not overtaken by the next fragment's arrival)
      volatile int* const arrived = misc + 4 + 2 * (f.idx & 1) + t;
      if ((threadIdx.x & 127) == 0) *arrived = atom_add_acq_rel_gpu(counter, 1);
      if (!(ok = stream_sync())) break;
      const bool last = *arrived == total - 1;
      if (last) {
        __threadfence();
        if (warp_on && join_rows<KVT, D, CG>(p, f, U, nw, c0, c1, rank, t, wq, row0, rows, slot_kind) && lane == 0)
          atomicOr(misc + kRedo, redo_bits(f.whole, slot_kind, t));
        if ((threadIdx.x & 127) == 0) *counter = 0;  // ready for the next call
        if (f.whole) {
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(Tr::JD + slot));
        }
      }
    }

    // ---- rows that are not finite, from the definition: they may owe it to a V row that they do not see.  All fragments
    // are done, and nothing but the end of the kernel waits for these warps.
    named_barrier_sync(1, 256);  // the CTA's rows are stored
    const int redo = *static_cast<volatile int*>(misc + kRedo);
    if (redo != 0) {
      start_frags();
      while (next_frag(wf, prefix, p)) {
        const int rps = stream_rows(a.group), kind = slot_kind_of(f.whole, f.idx);
        for (int x = 0; x < (p.paired ? 2 : 1); ++x) {
          const int bits = redo_bits(f.whole, kind, x) | (p.paired ? 0 : redo_bits(f.whole, kind, 1));
          if ((redo & bits) == 0) continue;
          const int first_row = row_tile(f.m, x) * rps, rows = min(rps, f.v.L * a.group - first_row);
          for (int k = warp - 4; k < rows; k += 8) {
            const int i = (first_row + k) / a.group, h = f.kvh * a.group + (first_row + k) - i * a.group;
            if (row_not_finite<D>(a, (static_cast<int64_t>(f.v.row0) + i) * a.num_heads + h))
              attend_row<KVT, D>(a, f.s, f.v, i, h);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync_all();  // nobody uses the peer's shared memory or TMEM any more
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<CG>(tmem, 512);
  }
}

}  // namespace pa
