// pa_evict.cu - row moves inside the paged cache: the commit of a drafted
// tree's accepted path, and the eviction by accumulated attention weight.
#include "pa_common.cuh"
#include "pa_ops.h"

namespace pa {
namespace {

// Byte offset of the row of position t of (sequence table row, KV head); false
// when the table entry is outside the pool (the error bit is set).
__device__ __forceinline__ bool row_offset(const int32_t* table, int t, int kvh, int Hkv, int B, int shift,
                                           int64_t num_blocks, int row_bytes, unsigned int* err, int64_t* off) {
  const int pb = __ldg(table + (t >> shift));
  if (pb < 0 || pb >= num_blocks) {
    raise_error(err, PA_DEVERR_BLOCK_ID);
    return false;
  }
  *off = ((static_cast<int64_t>(pb) * Hkv + kvh) * B + (t & (B - 1))) * row_bytes;
  return true;
}

// ------------------------------------------------------------------ commit
//
// One CTA per (sequence, KV head, pool).  Source and destination rows of a
// path overlap, so the CTA holds the whole path (at most 256 rows of 256
// bytes, 64 bytes in registers per thread and pass) before it writes.
constexpr int kCommitThreads = 256;
constexpr int kCommitMax = 16;  // 16-byte chunks a thread holds

__global__ void __launch_bounds__(kCommitThreads) commit_tree_kernel(const CommitArgs a) {
  griddep_launch_dependents();
  const int kvh = blockIdx.x, s = blockIdx.y, which = blockIdx.z;
  const int cap = a.max_blocks_per_seq << a.block_shift;
  const int T = a.seq_lens[s];
  const int L = a.q_starts[s + 1] - a.q_starts[s];
  const int n = a.path_lens[s];
  const int first = T - L;
  __shared__ int bad;
  if (threadIdx.x == 0) bad = (T < 0 || T > cap || L < 0 || first < 0 || n < 0 || n > a.max_path || n > L) ? 1 : 0;
  __syncthreads();
  if (!bad) {
    for (int i = threadIdx.x; i < n; i += kCommitThreads) {
      const int node = a.path[static_cast<int64_t>(s) * a.max_path + i];
      if (node < 0 || node >= L) bad = 1;
    }
  }
  __syncthreads();
  if (bad) {
    if (kvh == 0 && which == 0 && threadIdx.x == 0) {
      raise_error(a.err, PA_DEVERR_PATH);
      a.new_lens[s] = T;
    }
    return;
  }
  if (kvh == 0 && which == 0 && threadIdx.x == 0) a.new_lens[s] = first + n;
  uint8_t* cache = static_cast<uint8_t*>(which ? a.v_cache : a.k_cache);
  const int32_t* table = a.block_tables + static_cast<int64_t>(s) * a.max_blocks_per_seq;
  const int chunks = a.row_bytes >> 4, total = n * chunks;
  uint4 held[kCommitMax];
  int64_t at[kCommitMax];
#pragma unroll
  for (int j = 0; j < kCommitMax; ++j) {
    const int x = threadIdx.x + j * kCommitThreads;
    at[j] = -1;
    if (x < total) {
      const int i = x / chunks, c = x - i * chunks;
      const int node = a.path[static_cast<int64_t>(s) * a.max_path + i];
      int64_t src, dst;
      if (node != i &&
          row_offset(table, first + node, kvh, a.num_kv_heads, a.block_size, a.block_shift, a.num_blocks, a.row_bytes,
                     a.err, &src) &&
          row_offset(table, first + i, kvh, a.num_kv_heads, a.block_size, a.block_shift, a.num_blocks, a.row_bytes,
                     a.err, &dst)) {
        held[j] = *reinterpret_cast<const uint4*>(cache + src + 16 * c);
        at[j] = dst + 16 * c;
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kCommitMax; ++j)
    if (at[j] >= 0) *reinterpret_cast<uint4*>(cache + at[j]) = held[j];
}

// ------------------------------------------------------------------ eviction: row moves
//
// A warp moves 32 rows of K and V: its lanes look up one row's source and
// destination each (one round trip for all 32), then row_bytes / 16 lanes copy
// a row 16 bytes each, kMoves of them in flight before the first is stored.
constexpr int kMoves = 8;

__device__ __forceinline__ void move_rows(const EvictArgs& a, int s, int kvh, const int32_t* kept, int i0, int n) {
  const int lane = threadIdx.x & 31;
  const int32_t* table = a.block_tables + static_cast<int64_t>(s) * a.max_blocks_per_seq;
  const int32_t* dtable = a.dst_tables + static_cast<int64_t>(s) * a.max_dst_blocks;
  int64_t src = -1, dst = -1;
  if (i0 + lane < n) {
    if (!row_offset(table, kept[i0 + lane], kvh, a.num_kv_heads, a.block_size, a.block_shift, a.num_blocks, a.row_bytes,
                    a.err, &src) ||
        !row_offset(dtable, i0 + lane, kvh, a.num_kv_heads, a.block_size, a.block_shift, a.num_blocks, a.row_bytes, a.err,
                    &dst))
      dst = -1;
  }
  const int shift = a.row_bytes == 256 ? 4 : (a.row_bytes == 128 ? 3 : 2);  // log2 of the 16-byte chunks of a row
  const int sub = lane >> shift, c = (lane & ((1 << shift) - 1)) * 16, step = 32 >> shift;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    uint8_t* const cache = static_cast<uint8_t*>(which ? a.v_cache : a.k_cache);
    for (int r0 = 0; r0 < 32; r0 += step * kMoves) {
      uint4 held[kMoves];
      int64_t to[kMoves];
#pragma unroll
      for (int k = 0; k < kMoves; ++k) {
        const int r = r0 + step * k + sub;
        const int64_t from = __shfl_sync(0xffffffffu, src, r & 31);
        to[k] = __shfl_sync(0xffffffffu, dst, r & 31);
        if (r >= 32) to[k] = -1;
        if (to[k] >= 0) held[k] = *reinterpret_cast<const uint4*>(cache + from + c);
      }
#pragma unroll
      for (int k = 0; k < kMoves; ++k)
        if (to[k] >= 0) *reinterpret_cast<uint4*>(cache + to[k] + c) = held[k];
    }
  }
}

constexpr int kGatherWarps = 4;

__global__ void __launch_bounds__(kGatherWarps * 32) evict_gather_kernel(const EvictArgs a) {
  griddep_wait();
  const int s = blockIdx.z, kvh = blockIdx.y;
  const int cap = a.max_blocks_per_seq << a.block_shift;
  const int n = min(max(0, min(a.seq_lens[s], cap)), a.budget);
  const int i0 = (blockIdx.x * kGatherWarps + (threadIdx.x >> 5)) * 32;
  if (i0 >= n) return;
  move_rows(a, s, kvh, a.kept + (static_cast<int64_t>(s) * a.num_kv_heads + kvh) * a.budget, i0, n);
}

// ------------------------------------------------------------------ eviction: selection
//
// One CTA per (sequence, KV head), each warp a contiguous part of its
// positions.  A weight's key is an unsigned integer with the same order: minus
// zero counts as zero, NaN (1) stands below minus infinity, the always-kept
// positions stand above everything, and no position (0) below it.  So the kept
// positions are those of the `budget` largest keys.  The key of that rank is
// narrowed down 11 bits at a time by a histogram in shared memory; as soon as
// the keys that share the leading digits fit the CTA, one per thread, its
// remaining bits follow from one count over the CTA each (and none are needed
// when all of those are kept).  Then each warp counts what it keeps, and after
// one scan over the warps writes its kept positions in order: those above the
// key, and the first `ties` equal to it.  Up to 32768 positions the keys are
// made once and stay in registers; beyond, the weights are read again (from L2)
// in each pass.
// (Moving few rows in the same CTA instead of a second, overlapping launch was
// slower: 21.9 against 18 us for 256 rows of 32 pairs.)
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelHeld = 32;  // keys a thread holds, or has in flight
constexpr int kBins = 2048;
constexpr uint32_t kAlways = 0xffffffffu;

__device__ __forceinline__ uint32_t weight_key(float x) {
  if (x != x) return 1u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
  griddep_launch_dependents();
  const int kvh = blockIdx.x, s = blockIdx.y;
  const int cap = a.max_blocks_per_seq << a.block_shift;
  int T = a.seq_lens[s];
  if (T < 0 || T > cap) {
    if (kvh == 0 && threadIdx.x == 0) raise_error(a.err, PA_DEVERR_SEQ_LEN);
    T = T < 0 ? 0 : cap;
  }
  const float* mass = a.mass + s * a.mass_stride_seq + kvh * a.mass_stride_head;
  int32_t* kept = a.kept + (static_cast<int64_t>(s) * a.num_kv_heads + kvh) * a.budget;
  float* mass_out = a.mass_out + (static_cast<int64_t>(s) * a.num_kv_heads + kvh) * a.budget;
  if (kvh == 0 && threadIdx.x == 0) a.new_lens[s] = min(T, a.budget);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (T <= a.budget) {
    for (int t = threadIdx.x; t < T; t += kSelThreads) {
      kept[t] = t;
      mass_out[t] = mass[t];
    }
    return;
  }
  __shared__ int hist[kBins];
  __shared__ uint32_t few[kSelThreads];
  __shared__ int wsum[2][kSelWarps];
  __shared__ int pick[3], num_few;
  const int lo = a.sinks, hi = T - a.recent;  // outside: always kept
  // this warp's positions [w0, w1): a multiple of 32, lane l holding w0 + 32 k + l
  const int part = ((T + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int w0 = min(T, warp * part), w1 = min(T, w0 + part);
  const bool held = part <= 32 * kSelHeld;
  uint32_t y[kSelHeld];
  auto fetch = [&](int t0) {
    float x[kSelHeld];
#pragma unroll
    for (int k = 0; k < kSelHeld; ++k) {
      const int t = t0 + 32 * k + lane;
      x[k] = t < w1 ? __ldg(mass + t) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kSelHeld; ++k) {
      const int t = t0 + 32 * k + lane;
      y[k] = t >= w1 ? 0u : (t < lo || t >= hi) ? kAlways : weight_key(x[k]);
    }
  };
  if (held) fetch(w0);
  // body(key, position of the chunk's first lane) over the warp's positions, a chunk of 32 at a time
  auto each = [&](auto body) {
#pragma unroll 1
    for (int t0 = w0; t0 < w1; t0 += 32 * kSelHeld) {
      if (!held) fetch(t0);
#pragma unroll
      for (int k = 0; k < kSelHeld; ++k)
        if (t0 + 32 * k < w1) body(y[k], t0 + 32 * k);
    }
  };
  // the key: everything above `key` is kept, and `ties` of those equal to it
  uint32_t key = 0u, prefix = 0u, mask = 0u;
  int ties = 0, need = a.budget, shift = 21;
#pragma unroll 1
  for (int digit = 0; digit < 3; ++digit) {
    const uint32_t dmask = digit < 2 ? 0x7ffu : 0x3ffu;
    for (int i = threadIdx.x; i < kBins; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    each([&](uint32_t v, int) {
      if ((v & mask) == prefix) atomicAdd(&hist[(v >> shift) & dmask], 1);
    });
    __syncthreads();
    // thread i holds bins kBins - 1 - 2 i and the one below: the digit is the first from above that brings the count to need
    {
      const int b = kBins - 1 - 2 * static_cast<int>(threadIdx.x);
      const int c0 = hist[b], c1 = hist[b - 1];
      int upto = c0 + c1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      if (lane == 31) wsum[0][warp] = upto;
      __syncthreads();
      int w = lane < warp ? wsum[0][lane] : 0;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
      const int before = w + upto - c0 - c1;
      if (before < need && need <= before + c0 + c1) {
        const bool first = need <= before + c0;
        pick[0] = first ? b : b - 1;
        pick[1] = need - before - (first ? 0 : c0);  // still to be found in the bin
        pick[2] = first ? c0 : c1;                   // its size
      }
      if (threadIdx.x == 0) num_few = 0;
      __syncthreads();
    }
    prefix |= static_cast<uint32_t>(pick[0]) << shift;
    mask |= dmask << shift;
    need = pick[1];
    const int size = pick[2];
    if (need == size) {  // all of them: everything from prefix on (not all positions are kept, so prefix > 0 here)
      key = prefix - 1u;
      ties = 0;
      break;
    }
    if (digit == 2) {
      key = prefix;
      ties = need;
      break;
    }
    if (size <= kSelThreads) {
      each([&](uint32_t v, int) {
        if ((v & mask) == prefix) {
          const int at = atomicAdd(&num_few, 1);
          if (at < kSelThreads) few[at] = v;  // (lanes past the end hold 0 and may add to the lowest bin)
        }
      });
      __syncthreads();
      const bool mine = static_cast<int>(threadIdx.x) < size;
      const uint32_t v = mine ? few[threadIdx.x] : 0u;
      // the largest value of the remaining bits with at least `need` keys from it on
#pragma unroll 1
      for (int b = shift - 1; b >= 0; --b) {
        const uint32_t with = prefix | (1u << b);
        if (__syncthreads_count(mine && v >= with) >= need) prefix = with;
      }
      key = prefix;
      ties = need - __syncthreads_count(mine && v > key);
      break;
    }
    shift = digit == 0 ? 10 : 0;
  }
  int sure = 0, equal = 0;
  each([&](uint32_t v, int) {
    sure += __popc(__ballot_sync(0xffffffffu, v > key));
    equal += __popc(__ballot_sync(0xffffffffu, v == key));
  });
  __syncthreads();  // wsum is free
  if (lane == 0) {
    wsum[0][warp] = sure;
    wsum[1][warp] = equal;
  }
  __syncthreads();
  int s0 = lane < warp ? wsum[0][lane] : 0, e0 = lane < warp ? wsum[1][lane] : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s0 += __shfl_xor_sync(0xffffffffu, s0, o);
    e0 += __shfl_xor_sync(0xffffffffu, e0, o);
  }
  const unsigned below = (1u << lane) - 1u;
  each([&](uint32_t v, int t0) {
    const bool above = v > key, same = v == key;
    const unsigned by = __ballot_sync(0xffffffffu, above), be = __ballot_sync(0xffffffffu, same);
    if (by | be) {
      const int eq = e0 + __popc(be & below);  // equal ones before this position
      if (above || (same && eq < ties)) {
        const int at = s0 + __popc(by & below) + min(eq, ties);
        kept[at] = t0 + lane;
        mass_out[at] = __ldg(mass + t0 + lane);
      }
      s0 += __popc(by);
      e0 += __popc(be);
    }
  });
}

}  // namespace

cudaError_t launch_commit_tree(const CommitArgs& a, cudaStream_t stream) {
  (void)cudaGetLastError();
  commit_tree_kernel<<<dim3(a.num_kv_heads, a.num_seqs, 2), kCommitThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream) {
  (void)cudaGetLastError();
  const int cap = a.max_blocks_per_seq << a.block_shift;
  const int rows = a.budget < cap ? a.budget : cap;
  evict_select_kernel<<<dim3(a.num_kv_heads, a.num_seqs), kSelThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // the moves may be set up while the selection runs; they wait for it before they read
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((rows + kGatherWarps * 32 - 1) / (kGatherWarps * 32), a.num_kv_heads, a.num_seqs);
  cfg.blockDim = dim3(kGatherWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, evict_gather_kernel, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace pa
