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

// ------------------------------------------------------------------ eviction: selection
//
// One CTA per (sequence, KV head).  A weight's key is an unsigned integer with
// the same order (NaN: 0, below minus infinity; minus zero counts as zero).
// The key of rank `need` among the middle positions is found digit by digit, 8
// bits a pass, from histograms in shared memory; then each warp takes a
// contiguous part of the positions, counts what it keeps, and after one scan
// over the warps writes its kept positions: those above the key, and the first
// `ties` equal to it.
//
// Weights share few leading digits (a handful of exponents), so lanes of one
// warp would queue at the same counter: every lane has a column of counters of
// its own, on its own bank.
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelUnroll = 8;  // weights a thread has in flight

__device__ __forceinline__ uint32_t weight_key(float x) {
  if (x != x) return 0u;
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
  if (T <= a.budget) {
    for (int t = threadIdx.x; t < T; t += kSelThreads) {
      kept[t] = t;
      mass_out[t] = mass[t];
    }
    return;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lo = a.sinks, hi = T - a.recent;  // the middle positions
  int need = a.budget - a.sinks - a.recent;   // < hi - lo
  const bool any = need > 0;
  extern __shared__ int hist[];               // [256][32]
  __shared__ int bin[256];
  __shared__ int pick[2];
  uint32_t prefix = 0u, mask = 0u;
  if (any) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = threadIdx.x; i < 256 * 32; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int t0 = lo + static_cast<int>(threadIdx.x); t0 < hi; t0 += kSelThreads * kSelUnroll) {
        float x[kSelUnroll];
#pragma unroll
        for (int k = 0; k < kSelUnroll; ++k) {
          const int t = t0 + k * kSelThreads;
          x[k] = t < hi ? __ldg(mass + t) : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kSelUnroll; ++k) {
          const uint32_t key = weight_key(x[k]);
          if (t0 + k * kSelThreads < hi && (key & mask) == prefix) atomicAdd(&hist[((key >> shift) & 255u) * 32 + lane], 1);
        }
      }
      __syncthreads();
      for (int b = warp; b < 256; b += kSelWarps) {  // a bin's 32 columns
        int c = hist[b * 32 + lane];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
        if (lane == 0) bin[b] = c;
      }
      __syncthreads();
      if (warp == 0) {
        // lane i holds the bins 255 - 8 i .. 248 - 8 i: the digit is the first, from above, that brings the count to `need`
        int c[8], sum = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          c[k] = bin[255 - 8 * lane - k];
          sum += c[k];
        }
        int before = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, before, o);
          if (lane >= o) before += y;
        }
        before -= sum;
        if (before < need && need <= before + sum) {
          int left = need - before;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if (left > 0 && left <= c[k]) {
              pick[0] = 255 - 8 * lane - k;
              pick[1] = left;
            }
            left -= c[k];
          }
        }
      }
      __syncthreads();
      prefix |= static_cast<uint32_t>(pick[0]) << shift;
      mask |= 255u << shift;
      need = pick[1];
    }
  }
  const int ties = need;  // how many of the middle positions equal to the key are kept
  // each warp: positions [w0, w1), a multiple of 32 long
  const int part = ((T + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int w0 = min(T, warp * part), w1 = min(T, w0 + part);
  auto classify = [&](int t, float x, bool* equal) -> bool {
    *equal = false;
    if (t >= w1) return false;
    if (t < lo || t >= hi) return true;
    if (!any) return false;
    const uint32_t k = weight_key(x);
    *equal = k == prefix;
    return k > prefix;
  };
  int sure = 0, equal = 0;
  for (int t0 = w0; t0 < w1; t0 += 32 * kSelUnroll) {
    float x[kSelUnroll];
#pragma unroll
    for (int k = 0; k < kSelUnroll; ++k) {
      const int t = t0 + 32 * k + lane;
      x[k] = t < w1 ? __ldg(mass + t) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kSelUnroll; ++k) {
      bool e;
      const bool y = classify(t0 + 32 * k + lane, x[k], &e);
      sure += __popc(__ballot_sync(0xffffffffu, y));
      equal += __popc(__ballot_sync(0xffffffffu, e));
    }
  }
  __shared__ int wsure[kSelWarps], wequal[kSelWarps];
  if (lane == 0) {
    wsure[warp] = sure;
    wequal[warp] = equal;
  }
  __syncthreads();
  int s0 = lane < warp ? wsure[lane] : 0, e0 = lane < warp ? wequal[lane] : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s0 += __shfl_xor_sync(0xffffffffu, s0, o);
    e0 += __shfl_xor_sync(0xffffffffu, e0, o);
  }
  for (int t0 = w0; t0 < w1; t0 += 32 * kSelUnroll) {
    float x[kSelUnroll];
#pragma unroll
    for (int k = 0; k < kSelUnroll; ++k) {
      const int t = t0 + 32 * k + lane;
      x[k] = t < w1 ? __ldg(mass + t) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kSelUnroll; ++k) {
      const int t = t0 + 32 * k + lane;
      bool e;
      const bool y = classify(t, x[k], &e);
      const unsigned by = __ballot_sync(0xffffffffu, y), be = __ballot_sync(0xffffffffu, e);
      const unsigned below = (1u << lane) - 1u;
      const int eq = e0 + __popc(be & below);  // equal ones before this position
      if (y || (e && eq < ties)) {
        const int at = s0 + __popc(by & below) + min(eq, ties);
        kept[at] = t;
        mass_out[at] = x[k];
      }
      s0 += __popc(by);
      e0 += __popc(be);
    }
  }
}

// ------------------------------------------------------------------ eviction: row moves
//
// A warp moves 32 rows of K and V: its lanes look up one row's source and
// destination each (one round trip for all 32), then row_bytes / 16 lanes copy
// a row 16 bytes each, kMoves of them in flight before the first is stored.
constexpr int kGatherWarps = 4;
constexpr int kMoves = 8;

__global__ void __launch_bounds__(kGatherWarps * 32) evict_gather_kernel(const EvictArgs a) {
  griddep_wait();
  const int s = blockIdx.z, kvh = blockIdx.y;
  const int cap = a.max_blocks_per_seq << a.block_shift;
  const int n = min(max(0, min(a.seq_lens[s], cap)), a.budget);
  const int lane = threadIdx.x & 31;
  const int i0 = (blockIdx.x * kGatherWarps + (threadIdx.x >> 5)) * 32;
  if (i0 >= n) return;
  const int32_t* kept = a.kept + (static_cast<int64_t>(s) * a.num_kv_heads + kvh) * a.budget;
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
  const int shift = a.row_bytes == 256 ? 4 : 3;  // log2 of the 16-byte chunks of a row
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

}  // namespace

cudaError_t launch_commit_tree(const CommitArgs& a, cudaStream_t stream) {
  (void)cudaGetLastError();
  commit_tree_kernel<<<dim3(a.num_kv_heads, a.num_seqs, 2), kCommitThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream) {
  (void)cudaGetLastError();
  evict_select_kernel<<<dim3(a.num_kv_heads, a.num_seqs), kSelThreads, 256 * 32 * sizeof(int), stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // the moves may be set up while the selection runs; they wait for it before they read
  const int cap = a.max_blocks_per_seq << a.block_shift;
  const int rows = a.budget < cap ? a.budget : cap;
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
