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
// bits a pass, from histograms in shared memory; then one ordered pass writes
// the kept positions: those above the key, and the first `ties` equal to it.
constexpr int kSelThreads = 1024;

__device__ __forceinline__ uint32_t weight_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
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
  const int lo = a.sinks, hi = T - a.recent;  // the middle positions
  int need = a.budget - a.sinks - a.recent;   // < hi - lo
  __shared__ int hist[256];
  __shared__ int pick[2];
  uint32_t prefix = 0u, mask = 0u;
  if (need > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = threadIdx.x; i < 256; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int t = lo + threadIdx.x; t < hi; t += kSelThreads) {
        const uint32_t k = weight_key(mass[t]);
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1);
      }
      __syncthreads();
      if (threadIdx.x == 0) {
        int left = need, d = 255;
        while (hist[d] < left) left -= hist[d--];
        pick[0] = d;
        pick[1] = left;
      }
      __syncthreads();
      prefix |= static_cast<uint32_t>(pick[0]) << shift;
      mask |= 255u << shift;
      need = pick[1];
      __syncthreads();
    }
  }
  const int ties = need;  // how many of the middle positions equal to the key are kept
  const bool any = a.budget > a.sinks + a.recent;
  // ordered pass: (kept, equal) counts scanned over the CTA, 1024 positions at a time
  __shared__ int wsum[32];
  int base = 0, eq_base = 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int t0 = 0; t0 < T; t0 += kSelThreads) {
    const int t = t0 + threadIdx.x;
    bool sure = false, equal = false;
    float x = 0.f;
    if (t < T) {
      x = mass[t];
      if (t < lo || t >= hi) {
        sure = true;
      } else if (any) {
        const uint32_t k = weight_key(x);
        sure = k > prefix;
        equal = k == prefix;
      }
    }
    // equal ones before this position
    const unsigned be = __ballot_sync(0xffffffffu, equal), bs = __ballot_sync(0xffffffffu, sure);
    if (lane == 0) wsum[warp] = __popc(be) | (__popc(bs) << 16);
    __syncthreads();
    int eq = eq_base, eq_all = 0, su = 0, su_all = 0;
    for (int w = 0; w < 32; ++w) {
      const int e = wsum[w] & 0xffff, k = wsum[w] >> 16;
      if (w < warp) {
        eq += e;
        su += k;
      }
      eq_all += e;
      su_all += k;
    }
    eq += __popc(be & ((1u << lane) - 1u));
    su += __popc(bs & ((1u << lane) - 1u));
    const bool keep = sure || (equal && eq < ties);
    if (keep) {
      const int at = base + su + min(eq, ties) - min(eq_base, ties);
      kept[at] = t;
      mass_out[at] = x;
    }
    base += su_all + min(eq_base + eq_all, ties) - min(eq_base, ties);
    eq_base += eq_all;
    __syncthreads();
  }
}

// ------------------------------------------------------------------ eviction: row moves
//
// 16 bytes per thread: a row is row_bytes / 16 neighbouring threads.
constexpr int kGatherThreads = 256;

__global__ void __launch_bounds__(kGatherThreads) evict_gather_kernel(const EvictArgs a) {
  const int s = blockIdx.z, kvh = blockIdx.y >> 1, which = blockIdx.y & 1;
  const int cap = a.max_blocks_per_seq << a.block_shift;
  const int n = min(max(0, min(a.seq_lens[s], cap)), a.budget);
  const int chunks = a.row_bytes >> 4;
  uint8_t* cache = static_cast<uint8_t*>(which ? a.v_cache : a.k_cache);
  const int32_t* kept = a.kept + (static_cast<int64_t>(s) * a.num_kv_heads + kvh) * a.budget;
  const int32_t* table = a.block_tables + static_cast<int64_t>(s) * a.max_blocks_per_seq;
  const int32_t* dtable = a.dst_tables + static_cast<int64_t>(s) * a.max_dst_blocks;
  for (int x = blockIdx.x * kGatherThreads + threadIdx.x; x < n * chunks; x += gridDim.x * kGatherThreads) {
    const int i = x / chunks, c = x - i * chunks;
    int64_t src, dst;
    if (row_offset(table, kept[i], kvh, a.num_kv_heads, a.block_size, a.block_shift, a.num_blocks, a.row_bytes, a.err,
                   &src) &&
        row_offset(dtable, i, kvh, a.num_kv_heads, a.block_size, a.block_shift, a.num_blocks, a.row_bytes, a.err,
                   &dst))
      *reinterpret_cast<uint4*>(cache + dst + 16 * c) = *reinterpret_cast<const uint4*>(cache + src + 16 * c);
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
  evict_select_kernel<<<dim3(a.num_kv_heads, a.num_seqs), kSelThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int cap = a.max_blocks_per_seq << a.block_shift;
  const int64_t work = static_cast<int64_t>(a.budget < cap ? a.budget : cap) * (a.row_bytes >> 4);
  const int64_t gx = (work + kGatherThreads - 1) / kGatherThreads;
  evict_gather_kernel<<<dim3(static_cast<unsigned>(gx < 1024 ? gx : 1024), 2 * a.num_kv_heads, a.num_seqs), kGatherThreads,
                        0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace pa
