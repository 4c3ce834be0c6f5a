// pa_evict.cu - row moves inside the paged cache: the commit of a drafted
// tree's accepted path, and the eviction by accumulated attention weight.
#include <type_traits>

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
// What bounds it: memory traffic.  4096 rows of 8 x 8 pairs, 256 bytes each, K
// and V: 42 us for 268 MB read and written, of which DRAM moves 222 MB in that
// time (5.2 TB/s; the last writes leave L2 later).  256 or 512 rows of 4 x 8
// pairs: 11 us from a cold cache, its chain of dependent reads (kept position,
// table, row).
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
// One CTA per (sequence, KV head), or a cluster of them when there are few
// pairs and many positions; each warp has a contiguous part of the positions.
// A weight's key is an unsigned integer with the same order: minus zero counts
// as zero, NaN (1) stands below minus infinity, and the always-kept positions
// stand above everything.  So the kept positions are those of the `budget`
// largest keys.  The key of that rank is narrowed down 11 bits at a time by a
// histogram in shared memory; as soon as the keys that share the leading digits
// fit the CTA, one per thread, the other positions are left out of the next
// digits (and none are needed when all of those are kept).  Then each warp
// counts what it keeps, and after one scan over the warps writes its kept
// positions in order: those above the key, and the first `ties` equal to it.
// CTAs of a cluster exchange their histograms and their warps' counts; all of
// them find the same key.
//
// The keys of a CTA's first kSelHeld positions are made once and stay in shared
// memory; beyond, the weights are read again (from L2) in each pass.  (Keys in
// registers took the same passes unrolled 32 times, whose code alone, fetched
// once per launch, cost microseconds: 16.4 against 12.5 us for 4 x 8 pairs of
// 300 to 1100 positions with their moves.)
//
// What bounds it: the chain of passes and barriers in few CTAs.  4 x 8 pairs of
// 300 to 1100 positions: 7.2 us, of 4096: 8.3 us; 8 x 8 pairs of 32768 positions:
// 24 us in one CTA each, 18 us in two.  (Moving few rows in the same CTA instead of a
// second, overlapping launch was slower: 21.9 against 18 us for 256 rows of 32
// pairs, at the time.)
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelHeld = 48 * 1024;
constexpr int kBins = 2048;
constexpr uint32_t kAlways = 0xffffffffu;

__device__ __forceinline__ uint32_t weight_key(float x) {
  if (x != x) return 1u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ int2 ld_cluster2(const int* p, uint32_t rank) {
  int2 v;
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(cluster_addr(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

template <bool CLUSTER>
__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(const EvictArgs a) {
  griddep_launch_dependents();
  uint32_t rank = 0, ctas = 1;
  if constexpr (CLUSTER) {
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
  }
  const int kvh = blockIdx.x / ctas, s = blockIdx.y;
  const int cap = a.max_blocks_per_seq << a.block_shift;
  int T = a.seq_lens[s];
  if (T < 0 || T > cap) {
    if (blockIdx.x == 0 && threadIdx.x == 0) raise_error(a.err, PA_DEVERR_SEQ_LEN);
    T = T < 0 ? 0 : cap;
  }
  const float* mass = a.mass + s * a.mass_stride_seq + kvh * a.mass_stride_head;
  int32_t* kept = a.kept + (static_cast<int64_t>(s) * a.num_kv_heads + kvh) * a.budget;
  float* mass_out = a.mass_out + (static_cast<int64_t>(s) * a.num_kv_heads + kvh) * a.budget;
  if (blockIdx.x == 0 && threadIdx.x == 0) a.new_lens[s] = min(T, a.budget);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (T <= a.budget) {
    for (int t = rank * kSelThreads + threadIdx.x; t < T; t += ctas * kSelThreads) {
      kept[t] = t;
      mass_out[t] = mass[t];
    }
    return;
  }
  extern __shared__ __align__(16) uint32_t keys[];  // of the CTA's first kSelHeld positions
  __shared__ __align__(16) int hists[CLUSTER ? 3 : 1][kBins];  // (the other CTAs may still read the last digit's)
  __shared__ uint32_t few[kSelThreads];
  __shared__ int wsum[kSelWarps];
  __shared__ int2 counts[kSelWarps];
  __shared__ int pick[3], num_few;
  const int lo = a.sinks, hi = T - a.recent;  // outside: always kept
  // this warp's positions [w0, w1); lane l takes w0 + 32 k + l
  const int part = (T + ctas * kSelThreads - 1) / (ctas * kSelThreads) * 32;
  const int c0 = rank * kSelWarps * part, held = c0 + kSelHeld;
  const int w0 = min(T, c0 + warp * part), w1 = min(T, w0 + part);
  for (int t = w0 + lane; t < min(w1, held); t += 32)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(keys + (t - c0))), "l"(mass + t) : "memory");
  for (int i = threadIdx.x; i < (CLUSTER ? 3 : 1) * kBins; i += kSelThreads) hists[0][i] = 0;
  if (threadIdx.x == 0) num_few = 0;
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  auto sync_all = [&] {  // the CTAs that share the positions
    if constexpr (CLUSTER) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
  };
  auto key_of = [&](int t, float x) { return t < lo || t >= hi ? kAlways : weight_key(x); };
  // body(position, key) over the warp's positions; made: the keys stand in shared memory
  auto each = [&](auto made, auto body) {
    const int in_shared = min(w1, held);
    uint32_t* const at = keys - c0;
#pragma unroll 8
    for (int t = w0 + lane; t < in_shared; t += 32) {
      if constexpr (decltype(made)::value) {
        body(t, at[t]);
      } else {
        const uint32_t v = key_of(t, __uint_as_float(at[t]));
        at[t] = v;
        body(t, v);
      }
    }
#pragma unroll 1
    for (int t = max(w0, held) + lane; t < w1; t += 32) body(t, key_of(t, __ldg(mass + t)));
  };
  // the key: everything above `key` is kept, and `ties` of those equal to it
  uint32_t key = 0u, prefix = 0u, mask = 0u, own = 0u;
  int ties = 0, need = a.budget;
  bool small = false, mine = false;  // the keys that are left are one per thread (its own, if `mine`)
#pragma unroll 1
  for (int digit = 0; digit < 3; ++digit) {
    const uint32_t dmask = digit < 2 ? 0x7ffu : 0x3ffu;
    const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0;
    int* const hist = hists[CLUSTER ? digit : 0];
    if (digit == 0) {
      each(std::false_type(), [&](int, uint32_t v) { atomicAdd(&hist[v >> 21], 1); });
    } else if (small) {
      if (mine && (own & mask) == prefix) atomicAdd(&hist[(own >> shift) & dmask], 1);
    } else {
      each(std::true_type(), [&](int, uint32_t v) {
        if ((v & mask) == prefix) atomicAdd(&hist[(v >> shift) & dmask], 1);
      });
    }
    sync_all();
    // thread i holds bins kBins - 1 - 2 i and the one below: the digit is the first from above that brings the count to need
    const int b = kBins - 1 - 2 * static_cast<int>(threadIdx.x);
    int n0 = hist[b], n1 = hist[b - 1];
    if constexpr (CLUSTER) {
      for (uint32_t r = 1; r < ctas; ++r) {
        const int2 n = ld_cluster2(&hist[b - 1], (rank + r) % ctas);
        n0 += n.y;
        n1 += n.x;
      }
    } else {
      hist[b] = hist[b - 1] = 0;
    }
    int upto = n0 + n1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) wsum[warp] = upto;
    __syncthreads();
    const int before = __reduce_add_sync(0xffffffffu, lane < warp ? wsum[lane] : 0) + upto - n0 - n1;
    if (before < need && need <= before + n0 + n1) {
      const bool first = need <= before + n0;
      pick[0] = first ? b : b - 1;
      pick[1] = need - before - (first ? 0 : n0);  // still to be found in the bin
      pick[2] = first ? n0 : n1;                   // its size
    }
    __syncthreads();
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
    if (!small && size <= kSelThreads) {
      each(std::true_type(), [&](int, uint32_t v) {
        if ((v & mask) == prefix) few[atomicAdd(&num_few, 1)] = v;
      });
      __syncthreads();
      small = true;
      mine = static_cast<int>(threadIdx.x) < num_few;
      own = mine ? few[threadIdx.x] : 0u;
    }
  }
  int sure = 0, equal = 0;
  each(std::true_type(), [&](int, uint32_t v) {
    sure += v > key ? 1 : 0;
    equal += v == key ? 1 : 0;
  });
  sure = __reduce_add_sync(0xffffffffu, sure);
  equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 0) counts[warp] = make_int2(sure, equal);
  sync_all();
  // what the warps before this one, in its CTA and in those before, keep
  int2 n = lane < warp ? counts[lane] : make_int2(0, 0);
  for (uint32_t r = 0; CLUSTER && r < rank; ++r) {
    const int2 v = ld_cluster2(reinterpret_cast<const int*>(counts + lane), r);
    n.x += v.x;
    n.y += v.y;
  }
  int s0 = __reduce_add_sync(0xffffffffu, n.x), e0 = __reduce_add_sync(0xffffffffu, n.y);
  if constexpr (CLUSTER) cluster_arrive();  // the others' shared memory has been read
  const unsigned below = (1u << lane) - 1u;
#pragma unroll 4
  for (int t0 = w0; t0 < w1; t0 += 32) {
    const int t = t0 + lane;
    const uint32_t v = t >= w1 ? 0u : t < held ? keys[t - c0] : key_of(t, __ldg(mass + t));
    const bool above = v > key, same = t < w1 && v == key;
    const unsigned by = __ballot_sync(0xffffffffu, above), be = __ballot_sync(0xffffffffu, same);
    const int eq = e0 + __popc(be & below);  // equal ones before this position
    if (above || (same && eq < ties)) {
      const int at = s0 + __popc(by & below) + min(eq, ties);
      kept[at] = t;
      // the key gives the weight back, but for the always-kept and NaN
      mass_out[at] = v == kAlways || v == 1u ? __ldg(mass + t)
                                             : __uint_as_float(v ^ ((v >> 31) ? 0x80000000u : 0xffffffffu));
    }
    s0 += __popc(by);
    e0 += __popc(be);
  }
  if constexpr (CLUSTER) cluster_wait();
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
  // CTAs that share a pair: up to 8192 positions each while the device has SMs for all (a CTA fills one), and as many as
  // hold all keys.  A cluster costs about 4 us to start, so none up to 16384 positions.  Both kernels in us with clusters
  // of 1 / 2 / 4 / 8, positions x pairs to kept rows: 32768 x 32 to 4096 57 / 52 / 50 / 65, 32768 x 64 to 4096
  // 77 / 73 / 77 / 101, 16384 x 32 to 1024 30 / 30 / 31 / 40, 131072 x 8 to 4096 212 / 118 / 46 / 42.
  const int64_t pairs = static_cast<int64_t>(a.num_kv_heads) * a.num_seqs;
  int ctas = 1;
  cudaError_t e = cudaSuccess;
  if (cap > 2 * 8192) {
    int dev = 0, sms = 0;
    e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    while (ctas < 8 && ((cap / ctas > 8192 && 2 * ctas * pairs <= sms) || cap / ctas > kSelHeld)) ctas *= 2;
  }
  const int most = cap / ctas + kSelThreads;  // positions of a CTA
  auto* const select = ctas > 1 ? evict_select_kernel<true> : evict_select_kernel<false>;
  cudaLaunchConfig_t sel = {};
  sel.gridDim = dim3(a.num_kv_heads * ctas, a.num_seqs);
  sel.blockDim = dim3(kSelThreads);
  sel.dynamicSmemBytes = (most < kSelHeld ? most : kSelHeld) * sizeof(uint32_t);
  sel.stream = stream;
  if (ctas > 1 || sel.dynamicSmemBytes > 32 * 1024) {  // with the 13 KB that are static, up to 48 KB need no leave
    e = cudaFuncSetAttribute(select, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelHeld * 4);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute cluster[1];
  cluster[0].id = cudaLaunchAttributeClusterDimension;
  cluster[0].val.clusterDim.x = ctas;
  cluster[0].val.clusterDim.y = cluster[0].val.clusterDim.z = 1;
  sel.attrs = cluster;
  sel.numAttrs = ctas > 1 ? 1 : 0;
  e = cudaLaunchKernelEx(&sel, select, a);
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
