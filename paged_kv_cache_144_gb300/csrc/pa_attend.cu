// pa_attend.cu - attention of ragged query rows over the paged cache with
// score modifiers, and the accumulation of each cached position's weight.
#include <cstring>

#include "pa_attend_tc.cuh"

namespace pa {
namespace {

// Which kernel serves a call, by its rows (queries x query heads per KV head) and by the table's positions over all
// sequences and KV heads.  The decode kernel's variants read the cache once per 16 rows; the tensor-core kernel's time hardly
// depends on the rows below 128, but has about 50 us of start and joins, and widens 8-bit codes.  Measured, head size 128,
// lengths of 1/2 to 1 of the table, decode kernel / tensor cores, us:
//   bf16, 2^20 positions: 32 rows 120 / 153, 48 rows 162 / 156, 64 rows 236 / 157;  2^21: 32 rows 241 / 201, 64 rows 456 / 204
//   bf16, 2^19 positions: 32 rows 72 / 103, 48 rows 90 / 101, 64 rows 127 / 105;  2^16: 64 rows 27 / 63
//   e4m3, 2^20 positions: 32 rows 135 / 254, 48 rows 192 / 255, 64 rows 281 / 257;  2^19: 64 rows 134 / 131
constexpr int kFewRows = 64;
bool few_rows(int64_t rows, int64_t positions, bool q8) {
  const int64_t row_groups = (rows + 15) / 16;
  return rows <= 16 || (rows <= kFewRows && positions <= int64_t{1} << ((q8 ? 23 : 22) - row_groups));
}
// Units charged per fragment in their balanced split, as in pa_decode.  4 trees of 5 to 16 nodes over 20 to 300 tokens with
// 1 / 2 / 3 / 5 units: 27.5 / 23.5 / 26.8 / 30.7 us with the commit (fewer, longer pieces against joins); 32 x 4K decode steps
// 52.1 / 51.9 / 51.6 / 51.7.
constexpr int kDecodeFragCost = 2;

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Arrival counters live at the start of the workspace, which is zero between calls.  Up to kCounters of them fit the fixed
// area that calls of any shape share; a call with more clears them itself first (its batch is large enough not to notice).
constexpr size_t kCounters = 1 << 16;

// Batches for which the decode kernel's launch shape is computed: powers of two up to 64, then steps of an eighth of the next
// power of two, 64 at least; a batch takes the next one's shape.  (Its per-sequence arrays take shared memory from the rings, so
// warps, and the workspace that their records take, fall as a batch grows, in steps; with few different shapes
// attend_workspace_bytes can look at all of them.)
int shape_step(int num_seqs) {
  int n = 1;
  while (n < num_seqs) n *= 2;
  return n <= 64 ? n : (n / 8 > 64 ? n / 8 : 64);
}
int shape_seqs(int num_seqs) {
  const int step = shape_step(num_seqs);
  return (num_seqs + step - 1) / step * step;
}
int smaller_shape(int num_seqs) {  // the next smaller of them, or 0
  const int n = shape_seqs(num_seqs);
  return n <= 64 ? n / 2 : n - shape_step(n);
}

// How a call of these sizes runs, and what it keeps in the workspace.
struct Plan {
  enum Kind { kFew, kTensor } kind;
  int cg;                     // kTensor: CTAs that share a tile (1, or a cluster of 2)
  int paired;                 // kTensor: the streams are two row tiles
  int seg_rows;               // kTensor: rows of a segment
  DecodeKey key;              // kFew: the decode kernel's variant and geometry
  DecodeGeometry geo;
  int ctas;
  int rec_rows, slots;
  size_t num_counters;
  size_t records, pending, stats, scores, bytes;  // offsets of the parts, total
  int score_stride;
};

// prefer: the kernel to plan for where both may serve such a call, or -1: the one that does.
bool make_plan(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq,
               int max_q_len, int q_dtype, int kv_dtype, bool tree, bool accumulate, int prefer, Plan* pl) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return false;
  const int group = num_heads / num_kv_heads;
  const int64_t rows = static_cast<int64_t>(max_q_len) * group;
  const bool q8 = kv_dtype == PA_FP8_E4M3 || kv_dtype == PA_INT8;
  pl->ctas = sms;
  const int rps = stream_rows(group);
  pl->cg = q8 || (head_dim == 128 && rows > rps) ? 2 : 1;
  pl->paired = rows > static_cast<int64_t>(rps) * pl->cg ? 1 : 0;
  pl->seg_rows = rps * pl->cg * (pl->paired ? 2 : 1);
  const int few = tuning_override("PA_ATTEND_FEW_ROWS");  // tuning
  const int64_t positions = static_cast<int64_t>(num_seqs) * num_kv_heads * max_blocks_per_seq * block_size;
  const bool chosen = prefer >= 0 ? prefer == Plan::kFew : few >= 0 ? rows <= few : few_rows(rows, positions, q8);
  const bool is_few = rows <= kFewRows && (accumulate || chosen);
  pl->kind = is_few ? Plan::kFew : Plan::kTensor;
  size_t records = 0, pending = 0;
  pl->num_counters = 0;
  if (pl->kind == Plan::kFew) {
    const int gm = max_q_len == 1 && group <= 8 && !tree ? 8 : 16;
    pl->key.q_dtype = q_dtype;
    pl->key.kv_dtype = kv_dtype;
    pl->key.head_dim = head_dim;
    pl->key.gmax = gm;
    pl->key.unit_rows = q8 && block_size >= 16 && gm == 8 ? 64 : 32;
    pl->key.append = 2;
    pl->key.row_groups = gm == 16 ? static_cast<int>((rows + 15) / 16) : 1;
    if (!decode_geometry(pl->key, shape_seqs(num_seqs), &pl->geo)) return false;
    const size_t warps = static_cast<size_t>(pl->geo.ctas) * pl->geo.warps_per_cta;
    pl->num_counters = static_cast<size_t>(num_seqs) * num_kv_heads * pl->geo.row_groups;
    records = 2 * warps * pl->geo.record_floats * sizeof(float);
    pending = 2 * warps * sizeof(int);
  } else {
    pl->ctas = sms / pl->cg * pl->cg;
    pl->rec_rows = rows < rps ? static_cast<int>((rows + 7) / 8 * 8) : kTile;
    pl->slots = pl->paired ? 2 : 4;
    pl->num_counters = pl->paired ? 2 * static_cast<size_t>(sms) : static_cast<size_t>(num_seqs) * num_kv_heads * pl->cg;
    records = static_cast<size_t>(sms) * pl->slots * 2 * pl->rec_rows * (head_dim + 2) * sizeof(float);  // (32-byte multiples)
  }
  size_t at = up256((pl->num_counters > kCounters ? pl->num_counters : kCounters) * sizeof(int));
  pl->records = at;
  at += up256(records);
  pl->pending = at;
  at += up256(pending);
  pl->stats = at;
  pl->score_stride = max_blocks_per_seq * block_size;
  if (accumulate) at += up256(static_cast<size_t>(num_seqs) * num_heads * sizeof(float2));
  pl->scores = at;
  if (accumulate) at += up256(static_cast<size_t>(num_seqs) * num_heads * pl->score_stride * sizeof(float));
  pl->bytes = at;
  return true;
}

// The decode kernel's variants with score modifiers.
cudaError_t launch_few(const AttendParams& a, const Plan& pl, uint8_t* ws, cudaStream_t stream) {
  DecodeParams p;
  memset(&p, 0, sizeof(p));
  p.out = a.out;
  p.out_dtype = a.out_dtype;
  p.q = a.q;
  p.q_stride = a.q_stride;
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.k_zero_point = a.k_zero_point;
  p.v_zero_point = a.v_zero_point;
  p.block_tables = a.block_tables;
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.seq_lens = a.seq_lens;
  p.num_blocks = a.num_blocks;
  p.num_seqs = a.num_seqs;
  p.num_heads = a.num_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.group = a.group;
  p.qk_scale_log2 = a.scale * 1.4426950408889634f;
  p.block_size = a.block_size;
  p.block_shift = a.block_shift;
  p.frag_cost = kDecodeFragCost;
  p.window = a.window;
  p.q_len = 1;
  p.k_cache = const_cast<void*>(a.k_cache);
  p.v_cache = const_cast<void*>(a.v_cache);
  p.seg_counters = reinterpret_cast<int*>(ws);
  p.part_records = reinterpret_cast<float*>(ws + pl.records);
  p.pending = reinterpret_cast<int*>(ws + pl.pending);
  p.pending_cap = 2;
  p.err = a.err;
  p.stages = pl.geo.stages;
  p.row_groups = pl.geo.row_groups;
  p.stage_bytes = pl.geo.stage_bytes;
  p.wait_limit_ns = a.wait_limit_ns;
  p.att = a;
  const int eb = a.kv_dtype == PA_FP8_E4M3 || a.kv_dtype == PA_INT8 ? 1 : 2;
  const int box = a.block_size < pl.geo.unit_rows ? a.block_size : pl.geo.unit_rows;
  CUtensorMap tk, tv;
  if (!encode_cache_map(&tk, a.k_cache, a.num_blocks, a.num_kv_heads, a.block_size, a.head_dim, eb, box) ||
      !encode_cache_map(&tv, a.v_cache, a.num_blocks, a.num_kv_heads, a.block_size, a.head_dim, eb, box))
    return cudaErrorInvalidValue;
  return launch_decode(pl.key, pl.geo, p, tk, tv, stream, a.pdl);
}

// 4-D view of a 16-bit pool: {64 elements, 8 rows, 128-byte halves of a row, groups of 8 rows}; one box = box_rows
// rows, landing as [group][half][8 rows][128 bytes], swizzled by row.
bool encode_tile_map(CUtensorMap* map, const void* cache, int64_t rows, int head_dim, int box_rows, int box_halves) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t row_bytes = static_cast<cuuint64_t>(head_dim) * 2;
  const cuuint32_t halves = static_cast<cuuint32_t>(row_bytes / 128);
  cuuint64_t dims[4] = {64, 8, halves, static_cast<cuuint64_t>(rows / 8)};
  cuuint64_t strides[3] = {row_bytes, 128, 8 * row_bytes};
  cuuint32_t box[4] = {64, 8, static_cast<cuuint32_t>(box_halves), static_cast<cuuint32_t>(box_rows / 8)};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<void*>(cache), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 2-D view of an 8-bit pool: {row bytes, rows}; one box = box_rows rows of box_bytes bytes, as they are.
bool encode_code_map(CUtensorMap* map, const void* cache, int64_t rows, int row_bytes, int box_rows, int box_bytes) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(row_bytes)};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(box_bytes), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(cache), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 4-D view of the query rows: {64 elements, heads, tokens, 128-byte halves of a row}; one box = 128 / group tokens by the
// group's heads, landing as [half][token, head][128 bytes], swizzled by row; zero past the last token.
bool encode_query_map(CUtensorMap* map, const AttendParams& a) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint32_t halves = static_cast<cuuint32_t>(a.head_dim / 64);
  cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(a.num_heads), static_cast<cuuint64_t>(a.num_tokens), halves};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(a.head_dim) * 2, static_cast<cuuint64_t>(a.q_stride) * 2, 128};
  cuuint32_t box[4] = {64, static_cast<cuuint32_t>(a.group), static_cast<cuuint32_t>(kTile / a.group), halves};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<void*>(a.q), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename KVT, int D, int CG, bool SPLIT>
cudaError_t launch_tc_as(const AttendParams& a, const Plan& pl, uint8_t* ws, cudaStream_t stream) {
  using Tr = TcTraits<KVT, D, CG>;
  TcParams p;
  p.a = a;
  p.paired = pl.paired;
  p.seg_rows = pl.seg_rows;
  p.max_segments = static_cast<float>(a.num_seqs) * a.num_kv_heads * ((a.max_q_len * a.group + pl.seg_rows - 1) / pl.seg_rows);
  p.rec_rows = pl.rec_rows;
  p.slots = pl.slots;
  p.counters = reinterpret_cast<int*>(ws);
  p.records = reinterpret_cast<float*>(ws + pl.records);
  CUtensorMap tk, tv, tq;
  const int64_t rows = a.num_blocks * a.num_kv_heads * a.block_size;
  auto box = [&](int most) { return a.block_size < most ? a.block_size : most; };
  const bool maps = Tr::B8 ? encode_code_map(&tk, a.k_cache, rows, D, box(Tr::KROWS), D) &&
                                 encode_code_map(&tv, a.v_cache, rows, D, box(kTile), D / CG)
                           : encode_tile_map(&tk, a.k_cache, rows, D, box(Tr::KROWS), Tr::NH) &&
                                 encode_tile_map(&tv, a.v_cache, rows, D, box(kTile), Tr::VH);
  if (!maps || !encode_query_map(&tq, a)) return cudaErrorInvalidValue;
  auto kern = attend_tc_kernel<KVT, D, CG, SPLIT>;
  const size_t smem = Tr::smem_bytes(a.num_seqs);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(pl.ctas);
  cfg.blockDim = dim3(Tr::THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CG;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.pdl ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kern, tk, tv, tq, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename KVT, int D, int CG>
cudaError_t launch_tc(const AttendParams& a, const Plan& pl, uint8_t* ws, cudaStream_t stream) {
  // the second product is free where memory traffic bounds the call, and wanted where the output keeps its precision
  return !pl.paired || a.out_dtype == PA_F32 ? launch_tc_as<KVT, D, CG, true>(a, pl, ws, stream)
                                             : launch_tc_as<KVT, D, CG, false>(a, pl, ws, stream);
}

// mass[s][kvh][t] += sum over the group of exp2(score - max) / sum, from the stored scores, whose heads stand side by side:
// kMassKeys positions per thread, a CTA's threads on consecutive ones.  (A weight is known only when its row's last position
// has been seen, so the attention stores the scores and this kernel follows.)
// What bounds it: memory and L2 traffic, 4 G + 8 bytes per position and KV head.  8 heads of 32 x up to 4096 positions, G = 4:
// 5.5 us; of 8 x 32768, G = 8: 16 us (84 MB, 5.2 TB/s).
constexpr int kMassThreads = 128, kMassKeys = 4;
__global__ void __launch_bounds__(kMassThreads) attend_add_mass_kernel(const AttendParams p) {
  griddep_wait();
  const int s = blockIdx.z, kvh = blockIdx.y, G = p.group;
  const SeqView v = seq_view(p, s, false);
  if (v.L != 1) return;
  const RowBounds rb = row_bounds(p, v, seq_prefix(p, s, v.T), 0);
  const int t0 = blockIdx.x * kMassThreads * kMassKeys;
  if (t0 + kMassThreads * kMassKeys <= rb.lo || t0 >= rb.hi) return;
  const int64_t row0 = static_cast<int64_t>(s) * p.num_heads + kvh * G;
  const float* const sc = p.scores + (static_cast<int64_t>(s) * p.num_kv_heads + kvh) * p.score_stride * G;
  float* const mass = p.mass + s * p.mass_stride_seq + kvh * p.mass_stride_head;
  float sum[kMassKeys] = {}, old[kMassKeys];
  bool in[kMassKeys];  // (scores outside [lo, hi) were not stored)
#pragma unroll
  for (int k = 0; k < kMassKeys; ++k) {
    const int t = t0 + k * kMassThreads + threadIdx.x;
    in[k] = t >= rb.lo && t < rb.hi;
    old[k] = in[k] ? mass[t] : 0.f;
  }
  auto add = [&](int k, float z, float2 ml, float inv) { sum[k] = fmaf(exp2f(z - ml.x), inv, sum[k]); };
  if ((G & 3) == 0) {
#pragma unroll 2
    for (int g = 0; g < G; g += 4) {
      float4 x[kMassKeys];
#pragma unroll
      for (int k = 0; k < kMassKeys; ++k) {
        const int t = t0 + k * kMassThreads + threadIdx.x;
        if (in[k]) x[k] = *reinterpret_cast<const float4*>(sc + static_cast<int64_t>(t) * G + g);
      }
      float2 ml[4];
      float inv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ml[i] = p.row_stats[row0 + g + i];
        inv[i] = __frcp_rn(ml[i].y);
      }
#pragma unroll
      for (int k = 0; k < kMassKeys; ++k) {
        if (!in[k]) continue;
        add(k, x[k].x, ml[0], inv[0]);
        add(k, x[k].y, ml[1], inv[1]);
        add(k, x[k].z, ml[2], inv[2]);
        add(k, x[k].w, ml[3], inv[3]);
      }
    }
  } else {
    for (int g = 0; g < G; ++g) {
      const float2 ml = p.row_stats[row0 + g];
      const float inv = __frcp_rn(ml.y);
#pragma unroll
      for (int k = 0; k < kMassKeys; ++k) {
        const int t = t0 + k * kMassThreads + threadIdx.x;
        if (in[k]) add(k, sc[static_cast<int64_t>(t) * G + g], ml, inv);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kMassKeys; ++k)
    if (in[k]) mass[t0 + k * kMassThreads + threadIdx.x] = old[k] + sum[k];
}

}  // namespace

size_t attend_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                              int max_blocks_per_seq, int max_q_len, int kv_dtype, bool accumulate) {
  // The largest need on either kernel, with and without a tree, with either query type that the caches take, and of calls with
  // fewer sequences, queries or blocks: records change with the launch shape (shape_seqs; all else grows with the batch and its
  // blocks), and where the rows fill another 16 up to 64, a stream or a pair.
  const int group = num_heads / num_kv_heads, per_stream = stream_rows(group) / group;
  const int lens[] = {1,          16 / group,     16 / group + 1, 32 / group,     32 / group + 1, 48 / group, 48 / group + 1,
                      64 / group, 64 / group + 1, per_stream,     per_stream + 1, 2 * per_stream, max_q_len};
  constexpr int kLens = sizeof(lens) / sizeof(lens[0]);
  size_t most = 0;
  for (int i = 0; i < 8; ++i) {
    const int q_dtype = i & 1 ? PA_BF16 : PA_F16, prefer = i & 2 ? Plan::kFew : Plan::kTensor;
    if ((kv_dtype == PA_F16 || kv_dtype == PA_BF16) && q_dtype != kv_dtype) continue;
    for (int x = 0; x < kLens; ++x) {
      const int len = lens[x];
      bool again = len < 1 || len > max_q_len;
      for (int y = 0; y < x; ++y) again = again || lens[y] == len;
      if (again) continue;
      for (int seqs = num_seqs > 1 ? num_seqs : 1; seqs >= 1; seqs = smaller_shape(seqs)) {
        Plan pl;
        if (!make_plan(seqs, num_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq, len, q_dtype, kv_dtype,
                       (i & 4) != 0, accumulate, prefer, &pl))
          return static_cast<size_t>(-1);
        most = pl.bytes > most ? pl.bytes : most;
      }
    }
  }
  return most;
}

int launch_attend(AttendParams p, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  (void)cudaGetLastError();
  Plan pl;
  if (!make_plan(p.num_seqs, p.num_heads, p.num_kv_heads, p.head_dim, p.block_size, p.max_blocks_per_seq, p.max_q_len,
                 p.q_dtype, p.kv_dtype, p.tree_mask != nullptr, p.mass != nullptr, -1, &pl))
    return cuda_status(cudaErrorInvalidDevice, "pa_attend plan");
  if (!workspace || workspace_bytes < pl.bytes || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return PA_ERR_WORKSPACE;
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  p.row_stats = reinterpret_cast<float2*>(ws + pl.stats);
  p.scores = reinterpret_cast<float*>(ws + pl.scores);
  p.score_stride = pl.score_stride;
  cudaError_t e = cudaSuccess;
  if (pl.num_counters > kCounters) {
    e = cudaMemsetAsync(ws, 0, pl.num_counters * sizeof(int), stream);
    p.pdl = false;  // the kernel before this one is no longer the stream's last work
  }
  if (e != cudaSuccess) return cuda_status(e, "pa_attend counters");
  if (pl.kind == Plan::kFew) {
    e = launch_few(p, pl, ws, stream);
  } else if (p.kv_dtype == PA_FP8_E4M3) {
    e = launch_tc<e4m3_t, 128, 2>(p, pl, ws, stream);
  } else if (p.kv_dtype == PA_INT8) {
    e = launch_tc<i8_t, 128, 2>(p, pl, ws, stream);
  } else if (p.kv_dtype == PA_F16) {
    e = p.head_dim == 64 ? launch_tc<f16_t, 64, 1>(p, pl, ws, stream)
        : pl.cg == 1     ? launch_tc<f16_t, 128, 1>(p, pl, ws, stream)
                         : launch_tc<f16_t, 128, 2>(p, pl, ws, stream);
  } else {
    e = p.head_dim == 64 ? launch_tc<bf16_t, 64, 1>(p, pl, ws, stream)
        : pl.cg == 1     ? launch_tc<bf16_t, 128, 1>(p, pl, ws, stream)
                         : launch_tc<bf16_t, 128, 2>(p, pl, ws, stream);
  }
  if (e == cudaSuccess && p.mass) {
    const int cap = p.max_blocks_per_seq << p.block_shift;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((cap + kMassKeys * kMassThreads - 1) / (kMassKeys * kMassThreads), p.num_kv_heads, p.num_seqs);
    cfg.blockDim = dim3(kMassThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, attend_add_mass_kernel, p);
    if (e == cudaSuccess) e = cudaGetLastError();
  }
  return cuda_status(e, "pa_attend launch");
}

}  // namespace pa
