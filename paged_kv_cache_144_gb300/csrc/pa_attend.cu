// pa_attend.cu - attention of ragged query rows over the paged cache with
// score modifiers, and the accumulation of each cached position's weight.
#include "pa_attend_tc.cuh"

namespace pa {
namespace {

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// How a call of these sizes runs, and what it keeps in the workspace.
struct Plan {
  int ctas;
  int paired;
  int rec_rows, slots;
  size_t counters, records, stats, scores, bytes;  // offsets of the parts, total
  int score_stride;
};

bool make_plan(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int cap, int max_q_len, bool accumulate,
               Plan* pl) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return false;
  const int64_t rows = static_cast<int64_t>(max_q_len) * (num_heads / num_kv_heads);
  pl->ctas = sms;
  pl->paired = rows > kTile ? 1 : 0;
  pl->rec_rows = pl->paired ? kTile : static_cast<int>((rows + 7) / 8 * 8);
  pl->slots = pl->paired ? 2 : 4;
  size_t at = 0;
  pl->counters = at;
  at += up256((pl->paired ? 2 * static_cast<size_t>(sms) : static_cast<size_t>(num_seqs) * num_kv_heads) * sizeof(int));
  pl->records = at;
  at += up256(static_cast<size_t>(sms) * pl->slots * 2 * pl->rec_rows * (head_dim + 2) * sizeof(float));
  pl->stats = at;
  pl->score_stride = (cap + kTile - 1) / kTile * kTile;
  if (accumulate) at += up256(static_cast<size_t>(num_seqs) * num_heads * sizeof(float2));
  pl->scores = at;
  if (accumulate) at += up256(static_cast<size_t>(num_seqs) * num_heads * pl->score_stride * sizeof(float));
  pl->bytes = at;
  return true;
}

// 4-D view of a 16-bit pool: {64 elements, 8 rows, 128-byte halves of a row, groups of 8 rows}; one box = box_rows
// rows, landing as [group][half][8 rows][128 bytes], swizzled by row.
bool encode_tile_map(CUtensorMap* map, const void* cache, int64_t rows, int head_dim, int box_rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t row_bytes = static_cast<cuuint64_t>(head_dim) * 2;
  const cuuint32_t halves = static_cast<cuuint32_t>(row_bytes / 128);
  cuuint64_t dims[4] = {64, 8, halves, static_cast<cuuint64_t>(rows / 8)};
  cuuint64_t strides[3] = {row_bytes, 128, 8 * row_bytes};
  cuuint32_t box[4] = {64, 8, halves, static_cast<cuuint32_t>(box_rows / 8)};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<void*>(cache), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename KVT, int D>
cudaError_t launch_tc(const AttendParams& a, const Plan& pl, uint8_t* ws, cudaStream_t stream) {
  using Tr = TcTraits<KVT, D>;
  TcParams p;
  p.a = a;
  p.paired = pl.paired;
  // the second product is free where memory traffic bounds the call, and wanted where the output keeps its precision
  p.split_p = (!pl.paired || a.out_dtype == PA_F32) ? 1 : 0;
  p.rec_rows = pl.rec_rows;
  p.slots = pl.slots;
  p.counters = reinterpret_cast<int*>(ws + pl.counters);
  p.records = reinterpret_cast<float*>(ws + pl.records);
  p.scores = reinterpret_cast<float*>(ws + pl.scores);
  p.score_stride = pl.score_stride;
  CUtensorMap tk, tv;
  const int64_t rows = a.num_blocks * a.num_kv_heads * a.block_size;
  const int box = a.block_size < kTile ? a.block_size : kTile;
  if (!encode_tile_map(&tk, a.k_cache, rows, D, box) || !encode_tile_map(&tv, a.v_cache, rows, D, box))
    return cudaErrorInvalidValue;
  auto kern = attend_tc_kernel<KVT, D>;
  const size_t smem = Tr::smem_bytes(a.num_seqs);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(pl.ctas);
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.pdl ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, kern, tk, tv, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

constexpr int kRowWarps = 4;

// One warp per (query, head).
template <typename KVT, int D>
__global__ void __launch_bounds__(kRowWarps * 32) attend_rows_kernel(const AttendParams p) {
  __shared__ float qs[kRowWarps][D];
  griddep_wait();
  const int s = blockIdx.y;
  const SeqView v = seq_view(p, s, blockIdx.x == 0 && threadIdx.x == 0);
  for (int64_t x = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
       x < static_cast<int64_t>(v.L) * p.num_heads; x += static_cast<int64_t>(gridDim.x) * kRowWarps) {
    const int h = static_cast<int>(x % p.num_heads), i = static_cast<int>(x / p.num_heads);
    const float2 ml = attend_row<KVT, D>(p, s, v, i, h, qs[threadIdx.x >> 5]);
    if (p.mass && (threadIdx.x & 31) == 0) p.row_stats[static_cast<int64_t>(s) * p.num_heads + h] = ml;
  }
}

// mass[s][kvh][t] += sum over the group of softmax weights: one thread per
// position, the scores computed again from q and K.
template <typename KVT, int D>
__global__ void __launch_bounds__(128) attend_mass_kernel(const AttendParams p) {
  const int s = blockIdx.z, kvh = blockIdx.y;
  const SeqView v = seq_view(p, s, false);
  const int t = blockIdx.x * 128 + threadIdx.x;
  if (t >= v.T || v.L != 1) return;
  const RowBounds rb = row_bounds(p, v, seq_prefix(p, s, v.T), 0);
  if (t < rb.lo || t >= rb.hi) return;
  float ks = 1.f;
  int kz = 0;
  if constexpr (elem<KVT>::bytes == 1) ks = __ldg(p.k_scale + kvh);
  if constexpr (std::is_same<KVT, i8_t>::value) kz = __ldg(p.k_zero_point + kvh);
  int pb = __ldg(p.block_tables + static_cast<int64_t>(s) * p.max_blocks_per_seq + (t >> p.block_shift));
  if (pb < 0 || pb >= p.num_blocks) pb = 0;
  const uint8_t* kr = static_cast<const uint8_t*>(p.k_cache) +
                      ((static_cast<int64_t>(pb) * p.num_kv_heads + kvh) * p.block_size + (t & (p.block_size - 1))) *
                          (D * elem<KVT>::bytes);
  float sum = 0.f;
  for (int g = 0; g < p.group; ++g) {
    const int h = kvh * p.group + g;
    const int64_t e = static_cast<int64_t>(v.row0) * p.q_stride + static_cast<int64_t>(h) * D;
    float x = 0.f;
    for (int c = 0; c < D; ++c)
      x = fmaf(p.q_dtype == PA_BF16 ? load_scalar<bf16_t>(p.q, e + c) : load_scalar<f16_t>(p.q, e + c),
               cache_elem<KVT>(kr, c, kz), x);
    x *= p.scale * ks;
    if (p.softcap > 0.f) x = cap_score(x, p.softcap, 2.f * 1.4426950408889634f / p.softcap);
    if (p.slopes) x -= __ldg(p.slopes + h) * static_cast<float>(abs(rb.pos - t));
    const float2 ml = p.row_stats[static_cast<int64_t>(s) * p.num_heads + h];
    sum += exp2f(x * 1.4426950408889634f - ml.x) / ml.y;
  }
  p.mass[s * p.mass_stride_seq + kvh * p.mass_stride_head + t] += sum;
}

// mass[s][kvh][t] += sum over the group of exp2(score - max) / sum, from the stored scores: one thread per position.
__global__ void __launch_bounds__(256) attend_add_mass_kernel(const AttendParams p, const float* scores, int score_stride) {
  const int s = blockIdx.z, kvh = blockIdx.y;
  const SeqView v = seq_view(p, s, false);
  if (v.L != 1) return;
  const RowBounds rb = row_bounds(p, v, seq_prefix(p, s, v.T), 0);
  const int t = blockIdx.x * 256 + threadIdx.x;
  if (t < rb.lo || t >= rb.hi) return;
  float sum = 0.f;
  for (int g = 0; g < p.group; ++g) {
    const int64_t row = static_cast<int64_t>(s) * p.num_heads + kvh * p.group + g;
    const float2 ml = p.row_stats[row];
    sum += exp2f(scores[row * score_stride + t] - ml.x) / ml.y;
  }
  p.mass[s * p.mass_stride_seq + kvh * p.mass_stride_head + t] += sum;
}

template <typename KVT, int D>
cudaError_t launch_t(const AttendParams& p, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(p.max_q_len) * p.num_heads;
  const int64_t gx = (rows + kRowWarps - 1) / kRowWarps;
  attend_rows_kernel<KVT, D><<<dim3(static_cast<unsigned>(gx < 4096 ? gx : 4096), p.num_seqs), kRowWarps * 32, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && p.mass) {
    const int cap = p.max_blocks_per_seq << p.block_shift;
    attend_mass_kernel<KVT, D><<<dim3((cap + 127) / 128, p.num_kv_heads, p.num_seqs), 128, 0, stream>>>(p);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace

size_t attend_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                              int max_blocks_per_seq, int max_q_len, int kv_dtype, bool accumulate) {
  Plan pl;
  if (!make_plan(num_seqs, num_heads, num_kv_heads, head_dim, max_blocks_per_seq * block_size, max_q_len, accumulate, &pl))
    return static_cast<size_t>(-1);
  return pl.bytes;
}

cudaError_t launch_attend(AttendParams p, void* workspace, cudaStream_t stream) {
  (void)cudaGetLastError();
  Plan pl;
  if (!make_plan(p.num_seqs, p.num_heads, p.num_kv_heads, p.head_dim, p.max_blocks_per_seq * p.block_size, p.max_q_len,
                 p.mass != nullptr, &pl))
    return cudaErrorInvalidDevice;
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  p.row_stats = reinterpret_cast<float2*>(ws + pl.stats);
  cudaError_t e = cudaSuccess;
  if (p.kv_dtype == PA_F16 || p.kv_dtype == PA_BF16) {
    if (p.kv_dtype == PA_F16)
      e = p.head_dim == 128 ? launch_tc<f16_t, 128>(p, pl, ws, stream) : launch_tc<f16_t, 64>(p, pl, ws, stream);
    else
      e = p.head_dim == 128 ? launch_tc<bf16_t, 128>(p, pl, ws, stream) : launch_tc<bf16_t, 64>(p, pl, ws, stream);
    if (e == cudaSuccess && p.mass) {
      const int cap = p.max_blocks_per_seq << p.block_shift;
      attend_add_mass_kernel<<<dim3((cap + 255) / 256, p.num_kv_heads, p.num_seqs), 256, 0, stream>>>(
          p, reinterpret_cast<const float*>(ws + pl.scores), pl.score_stride);
      e = cudaGetLastError();
    }
    return e;
  }
  return p.kv_dtype == PA_FP8_E4M3 ? launch_t<e4m3_t, 128>(p, stream) : launch_t<i8_t, 128>(p, stream);
}

}  // namespace pa
