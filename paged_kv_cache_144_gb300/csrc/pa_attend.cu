// pa_attend.cu - attention of ragged query rows over the paged cache with
// score modifiers, and the accumulation of each cached position's weight.
#include "pa_attend.cuh"

namespace pa {
namespace {

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

size_t attend_workspace_bytes(int num_seqs, int num_heads, int, int, int, int, int, int, bool accumulate) {
  return accumulate ? sizeof(float2) * static_cast<size_t>(num_seqs) * num_heads : 0;
}

cudaError_t launch_attend(AttendParams p, void* workspace, cudaStream_t stream) {
  (void)cudaGetLastError();
  p.row_stats = p.mass ? static_cast<float2*>(workspace) : nullptr;
  switch (p.kv_dtype) {
    case PA_F16: return p.head_dim == 128 ? launch_t<f16_t, 128>(p, stream) : launch_t<f16_t, 64>(p, stream);
    case PA_BF16: return p.head_dim == 128 ? launch_t<bf16_t, 128>(p, stream) : launch_t<bf16_t, 64>(p, stream);
    case PA_FP8_E4M3: return launch_t<e4m3_t, 128>(p, stream);
    default: return launch_t<i8_t, 128>(p, stream);
  }
}

}  // namespace pa
