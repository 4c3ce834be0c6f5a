// pa_read.cu - cached rows read back as values, by slot.
//
// Mathematics: 16-bit rows as they are, e4m3 code * scale[h], int8 (code -
// zero_point[h]) * scale[h], 4-bit code * scale + zero of the row's own pair, in
// float32, rounded once to the output's type.
//
// Work: D / 8 threads take a row, 8 values each, so that a 16-bit output leaves
// in 16-byte pieces and a row's codes arrive in whole sectors; K and V of kRows
// rows of a thread are on their way at once.  Rows are taken in the order of the
// output.
//
// What bounds it: memory traffic (device times, caches cold).  32768 rows of 8
// heads of 128 as bf16: from 4 bits 30.4 us, 5.6 TB/s of the 170 MB read and written
// (82 % of a plain copy); from e4m3 33.4 (89 %), from bf16 42.7 (93 %).  333 rows:
// 3.6 us, two dependent loads.  K and V under way together, the slot read once, for
// two rows of a thread: 38.5 -> 30.4; four rows 30.6, 256 threads 32.1.
#include <type_traits>

#include "pa_common.cuh"
#include "pa_ops.h"

namespace pa {
namespace {

constexpr int kThreads = 128;
constexpr int kRows = 2;

template <typename KVT> struct Codes { using type = uint2; };  // what a thread loads: 8 values
template <> struct Codes<f16_t> { using type = uint4; };
template <> struct Codes<bf16_t> { using type = uint4; };
template <> struct Codes<i4_t> { using type = uint32_t; };

template <typename KVT, int D>
__global__ void __launch_bounds__(kThreads) read_cache_kernel(const ReadArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  using C = typename Codes<KVT>::type;
  constexpr int L = D / 8, STEP = kThreads / L;  // threads of a row, rows of a step
  const int l = static_cast<int>(threadIdx.x) % L, Hk = a.num_kv_heads, B = a.block_size;
  const int64_t total = a.num_tokens * Hk;
  const int64_t x0 = static_cast<int64_t>(blockIdx.x) * (STEP * kRows) + threadIdx.x / L;
  C code[kRows][2];
  uint32_t pair[kRows][2];
  int64_t tok[kRows];  // (-1: no such row)
  int head[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int64_t x = x0 + k * STEP;
    tok[k] = -1;
    head[k] = 0;
    if (x >= total) continue;
    const int64_t n = x < (int64_t{1} << 32) ? static_cast<uint32_t>(x) / static_cast<uint32_t>(Hk) : x / Hk;
    const int64_t slot = a.slots[n];
    head[k] = static_cast<int>(x - n * Hk);
    if (slot < 0) continue;  // padding
    if (slot >= a.num_blocks * B) {
      if (l == 0 && head[k] == 0) raise_error(a.err, PA_DEVERR_SLOT);
      continue;
    }
    tok[k] = n;
    const int64_t blk = slot >> a.block_shift, tile = blk * Hk + head[k];
    const int row = static_cast<int>(slot - (blk << a.block_shift));
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const uint8_t* const cache = static_cast<const uint8_t*>(v ? a.v_cache : a.k_cache);
      if constexpr (std::is_same<KVT, i4_t>::value) {
        const uint8_t* const at = cache + tile * (static_cast<int64_t>(B) * int4_row_bytes(D));
        code[k][v] = reinterpret_cast<const uint32_t*>(at + row * (D / 2))[l];
        pair[k][v] = reinterpret_cast<const uint32_t*>(at + B * (D / 2))[row];
      } else {
        code[k][v] = reinterpret_cast<const C*>(cache + (tile * B + row) * (D * elem<KVT>::bytes))[l];
      }
    }
  }
#pragma unroll
  for (int x2 = 0; x2 < 2 * kRows; ++x2) {
    const int k = x2 >> 1;
    const bool is_v = x2 & 1;
    if (tok[k] < 0) continue;
    float x[8];
    if constexpr (std::is_same<KVT, i4_t>::value) {
      const float2 sz = widen2<f16_t>(pair[k][is_v]);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        x[i] = fmaf(static_cast<float>((code[k][is_v] >> (16 * (i & 1) + 4 * (i >> 1))) & 15u), sz.x, sz.y);
    } else if constexpr (elem<KVT>::bytes == 2) {
      const uint32_t r[4] = {code[k][is_v].x, code[k][is_v].y, code[k][is_v].z, code[k][is_v].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = widen2<KVT>(r[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    } else {
      const float s = __ldg((is_v ? a.v_scale : a.k_scale) + head[k]);
      const uint32_t r[2] = {code[k][is_v].x, code[k][is_v].y};
      if constexpr (std::is_same<KVT, e4m3_t>::value) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = widen2_e4m3(r[i >> 1] >> (16 * (i & 1)));
          x[2 * i] = f.x * s;
          x[2 * i + 1] = f.y * s;
        }
      } else {
        const int zp = __ldg((is_v ? a.v_zero_point : a.k_zero_point) + head[k]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          x[i] = static_cast<float>(static_cast<int>(static_cast<int8_t>(r[i >> 2] >> (8 * (i & 3)))) - zp) * s;
      }
    }
    const int64_t o = tok[k] * (is_v ? a.v_stride : a.k_stride) + static_cast<int64_t>(head[k]) * D + 8 * l;
    void* const out = is_v ? a.v_out : a.k_out;
    if (a.out_dtype == PA_F32) {
      float4* const to = reinterpret_cast<float4*>(static_cast<float*>(out) + o);
      to[0] = make_float4(x[0], x[1], x[2], x[3]);
      to[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
      uint4 w;
      if (a.out_dtype == PA_BF16)
        w = make_uint4(pack2<true>(x[0], x[1]), pack2<true>(x[2], x[3]), pack2<true>(x[4], x[5]), pack2<true>(x[6], x[7]));
      else
        w = make_uint4(pack2<false>(x[0], x[1]), pack2<false>(x[2], x[3]), pack2<false>(x[4], x[5]), pack2<false>(x[6], x[7]));
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + o) = w;
    }
  }
}

template <typename KVT, int D>
cudaError_t launch_as(const ReadArgs& a, cudaStream_t stream) {
  constexpr int PER = kThreads / (D / 8) * kRows;
  const int64_t total = a.num_tokens * a.num_kv_heads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((total + PER - 1) / PER));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.pdl ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, read_cache_kernel<KVT, D>, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_read_cache(const ReadArgs& a, cudaStream_t stream) {
  (void)cudaGetLastError();
  const bool d64 = a.head_dim == 64;
  switch (a.kv_dtype) {
    case PA_INT4: return launch_as<i4_t, 128>(a, stream);
    case PA_FP8_E4M3: return d64 ? launch_as<e4m3_t, 64>(a, stream) : launch_as<e4m3_t, 128>(a, stream);
    case PA_INT8: return d64 ? launch_as<i8_t, 64>(a, stream) : launch_as<i8_t, 128>(a, stream);
    case PA_F16: return d64 ? launch_as<f16_t, 64>(a, stream) : launch_as<f16_t, 128>(a, stream);
    default: return d64 ? launch_as<bf16_t, 64>(a, stream) : launch_as<bf16_t, 128>(a, stream);
  }
}

}  // namespace pa
