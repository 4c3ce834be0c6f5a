// pa_attend_tc_launch.cuh - host side of the tensor-core attention kernel: tensor
// maps and the launch of one variant.  Included by one translation unit per
// cache type.
#pragma once

#include "pa_attend_plan.h"
#include "pa_attend_tc.cuh"

namespace pa {
namespace {

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

template <typename KVT, int D, int CG, bool SPLIT, bool SINKS>
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
  CUtensorMap tk = {}, tv = {}, tq;  // (4-bit caches: bulk copies, no maps of K and V)
  const int64_t rows = a.num_blocks * a.num_kv_heads * a.block_size;
  auto box = [&](int most) { return a.block_size < most ? a.block_size : most; };
  const bool maps = Tr::B4   ? true
                    : Tr::B8 ? encode_code_map(&tk, a.k_cache, rows, D, box(Tr::KROWS), D) &&
                                 encode_code_map(&tv, a.v_cache, rows, D, box(kTile), D / CG)
                           : encode_tile_map(&tk, a.k_cache, rows, D, box(Tr::KROWS), Tr::NH) &&
                                 encode_tile_map(&tv, a.v_cache, rows, D, box(kTile), Tr::VH);
  if (!maps || !encode_query_map(&tq, a)) return cudaErrorInvalidValue;
  auto kern = attend_tc_kernel<KVT, D, CG, SPLIT, SINKS>;
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
  const bool split = !pl.paired || a.out_dtype == PA_F32;
  // (sinks apart: their masks and tile numbers cost a call without them 5 % of its time)
  if (a.sinks > 0 || std::is_same<KVT, i4_t>::value)
    return split ? launch_tc_as<KVT, D, CG, true, true>(a, pl, ws, stream) : launch_tc_as<KVT, D, CG, false, true>(a, pl, ws, stream);
  if constexpr (!std::is_same<KVT, i4_t>::value)
    return split ? launch_tc_as<KVT, D, CG, true, false>(a, pl, ws, stream) : launch_tc_as<KVT, D, CG, false, false>(a, pl, ws, stream);
}

}  // namespace
}  // namespace pa
