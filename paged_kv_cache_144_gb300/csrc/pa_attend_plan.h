// pa_attend_plan.h - how a pa_attend call runs, and the launches of the
// tensor-core kernel, one translation unit per cache type.
#pragma once

#include "pa_ops.h"

namespace pa {

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

cudaError_t launch_tc_f16(const AttendParams& a, const Plan& pl, uint8_t* ws, cudaStream_t stream);
cudaError_t launch_tc_bf16(const AttendParams& a, const Plan& pl, uint8_t* ws, cudaStream_t stream);
cudaError_t launch_tc_fp8(const AttendParams& a, const Plan& pl, uint8_t* ws, cudaStream_t stream);
cudaError_t launch_tc_int8(const AttendParams& a, const Plan& pl, uint8_t* ws, cudaStream_t stream);
cudaError_t launch_tc_int4(const AttendParams& a, const Plan& pl, uint8_t* ws, cudaStream_t stream);

// One query per sequence over a 4-bit cache, up to 8 heads per KV head: attend_int4_kernel.
bool int4_geometry(int num_seqs, DecodeGeometry* geo);
cudaError_t launch_int4(const DecodeGeometry& geo, const DecodeParams& p, int q_dtype, cudaStream_t stream, bool pdl);

}  // namespace pa
