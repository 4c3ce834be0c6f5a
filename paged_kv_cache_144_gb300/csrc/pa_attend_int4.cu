// pa_attend_int4.cu - the launch of attend_int4_kernel, in its own translation
// unit so the build compiles it in parallel.
#include "pa_attend_int4.cuh"

#include "pa_attend_plan.h"

namespace pa {

bool int4_geometry(int num_seqs, DecodeGeometry* g) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return false;
  g->warps_per_cta = Int4Traits::WARPS;
  g->stages = 0;
  g->ctas = sms;
  g->smem_bytes = Int4Traits::smem_bytes(num_seqs);
  g->record_floats = Int4Traits::REC;
  g->stage_bytes = 0;
  g->unit_rows = Int4Traits::UR;
  g->row_groups = 1;
  return true;
}

namespace {

template <typename QT, int BX, bool SPLIT>
cudaError_t launch_as(const DecodeGeometry& g, const DecodeParams& p, cudaStream_t stream, bool pdl) {
  auto kern = attend_int4_kernel<QT, BX, SPLIT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(g.smem_bytes));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(g.ctas);
  cfg.blockDim = dim3(g.warps_per_cta * 32);
  cfg.dynamicSmemBytes = g.smem_bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, kern, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename QT, bool SPLIT>
cudaError_t launch_bx(const DecodeGeometry& g, const DecodeParams& p, cudaStream_t stream, bool pdl) {
  static_assert(Int4Traits::UR == 64, "blocks of a unit");
  switch (p.block_size) {
    case 8: return launch_as<QT, 8, SPLIT>(g, p, stream, pdl);
    case 16: return launch_as<QT, 4, SPLIT>(g, p, stream, pdl);
    case 32: return launch_as<QT, 2, SPLIT>(g, p, stream, pdl);
    default: return launch_as<QT, 1, SPLIT>(g, p, stream, pdl);
  }
}

// One f16 value per weight where the output is bf16: off by 2^-11 of it, against the output's own 2^-8 (2^-11 for f16, which
// takes two: +3 % of the time).
template <typename QT>
cudaError_t launch_q(const DecodeGeometry& g, const DecodeParams& p, cudaStream_t stream, bool pdl) {
  return p.out_dtype == PA_BF16 ? launch_bx<QT, false>(g, p, stream, pdl) : launch_bx<QT, true>(g, p, stream, pdl);
}

}  // namespace

cudaError_t launch_int4(const DecodeGeometry& g, const DecodeParams& p, int q_dtype, cudaStream_t stream, bool pdl) {
  (void)cudaGetLastError();
  return q_dtype == PA_BF16 ? launch_q<bf16_t>(g, p, stream, pdl) : launch_q<f16_t>(g, p, stream, pdl);
}

}  // namespace pa
