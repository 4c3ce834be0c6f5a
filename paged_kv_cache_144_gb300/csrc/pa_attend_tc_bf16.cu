// pa_attend_tc_bf16.cu - the tensor-core attention kernel over bf16 caches.
#include "pa_attend_tc_launch.cuh"

namespace pa {

cudaError_t launch_tc_bf16(const AttendParams& a, const Plan& pl, uint8_t* ws, cudaStream_t stream) {
  if (a.head_dim == 64) return launch_tc<bf16_t, 64, 1>(a, pl, ws, stream);
  return pl.cg == 1 ? launch_tc<bf16_t, 128, 1>(a, pl, ws, stream) : launch_tc<bf16_t, 128, 2>(a, pl, ws, stream);
}

}  // namespace pa
