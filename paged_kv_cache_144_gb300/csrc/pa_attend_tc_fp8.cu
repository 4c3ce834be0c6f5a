// pa_attend_tc_fp8.cu - the tensor-core attention kernel over FP8-e4m3 caches.
#include "pa_attend_tc_launch.cuh"

namespace pa {

cudaError_t launch_tc_fp8(const AttendParams& a, const Plan& pl, uint8_t* ws, cudaStream_t stream) {
  return launch_tc<e4m3_t, 128, 2>(a, pl, ws, stream);
}

}  // namespace pa
