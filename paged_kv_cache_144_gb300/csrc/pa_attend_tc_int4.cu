// pa_attend_tc_int4.cu - the tensor-core attention kernel over 4-bit caches.
#include "pa_attend_tc_launch.cuh"

namespace pa {

cudaError_t launch_tc_int4(const AttendParams& a, const Plan& pl, uint8_t* ws, cudaStream_t stream) {
  return launch_tc<i4_t, 128, 2>(a, pl, ws, stream);
}

}  // namespace pa
