// pa_decode_int4.cu - the decode variants of pa_attend over 4-bit caches, in their own
// translation unit so the build compiles them in parallel.  This file is the
// only place these kernels are instantiated.
#include "pa_decode.cuh"
#include "pa_decode_variants.h"

namespace pa {
PA_DECODE_VARIANTS_INT4(PA_DEFINE_VARIANT)
}  // namespace pa
