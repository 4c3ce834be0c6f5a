// pa_decode_sinks16.cu - the decode variants with score modifiers and sinks (16-bit caches), in their own
// translation unit so the build compiles them in parallel.  This file is the
// only place these kernels are instantiated.
#include "pa_decode.cuh"
#include "pa_decode_variants.h"

namespace pa {
PA_DECODE_VARIANTS_SINKS16(PA_DEFINE_VARIANT)
}  // namespace pa
