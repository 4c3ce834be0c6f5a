// pa_decode_sinks8.cu - the decode variants with score modifiers and sinks (8-bit caches), in their own
// translation unit so the build compiles them in parallel.  This file is the
// only place these kernels are instantiated.
#include "pa_decode.cuh"
#include "pa_decode_variants.h"

namespace pa {
PA_DECODE_VARIANTS_SINKS8(PA_DEFINE_VARIANT)
}  // namespace pa
