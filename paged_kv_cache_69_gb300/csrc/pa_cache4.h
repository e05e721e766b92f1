// pa_cache4.h -- host entry of the 4-bit cache write (pa_cache4.cu), called
// by pa_reshape_and_cache once the arguments shared by every cache type are
// checked.
#pragma once

#include <type_traits>

#include "../../include/pa.h"

namespace pa {
pa_status write_int4(void* kc, void* vc, const void* key, const void* value, pa_dtype src, const int64_t* slots, int T,
                     int Hkv, int D, int bs, int NB, int32_t* err, cudaStream_t stream);
}  // namespace pa
