// pa_decode_int4.h -- host entry of attention over 4-bit pools, called once
// the arguments shared by every cache type are checked.
#pragma once

#include "../../include/pa.h"

namespace pa {
pa_status decode_int4(void* out, const void* q, pa_dtype q_dtype, const void* k, const void* v, const int32_t* tables,
                      int MB, const int32_t* lens, int B, int Hq, int Hkv, int D, int bs, int NB, float scale,
                      int32_t* err, cudaStream_t stream, const int32_t* q_start, int QL, int total_q);
}  // namespace pa
