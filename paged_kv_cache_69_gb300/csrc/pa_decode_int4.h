// pa_decode_int4.h -- host entry of attention over 4-bit pools, called once
// the arguments shared by every cache type are checked and the workspace is
// carved.
#pragma once

#include "pa_kernels.h"

namespace pa {

struct Int4Call {
    void* out;
    const void* q;
    pa_dtype q_dtype;
    const void* k;
    const void* v;
    const int32_t* tables;
    int MB;
    const int32_t* lens;
    int B, Hq, Hkv, D, bs, NB;
    float scale;
    int partition_tokens;
    Workspace ws;
    int32_t* err;
    cudaStream_t stream;
    const int32_t* q_start;       // null: one query token per sequence
    int QL, total_q;
    int sms, max_smem;
    const WeightsOut* weights;    // null but for pa_decode_weights
};
pa_status decode_int4(const Int4Call& c);

}  // namespace pa
