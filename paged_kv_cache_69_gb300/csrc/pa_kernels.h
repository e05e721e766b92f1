// pa_kernels.h -- lookup of the decode kernel instantiations (host side).
#pragma once

#include "../../include/pa.h"

namespace pa {
struct DecodeParams;
// The parts of a decode workspace (pa_api.cu lays them out).
struct Workspace {
    int4* split_list;
    int* totals;
    float2* part_ml;
    float* part_acc;
    int max_slots;
};
// Launch of the log-sum-exp merge behind a main kernel's (limit: f16 outputs
// stay within +-65504), and behind that, if
// p.scores is set, of the kernel that adds the weights up.
pa_status launch_merge(const DecodeParams& p, pa_dtype out, bool split_heads, int sms, cudaStream_t stream, bool limit = false);
// What pa_decode_weights adds to a decode call: the pool that is added to, the
// new tokens' counts (or null) and where the scores, (m, l) and first chunks go.
struct WeightsOut {
    float* weights;
    const int32_t* fresh;
    float* scores;
    float2* lse;
    int* chunk0;
};
pa_status launch_weights(const DecodeParams& p, const WeightsOut& w, cudaStream_t stream);
// Kernel entry for the given cache dtype, query dtype and head_dim, or null.
const void* decode_kernel_tc(pa_dtype kv, pa_dtype q, int D);
const void* decode_kernel_simt(pa_dtype kv, pa_dtype q, int D);
// fp8 cache (e4m3 or e5m2), tensor cores with fp8 operands, 32-token chunks.
const void* decode_kernel_e4m3(pa_dtype kv, pa_dtype q, int D);
// the same for GQA groups of at most 4 heads: keys as the MMA rows.
const void* decode_kernel_fp8t(pa_dtype kv, pa_dtype q, int D);
// several (causal) query tokens per sequence, tensor cores.
const void* decode_kernel_mq(pa_dtype kv, pa_dtype q, int D);
// the same on the 5th-generation tensor cores (tcgen05, accumulators in
// tensor memory), 16-bit caches, more than 16 (token, head) rows per KV
// head; chunks of CT = 32 tokens.
const void* decode_kernel_mq_um(pa_dtype kv, pa_dtype q, int D, int CT);
// Log-sum-exp merge; split_heads: several warps per (sequence, head), for
// partitioned sequences with many partials.
const void* reduce_kernel(pa_dtype out, int D, bool split_heads, bool limit);
// pa_decode with the weights added up.
pa_status decode_with_weights(const WeightsOut& w, void* out, const void* q, pa_dtype q_dtype, const void* k_cache,
                              const void* v_cache, pa_dtype kv_dtype, const int32_t* block_tables, int MB,
                              const int32_t* seq_lens, int B, int Hq, int Hkv, int D, int bs, int NB, float scale,
                              float k_scale, float v_scale, void* workspace, size_t workspace_bytes,
                              int32_t* err_flag, cudaStream_t stream);
// The 16-token kernels that keep the scores (f32 caches: CUDA cores), and the
// merge that keeps (m, l).
const void* decode_kernel_weights(pa_dtype kv, pa_dtype q, int D);
const void* reduce_kernel_weights(pa_dtype out, int D, bool limit);
}  // namespace pa
