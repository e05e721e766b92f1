// pa_weights.cu -- pa_decode_weights: a decode step that also adds each key's
// softmax weight, summed over the query heads of its group, to a pool of
// accumulated weights.
//
// The output is pa_decode's.  The weights come from one CTA per (sequence, KV
// head): for each head of the group a first pass over the keys finds the
// maximum and the sum of the softmax, a second adds exp(s - max) / sum to the
// keys' entries; scores in f32, one thread per key.
#include "pa_common.h"
#include "pa_int4.cuh"
#include "pa_kernels.h"

namespace pa {

struct WeightsArgs {
    float* weights;               // [NB][Hkv][bs]
    const void* q;
    const uint8_t* k;
    const int32_t* tables;
    const int32_t* lens;
    const int32_t* fresh;
    int32_t* err;
    int MB, Hq, Hkv, G, D, bs, NB;
    float qk_scale;               // scale * log2(e) (* k_scale for fp8)
};

struct Int4T { static constexpr pa_dtype code = PA_INT4; static constexpr int bytes = 0; };
constexpr int WT_THREADS = 256;

// <q, K_t> of one key row.
template <class KV>
__device__ __forceinline__ float key_dot(const WeightsArgs& a, const float* q, int block, int off, int g) {
    float s = 0.f;
    if constexpr (KV::code == PA_INT4) {
        const uint8_t* b = a.k + static_cast<size_t>(block) * a.bs * a.Hkv * (a.D / 2 + INT4_PARAM_BYTES);
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(b + int4_param_off(g, off, a.bs, a.D, a.Hkv)));
        const uint8_t* c = b + int4_code_off(g, off, a.bs, a.D);
        for (int d = 0; d < a.D; d += 2) {
            const uint32_t x = c[d / 2];
            s = fmaf(q[d], int4_value(x & 15u, p.y, p.x), s);
            s = fmaf(q[d + 1], int4_value(x >> 4, p.y, p.x), s);
        }
    } else {
        const typename KV::T* row = reinterpret_cast<const typename KV::T*>(a.k) +
                                    ((static_cast<size_t>(block) * a.bs + off) * a.Hkv + g) * a.D;
        for (int d = 0; d < a.D; ++d) {
            float x;
            if constexpr (KV::code == PA_FP8_E4M3) x = fp8_to_float(row[d]);
            else if constexpr (KV::code == PA_FP8_E5M2) x = e5m2_to_float(row[d]);
            else x = to_float(row[d]);
            s = fmaf(q[d], x, s);
        }
    }
    return s * a.qk_scale;
}

template <class KV, class QT>
__global__ void __launch_bounds__(WT_THREADS)
weights_kernel(const __grid_constant__ WeightsArgs a) {
    __shared__ float q[128];
    __shared__ float rm[WT_THREADS / 32], rs[WT_THREADS / 32];
    grid_dependency_wait();
    const int i = blockIdx.x, g = blockIdx.y, tid = threadIdx.x;
    const int L = min(max(a.lens[i], 0), a.MB * a.bs);
    const int first_fresh = L - (a.fresh ? min(max(a.fresh[i], 0), L) : min(L, 1));
    const int32_t* bt = a.tables + static_cast<size_t>(i) * a.MB;
    for (int r = 0; r < a.G; ++r) {
        __syncthreads();
        const typename QT::T* qr = static_cast<const typename QT::T*>(a.q) +
                                   (static_cast<size_t>(i) * a.Hq + g * a.G + r) * a.D;
        for (int d = tid; d < a.D; d += WT_THREADS) q[d] = to_float(qr[d]);
        __syncthreads();
        float m = -INFINITY, l = 0.f;
        for (int t = tid; t < L; t += WT_THREADS) {
            const int b = bt[t / a.bs];
            if (b < 0 || b >= a.NB) continue;
            const float s = key_dot<KV>(a, q, b, t % a.bs, g);
            const float mn = fmaxf(m, s);
            l = l * exp2f(m - mn) + exp2f(s - mn);
            m = mn;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, m, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
            const float mn = fmaxf(fmaxf(m, m2), -1e38f);
            l = l * exp2f(m - mn) + l2 * exp2f(m2 - mn);
            m = mn;
        }
        if ((tid & 31) == 0) { rm[tid >> 5] = m; rs[tid >> 5] = l; }
        __syncthreads();
        float M = -1e38f, den = 0.f;
        for (int w = 0; w < WT_THREADS / 32; ++w) M = fmaxf(M, rm[w]);
        for (int w = 0; w < WT_THREADS / 32; ++w) den += rs[w] * exp2f(rm[w] - M);
        for (int t = tid; t < L; t += WT_THREADS) {
            const int b = bt[t / a.bs];
            if (b < 0 || b >= a.NB) continue;
            const float p = exp2f(key_dot<KV>(a, q, b, t % a.bs, g) - M) / den;
            float* w = a.weights + (static_cast<size_t>(b) * a.Hkv + g) * a.bs + t % a.bs;
            *w = (r == 0 && t >= first_fresh) ? p : *w + p;
        }
    }
}

template <class KV>
static const void* weights_fn(pa_dtype q) {
    if (q == PA_F32) return reinterpret_cast<const void*>(&weights_kernel<KV, F32T>);
    if (q == PA_F16) return reinterpret_cast<const void*>(&weights_kernel<KV, F16T>);
    return reinterpret_cast<const void*>(&weights_kernel<KV, BF16T>);
}

}  // namespace pa

using namespace pa;

extern "C" size_t pa_decode_weights_workspace_size(int num_seqs, int num_q_heads, int max_seq_len, int head_dim) {
    return pa_decode_workspace_size(num_seqs, num_q_heads, max_seq_len, head_dim, 0);
}

extern "C" pa_status pa_decode_weights(void* out, float* weights, const void* q, pa_dtype q_dtype,
                                       const void* k_cache, const void* v_cache, pa_dtype kv_dtype,
                                       const int32_t* block_tables, int max_blocks_per_seq,
                                       const int32_t* seq_lens, const int32_t* fresh, int num_seqs, int num_q_heads,
                                       int num_kv_heads, int head_dim, int block_size, int num_blocks,
                                       float scale, float k_scale, float v_scale, void* workspace,
                                       size_t workspace_bytes, int32_t* err_flag, cudaStream_t stream) {
    clear_error();
    if (num_seqs > 0 && !weights) return fail(PA_ERR_INVALID_ARG, "decode_weights: null pointer");
    if (num_seqs > 0 && !aligned16(weights)) return fail(PA_ERR_INVALID_ARG, "decode_weights: weights must be 16-byte aligned");
    const pa_status st = decode_weights_out(out, q, q_dtype, k_cache, v_cache, kv_dtype, block_tables,
                                            max_blocks_per_seq, seq_lens, num_seqs, num_q_heads, num_kv_heads, head_dim,
                                            block_size, num_blocks, scale, k_scale, v_scale, workspace,
                                            workspace_bytes, err_flag, stream);
    if (st != PA_OK || num_seqs == 0) return st;
    WeightsArgs a{weights, q, static_cast<const uint8_t*>(k_cache), block_tables, seq_lens, fresh, err_flag,
                  max_blocks_per_seq, num_q_heads, num_kv_heads, num_q_heads / num_kv_heads, head_dim, block_size,
                  num_blocks, scale * 1.4426950408889634f * (is_fp8(kv_dtype) ? k_scale : 1.f)};
    const void* fn = kv_dtype == PA_F32 ? weights_fn<F32T>(q_dtype) : kv_dtype == PA_F16 ? weights_fn<F16T>(q_dtype)
                     : kv_dtype == PA_BF16 ? weights_fn<BF16T>(q_dtype)
                     : kv_dtype == PA_FP8_E4M3 ? weights_fn<FP8T>(q_dtype)
                     : kv_dtype == PA_FP8_E5M2 ? weights_fn<E5M2T>(q_dtype) : weights_fn<Int4T>(q_dtype);
    void* args[] = {&a};
    const cudaError_t e = cudaLaunchKernel(fn, dim3(static_cast<unsigned>(num_seqs), static_cast<unsigned>(num_kv_heads)),
                                           dim3(WT_THREADS), args, 0, stream);
    return e == cudaSuccess ? PA_OK : fail_cuda("decode_weights launch", e);
}
