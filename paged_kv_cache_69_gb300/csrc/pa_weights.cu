// pa_weights.cu -- pa_decode_weights: a decode step that also adds each key's
// softmax weight, summed over the query heads of its group, to a pool of
// accumulated weights.
//
// The decode kernels keep what they have in hand: the scores of each chunk
// (f32, log2 units, [chunk][head][token]) and, per sequence and head, the
// maximum m and the sum l of the softmax, from the segment that covers a whole
// sequence or from the merge.  The kernel here then forms
//   w[g][t] = sum over the heads h of group g of 2^(s[h][t] - m[h]) / l[h]
// and adds it to the entry of each token.  Reading the scores back costs
// 4 bytes per token and query head, where a second pass over the keys would
// cost head_dim elements per KV head.  A thread takes four tokens of one KV
// head: 16-byte loads of each head's scores and one 16-byte update.
//
// Measured: the 7B-like batch of 64 in f16 118 us, of which pa_decode alone
// takes 92 (514 MB of keys and values; 28 MB of scores written and read, 8 MB
// of weights updated); 8 sequences of 32k-131k tokens in 4 bits 221 against
// 183 (83 MB of scores, written and read).  The rest is the merge's and this
// kernel's start and end behind the decode kernel.  Keys and values are marked
// to leave L2 first, so that most scores are still there when they are read.
// A batch of 64 and 287306 tokens in e4m3 takes 105 us (pa_decode's own fp8
// kernel 71, bytes 45), in 4 bits 60 (52, 25), in f32 3720 (3830, 175; CUDA
// cores).  The scores have room for every place of the table, 4 bytes per query
// head, and the grid covers it: under tables for 131072 tokens those 64
// sequences need 945 MB of workspace instead of 64 and 7 to 10 us more.
#include <cuda.h>

#include "pa_common.h"
#include "pa_decode_kernel.cuh"
#include "pa_kernels.h"

namespace pa {

constexpr int WT_THREADS = 256;
constexpr int WT_STEPS = 4;                   // token spans of a CTA, one after another

// NH: heads of a group whose scores are loaded at once.
// What kernels before the decode kernel wrote is final when this grid starts
// (it follows the merge's start, that the decode kernel's wait), so lengths
// and tables are read before the wait for this call's own results.
template <int NH>
__global__ void __launch_bounds__(WT_THREADS, NH == 4 ? 4 : 3)
weights_kernel(const __grid_constant__ DecodeParams p, float* __restrict__ weights, const int32_t* __restrict__ fresh,
               int quads, int bs_log2, int ct_log2) {
    // consecutive threads: consecutive quads of tokens of one KV head
    const int i = blockIdx.y, x = threadIdx.x, g = blockIdx.z * (WT_THREADS / quads) + x / quads;
    const int span = 4 * quads, t0 = static_cast<int>(blockIdx.x) * WT_STEPS * span;
    int t = t0 + 4 * (x & (quads - 1));
    const int maxL = p.MB << bs_log2;
    const int L = clamp_len(p.seq_lens[i], maxL);
    const int32_t* bt = p.block_tables + static_cast<size_t>(i) * p.MB;
    int next = t < maxL ? __ldg(bt + (t >> bs_log2)) : -1;
    const int old_until = L - (fresh ? min(max(fresh[i], 0), L) : 1);
    grid_dependency_wait();
    if (t0 >= L || g >= p.Hkv) return;
    const float* scores = score_row(p, p.chunk0[i], g * p.G);
    const float2* lse = p.lse + static_cast<size_t>(i) * p.Hq + g * p.G;
    const size_t chunk = static_cast<size_t>(p.Hq) << ct_log2;
#pragma unroll 1
    for (int k = 0; k < WT_STEPS && t < L; ++k, t += span) {
        const int b = next;
        next = t + span < maxL ? __ldg(bt + ((t + span) >> bs_log2)) : -1;
        if (b < 0 || b >= p.NB) continue;                     // a bad block is left out of the softmax, too
        float* dst = weights + ((static_cast<size_t>(b) * p.Hkv + g) << bs_log2) + (t & (p.bs - 1));
        const float4 old = *reinterpret_cast<const float4*>(dst);
        const float* sp = scores + (t >> ct_log2) * chunk + (t & (p.ct - 1));
        float w[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int r0 = 0; r0 < p.G; r0 += NH) {
            float4 s[NH];
#pragma unroll
            for (int r = 0; r < NH; ++r)
                if (r0 + r < p.G) s[r] = __ldcs(reinterpret_cast<const float4*>(sp + (static_cast<size_t>(r0 + r) << ct_log2)));
#pragma unroll
            for (int r = 0; r < NH; ++r)
                if (r0 + r < p.G) {
                    const float2 ml = lse[r0 + r];
                    // a head whose scores are all -infinity has the output 0, and no weights
                    const float m = ml.x == -INFINITY ? 0.f : ml.x, inv = ml.y == 0.f ? 0.f : 1.f / ml.y;
                    w[0] = fmaf(ex2_approx(s[r].x - m), inv, w[0]);
                    w[1] = fmaf(ex2_approx(s[r].y - m), inv, w[1]);
                    w[2] = fmaf(ex2_approx(s[r].z - m), inv, w[2]);
                    w[3] = fmaf(ex2_approx(s[r].w - m), inv, w[3]);
                }
        }
        float o[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (t + e < L) o[e] = (t + e < old_until ? o[e] : 0.f) + w[e];
        *reinterpret_cast<float4*>(dst) = make_float4(o[0], o[1], o[2], o[3]);
    }
}

pa_status launch_weights(const DecodeParams& p, const WeightsOut& w, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    // a CTA: WT_STEPS spans of 4 * quads tokens, of 256 / quads KV heads
    int quads = 8;
    while (quads < WT_THREADS && WT_THREADS / (2 * quads) >= p.Hkv) quads *= 2;
    const int heads = WT_THREADS / quads;
    cfg.gridDim = dim3(static_cast<unsigned>((static_cast<long long>(p.MB) * p.bs + WT_STEPS * 4 * quads - 1) / (WT_STEPS * 4 * quads)),
                       static_cast<unsigned>(p.B), static_cast<unsigned>((p.Hkv + heads - 1) / heads));
    cfg.blockDim = dim3(WT_THREADS);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    DecodeParams arg = p;
    float* weights = w.weights;
    const int32_t* fresh = w.fresh;
    int bs_log2 = 3, ct_log2 = 4;             // block sizes and chunks are powers of two
    while ((1 << bs_log2) < p.bs) ++bs_log2;
    while ((1 << ct_log2) < p.ct) ++ct_log2;
    void* args[] = {&arg, &weights, &fresh, &quads, &bs_log2, &ct_log2};
    const cudaError_t e = cudaLaunchKernelExC(&cfg, p.G <= 4 ? reinterpret_cast<const void*>(&weights_kernel<4>)
                                                          : reinterpret_cast<const void*>(&weights_kernel<8>), args);
    return e == cudaSuccess ? PA_OK : fail_cuda("decode_weights launch", e);
}

const void* decode_kernel_weights(pa_dtype kv, pa_dtype q, int D) {
#define PA_WT(KVT, QTT, DD, TC) reinterpret_cast<const void*>(&pa_decode_kernel<KVT, QTT, DD, TC, 16, false, false, false, true>)
#define PA_WTD(KVT, TC) (D == 128 ? PA_WT(KVT, KVT, 128, TC) : D == 64 ? PA_WT(KVT, KVT, 64, TC) : nullptr)
    if (kv == PA_F32 && q == PA_F32) return PA_WTD(F32T, false);
    if (kv == PA_F16 && q == PA_F16) return PA_WTD(F16T, true);
    if (kv == PA_BF16 && q == PA_BF16) return PA_WTD(BF16T, true);
    if (D != 128) return nullptr;
    if (kv == PA_FP8_E4M3) return q == PA_F16 ? PA_WT(FP8T, F16T, 128, true) : q == PA_BF16 ? PA_WT(FP8T, BF16T, 128, true) : nullptr;
    if (kv == PA_FP8_E5M2) return q == PA_F16 ? PA_WT(E5M2T, F16T, 128, true) : q == PA_BF16 ? PA_WT(E5M2T, BF16T, 128, true) : nullptr;
#undef PA_WTD
#undef PA_WT
    return nullptr;
}

const void* reduce_kernel_weights(pa_dtype out, int D, F16Out limit) {
#define PA_RED(T) (D == 128 ? reinterpret_cast<const void*>(&pa_reduce_kernel<T, 128, 1, true>) \
                   : D == 64 ? reinterpret_cast<const void*>(&pa_reduce_kernel<T, 64, 1, true>) : nullptr)
    if (out == PA_F32) return PA_RED(float);
    if (out == PA_F16)
        return limit == F16Out::LIMITED ? PA_RED(LimitedHalf) : limit == F16Out::FINITE ? PA_RED(FiniteHalf) : PA_RED(__half);
    if (out == PA_BF16) return PA_RED(__nv_bfloat16);
#undef PA_RED
    return nullptr;
}

static size_t wt_align(size_t x) { return (x + 255) & ~size_t(255); }
// A chunk has at most 128 tokens (4-bit caches).
static size_t score_bytes(int B, int Hq, int max_len) {
    return sizeof(float) * static_cast<size_t>(B) * ((static_cast<size_t>(max_len) + 127) / 128 * 128) * Hq;
}

}  // namespace pa

using namespace pa;

extern "C" size_t pa_decode_weights_workspace_size(int num_seqs, int num_q_heads, int max_seq_len, int head_dim) {
    const size_t base = pa_decode_workspace_size(num_seqs, num_q_heads, max_seq_len, head_dim, 0);
    if (base == 0) return 0;
    return wt_align(base) + wt_align(sizeof(int) * static_cast<size_t>(num_seqs)) +
           wt_align(sizeof(float2) * static_cast<size_t>(num_seqs) * num_q_heads) +
           wt_align(score_bytes(num_seqs, num_q_heads, max_seq_len));
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
    if (num_seqs > 65535) return fail(PA_ERR_UNSUPPORTED, "decode_weights: more than 65535 sequences");
    WeightsOut w{weights, fresh, nullptr, nullptr, nullptr};
    if (num_seqs > 0 && num_q_heads > 0 && head_dim > 0 && max_blocks_per_seq > 0 && block_size > 0 &&
        static_cast<long long>(max_blocks_per_seq) * block_size < (1LL << 30) && workspace) {
        // the parts behind pa_decode's workspace; a missing device is reported below
        const int max_len = max_blocks_per_seq * block_size;
        const size_t base = pa_decode_workspace_size(num_seqs, num_q_heads, max_len, head_dim, 0);
        if (base != 0) {
            if (workspace_bytes < pa_decode_weights_workspace_size(num_seqs, num_q_heads, max_len, head_dim))
                return fail(PA_ERR_WORKSPACE, "decode_weights: workspace smaller than pa_decode_weights_workspace_size()");
            uint8_t* ws = static_cast<uint8_t*>(workspace) + wt_align(base);
            w.chunk0 = reinterpret_cast<int*>(ws); ws += wt_align(sizeof(int) * static_cast<size_t>(num_seqs));
            w.lse = reinterpret_cast<float2*>(ws); ws += wt_align(sizeof(float2) * static_cast<size_t>(num_seqs) * num_q_heads);
            w.scores = reinterpret_cast<float*>(ws);
        }
    }
    return decode_with_weights(w, out, q, q_dtype, k_cache, v_cache, kv_dtype, block_tables, max_blocks_per_seq,
                               seq_lens, num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, scale,
                               k_scale, v_scale, workspace, workspace_bytes, err_flag, stream);
}
