// pa_shared.cu -- pa_decode_shared: a decode step of sequences that share
// prefixes, each prefix attended once for all sequences of its group.
//
// With P tokens shared, L_i of sequence i and weights e_t = exp(s_t - m),
//     out = (sum_{t<P} e_t V_t + sum_{P<=t<L_i} e_t V_t) / (sum_{t<P} e_t + sum_{P<=t<L_i} e_t)
// The first sums are one product over the prefix for the (sequence, head) rows of
// the whole group: the prompt kernel, each KV head's rows in tiles of 128, cut into
// ranges of keys.  The second ones are a decode step over the tables behind the
// prefix: the decode kernel.  Both leave partials (reference, l, O), which the kernel
// here merges, one warp per (sequence, head).  A prefix is read once per KV head and
// 256 rows instead of once per sequence.
//
// Three launches, each the dependent of the one before.  128 sequences behind 32768 tokens,
// 32/8 heads x 128, bf16, 20-2048 tokens of their own: 165 us (the bytes alone 99): the prefix 59
// (tensor cores 56% of their cycles, DRAM 30%: one span of 28 chunks per CTA, whose start and end
// nothing covers), the tails 92 (HBM, 5.9 TB/s), the merge 13 (a chain of dependent loads).  32
// groups of four behind 2048, 28/4 heads: 68 = 38 + 22 + 11; the prefix there has 28 of an item's 256
// rows, so that the score, softmax and product of a chunk follow one another (tensor cores 24%,
// DRAM 47%).  pa_decode on the first batch would read 17 GB, some 2500 us.
#include <cuda.h>

#include <algorithm>

#include "pa_common.h"
#include "pa_decode_kernel.cuh"
#include "pa_kernels.h"
#include "pa_launch.h"
#include "pa_prompt.h"
#include "pa_prompt_kernel.cuh"

namespace pa {

const void* decode_kernel_tail(pa_dtype kv, int D) {
#define PA_TAIL(KVT, DD) reinterpret_cast<const void*>(&pa_decode_kernel<KVT, KVT, DD, true, 16, false, false, false, false, true>)
    if (kv == PA_F16) return D == 128 ? PA_TAIL(F16T, 128) : D == 64 ? PA_TAIL(F16T, 64) : nullptr;
    if (kv == PA_BF16) return D == 128 ? PA_TAIL(BF16T, 128) : D == 64 ? PA_TAIL(BF16T, 64) : nullptr;
#undef PA_TAIL
    return nullptr;
}

// Partials of one (sequence, head): first those of the prefix's ranges, then those
// of the decode kernel's segments.  A lane names one partial; the columns of eight
// are in flight at a time.
template <typename OutT, int D>
__global__ void __launch_bounds__(128)
shared_merge_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ PromptParams s) {
    constexpr int DPL = D / 32;
    const int lane = threadIdx.x & 31;
    const long long w = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (w >= static_cast<long long>(p.B) * p.Hq) return;
    const int i = static_cast<int>(w / p.Hq), h = static_cast<int>(w - static_cast<long long>(i) * p.Hq);
    const int g = prompt_seq_of(s, i);
    PromptSeq q{0, 0, 0, 0, 0};
    if (g >= 0) q = prompt_seq(s, g, false);
    grid_dependency_wait();
    const int parts = min(max(s.cut[0].x, 0), s.splits);   // (behind a wait that ran out it may be anything)
    const int tail = p.seq_lens[i];
    if (tail < 0) return;
    // the prefix's partials: one per range of keys
    const int n1 = q.L > 0 ? parts : 0;
    const size_t at1 = static_cast<size_t>(w) * parts;
    // the tail's: slot range + unit for each range that holds some of its chunks
    int n2 = 0, r0 = 0, U = 0, S = 0, nch = 0;
    long long W = 0;
    bool dense = true;
    if (tail > 0) {
        S = p.chunk0[i];
        U = p.unit0[i];
        nch = cdiv_i(tail, p.ct);
        W = stream_weight(p, p.totals[0], p.totals[1]);
        r0 = range_of_pos(chunk_pos(p, S, U), W, p.NR);
        n2 = range_of_pos(chunk_pos(p, S + nch - 1, U), W, p.NR) - r0 + 1;
        dense = p.totals[0] >= p.NR || dense_ranges(p, W);
    }
    float M = -INFINITY, den = 0.f, num[DPL];
#pragma unroll
    for (int c = 0; c < DPL; ++c) num[c] = 0.f;
    for (int b = 0; b < n1 + n2; b += 32) {
        const int k = b + lane;
        const float* acc = nullptr;
        float2 ml = make_float2(-INFINITY, 0.f);
        if (k < n1) {
            const size_t at = at1 + k;
            ml = s.part_ml[at];
            acc = s.part_acc + at * D;
        } else if (k < n1 + n2) {
            const int r = r0 + k - n1, slot = r + U;
            if (slot < p.max_slots &&
                (dense || unit_in_range(r, S, S + nch, static_cast<long long>(p.WS) * (U + 1), W, p.NR, p.WQ))) {
                const size_t at = static_cast<size_t>(slot) * p.Hq + h;
                ml = p.part_ml[at];
                acc = p.part_acc + at * D;
            }
        }
        if (ml.y == 0.f) { acc = nullptr; ml.x = -INFINITY; }      // nothing in it
        float top = ml.x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float Mn = fmaxf(M, top), Mu = Mn > -INFINITY ? Mn : 0.f;
        const float old = exp2f(M - Mu), e = acc ? exp2f(ml.x - Mu) : 0.f;
        float wl = acc ? e * ml.y : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) wl += __shfl_xor_sync(0xffffffffu, wl, o);
        den = den * old + wl;
        M = Mn;
#pragma unroll
        for (int c = 0; c < DPL; ++c) num[c] *= old;
        uint32_t left = __ballot_sync(0xffffffffu, acc != nullptr);
        while (left) {
            constexpr int NB = 8;
            float v[NB][DPL], f[NB];
#pragma unroll
            for (int t = 0; t < NB; ++t) {
                const int src = left ? __ffs(left) - 1 : 0;
                const bool on = left != 0;
                left &= left - 1;
                const float* a = reinterpret_cast<const float*>(
                    __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(acc), src));
                f[t] = __shfl_sync(0xffffffffu, e, src);
                if (on) {
                    VecF<DPL>::load(a + lane * DPL, v[t]);
                } else {
                    f[t] = 0.f;
#pragma unroll
                    for (int c = 0; c < DPL; ++c) v[t][c] = 0.f;
                }
            }
#pragma unroll
            for (int t = 0; t < NB; ++t)
#pragma unroll
                for (int c = 0; c < DPL; ++c) num[c] = fmaf(f[t], v[t][c], num[c]);
        }
    }
    const float inv = den != 0.f ? 1.f / den : 0.f;
    OutT* o = static_cast<OutT*>(p.out) + (static_cast<size_t>(i) * p.Hq + h) * D + lane * DPL;
#pragma unroll
    for (int c = 0; c < DPL; ++c) o[c] = from_float<OutT>(num[c] * inv);
}

pa_status launch_shared_merge(const DecodeParams& p, const Tails& t, pa_dtype out, cudaStream_t stream) {
    const void* kern = out == PA_F16 ? (p.D == 128 ? reinterpret_cast<const void*>(&shared_merge_kernel<FiniteHalf, 128>)
                                                   : reinterpret_cast<const void*>(&shared_merge_kernel<FiniteHalf, 64>))
                                     : (p.D == 128 ? reinterpret_cast<const void*>(&shared_merge_kernel<__nv_bfloat16, 128>)
                                                   : reinterpret_cast<const void*>(&shared_merge_kernel<__nv_bfloat16, 64>));
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>((static_cast<long long>(p.B) * p.Hq + 3) / 4));
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* args[] = {const_cast<DecodeParams*>(&p), const_cast<PromptParams*>(t.prefix)};
    const cudaError_t e = cudaLaunchKernelExC(&cfg, kern, args);
    return e == cudaSuccess ? PA_OK : fail_cuda("decode_shared: merge launch", e);
}

static size_t round256(size_t x) { return (x + 255) & ~size_t(255); }
static size_t ints(int n) { return round256(sizeof(int32_t) * static_cast<size_t>(n)); }

}  // namespace pa

using namespace pa;

extern "C" size_t pa_decode_shared_workspace_size(int num_seqs, int num_groups, int num_q_heads, int num_kv_heads,
                                                  int max_seq_len, int head_dim) {
    if (num_groups < 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0 || num_q_heads / num_kv_heads > PT_M) return 0;
    const size_t base = pa_decode_workspace_size(num_seqs, num_q_heads, max_seq_len, head_dim, 0);
    DeviceInfo dev;
    if (base == 0 || !device_info(dev)) return 0;
    return round256(base) + 4 * ints(num_seqs) +
           prompt_part_bytes(num_seqs, num_q_heads, head_dim, true, dev.sms);
}

extern "C" pa_status pa_decode_shared(void* out, const void* q, pa_dtype q_dtype, const void* k_cache, const void* v_cache,
                                      pa_dtype kv_dtype, const int32_t* block_tables, int max_blocks_per_seq,
                                      const int32_t* seq_lens, const int32_t* group_start, const int32_t* prefix_lens,
                                      int num_seqs, int num_groups, int num_q_heads, int num_kv_heads, int head_dim,
                                      int block_size, int num_blocks, float scale, void* workspace, size_t workspace_bytes,
                                      int32_t* err_flag, cudaStream_t stream) {
    clear_error();
    const int B = num_seqs, Hq = num_q_heads, Hkv = num_kv_heads, D = head_dim, MB = max_blocks_per_seq;
    if (B < 0 || num_groups < 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || block_size <= 0 || num_blocks <= 0 || MB <= 0)
        return fail(PA_ERR_INVALID_ARG, "decode_shared: sizes must be positive (num_seqs and num_groups >= 0)");
    if (B == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !seq_lens || !group_start || (num_groups > 0 && !prefix_lens))
        return fail(PA_ERR_INVALID_ARG, "decode_shared: null pointer");
    if (!valid_dtype(q_dtype) || !valid_cache_dtype(kv_dtype)) return fail(PA_ERR_INVALID_ARG, "decode_shared: unknown dtype");
    if (Hq % Hkv != 0) return fail(PA_ERR_INVALID_ARG, "decode_shared: num_q_heads must be a multiple of num_kv_heads");
    if (q_dtype != kv_dtype || (q_dtype != PA_F16 && q_dtype != PA_BF16))
        return fail(PA_ERR_UNSUPPORTED, "decode_shared: f16 or bf16 queries and caches of one type");
    if (D != 64 && D != 128) return fail(PA_ERR_UNSUPPORTED, "decode_shared: head_dim must be 64 or 128");
    if (block_size != 8 && block_size != 16 && block_size != 32 && block_size != 64 && block_size != 128)
        return fail(PA_ERR_UNSUPPORTED, "decode_shared: block_size must be 8, 16, 32, 64 or 128");
    if (Hq / Hkv > PT_M) return fail(PA_ERR_UNSUPPORTED, "decode_shared: at most 128 query heads per KV head");
    if (Hkv > 256) return fail(PA_ERR_UNSUPPORTED, "decode_shared: num_kv_heads must be <= 256");
    if (static_cast<long long>(num_blocks) * block_size >= (1LL << 31) - PT_M ||
        static_cast<long long>(MB) * block_size >= (1LL << 30) ||
        (static_cast<long long>(B) + num_groups) * Hq >= (1LL << 31))
        return fail(PA_ERR_UNSUPPORTED, "decode_shared: pool, table or batch too large for 32-bit row coordinates");
    if (!aligned16(q) || !aligned16(out) || !aligned16(k_cache) || !aligned16(v_cache))
        return fail(PA_ERR_INVALID_ARG, "decode_shared: q, out, k_cache and v_cache must be 16-byte aligned");
    DeviceInfo dev;
    if (!device_info(dev)) return fail(PA_ERR_CUDA, "decode_shared: cannot query the current device");
    if (!workspace) return fail(PA_ERR_WORKSPACE, "decode_shared: workspace pointer is null");
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return fail(PA_ERR_WORKSPACE, "decode_shared: workspace must be 256-byte aligned");
    const int max_len = MB * block_size;
    if (workspace_bytes < pa_decode_shared_workspace_size(B, num_groups, Hq, Hkv, max_len, D))
        return fail(PA_ERR_WORKSPACE, "decode_shared: workspace smaller than pa_decode_shared_workspace_size()");
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const size_t base = round256(pa_decode_workspace_size(B, Hq, max_len, D, 0));
    int32_t* part[4];
    for (int x = 0; x < 4; ++x) part[x] = reinterpret_cast<int32_t*>(ws + base + x * ints(B));
    const PromptPlan plan = prompt_plan(num_groups, B, Hq, Hkv, D, max_len, false, true, dev.sms);
    const PromptCall c{"decode_shared", out, q, q_dtype, k_cache, v_cache, group_start, nullptr, prefix_lens, block_tables,
                       num_groups, Hq, Hkv, D, B, 0, block_size, num_blocks, MB, scale, true, seq_lens, part[0], part[1],
                       err_flag, stream};
    PromptParams pp;
    const pa_status st = launch_prompt(c, plan, ws + base + 4 * ints(B), &pp);
    if (st != PA_OK) return st;
    const Tails t{part[0], part[1], part[2], part[3], &pp};
    return decode_tails(t, out, q, q_dtype, k_cache, v_cache, kv_dtype, block_tables, MB, seq_lens, B, Hq, Hkv, D, block_size,
                        num_blocks, scale, workspace, base, err_flag, stream);
}
