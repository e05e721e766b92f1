// pa_prefill.cu -- pa_prefill and pa_prefill_cached: causal attention of whole
// prompts, with K and V contiguous or in the paged pool.  Argument checks, the
// plan and the launches; the kernel is in pa_prompt_kernel.cuh.
#include <cuda.h>

#include <algorithm>
#include <cmath>
#include <cstdio>

#include "pa_kernels.h"
#include "pa_launch.h"
#include "pa_prompt.h"
#include "pa_prompt_kernel.cuh"

namespace pa {

// Prefills of more rounds of items than this are not cut: their last, lightest round
// is at most a tenth of the whole.  Nor those whose last round cannot hold items of more
// chunks than PT_CUT: the merge's launch alone costs 2 us, two chunks' time (eight prompts of
// 1024 tokens 86.7 us with it, 83.9 without; one of 512 22.3 and 20.0; 256 tokens behind
// 65280, 512 chunks, 222 cut and 671 not).
constexpr int PT_ROUNDS = 8, PT_CUT = 12;

static size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// At most so many items per KV head: a sequence of n tokens has 1 + floor((n - 1) / TT).
static long long prompt_items(int B, int total_q, int TT) { return B + std::max(0, total_q - B) / TT; }

// Rows of partials of a prefill: it cuts fewer items than it has CTAs, into at most 2 ranges
// per CTA in all, each with both tiles' rows.
static size_t prefill_rows(int sms) { return 2 * static_cast<size_t>(sms) * 2 * PT_M; }

static size_t ml_size(size_t rows) { return up256(rows * sizeof(float2)); }
static size_t acc_size(size_t rows, int D) { return up256(rows * D * sizeof(float)); }
static size_t cut_size(int sms) { return up256((1 + static_cast<size_t>(sms)) * sizeof(int4)); }

PromptPlan prompt_plan(int B, int total_q, int Hq, int Hkv, int D, int max_keys, bool prompts, bool shared,
                       int sms) {
    PromptPlan pl;
    const int TT = 2 * (PT_M / (Hq / Hkv));
    const long long items = prompt_items(B, total_q, TT) * Hkv;
    const int chunks = std::max(1, (max_keys + PT_M - 1) / PT_M);
    if (shared) {
        const long long places = static_cast<long long>(total_q / TT + B + 1) * Hkv;
        pl.splits = static_cast<int>(std::min<long long>({1 + 2 * sms / places, chunks, 32}));
    } else if (items <= PT_ROUNDS * static_cast<long long>(sms)) {
        // whole prompts have items of every length: the r lightest attend at most r / Hkv
        // items' tokens
        const int last = prompts ? std::min(chunks, (sms * TT + PT_M * Hkv - 1) / (PT_M * Hkv)) : chunks;
        if (last > PT_CUT) pl.splits = std::min(chunks, 32);
    }
    pl.grid = static_cast<int>(std::max(1LL, std::min<long long>(items * pl.splits, sms)));
    if (pl.splits > 1 || shared) {
        const size_t rows = shared ? static_cast<size_t>(total_q) * Hq * pl.splits : prefill_rows(sms);
        pl.cut_bytes = cut_size(sms);
        pl.ml_bytes = ml_size(rows);
        pl.acc_bytes = acc_size(rows, D);
    }
    return pl;
}

size_t prompt_part_bytes(int total_q, int Hq, int D, bool shared, int sms) {
    size_t rows = prefill_rows(sms);
    if (shared) {
        // total_q Hq rows, each in 1 + floor(2 sms / places) ranges, of which there are 32 at most.  There
        // are more places than total_q Hq / (2 PT_M), so that the second term has fewer rows
        // than 2 sms x 2 PT_M, with fewer sequences too.
        const size_t once = static_cast<size_t>(total_q) * Hq;
        rows = std::min(once + rows, 32 * once);
    }
    return cut_size(sms) + ml_size(rows) + acc_size(rows, D);
}

static CUresult encode4(CUtensorMap* m, pa_dtype dt, const void* base, cuuint64_t d1, cuuint64_t d2, cuuint64_t planes,
                        cuuint64_t s1, cuuint64_t s2, cuuint32_t b1, cuuint32_t b2) {
    const EncodeTiledFn enc = encode_fn();
    if (!enc) return CUDA_ERROR_NOT_FOUND;
    const cuuint64_t dims[4] = {64, d1, d2, planes};
    const cuuint64_t strides[3] = {s1, s2, 128};
    const cuuint32_t box[4] = {64, b1, b2, 1}, es[4] = {1, 1, 1, 1};
    return enc(m, tmap_type(dt), 4, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// Pool rows by groups of eight: a box holds [group][plane][row][128 bytes].
static CUresult encode_pool(CUtensorMap* m, pa_dtype dt, const void* base, cuuint64_t rows, cuuint64_t Hkv, int D, int rpb) {
    const EncodeTiledFn enc = encode_fn();
    if (!enc) return CUDA_ERROR_NOT_FOUND;
    const cuuint64_t planes = D / 64, row = Hkv * D * 2;
    const cuuint64_t dims[5] = {64, 8, planes, rows / 8, Hkv};
    const cuuint64_t strides[4] = {row, 128, 8 * row, static_cast<cuuint64_t>(D) * 2};
    const cuuint32_t box[5] = {64, 8, static_cast<cuuint32_t>(planes), static_cast<cuuint32_t>(rpb / 8), 1}, es[5] = {1, 1, 1, 1, 1};
    return enc(m, tmap_type(dt), 5, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

template <class KV, int D, bool PAGED, bool SHARED = false>
static cudaError_t launch(const PromptParams& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                          cudaStream_t stream) {
    const void* kern = reinterpret_cast<const void*>(&prompt_kernel<KV, D, PAGED, SHARED>);
    cudaError_t e = allow_shared(kern, PromptLayout<D>::BYTES);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(p.grid));
    cfg.blockDim = dim3(PT_THREADS);
    cfg.dynamicSmemBytes = PromptLayout<D>::BYTES;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* args[] = {const_cast<PromptParams*>(&p), const_cast<CUtensorMap*>(&tq), const_cast<CUtensorMap*>(&tk),
                    const_cast<CUtensorMap*>(&tv)};
    if ((e = cudaLaunchKernelExC(&cfg, kern, args)) != cudaSuccess || p.splits == 1 || SHARED) return e;
    cfg.gridDim = dim3(static_cast<unsigned>(p.grid * (2 * PT_M / PT_MERGE_ROWS)));
    cfg.blockDim = dim3(32 * PT_MERGE_WARPS);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(&prompt_merge_kernel<KV, D>), args);
}

static pa_status bad(const PromptCall& c, pa_status st, const char* what) {
    char msg[192];
    std::snprintf(msg, sizeof msg, "%s: %s", c.who, what);
    return fail(st, msg);
}

pa_status launch_prompt(const PromptCall& c, const PromptPlan& plan, void* parts, PromptParams* p_out) {
    DeviceInfo dev;
    if (!device_info(dev)) return bad(c, PA_ERR_CUDA, "cannot query the current device");
    const int G = c.Hq / c.Hkv;
    PromptParams p{};
    p.out = c.out;
    p.q_start = c.q_start; p.k_start = c.k_start; p.seq_lens = c.seq_lens; p.block_tables = c.block_tables;
    p.err_flag = c.err_flag;
    p.B = c.B; p.Hq = c.Hq; p.Hkv = c.Hkv; p.G = G; p.bs = c.bs; p.NB = c.NB; p.MB = c.MB;
    p.total_q = c.total_q; p.total_k = c.total_k;
    p.tokens = PT_M / G;
    p.div_tt = make_div(2 * p.tokens);
    p.div_hkv = make_div(c.Hkv);
    p.splits = plan.splits;
    p.grid = plan.grid;
    p.causal = !c.shared;
    p.shared = c.shared;
    p.lens = c.lens; p.tail_lens = c.tail_lens; p.tail_blk = c.tail_blk;
    p.rpb = c.k_start ? PT_M : std::min(c.bs, PT_M);
    while ((1 << p.bs_log2) < c.bs) ++p.bs_log2;           // block sizes are powers of two
    while ((1 << p.rpb_log2) < p.rpb) ++p.rpb_log2;
    if (plan.acc_bytes) {
        uint8_t* at = static_cast<uint8_t*>(parts);
        p.cut = reinterpret_cast<int4*>(at);
        p.part_ml = reinterpret_cast<float2*>(at + plan.cut_bytes);
        p.part_acc = reinterpret_cast<float*>(at + plan.cut_bytes + plan.ml_bytes);
    }
    // scale enters as a positive factor of the scores' exponent; its sign goes into the MMA
    p.c = std::max(std::fabs(c.scale) * 1.4426950408889634f, 1.17549435e-38f);
    p.negate = c.scale < 0.f ? 1u << 13 : 0u;
    const cuuint64_t D2 = static_cast<cuuint64_t>(c.D) * 2, planes = c.D / 64;
    alignas(64) CUtensorMap tq, tk, tv;
    CUresult r = encode4(&tq, c.dtype, c.q, c.Hq, c.total_q, planes, D2, D2 * c.Hq, G, p.tokens);
    const void* src[2] = {c.k ? c.k : c.q, c.v ? c.v : c.q};     // (no keys: nothing is read)
    CUtensorMap* map[2] = {&tk, &tv};
    for (int x = 0; x < 2 && r == CUDA_SUCCESS; ++x)
        r = c.k_start ? encode4(map[x], c.dtype, src[x], std::max(c.total_k, 1), c.Hkv, planes, D2 * c.Hkv, D2, PT_M, 1)
                      : encode_pool(map[x], c.dtype, src[x], static_cast<cuuint64_t>(c.NB) * c.bs, c.Hkv, c.D, p.rpb);
    if (r != CUDA_SUCCESS) {
        char msg[96];
        std::snprintf(msg, sizeof msg, "cuTensorMapEncodeTiled failed (CUresult %d)", static_cast<int>(r));
        return bad(c, PA_ERR_CUDA, msg);
    }
    cudaError_t e;
#define PA_PROMPT(KVT, DD)                                                  \
    (c.shared    ? launch<KVT, DD, true, true>(p, tq, tk, tv, c.stream)     \
     : c.k_start ? launch<KVT, DD, false>(p, tq, tk, tv, c.stream)          \
                 : launch<KVT, DD, true>(p, tq, tk, tv, c.stream))
    if (c.dtype == PA_F16) e = c.D == 128 ? PA_PROMPT(F16T, 128) : PA_PROMPT(F16T, 64);
    else e = c.D == 128 ? PA_PROMPT(BF16T, 128) : PA_PROMPT(BF16T, 64);
#undef PA_PROMPT
    if (p_out) *p_out = p;
    if (e != cudaSuccess) {
        char msg[96];
        std::snprintf(msg, sizeof msg, "%s: kernel launch", c.who);
        return fail_cuda(msg, e);
    }
    return PA_OK;
}

// The checks of both calls, the plan and the launches.
static pa_status prefill(const PromptCall& c, pa_dtype kv_dtype, void* workspace, size_t workspace_bytes) {
    if (c.B < 0 || c.Hq <= 0 || c.Hkv <= 0 || c.D <= 0 || c.total_q < 0 || c.total_k < 0 || c.bs <= 0 || c.NB <= 0 || c.MB <= 0)
        return bad(c, PA_ERR_INVALID_ARG, "sizes must be positive (num_seqs and row counts >= 0)");
    if (c.B == 0 || c.total_q == 0) return PA_OK;
    const bool keys = !c.k_start || c.total_k > 0;         // without keys there are no K and V
    if (!c.out || !c.q || (keys && (!c.k || !c.v)) || !c.q_start || !(c.k_start || (c.block_tables && c.seq_lens)))
        return bad(c, PA_ERR_INVALID_ARG, "null pointer");
    if (!valid_dtype(c.dtype) || !valid_cache_dtype(kv_dtype)) return bad(c, PA_ERR_INVALID_ARG, "unknown dtype");
    if (c.Hq % c.Hkv != 0) return bad(c, PA_ERR_INVALID_ARG, "num_q_heads must be a multiple of num_kv_heads");
    if (c.dtype != kv_dtype || (c.dtype != PA_F16 && c.dtype != PA_BF16))
        return bad(c, PA_ERR_UNSUPPORTED, "q, K and V must be f16 or bf16, all of one type");
    if (c.D != 64 && c.D != 128) return bad(c, PA_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
    if (c.Hq / c.Hkv > PT_M) return bad(c, PA_ERR_UNSUPPORTED, "at most 128 query heads per KV head");
    if (c.Hkv > 256) return bad(c, PA_ERR_UNSUPPORTED, "num_kv_heads must be <= 256");
    if (c.block_tables && c.bs != 8 && c.bs != 16 && c.bs != 32 && c.bs != 64 && c.bs != 128)
        return bad(c, PA_ERR_UNSUPPORTED, "block_size must be 8, 16, 32, 64 or 128");
    if (static_cast<long long>(c.NB) * c.bs >= (1LL << 31) - PT_M || static_cast<long long>(c.MB) * c.bs >= (1LL << 30) ||
        c.total_q >= (1 << 30) || c.total_k >= (1 << 30) || (static_cast<long long>(c.total_q) + c.B) * c.Hq >= (1LL << 31))
        return bad(c, PA_ERR_UNSUPPORTED, "pool, table or batch too large for 32-bit row coordinates");
    if (!aligned16(c.q) || !aligned16(c.out) || !aligned16(c.k) || !aligned16(c.v))
        return bad(c, PA_ERR_INVALID_ARG, "q, out, K and V must be 16-byte aligned");
    DeviceInfo dev;
    if (!device_info(dev)) return bad(c, PA_ERR_CUDA, "cannot query the current device");
    const int max_keys = c.k_start ? c.total_k : c.MB * c.bs;
    const PromptPlan plan = prompt_plan(c.B, c.total_q, c.Hq, c.Hkv, c.D, max_keys, c.k_start == c.q_start, false, dev.sms);
    if (plan.acc_bytes) {
        if (!workspace) return bad(c, PA_ERR_WORKSPACE, "workspace pointer is null");
        if (workspace_bytes < plan.bytes())
            return bad(c, PA_ERR_WORKSPACE, "workspace smaller than pa_prefill_workspace_size()");
        if (reinterpret_cast<uintptr_t>(workspace) & 255u)
            return bad(c, PA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    }
    return launch_prompt(c, plan, workspace, nullptr);
}

}  // namespace pa

using namespace pa;

extern "C" size_t pa_prefill_workspace_size(int num_seqs, int total_q, int num_q_heads, int num_kv_heads, int head_dim) {
    if (num_seqs < 0 || total_q < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
        num_q_heads % num_kv_heads != 0 || num_q_heads / num_kv_heads > PT_M)
        return 0;
    DeviceInfo dev;
    if (!device_info(dev)) return 0;
    return prompt_part_bytes(total_q, num_q_heads, head_dim, false, dev.sms);
}

extern "C" pa_status pa_prefill(void* out, const void* q, const void* key, const void* value, pa_dtype dtype,
                                const int32_t* q_start, const int32_t* k_start, int num_seqs, int total_q, int total_k,
                                int num_q_heads, int num_kv_heads, int head_dim, float scale, void* workspace,
                                size_t workspace_bytes, int32_t* err_flag, cudaStream_t stream) {
    clear_error();
    PromptCall c{"prefill", out, q, dtype, key, value, q_start, k_start ? k_start : q_start, nullptr, nullptr, num_seqs,
                 num_q_heads, num_kv_heads, head_dim, total_q, total_k, PT_M, 1, 1, scale, false, nullptr, nullptr, nullptr, err_flag, stream};
    return prefill(c, dtype, workspace, workspace_bytes);
}

extern "C" pa_status pa_prefill_cached(void* out, const void* q, pa_dtype q_dtype, const void* k_cache, const void* v_cache,
                                       pa_dtype kv_dtype, const int32_t* block_tables, int max_blocks_per_seq,
                                       const int32_t* seq_lens, const int32_t* q_start, int num_seqs, int total_q,
                                       int num_q_heads, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                                       float scale, void* workspace, size_t workspace_bytes, int32_t* err_flag,
                                       cudaStream_t stream) {
    clear_error();
    PromptCall c{"prefill_cached", out, q, q_dtype, k_cache, v_cache, q_start, nullptr, seq_lens, block_tables, num_seqs,
                 num_q_heads, num_kv_heads, head_dim, total_q, 0, block_size, num_blocks, max_blocks_per_seq, scale, false, nullptr,
                 nullptr, nullptr, err_flag, stream};
    return prefill(c, kv_dtype, workspace, workspace_bytes);
}
