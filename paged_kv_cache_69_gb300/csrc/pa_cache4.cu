// pa_cache4.cu -- writes into 4-bit pools (pa_reshape_and_cache with
// PA_INT4) and reads of cached rows back as values (pa_gather_cache, every
// cache type).
//
// A unit of work is one (token, KV head, K or V) row: head_dim / 8 lanes take
// 8 elements each with 16-byte accesses.  The write reduces the row's
// extremes over those lanes, rounds (step, low) once and stores 8 codes per
// lane as one word, so a row is one contiguous 64-byte (head_dim 128) store;
// the gather is the same in the other direction.  Both move each byte once and
// keep nothing between rows: they are bound by HBM once a few thousand rows
// are in flight, and by the launch for the tokens of a decode step.
#include <cstdio>

#include "pa_cache4.h"
#include "pa_common.h"
#include "pa_int4.cuh"

namespace pa {

constexpr int ROW_THREADS = 256;

// 8 consecutive elements as floats.
template <class S>
__device__ __forceinline__ void load8(const uint8_t* src, float (&x)[8]) {
    if constexpr (S::code == PA_F32) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(src));
        const float4 b = __ldg(reinterpret_cast<const float4*>(src) + 1);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
        const uint4 r = __ldg(reinterpret_cast<const uint4*>(src));
        const typename S::T* e = reinterpret_cast<const typename S::T*>(&r);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = to_float(e[k]);
    }
}
template <class S>
__device__ __forceinline__ void store8(uint8_t* dst, const float (&x)[8]) {
    if constexpr (S::code == PA_F32) {
        reinterpret_cast<float4*>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4*>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        constexpr bool bf = S::code == PA_BF16;
        *reinterpret_cast<uint4*>(dst) = make_uint4(pack2(x[0], x[1], bf), pack2(x[2], x[3], bf),
                                                    pack2(x[4], x[5], bf), pack2(x[6], x[7], bf));
    }
}

// The (token, head, K|V) row of this thread's lane group, or false behind the
// last.  Rows run over K then V, heads inside tokens.
struct RowId {
    int64_t t, slot;
    int h;
    bool v;
};
template <int D>
__device__ __forceinline__ bool row_id(const int64_t* slots, int64_t T, int Hkv, int64_t nslots, int32_t* err,
                                       RowId& r) {
    constexpr int LPR = D / 8;                       // lanes per row
    const int64_t u = (static_cast<int64_t>(blockIdx.x) * ROW_THREADS + threadIdx.x) / LPR;
    const int64_t n = T * Hkv;
    if (u >= 2 * n) return false;
    r.v = u >= n;
    const int64_t w = r.v ? u - n : u;
    r.t = w / Hkv;
    r.h = static_cast<int>(w - r.t * Hkv);
    r.slot = __ldg(slots + r.t);
    if (r.slot < 0) return false;
    if (r.slot >= nslots) {
        if (threadIdx.x % LPR == 0) raise_flag(err, PA_ERRBIT_BAD_SLOT);
        return false;
    }
    return true;
}

template <class S, int D>
__global__ void __launch_bounds__(ROW_THREADS)
write4_kernel(uint8_t* __restrict__ kc, uint8_t* __restrict__ vc, const uint8_t* __restrict__ key,
              const uint8_t* __restrict__ value, const int64_t* __restrict__ slots, int64_t T, int Hkv, int bs,
              int64_t nslots, int32_t* err) {
    grid_dependents_launch();
    constexpr int LPR = D / 8;
    RowId r;
    const bool on = row_id<D>(slots, T, Hkv, nslots, err, r);
    const int j = threadIdx.x % LPR;
    float x[8];
    float mn = INFINITY, mx = -INFINITY;
    int nan = 0;
    if (on) {
        load8<S>((r.v ? value : key) + ((static_cast<size_t>(r.t) * Hkv + r.h) * D + j * 8) * S::bytes, x);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            nan |= isnan(x[k]);
            x[k] = fminf(fmaxf(x[k], -65504.f), 65504.f);
            mn = fminf(mn, x[k]);
            mx = fmaxf(mx, x[k]);
        }
    }
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) {          // groups are whole: a warp's lanes all take part
        mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        nan |= __shfl_xor_sync(0xffffffffu, nan, o);
    }
    if (!on) return;
    __half step, low;
    int4_params(mn, mx, step, low);
    uint32_t w = 0;
    if (nan) {
        step = low = __ushort_as_half(0x7e00);
    } else {
        const float fl = __half2float(low), fs = __half2float(step);
        if (fs > 0.f) {
            const float rs = 1.f / fs;
#pragma unroll
            for (int k = 0; k < 8; ++k) w |= int4_code(x[k], fl, fs, rs) << (4 * k);
        }
    }
    const int64_t b = r.slot / bs;
    const int off = static_cast<int>(r.slot - b * bs);
    uint8_t* blk = (r.v ? vc : kc) + static_cast<size_t>(b) * bs * Hkv * (D / 2 + INT4_PARAM_BYTES);
    *reinterpret_cast<uint32_t*>(blk + int4_code_off(r.h, off, bs, D) + 4 * j) = w;
    if (j == 0)
        *reinterpret_cast<__half2*>(blk + int4_param_off(r.h, off, bs, D, Hkv)) = __halves2half2(step, low);
}

// Rows of a 4-bit pool as values.
template <class S, int D>
__global__ void __launch_bounds__(ROW_THREADS)
gather4_kernel(uint8_t* __restrict__ key, uint8_t* __restrict__ value, const uint8_t* __restrict__ kc,
               const uint8_t* __restrict__ vc, const int64_t* __restrict__ slots, int64_t T, int Hkv, int bs,
               int64_t nslots, int32_t* err) {
    constexpr int LPR = D / 8;
    RowId r;
    if (!row_id<D>(slots, T, Hkv, nslots, err, r)) return;
    const int j = threadIdx.x % LPR;
    const int64_t b = r.slot / bs;
    const int off = static_cast<int>(r.slot - b * bs);
    const uint8_t* blk = (r.v ? vc : kc) + static_cast<size_t>(b) * bs * Hkv * (D / 2 + INT4_PARAM_BYTES);
    const uint32_t w = *reinterpret_cast<const uint32_t*>(blk + int4_code_off(r.h, off, bs, D) + 4 * j);
    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(blk + int4_param_off(r.h, off, bs, D, Hkv)));
    float x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = int4_value((w >> (4 * k)) & 15u, p.y, p.x);
    store8<S>((r.v ? value : key) + ((static_cast<size_t>(r.t) * Hkv + r.h) * D + j * 8) * S::bytes, x);
}

// Rows of the other caches: bits for equal types, fp8 codes times their scale
// otherwise (rounded to f32, then to the destination type).
template <class KV, class S, int D>
__global__ void __launch_bounds__(ROW_THREADS)
gather_kernel(uint8_t* __restrict__ key, uint8_t* __restrict__ value, const uint8_t* __restrict__ kc,
              const uint8_t* __restrict__ vc, const int64_t* __restrict__ slots, int64_t T, int Hkv,
              int64_t nslots, float k_scale, float v_scale, int32_t* err) {
    constexpr int LPR = D / 8;
    RowId r;
    if (!row_id<D>(slots, T, Hkv, nslots, err, r)) return;
    const int j = threadIdx.x % LPR;
    const uint8_t* src = (r.v ? vc : kc) + ((static_cast<size_t>(r.slot) * Hkv + r.h) * D + j * 8) * KV::bytes;
    uint8_t* dst = (r.v ? value : key) + ((static_cast<size_t>(r.t) * Hkv + r.h) * D + j * 8) * S::bytes;
    if constexpr (KV::code == S::code) {
        if constexpr (KV::bytes == 4) {
            const uint4 a = reinterpret_cast<const uint4*>(src)[0], b = reinterpret_cast<const uint4*>(src)[1];
            reinterpret_cast<uint4*>(dst)[0] = a;
            reinterpret_cast<uint4*>(dst)[1] = b;
        } else {
            *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
        }
    } else {
        const uint2 raw = *reinterpret_cast<const uint2*>(src);
        const float sc = r.v ? v_scale : k_scale;
        float x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint8_t c = static_cast<uint8_t>((k < 4 ? raw.x : raw.y) >> (8 * (k & 3)));
            x[k] = (KV::code == PA_FP8_E5M2 ? e5m2_to_float(c) : fp8_to_float(c)) * sc;
        }
        store8<S>(dst, x);
    }
}

static unsigned row_grid(int64_t T, int Hkv, int D) {
    return static_cast<unsigned>((2 * T * Hkv * (D / 8) + ROW_THREADS - 1) / ROW_THREADS);
}

pa_status write_int4(void* kc, void* vc, const void* key, const void* value, pa_dtype src, const int64_t* slots, int T,
                     int Hkv, int D, int bs, int NB, int32_t* err, cudaStream_t stream) {
    if (D != 64 && D != 128) return fail(PA_ERR_UNSUPPORTED, "reshape_and_cache: a 4-bit cache needs head_dim 64 or 128");
    if (bs % 8 != 0) return fail(PA_ERR_UNSUPPORTED, "reshape_and_cache: a 4-bit cache needs a block_size of a multiple of 8");
    if (static_cast<int64_t>(T) * Hkv > (1LL << 34)) return fail(PA_ERR_UNSUPPORTED, "reshape_and_cache: too many rows");
    const int64_t nslots = static_cast<int64_t>(NB) * bs;
    const unsigned grid = row_grid(T, Hkv, D);
#define PA_W4(ST, DD)                                                                                              \
    write4_kernel<ST, DD><<<grid, ROW_THREADS, 0, stream>>>(                                                        \
        static_cast<uint8_t*>(kc), static_cast<uint8_t*>(vc), static_cast<const uint8_t*>(key),                     \
        static_cast<const uint8_t*>(value), slots, T, Hkv, bs, nslots, err)
#define PA_W4D(ST) do { if (D == 128) PA_W4(ST, 128); else PA_W4(ST, 64); } while (0)
    switch (src) {
        case PA_F32: PA_W4D(F32T); break;
        case PA_F16: PA_W4D(F16T); break;
        case PA_BF16: PA_W4D(BF16T); break;
        default: return fail(PA_ERR_UNSUPPORTED, "reshape_and_cache: a 4-bit cache needs an f32, f16 or bf16 source");
    }
#undef PA_W4D
#undef PA_W4
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? PA_OK : fail_cuda("reshape_and_cache launch", e);
}

template <class KV, class S>
static void launch_gather(uint8_t* key, uint8_t* value, const uint8_t* kc, const uint8_t* vc, const int64_t* slots,
                          int T, int Hkv, int D, int bs, int64_t nslots, float ks, float vs, int32_t* err,
                          cudaStream_t stream) {
    const unsigned grid = row_grid(T, Hkv, D);
    if constexpr (std::is_same<KV, void>::value) {
        if (D == 128) gather4_kernel<S, 128><<<grid, ROW_THREADS, 0, stream>>>(key, value, kc, vc, slots, T, Hkv, bs, nslots, err);
        else gather4_kernel<S, 64><<<grid, ROW_THREADS, 0, stream>>>(key, value, kc, vc, slots, T, Hkv, bs, nslots, err);
    } else {
        if (D == 128) gather_kernel<KV, S, 128><<<grid, ROW_THREADS, 0, stream>>>(key, value, kc, vc, slots, T, Hkv, nslots, ks, vs, err);
        else gather_kernel<KV, S, 64><<<grid, ROW_THREADS, 0, stream>>>(key, value, kc, vc, slots, T, Hkv, nslots, ks, vs, err);
    }
}

}  // namespace pa

using namespace pa;

extern "C" pa_status pa_gather_cache(void* key, void* value, pa_dtype dst_dtype, const void* k_cache,
                                     const void* v_cache, pa_dtype kv_dtype, const int64_t* slot_mapping,
                                     int num_tokens, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                                     float k_scale, float v_scale, int32_t* err_flag, cudaStream_t stream) {
    clear_error();
    if (num_tokens < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks <= 0)
        return fail(PA_ERR_INVALID_ARG, "gather_cache: sizes must be positive (num_tokens >= 0)");
    if (num_tokens == 0) return PA_OK;
    if (!k_cache || !v_cache || !key || !value || !slot_mapping)
        return fail(PA_ERR_INVALID_ARG, "gather_cache: null pointer");
    if (!valid_cache_dtype(kv_dtype) || !valid_dtype(dst_dtype))
        return fail(PA_ERR_INVALID_ARG, "gather_cache: unknown dtype");
    if (head_dim != 64 && head_dim != 128) return fail(PA_ERR_UNSUPPORTED, "gather_cache: head_dim must be 64 or 128");
    if (is_int4(kv_dtype) && block_size % 8 != 0)
        return fail(PA_ERR_UNSUPPORTED, "gather_cache: a 4-bit cache needs a block_size of a multiple of 8");
    if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(key) || !aligned16(value))
        return fail(PA_ERR_INVALID_ARG, "gather_cache: caches and destinations must be 16-byte aligned");
    if (static_cast<int64_t>(num_tokens) * num_kv_heads > (1LL << 34))
        return fail(PA_ERR_UNSUPPORTED, "gather_cache: too many rows");
    if (is_fp8(dst_dtype)) return fail(PA_ERR_UNSUPPORTED, "gather_cache: the destination must be f32, f16 or bf16");
    if (is_fp8(kv_dtype) && (!(k_scale > 0.f) || !(v_scale > 0.f) || !isfinite_host(k_scale) || !isfinite_host(v_scale)))
        return fail(PA_ERR_INVALID_ARG, "gather_cache: fp8 scales must be finite and > 0");
    if (!is_fp8(kv_dtype) && !is_int4(kv_dtype) && kv_dtype != dst_dtype)
        return fail(PA_ERR_UNSUPPORTED, "gather_cache: the destination type must equal the cache's (fp8 and 4-bit caches excepted)");
    const int64_t nslots = static_cast<int64_t>(num_blocks) * block_size;
#define PA_GA(KV, ST)                                                                                              \
    launch_gather<KV, ST>(static_cast<uint8_t*>(key), static_cast<uint8_t*>(value),                                 \
                          static_cast<const uint8_t*>(k_cache), static_cast<const uint8_t*>(v_cache), slot_mapping, \
                          num_tokens, num_kv_heads, head_dim, block_size, nslots, k_scale, v_scale, err_flag, stream)
#define PA_GADST(KV) do { if (dst_dtype == PA_F32) PA_GA(KV, F32T); else if (dst_dtype == PA_F16) PA_GA(KV, F16T); else PA_GA(KV, BF16T); } while (0)
    switch (kv_dtype) {
        case PA_F32: PA_GA(F32T, F32T); break;
        case PA_F16: PA_GA(F16T, F16T); break;
        case PA_BF16: PA_GA(BF16T, BF16T); break;
        case PA_FP8_E4M3: PA_GADST(FP8T); break;
        case PA_FP8_E5M2: PA_GADST(E5M2T); break;
        default: PA_GADST(void); break;
    }
#undef PA_GADST
#undef PA_GA
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? PA_OK : fail_cuda("gather_cache launch", e);
}

extern "C" size_t pa_block_bytes(pa_dtype kv_dtype, int num_kv_heads, int head_dim, int block_size) {
    if (!valid_cache_dtype(kv_dtype) || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0) return 0;
    return static_cast<size_t>(block_size) * num_kv_heads * row_bytes(kv_dtype, head_dim);
}
