// pa_cache4.cu -- writes into 4-bit pools (pa_reshape_and_cache with
// PA_INT4) and reads of cached rows back as values (pa_gather_cache, every
// cache type).
//
// A unit of work is one (token, KV head, K or V) row: head_dim / 16 lanes take
// 16 elements each with 16-byte accesses.  The write reduces the row's
// extremes over those lanes, rounds (step, low) once and stores 16 codes per
// lane, so a row is one contiguous 64-byte (head_dim 128) store; the gather is
// the same in the other direction.  Both move each byte once.  The write is
// bound by its arithmetic (16 elements per lane halve what a row costs beside
// its elements; codes come from plain f32 quotients but for the few next to
// a border), the gather by HBM, both by the launch for the tokens of a step.
// 65536 tokens of 8 heads x 128, bf16: 105 us (HBM alone 50) and 64 us (50).
// Reads of the other caches move bits, or widen fp8: the same tokens of f16 82 us
// (79), f32 166 (159), e4m3 to bf16 72 (60), 4 bits and e4m3 to f32 137 and 140
// (90 and 99).
#include <cstdio>

#include "pa_cache4.h"
#include "pa_common.h"
#include "pa_int4.cuh"

namespace pa {

constexpr int ROW_THREADS = 256;
// Elements per lane.  (32 in the write: 108 us as with 16, and 2 us more for
// the 64 tokens of a step.)
constexpr int EPL = 16;

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

// x / d for a divisor that is the same for a whole launch: m = ceil(2^32 / d)
// gives a quotient that is right or one too large.
struct Div {
    uint32_t d, m;
};
__device__ __forceinline__ uint32_t div_by(uint32_t x, Div v) {
    if (v.d == 1) return x;
    const uint32_t q = __umulhi(x, v.m);
    return q - (q * v.d > x ? 1u : 0u);
}

struct RowArgs {
    const int64_t* slots;
    uint32_t rows, nslots;                           // tokens x heads; slots of the pool
    Div heads, bs;
    int32_t* err;
};

// The (token, head) row of this thread's lane group, in K (blockIdx.y 0) or V:
// false behind the last.
struct RowId {
    uint32_t t, h, blk, off;
};
template <int LPR>                                   // lanes per row
__device__ __forceinline__ bool row_id(const RowArgs& a, RowId& r) {
    const uint32_t u = blockIdx.x * (ROW_THREADS / LPR) + threadIdx.x / LPR;
    r.t = div_by(u, a.heads);
    r.h = u - r.t * a.heads.d;
    return u < a.rows;
}
// Its place in the pool: false for padding and, flagged, outside the pool.
template <int LPR>
__device__ __forceinline__ bool row_place(const RowArgs& a, int64_t slot, RowId& r) {
    if (slot < 0) return false;
    if (slot >= static_cast<int64_t>(a.nslots)) {
        if (threadIdx.x % LPR == 0) raise_flag(a.err, PA_ERRBIT_BAD_SLOT);
        return false;
    }
    r.blk = div_by(static_cast<uint32_t>(slot), a.bs);
    r.off = static_cast<uint32_t>(slot) - r.blk * a.bs.d;
    return true;
}

template <class S, int D>
__global__ void __launch_bounds__(ROW_THREADS)
write4_kernel(uint8_t* __restrict__ kc, uint8_t* __restrict__ vc, const uint8_t* __restrict__ key,
              const uint8_t* __restrict__ value, const __grid_constant__ RowArgs a) {
    grid_dependents_launch();
    constexpr int LPR = D / EPL;
    const bool v = blockIdx.y != 0;
    RowId r;
    bool on = row_id<LPR>(a, r);
    const int j = threadIdx.x % LPR;
    constexpr int NW = EPL / 8;                    // code words per lane
    float x[NW][8];
    float mn = INFINITY, mx = -INFINITY;
    int64_t slot = -1;
    if (on) {                                        // the source row and its slot load together
        slot = __ldg(a.slots + r.t);
        const uint8_t* src = (v ? value : key) + ((static_cast<size_t>(r.t) * a.heads.d + r.h) * D + j * EPL) * S::bytes;
#pragma unroll
        for (int y = 0; y < NW; ++y) load8<S>(src + 8 * y * S::bytes, x[y]);
#pragma unroll
        for (int k = 0; k < EPL; ++k) {
            mn = min_nan(mn, x[k / 8][k % 8]);
            mx = max_nan(mx, x[k / 8][k % 8]);
        }
    }
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) {          // groups are whole: a warp's lanes all take part
        mn = min_nan(mn, __shfl_xor_sync(0xffffffffu, mn, o));
        mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    }
    on = on && row_place<LPR>(a, slot, r);
    if (!on) return;
    const bool nan = mn != mn;
    if (mx > 65504.f || mn < -65504.f) {
#pragma unroll
        for (int k = 0; k < EPL; ++k) x[k / 8][k % 8] = fminf(fmaxf(x[k / 8][k % 8], -65504.f), 65504.f);
        mn = fminf(fmaxf(mn, -65504.f), 65504.f);
        mx = fminf(fmaxf(mx, -65504.f), 65504.f);
    }
    __half step, low;
    int4_params(mn, mx, step, low);
    uint32_t w[NW] = {};
    if (nan) {
        step = low = __ushort_as_half(0x7e00);
    } else {
        const float fl = __half2float(low), fs = __half2float(step);
        if (fs > 0.f) {
            const float r15 = rcp_approx(15.f * fs);      // 15 * step is exact
            float near = 0.f;
#pragma unroll
            for (int y = 0; y < NW; ++y) w[y] = int4_codes8(x[y], fl, r15, near);
            if (near > INT4_NEAR) {
                const float rs = 1.f / fs;
#pragma unroll
                for (int y = 0; y < NW; ++y) {
                    w[y] = 0;
#pragma unroll
                    for (int k = 0; k < 8; ++k) w[y] |= int4_code(x[y][k], fl, fs, rs) << (4 * k);
                }
            }
        }
    }
    uint8_t* blk = (v ? vc : kc) + static_cast<size_t>(r.blk) * a.bs.d * a.heads.d * (D / 2 + INT4_PARAM_BYTES);
    *reinterpret_cast<uint2*>(blk + int4_code_off(r.h, r.off, a.bs.d, D) + 8 * j) = make_uint2(w[0], w[1]);
    if (j == 0)
        *reinterpret_cast<__half2*>(blk + int4_param_off(r.h, r.off, a.bs.d, D, a.heads.d)) = __halves2half2(step, low);
}

// Rows of a 4-bit pool as values.
template <class S, int D>
__global__ void __launch_bounds__(ROW_THREADS)
gather4_kernel(uint8_t* __restrict__ key, uint8_t* __restrict__ value, const uint8_t* __restrict__ kc,
               const uint8_t* __restrict__ vc, const __grid_constant__ RowArgs a) {
    constexpr int LPR = D / EPL;
    const bool v = blockIdx.y != 0;
    RowId r;
    if (!row_id<LPR>(a, r) || !row_place<LPR>(a, __ldg(a.slots + r.t), r)) return;
    const int j = threadIdx.x % LPR;
    const uint8_t* blk = (v ? vc : kc) + static_cast<size_t>(r.blk) * a.bs.d * a.heads.d * (D / 2 + INT4_PARAM_BYTES);
    const uint2 w = *reinterpret_cast<const uint2*>(blk + int4_code_off(r.h, r.off, a.bs.d, D) + 8 * j);
    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(blk + int4_param_off(r.h, r.off, a.bs.d, D, a.heads.d)));
    uint8_t* dst = (v ? value : key) + ((static_cast<size_t>(r.t) * a.heads.d + r.h) * D + j * EPL) * S::bytes;
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        float x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            x[k] = int4_value(((y ? w.y : w.x) >> (4 * k)) & 15u, p.y, p.x);
            if constexpr (S::code == PA_F16) x[k] = limit_f16(x[k]);
        }
        store8<S>(dst + 8 * y * S::bytes, x);
    }
}

// Rows of the other caches: bits for equal types, fp8 codes times their scale
// otherwise (rounded to f32, then to the destination type).
template <class KV, class S, int D>
__global__ void __launch_bounds__(ROW_THREADS)
gather_kernel(uint8_t* __restrict__ key, uint8_t* __restrict__ value, const uint8_t* __restrict__ kc,
              const uint8_t* __restrict__ vc, float k_scale, float v_scale, const __grid_constant__ RowArgs a) {
    constexpr int LPR = D / EPL;
    const bool v = blockIdx.y != 0;
    RowId r;
    if (!row_id<LPR>(a, r) || !row_place<LPR>(a, __ldg(a.slots + r.t), r)) return;
    const int j = threadIdx.x % LPR;
    const size_t slot = static_cast<size_t>(r.blk) * a.bs.d + r.off;
    const uint8_t* src = (v ? vc : kc) + ((slot * a.heads.d + r.h) * D + j * EPL) * KV::bytes;
    uint8_t* dst = (v ? value : key) + ((static_cast<size_t>(r.t) * a.heads.d + r.h) * D + j * EPL) * S::bytes;
    if constexpr (KV::code == S::code) {
        constexpr int N = EPL * KV::bytes / 16;
        uint4 x[N];
#pragma unroll
        for (int y = 0; y < N; ++y) x[y] = reinterpret_cast<const uint4*>(src)[y];
#pragma unroll
        for (int y = 0; y < N; ++y) reinterpret_cast<uint4*>(dst)[y] = x[y];
    } else {
        const uint4 raw = *reinterpret_cast<const uint4*>(src);
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
        const float sc = v ? v_scale : k_scale;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            float x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint8_t c = static_cast<uint8_t>(w[2 * y + k / 4] >> (8 * (k & 3)));
                x[k] = (KV::code == PA_FP8_E5M2 ? e5m2_to_float(c) : fp8_to_float(c)) * sc;
            }
            store8<S>(dst + 8 * y * S::bytes, x);
        }
    }
}

static Div make_div(int d) {
    return Div{static_cast<uint32_t>(d), static_cast<uint32_t>(((1ull << 32) + d - 1) / d)};
}
static RowArgs row_args(const int64_t* slots, int T, int Hkv, int bs, int NB, int32_t* err) {
    return RowArgs{slots, static_cast<uint32_t>(T) * static_cast<uint32_t>(Hkv), static_cast<uint32_t>(NB) * static_cast<uint32_t>(bs),
                   make_div(Hkv), make_div(bs), err};
}
// Row and slot numbers in 31 bits, as the decode kernels ask for.
static bool rows_fit(int T, int Hkv, int bs, int NB) {
    return static_cast<int64_t>(T) * Hkv < (1LL << 31) && static_cast<int64_t>(NB) * bs < (1LL << 31);
}
static dim3 row_grid(const RowArgs& a, int lanes_per_row) {
    const uint32_t per = ROW_THREADS / lanes_per_row;
    return dim3((a.rows + per - 1) / per, 2);
}

pa_status write_int4(void* kc, void* vc, const void* key, const void* value, pa_dtype src, const int64_t* slots, int T,
                     int Hkv, int D, int bs, int NB, int32_t* err, cudaStream_t stream) {
    if (D != 64 && D != 128) return fail(PA_ERR_UNSUPPORTED, "reshape_and_cache: a 4-bit cache needs head_dim 64 or 128");
    if (bs % 8 != 0) return fail(PA_ERR_UNSUPPORTED, "reshape_and_cache: a 4-bit cache needs a block_size of a multiple of 8");
    if (!rows_fit(T, Hkv, bs, NB)) return fail(PA_ERR_UNSUPPORTED, "reshape_and_cache: pool or call too large for 32-bit row numbers");
    if (!block_fits(PA_INT4, Hkv, D, bs)) return fail(PA_ERR_UNSUPPORTED, "reshape_and_cache: a 4-bit block of 2 GB or more");
    const RowArgs a = row_args(slots, T, Hkv, bs, NB, err);
    const dim3 grid = row_grid(a, D / EPL);
#define PA_W4(ST, DD)                                                                                              \
    write4_kernel<ST, DD><<<grid, ROW_THREADS, 0, stream>>>(                                                        \
        static_cast<uint8_t*>(kc), static_cast<uint8_t*>(vc), static_cast<const uint8_t*>(key),                     \
        static_cast<const uint8_t*>(value), a)
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
static void launch_gather(uint8_t* key, uint8_t* value, const uint8_t* kc, const uint8_t* vc, int D, float ks, float vs,
                          const RowArgs& a, cudaStream_t stream) {
    const dim3 grid = row_grid(a, D / EPL);
    if constexpr (std::is_same<KV, void>::value) {
        if (D == 128) gather4_kernel<S, 128><<<grid, ROW_THREADS, 0, stream>>>(key, value, kc, vc, a);
        else gather4_kernel<S, 64><<<grid, ROW_THREADS, 0, stream>>>(key, value, kc, vc, a);
    } else {
        if (D == 128) gather_kernel<KV, S, 128><<<grid, ROW_THREADS, 0, stream>>>(key, value, kc, vc, ks, vs, a);
        else gather_kernel<KV, S, 64><<<grid, ROW_THREADS, 0, stream>>>(key, value, kc, vc, ks, vs, a);
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
    if (!rows_fit(num_tokens, num_kv_heads, block_size, num_blocks))
        return fail(PA_ERR_UNSUPPORTED, "gather_cache: pool or call too large for 32-bit row numbers");
    if (is_int4(kv_dtype) && !block_fits(kv_dtype, num_kv_heads, head_dim, block_size))
        return fail(PA_ERR_UNSUPPORTED, "gather_cache: a 4-bit block of 2 GB or more");
    if (is_fp8(dst_dtype)) return fail(PA_ERR_UNSUPPORTED, "gather_cache: the destination must be f32, f16 or bf16");
    if (is_fp8(kv_dtype) && (!(k_scale > 0.f) || !(v_scale > 0.f) || !isfinite_host(k_scale) || !isfinite_host(v_scale)))
        return fail(PA_ERR_INVALID_ARG, "gather_cache: fp8 scales must be finite and > 0");
    if (!is_fp8(kv_dtype) && !is_int4(kv_dtype) && kv_dtype != dst_dtype)
        return fail(PA_ERR_UNSUPPORTED, "gather_cache: the destination type must equal the cache's (fp8 and 4-bit caches excepted)");
    const RowArgs a = row_args(slot_mapping, num_tokens, num_kv_heads, block_size, num_blocks, err_flag);
#define PA_GA(KV, ST)                                                                                              \
    launch_gather<KV, ST>(static_cast<uint8_t*>(key), static_cast<uint8_t*>(value),                                 \
                          static_cast<const uint8_t*>(k_cache), static_cast<const uint8_t*>(v_cache), head_dim,     \
                          k_scale, v_scale, a, stream)
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
