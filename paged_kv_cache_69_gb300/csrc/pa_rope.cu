// pa_rope.cu -- pa_rope_and_cache: new tokens' queries and keys rotated by
// their positions, K and V written into the pool, in one pass.
//
// A pair (a, b) of a row's first rot_dim elements turns by the angle of its
// token's position, whose cosine c and sine s come from a table:
//     a' = a c - b s,   b' = b c + a s   in f32, rounded once to the row's type.
// Pair i is (x[i], x[i + rot_dim / 2]) or, interleaved, (x[2 i], x[2 i + 1]).  With
// several axes of positions the pairs are dealt out to them in sections.  The
// pool gets what pa_reshape_and_cache would write of the rotated key.
//
// head_dim / 16 lanes hold a row, two groups of 8 elements each: the two halves of
// eight pairs, so that a turn stays in a lane and both are whole 16- or 32-byte
// accesses.  A lane takes NR rows of one token -- query, key and value heads in
// this order -- whose loads are all in flight before the first is used; its eight
// (c, s) serve them all.
//
// Bound by HBM on prompts: 65536 tokens of 32/8 heads x 128, bf16, 248 us, 6640 GB/s
// (326 without the hints that rows pass once, or with 256 threads; 2, 3, 6 and 8 rows
// per lane: 287, 294, 305, 436).  Slots in any order: 277 us, into 8-bit pools 315, into 4-bit
// ones 465 (a row's extremes and codes: 3.1 TB/s), with key_out 9 to 15 more.  On the 64 tokens of a
// decode step by the launch and one chain of loads (position, then table), 4.2-6.2 us, whatever
// the pool.
#include <algorithm>
#include <climits>
#include <cstdio>

#include "pa_common.h"
#include "pa_int4.cuh"
#include "pa_rows.cuh"

namespace pa {

constexpr int ROPE_THREADS = 128;
constexpr int ROPE_AXES = 4;

struct RopeArgs {
    uint8_t *kc, *vc;
    uint8_t *q_out, *key_out;                  // may be q and key: plain loads, not the read-only path
    const uint8_t *q, *key, *value;
    const int64_t *positions, *slots;          // positions [axes][T]
    const float* table;                        // [max_pos][rot]
    int32_t* err;
    int T, Hq, Hkv, D, rot, interleaved, axes, max_pos;
    int end[ROPE_AXES];                        // pairs below end[a] belong to axis a or an earlier one
    uint32_t units;                            // tokens x chunks of rows
    Div chunks, bs;
    int64_t nslots;
    float k_scale, v_scale;
};

// 8 elements as they lie in memory: what does not turn keeps its bits.  ONCE: rows of a
// prompt, which pass through L2 on their way; those of a step are read again at once.
template <class S, bool ONCE>
struct Eight {
    uint4 r[S::bytes / 2];
    __device__ __forceinline__ void load(const uint8_t* src) {
#pragma unroll
        for (int y = 0; y < S::bytes / 2; ++y) r[y] = ONCE ? __ldcs(reinterpret_cast<const uint4*>(src) + y) : reinterpret_cast<const uint4*>(src)[y];
    }
    __device__ __forceinline__ void store(uint8_t* dst) const {
#pragma unroll
        for (int y = 0; y < S::bytes / 2; ++y) {
            if constexpr (ONCE) __stcs(reinterpret_cast<uint4*>(dst) + y, r[y]);
            else reinterpret_cast<uint4*>(dst)[y] = r[y];
        }
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const typename S::T* e = reinterpret_cast<const typename S::T*>(r);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = to_float(e[k]);
    }
    __device__ __forceinline__ void set(const float (&x)[8]) { store8<S>(reinterpret_cast<uint8_t*>(r), x); }
};

template <class F8>
__device__ __forceinline__ uint2 fp8_of(const float (&x)[8], float scale) {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 8; ++k)
        w[k >> 2] |= static_cast<uint32_t>(__nv_cvt_float_to_fp8(__fdiv_rn(x[k], scale), __NV_SATFINITE,
                                                                 F8::code == PA_FP8_E5M2 ? __NV_E5M2 : __NV_E4M3))
                     << (8 * (k & 3));
    return make_uint2(w[0], w[1]);
}

struct Int4T { static constexpr int bytes = 0; static constexpr pa_dtype code = PA_INT4; };

// S: type of the rows, KV: of the pool, NR: rows per lane.
template <class S, class KV, int NR>
__global__ void __launch_bounds__(ROPE_THREADS)
rope_kernel(const __grid_constant__ RopeArgs a) {
    grid_dependents_launch();
    const int lpr = a.D / 16;
    const int j = threadIdx.x & (lpr - 1);
    const uint32_t u = blockIdx.x * (ROPE_THREADS / lpr) + threadIdx.x / lpr;
    if (u >= a.units) return;
    const uint32_t group = ((1u << lpr) - 1u) << (threadIdx.x & 31 & ~(lpr - 1));
    const uint32_t t = div_by(u, a.chunks);
    const int row0 = static_cast<int>(u - t * a.chunks.d) * NR, rows = a.Hq + 2 * a.Hkv;
    // the lane's elements: both halves of pairs 8 j .. 8 j + 7, or 16 that do not turn
    const bool turns = 8 * j < a.rot / 2;
    const int e0 = turns && !a.interleaved ? 8 * j : 16 * j;
    const int e1 = turns && !a.interleaved ? 8 * j + a.rot / 2 : 16 * j + 8;
    const int64_t slot = a.slots[t];
    int64_t pos[ROPE_AXES];
    bool in = true;
#pragma unroll
    for (int x = 0; x < ROPE_AXES; ++x) {
        pos[x] = x < a.axes ? a.positions[static_cast<size_t>(x) * a.T + t] : 0;
        in = in && pos[x] >= 0 && pos[x] < a.max_pos;
    }
    Eight<S, (NR > 1)> x0[NR], x1[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        const int row = row0 + n;
        const uint8_t* src = row < a.Hq ? a.q : row < a.Hq + a.Hkv ? a.key : a.value;
        const int h = row < a.Hq ? row : row < a.Hq + a.Hkv ? row - a.Hq : row - a.Hq - a.Hkv;
        const size_t at = (static_cast<size_t>(t) * (row < a.Hq ? a.Hq : a.Hkv) + h) * a.D;
        if (row < rows) {
            x0[n].load(src + (at + e0) * S::bytes);
            x1[n].load(src + (at + e1) * S::bytes);
        }
    }
    if (slot < 0) return;                                  // padding
    if (slot >= a.nslots || !in) {
        if (j == 0) raise_flag(a.err, (slot >= a.nslots ? PA_ERRBIT_BAD_SLOT : 0u) | (in ? 0u : PA_ERRBIT_BAD_POSITION));
        return;
    }
    if (turns && row0 < a.Hq + a.Hkv) {
        float c[8], s[8];
        // the axis of the lane's first pair, and whether the others share it
        int64_t p = pos[0];
        int end = a.end[0];
#pragma unroll
        for (int x = 1; x < ROPE_AXES; ++x)
            if (8 * j >= a.end[x - 1]) { p = pos[x]; end = a.end[x]; }
        const float* at = a.table + static_cast<size_t>(p) * a.rot + 8 * j;
        if (8 * j + 8 <= end) {
#pragma unroll
            for (int y = 0; y < 8; y += 4) {
                const float4 v = __ldg(reinterpret_cast<const float4*>(at + y));
                const float4 w = __ldg(reinterpret_cast<const float4*>(at + a.rot / 2 + y));
                c[y] = v.x; c[y + 1] = v.y; c[y + 2] = v.z; c[y + 3] = v.w;
                s[y] = w.x; s[y + 1] = w.y; s[y + 2] = w.z; s[y + 3] = w.w;
            }
        } else {
#pragma unroll
            for (int y = 0; y < 8; ++y) {
                const int i = 8 * j + y;
                p = pos[0];
#pragma unroll
                for (int x = 1; x < ROPE_AXES; ++x)
                    if (i >= a.end[x - 1]) p = pos[x];
                c[y] = __ldg(a.table + static_cast<size_t>(p) * a.rot + i);
                s[y] = __ldg(a.table + static_cast<size_t>(p) * a.rot + a.rot / 2 + i);
            }
        }
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            if (row0 + n >= a.Hq + a.Hkv) continue;
            float f[8], g[8];
            x0[n].get(f);
            x1[n].get(g);
#pragma unroll
            for (int y = 0; y < 8; ++y) {
                float& u = a.interleaved ? (y < 4 ? f[2 * (y & 3)] : g[2 * (y & 3)]) : f[y];
                float& w = a.interleaved ? (y < 4 ? f[2 * (y & 3) + 1] : g[2 * (y & 3) + 1]) : g[y];
                const float p0 = u * c[y] - w * s[y], p1 = w * c[y] + u * s[y];
                u = p0;
                w = p1;
            }
            x0[n].set(f);
            x1[n].set(g);
        }
    }
    const uint32_t blk = KV::code == PA_INT4 ? div_by(static_cast<uint32_t>(slot), a.bs) : 0;
    const uint32_t off = KV::code == PA_INT4 ? static_cast<uint32_t>(slot) - blk * a.bs.d : 0;
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        const int row = row0 + n;
        if (row >= rows) break;
        if (row < a.Hq) {
            uint8_t* dst = a.q_out + (static_cast<size_t>(t) * a.Hq + row) * a.D * S::bytes;
            x0[n].store(dst + e0 * S::bytes);
            x1[n].store(dst + e1 * S::bytes);
            continue;
        }
        const bool v = row >= a.Hq + a.Hkv;
        const int h = row - a.Hq - (v ? a.Hkv : 0);
        if (!v && a.key_out) {
            uint8_t* dst = a.key_out + (static_cast<size_t>(t) * a.Hkv + h) * a.D * S::bytes;
            x0[n].store(dst + e0 * S::bytes);
            x1[n].store(dst + e1 * S::bytes);
        }
        uint8_t* pool = v ? a.vc : a.kc;
        if constexpr (KV::code == PA_INT4) {
            float x[2][8];
            float mn = INFINITY, mx = -INFINITY;
            x0[n].get(x[0]);
            x1[n].get(x[1]);
#pragma unroll
            for (int y = 0; y < 8; ++y) {
                mn = min_nan(mn, min_nan(x[0][y], x[1][y]));
                mx = max_nan(mx, max_nan(x[0][y], x[1][y]));
            }
            for (int o = lpr / 2; o > 0; o >>= 1) {        // the row's lanes are together here
                mn = min_nan(mn, __shfl_xor_sync(group, mn, o));
                mx = max_nan(mx, __shfl_xor_sync(group, mx, o));
            }
            __half step, low;
            uint32_t w[2];
            int4_quantise(x, mn, mx, step, low, w);
            uint8_t* b = pool + static_cast<size_t>(blk) * a.bs.d * a.Hkv * (a.D / 2 + INT4_PARAM_BYTES);
            uint8_t* codes = b + int4_code_off(h, off, a.bs.d, a.D);
            *reinterpret_cast<uint32_t*>(codes + e0 / 2) = w[0];
            *reinterpret_cast<uint32_t*>(codes + e1 / 2) = w[1];
            if (j == 0)
                *reinterpret_cast<__half2*>(b + int4_param_off(h, off, a.bs.d, a.D, a.Hkv)) = __halves2half2(step, low);
        } else {
            uint8_t* dst = pool + (static_cast<size_t>(slot) * a.Hkv + h) * a.D * KV::bytes;
            if constexpr (KV::bytes == 1) {
                const float sc = v ? a.v_scale : a.k_scale;
                float x[8];
                x0[n].get(x);
                *reinterpret_cast<uint2*>(dst + e0) = fp8_of<KV>(x, sc);
                x1[n].get(x);
                *reinterpret_cast<uint2*>(dst + e1) = fp8_of<KV>(x, sc);
            } else {
                x0[n].store(dst + e0 * KV::bytes);
                x1[n].store(dst + e1 * KV::bytes);
            }
        }
    }
}

template <class S, class KV>
static cudaError_t launch_rope(RopeArgs a, cudaStream_t stream) {
    const int rows = a.Hq + 2 * a.Hkv, lpr = a.D / 16;
    const auto go = [&](auto kern, int nr) {
        a.chunks = make_div((rows + nr - 1) / nr);
        a.units = static_cast<uint32_t>(a.T) * a.chunks.d;
        const uint32_t per = ROPE_THREADS / lpr;
        kern<<<(a.units + per - 1) / per, ROPE_THREADS, 0, stream>>>(a);
    };
    // Four rows per lane on prompts; the few tokens of a decode step spread over more lanes.  The
    // border lies where it does at 36 rows a token of 128 16-bit elements (one row against four: 64
    // tokens 5.7 and 7.6 us, 256 5.7 and 7.3, 455 7.0 and 7.6, 1024 9.8 and 7.7, 16384 68 and 54).  At
    // head_dim 64, where as many rows are half the threads, four are never the faster: 18 rows of
    // bf16 and 2048, 5003 and 16384 tokens 6.2, 8.3 and 17.9 us with one, 6.3, 8.4 and 18.4 with four; 8
    // rows of f32 and 2048 and 5003 tokens 6.2 and 6.7 against 6.3 and 8.4.
    if (static_cast<long long>(a.T) * rows >= 16384) go(rope_kernel<S, KV, 4>, 4);
    else go(rope_kernel<S, KV, 1>, 1);
    return cudaGetLastError();
}

}  // namespace pa

using namespace pa;

extern "C" pa_status pa_rope_and_cache(void* k_cache, void* v_cache, pa_dtype kv_dtype, void* q_out, void* key_out,
                                       const void* q, const void* key, const void* value, pa_dtype src_dtype,
                                       const int64_t* positions, int num_axes, const int* sections, const float* cos_sin,
                                       int max_positions, int rot_dim, int interleaved, const int64_t* slot_mapping,
                                       int num_tokens, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                       int num_blocks, float k_scale, float v_scale, int32_t* err_flag, cudaStream_t stream) {
    clear_error();
    if (num_tokens < 0 || num_q_heads < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks <= 0 ||
        max_positions <= 0)
        return fail(PA_ERR_INVALID_ARG, "rope_and_cache: sizes must be positive (num_tokens and num_q_heads >= 0)");
    if (head_dim != 64 && head_dim != 128) return fail(PA_ERR_UNSUPPORTED, "rope_and_cache: head_dim must be 64 or 128");
    if (rot_dim <= 0 || rot_dim > head_dim || rot_dim % 16 != 0)
        return fail(PA_ERR_INVALID_ARG, "rope_and_cache: rot_dim must be a multiple of 16, at most head_dim");
    if (num_axes < 1 || num_axes > ROPE_AXES)
        return fail(PA_ERR_UNSUPPORTED, "rope_and_cache: 1 to 4 axes of positions");
    RopeArgs a{};
    for (int x = 0; x < ROPE_AXES; ++x) a.end[x] = INT_MAX;
    if (num_axes > 1) {
        if (!sections) return fail(PA_ERR_INVALID_ARG, "rope_and_cache: several axes need sections");
        long long sum = 0;
        for (int x = 0; x < num_axes; ++x) {
            if (sections[x] < 0) return fail(PA_ERR_INVALID_ARG, "rope_and_cache: a section must not be negative");
            sum += sections[x];
            if (x < num_axes - 1) a.end[x] = static_cast<int>(std::min<long long>(sum, INT_MAX));
        }
        if (sum != rot_dim / 2) return fail(PA_ERR_INVALID_ARG, "rope_and_cache: the sections must add up to rot_dim / 2");
    }
    if (num_tokens == 0) return PA_OK;
    if (!k_cache || !v_cache || !key || !value || !positions || !cos_sin || !slot_mapping || (num_q_heads > 0 && (!q || !q_out)))
        return fail(PA_ERR_INVALID_ARG, "rope_and_cache: null pointer");
    if (!valid_cache_dtype(kv_dtype) || !valid_dtype(src_dtype)) return fail(PA_ERR_INVALID_ARG, "rope_and_cache: unknown dtype");
    if (is_fp8(src_dtype)) return fail(PA_ERR_UNSUPPORTED, "rope_and_cache: the source must be f32, f16 or bf16");
    if (!is_fp8(kv_dtype) && !is_int4(kv_dtype) && src_dtype != kv_dtype)
        return fail(PA_ERR_UNSUPPORTED, "rope_and_cache: source dtype must equal cache dtype (fp8 and 4-bit caches excepted)");
    if (is_fp8(kv_dtype) && (!(k_scale > 0.f) || !(v_scale > 0.f) || !isfinite_host(k_scale) || !isfinite_host(v_scale)))
        return fail(PA_ERR_INVALID_ARG, "rope_and_cache: fp8 scales must be finite and > 0");
    for (const void* p : {static_cast<const void*>(k_cache), static_cast<const void*>(v_cache), static_cast<const void*>(q_out),
                          static_cast<const void*>(key_out), q, key, value, static_cast<const void*>(cos_sin)})
        if (!aligned16(p)) return fail(PA_ERR_INVALID_ARG, "rope_and_cache: tensors must be 16-byte aligned");
    if (is_int4(kv_dtype) && block_size % 8 != 0)
        return fail(PA_ERR_UNSUPPORTED, "rope_and_cache: a 4-bit cache needs a block_size of a multiple of 8");
    if (is_int4(kv_dtype) && !block_fits(kv_dtype, num_kv_heads, head_dim, block_size))
        return fail(PA_ERR_UNSUPPORTED, "rope_and_cache: a 4-bit block of 2 GB or more");
    if (static_cast<long long>(num_tokens) * (num_q_heads + 2LL * num_kv_heads) >= (1LL << 31) ||
        static_cast<long long>(num_blocks) * block_size >= (1LL << 31))
        return fail(PA_ERR_UNSUPPORTED, "rope_and_cache: pool or call too large for 32-bit row numbers");
    a.kc = static_cast<uint8_t*>(k_cache); a.vc = static_cast<uint8_t*>(v_cache);
    a.q_out = static_cast<uint8_t*>(q_out); a.key_out = static_cast<uint8_t*>(key_out);
    a.q = static_cast<const uint8_t*>(q); a.key = static_cast<const uint8_t*>(key); a.value = static_cast<const uint8_t*>(value);
    a.positions = positions; a.slots = slot_mapping; a.table = cos_sin; a.err = err_flag;
    a.T = num_tokens; a.Hq = num_q_heads; a.Hkv = num_kv_heads; a.D = head_dim; a.rot = rot_dim; a.interleaved = interleaved;
    a.axes = num_axes; a.max_pos = max_positions;
    a.bs = make_div(block_size);
    a.nslots = static_cast<int64_t>(num_blocks) * block_size;
    a.k_scale = k_scale; a.v_scale = v_scale;
    cudaError_t e;
#define PA_ROPE(ST)                                                                                    \
    switch (kv_dtype) {                                                                                \
        case PA_FP8_E4M3: e = launch_rope<ST, FP8T>(a, stream); break;                                 \
        case PA_FP8_E5M2: e = launch_rope<ST, E5M2T>(a, stream); break;                                \
        case PA_INT4: e = launch_rope<ST, Int4T>(a, stream); break;                                    \
        default: e = launch_rope<ST, ST>(a, stream); break;                                            \
    }
    switch (src_dtype) {
        case PA_F32: PA_ROPE(F32T) break;
        case PA_F16: PA_ROPE(F16T) break;
        default: PA_ROPE(BF16T) break;
    }
#undef PA_ROPE
    return e == cudaSuccess ? PA_OK : fail_cuda("rope_and_cache launch", e);
}
