// pa_decode_int4.cu -- attention over 4-bit pools (pa_decode and pa_attention
// with PA_INT4).
//
// One CTA per (sequence, query token, query head).  Warp w takes tokens w,
// w + 4, ... of the sequence; a lane holds head_dim / 32 dimensions, so a
// score is a 5-step warp sum, and each warp runs its own online softmax
// (maximum and sum in f32, log2 domain).  The warps' results are joined by
// their maxima through shared memory.  K and V are expanded in f32:
// low + step * code.
#include "pa_common.h"
#include "pa_decode_int4.h"
#include "pa_int4.cuh"

namespace pa {

struct Int4Args {
    void* out;
    const void* q;
    const uint8_t* k;
    const uint8_t* v;
    const int32_t* tables;
    const int32_t* lens;
    const int32_t* q_start;
    int32_t* err;
    int MB, Hq, Hkv, G, bs, NB, total_q, QL;
    float qk_scale;               // scale * log2(e)
};

constexpr int I4_WARPS = 4;

template <class QT, int D>
__global__ void __launch_bounds__(I4_WARPS * 32)
int4_row_kernel(const __grid_constant__ Int4Args a) {
    constexpr int E = D / 32;     // dimensions per lane
    using T = typename QT::T;
    __shared__ float sm[I4_WARPS], sl[I4_WARPS], sacc[I4_WARPS][D];
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int i = blockIdx.x, j = blockIdx.y, h = blockIdx.z, g = h / a.G;
    int row = i, n = 1;
    if (a.q_start) {
        const int s0 = a.q_start[i], s1 = a.q_start[i + 1];
        if (s0 < 0 || s1 < s0 || s1 > a.total_q || s1 - s0 > a.QL) {
            if (threadIdx.x == 0) raise_flag(a.err, PA_ERRBIT_BAD_QUERY);
            return;
        }
        row = s0 + j;
        n = s1 - s0;
    }
    if (j >= n) return;
    const int Lraw = a.lens[i], maxL = a.MB * a.bs;
    if ((Lraw < 0 || Lraw > maxL) && threadIdx.x == 0) raise_flag(a.err, PA_ERRBIT_SEQ_TOO_LONG);
    const int L = min(max(Lraw, 0), maxL);
    const int last = L - n + j;                     // last position attended
    const T* qr = static_cast<const T*>(a.q) + (static_cast<size_t>(row) * a.Hq + h) * D + lane * E;
    float q[E], acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) { q[e] = to_float(qr[e]); acc[e] = 0.f; }
    float m = -INFINITY, l = 0.f;
    const size_t bb = static_cast<size_t>(a.bs) * a.Hkv * (D / 2 + INT4_PARAM_BYTES);
    for (int t = w; t <= last; t += I4_WARPS) {
        const int b = a.tables[static_cast<size_t>(i) * a.MB + t / a.bs], off = t % a.bs;
        if (b < 0 || b >= a.NB) {
            if (lane == 0) raise_flag(a.err, PA_ERRBIT_BAD_BLOCK);
            continue;
        }
        const uint32_t co = int4_code_off(g, off, a.bs, D) + lane * E / 2, po = int4_param_off(g, off, a.bs, D, a.Hkv);
        const uint8_t* kb = a.k + b * bb;
        const uint8_t* vb = a.v + b * bb;
        uint32_t kc, vc;
        if constexpr (E == 4) {
            kc = *reinterpret_cast<const uint16_t*>(kb + co);
            vc = *reinterpret_cast<const uint16_t*>(vb + co);
        } else {
            kc = kb[co];
            vc = vb[co];
        }
        const float2 kp = __half22float2(*reinterpret_cast<const __half2*>(kb + po));
        const float2 vp = __half22float2(*reinterpret_cast<const __half2*>(vb + po));
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(q[e], int4_value((kc >> (4 * e)) & 15u, kp.y, kp.x), s);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        s *= a.qk_scale;
        const float mn = fmaxf(m, s), al = exp2f(m - mn), p = exp2f(s - mn);
        m = mn;
        l = l * al + p;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * al + p * int4_value((vc >> (4 * e)) & 15u, vp.y, vp.x);
    }
    if (lane == 0) { sm[w] = m; sl[w] = l; }
#pragma unroll
    for (int e = 0; e < E; ++e) sacc[w][lane * E + e] = acc[e];
    __syncthreads();
    float M = -INFINITY;
#pragma unroll
    for (int x = 0; x < I4_WARPS; ++x) M = fmaxf(M, sm[x]);
    if (M == -INFINITY) M = 0.f;
    float den = 0.f;
#pragma unroll
    for (int x = 0; x < I4_WARPS; ++x) den += exp2f(sm[x] - M) * sl[x];
    T* o = static_cast<T*>(a.out) + (static_cast<size_t>(row) * a.Hq + h) * D;
    for (int d = threadIdx.x; d < D; d += I4_WARPS * 32) {
        float num = 0.f;
#pragma unroll
        for (int x = 0; x < I4_WARPS; ++x) num += exp2f(sm[x] - M) * sacc[x][d];
        o[d] = from_float<T>(den == 0.f ? 0.f : num / den);
    }
}

pa_status decode_int4(void* out, const void* q, pa_dtype q_dtype, const void* k, const void* v, const int32_t* tables,
                      int MB, const int32_t* lens, int B, int Hq, int Hkv, int D, int bs, int NB, float scale,
                      int32_t* err, cudaStream_t stream, const int32_t* q_start, int QL, int total_q) {
    Int4Args a{};
    a.out = out; a.q = q; a.k = static_cast<const uint8_t*>(k); a.v = static_cast<const uint8_t*>(v);
    a.tables = tables; a.lens = lens; a.q_start = q_start; a.err = err;
    a.MB = MB; a.Hq = Hq; a.Hkv = Hkv; a.G = Hq / Hkv; a.bs = bs; a.NB = NB; a.total_q = total_q; a.QL = QL;
    a.qk_scale = scale * 1.4426950408889634f;
    if (Hq > 65535) return fail(PA_ERR_UNSUPPORTED, "decode: more than 65535 query heads");
    const dim3 grid(static_cast<unsigned>(B), static_cast<unsigned>(QL), static_cast<unsigned>(Hq));
    const bool h = q_dtype == PA_F16;
    if (D == 128) {
        if (h) int4_row_kernel<F16T, 128><<<grid, I4_WARPS * 32, 0, stream>>>(a);
        else int4_row_kernel<BF16T, 128><<<grid, I4_WARPS * 32, 0, stream>>>(a);
    } else {
        if (h) int4_row_kernel<F16T, 64><<<grid, I4_WARPS * 32, 0, stream>>>(a);
        else int4_row_kernel<BF16T, 64><<<grid, I4_WARPS * 32, 0, stream>>>(a);
    }
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? PA_OK : fail_cuda("decode: launch", e);
}

}  // namespace pa
