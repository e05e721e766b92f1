// pa_rows.cuh -- pieces of kernels that move rows of cached elements: eight
// elements at a time as floats, and divisions by numbers fixed for a launch.
#pragma once

#include <cstdint>

#include "pa_device.cuh"

namespace pa {

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
inline Div make_div(int d) {
    return Div{static_cast<uint32_t>(d), static_cast<uint32_t>(((1ull << 32) + d - 1) / d)};
}

}  // namespace pa
