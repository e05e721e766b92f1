// pa_common.h -- host-side helpers shared by the library's translation units:
// status reporting (a thread-local detail string) and argument checks.
#pragma once

#include <cmath>
#include <cstdint>
#include <cuda_runtime_api.h>

#include "../../include/pa.h"

namespace pa {

void clear_error();
pa_status fail(pa_status s, const char* what);
pa_status fail_cuda(const char* what, cudaError_t e);

inline bool is_fp8(pa_dtype d) { return d == PA_FP8_E4M3 || d == PA_FP8_E5M2; }
inline bool is_int4(pa_dtype d) { return d == PA_INT4; }
// element types of tensors; PA_INT4 is a cache type only
inline bool valid_dtype(pa_dtype d) { return d == PA_F32 || d == PA_F16 || d == PA_BF16 || is_fp8(d); }
inline bool valid_cache_dtype(pa_dtype d) { return valid_dtype(d) || is_int4(d); }
inline int dtype_bytes(pa_dtype d) { return d == PA_F32 ? 4 : (is_fp8(d) ? 1 : 2); }
// bytes of one token's K (or V) row of one head in a pool: 4-bit codes and
// their (step, low) pair, or the elements
inline int row_bytes(pa_dtype d, int head_dim) { return is_int4(d) ? head_dim / 2 + 4 : head_dim * dtype_bytes(d); }
// The limit on a kernel's dynamic shared memory belongs to the kernel, not to a
// launch: every call sets the same value, so that calls of other host threads
// between this one and its launch change nothing.
cudaError_t allow_shared(const void* kernel, int bytes);
// Blocks of 2 GB and more: places inside a block are counted in 32 bits.
inline bool block_fits(pa_dtype d, int num_kv_heads, int head_dim, int block_size) {
    return static_cast<double>(num_kv_heads) * block_size * row_bytes(d, head_dim) < 2147483648.0;
}
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool isfinite_host(float x) { return std::isfinite(x); }

}  // namespace pa
