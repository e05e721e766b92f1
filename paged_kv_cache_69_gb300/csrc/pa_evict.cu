// pa_evict.cu -- eviction from a paged cache by accumulated attention weight.
//
// For a sequence of L > budget tokens and one KV head, the kept tokens are
// the first num_sink, the last num_recent and, of those between, the
// budget - num_sink - num_recent of largest weight (ties: the lower
// position).  The kept rows move to positions 0 .. budget - 1:
//   heavy = budget - num_recent;
//   a kept row below `heavy` stays; the i-th position below it that is not
//   kept takes the i-th kept row from [heavy, L - num_recent);
//   the recent rows move, in order, to [heavy, budget).
// Attention does not depend on the order of the rows, so only the rows that
// change places are moved, and the recent ones stay last for the next call.
//
// evict_select_kernel: one CTA per (sequence, KV head).  The k-th largest
// weight is found by a radix select over order-preserving 32-bit keys (four
// 8-bit digits, a histogram each); one more pass in position order ranks the
// ties, lists the free places below `heavy` and the kept rows behind it.
// evict_move_kernel: a CTA moves a slice of 64 bytes (or less) of a head's
// rows of one plane (K, V, the 4-bit parameters, the weights).  Slices share
// no bytes, so the order that an in-place move needs holds inside a CTA.
#include <algorithm>

#include "pa_common.h"
#include "pa_device.cuh"

namespace pa {

constexpr int EV_SEL_THREADS = 512;
constexpr int EV_MOVE_THREADS = 256;
constexpr int EV_MAX_SLICES = 64;
constexpr int EV_UNROLL = 4;

// A row's place: base + block * block_stride + offset * tok_stride + head * head_stride.
struct EvictPlane {
    uint8_t* base;
    size_t block_stride;
    uint32_t tok_stride, head_stride;
};
struct EvictSlice {
    int plane, col, width, unit;      // bytes [col, col + width) of a row, moved in units of 16 or 4 bytes
};
struct EvictRow {
    int len, new_len, moves, ok;
};
struct EvictArgs {
    EvictPlane plane[5];
    EvictSlice slice[EV_MAX_SLICES];
    const float* weights;
    const int32_t* tables;
    const int32_t* new_tables;        // null: in place
    const int32_t* lens;
    int32_t* new_lens;
    int32_t* kept;                    // [rows][budget]
    int32_t* holes;                   // [rows][budget] places below heavy that take a row
    int32_t* fills;                   // [rows][budget] the rows they take
    EvictRow* rows;
    int32_t* err;
    int MB, newMB, B, Hkv, bs, shift, NB, budget, sink, recent, per_part;
};

// Larger weights have larger keys; -0 equals 0; NaN is below everything.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0u;
    const uint32_t b = w == 0.f ? 0u : __float_as_uint(w);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ int block_scan_excl(int v, int* warp_sums, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int s = lane < nw ? warp_sums[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        if (lane < nw) warp_sums[lane] = s;
    }
    __syncthreads();
    total = warp_sums[nw - 1];
    const int r = x - v + (warp ? warp_sums[warp - 1] : 0);
    __syncthreads();
    return r;
}

__global__ void __launch_bounds__(EV_SEL_THREADS)
evict_select_kernel(const __grid_constant__ EvictArgs a) {
    __shared__ int hist[256];
    __shared__ int sums[32];
    __shared__ int s_bad, s_digit, s_above;
    const int row = blockIdx.x, i = row / a.Hkv, g = row - i * a.Hkv, tid = threadIdx.x;
    const int32_t* bt = a.tables + static_cast<size_t>(i) * a.MB;
    int32_t* kept = a.kept + static_cast<size_t>(row) * a.budget;
    int32_t* holes = a.holes + static_cast<size_t>(row) * a.budget;
    int32_t* fills = a.fills + static_cast<size_t>(row) * a.budget;
    const int L = a.lens[i];
    const int n = min(L, a.budget);
    if (tid == 0) s_bad = 0;
    __syncthreads();
    bool bad_len = L < 0 || static_cast<long long>(L) > static_cast<long long>(a.MB) * a.bs;
    if (a.new_tables) bad_len = bad_len || static_cast<long long>(n) > static_cast<long long>(a.newMB) * a.bs;
    if (!bad_len) {
        bool bad = false;
        for (int j = tid; j < (L + a.bs - 1) >> a.shift; j += blockDim.x) bad |= bt[j] < 0 || bt[j] >= a.NB;
        if (a.new_tables) {
            const int32_t* nt = a.new_tables + static_cast<size_t>(i) * a.newMB;
            for (int j = tid; j < (n + a.bs - 1) >> a.shift; j += blockDim.x) bad |= nt[j] < 0 || nt[j] >= a.NB;
        }
        if (bad) s_bad = 1;
    }
    __syncthreads();
    if (bad_len || s_bad) {
        if (tid == 0) {
            raise_flag(a.err, bad_len ? PA_ERRBIT_SEQ_TOO_LONG : PA_ERRBIT_BAD_BLOCK);
            a.rows[row] = EvictRow{L, a.new_tables ? 0 : L, 0, 0};
        }
        for (int j = tid; j < a.budget; j += blockDim.x) kept[j] = -1;
        return;
    }
    if (L <= a.budget) {
        for (int j = tid; j < a.budget; j += blockDim.x) kept[j] = j < L ? j : -1;
        if (tid == 0) a.rows[row] = EvictRow{L, L, 0, 1};
        return;
    }
    const int heavy = a.budget - a.recent, end = L - a.recent;
    const int k = heavy - a.sink;
    auto key_at = [&](int pos) -> uint32_t {
        const size_t b = static_cast<size_t>(bt[pos >> a.shift]);
        return weight_key(a.weights[(b * a.Hkv + g) * a.bs + (pos & (a.bs - 1))]);
    };
    // the k-th largest key, digit by digit from the top
    uint32_t thr = 0;
    int need = k;                                   // ties with thr that are kept
    for (int d = 24; d >= 0 && k > 0; d -= 8) {
        for (int b = tid; b < 256; b += blockDim.x) hist[b] = 0;
        __syncthreads();
        for (int pos = a.sink + tid; pos < end; pos += blockDim.x) {
            const uint32_t key = key_at(pos);
            if (d == 24 || (key >> (d + 8)) == (thr >> (d + 8))) atomicAdd(&hist[(key >> d) & 255u], 1);
        }
        __syncthreads();
        // digits from the largest down: thread t < 256 holds digit 255 - t
        int total;
        const int c = tid < 256 ? hist[255 - tid] : 0;
        const int before = block_scan_excl(c, sums, total);
        if (tid < 256 && before < need && need <= before + c) { s_digit = 255 - tid; s_above = before; }
        __syncthreads();
        thr |= static_cast<uint32_t>(s_digit) << d;
        need -= s_above;
        __syncthreads();
    }
    for (int j = tid; j < a.budget; j += blockDim.x) kept[j] = j < heavy ? j : end + (j - heavy);
    int ties = 0, nh = 0, nf = 0;
    for (int p0 = 0; p0 < end; p0 += blockDim.x) {
        const int pos = p0 + tid;
        uint32_t key = 0;
        const bool cand = pos >= a.sink && pos < end && k > 0;
        if (cand) key = key_at(pos);
        int total;
        const bool tie = cand && key == thr;
        const int rank = ties + block_scan_excl(tie ? 1 : 0, sums, total);
        ties += total;
        const bool keep = pos < a.sink || (cand && (key > thr || (tie && rank < need)));
        const bool hole = pos < heavy && !keep, fill = pos >= heavy && pos < end && keep;
        const int at = block_scan_excl((hole ? 1 : 0) | (fill ? 0x10000 : 0), sums, total);
        if (hole) holes[nh + (at & 0xffff)] = pos;
        if (fill) fills[nf + (at >> 16)] = pos;
        nh += total & 0xffff;
        nf += total >> 16;
    }
    __syncthreads();                               // the lists are this CTA's own writes
    for (int r = tid; r < nf; r += blockDim.x) kept[holes[r]] = fills[r];
    if (tid == 0) a.rows[row] = EvictRow{L, a.budget, nf, 1};
}

template <typename T>
__device__ __forceinline__ void evict_move(const EvictArgs& a, const EvictPlane& pl, const EvictSlice& sl, int row,
                                           const EvictRow& r) {
    constexpr int U = EV_UNROLL;
    const int i = row / a.Hkv, g = row - i * a.Hkv;
    const int lpr = sl.width / static_cast<int>(sizeof(T)), R = EV_MOVE_THREADS / lpr;
    const int rr = threadIdx.x / lpr, lane = threadIdx.x - rr * lpr;
    const bool on = rr < R;
    const int32_t* bt = a.tables + static_cast<size_t>(i) * a.MB;
    const int32_t* nt = a.new_tables ? a.new_tables + static_cast<size_t>(i) * a.newMB : bt;
    uint8_t* base = pl.base + static_cast<size_t>(g) * pl.head_stride + sl.col + lane * sizeof(T);
    auto at = [&](const int32_t* t, int pos) -> T* {
        return reinterpret_cast<T*>(base + static_cast<size_t>(t[pos >> a.shift]) * pl.block_stride +
                                    static_cast<size_t>(pos & (a.bs - 1)) * pl.tok_stride);
    };
    T v[U];
    if (a.new_tables) {
        const int32_t* map = a.kept + static_cast<size_t>(row) * a.budget;
        const int lo = blockIdx.z * a.per_part, hi = min(r.new_len, lo + a.per_part);
        for (int j0 = lo + rr; j0 < hi && on; j0 += R * U) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (j0 + u * R < hi) v[u] = *at(bt, map[j0 + u * R]);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (j0 + u * R < hi) *at(nt, j0 + u * R) = v[u];
        }
        return;
    }
    // kept rows from behind `heavy` into the free places below it
    const int32_t* holes = a.holes + static_cast<size_t>(row) * a.budget;
    const int32_t* fills = a.fills + static_cast<size_t>(row) * a.budget;
    for (int j0 = rr; j0 < r.moves && on; j0 += R * U) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (j0 + u * R < r.moves) v[u] = *at(bt, fills[j0 + u * R]);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (j0 + u * R < r.moves) *at(bt, holes[j0 + u * R]) = v[u];
    }
    if (r.len <= a.budget) return;
    // The recent rows, in order: a row's new place may be another recent
    // row's old one, always an earlier row of the list, so a step's rows are
    // all read before any of them is written.
    const int from = r.len - a.recent, to = a.budget - a.recent;
    for (int b0 = 0; b0 < a.recent; b0 += R * U) {
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = b0 + rr + u * R;
            if (on && j < a.recent) v[u] = *at(bt, from + j);
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = b0 + rr + u * R;
            if (on && j < a.recent) *at(bt, to + j) = v[u];
        }
    }
}

__global__ void __launch_bounds__(EV_MOVE_THREADS)
evict_move_kernel(const __grid_constant__ EvictArgs a) {
    const int row = blockIdx.x;
    const EvictRow r = a.rows[row];
    if (threadIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && row % a.Hkv == 0) a.new_lens[row / a.Hkv] = r.new_len;
    if (!r.ok) return;
    const EvictSlice sl = a.slice[blockIdx.y];
    if (sl.unit == 16) evict_move<uint4>(a, a.plane[sl.plane], sl, row, r);
    else evict_move<uint32_t>(a, a.plane[sl.plane], sl, row, r);
}

static size_t ev_align(size_t x) { return (x + 255) & ~size_t(255); }

static size_t evict_ws(int B, int Hkv, int budget) {
    const size_t rows = static_cast<size_t>(B) * Hkv;
    return ev_align(rows * sizeof(EvictRow)) + 3 * ev_align(rows * budget * sizeof(int32_t));
}

}  // namespace pa

using namespace pa;

extern "C" size_t pa_evict_workspace_size(int num_seqs, int num_kv_heads, int max_seq_len, int budget) {
    if (num_seqs < 0 || num_kv_heads <= 0 || max_seq_len < 0 || budget <= 0) return 0;
    return std::max<size_t>(256, evict_ws(num_seqs, num_kv_heads, budget));
}

extern "C" pa_status pa_evict(void* k_cache, void* v_cache, pa_dtype kv_dtype, float* weights,
                              const int32_t* block_tables, int max_blocks_per_seq, const int32_t* seq_lens,
                              const int32_t* new_block_tables, int new_max_blocks_per_seq, int32_t* new_seq_lens,
                              int32_t* kept, int num_seqs, int num_kv_heads, int head_dim, int block_size,
                              int num_blocks, int budget, int num_sink, int num_recent, void* workspace,
                              size_t workspace_bytes, int32_t* err_flag, cudaStream_t stream) {
    clear_error();
    if (num_seqs < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks <= 0 ||
        max_blocks_per_seq <= 0 || (new_block_tables && new_max_blocks_per_seq <= 0))
        return fail(PA_ERR_INVALID_ARG, "evict: sizes must be positive (num_seqs >= 0)");
    if (budget <= 0 || num_sink < 0 || num_recent < 0 || static_cast<long long>(num_sink) + num_recent > budget)
        return fail(PA_ERR_INVALID_ARG, "evict: budget must be positive and hold num_sink + num_recent tokens");
    if (num_seqs == 0) return PA_OK;
    if (!k_cache || !v_cache || !weights || !block_tables || !seq_lens || !new_seq_lens)
        return fail(PA_ERR_INVALID_ARG, "evict: null pointer");
    if (!valid_cache_dtype(kv_dtype)) return fail(PA_ERR_INVALID_ARG, "evict: unknown dtype");
    if (block_size != 8 && block_size != 16 && block_size != 32 && block_size != 64 && block_size != 128)
        return fail(PA_ERR_UNSUPPORTED, "evict: block_size must be 8, 16, 32, 64 or 128");
    if (is_int4(kv_dtype) && head_dim != 64 && head_dim != 128)
        return fail(PA_ERR_UNSUPPORTED, "evict: a 4-bit cache needs head_dim 64 or 128");
    const int rb = is_int4(kv_dtype) ? head_dim / 2 : head_dim * dtype_bytes(kv_dtype);
    if (rb % 16 != 0 || rb > 1024) return fail(PA_ERR_UNSUPPORTED, "evict: a head's row must be a multiple of 16 bytes, at most 1024");
    if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(weights))
        return fail(PA_ERR_INVALID_ARG, "evict: caches and weights must be 16-byte aligned");
    if (static_cast<long long>(max_blocks_per_seq) * block_size >= (1LL << 30) ||
        static_cast<long long>(num_blocks) * block_size >= (1LL << 31) ||
        static_cast<long long>(num_seqs) * num_kv_heads >= (1LL << 31))
        return fail(PA_ERR_UNSUPPORTED, "evict: pool, table or batch too large");
    if (!workspace) return fail(PA_ERR_WORKSPACE, "evict: workspace pointer is null");
    if (workspace_bytes < evict_ws(num_seqs, num_kv_heads, budget))
        return fail(PA_ERR_WORKSPACE, "evict: workspace smaller than pa_evict_workspace_size()");
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return fail(PA_ERR_WORKSPACE, "evict: workspace must be 256-byte aligned");

    EvictArgs a{};
    const uint32_t Hkv = static_cast<uint32_t>(num_kv_heads), bs = static_cast<uint32_t>(block_size);
    int ns = 0, np = 0;
    auto add_plane = [&](uint8_t* base, size_t bstride, uint32_t tstride, uint32_t hstride, int width, int unit) {
        a.plane[np] = EvictPlane{base, bstride, tstride, hstride};
        for (int c = 0; c < width; c += 64) a.slice[ns++] = EvictSlice{np, c, std::min(64, width - c), unit};
        ++np;
    };
    for (int kv = 0; kv < 2; ++kv) {
        uint8_t* base = static_cast<uint8_t*>(kv ? v_cache : k_cache);
        if (is_int4(kv_dtype)) {
            const size_t bb = static_cast<size_t>(bs) * Hkv * (rb + 4);
            add_plane(base, bb, static_cast<uint32_t>(rb), bs * rb, rb, 16);
            add_plane(base + static_cast<size_t>(bs) * Hkv * rb, bb, 4, bs * 4, 4, 4);
        } else {
            add_plane(base, static_cast<size_t>(bs) * Hkv * rb, Hkv * rb, static_cast<uint32_t>(rb), rb, 16);
        }
    }
    add_plane(reinterpret_cast<uint8_t*>(weights), static_cast<size_t>(bs) * Hkv * 4, 4, bs * 4, 4, 4);

    a.weights = weights;
    a.tables = block_tables; a.new_tables = new_block_tables; a.lens = seq_lens; a.new_lens = new_seq_lens;
    a.err = err_flag;
    a.MB = max_blocks_per_seq; a.newMB = new_max_blocks_per_seq; a.B = num_seqs; a.Hkv = num_kv_heads;
    a.bs = block_size; a.NB = num_blocks; a.budget = budget; a.sink = num_sink; a.recent = num_recent;
    for (a.shift = 3; (1 << a.shift) < block_size; ++a.shift) {}
    const size_t rows = static_cast<size_t>(num_seqs) * num_kv_heads;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const size_t list = ev_align(rows * budget * sizeof(int32_t));
    a.rows = reinterpret_cast<EvictRow*>(ws); ws += ev_align(rows * sizeof(EvictRow));
    a.holes = reinterpret_cast<int32_t*>(ws); ws += list;
    a.fills = reinterpret_cast<int32_t*>(ws); ws += list;
    a.kept = kept ? kept : reinterpret_cast<int32_t*>(ws);
    a.per_part = new_block_tables ? 1024 : budget;

    evict_select_kernel<<<static_cast<unsigned>(rows), EV_SEL_THREADS, 0, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail_cuda("evict: selection launch", e);
    const dim3 grid(static_cast<unsigned>(rows), static_cast<unsigned>(ns),
                    static_cast<unsigned>((budget + a.per_part - 1) / a.per_part));
    if (grid.z > 65535u) return fail(PA_ERR_UNSUPPORTED, "evict: budget too large");
    evict_move_kernel<<<grid, EV_MOVE_THREADS, 0, stream>>>(a);
    e = cudaGetLastError();
    return e == cudaSuccess ? PA_OK : fail_cuda("evict: move launch", e);
}
