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
// evict_select_kernel: a cluster of 1 to 8 CTAs per (sequence, KV head), each
// with a contiguous part of its tokens.  The weights are read once, turned
// into order-preserving 32-bit keys and kept in shared memory; the k-th
// largest is found by a radix select of three digits (11, 11, 10 bits): each
// CTA counts its part, adds its bins that are not empty to the first CTA's
// (atomics in distributed shared memory; reading all bins of all CTAs took
// most of 160 us on 64 rows of 32k to 131k tokens), and that one finds the
// digit; where a whole bin is kept, the digits behind it are left out.  A
// thread then owns a run of consecutive tokens: it turns its keys into two masks
// (above the threshold, tied with it), ranks its ties, counts the free places
// below `heavy` and the kept rows behind it, and writes both lists in position
// order.  Those 64 rows to 4096 tokens each: 52 us, bound by the passes over
// shared memory and the barriers between them (24 MB of weights; three CTAs per
// SM instead of two 7 us slower, copies of the bins by lane 2 to 17).
// evict_move_kernel: a CTA moves a slice of a head's rows of one plane (K, V,
// the 4-bit parameters, the weights).  Slices share no bytes, so the order
// that an in-place move needs holds inside a CTA.  In place a slice is 64 bytes
// wide, so that the few hundred rows of a steady eviction take one or two
// steps; into other blocks 256 bytes, and the rows are cut over CTAs as well
// (64-byte slices of 4096 rows moved 4.5 TB/s, 256-byte ones 5.6).
//
// The launch follows what the table could hold, since the host does not see the
// lengths: 64 sequences of 2064 tokens one block over their budget take 27 us in
// f16, 22 in e4m3 and 20 in 4 bits under a tight table, but 111, 106 and 105
// under one for 131072 tokens (8 CTAs per row, most with little to do) and 123,
// 118 and 117 under one for 262144 (weights read again in every pass); 8 prompts
// of 47k to 131k tokens brought to 4096 102, 83 and 80 under 131072, and 154, 138
// and 130 under 262144.  So tables no wider than the batch needs are the faster
// ones.
#include <algorithm>

#include "pa_common.h"
#include "pa_device.cuh"

namespace pa {

constexpr int EV_SEL_THREADS = 512;
constexpr int EV_MOVE_THREADS = 256;
constexpr int EV_MAX_SLICES = 64;
constexpr int EV_UNROLL = 4;
// Tables hold less than 2^30 tokens; a position past the budget by a grid's
// stride still fits 32 bits.
constexpr int EV_MAX_BUDGET = 1 << 30;

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

// Exclusive prefix sum over the block; `total` is the block's sum.
__device__ __forceinline__ int block_scan_excl(int v, int* warp_sums, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int NW = EV_SEL_THREADS / 32;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();                            // the sums of the scan before are read
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int s = lane < NW ? warp_sums[lane] : 0;    // every warp scans the warps' sums
#pragma unroll
    for (int o = 1; o < NW; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    total = __shfl_sync(0xffffffffu, s, NW - 1);
    const int before = __shfl_sync(0xffffffffu, s, max(warp - 1, 0));
    return x - v + (warp ? before : 0);
}

// Thread-block clusters (PTX ISA: barrier.cluster, mapa, ld.shared::cluster).
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %cluster_nctaid.x;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void peer_add(int* p, int v, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("red.relaxed.cluster.shared::cluster.add.s32 [%0], %1;" :: "r"(a), "r"(v) : "memory");
}
// The int at the same shared address in CTA `rank` of the cluster.
__device__ __forceinline__ int peer_int(const int* p, uint32_t rank) {
    uint32_t a;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

// Sum of the ints at *p in the CTAs of lower rank, and in all; every lane.
__device__ __forceinline__ void peer_prefix(const int* p, int rank, int C, int& lower, int& all) {
    const int lane = threadIdx.x & 31;
    const int v = lane < C ? peer_int(p, lane) : 0;
    lower = __reduce_add_sync(0xffffffffu, lane < rank ? v : 0);
    all = __reduce_add_sync(0xffffffffu, v);
}

constexpr int EV_BINS = 2048;
constexpr int EV_CACHE = 24576;            // keys that a CTA keeps at most (101 KB with padding)
constexpr int EV_MAX_CLUSTER = 8;

// CACHED: a CTA's keys stay in shared memory; else (sequences beyond
// 8 * EV_CACHE tokens) every pass reads the weights again.
template <bool CACHED>
__global__ void __launch_bounds__(EV_SEL_THREADS)
evict_select_kernel(const __grid_constant__ EvictArgs a) {
    __shared__ int hist[EV_BINS];
    __shared__ int sums[EV_SEL_THREADS / 32];
    __shared__ int s_bad, s_digit, s_above, s_count, s_ties, s_nh, s_nf;
    extern __shared__ uint32_t s_keys[];
    constexpr int NT = EV_SEL_THREADS;
    grid_dependents_launch();
    const int C = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
    const int row = blockIdx.x / C, i = row / a.Hkv, g = row - i * a.Hkv, tid = threadIdx.x;
    const int32_t* bt = a.tables + static_cast<size_t>(i) * a.MB;
    int32_t* kept = a.kept + static_cast<size_t>(row) * a.budget;
    int32_t* holes = a.holes + static_cast<size_t>(row) * a.budget;
    int32_t* fills = a.fills + static_cast<size_t>(row) * a.budget;
    const int L = a.lens[i];
    const int n = min(L, a.budget);
    if (tid == 0) s_bad = 0;
    for (int x = tid; x < EV_BINS; x += NT) hist[x] = 0;
    __syncthreads();
    bool bad_len = L < 0 || static_cast<long long>(L) > static_cast<long long>(a.MB) * a.bs;
    if (a.new_tables) bad_len = bad_len || static_cast<long long>(n) > static_cast<long long>(a.newMB) * a.bs;
    // blocks of table t from j0 on, up to j1, over `of` CTAs of the cluster
    auto check = [&](const int32_t* t, int j0, int j1, int of) {
        bool bad = false;
        for (int j = j0 + (of > 1 ? rank * NT : 0) + tid; j < j1; j += of * NT) bad |= t[j] < 0 || t[j] >= a.NB;
        if (bad) s_bad = 1;
    };
    auto blocks = [&](int tokens) { return (tokens + a.bs - 1) >> a.shift; };
    const int32_t* nt = a.new_tables ? a.new_tables + static_cast<size_t>(i) * a.newMB : nullptr;
    auto skip = [&](uint32_t bit) {
        if (tid == 0) {
            raise_flag(a.err, bit);
            a.rows[row] = EvictRow{L, a.new_tables ? 0 : L, 0, 0};
        }
        for (int j = tid; j < a.budget; j += NT) kept[j] = -1;
    };
    // The CTAs of a cluster see the same lengths and tables: where one leaves,
    // all do, and before the first cluster barrier or behind one.
    if (bad_len) {
        if (rank == 0) skip(PA_ERRBIT_SEQ_TOO_LONG);
        return;
    }
    if (L <= a.budget) {
        if (rank != 0) return;
        check(bt, 0, blocks(L), 1);
        if (nt) check(nt, 0, blocks(n), 1);
        __syncthreads();
        if (s_bad) { skip(PA_ERRBIT_BAD_BLOCK); return; }
        for (int j = tid; j < a.budget; j += NT) kept[j] = j < L ? j : -1;
        if (tid == 0) a.rows[row] = EvictRow{L, L, 0, 1};
        return;
    }
    const int heavy = a.budget - a.recent, end = L - a.recent;
    auto sync = [&] { if (C > 1) cluster_sync(); else __syncthreads(); };
    const int k = heavy - a.sink;                   // tokens chosen by weight, of [sink, end)
    const int seg = ((end + C - 1) / C + 3) & ~3;   // this CTA: tokens [lo, hi)
    const int lo = min(rank * seg, end), hi = min(end, lo + seg);
    const float* wg = a.weights + static_cast<size_t>(g) * a.bs;
    const size_t wstride = static_cast<size_t>(a.Hkv) * a.bs;
    auto slot_of = [](int x) { return x + (x >> 5); };                 // a run per thread: no bank conflicts
    auto key_at = [&](int pos) -> uint32_t {
        if constexpr (CACHED) return s_keys[slot_of(pos - lo)];
        return weight_key(wg[static_cast<size_t>(bt[pos >> a.shift]) * wstride + (pos & (a.bs - 1))]);
    };
    const int first = max(lo, a.sink);              // candidates: [first, hi)
    uint32_t thr = 0;
    int need = k;                                   // ties with thr that are kept
    // blocks that the weights below do not pass
    check(bt, k > 0 ? end >> a.shift : 0, blocks(L), C);
    if (nt) check(nt, 0, blocks(n), C);
    if (k > 0) {
        // weights by 16 bytes, four in flight: keys, and the first digit's counts
        constexpr int U = 4;
        for (int p0 = lo + 4 * tid; p0 < hi; p0 += 4 * NT * U) {
            int blk[U];
            float4 w[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int pos = p0 + u * 4 * NT;
                blk[u] = pos < hi ? __ldg(bt + (pos >> a.shift)) : 0;
                if (blk[u] < 0 || blk[u] >= a.NB) { blk[u] = 0; s_bad = 1; }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int pos = p0 + u * 4 * NT;
                if (pos < hi) w[u] = *reinterpret_cast<const float4*>(wg + static_cast<size_t>(blk[u]) * wstride + (pos & (a.bs - 1)));
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int pos = p0 + u * 4 * NT;
                const float v[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (pos + e < hi) {
                        const uint32_t key = weight_key(v[e]);
                        if constexpr (CACHED) s_keys[slot_of(pos + e - lo)] = key;
                        if (pos + e >= first) atomicAdd(&hist[key >> 21], 1);
                    }
            }
        }
    }
    sync();                                         // the first CTA's bins are zeroed, every part's blocks checked
    int total, lower, bad = s_bad;
    if (C > 1) peer_prefix(&s_bad, rank, C, lower, bad);
    if (bad) {
        sync();                                     // every peer has read
        if (rank == 0) skip(PA_ERRBIT_BAD_BLOCK);
        return;
    }
    if (k > 0) {
#pragma unroll 1
        for (int d = 0; d < 3; ++d) {
            const int shift = d == 0 ? 21 : d == 1 ? 10 : 0;
            if (d > 0) {
                const int up = d == 1 ? 21 : 10;    // bits decided so far
#pragma unroll 4
                for (int pos = first + tid; pos < hi; pos += NT) {
                    const uint32_t key = key_at(pos);
                    if ((key >> up) == (thr >> up)) atomicAdd(&hist[(key >> shift) & (d == 1 ? 2047u : 1023u)], 1);
                }
            }
            if (C > 1) {
                __syncthreads();
                if (rank > 0)
                    for (int x = tid; x < EV_BINS; x += NT)
                        if (const int v = hist[x]) {
                            peer_add(&hist[x], v, 0);
                            hist[x] = 0;
                        }
            }
            sync();
            if (rank == 0) {
                // digits from the largest down, EV_BINS / NT per thread
                constexpr int PB = EV_BINS / NT;
                int cnt[PB], mine = 0;
#pragma unroll
                for (int e = 0; e < PB; ++e) {
                    cnt[e] = hist[EV_BINS - 1 - (tid * PB + e)];
                    hist[EV_BINS - 1 - (tid * PB + e)] = 0;         // for the next digit
                    mine += cnt[e];
                }
                int before = block_scan_excl(mine, sums, total);
                if (before < need && need <= before + mine) {
#pragma unroll
                    for (int e = 0; e < PB; ++e) {
                        if (before < need && need <= before + cnt[e]) {
                            s_digit = EV_BINS - 1 - (tid * PB + e);
                            s_above = before;
                            s_count = cnt[e];
                        }
                        before += cnt[e];
                    }
                }
            }
            sync();
            thr |= static_cast<uint32_t>(C > 1 ? peer_int(&s_digit, 0) : s_digit) << shift;
            need -= C > 1 ? peer_int(&s_above, 0) : s_above;
            // the whole bin is kept: the other digits decide nothing
            if (need == (C > 1 ? peer_int(&s_count, 0) : s_count) && d < 2 && thr > 0) {
                --thr;
                need = 0;
                break;
            }
        }
    }
    for (int j = rank * NT + tid; j < a.budget; j += C * NT) kept[j] = j < heavy ? j : end + (j - heavy);
    const int run = (hi - lo + NT - 1) / NT, r0 = min(hi, lo + tid * run), r1 = min(hi, r0 + run);
    int mine = 0, all;
    // One pass over a thread's run: which keys pass the threshold and which
    // tie with it, a bit each (a run has at most EV_CACHE / NT of them); without
    // the keys at hand, the ties are counted here and the rest is walked below.
    static_assert(EV_CACHE / NT <= 64, "a run's bits");
    uint64_t above = 0, tie = 0;
    auto bits = [](int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1; };
    const uint64_t in_run = bits(r1 - r0);
    if constexpr (CACHED) {
        if (k > 0) {
            uint32_t gt[2] = {0, 0}, eq[2] = {0, 0};
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const int from = r0 + 32 * w, n = min(32, r1 - from);
                uint32_t bit = 1;
#pragma unroll 4
                for (int x = 0; x < n; ++x, bit += bit) {
                    const uint32_t key = key_at(from + x);
                    if (key > thr) gt[w] |= bit;
                    if (key == thr) eq[w] |= bit;
                }
            }
            above = static_cast<uint64_t>(gt[1]) << 32 | gt[0];
            tie = static_cast<uint64_t>(eq[1]) << 32 | eq[0];
        }
        const uint64_t sinks = bits(a.sink - r0) & in_run;
        above |= sinks;
        tie &= ~sinks;
        mine = __popcll(tie);
    } else if (k > 0) {
#pragma unroll 4
        for (int pos = max(r0, a.sink); pos < r1; ++pos) mine += key_at(pos) == thr ? 1 : 0;
    }
    int ties = block_scan_excl(mine, sums, total);
    if (C > 1) {
        if (tid == 0) s_ties = total;
        cluster_sync();
        peer_prefix(&s_ties, rank, C, lower, all);
        ties += lower;
    }
    // one walk over the run: f(position, kept)
    auto walk = [&](auto f) {
        int t = ties;
#pragma unroll 4
        for (int pos = r0; pos < r1; ++pos) {
            bool keep = pos < a.sink;
            if (!keep && k > 0) {
                const uint32_t key = key_at(pos);
                keep = key > thr;
                if (key == thr) keep = t++ < need;
            }
            f(pos, keep);
        }
    };
    int h = 0, f = 0;
    uint64_t hole = 0, fill = 0;
    if constexpr (CACHED) {
        uint64_t kept_ties = tie;
        for (int drop = mine - max(need - ties, 0); drop > 0; --drop) kept_ties &= ~(1ull << (63 - __clzll(kept_ties)));
        const uint64_t keep = above | kept_ties, below = bits(heavy - r0);
        hole = in_run & below & ~keep;
        fill = keep & ~below;
        h = __popcll(hole);
        f = __popcll(fill);
    } else {
        walk([&](int pos, bool keep) {
            h += (pos < heavy && !keep) ? 1 : 0;
            f += (pos >= heavy && keep) ? 1 : 0;
        });
    }
    int h0, f0, nf;
    if constexpr (CACHED) {                        // counts of at most EV_CACHE: both in one scan
        const int at = block_scan_excl(h | (f << 16), sums, total);
        h0 = at & 0xffff; f0 = at >> 16;
        h = total & 0xffff; nf = total >> 16;
    } else {
        h0 = block_scan_excl(h, sums, h);
        f0 = block_scan_excl(f, sums, nf);
    }
    if (C > 1) {
        if (tid == 0) { s_nh = h; s_nf = nf; }
        cluster_sync();
        peer_prefix(&s_nh, rank, C, lower, all);
        h0 += lower;
        peer_prefix(&s_nf, rank, C, lower, all);
        f0 += lower;
        nf = all;
    }
    if constexpr (CACHED) {
        for (; hole; hole &= hole - 1) holes[h0++] = r0 + __ffsll(hole) - 1;
        for (; fill; fill &= fill - 1) fills[f0++] = r0 + __ffsll(fill) - 1;
    } else {
        walk([&](int pos, bool keep) {
            if (pos < heavy && !keep) holes[h0++] = pos;
            if (pos >= heavy && keep) fills[f0++] = pos;
        });
    }
    __threadfence();
    sync();                                        // every list entry written, every peer's counts read
    for (int r = rank * NT + tid; r < nf; r += C * NT) kept[__ldcg(holes + r)] = __ldcg(fills + r);
    if (rank == 0 && tid == 0) a.rows[row] = EvictRow{L, a.budget, nf, 1};
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
    // First the kept rows from behind `heavy`, into the free places below it,
    // then the recent rows, in order.  A new place of a recent row may be the
    // old one of a row that comes no later in this list, and one below `heavy`
    // of none: a step's rows are all read before any of them is written.
    if (r.len <= a.budget) return;
    const int32_t* holes = a.holes + static_cast<size_t>(row) * a.budget;
    const int32_t* fills = a.fills + static_cast<size_t>(row) * a.budget;
    const int n = r.moves + a.recent, from = r.len - a.recent - r.moves, to = a.budget - a.recent - r.moves;
    for (int b0 = 0; b0 < n; b0 += R * U) {
        T* dst[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = b0 + rr + u * R;
            const bool fill = j < r.moves;
            const int src = !on || j >= n ? -1 : fill ? fills[j] : from + j;
            if (src >= 0) {
                v[u] = *at(bt, src);
                dst[u] = at(bt, fill ? holes[j] : to + j);
            } else {
                dst[u] = nullptr;
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (dst[u]) *dst[u] = v[u];
    }
}

__global__ void __launch_bounds__(EV_MOVE_THREADS)
evict_move_kernel(const __grid_constant__ EvictArgs a) {
    grid_dependency_wait();
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
    if (num_seqs < 0 || num_kv_heads <= 0 || max_seq_len < 0 || budget <= 0 || budget > EV_MAX_BUDGET) return 0;
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
    if (budget > EV_MAX_BUDGET) return fail(PA_ERR_UNSUPPORTED, "evict: budget above 2^30");
    if (block_size != 8 && block_size != 16 && block_size != 32 && block_size != 64 && block_size != 128)
        return fail(PA_ERR_UNSUPPORTED, "evict: block_size must be 8, 16, 32, 64 or 128");
    if (is_int4(kv_dtype) && head_dim != 64 && head_dim != 128)
        return fail(PA_ERR_UNSUPPORTED, "evict: a 4-bit cache needs head_dim 64 or 128");
    if (head_dim > 1024 || !block_fits(kv_dtype, num_kv_heads, head_dim, block_size) ||
        !block_fits(PA_F32, num_kv_heads, 1, block_size))
        return fail(PA_ERR_UNSUPPORTED, "evict: a row above 1024 elements, or a block of 2 GB or more");
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
        const int w = new_block_tables ? 256 : 64;
        for (int c = 0; c < width; c += w) a.slice[ns++] = EvictSlice{np, c, std::min(w, width - c), unit};
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
    a.per_part = new_block_tables ? 256 : budget;

    // Clusters: as many CTAs as keep a part within EV_CACHE tokens, and more
    // while the rows would leave SMs idle and parts stay above 2048 tokens.
    const int max_len = max_blocks_per_seq * block_size;
    int C = 1;
    while (C < EV_MAX_CLUSTER && (max_len > C * EV_CACHE || (rows * C < 256 && max_len > C * 2048))) C *= 2;
    const bool cached = max_len <= C * EV_CACHE;
    const int part = std::min(EV_CACHE, (max_len + C - 1) / C + 4);
    const size_t smem = cached ? sizeof(uint32_t) * static_cast<size_t>(part + part / 32 + 1) : 0;
    const void* sel = cached ? reinterpret_cast<const void*>(&evict_select_kernel<true>)
                             : reinterpret_cast<const void*>(&evict_select_kernel<false>);
    cudaError_t e = cudaSuccess;
    if (cached) {
        e = allow_shared(sel, static_cast<int>(sizeof(uint32_t) * (EV_CACHE + EV_CACHE / 32 + 1)));
        if (e != cudaSuccess) return fail_cuda("evict: set shared memory size", e);
    }
    const dim3 grid(static_cast<unsigned>(rows), static_cast<unsigned>(ns),
                    static_cast<unsigned>((budget + a.per_part - 1) / a.per_part));
    if (grid.z > 65535u || rows * C > 0x7fffffffu) return fail(PA_ERR_UNSUPPORTED, "evict: budget or batch too large");
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(C);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(rows * C));
    cfg.blockDim = dim3(EV_SEL_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* args[] = {&a};
    e = cudaLaunchKernelExC(&cfg, sel, args);
    if (e != cudaSuccess) return fail_cuda("evict: selection launch", e);
    // becomes resident while the selection runs, and waits for it
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(EV_MOVE_THREADS);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(&evict_move_kernel), args);
    return e == cudaSuccess ? PA_OK : fail_cuda("evict: move launch", e);
}
