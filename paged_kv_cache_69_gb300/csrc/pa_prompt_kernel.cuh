// pa_prompt_kernel.cuh -- attention of many query rows over long runs of keys
// on the 5th-generation tensor cores: pa_prefill and pa_prefill_cached (causal,
// every query token of a prompt) and the shared part of pa_decode_shared (one
// query token of each sequence of a group, all attending one prefix).
//
// What is computed.  Sequence i has n_i query tokens (rows q_start[i] on of q)
// and L_i keys; token j at position p = L_i - n_i + j attends the keys t <= p
// (causal), or all of them:
//   s_t = scale <q, K_t>,  out = sum_t exp(s_t - m) V_t / sum_t exp(s_t - m).
// In one pass over the keys: with a reference r per row, P_t = 2^(c s_t - r) and
// l = sum P_t, O = sum P_t V_t; when a score passes the reference by more than
// 2^8, r moves to the row's maximum and l and O are multiplied by 2^(r_old - r).
// The quotient O / l does not depend on r.
//
// How.  The query heads of a KV head's group are packed: tile row u is token
// u / G, head u % G, so that K and V are read once for the whole group.  An item
// is 2 x 128 rows of one (sequence, KV head) and its keys, 128 at a time:
//   - one producer warp finds the items and copies Q, K and V by TMA (128-byte
//     swizzle; paged K and V block by block through the table);
//   - one thread issues S_q = Q_q K^T and O_q += P_q V (q = 0, 1) as 128x128x16
//     MMAs; S, P and O live in tensor memory (P over the columns of its S);
//   - two groups of four warps run the softmax, one row per thread: while one of
//     them works on its S, the tensor cores work for the other.
// Order of the MMAs: ... P0 V(j), S0(j+1), P1 V(j), S1(j+1) ...; a commit covers
// everything issued before it, so "S_q(j+1) is there" also says that P_q V(j) is
// in O_q, and the softmax warps may rescale O_q without a barrier of its own.
//
// CTAs are persistent.  Items go out by length, longest first and in turns of
// alternating direction, which balances causal items without a counter in memory;
// with fewer items than CTAs each is cut into `splits` ranges of keys, merged
// by prompt_merge_kernel.
#pragma once

#include <cuda.h>

#include <climits>
#include <cstdint>
#include <type_traits>

#include "pa_device.cuh"

namespace pa {

constexpr int PT_M = 128;              // rows of a tile, keys of a chunk
constexpr int PT_THREADS = 384;        // 2 x 4 softmax warps, the MMA warp, the producer, the scheduler, one idle
constexpr int PT_ITEMS = 4;            // items that the scheduler may be ahead
constexpr int PT_PARTS = 2;            // parts of P that the second product starts on
constexpr int PT_KNOWN = 1024;         // sequences whose items' numbers are kept
// Registers of a softmax thread and of the others (two thirds and one third of the
// block's 168 each at launch): the softmax holds a row of S.
constexpr int PT_REGS = 208, PT_REGS_FEW = 88;
constexpr float PT_SLACK = 8.f;        // log2 that a score may pass the reference by

struct PromptParams {
    void* out;
    const int32_t* q_start;            // [B + 1] query rows (members of each group in shared mode)
    const int32_t* k_start;            // [B + 1] rows of contiguous K and V, or null
    const int32_t* seq_lens;           // [B] keys, paged; shared mode: prefix lengths
    const int32_t* block_tables;       // paged: [rows][MB]
    int32_t* err_flag;
    float* part_acc;                   // [slot][2][128][D] with splits > 1
    float2* part_ml;                   // [slot][2][128] (reference in log2 units, l)
    int B, Hq, Hkv, G, bs, NB, MB;
    int total_q, total_k;
    int tokens;                        // query tokens per tile, 128 / G
    int splits, causal, shared;
    // shared mode: lengths of the sequences, and what the decode kernel behind takes
    const int32_t* lens;               // [total_q]
    int32_t *tail_lens, *tail_blk;
    int rpb;                           // rows per TMA box of K and V
    float c;                           // |scale| log2(e)
    uint32_t negate;                   // instruction descriptor bit of -Q, for scale < 0
};

// An item as the producer hands it on.
struct PromptItem {
    int live;                          // 0: no more items (the rest is unset)
    int row0, ntok;                    // first query row, query tokens of both tiles
    int pos0, L;                       // position of the first token, keys of the sequence
    int t0, e[2];                      // chunks [t0, e[q]) of tile q
    int h, slot;                       // KV head; partial slot
    int idx;                           // sequence (or group)
};

// Non-finite values of V among keys that some row of the tile must not see: the
// first such key of each column, by kind (NaN, +infinity, -infinity).
struct PromptFix {
    int any;
    int first[3][PT_M];
};

struct PromptBars {
    uint64_t q_full[2], q_empty[2], s_full[2], p_full[2][PT_PARTS], o_full[2];
    uint64_t i_full[PT_ITEMS], i_empty[PT_ITEMS];
    uint64_t fin;
    uint32_t tmem;
    int any_bad;                       // a block id outside the pool was met
};

template <int D>
struct PromptLayout {
    static constexpr uint32_t TILE = PT_M * D * 2;               // bytes of 128 rows
    static constexpr uint32_t PLANE = PT_M * 128;                // a plane of 64 columns
    static constexpr int STAGES = D == 128 ? 4 : 8;              // of K or V
    static constexpr uint32_t Q = 0, KV = 2 * TILE, END = KV + STAGES * TILE;
    static constexpr uint32_t FULL = END, EMPTY = FULL + 8 * STAGES, BARS = EMPTY + 8 * STAGES;
    static constexpr uint32_t ITEM = (BARS + sizeof(PromptBars) + 15) & ~15u;
    static constexpr uint32_t FIX = ITEM + PT_ITEMS * ((sizeof(PromptItem) + 15) & ~15u);
    static constexpr uint32_t BAD = (FIX + PT_ITEMS * sizeof(PromptFix) + 15) & ~15u;   // uint4 per stage
    static constexpr uint32_t STAGE = (BAD + 16 * STAGES + 127) & ~127u;     // 2 KB per softmax warp
    static constexpr uint32_t KNOWN = STAGE + 8 * 2048;          // (level, items) of the first sequences
    static constexpr uint32_t BYTES = KNOWN + 8 * PT_KNOWN + 1024;   // + alignment of the base
    static_assert(BYTES <= 227 * 1024, "shared memory of a CTA");
    static constexpr uint32_t TCOLS = 512;                       // S0, S1, O0, O1
    static constexpr uint32_t OCOL = 256;
};

// ---------------------------------------------------------------------------
// sequences and items
// ---------------------------------------------------------------------------
struct PromptSeq {
    int row0, n, L;                    // query rows, keys
    int a, c;                          // level of the first item, items
};

// Shared mode: a group of fewer (sequence, head) rows than this, or with fewer
// shared tokens, is left to the decode kernel, prefix and all.
constexpr int PT_SHARED_ROWS = 8, PT_SHARED_KEYS = 64;

// The tokens of group i's prefix that are attended once: whole blocks.
__device__ __forceinline__ int shared_prefix(const PromptParams& p, int i, int n) {
    const int P = __ldg(p.seq_lens + i);
    if (P < PT_SHARED_KEYS || n * p.G < PT_SHARED_ROWS) return 0;
    return min(P, p.MB * p.bs) / p.bs * p.bs;
}

// Sequence (or group) i; n = 0 where its numbers do not fit.
__device__ __forceinline__ PromptSeq prompt_seq(const PromptParams& p, int i, bool report) {
    PromptSeq s{0, 0, 0, 0, 0};
    const int a = __ldg(p.q_start + i), b = __ldg(p.q_start + i + 1);
    bool ok = a >= 0 && b >= a && b <= p.total_q;
    uint32_t bit = PA_ERRBIT_BAD_QUERY;
    if (p.k_start) {
        const int ka = __ldg(p.k_start + i), kb = __ldg(p.k_start + i + 1);
        ok = ok && ka >= 0 && kb >= ka && kb <= p.total_k;
        s.L = kb - ka;
    } else if (p.shared) {
        s.L = ok ? shared_prefix(p, i, b - a) : 0;
    } else {
        s.L = __ldg(p.seq_lens + i);
        if (ok && (s.L < 0 || s.L > p.MB * p.bs)) { ok = false; bit = PA_ERRBIT_SEQ_TOO_LONG; }
    }
    if (!ok) {
        if (report) raise_flag(p.err_flag, bit);
        return PromptSeq{0, 0, 0, 0, 0};
    }
    s.row0 = a;
    s.n = b - a;
    const int TT = 2 * p.tokens;
    if (p.shared) {
        s.c = s.L > 0 ? (s.n + TT - 1) / TT : 0;
        s.a = s.L / TT;
    } else {
        s.c = (s.n + TT - 1) / TT;
        s.a = max(0, s.L - s.n) / TT;
    }
    return s;
}

// Items of the sequence at level u and above: causal items lie one to a level from a
// on, the items of a group all at a.
__device__ __forceinline__ int items_from(const PromptParams& p, const PromptSeq& s, int u) {
    return p.shared ? (s.a >= u ? s.c : 0) : min(max(s.a + s.c - u, 0), s.c);
}

// The items of the launch in order of length, for one warp.
struct PromptOrder {
    int2* known;                       // (a, c) of the first PT_KNOWN sequences
    int hi;                            // no item that is still to come lies above this level
    int total;                         // items per KV head

    __device__ __forceinline__ PromptSeq seq(const PromptParams& p, int i) const {
        if (i >= PT_KNOWN) return prompt_seq(p, i, false);
        const int2 x = known[i];
        return PromptSeq{0, 0, 0, x.x, x.y};
    }
    __device__ __forceinline__ int count_from(const PromptParams& p, int u) const {
        int x = 0;
        for (int i = threadIdx.x & 31; i < p.B; i += 32) x += items_from(p, seq(p, i), u);
        return __reduce_add_sync(0xffffffffu, x);
    }
    __device__ __forceinline__ void init(const PromptParams& p, int2* smem) {
        const bool report = blockIdx.x == 0;
        known = smem;
        int top = 0, n = 0;
        for (int i = threadIdx.x & 31; i < p.B; i += 32) {
            const PromptSeq s = prompt_seq(p, i, report);
            if (i < PT_KNOWN) known[i] = make_int2(s.a, s.c);
            if (s.c > 0) top = max(top, p.shared ? s.a : s.a + s.c - 1);
            n += s.c;
        }
        __syncwarp();
        total = __reduce_add_sync(0xffffffffu, n);
        hi = __reduce_max_sync(0xffffffffu, top);
    }
    // Item k (below total): its sequence's index and numbers, its number in the sequence.
    __device__ __forceinline__ void find(const PromptParams& p, int k, int& idx, PromptSeq& s, int& t) {
        // the largest level that more than k items lie at or above: down from the last
        // one in growing steps, then between the last two
        int lo = hi, step = 1;
        while (lo > 0 && count_from(p, lo) <= k) {
            hi = lo - 1;
            lo = max(0, lo - step);
            step *= 2;
        }
        while (lo < hi) {
            const int u = (lo + hi + 1) >> 1;
            if (count_from(p, u) > k) lo = u; else hi = u - 1;
        }
        int r = k - count_from(p, hi + 1);
        const int lane = threadIdx.x & 31;
        for (int i0 = 0; i0 < p.B; i0 += 32) {
            PromptSeq x{0, 0, 0, 0, 0};
            if (i0 + lane < p.B) x = seq(p, i0 + lane);
            const int own = items_from(p, x, hi) - items_from(p, x, hi + 1);
            const int all = __reduce_add_sync(0xffffffffu, own);
            if (r >= all) {
                r -= all;
                continue;
            }
            int inc = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            const int src = __ffs(__ballot_sync(0xffffffffu, inc > r)) - 1;
            const int before = __shfl_sync(0xffffffffu, inc - own, src);
            idx = i0 + src;
            s = prompt_seq(p, idx, false);
            t = p.shared ? r - before : hi - s.a;
            return;
        }
        idx = 0;                       // not reached: k < total
        s = PromptSeq{0, 0, 0, 0, 0};
        t = 0;
    }
};

// The place of an item among the partials: sequences take floor(n / 2 tokens) + 1
// places each, counted from their first query row, without a sum over the batch.
__host__ __device__ __forceinline__ int prompt_slot(int row0, int i, int t, int tokens) {
    return row0 / (2 * tokens) + i + t;
}

// ---------------------------------------------------------------------------
// tensor memory and packed arithmetic
// ---------------------------------------------------------------------------
// D += A B with A (16-bit pairs) in tensor memory, issued by one thread.
__device__ __forceinline__ void umma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        :: "r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u) : "memory");
}
// 32 consecutive columns of the warp's 32 lanes.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        :: "r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
           "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
template <int N> __device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(N)); }
template <int N> __device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(N)); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return d;
}

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------
template <class KV, int D>
struct PromptKernel {
    using E = typename KV::T;
    using Lay = PromptLayout<D>;
    static constexpr bool BF16 = KV::code == PA_BF16;
    static constexpr int PLANES = D / 64;
    static constexpr int S = Lay::STAGES;
    // P is kept above 2^-24 for f16 operands: its largest is about 2^7 there, at most
    // 2^15, so that weights down to 2^-31 of a row's largest still count (11 bits down
    // to 2^-21); bf16 has the range of f32 and needs none of it.
    static constexpr float LIFT = BF16 ? 0.f : 7.f;

    static __device__ __forceinline__ bool wait(const PromptParams& p, uint64_t* bar, uint32_t parity) {
        if (mbar_wait_bounded(bar, parity)) return true;
        raise_flag(p.err_flag, PA_ERRBIT_WAIT_TIMEOUT);
        return false;
    }

    // ---------------- scheduler: one warp finds the CTA's items ----------------
    static __device__ void schedule(const PromptParams& p, PromptBars* b, PromptItem* items, PromptFix* fix, int2* known) {
        const int lane = threadIdx.x & 31;
        PromptOrder order;
        order.init(p, known);
        const int total = order.total * p.Hkv * p.splits;
        const int TT = 2 * p.tokens;
        for (int turn = 0;; ++turn) {
            const int slot = turn % PT_ITEMS;
            bool ok = true;
            if (turn >= PT_ITEMS) ok = wait(p, &b->i_empty[slot], (turn / PT_ITEMS - 1) & 1u);
            if (!__all_sync(0xffffffffu, ok)) return;
            // turns of alternating direction: CTA b takes b, 2 grid - 1 - b, 2 grid + b, ...
            // (k is below the next turn's first number: behind the last item there are no more turns)
            const int k = turn * gridDim.x + (turn & 1 ? static_cast<int>(gridDim.x) - 1 - static_cast<int>(blockIdx.x)
                                                       : static_cast<int>(blockIdx.x));
            PromptItem it{};
            if (k < total) {
                const int part = k % p.splits, kh = k / p.splits;
                PromptSeq s;
                int t;
                order.find(p, kh / p.Hkv, it.idx, s, t);
                it.live = 1;
                it.h = kh % p.Hkv;
                it.row0 = s.row0 + t * TT;
                it.ntok = min(TT, s.n - t * TT);
                it.pos0 = s.L - s.n + t * TT;
                it.L = s.L;
                int e[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int nt = min(max(it.ntok - q * p.tokens, 0), p.tokens);
                    const int end = p.causal ? it.pos0 + q * p.tokens + nt : s.L;    // keys of the tile's last row
                    e[q] = nt > 0 && end > 0 ? (end + PT_M - 1) / PT_M : 0;
                }
                const int most = max(e[0], e[1]);
                it.t0 = static_cast<int>(static_cast<long long>(most) * part / p.splits);
                const int t1 = static_cast<int>(static_cast<long long>(most) * (part + 1) / p.splits);
                it.e[0] = max(it.t0, min(e[0], t1));
                it.e[1] = max(it.t0, min(e[1], t1));
                it.slot = (prompt_slot(s.row0, it.idx, t, p.tokens) * p.Hkv + it.h) * p.splits + part;
            }
            if (lane == 0) {
                items[slot] = it;
                fix[slot].any = 0;
            }
#pragma unroll
            for (int x = 0; x < 3; ++x)
                for (int d = lane; d < D; d += 32) fix[slot].first[x][d] = INT_MAX;
            __syncwarp();
            if (lane == 0) mbar_arrive(&b->i_full[slot]);
            if (!it.live) return;
        }
    }

    // ---------------- producer ----------------
    static __device__ void producer(const PromptParams& p, uint8_t* base, uint64_t* full, uint64_t* empty, PromptBars* b,
                                    const PromptItem* items, uint4* bad, const CUtensorMap* tq, const CUtensorMap* tk,
                                    const CUtensorMap* tv) {
        const int lane = threadIdx.x & 31;
        const uint32_t q_bytes = static_cast<uint32_t>(p.tokens * p.G) * 128u * PLANES;
        const int nb = PT_M / p.rpb;                       // boxes of a chunk and plane
        int issued = 0, qload[2] = {0, 0};
        bool ok = true;
        for (int turn = 0; ok; ++turn) {
            const int is = turn % PT_ITEMS;
            ok = __all_sync(0xffffffffu, wait(p, &b->i_full[is], (turn / PT_ITEMS) & 1u));
            if (!ok) break;
            const PromptItem it = items[is];
            __syncwarp();
            if (lane == 0) mbar_arrive(&b->i_empty[is]);
            if (!it.live) break;
            // the query rows of each tile that has keys
            auto queries = [&](int q) {
                if (it.e[q] <= it.t0) return;
                if (qload[q] > 0) ok = ok && wait(p, &b->q_empty[q], (qload[q] - 1) & 1u);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) return;
                ++qload[q];
                if (lane == 0) {
                    mbar_arrive_expect_tx(&b->q_full[q], q_bytes);
#pragma unroll
                    for (int pl = 0; pl < PLANES; ++pl)
                        tma_load_4d(base + Lay::Q + q * Lay::TILE + pl * Lay::PLANE, tq, &b->q_full[q], 0, it.h * p.G,
                                    it.row0 + q * p.tokens, pl);
                }
            };
            const int n = max(it.e[0], it.e[1]) - it.t0;
            if (n == 0) continue;
            const int32_t* table = nullptr;
            int k0 = 0;
            if (p.k_start) k0 = __ldg(p.k_start + it.idx);
            else table = p.block_tables + static_cast<size_t>(p.shared ? __ldg(p.q_start + it.idx) : it.idx) * p.MB;
            const int nblk = (it.L + p.bs - 1) / p.bs;     // paged: blocks that the sequence uses
            // lane x < nb copies box x of each chunk; the next chunk's table entry is read ahead
            auto entry = [&](int t) -> int {               // first pool row of the lane's box in chunk t, or -1
                const int tok = t * PT_M + lane * p.rpb;
                const int j = tok / p.bs;
                if (lane >= nb || j >= nblk) return -1;
                const int id = __ldg(table + j);
                return id < 0 || id >= p.NB ? -2 : id * p.bs + (tok - j * p.bs);
            };
            int next = table ? entry(it.t0) : 0;
            for (int j = 0; j < n && ok; ++j) {
                if (j == 0) queries(0);
                if (j == 0 && ok) queries(1);
                if (!ok) break;
                const int t = it.t0 + j;
                int row = next;
                if (table) {
                    if (j + 1 < n) next = entry(t + 1);
                } else {
                    row = k0 + t * PT_M;
                }
                uint4 mask = make_uint4(0, 0, 0, 0);
                if (table) {
                    const uint32_t miss = __ballot_sync(0xffffffffu, row == -2);
                    if (miss) {                            // keys of blocks outside the pool are left out
                        if (lane == 0) {
                            raise_flag(p.err_flag, PA_ERRBIT_BAD_BLOCK);
                            *reinterpret_cast<volatile int*>(&b->any_bad) = 1;
                        }
                        uint32_t w[4] = {0, 0, 0, 0};
                        for (int x = 0; x < nb; ++x)
                            if ((miss >> x) & 1u)
                                for (int y = x * p.rpb; y < (x + 1) * p.rpb; ++y) w[y >> 5] |= 1u << (y & 31);
                        mask = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                // boxes without rows start behind the pool, where TMA fills in zeros
                const int at = table ? (row >= 0 ? row : p.NB * p.bs) : row;
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const int st = issued % S;
                    if (issued >= S) ok = ok && wait(p, &empty[st], (issued / S - 1) & 1u);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    uint8_t* dst = base + Lay::KV + st * Lay::TILE;
                    if (lane == 0) {
                        if (v) bad[st] = mask;
                        mbar_arrive_expect_tx(&full[st], Lay::TILE);
                    }
                    __syncwarp();
                    if (lane < nb) {
#pragma unroll
                        for (int pl = 0; pl < PLANES; ++pl)
                            tma_load_4d(dst + pl * Lay::PLANE + lane * p.rpb * 128, v ? tv : tk, &full[st], 0, at, it.h, pl);
                    }
                    ++issued;
                }
            }
        }
        // every copy must land before the CTA exits
        for (int st = max(0, issued - S); st < issued; ++st)
            if (!wait(p, &full[st % S], (st / S) & 1u)) break;
#pragma unroll
        for (int q = 0; q < 2; ++q)
            if (qload[q] > 0) wait(p, &b->q_full[q], (qload[q] - 1) & 1u);
    }

    // ---------------- MMA issue (one thread) ----------------
    static __device__ void mma(const PromptParams& p, uint8_t* base, uint64_t* full, uint64_t* empty, PromptBars* b,
                               const PromptItem* items) {
        const uint32_t tm = b->tmem;
        const uint32_t id_s = umma_idesc_f16(BF16, PT_M, PT_M, false, false) | p.negate;
        const uint32_t id_o = umma_idesc_f16(BF16, PT_M, D, false, true);
        const uint32_t qb = smem_u32(base + Lay::Q), kvb = smem_u32(base + Lay::KV);
        int used = 0;                                      // stages gone through
        int qn[2] = {0, 0};
        uint32_t pn[2] = {0, 0};
        bool ok = true;
        auto score = [&](int q, int st, bool last) {       // S_q = Q_q K^T
            const uint32_t kb = kvb + st * Lay::TILE, qa = qb + q * Lay::TILE;
            tc05_fence_after();
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = static_cast<uint32_t>(kk >> 2) * Lay::PLANE + static_cast<uint32_t>(kk & 3) * 32u;
                umma_f16(tm + q * PT_M, umma_desc(qa + off, 16u, 1024u, 2u), umma_desc(kb + off, 16u, 1024u, 2u), id_s, kk > 0);
            }
            umma_commit(&b->s_full[q]);
            if (last) umma_commit(&b->q_empty[q]);
        };
        auto value = [&](int q, int st, bool first) {      // O_q (+)= P_q V, as the parts of P come
            const uint32_t vb = kvb + st * Lay::TILE;
            const uint32_t phase = pn[q]++ & 1u;
#pragma unroll
            for (int part = 0; part < PT_PARTS; ++part) {
                if (!wait(p, &b->p_full[q][part], phase)) return false;
                tc05_fence_after();
#pragma unroll
                for (int x = 0; x < PT_M / 16 / PT_PARTS; ++x) {
                    const int kk = part * (PT_M / 16 / PT_PARTS) + x;
                    umma_f16_ta(tm + Lay::OCOL + q * D, tm + q * PT_M + kk * 8,
                                umma_desc(vb + kk * 2048u, Lay::PLANE, 1024u, 2u), id_o, !first || kk > 0);
                }
            }
            return true;
        };
        for (int turn = 0; ok; ++turn) {
            const int is = turn % PT_ITEMS;
            if (!(ok = wait(p, &b->i_full[is], (turn / PT_ITEMS) & 1u))) break;
            const PromptItem it = items[is];
            mbar_arrive(&b->i_empty[is]);
            if (!it.live) break;
            const int n0 = it.e[0] - it.t0, n1 = it.e[1] - it.t0, n = max(n0, n1);
            if (n == 0) continue;
            // chunk j: K in stage 2 j of the item's, V in the one behind it
            if (!(ok = wait(p, &full[used % S], (used / S) & 1u))) break;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                if ((q ? n1 : n0) == 0) continue;
                if (!(ok = wait(p, &b->q_full[q], qn[q]++ & 1u))) break;
                score(q, used % S, (q ? n1 : n0) == 1);
            }
            if (!ok) break;
            umma_commit(&empty[used % S]);
            ++used;
            for (int j = 0; j < n && ok; ++j) {
                const int vs = used % S, ks = (used + 1) % S;
                if (!(ok = wait(p, &full[vs], (used / S) & 1u))) break;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int nq = q ? n1 : n0;
                    if (j < nq) {
                        if (!(ok = value(q, vs, j == 0))) break;
                        if (j == nq - 1) umma_commit(&b->o_full[q]);
                    }
                    if (q == 1) umma_commit(&empty[vs]);
                    if (q == 0 && j + 1 < n && !(ok = wait(p, &full[ks], ((used + 1) / S) & 1u))) break;
                    if (j + 1 < nq) score(q, ks, j + 1 == nq - 1);
                }
                if (!ok) break;
                if (j + 1 < n) umma_commit(&empty[ks]);
                used += j + 1 < n ? 2 : 1;
            }
        }
        // nothing may still read shared or tensor memory when the CTA frees them
        umma_commit(&b->fin);
        wait(p, &b->fin, 0u);
    }

    // ---------------- softmax: tile q, one row per thread ----------------
    // Keys that some row of the tile must not see, in the chunk's V: rows behind the
    // sequence become zeros; elsewhere values that are not finite, whose product with
    // a weight of 0 would be NaN, are noted by column and first key, become zeros, and
    // come back at the end for the rows that do see them.
    static __device__ __noinline__ void mend_values(uint8_t* v, PromptFix* fix, int r, int lo, int tail, int key0) {
        constexpr int CH = D / 8;                          // 16-byte pieces of a row
        for (int x = r; x < (PT_M - lo) * CH; x += PT_M) {
            const int row = lo + x / CH, ch = x % CH;
            uint4* at = reinterpret_cast<uint4*>(v + (ch >> 3) * Lay::PLANE + swz128(row, ch & 7));
            if (row >= tail) continue;
            const uint4 raw = *at;
            uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
            constexpr uint32_t EXP = BF16 ? 0x7f80u : 0x7c00u;
            bool hit = false;
#pragma unroll
            for (int y = 0; y < 8; ++y) {
                const uint32_t bits = (w[y >> 1] >> (16 * (y & 1))) & 0xffffu;
                if ((bits & EXP) != EXP) continue;
                const int kind = (bits & 0x7fffu) != EXP ? 0 : bits >> 15 ? 2 : 1;
                atomicMin(&fix->first[kind][ch * 8 + y], key0 + row);
                w[y >> 1] &= 0xffff0000u >> (16 * (y & 1));
                hit = true;
            }
            if (hit) {
                *reinterpret_cast<volatile int*>(&fix->any) = 1;
                __threadfence_block();                     // noted before it is gone from V
                *at = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
    // The zeros, and whether there is anything to mend: 0 * x is NaN for an x that is
    // not finite.
    static __device__ __forceinline__ bool unfit_values(uint8_t* v, int r, int lo, int tail) {
        constexpr int CH = D / 8;
        using E2 = std::conditional_t<BF16, __nv_bfloat162, __half2>;
        E2 acc[2];
        uint32_t zero = 0;
        acc[0] = acc[1] = *reinterpret_cast<E2*>(&zero);
        const E2 none = acc[0];
        for (int x = r; x < (PT_M - lo) * CH; x += PT_M) {
            const int row = lo + x / CH, ch = x % CH;
            uint4* at = reinterpret_cast<uint4*>(v + (ch >> 3) * Lay::PLANE + swz128(row, ch & 7));
            if (row >= tail) {
                *at = make_uint4(0, 0, 0, 0);
                continue;
            }
            const uint4 raw = *at;
            const E2* e = reinterpret_cast<const E2*>(&raw);
#pragma unroll
            for (int y = 0; y < 4; ++y) acc[y & 1] = __hfma2(e[y], none, acc[y & 1]);
        }
        acc[0] = __hadd2(acc[0], acc[1]);
        return __hisnan(acc[0].x) || __hisnan(acc[0].y);
    }

    // 64 bytes of each of the warp's 32 rows to 32 places in memory, by way of shared
    // memory so that four lanes write one row's 64 bytes together.  dst(k): where lane's
    // row k * 8 + lane / 4 goes, or null.
    static __device__ __forceinline__ void put_rows(uint8_t* buf, int lane, const uint4 (&x)[4], uint8_t* const (&dst)[4],
                                                    int off) {
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 4; ++c)
            *reinterpret_cast<uint4*>(buf + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) = x[c];
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int row = k * 8 + (lane >> 2);
            const uint4 y = *reinterpret_cast<const uint4*>(buf + row * 64 + (((lane & 3) ^ ((row >> 1) & 3)) << 4));
            if (dst[k]) *reinterpret_cast<uint4*>(dst[k] + off + ((lane & 3) << 4)) = y;
        }
    }

    static __device__ void softmax(const PromptParams& p, int q, uint8_t* base, uint64_t* full, PromptBars* b,
                                   const PromptItem* items, PromptFix* fix, const uint4* bad) {
        const int r = threadIdx.x & (PT_M - 1);            // tile row = tensor-memory lane
        const int lane = threadIdx.x & 31;
        const uint32_t lanes = static_cast<uint32_t>(r & ~31) << 16;
        const uint32_t ts = b->tmem + lanes + q * PT_M, to = b->tmem + lanes + Lay::OCOL + q * D;
        uint8_t* buf = base + Lay::STAGE + (threadIdx.x >> 5) * 2048;
        const int tok = r / p.G;
        // (token, head) of the rows that this lane writes
        int wtok[4], whead[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int row = (r & ~31) + k * 8 + (lane >> 2);
            wtok[k] = row / p.G;
            whead[k] = row - wtok[k] * p.G;
        }
        const float c = p.c;
        uint32_t sn = 0, on = 0;
        int vstage = 1;                                    // stage of the item's first V
        for (int turn = 0;; ++turn) {
            const int is = turn % PT_ITEMS;
            if (!__all_sync(0xffffffffu, wait(p, &b->i_full[is], (turn / PT_ITEMS) & 1u))) return;
            const PromptItem it = items[is];
            if (!it.live) return;
            const int t1 = it.e[q];
            const int first = it.pos0 + q * p.tokens;      // position of the tile's first token
            const int last = p.causal ? first + tok : it.L - 1;                 // the row's last key
            const int seen = p.causal ? min(first, it.L - 1) : it.L - 1;        // the last key that every row sees
            float ref = -INFINITY;
            float2 sum = make_float2(0.f, 0.f);
            for (int t = it.t0; t < t1; ++t) {
                if (!__all_sync(0xffffffffu, wait(p, &b->s_full[q], sn++ & 1u))) return;
                tc05_fence_after();
                float s[PT_M];
#pragma unroll
                for (int x = 0; x < 4; ++x) tmem_ld32(ts + 32 * x, s + 32 * x);
                const int any_bad = p.block_tables ? *reinterpret_cast<volatile int*>(&b->any_bad) : 0;
                tmem_wait_ld();
                const int vs = vstage + 2 * (t - it.t0);
                const bool edge = t * PT_M + PT_M - 1 > seen;
                if (edge) {
                    const int rel = last - t * PT_M;
                    const int least = __reduce_min_sync(0xffffffffu, rel);
#pragma unroll
                    for (int x = 0; x < PT_M; x += 32) {
                        if (x + 31 <= least) continue;
#pragma unroll
                        for (int y = 0; y < 32; ++y) s[x + y] = x + y <= rel ? s[x + y] : -INFINITY;
                    }
                    if (!__all_sync(0xffffffffu, wait(p, &full[vs % S], (vs / S) & 1u))) return;
                }
                const auto highest = [&]() {
                    float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                    for (int x = 4; x < PT_M - 4; x += 8) {
#pragma unroll
                        for (int y = 0; y < 4; ++y) mx[y] = max3(mx[y], s[x + y], s[x + 4 + y]);
                    }
#pragma unroll
                    for (int y = 0; y < 4; ++y) mx[y] = fmaxf(mx[y], s[PT_M - 4 + y]);
                    return fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
                };
                float top = highest();
                if (any_bad) {                             // keys of blocks outside the pool
                    if (!__all_sync(0xffffffffu, wait(p, &full[vs % S], (vs / S) & 1u))) return;
                    const uint4 m4 = bad[vs % S];
                    const uint32_t w[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
                    for (int x = 0; x < PT_M; ++x)
                        if ((w[x >> 5] >> (x & 31)) & 1u) s[x] = -INFINITY;
                    top = highest();
                }
                // the reference moves at the row's first key and when it is passed by 2^8
                const bool move = top * c > ref + (PT_SLACK + LIFT) && top > -INFINITY;
                if (__any_sync(0xffffffffu, move)) {
                    const float to_ref = move ? top * c - LIFT : ref;
                    const float f = move ? exp2f(ref - to_ref) : 1.f;
                    ref = to_ref;
                    sum.x *= f;
                    sum.y *= f;
                    if (t > it.t0) {
#pragma unroll
                        for (int x = 0; x < D; x += 16) {
                            float o[16];
                            tmem_ld16(to + x, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int y = 0; y < 16; ++y) o[y] *= f;
                            tmem_st16(to + x, o);
                        }
                    }
                }
                if (edge) {
                    uint8_t* v = base + Lay::KV + (vs % S) * Lay::TILE;
                    const int lo = max(0, seen + 1 - t * PT_M), tail = it.L - t * PT_M;
                    if (unfit_values(v, r, lo, tail)) mend_values(v, fix + is, r, lo, tail, t * PT_M);
                    fence_proxy_async_smem();
                }
                const float neg = ref > -INFINITY ? -ref : 0.f;
                const float2 c2 = make_float2(c, c), n2 = make_float2(neg, neg);
                float2 acc = make_float2(0.f, 0.f);
#pragma unroll
                for (int part = 0; part < PT_PARTS; ++part) {
                    constexpr int W = PT_M / PT_PARTS;
#pragma unroll
                    for (int x = part * W; x < (part + 1) * W; x += 32) {
                        uint32_t w[16];
#pragma unroll
                        for (int y = 0; y < 32; y += 2) {
                            float2 e = fma2(make_float2(s[x + y], s[x + y + 1]), c2, n2);
                            e.x = ex2_approx(e.x);
                            e.y = ex2_approx(e.y);
                            if (y & 2) acc = add2(acc, e); else sum = add2(sum, e);
                            w[y >> 1] = pack2(e.x, e.y, BF16);
                        }
                        tmem_st16u(ts + x / 2, w);
                    }
                    tmem_wait_st();
                    tc05_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&b->p_full[q][part]);
                }
                sum = add2(sum, acc);
            }
            vstage += 2 * (max(it.e[0], it.e[1]) - it.t0);
            // ---- the tile's rows ----
            const float total = sum.x + sum.y;
            const bool direct = p.splits == 1 && !p.shared;
            const float inv = !direct ? 1.f : total != 0.f ? 1.f / total : 0.f;
            const bool any = t1 > it.t0;
            const size_t part0 = (static_cast<size_t>(it.slot) * 2 + q) * PT_M;
            uint8_t* dst[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const bool in = wtok[k] < p.tokens && q * p.tokens + wtok[k] < it.ntok;
                const size_t row = static_cast<size_t>(it.row0 + q * p.tokens + wtok[k]) * p.Hq + it.h * p.G + whead[k];
                dst[k] = !in ? nullptr
                         : direct ? static_cast<uint8_t*>(p.out) + row * D * 2
                         : any ? reinterpret_cast<uint8_t*>(p.part_acc + (part0 + (r & ~31) + k * 8 + (lane >> 2)) * D) : nullptr;
            }
            if (!direct && tok < p.tokens && q * p.tokens + tok < it.ntok) p.part_ml[part0 + r] = make_float2(ref, total);
            bool fixed = false;
            if (any) {
                if (!__all_sync(0xffffffffu, wait(p, &b->o_full[q], on++ & 1u))) return;
                tc05_fence_after();
                fixed = *reinterpret_cast<volatile int*>(&fix[is].any);
                __threadfence_block();
            }
#pragma unroll
            for (int x = 0; x < D; x += 32) {
                float o[32];
                if (any) {
                    tmem_ld32(to + x, o);
                    tmem_wait_ld();
                    if (fixed) {
#pragma unroll
                        for (int d = 0; d < 32; ++d) {
                            if (last >= fix[is].first[0][x + d]) o[d] = NAN;
                            if (last >= fix[is].first[1][x + d]) o[d] += INFINITY;
                            if (last >= fix[is].first[2][x + d]) o[d] -= INFINITY;
                        }
                    }
                } else {
#pragma unroll
                    for (int d = 0; d < 32; ++d) o[d] = 0.f;
                }
                uint4 w[4];
                if (direct) {
#pragma unroll
                    for (int d = 0; d < 4; ++d)
                        w[d] = make_uint4(pack2(o[8 * d] * inv, o[8 * d + 1] * inv, BF16), pack2(o[8 * d + 2] * inv, o[8 * d + 3] * inv, BF16),
                                          pack2(o[8 * d + 4] * inv, o[8 * d + 5] * inv, BF16), pack2(o[8 * d + 6] * inv, o[8 * d + 7] * inv, BF16));
                    put_rows(buf, lane, w, dst, x * 2);
                } else {
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
#pragma unroll
                        for (int d = 0; d < 4; ++d)
                            w[d] = make_uint4(__float_as_uint(o[16 * y + 4 * d]), __float_as_uint(o[16 * y + 4 * d + 1]),
                                              __float_as_uint(o[16 * y + 4 * d + 2]), __float_as_uint(o[16 * y + 4 * d + 3]));
                        put_rows(buf, lane, w, dst, (x + 16 * y) * 4);
                    }
                }
            }
            tc05_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&b->i_empty[is]);
        }
    }
};

// The sequence whose query rows hold `row`, or -1.
__device__ __forceinline__ int prompt_seq_of(const PromptParams& p, int row) {
    int lo = 0, hi = p.B;                                  // the last i with q_start[i] <= row
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (__ldg(p.q_start + m) <= row) lo = m; else hi = m;
    }
    return lo < p.B && __ldg(p.q_start + lo) <= row && row < __ldg(p.q_start + lo + 1) ? lo : -1;
}

// Shared mode: what each sequence has behind its group's prefix, for the decode
// kernel; -1 tokens for a sequence whose length does not fit.
__device__ __forceinline__ void write_tails(const PromptParams& p) {
    for (int i = blockIdx.x * PT_THREADS + threadIdx.x; i < p.total_q; i += gridDim.x * PT_THREADS) {
        const int g = prompt_seq_of(p, i);
        const int P = g >= 0 ? prompt_seq(p, g, false).L : 0;
        const int L = __ldg(p.lens + i);
        const bool ok = L >= P && L <= p.MB * p.bs;
        p.tail_lens[i] = ok ? L - P : -1;
        p.tail_blk[i] = P / p.bs;
    }
}

template <class KV, int D>
__global__ void __launch_bounds__(PT_THREADS, 1)
prompt_kernel(const __grid_constant__ PromptParams p, const __grid_constant__ CUtensorMap tq,
              const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv) {
    using K = PromptKernel<KV, D>;
    using Lay = PromptLayout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(base + Lay::FULL);
    uint64_t* empty = reinterpret_cast<uint64_t*>(base + Lay::EMPTY);
    PromptBars* b = reinterpret_cast<PromptBars*>(base + Lay::BARS);
    PromptItem* items = reinterpret_cast<PromptItem*>(base + Lay::ITEM);
    PromptFix* fix = reinterpret_cast<PromptFix*>(base + Lay::FIX);
    uint4* bad = reinterpret_cast<uint4*>(base + Lay::BAD);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < Lay::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int q = 0; q < 2; ++q) {
            mbar_init(&b->q_full[q], 1);
            mbar_init(&b->q_empty[q], 1);
            mbar_init(&b->s_full[q], 1);
            for (int x = 0; x < PT_PARTS; ++x) mbar_init(&b->p_full[q][x], 4);
            mbar_init(&b->o_full[q], 1);
        }
        for (int s = 0; s < PT_ITEMS; ++s) {
            mbar_init(&b->i_full[s], 1);
            mbar_init(&b->i_empty[s], 10);                 // 8 softmax warps, the MMA thread, the producer
        }
        mbar_init(&b->fin, 1);
        b->any_bad = 0;
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    __syncwarp();
    if (warp == 8) tmem_alloc<Lay::TCOLS>(&b->tmem);
    if (warp == 9 && lane == 0) {
        prefetch_tensormap(&tq);
        prefetch_tensormap(&tk);
        prefetch_tensormap(&tv);
    }
    tc05_fence_before();
    __syncthreads();
    tc05_fence_after();
    // a programmatic dependent of the kernel before it (the cache write): nothing that
    // it wrote is read before this
    grid_dependency_wait();
    grid_dependents_launch();
    if (p.shared) write_tails(p);
    if (warp >= 8) {
        regs_down<PT_REGS_FEW>();
        if (warp == 8) {
            if (elect_one()) K::mma(p, base, full, empty, b, items);
        } else if (warp == 9) {
            K::producer(p, base, full, empty, b, items, bad, &tq, &tk, &tv);
        } else if (warp == 10) {
            K::schedule(p, b, items, fix, reinterpret_cast<int2*>(base + Lay::KNOWN));
        }
    } else {
        regs_up<PT_REGS>();
        K::softmax(p, warp >> 2, base, full, b, items, fix, bad);
    }
    tc05_fence_before();
    __syncthreads();
    tc05_fence_after();
    __syncwarp();
    if (warp == 8) tmem_dealloc<Lay::TCOLS>(b->tmem);
}

// ---------------------------------------------------------------------------
// merge of the ranges of keys: out = sum_k 2^(r_k - M) O_k / sum_k 2^(r_k - M) l_k
// One warp per (query row, head).
// ---------------------------------------------------------------------------
template <class KV, int D>
__global__ void __launch_bounds__(256)
prompt_merge_kernel(const __grid_constant__ PromptParams p) {
    constexpr int DPL = D / 32;
    const int lane = threadIdx.x & 31;
    const long long w = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
    grid_dependency_wait();
    if (w >= static_cast<long long>(p.total_q) * p.Hq) return;
    const int row = static_cast<int>(w / p.Hq), h = static_cast<int>(w - static_cast<long long>(row) * p.Hq);
    const int i = prompt_seq_of(p, row);
    if (i < 0) return;
    const PromptSeq s = prompt_seq(p, i, false);
    if (s.n == 0) return;
    const int j = row - s.row0, t = j / (2 * p.tokens), u = j - t * 2 * p.tokens;
    const int q = u >= p.tokens, r = (u - q * p.tokens) * p.G + h % p.G;
    const size_t slot0 = (static_cast<size_t>(prompt_slot(s.row0, i, t, p.tokens)) * p.Hkv + h / p.G) * p.splits;
    float M = -INFINITY, den = 0.f, num[DPL];
#pragma unroll
    for (int x = 0; x < DPL; ++x) num[x] = 0.f;
    for (int k = 0; k < p.splits; ++k) {
        const size_t at = ((slot0 + k) * 2 + q) * PT_M + r;
        const float2 ml = p.part_ml[at];
        if (ml.y == 0.f) continue;
        const float Mn = fmaxf(M, ml.x), Mu = Mn > -INFINITY ? Mn : 0.f;
        const float a = exp2f(M - Mu), e = exp2f(ml.x - Mu);
        den = den * a + e * ml.y;
#pragma unroll
        for (int x = 0; x < DPL; ++x) num[x] = num[x] * a + e * p.part_acc[at * D + lane * DPL + x];
        M = Mn;
    }
    const float inv = den != 0.f ? 1.f / den : 0.f;
    typename KV::T* o = static_cast<typename KV::T*>(p.out) + (static_cast<size_t>(row) * p.Hq + h) * D + lane * DPL;
#pragma unroll
    for (int x = 0; x < DPL; ++x) o[x] = from_float<typename KV::T>(num[x] * inv);
}

}  // namespace pa
