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
// is 2 x 128 rows of one (sequence, KV head) and its keys, 128 at a time, and the
// warps of a CTA have a role each:
//   - the scheduler finds the items, the producer copies Q, K and V by TMA (128-byte
//     swizzle; paged K and V block by block through the table, K and V in a ring of
//     four tiles, eight at head_dim 64);
//   - one thread issues S_q = Q_q K^T and O_q += P_q V (q = 0, 1) as 128x128x16
//     MMAs; S, P and O live in tensor memory (P over the columns of its S);
//   - two groups of four warps run the softmax, one row per thread: while one of
//     them works on its S, the tensor cores work for the other;
//   - one warp keeps values that some row must not see from reaching it, four
//     write finished rows out while the next item's softmax is under way.
// Order of the MMAs: ... P0 V(j), S0(j+1), P1 V(j), S1(j+1) ...; a commit covers
// everything issued before it, so "S_q(j+1) is there" also says that P_q V(j) is
// in O_q, and the softmax warps may rescale O_q without a barrier of its own.
//
// CTAs are persistent.  Items go out by length, longest first and in turns of
// alternating direction, which balances causal items without a counter in memory;
// what is left of the last round (with few items, everything) is cut into ranges of
// keys where that pays, merged by prompt_merge_kernel.
//
// What bounds it, and what it measured.  A chunk takes a tile 4 x 128 x 128 x D
// flop: 1024 cycles at D = 128 if the tensor cores never wait.  One prompt of 32768
// tokens, 32/8 heads x 128, bf16: 4.8 ms, 1840 TFLOP/s (cuBLAS: 1980); D = 64 is
// bound by the softmax instead.  On the way there:
//   - MMAs and copies issued by an elected thread, whose operands the compiler may
//     keep in uniform registers (7.15 -> 5.3 ms; under `lane == 0` every MMA cost some
//     100 cycles to issue);
//   - P handed over in two parts (5.3 -> 5.1; four parts 5.1, and more to wait for);
//   - the roles' code kept small, since ten of them share the instruction cache: short
//     waits, rolled loops beside the hot ones (256 short prompts 627 -> 502 us);
//   - rows written out by warps of their own, items found by 32 bands of levels in
//     few instructions (502 -> 447; the first item is there after 9000 cycles, which
//     were 34000; 452-456 with f16 outputs limited and rows on any 16-byte boundary).
// Short prompts stay bound by what an item costs beside its chunks, about 8000 cycles.
// Not kept: the next item's scores ahead of the last products (no gain, more code);
// one tile's rows in both tiles, the chunks in turn (no gain as built, though neither memory
// nor the tensor cores bound such items: 47% and 24%); skipping masked columns and key steps
// (the tests cost more); one lane per block's copy.
#pragma once

#include <cuda.h>

#include <climits>
#include <cstdint>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_rows.cuh"

namespace pa {

constexpr int PT_M = 128;              // rows of a tile, keys of a chunk
constexpr int PT_THREADS = 512;        // 2 x 4 softmax warps, MMA, producer, scheduler, mender, 4 that write out
constexpr int PT_ITEMS = 4;            // items that the scheduler may be ahead
constexpr int PT_PARTS = 2;            // parts of P that the second product starts on
constexpr int PT_BAD = 8;              // chunks whose masks of bad blocks are kept: more than are under way
constexpr int PT_KNOWN = 1024;         // sequences whose items' numbers are kept
// Registers of a softmax thread, which holds a row of S, and of the others, out of
// the block's 128 each at launch.
constexpr int PT_REGS = 192, PT_REGS_FEW = 64;
static_assert(2 * PT_REGS + 2 * PT_REGS_FEW <= 4 * 128, "registers of the block");
constexpr float PT_SLACK = 8.f;        // log2 that a score may pass the reference by

struct PromptParams {
    void* out;
    const int32_t* q_start;            // [B + 1] query rows (members of each group in shared mode)
    const int32_t* k_start;            // [B + 1] rows of contiguous K and V, or null
    const int32_t* seq_lens;           // [B] keys, paged; shared mode: prefix lengths
    const int32_t* block_tables;       // paged: [rows][MB]
    int32_t* err_flag;
    float* part_acc;                   // [place][2][128][D]; shared mode: [sequence][head][range][D]
    float2* part_ml;                   // the same without D: (reference in log2 units, l)
    int B, Hq, Hkv, G, bs, NB, MB;
    int total_q, total_k;
    int tokens;                        // query tokens per tile, 128 / G
    int splits, causal, shared;        // splits: the most ranges that an item may be cut into
    int grid;                          // CTAs
    int4* cut;                         // for the merge: (b, cut items, a), and each one's (first row, tokens, head, place)
    // shared mode: lengths of the sequences, and what the decode kernel behind takes
    const int32_t* lens;               // [total_q]
    int32_t *tail_lens, *tail_blk;
    int rpb;                           // rows per TMA box of K and V
    int bs_log2, rpb_log2;
    Div div_tt, div_hkv;               // by 2 * tokens, by Hkv
    float c;                           // |scale| log2(e)
    uint32_t negate;                   // instruction descriptor bit of -Q, for scale < 0
};

// An item as the scheduler hands it on.
struct PromptItem {
    int live;                          // 0: no more items (the rest is unset)
    int row0, ntok;                    // first query row, query tokens of both tiles
    int pos0, L;                       // position of the first token, keys of the sequence
    int t0, e[2];                      // chunks [t0, e[q]) of tile q
    int h;                             // KV head
    int place;                         // of the partials, -1: rows of out; shared mode: the item's range of keys
    int ranges;                        // shared mode: how many there are
    int edge;                          // first chunk with keys that some row must not see
    int idx;                           // sequence (or group)
};

// Non-finite values of V among keys that some row of the tile must not see: the
// first such key of each column, by kind (NaN, +infinity, -infinity).
struct PromptFix {
    int any;
    int first[3][PT_M];
};

struct PromptBars {
    uint64_t q_full[2], q_empty[2], s_full[2], p_full[2][PT_PARTS], o_full[2], o_empty[2];
    uint64_t l_full[PT_ITEMS][2];      // (reference, l) of an item's tile
    uint64_t v_there, v_fit;           // an edge chunk's V has come, is mended; the edge chunks in turn
    uint64_t i_full[PT_ITEMS], i_empty[PT_ITEMS];
    uint64_t fin;
    uint32_t tmem;
    int any_bad;                       // a block id outside the pool was met
    alignas(16) int box[16];           // first groups of pool rows of a chunk's boxes
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
    static constexpr uint32_t BAD = (FIX + PT_ITEMS * sizeof(PromptFix) + 15) & ~15u;   // a uint4 each
    static constexpr uint32_t ROWS = (BAD + 16 * PT_BAD + 15) & ~15u;        // (reference, l) of each item's rows
    static constexpr uint32_t KNOWN = ROWS + PT_ITEMS * 2 * PT_M * 8;       // the first sequences' numbers
    static constexpr uint32_t BYTES = KNOWN + 16 * PT_KNOWN + 1024;   // + alignment of the base
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

// Shared mode: groups that would save fewer reads of a token than this are left to the
// decode kernel, prefix and all.  (28/4 heads x 128, 32 groups: two members with 1024
// tokens 46 us shared, 41 left to it; four 52 and 54; two with 4096 tokens 84 and 103.)
constexpr int PT_SHARED_SAVED = 2048;

// The tokens that group i shares, in whole blocks, and those of them that are attended once.
__device__ __forceinline__ int group_prefix(const PromptParams& p, int i) {
    return max(0, min(__ldg(p.seq_lens + i), p.MB * p.bs)) & ~(p.bs - 1);
}
__device__ __forceinline__ int shared_prefix(const PromptParams& p, int i, int n) {
    const int P = group_prefix(p, i);
    return static_cast<long long>(n - 1) * P >= PT_SHARED_SAVED ? P : 0;
}

__device__ __forceinline__ int prompt_items_of(const PromptParams& p, int n) {
    return static_cast<int>(div_by(n + 2 * p.tokens - 1, p.div_tt));
}

// Sequence (or group) i; n = 0 where its numbers do not fit or it has no items.
static __device__ __noinline__ PromptSeq prompt_seq(const PromptParams& p, int i, bool report) {
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
    if (p.shared && s.L == 0) s.n = 0;
    s.a = static_cast<int>(div_by(p.shared ? s.L : max(0, s.L - s.n), p.div_tt));
    s.c = prompt_items_of(p, s.n);
    return s;
}

// The sequence whose query rows hold `row`, or -1.
__device__ __forceinline__ int prompt_seq_of(const PromptParams& p, int row) {
    int lo = 0, hi = p.B;                                  // the last i with q_start[i] <= row
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (__ldg(p.q_start + m) <= row) lo = m; else hi = m;
    }
    return lo < p.B && __ldg(p.q_start + lo) <= row && row < __ldg(p.q_start + lo + 1) ? lo : -1;
}

// Shared mode: whether a row's group is `group` (groups whose entries fall back overlap; a row
// then belongs to one of them).
static __device__ __noinline__ bool prompt_member(const PromptParams& p, int row, int group) {
    return row < p.total_q && prompt_seq_of(p, row) == group;
}

// Items of a sequence of c items from level a on that lie at level u or above: causal
// items one to a level, the items of a group all at a.
__device__ __forceinline__ int items_from(const PromptParams& p, int a, int c, int u) {
    return p.shared ? (a >= u ? c : 0) : min(max(a + c - u, 0), c);
}

// The items of the launch in order of length, for one warp: in up to 32 bands of
// 2^shift levels, from the highest down, within one by sequence, the longest first.
// (Every instruction here runs once or a few times and is fetched from far away, 12
// cycles each: short code starts sooner than clever code.)
struct PromptOrder {
    int4* known;                       // (first row, tokens, keys, level) of the first PT_KNOWN sequences
    int top, total;                    // the highest level; items per KV head
    int shift;                         // 31: one band, the order does not matter
    int above;                         // lane u: items in band u and above
    int band, chunk, before;           // where the last item was found: the band's items before sequence 32 chunk

    __device__ __forceinline__ int4 seq(const PromptParams& p, int i) const {
        if (i >= p.B) return make_int4(0, 0, 0, 0);
        if (i < PT_KNOWN) return known[i];
        const PromptSeq s = prompt_seq(p, i, false);
        return make_int4(s.row0, s.n, s.L, s.a);
    }
    __device__ __forceinline__ void init(const PromptParams& p, int4* smem, bool report) {
        const int lane = threadIdx.x & 31;
        known = smem;
        int high = 0, n = 0;
#pragma unroll 1
        for (int i = lane; i < p.B; i += 32) {
            const PromptSeq s = prompt_seq(p, i, report);
            if (i < PT_KNOWN) known[i] = make_int4(s.row0, s.n, s.L, s.a);
            if (s.c > 0) high = max(high, p.shared ? s.a : s.a + s.c - 1);
            n += s.c;
        }
        __syncwarp();
        total = __reduce_add_sync(0xffffffffu, n);
        top = __reduce_max_sync(0xffffffffu, high);
        band = 32;
        chunk = before = 0;
        shift = 31;
        above = lane == 0 ? total : 0;
        if (total * p.Hkv <= p.grid) return;               // one round
        shift = max(0, 27 - __clz(top));                   // top >> shift < 32
        above = 0;
#pragma unroll 1
        for (int i0 = 0; i0 < p.B; i0 += 32) {
            const int4 s = seq(p, i0 + lane);
            const int c = prompt_items_of(p, s.y), m = min(32, p.B - i0);
#pragma unroll 1
            for (int j = 0; j < m; ++j)
                above += items_from(p, __shfl_sync(0xffffffffu, s.w, j), __shfl_sync(0xffffffffu, c, j), lane << shift);
        }
    }
    // Item k (below total, from call to call not smaller): its sequence's index and
    // numbers, its number in the sequence.
    __device__ __forceinline__ void find(const PromptParams& p, int k, int& idx, int4& s, int& t) {
        const int lane = threadIdx.x & 31;
        const int u = 31 - __clz(__ballot_sync(0xffffffffu, above > k) | 1u);
        const int next = __shfl_sync(0xffffffffu, above, (u + 1) & 31);
        if (u != band) { band = u; chunk = before = 0; }
        int r = k - (u == 31 ? 0 : next);
#pragma unroll 1
        for (;; ++chunk) {
            const int4 x = seq(p, 32 * chunk + lane);
            const int c = prompt_items_of(p, x.y);
            const int from = shift == 31 ? 0 : items_from(p, x.w, c, (u + 1) << shift);      // above the band
            const int own = (shift == 31 ? c : items_from(p, x.w, c, u << shift)) - from;
            int inc = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            const int all = __shfl_sync(0xffffffffu, inc, 31);
            if (r - before >= all && 32 * (chunk + 1) < p.B) {
                before += all;
                continue;
            }
            r -= before;
            const int src = 31 - __clz(__ballot_sync(0xffffffffu, inc - own <= r && own > 0) | 1u);
            t = __shfl_sync(0xffffffffu, c - 1 - from + inc - own, src) - r;
            idx = 32 * chunk + src;
            s = make_int4(__shfl_sync(0xffffffffu, x.x, src), __shfl_sync(0xffffffffu, x.y, src),
                          __shfl_sync(0xffffffffu, x.z, src), 0);
            return;
        }
    }
};

// How the items of a launch are cut: the first `whole` not at all; the others, one behind
// the other, into spans of a / b items each, a < b (or not at all, b = 1).  A span is at
// most the end of an item and the start of the next; all spans end at multiples of 1 / b of
// an item, so that items of one length read the same keys at the same time.
struct PromptCut {
    int whole, a, b;
};
// CTAs take whole rounds of items; what is left of the last round, the lightest items, is
// cut so that all CTAs have part of it.  (In shared mode all items are cut into b parts each.)
// With r items left, spans of a / b take ceil(w a / b) chunks' time of items of w chunks, and 6
// for each item that they are of (what an item costs beside its chunks); the merge takes 8.
// The rounds before leave CTAs unequal, so that the first, middle and last span count with
// what their CTA had before, and so does the last CTA.
// (2048 tokens behind 63488, 32/8 heads, 256 items: 1292 us, uncut 1354.  512 tokens each behind
// 100-8192, 28/4 heads, 232 items of unequal length: 126 uncut, 139 cut as if all were equal.)
__device__ __forceinline__ PromptCut prompt_cut(const PromptParams& p, const PromptOrder& order) {
    const int items = order.total * p.Hkv;
    PromptCut c{items, 1, 1};
    if (p.splits == 1) return c;
    const float grid = static_cast<float>(p.grid);
    const int R = p.shared ? 0 : static_cast<int>(floorf(__fdividef(items + 0.5f, grid)));
    c.whole = R * p.grid;
    const float r = static_cast<float>(items - c.whole);
    if (r == 0.f) return c;
    const float b = static_cast<float>((threadIdx.x & 31) + 1);
    const float full = ceilf(__fdividef(r * b - 0.5f, grid));
    const float a = p.shared ? 1.f : full, rounds = p.shared ? full : 1.f, part = __fdividef(a, b);
    const int spans = static_cast<int>(ceilf(__fdividef(r, part) - 0.01f));
    const int at[4] = {0, spans >> 1, spans - 1, p.grid - 1};      // places in the last round
    const int bands = order.shift == 31 ? 1 : 32;
    float w = 0.f, load[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int t = 0; t <= R; ++t) {
        int rank[4], u[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const int i = t == R ? static_cast<int>(at[y] * part) : (t ^ R) & 1 ? p.grid - 1 - at[y] : at[y];
            rank[y] = static_cast<int>(div_by(max(0, t * p.grid + i), p.div_hkv));
            u[y] = 0;
        }
#pragma unroll 1
        for (int x = 1; x < bands; ++x) {
            const int n = __shfl_sync(0xffffffffu, order.above, x);
#pragma unroll
            for (int y = 0; y < 4; ++y)
                if (n > rank[y]) u[y] = x;
        }
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            // chunks of the longest item of the band
            const int level = order.shift == 31 ? order.top : min(order.top, ((u[y] + 1) << order.shift) - 1);
            const float n = fmaxf(1.f, ceilf(static_cast<float>(level + 2) * static_cast<float>(2 * p.tokens) * (1.f / PT_M)));
            if (y == 0) w = n;
            if (t < R) load[y] += n + 6.f;
            else if (y < 3) load[y] += ceilf(n * part - 0.01f) + (a > 1.f ? 12.f : 6.f);
        }
    }
    float cost = rounds * fmaxf(fmaxf(load[0], load[1]), fmaxf(load[2], load[3])) + (b > 1.f && !p.shared ? 8.f : 0.f);
    if (b > 1.f && (b > static_cast<float>(p.splits) || b > w || a >= b || r * b > 2.f * grid * a)) cost = 1e9f;
    // the cheapest, of equal ones the first: costs are whole numbers below 2^26
    const int best = __reduce_min_sync(0xffffffffu, static_cast<uint32_t>(fminf(cost, 6.7e7f)) << 5 | (threadIdx.x & 31)) & 31;
    c.b = best + 1;
    c.a = static_cast<int>(__shfl_sync(0xffffffffu, a, best));
    return c;
}

// Number v in the order of a launch cut as c says: an item, or a span's first part or, second
// set, its other.  more: there is another; first: for an item's first part the item's number
// among the cut ones, else -1.
__device__ __forceinline__ PromptItem prompt_item(const PromptParams& p, PromptOrder& order, const PromptCut& c, int v,
                                                  bool second, int& first, bool& more) {
    const int TT = 2 * p.tokens;
    int k = v, from = 0, to = c.b, place = -1;             // parts from / b to to / b of item k
    first = -1;
    more = false;
    if (v >= c.whole && c.b > 1) {                         // at most two spans to a CTA
        const int span = v - c.whole;
        const int i = static_cast<int>(__fdividef(span * c.a + 0.5f, static_cast<float>(c.b))) + (second ? 1 : 0);
        k = c.whole + i;
        from = max(0, span * c.a - i * c.b);
        to = (span + 1) * c.a - i * c.b;
        more = to > c.b && k + 1 < order.total * p.Hkv;
        to = min(to, c.b);
        place = span + i;                                  // those of an item one behind the other
        if (from == 0) first = i;
    }
    const int kk = static_cast<int>(div_by(k, p.div_hkv));
    PromptItem it{};
    int4 s;
    int t;
    order.find(p, kk, it.idx, s, t);
    // (q_start that falls again and again could count past 32 bits)
    t = max(0, min(t, prompt_items_of(p, s.y) - 1));
    it.live = 1;
    it.h = k - kk * p.Hkv;
    it.row0 = s.x + t * TT;
    it.ntok = min(TT, s.y - t * TT);
    it.pos0 = s.z - s.y + t * TT;
    it.L = s.z;
    // keys of each tile's last row, in chunks
    const int n0 = min(it.ntok, p.tokens), n1 = it.ntok - n0;
    const int e0 = max(0, (p.causal ? it.pos0 + n0 : s.z) + PT_M - 1) / PT_M;
    const int e1 = n1 > 0 ? max(0, (p.causal ? it.pos0 + it.ntok : s.z) + PT_M - 1) / PT_M : 0;
    const int most = max(e0, e1);
    int t1 = most;
    if (c.b > 1) {                                         // (chunks < 2^23, b <= 32)
        it.t0 = most * from / c.b;
        t1 = most * to / c.b;
    }
    it.e[0] = max(it.t0, min(e0, t1));
    it.e[1] = max(it.t0, min(e1, t1));
    // the last key that every row of the first tile with chunks sees
    const int seen = p.causal ? min(it.pos0 + (it.e[0] > it.t0 ? 0 : p.tokens), it.L - 1) : it.L - 1;
    it.edge = max(0, seen + 1) / PT_M;
    it.place = p.shared ? from : place;
    it.ranges = c.b;
    return it;
}

// ---------------------------------------------------------------------------
// tensor memory and packed arithmetic
// ---------------------------------------------------------------------------
// The two halves of a descriptor of a 128-byte-swizzled operand (umma_desc): the
// address, to which steps along K are added, and what does not change.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) { return (addr >> 4) | (lbo >> 4) << 16; }
__host__ __device__ constexpr uint32_t desc_hi(uint32_t sbo) { return (sbo >> 4) | 1u << 14 | 2u << 29; }
// D (+)= A B, issued by one thread; A from shared memory or, 16-bit pairs, tensor memory.
template <bool ADD>
__device__ __forceinline__ void umma_ss(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t b_hi, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %6};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}"
        :: "r"(d_tmem), "r"(a), "r"(b), "r"(idesc), "n"(ADD ? 1 : 0), "n"(desc_hi(1024)), "r"(b_hi) : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b, uint32_t b_hi, uint32_t idesc,
                                        uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}"
        :: "r"(d_tmem), "r"(a_tmem), "r"(b), "r"(idesc), "r"(add), "r"(b_hi) : "memory");
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
// SHARED: the shared mode, whose rows go out as partials by (sequence, head).  (A kernel of its own:
// the places of both kinds worked out by one take 256 short prompts from 454 to 462 us.)
template <class KV, int D, bool PAGED, bool SHARED>
struct PromptKernel {
    using Lay = PromptLayout<D>;
    // K and V tiles in shared memory: 8-row groups of 128-byte rows GROUP bytes apart,
    // planes of 64 columns PLANE.  Contiguous: whole planes, a copy each.  Paged: the
    // planes of a group one behind the other, so that one copy brings a block's rows of
    // both and equal steps still lead from group to group.
    static constexpr uint32_t PLANE = PAGED ? 1024 : Lay::PLANE, GROUP = PAGED ? D / 64 * 1024 : 1024;
    static constexpr bool BF16 = KV::code == PA_BF16;
    static constexpr int PLANES = D / 64;
    static constexpr int S = Lay::STAGES;
    // P is kept above 2^-24 for f16 operands: its largest is about 2^7 there, at most
    // 2^15, so that weights down to 2^-31 of a row's largest still count (11 bits down
    // to 2^-21); bf16 has the range of f32 and needs none of it.
    static constexpr float LIFT = BF16 ? 0.f : 7.f;

    // Every wait ends after 2^31 cycles (about a second) at the latest.  The instructions
    // are few: what the ten roles of this kernel run has to share the instruction cache.
    // A wait for something that comes once per item may take as long as the item, of up to
    // 2^23 chunks: 16 times as much.
    template <int ROUNDS = 1>
    static __device__ __forceinline__ bool wait(const PromptParams& p, uint64_t* bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity)) return true;
#pragma unroll 1
        for (int x = 0; x < ROUNDS; ++x) {
            const uint32_t t0 = static_cast<uint32_t>(clock());
            do {
                if (mbar_try_wait(bar, parity)) return true;
            } while (static_cast<uint32_t>(clock()) - t0 < 0x80000000u);
        }
        raise_flag(p.err_flag, PA_ERRBIT_WAIT_TIMEOUT);
        return false;
    }
    static __device__ __forceinline__ bool wait_item(const PromptParams& p, uint64_t* bar, uint32_t parity) {
        return wait<16>(p, bar, parity);
    }

    // ---------------- scheduler: one warp finds the CTA's items ----------------
    static __device__ void schedule(const PromptParams& p, PromptBars* b, PromptItem* items, PromptFix* fix, int4* known) {
        const int lane = threadIdx.x & 31;
        PromptOrder order;
        order.init(p, known, blockIdx.x == 0);
        int total = order.total * p.Hkv;
        PromptCut c{total, 1, 1};
        bool more = false, planned = false;
        for (int turn = 0, round = 0;; ++turn) {
            const int slot = turn % PT_ITEMS;
            bool ok = true;
            if (turn >= PT_ITEMS) ok = wait_item(p, &b->i_empty[slot], (turn / PT_ITEMS - 1) & 1u);
            if (!__all_sync(0xffffffffu, ok)) return;
            if (!planned && (round == 1 || p.shared || total < p.grid)) {      // (behind a whole round its items go first)
                planned = true;
                c = prompt_cut(p, order);
                const int left = total - c.whole;
                total = c.whole + (c.b > 1 ? (left * c.b + c.a - 1) / c.a : left);
                if (p.cut && blockIdx.x == 0 && lane == 0) p.cut[0] = make_int4(c.b, c.b > 1 ? left : 0, c.a, 0);
            }
            // rounds of alternating direction: CTA b takes b, 2 grid - 1 - b, 2 grid + b, ...
            // (k is below the next round's first number: behind the last item there are no more rounds)
            const int k = round * gridDim.x + (round & 1 ? static_cast<int>(gridDim.x) - 1 - static_cast<int>(blockIdx.x)
                                                         : static_cast<int>(blockIdx.x));
            PromptItem it{};
            if (k < total) {
                int first;
                it = prompt_item(p, order, c, k, more, first, more);
                if (!p.shared && first >= 0 && lane == 0) p.cut[1 + first] = make_int4(it.row0, it.ntok, it.h, it.place);
            }
            if (!more) ++round;
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

    // The NB boxes of a paged tile; coordinates (column, row of a group, plane, group, head).
    template <int NB>
    static __device__ __forceinline__ void boxes(uint8_t* dst, const CUtensorMap* map, uint64_t* bar, const int* group, int h) {
        int g[NB];
#pragma unroll
        for (int x = 0; x < NB; ++x) g[x] = group[x];      // all under way before the first is used
#pragma unroll
        for (int x = 0; x < NB; ++x) tma_load_5d(dst + x * (PT_M / NB / 8) * GROUP, map, bar, 0, 0, 0, g[x], h);
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
            ok = __all_sync(0xffffffffu, wait_item(p, &b->i_full[is], (turn / PT_ITEMS) & 1u));
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
                if (elect_one()) {
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
            if constexpr (!PAGED) k0 = __ldg(p.k_start + it.idx);
            else table = p.block_tables + static_cast<size_t>(p.shared ? __ldg(p.q_start + it.idx) : it.idx) * p.MB;
            const int nblk = (it.L + p.bs - 1) >> p.bs_log2;     // paged: blocks that the sequence uses
            // lane x < nb copies box x of each chunk; the next chunk's table entry is read ahead
            auto entry = [&](int t) -> int {               // first pool row of the lane's box in chunk t, or -1
                const int tok = t * PT_M + (lane << p.rpb_log2);
                const int j = tok >> p.bs_log2;
                if (lane >= nb || j >= nblk) return -1;
                const int id = __ldg(table + j);
                return id < 0 || id >= p.NB ? -2 : (id << p.bs_log2) + (tok & (p.bs - 1));
            };
            int next = PAGED ? entry(it.t0) : 0;
#pragma unroll 1
            for (int q = 0; q < 2 && ok; ++q) queries(q);
#pragma unroll 1
            for (int j = 0; j < n && ok; ++j) {
                const int t = it.t0 + j;
                int row = next;
                if constexpr (PAGED) {
                    if (j + 1 < n) next = entry(t + 1);
                } else {
                    row = k0 + t * PT_M;
                }
                if constexpr (PAGED) {
                    // keys of blocks outside the pool are left out; this chunk's K is not on its
                    // way yet, so no softmax warp has come to it
                    const uint32_t miss = __ballot_sync(0xffffffffu, row == -2);
                    const int any_bad = *reinterpret_cast<volatile int*>(&b->any_bad);
                    if (miss | any_bad) {
                        uint32_t w = 0;                    // lane x: the keys 32 x .. 32 x + 31
#pragma unroll 1
                        for (int y = 0; y < 32; ++y) w |= (miss >> ((32 * (lane & 3) + y) >> p.rpb_log2) & 1u) << y;
                        if (lane < 4) reinterpret_cast<uint32_t*>(bad + (issued / 2) % PT_BAD)[lane] = w;
                        if (miss && lane == 0) {
                            raise_flag(p.err_flag, PA_ERRBIT_BAD_BLOCK);
                            *reinterpret_cast<volatile int*>(&b->any_bad) = 1;
                        }
                        __syncwarp();
                    }
                }
                // boxes without rows start behind the pool, where TMA fills in zeros
                const int at = PAGED && row < 0 ? p.NB << p.bs_log2 : row;
                if constexpr (PAGED) {
                    __syncwarp();
                    if (lane < 16) b->box[lane] = at >> 3;
                    __syncwarp();
                }
#pragma unroll 1
                for (int v = 0; v < 2; ++v) {
                    const int st = issued % S;
                    if (issued >= S) ok = ok && wait(p, &empty[st], (issued / S - 1) & 1u);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    uint8_t* dst = base + Lay::KV + st * Lay::TILE;
                    // One elected thread issues the copies, their number known to the compiler and the
                    // rows loaded ahead, so that operands stay in uniform registers: blocks of 8 and 16
                    // tokens then take no longer than those of 128 (with a lane per box 2.1 and 1.4
                    // times as long).
                    if (elect_one()) {
                        mbar_arrive_expect_tx(&full[st], Lay::TILE);
                        const CUtensorMap* map = v ? tv : tk;
                        if constexpr (PAGED) {
                            if (nb == 16) boxes<16>(dst, map, &full[st], b->box, it.h);
                            else if (nb == 8) boxes<8>(dst, map, &full[st], b->box, it.h);
                            else if (nb == 4) boxes<4>(dst, map, &full[st], b->box, it.h);
                            else if (nb == 2) boxes<2>(dst, map, &full[st], b->box, it.h);
                            else boxes<1>(dst, map, &full[st], b->box, it.h);
                        } else {
#pragma unroll
                            for (int pl = 0; pl < PLANES; ++pl)
                                tma_load_4d(dst + pl * PLANE, map, &full[st], 0, at, it.h, pl);
                        }
                    }
                    __syncwarp();
                    ++issued;
                }
            }
        }
        // every copy must land before the CTA exits
#pragma unroll 1
        for (int st = max(0, issued - S); st < issued; ++st)
            if (!wait(p, &full[st % S], (st / S) & 1u)) break;
#pragma unroll 1
        for (int q = 0; q < 2; ++q)
            if (qload[q] > 0) wait(p, &b->q_full[q], (qload[q] - 1) & 1u);
    }

    // ---------------- MMA issue (one thread) ----------------
    static __device__ void mma(const PromptParams& p, uint8_t* base, uint64_t* full, uint64_t* empty, PromptBars* b,
                               const PromptItem* items) {
        const uint32_t tm = b->tmem;
        const uint32_t id_s = umma_idesc_f16(BF16, PT_M, PT_M, false, false) | p.negate;
        const uint32_t id_o = umma_idesc_f16(BF16, PT_M, D, false, true);
        constexpr uint32_t hi = desc_hi(GROUP);
        const uint32_t qb = smem_u32(base + Lay::Q), kvb = smem_u32(base + Lay::KV);
        int used = 0;                                      // stages gone through
        int qn[2] = {0, 0};
        uint32_t pn[2] = {0, 0};
        uint32_t on[2] = {0, 0}, edges = 0;
        bool ok = true;
        auto score = [&](int q, int st, bool last) {       // S_q = Q_q K^T
            const uint32_t a = desc_lo(qb + q * Lay::TILE, 16), k = desc_lo(kvb + st * Lay::TILE, 16), d = tm + q * PT_M;
            tc05_fence_after();
            umma_ss<false>(d, a, k, hi, id_s);
#pragma unroll
            for (int kk = 1; kk < D / 16; ++kk) {
                constexpr uint32_t STEP = 32u >> 4;
                umma_ss<true>(d, a + (kk >> 2) * (Lay::PLANE >> 4) + (kk & 3) * STEP, k + (kk >> 2) * (PLANE >> 4) + (kk & 3) * STEP, hi,
                              id_s);
            }
            umma_commit(&b->s_full[q]);
            if (last) umma_commit(&b->q_empty[q]);
        };
        auto value = [&](int q, int st, bool first) {      // O_q (+)= P_q V, as the parts of P come
            // the O of the item before must have been taken out
            if (first && on[q]++ > 0 && !wait(p, &b->o_empty[q], on[q] & 1u)) return false;
            const uint32_t v = desc_lo(kvb + st * Lay::TILE, PLANE), d = tm + Lay::OCOL + q * D, a = tm + q * PT_M;
            const uint32_t phase = pn[q]++ & 1u;
#pragma unroll
            for (int part = 0; part < PT_PARTS; ++part) {
                if (!wait(p, &b->p_full[q][part], phase)) return false;
                tc05_fence_after();
#pragma unroll
                for (int x = 0; x < PT_M / 16 / PT_PARTS; ++x) {
                    const int kk = part * (PT_M / 16 / PT_PARTS) + x;
                    umma_ts(d, a + kk * 8, v + kk * (2 * GROUP >> 4), hi, id_o, kk > 0 || !first);
                }
            }
            return true;
        };
        for (int turn = 0; ok; ++turn) {
            const int is = turn % PT_ITEMS;
            if (!(ok = wait_item(p, &b->i_full[is], (turn / PT_ITEMS) & 1u))) break;
            const PromptItem it = items[is];
            mbar_arrive(&b->i_empty[is]);
            if (!it.live) break;
            const int n0 = it.e[0] - it.t0, n1 = it.e[1] - it.t0, n = max(n0, n1);
            if (n == 0) continue;
            // chunk j: K in stage 2 j of the item's, V in the one behind it
            if (!(ok = wait(p, &full[used % S], (used / S) & 1u))) break;
#pragma unroll 1
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
                const bool edge = it.t0 + j >= it.edge;
                if (edge) mbar_arrive(&b->v_there);        // mended while the softmax is at work on S
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int nq = q ? n1 : n0;
                    if (q == 0 && edge && !(ok = wait(p, &b->v_fit, edges++ & 1u))) break;
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

    // ---------------- mender: one warp ----------------
    // Keys that some row of an item must not see, in an edge chunk's V: values that are
    // not finite, whose product with a weight of 0 would be NaN, become zeros.  Those of the
    // sequence are noted by column and first key before, and come back at the end for the
    // rows that do see them.
    static __device__ __forceinline__ uint8_t* value_at(uint8_t* v, int row, int ch) {
        return v + (ch >> 3) * PLANE + (row >> 3) * GROUP + swz128(row & 7, ch & 7);
    }
    static __device__ __noinline__ void mend_values(uint8_t* v, PromptFix* fix, int lane, int lo, int tail, int key0) {
        constexpr int CH = D / 8;                          // 16-byte pieces of a row
#pragma unroll 1
        for (int x = lane; x < (PT_M - lo) * CH; x += 32) {
            const int row = lo + x / CH, ch = x % CH;
            uint4* at = reinterpret_cast<uint4*>(value_at(v, row, ch));
            if (row >= tail) {
                *at = make_uint4(0, 0, 0, 0);
                continue;
            }
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
    static __device__ void mend(const PromptParams& p, uint8_t* base, uint64_t* full, PromptBars* b, const PromptItem* items,
                                PromptFix* fix) {
        using E2 = std::conditional_t<BF16, __nv_bfloat162, __half2>;
        constexpr int U = 8;                               // accesses in flight
        const int lane = threadIdx.x & 31;
        const uint32_t zero = 0;
        const E2 none = *reinterpret_cast<const E2*>(&zero);
        int stage = 1;                                     // of the item's first V
        uint32_t edges = 0;
        for (int turn = 0;; ++turn) {
            const int is = turn % PT_ITEMS;
            if (!__all_sync(0xffffffffu, wait_item(p, &b->i_full[is], (turn / PT_ITEMS) & 1u))) return;
            const PromptItem it = items[is];
            if (!it.live) return;
            const int t1 = max(it.e[0], it.e[1]);
            const int seen = p.causal ? min(it.pos0 + (it.e[0] > it.t0 ? 0 : p.tokens), it.L - 1) : it.L - 1;
            for (int t = max(it.t0, it.edge); t < t1; ++t, ++edges) {
                const int vs = stage + 2 * (t - it.t0);
                // (full alone would not do: it may be rounds behind or ahead of a warp that
                // looks at some chunks only)
                if (!__all_sync(0xffffffffu, wait_item(p, &b->v_there, edges & 1u) && wait(p, &full[vs % S], (vs / S) & 1u))) return;
                uint8_t* v = base + Lay::KV + (vs % S) * Lay::TILE;
                const int lo = max(0, seen + 1 - t * PT_M), tail = min(PT_M, it.L - t * PT_M);
                // is there anything to mend from the 8-row group of row lo on?  0 * x is NaN for an
                // x that is not finite
                E2 acc[4] = {none, none, none, none};
                constexpr int SPANS = PAGED ? 1 : PLANES;   // stretches that lie together
                const int first = (lo >> 3) * GROUP, end = PT_M / 8 * GROUP;
#pragma unroll 1
                for (int span = 0; span < SPANS; ++span)
#pragma unroll 1
                for (int at = first + lane * 16; at < end; at += U * 512) {
                    uint4 raw[U];
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        raw[u] = at + u * 512 < end ? *reinterpret_cast<const uint4*>(v + span * PLANE + at + u * 512)
                                                    : make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const E2* e = reinterpret_cast<const E2*>(&raw[u]);
#pragma unroll
                        for (int y = 0; y < 4; ++y) acc[y] = __hfma2(e[y], none, acc[y]);
                    }
                }
                const E2 sum = __hadd2(__hadd2(acc[0], acc[1]), __hadd2(acc[2], acc[3]));
                if (__any_sync(0xffffffffu, __hisnan(sum.x) || __hisnan(sum.y)))
                    mend_values(v, fix + is, lane, lo, tail, t * PT_M);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&b->v_fit);
            }
            stage += 2 * (t1 - it.t0);
            __syncwarp();
            if (lane == 0) mbar_arrive(&b->i_empty[is]);
        }
    }

    // ---------------- softmax: tile q, one row per thread ----------------
    static __device__ void softmax(const PromptParams& p, int q, PromptBars* b, const PromptItem* items, const uint4* bad,
                                   float2* rows) {
        const int r = threadIdx.x & (PT_M - 1);            // tile row = tensor-memory lane
        const int lane = threadIdx.x & 31;
        const uint32_t lanes = static_cast<uint32_t>(r & ~31) << 16;
        const uint32_t ts = b->tmem + lanes + q * PT_M, to = b->tmem + lanes + Lay::OCOL + q * D;
        const int tok = r / p.G;
        const float c = p.c;
        uint32_t sn = 0;
        int chunk = 0;                                     // chunks of the items before
        for (int turn = 0;; ++turn) {
            const int is = turn % PT_ITEMS;
            if (!__all_sync(0xffffffffu, wait_item(p, &b->i_full[is], (turn / PT_ITEMS) & 1u))) return;
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
                const int any_bad = PAGED ? *reinterpret_cast<volatile int*>(&b->any_bad) : 0;
                tmem_wait_ld();
                const bool edge = t * PT_M + PT_M - 1 > seen;
                if (edge || any_bad) {
                    const int rel = last - t * PT_M;       // the row sees columns up to this one
                    const uint32_t* out = reinterpret_cast<const uint32_t*>(bad + (chunk + t - it.t0) % PT_BAD);
#pragma unroll
                    for (int x = 0; x < PT_M; x += 32) {
                        uint32_t w = rel - x >= 31 ? 0xffffffffu : rel < x ? 0u : (2u << (rel - x)) - 1u;
                        if (any_bad) w &= ~out[x / 32];
                        if (__all_sync(0xffffffffu, w == 0xffffffffu)) continue;
#pragma unroll
                        for (int y = 0; y < 32; ++y) s[x + y] = (w >> y) & 1u ? s[x + y] : -INFINITY;
                    }
                }
                float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int x = 4; x < PT_M - 4; x += 8) {
#pragma unroll
                    for (int y = 0; y < 4; ++y) mx[y] = max3(mx[y], s[x + y], s[x + 4 + y]);
                }
#pragma unroll
                for (int y = 0; y < 4; ++y) mx[y] = fmaxf(mx[y], s[PT_M - 4 + y]);
                const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
                // the reference moves at the row's first key and when it is passed by 2^8
                const bool move = top * c > ref + (PT_SLACK + LIFT) && top > -INFINITY;
                if (__any_sync(0xffffffffu, move)) {
                    const float to_ref = move ? top * c - LIFT : ref;
                    const float f = move ? exp2f(ref - to_ref) : 1.f;
                    ref = to_ref;
                    sum.x *= f;
                    sum.y *= f;
                    if (t > it.t0) {
#pragma unroll 1
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
            chunk += max(it.e[0], it.e[1]) - it.t0;
            // (reference, l) for the warps that write the rows out
            rows[(is * 2 + q) * PT_M + r] = make_float2(ref, sum.x + sum.y);
            __syncwarp();
            if (lane == 0) mbar_arrive(&b->l_full[is][q]);
            if (lane == 0) mbar_arrive(&b->i_empty[is]);
        }
    }

    // ---------------- rows out: four warps, both tiles in turn ----------------
    // 32 bytes: one access where the address is a multiple of 32 (`wide`), which a caller's
    // tensor need not be, else two of 16.  (Two of 16 always: 256 short prompts 476 us, so 456.)
    static __device__ __forceinline__ void put32(void* dst, const uint32_t (&w)[8], bool wide) {
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %9, 0;\n\t@p st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n\t"
                     "@!p st.global.v4.b32 [%0], {%1,%2,%3,%4};\n\t@!p st.global.v4.b32 [%0+16], {%5,%6,%7,%8};\n\t}"
                     :: "l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "r"(static_cast<int>(wide))
                     : "memory");
    }
    // Rows of f16 once more, where some quotient passes the largest f16 (as FiniteHalf says).
    // (Apart from the rows' own loop, which only looks for such quotients: limited there, 256 short
    // prompts take 465 us, so 455.)
    static __device__ __noinline__ void put_limited(uint32_t from, uint8_t* dst, float inv, bool mine) {
#pragma unroll 1
        for (int x = 0; x < D; x += 16) {
            float o[16];
            tmem_ld16(from + x, o);
            tmem_wait_ld();
            if (!mine) continue;
#pragma unroll
            for (int y = 0; y < 16; ++y) reinterpret_cast<FiniteHalf*>(dst)[x + y] = from_float<FiniteHalf>(o[y] * inv);
        }
    }
    // What mend_values took out, for a row that sees the keys up to `last`.
    static __device__ __noinline__ void unmend(void* row, bool direct, int last, const PromptFix* fix) {
        using E = typename KV::T;
#pragma unroll 1
        for (int d = 0; d < D; ++d) {
            const bool nan = last >= fix->first[0][d], up = last >= fix->first[1][d], down = last >= fix->first[2][d];
            if (!(nan || up || down)) continue;
            float x = direct ? to_float(static_cast<E*>(row)[d]) : static_cast<float*>(row)[d];
            if (nan) x = NAN;
            if (up) x += INFINITY;
            if (down) x -= INFINITY;
            if (direct) static_cast<E*>(row)[d] = from_float<E>(x);
            else static_cast<float*>(row)[d] = x;
        }
    }
    static __device__ void write_out(const PromptParams& p, PromptBars* b, const PromptItem* items, const PromptFix* fix,
                                     const float2* rows) {
        const int r = threadIdx.x & (PT_M - 1), lane = threadIdx.x & 31;
        const uint32_t lanes = static_cast<uint32_t>(r & ~31) << 16;
        const int tok = r / p.G, head = r - tok * p.G;
        // rows are 128 or 256 bytes: all of them lie as out itself does
        const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
        uint32_t n[2] = {0, 0};
        for (int turn = 0;; ++turn) {
            const int is = turn % PT_ITEMS;
            if (!__all_sync(0xffffffffu, wait_item(p, &b->i_full[is], (turn / PT_ITEMS) & 1u))) return;
            const PromptItem it = items[is];
            if (!it.live) return;
            const bool direct = !SHARED && it.place < 0;
#pragma unroll 1
            for (int q = 0; q < 2; ++q) {
                const uint32_t to = b->tmem + lanes + Lay::OCOL + q * D;
                const bool mine = tok < p.tokens && q * p.tokens + tok < it.ntok &&
                                  (!SHARED || prompt_member(p, it.row0 + q * p.tokens + tok, it.idx));
                const int last = p.causal ? it.pos0 + q * p.tokens + tok : it.L - 1;    // the row's last key
                const bool any = it.e[q] > it.t0;
                const size_t row = static_cast<size_t>(it.row0 + q * p.tokens + tok) * p.Hq + it.h * p.G + head;
                const size_t part = SHARED ? row * it.ranges + it.place : (static_cast<size_t>(direct ? 0 : it.place) * 2 + q) * PT_M + r;
                uint8_t* dst = direct ? static_cast<uint8_t*>(p.out) + row * D * 2 : reinterpret_cast<uint8_t*>(p.part_acc + part * D);
                if (!any) {                                // no keys: zeros, or an empty partial
                    const uint32_t w[8] = {};
                    if (mine && direct) {
#pragma unroll
                        for (int x = 0; x < D; x += 16) put32(dst + x * 2, w, wide);
                    }
                    if (mine && !direct) p.part_ml[part] = make_float2(-INFINITY, 0.f);
                    continue;
                }
                const uint32_t phase = n[q]++ & 1u;
                if (!__all_sync(0xffffffffu, wait_item(p, &b->l_full[is][q], (turn / PT_ITEMS) & 1u) && wait_item(p, &b->o_full[q], phase))) return;
                tc05_fence_after();
                const float2 ml = rows[(is * 2 + q) * PT_M + r];
                const float inv = !direct ? 1.f : ml.y != 0.f ? 1.f / ml.y : 0.f;
                const bool fixed = *reinterpret_cast<const volatile int*>(&fix[is].any);
                if (mine && !direct) p.part_ml[part] = ml;
                float top = 0.f;
#pragma unroll 1
                for (int x = 0; x < D; x += 32) {
                    float o[32];
                    tmem_ld32(to + x, o);
                    tmem_wait_ld();
                    if (!mine) continue;
                    uint32_t w[8];
                    if (direct) {
                        if constexpr (!BF16) {
#pragma unroll
                            for (int y = 0; y < 32; y += 2) top = max3(top, fabsf(o[y]), fabsf(o[y + 1]));
                        }
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
#pragma unroll
                            for (int d = 0; d < 8; ++d) w[d] = pack2(o[16 * y + 2 * d] * inv, o[16 * y + 2 * d + 1] * inv, BF16);
                            put32(dst + x * 2 + y * 32, w, wide);
                        }
                    } else {
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
#pragma unroll
                            for (int d = 0; d < 8; ++d) w[d] = __float_as_uint(o[8 * y + d]);
                            put32(dst + x * 4 + y * 32, w, true);     // (the workspace is 256-byte aligned)
                        }
                    }
                }
                if (!BF16 && __any_sync(0xffffffffu, direct && top * inv > 65504.f)) put_limited(to, dst, inv, mine);
                if (fixed && mine) unmend(dst, direct, last, fix + is);
                tc05_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&b->o_empty[q]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&b->i_empty[is]);
        }
    }
};

// Shared mode: what each sequence has behind its group's prefix, for the decode
// kernel; -1 tokens for a sequence whose length does not fit.
__device__ __forceinline__ void write_tails(const PromptParams& p) {
    for (int i = blockIdx.x * PT_THREADS + threadIdx.x; i < p.total_q; i += gridDim.x * PT_THREADS) {
        const int g = prompt_seq_of(p, i);
        int P = 0, least = 0;
        // (a group whose entries leave the batch has no say on its sequences)
        if (g >= 0 && __ldg(p.q_start + g) >= 0 && __ldg(p.q_start + g + 1) <= p.total_q) {
            P = prompt_seq(p, g, false).L;
            least = group_prefix(p, g);
        }
        const int L = __ldg(p.lens + i);
        const bool ok = L >= max(P, least) && L <= p.MB * p.bs;
        p.tail_lens[i] = ok ? L - P : -1;
        p.tail_blk[i] = P / p.bs;
    }
}

template <class KV, int D, bool PAGED, bool SHARED>
__global__ void __launch_bounds__(PT_THREADS, 1)
prompt_kernel(const __grid_constant__ PromptParams p, const __grid_constant__ CUtensorMap tq,
              const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv) {
    using K = PromptKernel<KV, D, PAGED, SHARED>;
    using Lay = PromptLayout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(base + Lay::FULL);
    uint64_t* empty = reinterpret_cast<uint64_t*>(base + Lay::EMPTY);
    PromptBars* b = reinterpret_cast<PromptBars*>(base + Lay::BARS);
    PromptItem* items = reinterpret_cast<PromptItem*>(base + Lay::ITEM);
    PromptFix* fix = reinterpret_cast<PromptFix*>(base + Lay::FIX);
    uint4* bad = reinterpret_cast<uint4*>(base + Lay::BAD);
    float2* rows = reinterpret_cast<float2*>(base + Lay::ROWS);
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
            mbar_init(&b->o_empty[q], 4);
            for (int x = 0; x < PT_ITEMS; ++x) mbar_init(&b->l_full[x][q], 4);
        }
        for (int s = 0; s < PT_ITEMS; ++s) {
            mbar_init(&b->i_full[s], 1);
            mbar_init(&b->i_empty[s], 15);                 // all warps but the scheduler; of the MMA warp one thread
        }
        mbar_init(&b->v_there, 1);
        mbar_init(&b->v_fit, 1);
        mbar_init(&b->fin, 1);
        b->any_bad = 0;
        for (int x = 0; x < PT_BAD; ++x) bad[x] = make_uint4(0, 0, 0, 0);
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
    if constexpr (SHARED) write_tails(p);
    if (warp >= 8) {
        regs_down<PT_REGS_FEW>();
        if (warp == 8) {
            if (elect_one()) K::mma(p, base, full, empty, b, items);
        } else if (warp == 9) {
            K::producer(p, base, full, empty, b, items, bad, &tq, &tk, &tv);
        } else if (warp == 10) {
            K::schedule(p, b, items, fix, reinterpret_cast<int4*>(base + Lay::KNOWN));
        } else if (warp == 11) {
            K::mend(p, base, full, b, items, fix);
        } else {
            K::write_out(p, b, items, fix, rows);
        }
    } else {
        regs_up<PT_REGS>();
        K::softmax(p, warp >> 2, b, items, bad, rows);
    }
    tc05_fence_before();
    __syncthreads();
    tc05_fence_after();
    __syncwarp();
    if (warp == 8) tmem_dealloc<Lay::TCOLS>(b->tmem);
}

// ---------------------------------------------------------------------------
// merge of the ranges of keys: out = sum_k 2^(r_k - M) O_k / sum_k 2^(r_k - M) l_k
// One CTA per 32 rows of a cut item, one warp per row at a time.
// ---------------------------------------------------------------------------
constexpr int PT_MERGE_WARPS = 8, PT_MERGE_ROWS = 32;

// Spans that cut item i < grid has part in, by the launch's entry n and the item's own; 0 where
// there is no such item, and for entries that cannot be one: behind a wait that ran out they
// are whatever the workspace held, and nothing outside the call's buffers may follow from them.
__host__ __device__ inline int cut_parts(const PromptParams& p, int i, int4 n, int4 item) {
    if (i >= n.y || n.x < 2 || n.x > 32 || n.z < 1 || n.z >= n.x) return 0;
    const int parts = ((i + 1) * n.x + n.z - 1) / n.z - i * n.x / n.z;      // at most n.x: an item has n.x / n.z of them
    const bool fits = item.x >= 0 && item.y >= 1 && item.y <= 2 * p.tokens && item.x <= p.total_q - item.y &&
                      item.z >= 0 && item.z < p.Hkv && item.w >= 0 && item.w <= 2 * p.grid - parts;
    return fits ? parts : 0;
}

template <class KV, int D>
__global__ void __launch_bounds__(32 * PT_MERGE_WARPS)
prompt_merge_kernel(const __grid_constant__ PromptParams p) {
    constexpr int DPL = D / 32, PER = 2 * PT_M / PT_MERGE_ROWS;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dependency_wait();
    const int i = blockIdx.x / PER;
    const int4 n = p.cut[0], item = p.cut[1 + i];          // (first row, tokens, head, place)
    const int parts = cut_parts(p, i, n, item);
    if (parts == 0) return;
    for (int y = warp; y < PT_MERGE_ROWS; y += PT_MERGE_WARPS) {
        const int x = (blockIdx.x % PER) * PT_MERGE_ROWS + y, q = x / PT_M, r = x % PT_M;
        const int tok = r / p.G;
        if (tok >= p.tokens || q * p.tokens + tok >= item.y) continue;
        const size_t at = (static_cast<size_t>(item.w) * 2 + q) * PT_M + r;
        const float2 ml = lane < parts ? p.part_ml[at + static_cast<size_t>(lane) * 2 * PT_M] : make_float2(-INFINITY, 0.f);
        float M = ml.x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        const float e = ml.y != 0.f ? exp2f(ml.x - (M > -INFINITY ? M : 0.f)) : 0.f;
        float den = ml.y != 0.f ? e * ml.y : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
        const uint32_t some = __ballot_sync(0xffffffffu, ml.y != 0.f);
        float num[DPL];
#pragma unroll
        for (int d = 0; d < DPL; ++d) num[d] = 0.f;
#pragma unroll 4
        for (int k = 0; k < parts; ++k) {
            const float f = __shfl_sync(0xffffffffu, e, k);
            if (!((some >> k) & 1u)) continue;
#pragma unroll
            for (int d = 0; d < DPL; ++d)
                num[d] = fmaf(f, p.part_acc[(at + static_cast<size_t>(k) * 2 * PT_M) * D + lane * DPL + d], num[d]);
        }
        const float inv = den != 0.f ? 1.f / den : 0.f;
        using OutT = std::conditional_t<KV::code == PA_F16, FiniteHalf, typename KV::T>;
        OutT* o = static_cast<OutT*>(p.out) +
                  (static_cast<size_t>(item.x + q * p.tokens + tok) * p.Hq + item.z * p.G + r - tok * p.G) * D + lane * DPL;
#pragma unroll
        for (int d = 0; d < DPL; ++d) o[d] = from_float<OutT>(num[d] * inv);
    }
}

}  // namespace pa
