// pa_decode_int4.cu -- attention over 4-bit pools (pa_decode, pa_attention and
// pa_decode_weights with PA_INT4).
//
// With K_t = low_t + step_t c_t (c the 4-bit codes of a row), for a query row q
//   <q, K_t> = step_t <q, c_t> + low_t sum(q)
//   sum_t p_t V_t = sum_t (p_t step_t) c_t + sum_t p_t low_t,
// so the codes enter the matrix products as they are and the two numbers of a
// row are applied to scores and probabilities.  An f16 number whose bits are
// a small integer n is n * 2^-24 (a subnormal, or the first binade, up to
// n = 2047): a mask turns packed codes into f16 pairs worth c * 2^-24 (low
// nibble of a byte) or 16 c * 2^-24 (high nibble), with no conversion, and the
// powers of two are taken out of the sums.
//
// The second product sums thousands of tokens in f32, and all codes are
// positive: its sum would grow with the number of tokens, while the output is
// what is left of it after low's part is taken off, so that every rounding of
// the accumulator weighs the more the longer the sequence is (0.0029 relative
// error at 131072 tokens, against 0.0017 of the bf16 output itself).  So the
// sum of 8 times the weights is formed beside it, by one more MMA per 16 tokens,
// and taken off every four chunks: the sums are then over (c - 8) step, and
// low + 8 step takes the place of low.
//
// Both products are transposed: S^T = K Q^T with 16 tokens and O^T = V^T P^T
// with 16 dimensions as the M rows of mma.sync m16n8k16 and 8 query rows as N,
// so a GQA group of up to 8 heads fills the tile.  head_dim is summed in an
// order that lets a lane read 16 bytes of a key at once (and the query rows
// are laid out to match); P^T goes from the accumulator layout of S^T to the
// operand layout of the second product by an 8 x 8 transpose (movmatrix).
//
// Work split, partials and the merge are the paged decode kernel's: the chunks
// of all sequences form one stream, cut into ranges of equal cost for
// persistent CTAs; one warp fills a ring of stages (a block's codes of the
// CTA's heads are one span, one bulk copy; its (step, low) pairs go by 16-byte
// cp.async, as short spans), the other warps each own 8 or 16 query rows of one
// KV head.  TS such warps share a chunk of 32 TS tokens, 32 each, and join
// their results in shared memory at the end of a segment.
//
// Measured (us, one call, against the bytes alone at the copy rate): the
// 7B-like batch of 64 (28 heads on 4, f16) 51 (23), the same with 1-4 query
// tokens 132 (23), 1024 sequences of 20-2048 tokens 62 (26), 8 sequences of
// 32k-131k tokens 183 (120).  The copies alone, the arithmetic left out, take
// 39, 66, 46 and 134, of which about 12 are the plan, the pipeline's fill and
// the merge.  No unit is full (issue 39 to 51%, tensor pipe 16 to 27%): beyond
// the copies the latency of one chunk's chain sets the pace, masks, products,
// scale, exponent, transpose, products, with 3 consumer warps per scheduler
// (2 of 16 rows); and every key costs its masks, its two numbers and the
// softmax of 8 rows whatever the rows hold.  What was tried beside this form,
// at the times of then (181, 64 and 129): two CTAs per SM with 64 tokens per
// warp (171 on the long sequences, but 76 on the short ones, where 32 tokens
// then took 70); four CTAs of 96 registers (227 on the long ones, spills);
// separate barriers for keys and values (193); for 8 rows one 16-token tile at a
// time (190; for 16 rows that form is the faster one, 146 against 175 on 1-4
// query tokens, the registers holding one tile).
#include <algorithm>
#include <cmath>
#include <cuda.h>

#include "pa_common.h"
#include "pa_decode_int4.h"
#include "pa_decode_kernel.cuh"
#include "pa_int4.cuh"
#include "pa_kernels.h"

namespace pa {

constexpr int I4_WT = 32;                   // tokens of a chunk that one warp takes
constexpr int I4_WARPS = 4;                 // consumer warps of a CTA, where the rows allow
// 16-token tiles that a warp carries through the two products at once, and
// CTAs per SM: as many as the registers hold.
constexpr int i4_tiles(int nqt) { return nqt == 1 ? 2 : 1; }
constexpr int i4_ctas(int nqt) { return nqt == 1 ? 3 : 2; }
constexpr int I4_MAX_STAGES = 8;
constexpr int I4_NQ = 2;                    // query ring slots
// log2 of how far above a row's reference its largest product may lie, and of
// where it lies when the reference has just moved: below 2^15, within f16, and
// few moves (8 apart, as of a softmax's reference)
constexpr float I4_ROOM = 14.f, I4_LIFT = 6.f;

struct I4Head {
    int tok0, slot, qrow0, qpos0, qn, qslot;
    uint32_t flags;                         // SEG_* bits, QLOAD, DIRECT, GAP
};
struct I4Desc {
    I4Head h;
    uint32_t vmask[I4_WARPS];               // tokens of the chunk that exist, 32 per warp
};

struct Int4Params {
    DecodeParams d;
    const uint8_t* k;
    const uint8_t* v;
    size_t block_bytes;
    uint32_t code_bytes, param_bytes;       // of one stage's K (or V)
    int RT;                                 // row tiles per KV head
    int TS;                                 // warps that share a chunk's tokens
    int nbox;                               // blocks of a chunk
    int bshift, rshift;                     // log2 of the block size, and of the rows that a block has in a chunk
    uint32_t join_off, frag_off;            // offsets of the join buffers and of the warps' query operands
};

// Bulk copy by 32-bit shared addresses.
__device__ __forceinline__ void bulk_load32(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 :: "r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

__device__ __forceinline__ void bulk_load32_hint(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar, uint64_t policy) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;"
                 :: "r"(dst), "l"(src), "r"(bytes), "r"(bar), "l"(policy) : "memory");
}
// 16-byte copy by the thread's own address, and this thread's arrival on `bar`
// once its copies so far have landed (counted in the barrier's 33 arrivals).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" :: "r"(bar) : "memory");
}

// ---------------------------------------------------------------------------
// producer: one warp; lane b copies block b of a chunk (or head b of a block
// that is longer than a chunk).
// ---------------------------------------------------------------------------
template <int D, bool WT>
__device__ __forceinline__ void int4_producer(const Int4Params& a, const Plan& pl, int hg, uint8_t* base,
                                              uint64_t* full, uint64_t* empty, uint64_t* qempty, I4Desc* descs) {
    const DecodeParams& p = a.d;
    const int lane = threadIdx.x & 31;
    const int S = p.stages, maxL = p.MB * p.bs, CT = p.ct;
    uint64_t policy = 0;
    if constexpr (WT) policy = l2_evict_first();
    int lbase = pl.seq, lval = 0;
    auto load_lens = [&](int first) {
        lbase = first;
        const int ii = first + lane;
        lval = ii < p.B ? clamp_len(__ldg(p.seq_lens + ii), maxL) : 0;
    };
    auto len_of = [&](int ii) -> int {
        if (ii >= p.B) return 0;
        if (ii - lbase >= 32) load_lens(ii);
        return __shfl_sync(0xffffffffu, lval, ii - lbase);
    };
    auto load_win = [&](int seq, int wb, int nblk) -> int {
        const int idx = wb + lane;
        return (seq < p.B && idx < nblk) ? __ldg(p.block_tables + static_cast<size_t>(seq) * p.MB + idx) : -1;
    };
    load_lens(pl.seq);
    int i = pl.seq, Si = pl.S, Ui = pl.U;
    int j = pl.cs - Si;
    const int nb = a.nbox;
    int wbase = (j * CT) >> a.bshift;                 // 32 table entries from here on, the next 32 in flight
    int wval = load_win(i, wbase, p.MB);
    int L = len_of(i);
    int qrow = i, qn = 1;
    auto load_q_rows = [&]() {
        if (i < p.B) {
            if (!query_rows(p, i, qrow, qn) && lane == 0) raise_flag(p.err_flag, PA_ERRBIT_BAD_QUERY);
        } else {
            qrow = 0; qn = 0;
        }
    };
    load_q_rows();
    int nch = cdiv_i(L, CT), nbl = cdiv_i(L, p.bs);
    int nseq = 0, nbase = 0, nval = -1;
    auto prefetch_next = [&]() {
        if (wbase + 32 < nbl) {
            nseq = i; nbase = wbase + 32; nval = load_win(i, nbase, nbl);
        } else {
            nseq = i + 1; nbase = 0; nval = load_win(i + 1, 0, cdiv_i(len_of(i + 1), p.bs));
        }
    };
    prefetch_next();
    const int range = blockIdx.x / p.NHG;
    const uint32_t head_codes = static_cast<uint32_t>(p.bs) * (D / 2);       // a block's codes of one head
    const int rows = 1 << a.rshift;                                          // rows of a block in a chunk
    const bool whole = p.bs <= CT;
    const uint32_t box_codes = static_cast<uint32_t>(p.HPC * rows) * (D / 2);
    const uint32_t qrow_bytes = static_cast<uint32_t>(p.HPC * p.G) * D * 2u;
    // The copies of a chunk are on the path from a stage coming free to its
    // refill, and one warp issues those of four: what a chunk needs beyond its
    // block ids is worked out per sequence or per CTA.
    const uint8_t* kcs = a.k + static_cast<size_t>(hg * p.HPC) * head_codes;
    const uint8_t* vcs = a.v + static_cast<size_t>(hg * p.HPC) * head_codes;
    const uint32_t base32 = smem_u32(base), full32 = smem_u32(full);
    const uint32_t my_codes = lane * box_codes;
    const uint32_t v_at = a.code_bytes + a.param_bytes;
    // Parameters are small next to what a bulk copy costs to issue: each lane
    // copies those of four tokens of a head, 16 bytes, for K and for V.
    const int prow = lane * 4, pbox = prow / (p.HPC * rows), phead = (prow >> a.rshift) % p.HPC;
    const bool pmine = prow < p.HPC * CT;
    const uint32_t my_params = a.code_bytes + prow * 4u;
    const size_t to_params = static_cast<size_t>(p.Hkv - hg * p.HPC) * head_codes +
                             static_cast<size_t>((hg * p.HPC + phead) * p.bs + (prow & (rows - 1))) * 4u;
    int issued = 0, qcount = 0, slot = 0, qs = 0;
    uint32_t round = 0, qround = 0;
    int jp = j, ju = 0;
    if (p.PC > 0) { ju = j / p.PC; jp = j - ju * p.PC; }
    bool ok = true;
    bool direct = (p.PC == 0 || nch <= p.PC) && Si >= pl.cs && Si + nch <= pl.ce;
    for (int k = pl.cs; k < pl.ce; ++k) {
        if (j >= nch) {
            do {
                Si += nch; Ui += n_units(L, p.PC, p.ct); ++i;
                L = len_of(i);
                load_q_rows();
                nch = cdiv_i(L, CT); nbl = cdiv_i(L, p.bs);
                j = 0; jp = 0; ju = 0;
                wbase = 0;
                wval = (nseq == i && nbase == 0) ? nval : load_win(i, 0, nbl);
                prefetch_next();
            } while (j >= nch);
            direct = (p.PC == 0 || nch <= p.PC) && Si >= pl.cs && Si + nch <= pl.ce;
        }
        const int tok0 = j * CT, b0 = tok0 >> a.bshift;
        if (b0 + nb - 1 >= wbase + 32) {
            if (nseq == i && nbase <= b0 && b0 + nb - 1 < nbase + 32) {
                wbase = nbase; wval = nval;
            } else {
                wbase = b0; wval = load_win(i, wbase, nbl);
            }
            prefetch_next();
        }
        const int ntok = min(CT, L - tok0);
        // lane b < nb: block b of the chunk
        const int id = __shfl_sync(0xffffffffu, wval, min(b0 + lane - wbase, 31));
        const uint32_t used = (1u << ((ntok + rows - 1) >> a.rshift)) - 1u;       // blocks with a token (at most 16)
        const bool good = ((used >> lane) & 1u) && static_cast<unsigned>(id) < static_cast<unsigned>(p.NB);
        const uint32_t goods = __ballot_sync(0xffffffffu, good);
        if (goods != used && lane == 0) raise_flag(p.err_flag, PA_ERRBIT_BAD_BLOCK);
        const bool seg_start = (k == pl.cs) || (jp == 0);
        const bool qload = seg_start && (k == pl.cs || j == 0);
        ok = issued < S || mbar_wait_bounded(&empty[slot], (round - 1) & 1u);
        if (qload && qcount >= I4_NQ) ok = mbar_wait_bounded(&qempty[qs], (qround - 1) & 1u) && ok;
        if (!__all_sync(0xffffffffu, ok)) {
            if (lane == 0) raise_flag(p.err_flag, PA_ERRBIT_WAIT_TIMEOUT);
            break;
        }
        if (lane == 0) {
            const bool part_end = p.PC > 0 && jp == p.PC - 1;
            uint32_t flags = 0;
            if (seg_start) flags |= SEG_START;
            if (qload) flags |= QLOAD;
            if (k == pl.ce - 1 || j == nch - 1 || part_end) flags |= SEG_END;
            if (k == pl.ce - 1 && part_end && j + 1 < nch) flags |= GAP;
            if (direct) flags |= DIRECT;
            I4Head d;
            d.tok0 = tok0; d.flags = flags; d.qn = qn;
            d.slot = range + Ui + ju;
            d.qslot = qload ? qs : (qs == 0 ? I4_NQ - 1 : qs - 1);
            d.qrow0 = qrow;
            d.qpos0 = L - qn;
            descs[slot].h = d;
            if (ntok == CT && goods == used) {
                for (int w = 0; w < CT / 32; ++w) descs[slot].vmask[w] = 0xffffffffu;
            } else {
                // tokens that exist and whose block is in the pool
                for (int w = 0; w < CT / 32; ++w) {
                    const int n = ntok - 32 * w;
                    uint32_t m = n >= 32 ? 0xffffffffu : n > 0 ? (1u << n) - 1u : 0u;
                    for (int t = 0; t < 32; t += 8)
                        if (!((goods >> ((32 * w + t) >> a.rshift)) & 1u)) m &= ~(0xffu << t);
                    descs[slot].vmask[w] = m;
                }
            }
            mbar_arrive_expect_tx(&full[slot], __popc(goods) * 2u * box_codes +
                                                   (qload ? static_cast<uint32_t>(qn) * qrow_bytes : 0u));
        }
        __syncwarp();
        const uint32_t stage = base32 + slot * p.stage_bytes, bar = full32 + slot * 8u;
        const int pid = __shfl_sync(0xffffffffu, id, pbox);
        if (pmine && ((goods >> pbox) & 1u)) {
            const size_t at = static_cast<size_t>(static_cast<unsigned>(pid)) * a.block_bytes + to_params +
                              (whole ? 0u : static_cast<uint32_t>(tok0 & (p.bs - 1)) * 4u);
            cp_async16(stage + my_params, kcs + at);
            cp_async16(stage + v_at + my_params, vcs + at);
        }
        cp_async_arrive(bar);
        if (whole) {
            if (good) {
                const size_t blk = static_cast<size_t>(static_cast<unsigned>(id)) * a.block_bytes;
                if constexpr (WT) {            // K and V pass once; the scores are read again
                    bulk_load32_hint(stage + my_codes, kcs + blk, box_codes, bar, policy);
                    bulk_load32_hint(stage + v_at + my_codes, vcs + blk, box_codes, bar, policy);
                } else {
                    bulk_load32(stage + my_codes, kcs + blk, box_codes, bar);
                    bulk_load32(stage + v_at + my_codes, vcs + blk, box_codes, bar);
                }
            }
        } else if (goods & 1u) {
            // a chunk is part of one block: a span per head
            const size_t blk = static_cast<size_t>(__shfl_sync(0xffffffffu, id, 0)) * a.block_bytes +
                               static_cast<size_t>(tok0 & (p.bs - 1)) * (D / 2);
            const uint32_t cb = CT * (D / 2);
            for (int h = lane; h < p.HPC; h += 32) {
                bulk_load32(stage + h * cb, kcs + blk + static_cast<size_t>(h) * head_codes, cb, bar);
                bulk_load32(stage + v_at + h * cb, vcs + blk + static_cast<size_t>(h) * head_codes, cb, bar);
            }
        }
        if (qload) {
            // the heads' rows of one query token are one span
            uint8_t* qd = base + p.q_off + qs * p.q_slot_bytes;
            for (int t = lane; t < qn; t += 32)
                bulk_load(qd + t * qrow_bytes,
                          static_cast<const uint8_t*>(p.q) + (static_cast<size_t>(qrow + t) * p.Hq + hg * p.HPC * p.G) * D * 2u,
                          qrow_bytes, &full[slot]);
            ++qcount;
            if (++qs == I4_NQ) { qs = 0; ++qround; }
        }
        ++issued;
        if (++slot == S) { slot = 0; ++round; }
        ++j;
        if (++jp == p.PC) { jp = 0; ++ju; }
    }
    // every copy lands before the CTA exits
    if (lane == 0) {
        for (int st = max(0, issued - S); st < issued; ++st) {
            if (!mbar_wait_bounded(&full[st % S], (st / S) & 1u)) {
                raise_flag(p.err_flag, PA_ERRBIT_WAIT_TIMEOUT);
                break;
            }
        }
    }
}

// Loads from shared memory by 32-bit address: the stage's address is computed
// from a rounded-up base, behind which the compiler would not see the address
// space and load through 64-bit generic addresses.
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t r;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a));
    return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 r;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
    return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
    return r;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" :: "r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ float2 lds_params(uint32_t a) {        // (step, low)
    const uint32_t r = lds32(a);
    return __half22float2(*reinterpret_cast<const __half2*>(&r));
}
// D = A B, f16 operands: mma_16816 with a zero accumulator.
__device__ __forceinline__ void mma_16816_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// Shuffle-reduce over the 8 lanes of equal lane % 4.
__device__ __forceinline__ float max_g4(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
__device__ __forceinline__ float sum_g4(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    x += __shfl_xor_sync(0xffffffffu, x, 8);
    return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

// The exponent of a row's step, whole: that of the smallest f16 for a step of
// 0 (its row still weighs by its low), and of the largest for what is none.
__device__ __forceinline__ float step_log2(float step) {
    const int e = static_cast<int>((__float_as_uint(step) >> 23) & 255u) - 127;
    return static_cast<float>(min(max(e, -24), 15));
}

template <typename T>
__device__ __forceinline__ uint32_t pack_out(float a, float b) {
    return pack2(a, b, std::is_same<T, __nv_bfloat16>::value);
}

// ---------------------------------------------------------------------------
// consumer: warp w owns NQT tiles of 8 query rows of one KV head.
// The products p step enter the second product rounded to f16 (11 bits),
// whatever the output's type: each rounding meets a c - 8, so the output's
// error is that of rounding p itself while the product is a normal f16.  The
// exponent's reference m is therefore one of the products, not of the scores:
// a row's largest s + log2(step) lies within [m + 6, m + 14], its largest
// product within [2^6, 2^15), and those down to 2^-20 to 2^-29 of it keep all
// 11 bits.  (References of scores and steps apart let one row with a large step
// and no weight push the others' products into subnormals: outputs of order one
// over 32768 keys were off by 0.07 to 0.17 with a step 8000 times the others'.
// Neither form is faster.)  Weights alone are then at most 2^38 and summed in
// f32.  WT: pa_decode_weights, the scores and (m, l) are kept.
// ---------------------------------------------------------------------------
template <class QT, int D, int NQT, bool WT>
__device__ __forceinline__ void int4_consumer(const Int4Params& a, const Plan& pl, int hg, int w, uint8_t* base,
                                              uint64_t* full, uint64_t* empty, uint64_t* qempty, uint64_t* joined,
                                              const I4Desc* descs) {
    using T = typename QT::T;
    constexpr int MT = i4_tiles(NQT);             // 16-token tiles at once
    constexpr int SUBS = I4_WT / (16 * MT);       // times that a chunk takes
    constexpr int KW = D / 32;                    // 32-bit code words of a key that a lane reads
    constexpr int OT = D / 16;                    // 16-dimension output tiles
    constexpr float UNIT = 16777216.f;            // 2^24: what an f16 with the bits of n is short of n
    const DecodeParams& p = a.d;
    const int lane = threadIdx.x & 31, g4 = lane >> 2, t4 = lane & 3;
    const int tile = w / a.TS, ts = w - tile * a.TS;      // (KV head, row tile), and its share of the tokens
    const int hl = tile / a.RT, rt = tile - hl * a.RT;
    const int S = p.stages;
    const int rows_total = p.QL * p.G;
    const uint32_t base32 = smem_u32(base);
    // Row r of a tile of 8 tokens is token tau(r) = r ^ (r / 2 % 2), on both
    // sides of P: the four tokens that a quarter of the V loads reads are then
    // two even and two odd 64-byte rows.
    const int tk = g4 ^ ((g4 >> 1) & 1);
    const int tv0 = (2 * t4) ^ (t4 & 1), tv1 = (2 * t4 + 1) ^ (t4 & 1);
    // A stage is K codes, K parameters, V codes, V parameters, each [block]
    // [head][row]; a block has 8 rows or a multiple.  Bytes from its start to
    // the codes of the first of each 8 tokens of this head, and to the
    // parameters of the lane's token of them.  With 8 rows per warp HPC * TS is
    // 4 and the distances inside a stage are constants of the code.
    const uint32_t POFF = NQT == 1 ? I4_WARPS * I4_WT * (D / 2) : a.code_bytes;
    const uint32_t VOFF = NQT == 1 ? I4_WARPS * I4_WT * (D / 2 + 4) : a.code_bytes + a.param_bytes;
    uint32_t c8[I4_WT / 8], p8[I4_WT / 8];
#pragma unroll
    for (int x = 0; x < I4_WT / 8; ++x) {
        const uint32_t t = I4_WT * ts + 8 * x, b = t >> a.rshift;
        const uint32_t row = ((b * p.HPC + hl) << a.rshift) + (t - (b << a.rshift));
        c8[x] = row * (D / 2);
        p8[x] = (row + tk) * 4u;
    }
    const uint32_t ok = tk * (D / 2) + t4 * (D / 8);                   // the lane's part of a key row
    const uint32_t ov0 = tv0 * (D / 2) + g4 * (D / 16), ov1 = tv1 * (D / 2) + g4 * (D / 16);   // and of two value rows

    float acc[OT][NQT][4];
    float eight[NQT][4];                          // 8 * (sum of the weights) since it was last taken off acc
    // The warp's query operand, [tile][word][lane] 16 bytes, kept in shared
    // memory: the registers it would take buy another CTA per SM.
    const uint32_t qf = base32 + a.frag_off + static_cast<uint32_t>(w * NQT * KW * 512) + lane * 16u;
    // rows 2 t4 and 2 t4 + 1 of each tile: reference of the exponent, sum of the
    // weights, sum of weight * (low + 8 step); the last two over the lane's tokens
    float m[NQT][2], l[NQT][2], c0[NQT][2];
    float sq[NQT][2];                             // sum of the query row, times the score scale
    float unit_qk = 0.f;                          // score of one unit of the codes' dot product
    int jt[NQT][2], lim[NQT][2];
    // the lane's scores of the next chunk, of its first row
    float* sdst = nullptr;
    int ct_log2 = 5;
    if constexpr (WT) {
        while ((1 << ct_log2) < p.ct) ++ct_log2;
        sdst = score_row(p, pl.cs, (hg * p.HPC + hl) * p.G + rt * NQT * 8 + 2 * t4) + I4_WT * ts + tk;
    }
    int in_rows = 0, joins = 0;
#pragma unroll
    for (int n = 0; n < NQT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int R = (rt * NQT + n) * 8 + 2 * t4 + e;
            jt[n][e] = R / p.G;
            if (R < rows_total) in_rows |= 1 << (2 * n + e);
            lim[n][e] = INT_MAX;
            sq[n][e] = 0.f;
        }

    for (int st = 0, k = pl.cs; k < pl.ce; ++k, ++st) {
        const int slot = st % S;
        if (!mbar_wait_bounded(&full[slot], (st / S) & 1u)) {
            if (lane == 0) raise_flag(p.err_flag, PA_ERRBIT_WAIT_TIMEOUT);
            return;
        }
        const I4Head d = descs[slot].h;
        const uint32_t vmask = descs[slot].vmask[ts];
        const uint32_t stage = base32 + slot * p.stage_bytes;
        if (d.flags & SEG_START) {
            if (d.flags & QLOAD) {
                // The B operand of this lane: row g4 of each tile, dimensions
                // [D/4 * t4, D/4 * (t4 + 1)) in the codes' order.  For bf16 rows a
                // power of two puts the warp's largest element into [2^13, 2^14):
                // their 8 bits fit an f16, except in elements below 2^-28 of the
                // largest, which are rounded to a multiple of 2^-38 of it.
                const uint8_t* qb = base + p.q_off + d.qslot * p.q_slot_bytes;
                uint32_t raw[NQT][KW][4];
#pragma unroll
                for (int n = 0; n < NQT; ++n) {
                    const int R = (rt * NQT + n) * 8 + g4, jj = R / p.G;
                    const bool on = R < rows_total && jj < d.qn;
                    const uint4* src = reinterpret_cast<const uint4*>(
                        qb + (static_cast<size_t>(jj * p.HPC + hl) * p.G + (R - jj * p.G)) * D * 2 + t4 * (D / 2));
#pragma unroll
                    for (int x = 0; x < KW; ++x) {
                        const uint4 r = on ? src[x] : make_uint4(0, 0, 0, 0);
                        raw[n][x][0] = r.x; raw[n][x][1] = r.y; raw[n][x][2] = r.z; raw[n][x][3] = r.w;
                    }
                }
                auto pair = [&](uint32_t x) -> float2 {
                    if constexpr (QT::code == PA_BF16) return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x));
                    else return __half22float2(*reinterpret_cast<const __half2*>(&x));
                };
                float f = 1.f;
                if constexpr (QT::code == PA_BF16) {
                    float mx = 0.f;
#pragma unroll
                    for (int n = 0; n < NQT; ++n)
#pragma unroll
                        for (int x = 0; x < KW; ++x)
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const float2 v = pair(raw[n][x][y]);
                                mx = fmaxf(mx, fmaxf(fabsf(v.x), fabsf(v.y)));
                            }
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                    // 2^(13 - exponent of the largest), from its exponent bits
                    const int ex = static_cast<int>(__float_as_uint(mx) >> 23) - 127;
                    if (mx > 0.f && ex < 128) f = __uint_as_float(static_cast<uint32_t>(min(13 - ex, 126) + 127) << 23);
                }
                const float qk = p.qk_scale / f;
                unit_qk = qk * UNIT;
#pragma unroll
                for (int n = 0; n < NQT; ++n) {
                    float s = 0.f;
#pragma unroll
                    for (int x = 0; x < KW; ++x) {
                        // words hold dims (0,1) (2,3) (4,5) (6,7): pairs (0,4) (2,6) (1,5) (3,7)
                        float2 v[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            v[y] = pair(raw[n][x][y]);
                            s += v[y].x + v[y].y;
                        }
                        sts128(qf + (n * KW + x) * 512u,
                               make_uint4(f32x2_to_f16x2(v[0].x * f, v[2].x * f), f32x2_to_f16x2(v[1].x * f, v[3].x * f),
                                          f32x2_to_f16x2(v[0].y * f, v[2].y * f), f32x2_to_f16x2(v[1].y * f, v[3].y * f)));
                    }
                    s += __shfl_xor_sync(0xffffffffu, s, 1);
                    s += __shfl_xor_sync(0xffffffffu, s, 2);
#pragma unroll
                    for (int e = 0; e < 2; ++e) sq[n][e] = __shfl_sync(0xffffffffu, s, (2 * t4 + e) * 4) * p.qk_scale;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&qempty[d.qslot]);
            }
#pragma unroll
            for (int n = 0; n < NQT; ++n) {
#pragma unroll
                for (int o = 0; o < OT; ++o) acc[o][n][0] = acc[o][n][1] = acc[o][n][2] = acc[o][n][3] = 0.f;
                eight[n][0] = eight[n][1] = eight[n][2] = eight[n][3] = 0.f;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    m[n][e] = -INFINITY; l[n][e] = c0[n][e] = 0.f;
                    if (p.q_start) lim[n][e] = ((in_rows >> (2 * n + e)) & 1) && jt[n][e] < d.qn ? d.qpos0 + jt[n][e] : -1;
                }
            }
        }
#pragma unroll 1
        for (int sub = 0; sub < SUBS; ++sub) {
            uint32_t c[2 * MT], pr[2 * MT];
#pragma unroll
            for (int x = 0; x < 2 * MT; ++x) {
                c[x] = stage + (SUBS > 1 && sub ? c8[(2 * MT + x) % (I4_WT / 8)] : c8[x]);
                pr[x] = stage + (SUBS > 1 && sub ? p8[(2 * MT + x) % (I4_WT / 8)] : p8[x]);
            }
            const int tok0 = d.tok0 + I4_WT * ts + 16 * MT * sub;
            const uint32_t vm = vmask >> (16 * MT * sub);
            constexpr uint32_t ALL = MT == 2 ? 0xffffffffu : 0xffffu;
            const bool all = (vm & ALL) == ALL;
            // ---- S^T = K Q^T ----
            // The steps along head_dim run outside the tiles: each product then
            // has 2 MT accumulators (the low and the high nibbles' of each
            // tile), whose dependent MMAs are that far apart.
            float s[MT][NQT][4];
            {
                uint32_t ka[MT][KW], kb[MT][KW];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const uint32_t at = c[2 * mt] + ok, bt = c[2 * mt + 1] + ok;
                    if constexpr (KW == 4) {
                        const uint4 x = lds128(at), y = lds128(bt);
                        ka[mt][0] = x.x; ka[mt][1] = x.y; ka[mt][2] = x.z; ka[mt][3] = x.w;
                        kb[mt][0] = y.x; kb[mt][1] = y.y; kb[mt][2] = y.z; kb[mt][3] = y.w;
                    } else {
                        const uint2 x = lds64(at), y = lds64(bt);
                        ka[mt][0] = x.x; ka[mt][1] = x.y; kb[mt][0] = y.x; kb[mt][1] = y.y;
                    }
                }
                float hi[MT][NQT][4];
#pragma unroll
                for (int x = 0; x < KW; ++x) {
                    uint4 f[NQT];
#pragma unroll
                    for (int n = 0; n < NQT; ++n) f[n] = lds128(qf + (n * KW + x) * 512u);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        const uint32_t a8 = ka[mt][x] >> 8, b8 = kb[mt][x] >> 8;
                        const uint32_t A1[4] = {ka[mt][x] & 0x000f000fu, kb[mt][x] & 0x000f000fu, a8 & 0x000f000fu, b8 & 0x000f000fu};
                        const uint32_t A2[4] = {ka[mt][x] & 0x00f000f0u, kb[mt][x] & 0x00f000f0u, a8 & 0x00f000f0u, b8 & 0x00f000f0u};
#pragma unroll
                        for (int n = 0; n < NQT; ++n) {
                            if (x == 0) {
                                mma_16816_zero(s[mt][n], A1, f[n].x, f[n].y);
                                mma_16816_zero(hi[mt][n], A2, f[n].z, f[n].w);
                            } else {
                                mma_16816<false>(s[mt][n], A1, f[n].x, f[n].y);
                                mma_16816<false>(hi[mt][n], A2, f[n].z, f[n].w);
                            }
                        }
                    }
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const float2 p0 = lds_params(pr[2 * mt] + POFF), p1 = lds_params(pr[2 * mt + 1] + POFF);
                    const float s0 = p0.x * unit_qk, s1 = p1.x * unit_qk;
#pragma unroll
                    for (int n = 0; n < NQT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            s[mt][n][e] = fmaf(fmaf(hi[mt][n][e], 0.0625f, s[mt][n][e]), e < 2 ? s0 : s1, (e < 2 ? p0.y : p1.y) * sq[n][e & 1]);
                }
            }
            // tokens that do not exist, or lie behind a row's position
            if (!all || (p.q_start && tok0 + 16 * MT - 1 > d.qpos0)) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int n = 0; n < NQT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int t = 16 * mt + 8 * (e >> 1) + tk;
                            if (!((vm >> t) & 1u) || tok0 + t > lim[n][e & 1]) s[mt][n][e] = -INFINITY;
                        }
            }
            if constexpr (WT) {
                // rows are heads here; 8 lanes store 8 tokens of a head, one sector
#pragma unroll
                for (int n = 0; n < NQT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if ((in_rows >> (2 * n + e)) & 1) {
                            float* dst = sdst + (static_cast<uint32_t>(n * 8 + e) << ct_log2) + 16 * MT * sub;
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt) {
                                dst[16 * mt] = s[mt][n][e];
                                dst[16 * mt + 8] = s[mt][n][e + 2];
                            }
                        }
            }
            // ---- V parameters: step and low + 8 step of the lane's two tokens of each tile ----
            float vs[MT][2], vl[MT][2];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 v = lds_params(pr[2 * mt + e] + VOFF + POFF);
                    vs[mt][e] = v.x; vl[mt][e] = fmaf(8.f, v.x, v.y);
                }
            if (!all) {                               // the pool may hold NaN where no token is
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (!((vm >> (16 * mt + 8 * e + tk)) & 1u)) vs[mt][e] = vl[mt][e] = 0.f;
            }
            // ---- online softmax (log2 domain) ----
            // The reference of a row moves only when a product may pass it by 2^14
            // (the lane's largest score and largest step, of different tokens at
            // worst, say when to look): a chunk mostly needs no exchange between
            // lanes but one vote.
            float smax = 0.f;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) smax = max_nan(smax, max_nan(fabsf(vs[mt][0]), fabsf(vs[mt][1])));
            const float top = I4_ROOM - step_log2(smax);
            bool far = smax != smax;                  // a row of NaN
#pragma unroll
            for (int n = 0; n < NQT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) mx = fmaxf(mx, fmaxf(s[mt][n][e], s[mt][n][e + 2]));
                    far = far || mx > m[n][e] + top;
                }
            if (__any_sync(0xffffffffu, far)) {
                float ls[MT][2];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (vs[mt][e] != vs[mt][e]) {
                            // a row of NaN spoils the query rows that attend it, and
                            // no other: its products with a weight of 0 would
#pragma unroll
                            for (int n = 0; n < NQT; ++n)
#pragma unroll
                                for (int x = 0; x < 2; ++x)
                                    if (s[mt][n][2 * e + x] != -INFINITY) c0[n][x] = __int_as_float(0x7fffffff);
                            vs[mt][e] = vl[mt][e] = 0.f;
                        }
                        ls[mt][e] = step_log2(vs[mt][e]);
                    }
#pragma unroll
                for (int n = 0; n < NQT; ++n) {
                    float f[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float t = -INFINITY;
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) t = fmaxf(t, fmaxf(s[mt][n][e] + ls[mt][0], s[mt][n][e + 2] + ls[mt][1]));
                        t = max_g4(t);
                        f[e] = 1.f;
                        if (t > m[n][e] + I4_ROOM) {
                            f[e] = ex2_approx(m[n][e] - (t - I4_LIFT));
                            m[n][e] = t - I4_LIFT;
                            l[n][e] *= f[e];
                            c0[n][e] *= f[e];
                        }
                    }
#pragma unroll
                    for (int o = 0; o < OT; ++o) {
                        acc[o][n][0] *= f[0]; acc[o][n][1] *= f[1]; acc[o][n][2] *= f[0]; acc[o][n][3] *= f[1];
                    }
                    eight[n][0] *= f[0]; eight[n][1] *= f[1]; eight[n][2] *= f[0]; eight[n][3] *= f[1];
                }
            }
            uint32_t pf[MT][NQT][2];
#pragma unroll
            for (int n = 0; n < NQT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float mu = m[n][e] == -INFINITY ? 0.f : m[n][e];
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        s[mt][n][e] = ex2_approx(s[mt][n][e] - mu);
                        s[mt][n][e + 2] = ex2_approx(s[mt][n][e + 2] - mu);
                        l[n][e] += s[mt][n][e] + s[mt][n][e + 2];
                        c0[n][e] = fmaf(s[mt][n][e], vl[mt][0], fmaf(s[mt][n][e + 2], vl[mt][1], c0[n][e]));
                    }
                }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const float w0 = vs[mt][0], w1 = vs[mt][1];
#pragma unroll
                for (int n = 0; n < NQT; ++n) {
                    const float x0 = s[mt][n][0] * w0, x1 = s[mt][n][1] * w0, x2 = s[mt][n][2] * w1, x3 = s[mt][n][3] * w1;
                    const uint32_t h0 = f32x2_to_f16x2(x0, x1), h1 = f32x2_to_f16x2(x2, x3);
                    pf[mt][n][0] = movmatrix(h0);
                    pf[mt][n][1] = movmatrix(h1);
                }
            }
            // ---- O^T += V^T P^T ----
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                // k columns 2 t4, 2 t4 + 1 and 8 on: four tokens of D / 8 dimensions
                const uint32_t r[4] = {c[2 * mt] + ov0 + VOFF, c[2 * mt] + ov1 + VOFF, c[2 * mt + 1] + ov0 + VOFF,
                                       c[2 * mt + 1] + ov1 + VOFF};
                constexpr int VW = D / 64;            // code words of a value that a lane reads
                uint32_t v[4][VW];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    if constexpr (VW == 2) {
                        const uint2 y = lds64(r[x]);
                        v[x][0] = y.x; v[x][1] = y.y;
                    } else {
                        v[x][0] = lds32(r[x]);
                    }
                }
                // pairs of tokens: q[half][word * 2 + upper] holds 4 dimensions of two tokens
                uint32_t q[2][2 * VW], q8[2][2 * VW];
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int y = 0; y < VW; ++y) {
                        q[x][2 * y] = __byte_perm(v[2 * x][y], v[2 * x + 1][y], 0x5410);
                        q[x][2 * y + 1] = __byte_perm(v[2 * x][y], v[2 * x + 1][y], 0x7632);
                        q8[x][2 * y] = q[x][2 * y] >> 8;
                        q8[x][2 * y + 1] = q[x][2 * y + 1] >> 8;
                    }
                const uint32_t mid[4] = {0x00080008u, 0x00080008u, 0x00080008u, 0x00080008u};   // code 8
#pragma unroll
                for (int n = 0; n < NQT; ++n) mma_16816<false>(eight[n], mid, pf[mt][n][0], pf[mt][n][1]);
#pragma unroll
                for (int o = 0; o < OT; ++o) {
                    // head_dim 128: tile o has dimensions 16 g4 + o and 16 g4 + 8 + o (nibble o of both words);
                    // 64: 8 g4 + o and 8 g4 + 4 + o (nibbles o and o + 4 of the one word)
                    constexpr int step = VW == 2 ? 2 : 1;
                    const int ia = VW == 2 ? o / 4 : 0, ib = ia + step;
                    const int nib = VW == 2 ? o % 4 : o;
                    const uint32_t mask = (nib & 1) ? 0x00f000f0u : 0x000f000fu;
                    const uint32_t A[4] = {(nib < 2 ? q[0][ia] : q8[0][ia]) & mask, (nib < 2 ? q[0][ib] : q8[0][ib]) & mask,
                                           (nib < 2 ? q[1][ia] : q8[1][ia]) & mask, (nib < 2 ? q[1][ib] : q8[1][ib]) & mask};
#pragma unroll
                    for (int n = 0; n < NQT; ++n) {
                        mma_16816<false>(acc[o][n], A, pf[mt][n][0], pf[mt][n][1]);
                    }
                }
            }
        }
        if ((st & 3) == 3 || (d.flags & SEG_END)) {
#pragma unroll
            for (int n = 0; n < NQT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
#pragma unroll
                    for (int o = 0; o < OT; ++o) acc[o][n][e] = fmaf(eight[n][e], (o & 1) ? -16.f : -1.f, acc[o][n][e]);
                    eight[n][e] = 0.f;
                }
        }
        if constexpr (WT) sdst += static_cast<size_t>(p.Hq) << ct_log2;
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[slot]);
        if (d.flags & SEG_END) {
            const bool direct = (d.flags & DIRECT) != 0;
            // warps ts > 0 hand (m, l, values) of their tokens to warp ts = 0
            constexpr int JF = D / 8 + 2;                 // floats per lane, tile and row of the pair
            float* jb = reinterpret_cast<float*>(base + a.join_off) + static_cast<size_t>(tile * (a.TS - 1)) * NQT * 2 * JF * 32 + lane;
            uint64_t* jfull = joined + 2 * tile;
            uint64_t* jfree = jfull + 1;
            if (a.TS > 1) {
                if (ts > 0) {
                    if (joins > 0 && !mbar_wait_bounded(jfree, (joins - 1) & 1u)) {
                        if (lane == 0) raise_flag(p.err_flag, PA_ERRBIT_WAIT_TIMEOUT);
                        return;
                    }
                } else if (!mbar_wait_bounded(jfull, joins & 1u)) {
                    if (lane == 0) raise_flag(p.err_flag, PA_ERRBIT_WAIT_TIMEOUT);
                    return;
                }
                ++joins;
            }
#pragma unroll
            for (int n = 0; n < NQT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float lt = sum_g4(l[n][e]);
                    const float ct = sum_g4(c0[n][e]);
                    // the lane's D / 8 dimensions from D / 8 * g4 on, in order
                    float v[D / 8];
#pragma unroll
                    for (int o = 0; o < OT; ++o) {
                        constexpr float LOW = UNIT, HIGH = UNIT * 0.0625f;
                        const float u = (o & 1) ? HIGH : LOW;
                        v[o] = fmaf(acc[o][n][e], u, ct);
                        v[OT + o] = fmaf(acc[o][n][2 + e], u, ct);
                    }
                    if (ts > 0) {
                        float* b = jb + static_cast<size_t>(((ts - 1) * NQT + n) * 2 + e) * JF * 32;
                        b[0] = m[n][e];
                        b[32] = lt;
#pragma unroll
                        for (int x = 0; x < D / 8; ++x) b[(2 + x) * 32] = v[x];
                        continue;
                    }
                    float mr = m[n][e];
                    for (int x = 1; x < a.TS; ++x) {
                        const float* b = jb + static_cast<size_t>(((x - 1) * NQT + n) * 2 + e) * JF * 32;
                        const float m2 = b[0], mn = fmaxf(mr, m2);
                        const float mu = mn == -INFINITY ? 0.f : mn;
                        const float f1 = ex2_approx(mr - mu), f2 = ex2_approx(m2 - mu);
                        mr = mn;
                        lt = lt * f1 + b[32] * f2;
#pragma unroll
                        for (int y = 0; y < D / 8; ++y) v[y] = v[y] * f1 + b[(2 + y) * 32] * f2;
                    }
                    const bool on = ((in_rows >> (2 * n + e)) & 1) && jt[n][e] < d.qn && (direct || d.slot < p.max_slots);
                    if (!on) continue;
                    const int R = (rt * NQT + n) * 8 + 2 * t4 + e;
                    const int head = (hg * p.HPC + hl) * p.G + (R - jt[n][e] * p.G);
                    if constexpr (WT) {
                        if (direct && g4 == 0) p.lse[static_cast<size_t>(d.qrow0) * p.Hq + head] = make_float2(mr, lt);
                    }
                    if (direct) {
                        const float sc = lt == 0.f ? 0.f : 1.f / lt;
#pragma unroll
                        for (int x = 0; x < D / 8; ++x) {
                            v[x] *= sc;
                            if constexpr (QT::code == PA_F16) v[x] = limit_f16(v[x]);
                        }
                        uint4* o = reinterpret_cast<uint4*>(static_cast<T*>(p.out) +
                                                            (static_cast<size_t>(d.qrow0 + jt[n][e]) * p.Hq + head) * D + g4 * (D / 8));
#pragma unroll
                        for (int x = 0; x < D / 64; ++x)
                            o[x] = make_uint4(pack_out<T>(v[8 * x], v[8 * x + 1]), pack_out<T>(v[8 * x + 2], v[8 * x + 3]),
                                              pack_out<T>(v[8 * x + 4], v[8 * x + 5]), pack_out<T>(v[8 * x + 6], v[8 * x + 7]));
                    } else {
                        const size_t prow = (static_cast<size_t>(d.slot) * p.QL + jt[n][e]) * p.Hq + head;
                        float4* o = reinterpret_cast<float4*>(p.part_acc + prow * D + g4 * (D / 8));
#pragma unroll
                        for (int x = 0; x < D / 32; ++x) o[x] = make_float4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
                        if (g4 == 0) p.part_ml[prow] = make_float2(mr, lt);
                    }
                }
            if (a.TS > 1) {
                __syncwarp();
                if (lane == 0) mbar_arrive(ts > 0 ? jfull : jfree);
            }
            if (ts == 0 && (d.flags & GAP) && !direct && d.slot + 1 < p.max_slots) {
                // the slot that a range end on a partition end skips: an empty partial
                for (int r = 0; r < 8 * NQT; ++r) {
                    const int R = rt * NQT * 8 + r, jj = R / p.G;
                    if (R >= rows_total) break;
                    const size_t prow = (static_cast<size_t>(d.slot + 1) * p.QL + jj) * p.Hq + (hg * p.HPC + hl) * p.G + (R - jj * p.G);
                    for (int x = lane; x < D / 4; x += 32)
                        reinterpret_cast<float4*>(p.part_acc + prow * D)[x] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (lane == 0) p.part_ml[prow] = make_float2(-INFINITY, 0.f);
                }
            }
        }
    }
}

// How many ranges a call without partitions is cut into.  With fewer chunks
// than ranges some would be empty, and the merge would look for a sequence's
// partials range by range: 123 of the 134 us of a call on three sequences of 5k
// to 23k tokens and one KV head.  And a chunk costs a CTA about 0.7 us, a
// partial the merge about 0.11: a sequence of n chunks in k ranges, 0.7 n / k +
// 0.11 k, is best off with k = sqrt(6 n) of them, so few sequences take
// sequences * sqrt(6 chunks per sequence) ranges where the GPU has more.  One
// sequence of 9000 tokens, 8 heads: 25 us (48 with a range per chunk); those
// three: 23 (39); one of 131072, one KV head 39 (60), 8 heads 76 (74).
__device__ __forceinline__ int int4_ranges(const DecodeParams& p, int2* scratch) {
    int c = 0;
    for (int i = threadIdx.x; i < p.B; i += blockDim.x) c += cdiv_i(clamp_len(p.seq_lens[i], p.MB * p.bs), p.ct);
    c = __reduce_add_sync(0xffffffffu, c);
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5].x = c;
    __syncthreads();
    c = 0;
    for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) c += scratch[w].x;
    __syncthreads();                           // the plan writes there
    const int even = static_cast<int>(sqrtf(6.f * static_cast<float>(c) * static_cast<float>(p.B)));
    return min(p.NR, max(1, min(c, even)));
}

// MAXW: consumer warps at most, CTAS: CTAs per SM that the registers are
// limited for.
template <class QT, int D, int NQT, bool WT, int MAXW, int CTAS>
__global__ void __launch_bounds__((MAXW + 1) * 32, CTAS)
int4_decode_kernel(const __grid_constant__ Int4Params a) {
    extern __shared__ uint8_t smem_raw[];
    const DecodeParams& p = a.d;
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    uint64_t* full = reinterpret_cast<uint64_t*>(base + p.bar_off);
    uint64_t* empty = full + I4_MAX_STAGES;
    uint64_t* qempty = empty + I4_MAX_STAGES;
    uint64_t* joined = qempty + I4_NQ;                     // (full, free) of each tile's join buffer
    I4Desc* descs = reinterpret_cast<I4Desc*>(joined + 2 * I4_WARPS);
    int2* scratch = reinterpret_cast<int2*>(descs + I4_MAX_STAGES);
    int4* s_first = reinterpret_cast<int4*>(scratch + 32);
    int2* s_tot = reinterpret_cast<int2*>(s_first + 1);
    int* s_end = reinterpret_cast<int*>(s_tot + 1);

    grid_dependency_wait();
    const int hg = blockIdx.x % p.NHG;
    const int range = blockIdx.x / p.NHG;
    Plan pl;
    DecodeParams plan_of = p;
    // (as many sequences as ranges hardly have fewer chunks, and counting those
    // of 1024 takes 3 us)
    if (p.PC == 0 && p.B < p.NR) plan_of.NR = int4_ranges(p, scratch);
    make_plan(plan_of, range, scratch, s_first, s_tot, s_end, pl);
    grid_dependents_launch();
    if (pl.cs >= pl.ce || pl.seq < 0) return;
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&full[s], 33);           // the bulk copies' bytes, and each lane's own copies
            mbar_init(&empty[s], p.NCW);
        }
        for (int s = 0; s < I4_NQ; ++s) mbar_init(&qempty[s], p.NCW);
        for (int s = 0; s < I4_WARPS; ++s) {
            mbar_init(&joined[2 * s], max(1, a.TS - 1));
            mbar_init(&joined[2 * s + 1], 1);
        }
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    __syncthreads();
    if (warp == p.NCW) int4_producer<D, WT>(a, pl, hg, base, full, empty, qempty, descs);
    else if (warp < p.NCW) int4_consumer<QT, D, NQT, WT>(a, pl, hg, warp, base, full, empty, qempty, joined, descs);
}

template <class QT, int D, int NQT, bool WT>
static const void* int4_fn_w(int ncw) {
    // more than four row tiles of a head: 65 to 128 rows, 16 per warp
    if constexpr (NQT == 2)
        if (ncw > I4_WARPS) return reinterpret_cast<const void*>(&int4_decode_kernel<QT, D, NQT, WT, 8, 1>);
    return reinterpret_cast<const void*>(&int4_decode_kernel<QT, D, NQT, WT, I4_WARPS, i4_ctas(NQT)>);
}
template <class QT, bool WT>
static const void* int4_fn(int D, int nqt, int ncw) {
    if (D == 128) return nqt == 1 ? int4_fn_w<QT, 128, 1, WT>(ncw) : int4_fn_w<QT, 128, 2, WT>(ncw);
    return nqt == 1 ? int4_fn_w<QT, 64, 1, WT>(ncw) : int4_fn_w<QT, 64, 2, WT>(ncw);
}

static int cdiv_ll(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }

pa_status decode_int4(const Int4Call& c) {
    const int G = c.Hq / c.Hkv, rows = c.QL * G, D = c.D;
    // 8 query rows per warp while a group fits, else 16: the codes of a key are
    // unpacked once per warp
    const int nqt = rows <= 8 ? 1 : 2;
    const int RT = cdiv_ll(rows, 8 * nqt);
    if (RT > 8) return fail(PA_ERR_UNSUPPORTED, "decode: more than 128 query rows per KV head");
    // Four consumer warps per CTA: HPC heads x RT row tiles x TS warps along
    // the tokens.  Two or more head groups keep three CTAs per SM within the
    // 2 x SMs ranges that the workspace has partials for.
    int HPC = 1;
    for (int h = 4; h > 1; h /= 2)
        if (c.Hkv % h == 0 && c.Hkv >= 2 * h && h * RT <= I4_WARPS) { HPC = h; break; }
    const int TS = std::max(1, I4_WARPS / (HPC * RT));
    const int NCW = HPC * RT * TS, CT = I4_WT * TS;
    Int4Params a{};
    DecodeParams& p = a.d;
    p.out = c.out; p.q = c.q; p.block_tables = c.tables; p.seq_lens = c.lens; p.err_flag = c.err;
    p.B = c.B; p.Hq = c.Hq; p.Hkv = c.Hkv; p.G = G; p.D = D; p.bs = c.bs; p.NB = c.NB; p.MB = c.MB;
    p.out_bytes = 2;
    p.HPC = HPC; p.NHG = c.Hkv / HPC; p.MT = RT; p.NCW = NCW;
    p.ct = CT;
    // partitions are whole chunks
    p.PC = cdiv_ll(c.partition_tokens, CT);
    p.q_start = c.q_start; p.QL = c.QL; p.total_q = c.q_start ? c.total_q : c.B;
    // A unit start is charged one and a half chunks: 1024 short sequences took
    // 69, 67, 64 and 66 us, a 7B-like batch 53, 52, 51 and 52, at 2, 3, 6 and 10.
    p.WQ = 4; p.WS = 6;
    p.qk_scale = c.scale * 1.4426950408889634f;
    p.v_scale = 1.f;
    a.k = static_cast<const uint8_t*>(c.k); a.v = static_cast<const uint8_t*>(c.v);
    a.block_bytes = static_cast<size_t>(c.bs) * c.Hkv * (D / 2 + INT4_PARAM_BYTES);
    a.code_bytes = static_cast<uint32_t>(HPC * CT * (D / 2));
    a.param_bytes = static_cast<uint32_t>(HPC * CT * INT4_PARAM_BYTES);
    a.RT = RT;
    a.TS = TS;
    a.nbox = c.bs <= CT ? CT / c.bs : 1;
    for (a.bshift = 3; (1 << a.bshift) < c.bs; ++a.bshift) {}
    for (a.rshift = 3; (1 << a.rshift) < std::min(c.bs, CT); ++a.rshift) {}
    p.stage_bytes = 2 * (a.code_bytes + a.param_bytes);
    p.q_bytes = static_cast<uint32_t>(c.QL * HPC * G * D * 2);
    p.q_slot_bytes = (p.q_bytes + 127u) & ~127u;
    const uint32_t join = static_cast<uint32_t>(HPC * RT * (TS - 1) * nqt * 2 * (D / 8 + 2) * 32 * 4);
    const uint32_t frags = static_cast<uint32_t>(NCW * nqt * (D / 32) * 512);
    const uint32_t extras = 1152;
    const long long fixed = static_cast<long long>(I4_NQ) * p.q_slot_bytes + join + frags + extras + 128;
    const long long sm = std::min(c.max_smem, 227 * 1024);
    const int threads = (NCW + 1) * 32;
    const int ctas = NCW <= I4_WARPS ? i4_ctas(nqt) : 1;
    int stages = 0;
    for (int n = ctas; n >= 1 && stages < 2; --n)
        stages = static_cast<int>(std::min<long long>(I4_MAX_STAGES, ((sm + 1024) / n - 1024 - fixed) / p.stage_bytes));
    if (stages < 2) return fail(PA_ERR_UNSUPPORTED, "decode: pipeline stages do not fit in shared memory");
    p.stages = stages;
    p.q_off = stages * p.stage_bytes;
    a.join_off = p.q_off + I4_NQ * p.q_slot_bytes;
    a.frag_off = a.join_off + join;
    p.bar_off = a.frag_off + frags;
    const size_t smem = 128 + p.bar_off + extras;
    p.split_list = c.ws.split_list; p.totals = c.ws.totals; p.max_slots = c.ws.max_slots;
    p.part_ml = c.ws.part_ml; p.part_acc = c.ws.part_acc;

    const bool h = c.q_dtype == PA_F16;
    const void* kern = c.weights ? (h ? int4_fn<F16T, true>(D, nqt, NCW) : int4_fn<BF16T, true>(D, nqt, NCW))
                                 : (h ? int4_fn<F16T, false>(D, nqt, NCW) : int4_fn<BF16T, false>(D, nqt, NCW));
    if (c.weights) { p.scores = c.weights->scores; p.lse = c.weights->lse; p.chunk0 = c.weights->chunk0; }
    cudaError_t ce = allow_shared(kern, c.max_smem);
    if (ce != cudaSuccess) return fail_cuda("decode: set shared memory size", ce);
    int per_sm = 0;
    ce = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, smem);
    if (ce != cudaSuccess) return fail_cuda("decode: occupancy query", ce);
    per_sm = std::max(1, per_sm);
    const long long chunk_bound = static_cast<long long>(c.B) * cdiv_ll(static_cast<long long>(c.MB) * c.bs, CT);
    long long NR = std::max(1LL, static_cast<long long>(per_sm) * c.sms / p.NHG);
    NR = std::min(NR, 2LL * c.sms);            // the workspace holds 2 x SMs ranges
    NR = std::min(NR, chunk_bound);
    p.NR = static_cast<int>(NR);

    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(NR * p.NHG));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = c.stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* args[] = {&a};
    ce = cudaLaunchKernelExC(&cfg, kern, args);
    if (ce != cudaSuccess) return fail_cuda("decode: main kernel launch", ce);
    const pa_status st = launch_merge(p, c.q_dtype, c.partition_tokens > 0, c.sms, c.stream, true);
    return st == PA_OK && c.weights ? launch_weights(p, *c.weights, c.stream) : st;
}

}  // namespace pa
