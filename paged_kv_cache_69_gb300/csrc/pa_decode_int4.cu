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
// Both products are transposed: S^T = K Q^T with 16 tokens and O^T = V^T P^T
// with 16 dimensions as the M rows of mma.sync m16n8k16 and 8 query rows as N,
// so a GQA group of up to 8 heads fills the tile.  head_dim is summed in an
// order that lets a lane read 16 bytes of a key at once (and the query rows
// are laid out to match); P^T goes from the accumulator layout of S^T to the
// operand layout of the second product by an 8 x 8 transpose (movmatrix).
//
// Work split, partials and the merge are the paged decode kernel's: the chunks
// (64 tokens here) of all sequences form one stream, cut into ranges of equal
// cost for persistent CTAs; one warp fills a ring of stages with contiguous
// bulk copies (a block's codes of the CTA's heads are one span, its
// parameters another), the other warps each own 8 or 16 query rows of one KV
// head.
#include <algorithm>
#include <cmath>
#include <cuda.h>

#include "pa_common.h"
#include "pa_decode_int4.h"
#include "pa_decode_kernel.cuh"
#include "pa_int4.cuh"
#include "pa_kernels.h"

namespace pa {

constexpr int I4_CT = 64;                   // tokens of a chunk
constexpr int I4_MT = I4_CT / 16;           // 16-token tiles of a chunk
constexpr int I4_MAX_STAGES = 8;
constexpr int I4_NQ = 2;                    // query ring slots

struct I4Desc {
    int seq, tok0, slot, qrow0, qpos0, qn;
    uint32_t flags;                         // SEG_* bits, QLOAD, DIRECT, GAP
    int qslot;
    uint64_t vmask;                         // tokens of the chunk that exist
};

struct Int4Params {
    DecodeParams d;
    const uint8_t* k;
    const uint8_t* v;
    size_t block_bytes;
    uint32_t code_bytes, param_bytes;       // of one stage's K (or V)
    int RT;                                 // row tiles (warps) per KV head
    int nbox;                               // blocks of a chunk
};

// ---------------------------------------------------------------------------
// producer: one warp; lane b copies block b of a chunk (or head b of a block
// that is longer than a chunk).
// ---------------------------------------------------------------------------
template <int D>
__device__ __forceinline__ void int4_producer(const Int4Params& a, const Plan& pl, int hg, uint8_t* base,
                                              uint64_t* full, uint64_t* empty, uint64_t* qempty, I4Desc* descs) {
    const DecodeParams& p = a.d;
    const int lane = threadIdx.x & 31;
    const int S = p.stages, maxL = p.MB * p.bs;
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
    int wbase = (j * I4_CT) / p.bs;                 // 32 table entries from here on, the next 32 in flight
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
    int nch = cdiv_i(L, I4_CT), nbl = cdiv_i(L, p.bs);
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
    const uint32_t params_at = static_cast<uint32_t>(p.Hkv) * head_codes;    // its parameters
    const int rows = min(p.bs, I4_CT);                                       // rows of a block in a chunk
    const bool whole = p.bs <= I4_CT;
    const uint32_t box_codes = static_cast<uint32_t>(p.HPC * rows) * (D / 2), box_params = static_cast<uint32_t>(p.HPC * rows) * 4u;
    int issued = 0, qcount = 0, slot = 0, qs = 0;
    uint32_t round = 0, qround = 0;
    int jp = j, ju = 0;
    if (p.PC > 0) { ju = j / p.PC; jp = j - ju * p.PC; }
    bool ok = true;
    for (int k = pl.cs; k < pl.ce; ++k) {
        while (j >= nch) {
            Si += nch; Ui += n_units(L, p.PC, p.ct); ++i;
            L = len_of(i);
            load_q_rows();
            nch = cdiv_i(L, I4_CT); nbl = cdiv_i(L, p.bs);
            j = 0; jp = 0; ju = 0;
            wbase = 0;
            wval = (nseq == i && nbase == 0) ? nval : load_win(i, 0, nbl);
            prefetch_next();
        }
        const int tok0 = j * I4_CT, b0 = tok0 / p.bs;
        if (b0 + nb - 1 >= wbase + 32) {
            if (nseq == i && nbase <= b0 && b0 + nb - 1 < nbase + 32) {
                wbase = nbase; wval = nval;
            } else {
                wbase = b0; wval = load_win(i, wbase, nbl);
            }
            prefetch_next();
        }
        const int ntok = min(I4_CT, L - tok0);
        // lane b < nb: block b of the chunk
        const int id = __shfl_sync(0xffffffffu, wval, min(b0 + lane - wbase, 31));
        const bool mine = lane < nb && lane * rows < ntok;
        const bool good = mine && id >= 0 && id < p.NB;
        if (mine && !good) raise_flag(p.err_flag, PA_ERRBIT_BAD_BLOCK);
        const uint32_t goods = __ballot_sync(0xffffffffu, good);
        uint64_t vmask = ntok >= 64 ? ~0ull : ((1ull << ntok) - 1ull);
        if (goods != __ballot_sync(0xffffffffu, mine)) {
            for (int b = 0; b < nb; ++b)
                if (!((goods >> b) & 1u)) {
                    const uint64_t r = rows >= 64 ? ~0ull : ((1ull << rows) - 1ull);
                    vmask &= ~(r << (b * rows));
                }
        }
        const bool seg_start = (k == pl.cs) || (jp == 0);
        const bool qload = seg_start && (k == pl.cs || j == 0);
        if (lane == 0) {
            if (issued >= S && !mbar_wait_bounded(&empty[slot], (round - 1) & 1u)) {
                raise_flag(p.err_flag, PA_ERRBIT_WAIT_TIMEOUT);
                ok = false;
            }
            if (ok && qload && qcount >= I4_NQ && !mbar_wait_bounded(&qempty[qs], (qround - 1) & 1u)) {
                raise_flag(p.err_flag, PA_ERRBIT_WAIT_TIMEOUT);
                ok = false;
            }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        const uint32_t qrow_bytes = static_cast<uint32_t>(p.HPC * p.G) * D * 2u;
        if (lane == 0) {
            const bool part_end = p.PC > 0 && jp == p.PC - 1;
            uint32_t flags = 0;
            if (seg_start) flags |= SEG_START;
            if (qload) flags |= QLOAD;
            if (k == pl.ce - 1 || j == nch - 1 || part_end) flags |= SEG_END;
            if (k == pl.ce - 1 && part_end && j + 1 < nch) flags |= GAP;
            if (n_units(L, p.PC, p.ct) == 1 && Si >= pl.cs && Si + nch <= pl.ce) flags |= DIRECT;
            I4Desc d;
            d.seq = i; d.tok0 = tok0; d.vmask = vmask; d.flags = flags; d.qn = qn;
            d.slot = range + Ui + ju;
            d.qslot = qload ? qs : (qs == 0 ? I4_NQ - 1 : qs - 1);
            d.qrow0 = qrow;
            d.qpos0 = L - qn;
            descs[slot] = d;
            const uint32_t boxes = __popc(goods);
            mbar_arrive_expect_tx(&full[slot], boxes * 2u * (box_codes + box_params) +
                                                   (qload ? static_cast<uint32_t>(qn) * qrow_bytes : 0u));
        }
        __syncwarp();
        uint8_t* kc = base + slot * p.stage_bytes;
        uint8_t* kp = kc + a.code_bytes;
        uint8_t* vc = kp + a.param_bytes;
        uint8_t* vp = vc + a.code_bytes;
        if (whole) {
            if (good) {
                const size_t blk = static_cast<size_t>(id) * a.block_bytes;
                const size_t cs = blk + static_cast<size_t>(hg * p.HPC) * head_codes;
                const size_t ps = blk + params_at + static_cast<size_t>(hg * p.HPC * p.bs) * 4u;
                bulk_load(kc + lane * box_codes, a.k + cs, box_codes, &full[slot]);
                bulk_load(kp + lane * box_params, a.k + ps, box_params, &full[slot]);
                bulk_load(vc + lane * box_codes, a.v + cs, box_codes, &full[slot]);
                bulk_load(vp + lane * box_params, a.v + ps, box_params, &full[slot]);
            }
        } else if (goods & 1u) {
            // a chunk is part of one block: a span per head
            const size_t blk = static_cast<size_t>(__shfl_sync(0xffffffffu, id, 0)) * a.block_bytes;
            const int t0 = tok0 % p.bs;
            const uint32_t cb = I4_CT * (D / 2), pb = I4_CT * 4;
            for (int h = lane; h < p.HPC; h += 32) {
                const size_t cs = blk + static_cast<size_t>(hg * p.HPC + h) * head_codes + static_cast<size_t>(t0) * (D / 2);
                const size_t ps = blk + params_at + static_cast<size_t>((hg * p.HPC + h) * p.bs + t0) * 4u;
                bulk_load(kc + h * cb, a.k + cs, cb, &full[slot]);
                bulk_load(kp + h * pb, a.k + ps, pb, &full[slot]);
                bulk_load(vc + h * cb, a.v + cs, cb, &full[slot]);
                bulk_load(vp + h * pb, a.v + ps, pb, &full[slot]);
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

template <typename T>
__device__ __forceinline__ uint32_t pack_out(float a, float b) {
    return pack2(a, b, std::is_same<T, __nv_bfloat16>::value);
}

// ---------------------------------------------------------------------------
// consumer: warp w owns NQT tiles of 8 query rows of one KV head.
// HL: each weight enters the second product as a pair of f16 numbers (the
// rounded weight and what the rounding lost).
// ---------------------------------------------------------------------------
template <class QT, int D, int NQT, bool HL>
__device__ __forceinline__ void int4_consumer(const Int4Params& a, const Plan& pl, int hg, int w, uint8_t* base,
                                              uint64_t* full, uint64_t* empty, uint64_t* qempty, const I4Desc* descs) {
    using T = typename QT::T;
    constexpr int KW = D / 32;                    // 32-bit code words of a key that a lane reads
    constexpr int OT = D / 16;                    // 16-dimension output tiles
    constexpr float UNIT = 16777216.f;            // 2^24: what an f16 with the bits of n is short of n
    const DecodeParams& p = a.d;
    const int lane = threadIdx.x & 31, g4 = lane >> 2, t4 = lane & 3;
    const int hl = w / a.RT, rt = w - hl * a.RT;
    const int S = p.stages;
    const int rows_total = p.QL * p.G;
    const int rows = min(p.bs, I4_CT);            // rows of a block in a chunk
    // Row r of a tile of 8 tokens is token tau(r) = r ^ (r / 2 % 2), on both
    // sides of P: the four tokens that a quarter of the V loads reads are then
    // two even and two odd 64-byte rows.
    const int tk = g4 ^ ((g4 >> 1) & 1);
    const int tv0 = (2 * t4) ^ (t4 & 1), tv1 = (2 * t4 + 1) ^ (t4 & 1);
    // byte offset of a token's row of this head in the stage's codes / parameters
    auto row_of = [&](int t) -> uint32_t {
        const int b = t / rows;
        return static_cast<uint32_t>((b * p.HPC + hl) * rows + (t - b * rows));
    };

    float acc[OT][NQT][4];
    uint32_t qf[NQT][KW][4];
    float m[NQT][2], l[NQT][2], c0[NQT][2];       // rows 2 t4 and 2 t4 + 1 of each tile
    float sq[NQT][2], qk[NQT][2];
    int jt[NQT][2], lim[NQT][2];
    float inv = 0.f;                              // power of two on step in the weights; 0: not set yet
    int in_rows = 0;
#pragma unroll
    for (int n = 0; n < NQT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int R = (rt * NQT + n) * 8 + 2 * t4 + e;
            jt[n][e] = R / p.G;
            if (R < rows_total) in_rows |= 1 << (2 * n + e);
            lim[n][e] = INT_MAX;
            sq[n][e] = qk[n][e] = 0.f;
        }

    for (int st = 0, k = pl.cs; k < pl.ce; ++k, ++st) {
        const int slot = st % S;
        if (!mbar_wait_bounded(&full[slot], (st / S) & 1u)) {
            if (lane == 0) raise_flag(p.err_flag, PA_ERRBIT_WAIT_TIMEOUT);
            return;
        }
        const I4Desc d = descs[slot];
        const uint8_t* kc = base + slot * p.stage_bytes;
        const uint8_t* kp = kc + a.code_bytes;
        const uint8_t* vc = kp + a.param_bytes;
        const uint8_t* vp = vc + a.code_bytes;
        if (d.flags & SEG_START) {
            if (d.flags & QLOAD) {
                // The B operand of this lane: row g4 of each tile, dimensions
                // [D/4 * t4, D/4 * (t4 + 1)) in the codes' order.  bf16 rows are
                // scaled by a power of two into f16's range (their 8 bits fit).
                const uint8_t* qb = base + p.q_off + d.qslot * p.q_slot_bytes;
#pragma unroll
                for (int n = 0; n < NQT; ++n) {
                    const int R = (rt * NQT + n) * 8 + g4, jj = R / p.G;
                    const bool on = R < rows_total && jj < d.qn;
                    const uint4* src = reinterpret_cast<const uint4*>(
                        qb + (static_cast<size_t>(jj * p.HPC + hl) * p.G + (R - jj * p.G)) * D * 2 + t4 * (D / 2));
                    uint32_t raw[KW][4];
#pragma unroll
                    for (int x = 0; x < KW; ++x) {
                        const uint4 r = on ? src[x] : make_uint4(0, 0, 0, 0);
                        raw[x][0] = r.x; raw[x][1] = r.y; raw[x][2] = r.z; raw[x][3] = r.w;
                    }
                    float f = 1.f;
                    if constexpr (QT::code == PA_BF16) {
                        float mx = 0.f;
#pragma unroll
                        for (int x = 0; x < KW; ++x)
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw[x][y]));
                                mx = fmaxf(mx, fmaxf(fabsf(v.x), fabsf(v.y)));
                            }
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                        // 2^(13 - exponent of the largest), from its exponent bits
                        const int ex = static_cast<int>(__float_as_uint(mx) >> 23) - 127;
                        if (mx > 0.f && ex < 128) f = __uint_as_float(static_cast<uint32_t>(min(13 - ex, 126) + 127) << 23);
#pragma unroll
                        for (int x = 0; x < KW; ++x)
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw[x][y]));
                                raw[x][y] = f32x2_to_f16x2(v.x * f, v.y * f);
                            }
                    }
                    float s = 0.f;
#pragma unroll
                    for (int x = 0; x < KW; ++x) {
                        // words hold dims (0,1) (2,3) (4,5) (6,7): pairs (0,4) (2,6) (1,5) (3,7)
                        qf[n][x][0] = __byte_perm(raw[x][0], raw[x][2], 0x5410);
                        qf[n][x][1] = __byte_perm(raw[x][1], raw[x][3], 0x5410);
                        qf[n][x][2] = __byte_perm(raw[x][0], raw[x][2], 0x7632);
                        qf[n][x][3] = __byte_perm(raw[x][1], raw[x][3], 0x7632);
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&raw[x][y]));
                            s += v.x + v.y;
                        }
                    }
                    s += __shfl_xor_sync(0xffffffffu, s, 1);
                    s += __shfl_xor_sync(0xffffffffu, s, 2);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        sq[n][e] = __shfl_sync(0xffffffffu, s, (2 * t4 + e) * 4);
                        qk[n][e] = p.qk_scale / __shfl_sync(0xffffffffu, f, (2 * t4 + e) * 4);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&qempty[d.qslot]);
            }
#pragma unroll
            for (int n = 0; n < NQT; ++n) {
#pragma unroll
                for (int o = 0; o < OT; ++o) acc[o][n][0] = acc[o][n][1] = acc[o][n][2] = acc[o][n][3] = 0.f;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    m[n][e] = -INFINITY; l[n][e] = 0.f; c0[n][e] = 0.f;
                    if (p.q_start) lim[n][e] = ((in_rows >> (2 * n + e)) & 1) && jt[n][e] < d.qn ? d.qpos0 + jt[n][e] : -1;
                }
            }
            inv = 0.f;
        }
        // ---- S^T = K Q^T over the chunk's tokens ----
        float s[I4_MT][NQT][4];
#pragma unroll
        for (int mt = 0; mt < I4_MT; ++mt) {
            const uint32_t r0 = row_of(16 * mt + tk), r1 = row_of(16 * mt + 8 + tk);
            uint32_t ka[KW], kb[KW];
            if constexpr (KW == 4) {
                const uint4 x = *reinterpret_cast<const uint4*>(kc + r0 * (D / 2) + t4 * 16);
                const uint4 y = *reinterpret_cast<const uint4*>(kc + r1 * (D / 2) + t4 * 16);
                ka[0] = x.x; ka[1] = x.y; ka[2] = x.z; ka[3] = x.w;
                kb[0] = y.x; kb[1] = y.y; kb[2] = y.z; kb[3] = y.w;
            } else {
                const uint2 x = *reinterpret_cast<const uint2*>(kc + r0 * (D / 2) + t4 * 8);
                const uint2 y = *reinterpret_cast<const uint2*>(kc + r1 * (D / 2) + t4 * 8);
                ka[0] = x.x; ka[1] = x.y; kb[0] = y.x; kb[1] = y.y;
            }
            float lo[NQT][4], hi[NQT][4];
#pragma unroll
            for (int n = 0; n < NQT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) lo[n][e] = hi[n][e] = 0.f;
#pragma unroll
            for (int x = 0; x < KW; ++x) {
                const uint32_t a8 = ka[x] >> 8, b8 = kb[x] >> 8;
                const uint32_t A1[4] = {ka[x] & 0x000f000fu, kb[x] & 0x000f000fu, a8 & 0x000f000fu, b8 & 0x000f000fu};
                const uint32_t A2[4] = {ka[x] & 0x00f000f0u, kb[x] & 0x00f000f0u, a8 & 0x00f000f0u, b8 & 0x00f000f0u};
#pragma unroll
                for (int n = 0; n < NQT; ++n) {
                    mma_16816<false>(lo[n], A1, qf[n][x][0], qf[n][x][1]);
                    mma_16816<false>(hi[n], A2, qf[n][x][2], qf[n][x][3]);
                }
            }
            const float2 p0 = __half22float2(*reinterpret_cast<const __half2*>(kp + r0 * 4));
            const float2 p1 = __half22float2(*reinterpret_cast<const __half2*>(kp + r1 * 4));
            const float s0 = p0.x * UNIT, s1 = p1.x * UNIT;
#pragma unroll
            for (int n = 0; n < NQT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float dot = fmaf(hi[n][e], 0.0625f, lo[n][e]);
                    s[mt][n][e] = fmaf(dot, e < 2 ? s0 : s1, (e < 2 ? p0.y : p1.y) * sq[n][e & 1]) * qk[n][e & 1];
                }
        }
        // tokens that do not exist, or lie behind a row's position
        const bool all = d.vmask == ~0ull;
        if (!all || (p.q_start && d.tok0 + I4_CT - 1 > d.qpos0)) {
#pragma unroll
            for (int mt = 0; mt < I4_MT; ++mt)
#pragma unroll
                for (int n = 0; n < NQT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int t = 16 * mt + 8 * (e >> 1) + tk;
                        if (!((d.vmask >> t) & 1ull) || d.tok0 + t > lim[n][e & 1]) s[mt][n][e] = -INFINITY;
                    }
        }
        // ---- V parameters: (step, low) of the lane's two tokens of each tile ----
        float vs[I4_MT][2], vl[I4_MT][2];
        float smax = 0.f;
#pragma unroll
        for (int mt = 0; mt < I4_MT; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = 16 * mt + 8 * e + tk;
                float2 v = __half22float2(*reinterpret_cast<const __half2*>(vp + row_of(t) * 4));
                if (!all && !((d.vmask >> t) & 1ull)) v = make_float2(0.f, 0.f);   // the pool may hold NaN there
                vs[mt][e] = v.x; vl[mt][e] = v.y;
                smax = fmaxf(smax, fabsf(v.x));
            }
        // Weights p * step enter an f16 operand: a power of two, common to the
        // segment, keeps the largest step's in [2^9, 2^15].
        smax = max_g4(smax);
        float grow = 1.f;
        if ((inv == 0.f && smax > 0.f) || smax * inv > 32768.f) {
            const int ex = static_cast<int>(__float_as_uint(smax) >> 23) - 127;
            const float ni = __uint_as_float(static_cast<uint32_t>(9 - ex + 127) << 23);
            if (inv != 0.f) grow = ni / inv;
            inv = ni;
        }
        // ---- online softmax (log2 domain) of the rows ----
        uint32_t pf[I4_MT][NQT][2], pl_[HL ? I4_MT : 1][NQT][2];
        float al[NQT][2];
        bool same = grow == 1.f;
#pragma unroll
        for (int n = 0; n < NQT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mx = -INFINITY;
#pragma unroll
                for (int mt = 0; mt < I4_MT; ++mt) mx = fmaxf(mx, fmaxf(s[mt][n][e], s[mt][n][e + 2]));
                const float mn = fmaxf(m[n][e], max_g4(mx));
                const float mu = mn == -INFINITY ? 0.f : mn;
                al[n][e] = ex2_approx(m[n][e] - mu);
                m[n][e] = mn;
                same = same && al[n][e] == 1.f;
                float ps = 0.f, cs = 0.f;
#pragma unroll
                for (int mt = 0; mt < I4_MT; ++mt) {
                    s[mt][n][e] = ex2_approx(s[mt][n][e] - mu);
                    s[mt][n][e + 2] = ex2_approx(s[mt][n][e + 2] - mu);
                    ps += s[mt][n][e] + s[mt][n][e + 2];
                    cs = fmaf(s[mt][n][e], vl[mt][0], fmaf(s[mt][n][e + 2], vl[mt][1], cs));
                }
                l[n][e] = fmaf(l[n][e], al[n][e], ps);
                c0[n][e] = fmaf(c0[n][e], al[n][e], cs);
            }
        }
#pragma unroll
        for (int mt = 0; mt < I4_MT; ++mt) {
            const float w0 = vs[mt][0] * inv, w1 = vs[mt][1] * inv;
#pragma unroll
            for (int n = 0; n < NQT; ++n) {
                const float x0 = s[mt][n][0] * w0, x1 = s[mt][n][1] * w0, x2 = s[mt][n][2] * w1, x3 = s[mt][n][3] * w1;
                const uint32_t h0 = f32x2_to_f16x2(x0, x1), h1 = f32x2_to_f16x2(x2, x3);
                pf[mt][n][0] = movmatrix(h0);
                pf[mt][n][1] = movmatrix(h1);
                if constexpr (HL) {
                    const float2 y0 = __half22float2(*reinterpret_cast<const __half2*>(&h0));
                    const float2 y1 = __half22float2(*reinterpret_cast<const __half2*>(&h1));
                    pl_[mt][n][0] = movmatrix(f32x2_to_f16x2(x0 - y0.x, x1 - y0.y));
                    pl_[mt][n][1] = movmatrix(f32x2_to_f16x2(x2 - y1.x, x3 - y1.y));
                }
            }
        }
        if (!__all_sync(0xffffffffu, same)) {
#pragma unroll
            for (int n = 0; n < NQT; ++n) {
                const float f0 = al[n][0] * grow, f1 = al[n][1] * grow;
#pragma unroll
                for (int o = 0; o < OT; ++o) {
                    acc[o][n][0] *= f0; acc[o][n][1] *= f1; acc[o][n][2] *= f0; acc[o][n][3] *= f1;
                }
            }
        }
        // ---- O^T += V^T P^T ----
#pragma unroll
        for (int mt = 0; mt < I4_MT; ++mt) {
            // k columns 2 t4, 2 t4 + 1 and 8 on: four tokens of D / 8 dimensions
            const uint32_t r[4] = {row_of(16 * mt + tv0), row_of(16 * mt + tv1), row_of(16 * mt + 8 + tv0),
                                   row_of(16 * mt + 8 + tv1)};
            constexpr int VW = D / 64;            // code words of a value that a lane reads
            uint32_t v[4][VW];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                if constexpr (VW == 2) {
                    const uint2 y = *reinterpret_cast<const uint2*>(vc + r[x] * (D / 2) + g4 * 8);
                    v[x][0] = y.x; v[x][1] = y.y;
                } else {
                    v[x][0] = *reinterpret_cast<const uint32_t*>(vc + r[x] * (D / 2) + g4 * 4);
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
                    if constexpr (HL) mma_16816<false>(acc[o][n], A, pl_[mt][n][0], pl_[mt][n][1]);
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[slot]);
        if (d.flags & SEG_END) {
            const bool direct = (d.flags & DIRECT) != 0;
            const float back = inv > 0.f ? UNIT / inv : 0.f;
#pragma unroll
            for (int n = 0; n < NQT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float lt = sum_g4(l[n][e]), ct = sum_g4(c0[n][e]);
                    const bool on = ((in_rows >> (2 * n + e)) & 1) && jt[n][e] < d.qn && (direct || d.slot < p.max_slots);
                    if (!on) continue;
                    const int R = (rt * NQT + n) * 8 + 2 * t4 + e;
                    const int head = (hg * p.HPC + hl) * p.G + (R - jt[n][e] * p.G);
                    const float sc = direct ? (lt == 0.f ? 0.f : 1.f / lt) : 1.f;
                    // the lane's D / 8 dimensions from D / 8 * g4 on, in order
                    float v[D / 8];
#pragma unroll
                    for (int o = 0; o < OT; ++o) {
                        const float u = (o & 1) ? back * 0.0625f : back;
                        v[o] = fmaf(acc[o][n][e], u, ct) * sc;
                        v[OT + o] = fmaf(acc[o][n][2 + e], u, ct) * sc;
                    }
                    if (direct) {
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
                        if (g4 == 0) p.part_ml[prow] = make_float2(m[n][e], lt);
                    }
                }
            if ((d.flags & GAP) && !direct && d.slot + 1 < p.max_slots) {
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

// MAXW: consumer warps at most; 4 leaves the registers for two CTAs per SM.
template <class QT, int D, int NQT, bool HL, int MAXW>
__global__ void __launch_bounds__((MAXW + 1) * 32, MAXW <= 4 ? 2 : 1)
int4_decode_kernel(const __grid_constant__ Int4Params a) {
    extern __shared__ uint8_t smem_raw[];
    const DecodeParams& p = a.d;
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    uint64_t* full = reinterpret_cast<uint64_t*>(base + p.bar_off);
    uint64_t* empty = full + I4_MAX_STAGES;
    uint64_t* qempty = empty + I4_MAX_STAGES;
    I4Desc* descs = reinterpret_cast<I4Desc*>(qempty + I4_NQ);
    int2* scratch = reinterpret_cast<int2*>(descs + I4_MAX_STAGES);
    int4* s_first = reinterpret_cast<int4*>(scratch + 32);
    int2* s_tot = reinterpret_cast<int2*>(s_first + 1);
    int* s_end = reinterpret_cast<int*>(s_tot + 1);

    grid_dependency_wait();
    const int hg = blockIdx.x % p.NHG;
    const int range = blockIdx.x / p.NHG;
    Plan pl;
    make_plan(p, range, scratch, s_first, s_tot, s_end, pl);
    grid_dependents_launch();
    if (pl.cs >= pl.ce || pl.seq < 0) return;
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], p.NCW);
        }
        for (int s = 0; s < I4_NQ; ++s) mbar_init(&qempty[s], p.NCW);
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    __syncthreads();
    if (warp == p.NCW) int4_producer<D>(a, pl, hg, base, full, empty, qempty, descs);
    else if (warp < p.NCW) int4_consumer<QT, D, NQT, HL>(a, pl, hg, warp, base, full, empty, qempty, descs);
}

template <class QT, int D, int NQT, bool HL>
static const void* int4_fn_w(int ncw) {
    if (ncw <= 4) return reinterpret_cast<const void*>(&int4_decode_kernel<QT, D, NQT, HL, 4>);
    return reinterpret_cast<const void*>(&int4_decode_kernel<QT, D, NQT, HL, 8>);
}
template <class QT, bool HL>
static const void* int4_fn(int D, int nqt, int ncw) {
    if (D == 128) return nqt == 1 ? int4_fn_w<QT, 128, 1, HL>(ncw) : int4_fn_w<QT, 128, 2, HL>(ncw);
    return nqt == 1 ? int4_fn_w<QT, 64, 1, HL>(ncw) : int4_fn_w<QT, 64, 2, HL>(ncw);
}

static int cdiv_ll(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }

pa_status decode_int4(const Int4Call& c) {
    const int G = c.Hq / c.Hkv, rows = c.QL * G, D = c.D;
    // 8 query rows per warp while a group fits, else 16: the codes of a key are
    // unpacked once per warp
    const int nqt = rows <= 8 ? 1 : 2;
    const int RT = cdiv_ll(rows, 8 * nqt);
    if (RT > 8) return fail(PA_ERR_UNSUPPORTED, "decode: more than 128 query rows per KV head");
    // heads per CTA: up to 4 warps (two CTAs per SM), at least one head
    int HPC = 1;
    for (int h = c.Hkv; h >= 1; --h)
        if (c.Hkv % h == 0 && h * RT <= std::max(4, RT)) { HPC = h; break; }
    const int NCW = HPC * RT;
    Int4Params a{};
    DecodeParams& p = a.d;
    p.out = c.out; p.q = c.q; p.block_tables = c.tables; p.seq_lens = c.lens; p.err_flag = c.err;
    p.B = c.B; p.Hq = c.Hq; p.Hkv = c.Hkv; p.G = G; p.D = D; p.bs = c.bs; p.NB = c.NB; p.MB = c.MB;
    p.out_bytes = 2;
    p.HPC = HPC; p.NHG = c.Hkv / HPC; p.MT = RT; p.NCW = NCW;
    p.ct = I4_CT;
    // partitions are whole chunks
    p.PC = cdiv_ll(c.partition_tokens, I4_CT);
    p.q_start = c.q_start; p.QL = c.QL; p.total_q = c.q_start ? c.total_q : c.B;
    p.WQ = 4; p.WS = 3;
    p.qk_scale = c.scale * 1.4426950408889634f;
    p.v_scale = 1.f;
    a.k = static_cast<const uint8_t*>(c.k); a.v = static_cast<const uint8_t*>(c.v);
    a.block_bytes = static_cast<size_t>(c.bs) * c.Hkv * (D / 2 + INT4_PARAM_BYTES);
    a.code_bytes = static_cast<uint32_t>(HPC * I4_CT * (D / 2));
    a.param_bytes = static_cast<uint32_t>(HPC * I4_CT * INT4_PARAM_BYTES);
    a.RT = RT;
    a.nbox = c.bs <= I4_CT ? I4_CT / c.bs : 1;
    p.stage_bytes = 2 * (a.code_bytes + a.param_bytes);
    p.q_bytes = static_cast<uint32_t>(c.QL * HPC * G * D * 2);
    p.q_slot_bytes = (p.q_bytes + 127u) & ~127u;
    const uint32_t extras = 1024;
    const long long fixed = static_cast<long long>(I4_NQ) * p.q_slot_bytes + extras + 128;
    const long long sm = std::min(c.max_smem, 227 * 1024);
    const int threads = (NCW + 1) * 32;
    int stages = 0;
    if (NCW <= 4) {
        const long long per_cta = (sm + 1024) / 2 - 1024 - fixed;
        const int s2 = static_cast<int>(std::min<long long>(I4_MAX_STAGES, per_cta / p.stage_bytes));
        if (s2 >= 2) stages = s2;
    }
    if (stages == 0) stages = static_cast<int>(std::min<long long>(I4_MAX_STAGES, (sm - fixed) / p.stage_bytes));
    if (stages < 2) return fail(PA_ERR_UNSUPPORTED, "decode: pipeline stages do not fit in shared memory");
    p.stages = stages;
    p.q_off = stages * p.stage_bytes;
    p.bar_off = p.q_off + I4_NQ * p.q_slot_bytes;
    const size_t smem = 128 + p.bar_off + extras;
    p.split_list = c.ws.split_list; p.totals = c.ws.totals; p.max_slots = c.ws.max_slots;
    p.part_ml = c.ws.part_ml; p.part_acc = c.ws.part_acc;

    const void* kern = c.q_dtype == PA_F16 ? int4_fn<F16T, true>(D, nqt, NCW) : int4_fn<BF16T, false>(D, nqt, NCW);
    cudaError_t ce = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (ce != cudaSuccess) return fail_cuda("decode: set shared memory size", ce);
    int per_sm = 0;
    ce = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, smem);
    if (ce != cudaSuccess) return fail_cuda("decode: occupancy query", ce);
    per_sm = std::max(1, per_sm);
    const long long chunk_bound = static_cast<long long>(c.B) * cdiv_ll(static_cast<long long>(c.MB) * c.bs, I4_CT);
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
    return launch_merge(p, c.q_dtype, c.partition_tokens > 0, c.sms, c.stream);
}

}  // namespace pa
