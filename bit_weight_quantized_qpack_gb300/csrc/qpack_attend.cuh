// qpack_attend.cuh — attention of one new token a sequence over the paged KV cache: the kernel, instantiated per cache
// type in qpack_attend_i8.cu, qpack_attend_f16.cu and qpack_attend_bf16.cu.
//
// The mathematics. One pass over the cache with a running maximum and sum (base 2): for tokens t, x_t = q~ . k'_t times
// scale log2 e, m' = max(m, x_t), l' = l 2^(m - m') + 2^(x_t - m'), o' = o 2^(m - m') + 2^(x_t - m') v'_t; out = o / l.
// Differences are taken between the products q~ . k'_t, before the factor: there they are exact near the maximum.
// Triples (m, l, o) over parts of a sequence join by the same rule, in any grouping; here always in a fixed order.
//
// What bounds it. Every cached byte is read once: 2 (D + D/16) bytes a token and key/value head in 8 bits, at D = 128
// 12.6 clocks of an SM's share of the copy rate (6787 GB/s over 152 SMs at 2.07 GHz). The two products take 4 D flops a
// token and query head, too much for the CUDA cores with eight heads a key head (2048 FMAs against 1610 issue slots in
// those 12.6 clocks). A query block has 1 to 16 rows where tcgen05.mma has at least 64, and its accumulators would have
// to come back from TMEM for every tile's softmax, so the products run on the warp-level mma.sync (m16n8k16): its
// fragments are registers, the softmax needs no exchange but two shuffles, and 32 instructions per 16 tokens keep the
// tensor pipe 30% busy. Unpacking the 8-bit cache is the largest part of the instructions (14 of some 23 a token and
// warp), and they are issued on half of the cycles.
//
// Measured: 64 sequences of 4096 to 8192 tokens, 64 query heads over 8, 8 bits: 139 us = 6180 GB/s, 91% of the copy
// rate; one sequence of 131071 tokens, 32 over 8: 53.4 us = 79%. What is left there is some 10 us a call, whatever its
// size: 2 us until the first copies start (lengths, then pages: dependent loads; queries are in registers after 4 us, in
// the last block after 8), 2 to 4 us by which the slowest SM ends after the middle one, 3 us for the joins of blocks, the
// launch. A row of 97 tokens takes 7 us. Sixteen query heads a key head are bound by the instructions instead (62% of the
// copy rate).
//
//   S = Q K^T:     A = queries (16 rows), B = 16 tokens x D. With up to eight query heads rows 0-7 hold the queries'
//                  leading 16-bit terms and rows 8-15 the remainders of the same heads, so one instruction takes both
//                  and S is the sum of two registers of a thread. With up to sixteen heads the remainders go in a
//                  second instruction.
//   O^T = V^T P^T: A = values transposed by ldmatrix, B = probabilities: S's accumulator layout is B's operand layout
//                  as it stands. Probabilities go in as two terms as well.
//
// Both terms carry 22 bits together: scores and sums then differ from fp32 arithmetic by less than the output's
// rounding, where a single fp16 term would add errors of that size. Queries are scaled by a power of two to a maximum in
// [2^13, 2^14) and probabilities by 2^12, so neither term meets fp16's range. Where the cache is bfloat16 two terms carry
// 16 bits: queries get a third term, and so do probabilities where the output is fp32 (2% of the time); a 16-bit output
// does not show their 2^-17. bfloat16 terms have fp32's range and stay as they are: scaled, the sums would pass it before
// the fp32 form's do.
//
// 8-bit elements become fp16(scale * code), exactly the cache's definition: a byte permute puts code + 128 under the
// exponent of 1024, one packed subtraction takes 1152 off (exact), one packed product rounds once: 1.75 instructions an
// element. ldmatrix moves pairs of bytes as 16-bit elements: for keys the four bytes of a thread are four consecutive
// d (the queries' fragments use the same order of d), for values two d of two tokens.
//
// Work is cut by tiles of 16 or 32 tokens, not by rows: lengths are known on the device only and may be anything, so
// each block adds up the rows' tiles and takes an equal share of all of them (consecutive tiles, through as many
// segments (row, key/value head, group of query heads) as it covers), and each of its warps an equal share of the
// block's. A warp owns a ring of cp.async stages and never waits for another warp until its share is done. A segment
// inside one warp's share is finished by that warp; one inside a block's share is joined in shared memory; one that
// spans blocks goes through the workspace, and the last block's warps to arrive join it. Where the segments are few and
// equally long, each gets a block.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qpack_dev.cuh"
#include "qpack_launch.h"
#include "qpack_paged.cuh"

namespace qpack {
namespace attend {

constexpr int MAX_ROWS = 1024;              // rows a launch
constexpr int MAX_COUNTERS = QPACK_KV_ATTEND_ZEROED / 4;    // of a launch: the front of the workspace

// Shape of an instance: NT groups of eight query heads, tiles of TOK tokens, W warps, a ring of STAGES tiles each.
// Accumulators and query fragments take D NT / 4 registers a thread each, so they bound W; shared memory bounds TOK and
// the stages. Measured (one block an SM throughout; us for one sequence of 131071 tokens / 64 of 4096 to 8192, 8 bits,
// D = 128): 8 warps x 32 tokens 54.9 / 141.3, 12 x 32 57.0 / 141.0, 10 x 32 59.5 / 151, 12 x 16 59.7 / 146, 16 x 16
// 60.9 / 147; two blocks of 4 warps an SM 57.9 / 140.7 where one of 8 had come to 52.3 / 136.8. At D = 64 and in fp16 at
// 128 twelve warps are up to 10% faster than eight on long caches (62 against 68 us) and 2% slower on short ones, although
// 20 bytes a thread spill in fp16; in bfloat16 at 128 their registers spill over the third terms (27.5 against 25.6 us).
// What else spills: 12 to 136 bytes where two groups of heads are held together (most in 8 bits at 128) or rows have 256
// elements. The other five instances of 64 and 128 elements with one group do not.
template <int KT, int D, int NT> struct Cfg {
    static constexpr int ES = KT == QPACK_KV_I8 ? 1 : 2;
    static constexpr int RB = D * ES;                           // bytes of a token's row
    static constexpr int SB = KT == QPACK_KV_I8 ? D / 16 : 0;   // bytes of its scales
    static constexpr int TOK = RB >= 256 ? 16 : 32;
    static constexpr int TILE = 2 * TOK * (RB + SB);            // keys, values, their scales
    static constexpr int W = RB == 512 ? 6 : D * NT >= 256 || (KT != QPACK_KV_F16 && D == 128) ? 8 : 12;
    // Two bfloat16 terms hold 16 bits: what an fp32 or rotated query has beyond waits in shared memory for a third product.
    static constexpr bool THREE = KT == QPACK_KV_BF16;
    static constexpr int Q3 = THREE ? D / 16 * 2 * NT * 128 : 0;    // bytes a warp
    static constexpr int ROOM = (222000 - W * Q3) / (W * TILE);
    static constexpr int STAGES = ROOM > 4 ? 4 : ROOM;
    static constexpr int NH = 8 * NT;
    static constexpr int PS = D + 4;                            // floats of a head in a partial, padded for the banks
    static constexpr int PF = NH * PS;                          // floats of a piece's accumulators
    static constexpr int VEC = NH * D / 4;                      // threads of a join, four accumulators each
    static constexpr int SLICES = VEC / 32;                     // warps of a join, each on its own
    static_assert(STAGES >= 2 && PF * 4 <= STAGES * TILE, "a warp's ring holds a partial");
    static_assert(2 * W <= 32, "a lane a piece");
    // Probabilities are held as 2^(x - m + P_BIAS), and queries are brought to a like height (the head of this file says why).
    static constexpr float P_BIAS = KT == QPACK_KV_BF16 ? 0.0f : 12.0f;
};

struct Params {
    AttendArgs a;
    int B, C, G;                // rows of this launch, groups of query heads, query heads a key/value head
    int row0;                   // first row of this launch
    int *counters;              // [segments][SLICES], zero between calls
    float4 *block_parts;        // [grid][2][VEC]: accumulators of a piece that leaves its block
    float2 *block_sums;         // [grid][2][VEC]: maximum and sum, once a thread
    float *warp_parts;          // [grid][W][PF]
};

static __device__ int g_fault_attend = 0;       // one a translation unit: one a cache type

__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
template <int N> __device__ __forceinline__ void cp_small(uint32_t dst, const void *src, bool ok) {
    if (N == 16)
        cp16(dst, src, ok);
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N == 16 ? 4 : N),
                     "r"(ok ? N : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t *r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t *r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// c += a b, m16n8k16, fp16 or bf16 operands.
template <int KT>
__device__ __forceinline__ void mma(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    if (KT == QPACK_KV_BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int V> struct Int { static constexpr int value = V; };

// N bytes (a multiple of 4, aligned to at most 16 of them) of shared memory as words.
template <int N> __device__ __forceinline__ void load_words(const unsigned char *p, uint32_t *w) {
    if (N % 16 == 0) {
#pragma unroll
        for (int i = 0; i < N / 16; ++i) {
            const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
            w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
        }
    } else if (N == 8) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x, w[1] = v.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    }
}

// Two fp32 as a packed pair of 16-bit terms, x in the low half, and the pair of what they leave.
template <int KT> __device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
    if (KT == QPACK_KV_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        const __nv_bfloat162 l = __floats2bfloat162_rn(x - __low2float(h), y - __high2float(h));
        hi = *reinterpret_cast<const uint32_t *>(&h);
        lo = *reinterpret_cast<const uint32_t *>(&l);
    } else {
        const __half2 h = __floats2half2_rn(x, y);
        const __half2 l = __floats2half2_rn(x - __low2float(h), y - __high2float(h));
        hi = *reinterpret_cast<const uint32_t *>(&h);
        lo = *reinterpret_cast<const uint32_t *>(&l);
    }
}

// What two bfloat16 terms leave of a pair, rounded to a third (exact for fp32 inputs: 24 bits in three terms of 8).
__device__ __forceinline__ uint32_t third_term(float x, float y, uint32_t hi, uint32_t lo) {
    const float a = x - __uint_as_float(hi << 16) - __uint_as_float(lo << 16);
    const float b = y - __uint_as_float(hi & 0xFFFF0000u) - __uint_as_float(lo & 0xFFFF0000u);
    const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&t);
}

// A thread's four elements of a 16-element chunk of queries, as loaded: i .. i + 3 (GAP 2) or i, i + 1 and GAP further.
// fp32 takes four words, the 16-bit types the first two. Loading and converting are apart, so that the loads' latency
// passes under the start of the cache's copies.
template <int GAP> __device__ __forceinline__ void load_q(const void *p, int dt, int64_t i, uint32_t *x) {
    if (dt == DT_F32) {
        const uint32_t *q = static_cast<const uint32_t *>(p) + i;
        if (GAP == 2) {
            const uint4 v = *reinterpret_cast<const uint4 *>(q);
            x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
        } else {
            const uint2 v = *reinterpret_cast<const uint2 *>(q), u = *reinterpret_cast<const uint2 *>(q + GAP);
            x[0] = v.x, x[1] = v.y, x[2] = u.x, x[3] = u.y;
        }
    } else {
        const uint16_t *q = static_cast<const uint16_t *>(p) + i;
        if (GAP == 2) {
            const uint2 v = *reinterpret_cast<const uint2 *>(q);
            x[0] = v.x, x[1] = v.y;
        } else {
            x[0] = *reinterpret_cast<const uint32_t *>(q);
            x[1] = *reinterpret_cast<const uint32_t *>(q + GAP);
        }
    }
}
__device__ __forceinline__ void convert_q(int dt, uint32_t *w, float *x) {
    if (dt == DT_F32) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(w[e]);
    } else if (dt == DT_F16) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = h2f_bits(uint16_t(e & 1 ? w[e / 2] >> 16 : w[e / 2] & 0xFFFFu));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
    }
}

// N = 1, 2 or 4 consecutive outputs, rounded once.
template <int N> __device__ __forceinline__ void store_out(void *p, int dt, int64_t i, const float *x) {
    if (dt == DT_F32) {
        float *o = static_cast<float *>(p) + i;
        if (N == 4) *reinterpret_cast<float4 *>(o) = make_float4(x[0], x[1], x[2], x[3]);
        else if (N == 2) *reinterpret_cast<float2 *>(o) = make_float2(x[0], x[1]);
        else *o = x[0];
        return;
    }
    uint16_t h[N];
#pragma unroll
    for (int e = 0; e < N; ++e) h[e] = dt == DT_F16 ? f2h_bits(x[e]) : __bfloat16_as_ushort(__float2bfloat16_rn(x[e]));
    uint16_t *o = static_cast<uint16_t *>(p) + i;
    if (N == 4)
        *reinterpret_cast<uint2 *>(o) = make_uint2(h[0] | uint32_t(h[1 % N]) << 16, h[2 % N] | uint32_t(h[3 % N]) << 16);
    else if (N == 2) *reinterpret_cast<uint32_t *>(o) = h[0] | uint32_t(h[1 % N]) << 16;
    else *o = h[0];
}

// A row's tokens [lo, len), its tiles from the multiple of TOK below lo.
struct Row {
    const int *table;
    unsigned lo, len, base;
    unsigned tiles;
};

template <int TOK> __device__ __forceinline__ Row row_of(const Params &p, int b, int *fault) {
    Row r;
    const AttendArgs &a = p.a;
    const int seq = a.seqs ? a.seqs[p.row0 + b] : p.row0 + b;
    int64_t len = 0;
    const bool known = seq >= 0 && seq < a.t.seqs;
    bool bad = !known;
    if (known) {
        len = a.t.lens[seq];
        const int64_t cap = int64_t(a.t.max_pages) * a.pool.page_tokens, top = cap < 0x7FFFFFFF ? cap : 0x7FFFFFFF;
        bad = len < 0 || len > top;
        len = len < 0 ? 0 : (len > top ? top : len);
    }
    if (bad && fault) atomicOr(fault, FAULT_PAGE);
    r.table = a.t.tables + (known ? int64_t(seq) * a.t.stride : 0);
    r.len = unsigned(len);
    r.lo = a.window > 0 && len > a.window ? unsigned(len - a.window) : 0u;
    r.base = r.lo / TOK * TOK;
    r.tiles = (r.len - r.base + TOK - 1) / TOK;
    return r;
}

// Shares are cut by work: a segment counts its tiles and SETUP more, the time that its queries and results take a warp
// (shares by tiles alone left blocks with many short segments 1.6 times as long as the others; 90 rows of 0 to 4000
// tokens: 1 37.4 us, 2 34.3, 3 34.2; 3072 segments of up to 40 tokens: 13.6, 13.4, 18.0). Positions ("units") run
// row by row and segment by segment, a segment's SETUP units first. The share of block i: equal pieces of `size` units,
// or (whole) segment i. The host keeps all numbers below 2^31.
constexpr unsigned SETUP = 2;
struct Plan {
    unsigned total, size;
    bool whole;
    int HC;                                                // segments a row
};
// a / b, b > 0. The set-up of a block is a chain of these; by an approximate quotient, put right in integers, each
// takes half as long as the general division.
__device__ __forceinline__ unsigned quot(unsigned a, unsigned b) {
    const float r = __fdividef(1.0f, float(b));
    unsigned q = unsigned(float(a) * r);
    q += int(float(int(a - q * b)) * r);                   // off by at most 2^9 before, by one after
    int rest = int(a - q * b);
    if (rest < 0) --q, rest += b;
    if (rest >= int(b)) ++q;
    return q;
}
// Units of a segment of row b (0: an empty row), and where the segment's begin.
__device__ __forceinline__ unsigned seg_units(const unsigned *cum, int b) { return cum[b + 1] - cum[b]; }
__device__ __forceinline__ unsigned seg_start(const Plan &pl, const unsigned *cum, int b, int hc) {
    return cum[b] * pl.HC + hc * seg_units(cum, b);
}
__device__ __forceinline__ void block_share(const Plan &pl, const unsigned *cum, int B, int i, unsigned &start,
                                            unsigned &end) {
    if (!pl.whole) {
        start = min(unsigned(i) * pl.size, pl.total), end = min(start + pl.size, pl.total);
        return;
    }
    start = end = pl.total;
    if (i >= B * pl.HC) return;
    const int b = quot(i, pl.HC);
    start = seg_start(pl, cum, b, i - b * pl.HC), end = start + seg_units(cum, b);
}
// The blocks that share a segment: the first holds it in its second slot of the workspace, the others, which begin inside
// it, in their first.
__device__ __forceinline__ void sharers(const Plan &pl, const unsigned *cum, int seg, int &first, int &count) {
    const int b = quot(seg, pl.HC);
    const unsigned s0 = seg_start(pl, cum, b, seg - b * pl.HC) + SETUP, n = seg_units(cum, b) - SETUP;    // its tiles
    first = int(quot(s0, pl.size));
    count = int(quot(s0 + n - 1, pl.size)) - first + 1;
}

// Where a tile lies: row, segment of the row, its key/value head and group of query heads, tile of the segment.
struct Cursor {
    int b, hc, h, q;
    unsigned ti;
    Row row;
};
// The first tile at or behind a unit that is not behind the last one.
template <int TOK>
__device__ __forceinline__ void seek(const Params &p, const Plan &pl, const unsigned *cum, unsigned unit, Cursor &c) {
    int lo = 0, hi = p.B;                                  // cum[lo] HC <= unit < cum[hi] HC
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cum[mid] * pl.HC <= unit) lo = mid; else hi = mid;
    }
    c.b = lo;
    c.row = row_of<TOK>(p, lo, nullptr);
    const unsigned rem = unit - cum[lo] * pl.HC, n = c.row.tiles + SETUP;
    c.hc = int(quot(rem, n));
    const unsigned at = rem - c.hc * n;
    c.ti = at > SETUP ? at - SETUP : 0;
    c.h = p.C == 1 ? c.hc : int(quot(c.hc, p.C));
    c.q = c.hc - c.h * p.C;
}
// The next segment; there is one.
template <int TOK>
__device__ __forceinline__ void next_segment(const Params &p, const Plan &pl, const unsigned *cum, Cursor &c) {
    c.ti = 0;
    ++c.hc;
    if (++c.q == p.C) c.q = 0, ++c.h;
    if (c.hc < pl.HC) return;
    c.hc = c.h = c.q = 0;
    int b = c.b + 1;
    while (cum[b + 1] == cum[b]) ++b;
    c.b = b;
    c.row = row_of<TOK>(p, b, nullptr);
}

// 1 / sum, or 0 where no token counted (a sum of NaN stays one).
__device__ __forceinline__ float inverse(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }
__device__ __forceinline__ float finite_base(float m) { return m == -INFINITY ? 0.0f : m; }
__device__ __forceinline__ float lse_of(float m, float l, float bias) {
    return l == 0.0f ? -INFINITY : (m - bias) * 0.6931471805599453f + logf(l);
}

// A triple of one head and four of its accumulators, joined with n <= N others.
struct Triple {
    float m = -INFINITY, l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    template <int N>
    __device__ __forceinline__ void add(const float (&mi)[N], const float (&li)[N], const float4 (&x)[N], int n) {
        float top = m;
#pragma unroll
        for (int i = 0; i < N; ++i) top = i < n ? fmaxf(top, mi[i]) : top;
        const float base = finite_base(top), f = ex2(m - base);
        m = top;
        l *= f, o.x *= f, o.y *= f, o.z *= f, o.w *= f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (i >= n) continue;
            const float h = ex2(mi[i] - base);
            l = fmaf(li[i], h, l);
            o.x = fmaf(x[i].x, h, o.x), o.y = fmaf(x[i].y, h, o.y);
            o.z = fmaf(x[i].z, h, o.z), o.w = fmaf(x[i].w, h, o.w);
        }
    }
};

// A piece of a segment that a warp leaves to the join: where its results go. The piece itself is in the warp's ring, or
// (far) in the workspace where the warp went on to another segment.
struct Piece {
    int64_t out, lse;           // element of the first head's results
    int seg, heads, far;        // segment; heads there are; seg < 0: no piece
};

template <int KT, int D, int NT>
__global__ void __launch_bounds__(Cfg<KT, D, NT>::W * 32, 1) attend_kernel(const __grid_constant__ Params p) {
    using F = Cfg<KT, D, NT>;
    constexpr int W = F::W, STAGES = F::STAGES, TILE = F::TILE, RB = F::RB, SB = F::SB, PS = F::PS, PF = F::PF;
    constexpr int TOK = F::TOK, CPR = RB / 16, CH = D / 16, NH = F::NH, TT = TOK / 8, THREADS = W * 32;
    constexpr bool I8 = KT == QPACK_KV_I8;
    extern __shared__ __align__(128) unsigned char smem[];
    // behind the rings: third terms, and the units before row b (of one segment a row)
    unsigned *cum = reinterpret_cast<unsigned *>(smem + W * (STAGES * TILE + F::Q3));
    __shared__ Piece s_piece[2 * W];
    __shared__ float s_m[2 * W][NH], s_l[2 * W][NH];       // a piece's maxima and sums
    __shared__ int s_runs[W][2 * W];                       // a warp's list of runs, by their first pieces
    __shared__ unsigned s_max;
    const AttendArgs &a = p.a;
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, j = lane & 3;
    const int T = a.pool.page_tokens, shift = 31 - __clz(T);

    pdl_launch_dependents();
    // Inputs, cache and workspace may be the previous grid's, lengths and tables among them: none of what is loaded below is
    // read-only for as long as this grid lives, and all of it is read by plain loads.
    pdl_wait();

    // -- the rows' tiles, and this block's share of them ------------------------------------------------------
    // Up to 32 rows are added up by every warp for itself (all write the same sums): no barrier before the copies (one
    // row of 2000 tokens 9.3 us instead of 9.9; more rows would be a longer loop in every warp).
    if (lane < 2) s_piece[2 * w + lane].seg = -1;
    const bool few = p.B <= 32;
    int *fault = blockIdx.x == 0 && (w == 0 || !few) ? &g_fault_attend : nullptr;
    if (!few) {
        for (int b = tid; b < p.B; b += THREADS) cum[b + 1] = row_of<TOK>(p, b, fault).tiles;
        __syncthreads();
    }
    unsigned longest = 0;                                  // tiles of the longest row
    if (few || w == 0) {
        unsigned carry = 0;
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            const int b = b0 + lane;
            unsigned x = b >= p.B ? 0u : few ? row_of<TOK>(p, b, fault).tiles : cum[b + 1];
            longest = max(longest, x);
            x = x ? x + SETUP : 0u;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            x += carry;
            if (b < p.B) cum[b + 1] = x;
            carry = __shfl_sync(0xffffffffu, x, 31);
        }
        longest = __reduce_max_sync(0xffffffffu, longest);
        if (lane == 0) cum[0] = 0, s_max = longest;
        __syncwarp();
    }
    if (!few) {
        __syncthreads();
        longest = s_max;
    }
    Plan pl;
    const unsigned grid = gridDim.x;
    pl.HC = a.pool.heads * p.C;
    pl.total = cum[p.B] * pl.HC;
    pl.size = max(quot(pl.total + grid - 1, grid), unsigned(W));        // at least a unit a warp
    // A block a segment, where there are blocks enough and the longest segment takes no more time than the equal shares and
    // the joins between blocks that they need (2.5 us, in which a block reads 112 KB): 112 segments of up to 1024 tokens
    // 13.6 us instead of 14.7, 144 of up to 4096 33.4 instead of 35.6; 112 of up to 4096 stay with equal shares, 29.9
    // instead of 32.5.
    pl.whole = p.B * pl.HC <= int(grid) && longest <= pl.size + 112 * 1024 / TILE;
    for (int b = blockIdx.x; b < p.B; b += grid) {
        if (cum[b + 1] != cum[b]) continue;                // an empty row
        const float zero = 0.0f;
        for (int i = tid; i < a.q_heads * D; i += THREADS)
            store_out<1>(a.out, a.odt, int64_t(p.row0 + b) * a.ldo + i, &zero);
        if (a.lse)
            for (int i = tid; i < a.q_heads; i += THREADS) a.lse[int64_t(p.row0 + b) * a.q_heads + i] = -INFINITY;
    }
    unsigned start, end;
    block_share(pl, cum, p.B, blockIdx.x, start, end);
    if (start >= end) return;

    // -- this warp's share -------------------------------------------------------------------------------------
    unsigned char *ring = smem + w * STAGES * TILE;
    const unsigned share = (end - start + W - 1) / W, w0 = min(start + w * share, end), w1 = min(w0 + share, end);
    Cursor ci;
    int nt = 0;                                            // its tiles
    if (w0 < w1) {
        seek<TOK>(p, pl, cum, w0, ci);
        // segments whose tiles the units [w0, w1) reach, from the first one's row on
        unsigned u = seg_start(pl, cum, ci.b, ci.hc) + SETUP;
        int b = ci.b, hc = ci.hc;
        for (;;) {
            const unsigned n = seg_units(cum, b) - SETUP, from = max(u, w0), to = min(u + n, w1);
            if (to > from) nt += to - from;
            if (u + n >= w1) break;
            u += n + SETUP;                                // the next segment's tiles; there is one, since w1 is behind it
            if (++hc == pl.HC) {
                hc = 0;
                do ++b; while (seg_units(cum, b) == 0);
            }
        }
    }
    if (nt > 0) {
        const uint32_t ring32 = smem_u32(ring);
        Cursor cc = ci;

        // The page of the tile, or of lane's token of it where pages are smaller than a tile; loaded a tile ahead of its
        // use.
        const bool large = T >= TOK;
        auto page_of = [&](const Cursor &c) {
            const unsigned t = c.row.base + c.ti * TOK + (large ? 0 : lane % TOK);
            return large || (t >= c.row.lo && t < c.row.len) ? c.row.table[t >> shift] : -1;
        };
        int entry = page_of(ci);
        // Starts the copies of the cursor's tile into a stage: chunk i * 32 + lane of the tile goes to its row, at its
        // place in the row xor the row's number, so that ldmatrix's eight rows meet different banks. Rows outside
        // [lo, len) and of pages outside the pool are filled with zeros.
        constexpr bool SWZ = RB % 128 == 0;
        const int r0 = lane / CPR;
        const uint32_t sw0 = r0 * RB + (((lane % CPR) ^ (SWZ ? r0 & 7 : (r0 >> 1) & 3)) << 4);
        const unsigned char *kbase = static_cast<const unsigned char *>(a.pool.k) + a.layer * a.pool.layer_stride * F::ES;
        const unsigned char *vbase = static_cast<const unsigned char *>(a.pool.v) + a.layer * a.pool.layer_stride * F::ES;
        const uint16_t *ksbase = I8 ? a.pool.k_scales + a.layer * a.pool.scale_layer_stride : nullptr;
        const uint16_t *vsbase = I8 ? a.pool.v_scales + a.layer * a.pool.scale_layer_stride : nullptr;
        auto issue = [&](uint32_t dst) {
            const unsigned t0 = ci.row.base + ci.ti * TOK;
            if (large && t0 >= ci.row.lo && ci.row.len - t0 >= TOK && unsigned(entry) < unsigned(a.pool.pages)) {
                // a whole tile of one page: consecutive rows
                const unsigned row = unsigned(ci.h * T) + (t0 & (T - 1));
                const int64_t at = (int64_t(entry) * a.pool.page_stride + row * unsigned(D)) * F::ES + lane * 16;
                const unsigned char *ks = kbase + at, *vs = vbase + at;
#pragma unroll
                for (int i = 0; i < TOK * CPR / 32; ++i) {
                    const uint32_t to = dst + i * 512 + (sw0 ^ (SWZ ? ((i * 32 / CPR) & 7) << 4 : 0));
                    cp16(to, ks + i * 512);
                    cp16(to + TOK * RB, vs + i * 512);
                }
                if (I8) {
                    const int64_t sat = int64_t(entry) * a.pool.scale_page_stride + (row + lane % TOK) * unsigned(D / 32);
                    const uint32_t to = dst + 2 * TOK * RB + lane * SB;
                    if (TOK == 32) {
                        cp_small<SB ? SB : 16>(to, ksbase + sat, true);
                        cp_small<SB ? SB : 16>(to + TOK * SB, vsbase + sat, true);
                    } else {
                        cp_small<SB ? SB : 16>(to, (lane < 16 ? ksbase : vsbase) + sat, true);
                    }
                }
            } else {
                const unsigned mine = t0 + lane % TOK;
                const bool in = mine >= ci.row.lo && mine < ci.row.len;
                const bool ok = in && unsigned(entry) < unsigned(a.pool.pages);
                if (in && !ok) atomicOr(&g_fault_attend, FAULT_PAGE);
                const unsigned okmask = __ballot_sync(0xffffffffu, ok);
                const int page = ok ? entry : 0;
                const unsigned slot = unsigned(ci.h * T) + (mine & (T - 1));
                const int64_t row = int64_t(page) * a.pool.page_stride + slot * unsigned(D);
                constexpr int HALF = TOK * CPR / 64;       // copies of half a tile
                if (TOK == 32 && T == 16 && okmask == 0xffffffffu) {
                    // a whole tile of two pages, the most common of the small ones: two runs of rows (48 rows of up to
                    // 8192 tokens 108.6 us instead of 113.9; with pages of 64 107.9)
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        const int64_t at = __shfl_sync(0xffffffffu, row, 16 * v) * F::ES + lane * 16;
                        const unsigned char *ks = kbase + at, *vs = vbase + at;
#pragma unroll
                        for (int i = 0; i < HALF; ++i) {
                            const int n = v * HALF + i;
                            const uint32_t to = dst + n * 512 + (sw0 ^ (SWZ ? ((n * 32 / CPR) & 7) << 4 : 0));
                            cp16(to, ks + i * 512);
                            cp16(to + TOK * RB, vs + i * 512);
                        }
                    }
                } else {
#pragma unroll 4
                    for (int i = 0; i < TOK * CPR / 32; ++i) {
                        const int idx = i * 32 + lane, r = idx / CPR, c = idx % CPR;
                        const int64_t off = __shfl_sync(0xffffffffu, row, r) * F::ES + c * 16;
                        const bool live = (okmask >> r) & 1;
                        const uint32_t to = dst + i * 512 + (sw0 ^ (SWZ ? ((i * 32 / CPR) & 7) << 4 : 0));
                        cp16(to, kbase + off, live);
                        cp16(to + TOK * RB, vbase + off, live);
                    }
                }
                if (I8) {
                    const int64_t sat = int64_t(page) * a.pool.scale_page_stride + slot * unsigned(D / 32);
                    const uint32_t to = dst + 2 * TOK * RB + lane * SB;
                    if (TOK == 32) {
                        cp_small<SB ? SB : 16>(to, ksbase + sat, ok);
                        cp_small<SB ? SB : 16>(to + TOK * SB, vsbase + sat, ok);
                    } else {
                        cp_small<SB ? SB : 16>(to, (lane < 16 ? ksbase : vsbase) + sat, ok);
                    }
                }
            }
        };
        int left = nt;                                     // tiles to issue
        auto advance = [&](int slot) {
            if (left > 0) {
                issue(ring32 + slot * TILE);
                if (--left) {
                    if (++ci.ti == ci.row.tiles) next_segment<TOK>(p, pl, cum, ci);
                    entry = page_of(ci);
                }
            }
            cp_commit();
        };

        // ldmatrix: lane addresses row lr of 16 tokens, chunk (even) + lane / 16
        const int lr = (lane & 7) + (lane & 8), lx = ((lane >> 4) ^ (SWZ ? lr & 7 : (lr >> 1) & 3)) << 4;
        constexpr int gap = I8 ? 2 : 8;                    // a thread's elements of a chunk: d0, + 1, + gap, + gap + 1
        const int d0 = I8 ? 4 * j : 2 * j;
        int slot = 0;
        for (int done = 0; done < nt;) {
            // -- a segment begins: its queries, rotated, scaled and split ---------------------------------------
            const bool whole = cc.ti == 0;
            const int count = min(int(cc.row.tiles - cc.ti), nt - done);
            uint32_t qf[CH][4 * NT];
            constexpr bool THREE = F::THREE;
            uint32_t *q3 = reinterpret_cast<uint32_t *>(smem + W * STAGES * TILE + w * F::Q3) + lane;
            bool third = false;                            // whether any query of the segment has a third term
            float qs[NT], m[NT], l[NT], mx[NT], acc[CH][NT][4];
            {
                uint32_t raw[NT][CH][4];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int head = cc.q * NH + 8 * n + g;
                    const int64_t at = int64_t(p.row0 + cc.b) * a.ldq + int64_t(cc.h * p.G + head) * D + d0;
#pragma unroll
                    for (int c = 0; c < CH; ++c) {
                        raw[n][c][0] = raw[n][c][1] = raw[n][c][2] = raw[n][c][3] = 0u;
                        if (head < p.G) load_q<gap>(a.q, a.qdt, at + 16 * c, raw[n][c]);
                    }
                }
                const int64_t pos = int64_t(cc.row.len) - 1;
                const bool turn = a.rope && pos < a.rope_rows;
                if (a.rope && !turn) atomicOr(&g_fault_attend, FAULT_PAGE);
                float2 co[CH / 2][2], si[CH / 2][2];
                auto fetch_rotation = [&] {
                    if (!turn) return;
                    const float *row = a.rope + pos * D + d0;
#pragma unroll
                    for (int c = 0; c < CH / 2; ++c)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            co[c][e] = *reinterpret_cast<const float2 *>(row + 16 * c + e * gap);
                            si[c][e] = *reinterpret_cast<const float2 *>(row + D / 2 + 16 * c + e * gap);
                        }
                };
                // The cache's copies are started behind these loads: before them, they held them up (by 2 us, of which
                // one was lost to the copies behind). Where the registers do not hold both, the rotation comes later.
                constexpr bool both = D * NT <= 128;
                if (both) fetch_rotation();
                if (done == 0) {
#pragma unroll
                    for (int st = 0; st < STAGES - 1; ++st) advance(st);
                }
                if (!both) fetch_rotation();
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    m[n] = mx[n] = -INFINITY;
                    l[n] = 0.0f;
                    float x[CH][4];
#pragma unroll
                    for (int c = 0; c < CH; ++c) convert_q(a.qdt, raw[n][c], x[c]);
                    if (turn) {
#pragma unroll
                        for (int c = 0; c < CH / 2; ++c)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float cs = e & 1 ? co[c][e >> 1].y : co[c][e >> 1].x;
                                const float sn = e & 1 ? si[c][e >> 1].y : si[c][e >> 1].x;
                                const float u = x[c][e], v = x[c + CH / 2][e];
                                x[c][e] = __fsub_rn(__fmul_rn(u, cs), __fmul_rn(v, sn));
                                x[c + CH / 2][e] = __fadd_rn(__fmul_rn(v, cs), __fmul_rn(u, sn));
                            }
                    }
                    float big = 0.0f;
#pragma unroll
                    for (int c = 0; c < CH; ++c)
#pragma unroll
                        for (int e = 0; e < 4; ++e) big = fmaxf(big, fabsf(x[c][e]));
                    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
                    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
                    // 2^(13 - exponent of the maximum), within fp32's normal range; 1 for zero, inf and NaN, and for bfloat16
                    // terms. The scale's sign goes with it, so that the largest score is the largest sum.
                    const int ex = __float_as_int(big) >> 23;
                    const int up = KT == QPACK_KV_BF16 || big == 0.0f || ex == 255 ? 127 : min(254, 267 - ex);
                    const float f = __int_as_float((up << 23) | (__float_as_int(a.scale) & 0x80000000));
                    const float back = __int_as_float(max(254 - up, 1) << 23);
                    qs[n] = fabsf(a.scale) * 1.4426950408889634f * back * (up == 254 ? 0.5f : 1.0f);
                    if (qs[n] == 0.0f) qs[n] = 0x1p-126f;   // a masked token's -inf stays one where the scale is 0
#pragma unroll
                    for (int c = 0; c < CH; ++c) {
                        uint32_t h0, l0, h1, l1;
                        split2<KT>(x[c][0] * f, x[c][1] * f, h0, l0);
                        split2<KT>(x[c][2] * f, x[c][3] * f, h1, l1);
                        if constexpr (NT == 1)
                            qf[c][0] = h0, qf[c][1] = l0, qf[c][2] = h1, qf[c][3] = l1;
                        else
                            qf[c][n] = h0, qf[c][2 + n] = h1, qf[c][4 + n] = l0, qf[c][6 + n] = l1;
                        if constexpr (THREE) {
                            const uint32_t t0 = third_term(x[c][0] * f, x[c][1] * f, h0, l0);
                            const uint32_t t1 = third_term(x[c][2] * f, x[c][3] * f, h1, l1);
                            q3[(c * 2 * NT + n) * 32] = t0;
                            q3[(c * 2 * NT + NT + n) * 32] = t1;
                            third |= ((t0 | t1) & 0x7FFF7FFFu) != 0;
                        }
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[c][n][r] = 0.0f;
                    }
                }
                if (THREE) third = __any_sync(0xffffffffu, third);
            }
            unsigned t0 = cc.row.base + cc.ti * TOK;
            for (int k = 0; k < count; ++k, t0 += TOK) {
                cp_wait<STAGES - 2>();
                __syncwarp();                              // the tile is there, and the stage before it is read
                advance(slot == 0 ? STAGES - 1 : slot - 1);
                const uint32_t st = ring32 + slot * TILE + lr * RB;
                const unsigned char *sk = ring + slot * TILE + 2 * TOK * RB, *sv = sk + TOK * SB;
                slot = slot + 1 == STAGES ? 0 : slot + 1;

                // -- scores ---------------------------------------------------------------------------------
                // The accumulators of the tile's eights of tokens (and with NT = 2 of leading terms and remainders) take
                // turns, so that no product waits for the one before it.
                float sc[TT][4], sl[TT][4];
#pragma unroll
                for (int t = 0; t < TT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[t][e] = sl[t][e] = 0.0f;
                uint32_t sw[TT][SB ? SB / 4 : 1];
                if (I8) {
#pragma unroll
                    for (int t = 0; t < TT; ++t) load_words<SB ? SB : 4>(sk + (g + 8 * t) * SB, sw[t]);
                }
#pragma unroll
                for (int c = 0; c < CH; c += I8 ? 2 : 1) {
#pragma unroll
                    for (int u = 0; u < TOK / 16; ++u) {
                        uint32_t r[4];
                        ldsm4((st + u * 16 * RB) + ((c * 16 * F::ES) ^ lx), r);
#pragma unroll
                        for (int v = 0; v < (I8 ? 2 : 1); ++v) {
                            const uint32_t *q = qf[c + v];
#pragma unroll
                            for (int t = 0; t < 2; ++t) {
                                uint32_t b0 = r[t], b1 = r[2 + t];
                                if constexpr (I8) {
                                    const uint32_t odd = (c / 2) & 1 ? 0x3232u : 0x1010u;
                                    const uint32_t s = __byte_perm(sw[2 * u + t][c / 4], 0u, odd);
                                    const uint32_t word = r[2 * v + t] ^ 0x80808080u;
                                    b0 = dequant2(word, 0x4140u, s), b1 = dequant2(word, 0x4342u, s);
                                }
                                mma<KT>(sc[2 * u + t], q[0], q[1], q[2], q[3], b0, b1);
                                if constexpr (NT == 2) mma<KT>(sl[2 * u + t], q[4], q[5], q[6], q[7], b0, b1);
                            }
                        }
                    }
                }
                if (THREE && third) {
#pragma unroll
                    for (int c = 0; c < CH; ++c)
#pragma unroll
                        for (int u = 0; u < TOK / 16; ++u) {
                            uint32_t r[4];
                            ldsm4((st + u * 16 * RB) + ((c * 16 * F::ES) ^ lx), r);
                            const uint32_t *q = q3 + c * 2 * NT * 32;      // a lane reads what it wrote
                            const uint32_t a0 = q[0], a2 = q[NT * 32];
                            const uint32_t a1 = NT == 2 ? q[32] : 0u, a3 = NT == 2 ? q[(2 * NT - 1) * 32] : 0u;
#pragma unroll
                            for (int t = 0; t < 2; ++t) mma<KT>(sl[2 * u + t], a0, a1, a2, a3, r[t], r[2 + t]);
                        }
                }
                if (NT == 2 || THREE) {
#pragma unroll
                    for (int t = 0; t < TT; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sc[t][e] += sl[t][e];
                }

                // -- softmax --------------------------------------------------------------------------------
                // s[n][2 t + e]: head g of group n, token 8 t + 2 j + e, before the factor qs > 0. The maximum m is held before
                // it too, and taken off first: the largest score's weight is then 2^12 without an error, so that a lone
                // token's value comes back unchanged, and none is larger, however large the scores are. mx is m with the
                // factor, for the joins: multiplied there instead, a call took 0.5 us more (one row of 2000 tokens 9.8 us).
                float s[NT][2 * TT];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2 * TT; ++e)
                        s[n][e] = NT == 1 ? sc[e >> 1][e & 1] + sc[e >> 1][2 + (e & 1)] : sc[e >> 1][2 * n + (e & 1)];
                if (t0 < cc.row.lo || cc.row.len - t0 < TOK) {
#pragma unroll
                    for (int e = 0; e < 2 * TT; ++e) {
                        const unsigned t = t0 + 8 * (e >> 1) + 2 * j + (e & 1);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            if (t < cc.row.lo || t >= cc.row.len) s[n][e] = -INFINITY;
                    }
                }
                bool up = false;
                float mt[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float x = s[n][0];
#pragma unroll
                    for (int e = 1; e < 2 * TT; ++e) x = fmaxf(x, s[n][e]);
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                    mt[n] = fmaxf(x, m[n]);
                    up |= mt[n] > m[n];
                }
                if (__any_sync(0xffffffffu, up)) {         // rare after the first tiles
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float nx = mt[n] * qs[n], f = ex2(mx[n] - finite_base(nx));
                        m[n] = mt[n], mx[n] = nx;
                        l[n] *= f;
                        const float f0 = __shfl_sync(0xffffffffu, f, 8 * j), f1 = __shfl_sync(0xffffffffu, f, 8 * j + 4);
#pragma unroll
                        for (int c = 0; c < CH; ++c) {
                            acc[c][n][0] *= f0;
                            acc[c][n][1] *= f1;
                            acc[c][n][2] *= f0;
                            acc[c][n][3] *= f1;
                        }
                    }
                }
                uint32_t ph[NT][TT], plo[NT][TT];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float top = finite_base(m[n]);
                    float sum = 0.0f;
#pragma unroll
                    for (int e = 0; e < 2 * TT; ++e) {
                        s[n][e] = ex2(fmaf(s[n][e] - top, qs[n], F::P_BIAS));
                        sum += s[n][e];
                    }
                    l[n] += sum;
#pragma unroll
                    for (int t = 0; t < TT; ++t) split2<KT>(s[n][2 * t], s[n][2 * t + 1], ph[n][t], plo[n][t]);
                }

                // -- values ---------------------------------------------------------------------------------
                if (THREE && a.odt == DT_F32) {
                    // what two bfloat16 terms leave of the probabilities, where the output keeps more than their 16 bits
#pragma unroll
                    for (int u = 0; u < TOK / 16; ++u) {
                        uint32_t pt[NT][2];
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int t = 0; t < 2; ++t)
                                pt[n][t] = third_term(s[n][4 * u + 2 * t], s[n][4 * u + 2 * t + 1], ph[n][2 * u + t], plo[n][2 * u + t]);
#pragma unroll
                        for (int c = 0; c < CH; ++c) {
                            uint32_t r[4];
                            ldsm4_t((st + (TOK + u * 16) * RB) + ((c * 16 * F::ES) ^ lx), r);
#pragma unroll
                            for (int n = 0; n < NT; ++n) mma<KT>(acc[c][n], r[0], r[2], r[1], r[3], pt[n][0], pt[n][1]);
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < TOK / 16; ++u) {
                    if (I8) {
                        // scales of tokens 2j and 2j + 1, and of 2j + 8 and 2j + 9: rows next to each other
                        uint32_t va[2][SB ? SB / 2 : 1];
#pragma unroll
                        for (int t = 0; t < 2; ++t) load_words<SB ? 2 * SB : 4>(sv + (2 * j + 8 * t + 16 * u) * SB, va[t]);
#pragma unroll
                        for (int c = 0; c < CH; c += 2) {
                            uint32_t r[4];
                            ldsm4_t((st + (TOK + u * 16) * RB) + ((c * 16) ^ lx), r);
                            const uint32_t sel = (c / 2) & 1 ? 0x7632u : 0x5410u;
                            const uint32_t s0 = __byte_perm(va[0][c / 4], va[0][(SB ? SB / 4 : 0) + c / 4], sel);
                            const uint32_t s1 = __byte_perm(va[1][c / 4], va[1][(SB ? SB / 4 : 0) + c / 4], sel);
#pragma unroll
                            for (int v = 0; v < 2; ++v) {
                                const uint32_t x0 = r[2 * v] ^ 0x80808080u, x1 = r[2 * v + 1] ^ 0x80808080u;
                                const uint32_t a0 = dequant2(x0, 0x4240u, s0), a1 = dequant2(x0, 0x4341u, s0);
                                const uint32_t a2 = dequant2(x1, 0x4240u, s1), a3 = dequant2(x1, 0x4341u, s1);
#pragma unroll
                                for (int n = 0; n < NT; ++n) {
                                    mma<KT>(acc[c + v][n], a0, a1, a2, a3, ph[n][2 * u], ph[n][2 * u + 1]);
                                    mma<KT>(acc[c + v][n], a0, a1, a2, a3, plo[n][2 * u], plo[n][2 * u + 1]);
                                }
                            }
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < CH; ++c) {
                            uint32_t r[4];
                            ldsm4_t((st + (TOK + u * 16) * RB) + ((c * 32) ^ lx), r);
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                mma<KT>(acc[c][n], r[0], r[2], r[1], r[3], ph[n][2 * u], ph[n][2 * u + 1]);
                                mma<KT>(acc[c][n], r[0], r[2], r[1], r[3], plo[n][2 * u], plo[n][2 * u + 1]);
                            }
                        }
                    }
                }
            }

            // -- the segment's end, or the share's --------------------------------------------------------------
            const bool ended = cc.ti + count == cc.row.tiles, last = done + count == nt;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                l[n] += __shfl_xor_sync(0xffffffffu, l[n], 1);
                l[n] += __shfl_xor_sync(0xffffffffu, l[n], 2);
            }
            // a thread's elements: heads 8 n + 2 j + (r & 1), d = 16 c + 2 g + (r >> 1) or 16 c + g + 8 (r >> 1)
            constexpr int gd = I8 ? 2 : 1, rd = I8 ? 1 : 8;
            if (ended && whole) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float inv = inverse(l[n]);
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float f = __shfl_sync(0xffffffffu, inv, 8 * j + 4 * r);
                        const int head = cc.q * NH + 8 * n + 2 * j + r;
                        if (head < p.G) {
                            const int64_t at = int64_t(p.row0 + cc.b) * a.ldo + int64_t(cc.h * p.G + head) * D + gd * g;
#pragma unroll
                            for (int c = 0; c < CH; ++c) {
                                const float o[2] = {acc[c][n][r] * f, acc[c][n][2 + r] * f};
                                if (I8) {
                                    store_out<2>(a.out, a.odt, at + 16 * c, o);
                                } else {
                                    store_out<1>(a.out, a.odt, at + 16 * c, o);
                                    store_out<1>(a.out, a.odt, at + 16 * c + 8, o + 1);
                                }
                            }
                        }
                    }
                    const int head = cc.q * NH + 8 * n + g;
                    if (a.lse && j == 0 && head < p.G)
                        a.lse[int64_t(p.row0 + cc.b) * a.q_heads + cc.h * p.G + head] = lse_of(mx[n], l[n], F::P_BIAS);
                }
            } else {
                // The first of two pieces waits in global memory (the ring is in use), the last one in the ring.
                if (last) {
                    cp_wait<0>();
                    __syncwarp();
                }
                const int at = 2 * w + (done == 0 ? 0 : 1);
                float *dst = last ? reinterpret_cast<float *>(ring) : p.warp_parts + (int64_t(blockIdx.x) * W + w) * PF;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int c = 0; c < CH; ++c)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            dst[(8 * n + 2 * j + (r & 1)) * PS + 16 * c + gd * g + rd * (r >> 1)] = acc[c][n][r];
                    if (j == 0) s_m[at][8 * n + g] = mx[n], s_l[at][8 * n + g] = l[n];
                }
                if (lane == 0) {
                    const int head = cc.h * p.G + cc.q * NH;
                    s_piece[at] = {int64_t(p.row0 + cc.b) * a.ldo + int64_t(head) * D,
                                   int64_t(p.row0 + cc.b) * a.q_heads + head, cc.b * pl.HC + cc.hc,
                                   min(NH, p.G - cc.q * NH), last ? 0 : 1};
                }
            }
            done += count;
            if (!last) next_segment<TOK>(p, pl, cum, cc);
        }
        cp_wait<0>();
    }
    __syncthreads();

    // -- joins ------------------------------------------------------------------------------------------------
    // Pieces in the order of their tiles, one a lane, runs of one segment among them; every warp finds the runs for
    // itself. A run that leaves the block's share (the first and the last may) goes to the workspace, the others are
    // finished. Of a run's pieces only the last can be far.
    const int seg = lane < 2 * W ? s_piece[lane].seg : -1;
    const unsigned valid = __ballot_sync(0xffffffffu, seg >= 0), below = valid & ((1u << lane) - 1u);
    if (!valid) return;
    const int prev = __shfl_sync(0xffffffffu, seg, below ? 31 - __clz(below) : 0);
    const bool begins = seg >= 0 && (!below || prev != seg);
    const unsigned starts = __ballot_sync(0xffffffffu, begins);
    const unsigned far = __ballot_sync(0xffffffffu, seg >= 0 && s_piece[lane < 2 * W ? lane : 0].far);
    bool before_me = false, outside = false;               // the segment begins before this block's share; leaves it
    if (begins) {
        const int b = quot(seg, pl.HC);
        const unsigned s0 = seg_start(pl, cum, b, seg - b * pl.HC);
        before_me = s0 + SETUP < start;
        outside = before_me || s0 + seg_units(cum, b) > end;
    }
    const unsigned outer = __ballot_sync(0xffffffffu, outside), early = __ballot_sync(0xffffffffu, before_me);
    int *s_run = s_runs[w];
    if (begins) s_run[__popc(starts & ((1u << lane) - 1u))] = lane;
    __syncwarp();
    constexpr int VEC = F::VEC;
    auto finish = [&](const Piece &pc, int head, int d, const Triple &t) {
        if (head >= pc.heads) return;
        const float f = inverse(t.l);
        const float x[4] = {t.o.x * f, t.o.y * f, t.o.z * f, t.o.w * f};
        store_out<4>(a.out, a.odt, pc.out + head * D + d, x);
        if (a.lse && d == 0) a.lse[pc.lse + head] = lse_of(t.m, t.l, F::P_BIAS);
    };
    const int todo = __popc(starts) * VEC;
    int left_base = 0, left_n = 0;                         // lane k: where the warp's k-th part that leaves the block is
    for (int i = tid; i < todo; i += THREADS) {
        const int p0 = s_run[i / VEC], e = i % VEC, head = e / (D / 4), d = e % (D / 4) * 4;
        const unsigned later = starts & ~((2u << p0) - 1u);
        const unsigned members = valid & ~((1u << p0) - 1u) & (later ? (later & -later) - 1u : 0xffffffffu);
        const int tail = 31 - __clz(members), away = (far >> tail) & 1, n = __popc(members) - away;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (away) {
            const float *far_part = p.warp_parts + (int64_t(blockIdx.x) * W + (tail >> 1)) * PF;
            o = *reinterpret_cast<const float4 *>(far_part + head * PS + d);
        }
        Triple t;
        for (int k0 = 0; k0 < n; k0 += 4) {                // the run's first piece, then one of each of the next warps
            float mi[4], li[4];
            float4 x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int at = k0 + k ? ((p0 >> 1) + min(k0 + k, n - 1)) * 2 : p0;
                mi[k] = s_m[at][head], li[k] = s_l[at][head];
                x[k] = *reinterpret_cast<const float4 *>(smem + (at >> 1) * STAGES * TILE + (head * PS + d) * 4);
            }
            t.add(mi, li, x, n - k0);
        }
        if (away) {
            const float mi[1] = {s_m[tail][head]}, li[1] = {s_l[tail][head]};
            const float4 x[1] = {o};
            t.add(mi, li, x, 1);
        }
        if (!((outer >> p0) & 1)) {
            finish(s_piece[p0], head, d, t);
            continue;
        }
        // A part for the workspace. A segment's first block has it in its second slot, the others, which begin inside the
        // segment, in their first.
        const int64_t mine = (int64_t(blockIdx.x) * 2 + ((early >> p0) & 1 ? 0 : 1)) * VEC + e;
        p.block_parts[mine] = t.o;
        p.block_sums[mine] = make_float2(t.m, t.l);
        if (lane == left_n) left_base = i - lane;
        ++left_n;
    }
    if (!left_n) return;
    // The segments' other blocks: each of the join's warps is on its own with its 32 x 4 accumulators of a segment. The
    // last of the blocks' warps to arrive joins them all, in the order of the blocks.
    __syncwarp();
    int first = 0, count = 0;
    bool am_last = false;
    if (lane < left_n) {
        const int s = s_piece[s_run[left_base / VEC]].seg;
        sharers(pl, cum, s, first, count);
        int *counter = p.counters + int64_t(s) * F::SLICES + left_base % VEC / 32, before;
        // releases the warp's part, acquires those that came before
        asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
        am_last = before == count - 1;
        if (am_last) *counter = 0;                         // ready for the next call
    }
    __syncwarp();
    for (unsigned mask = __ballot_sync(0xffffffffu, am_last); mask; mask &= mask - 1) {
        const int from = __ffs(mask) - 1, i = __shfl_sync(0xffffffffu, left_base, from) + lane;
        const int f0 = __shfl_sync(0xffffffffu, first, from), n = __shfl_sync(0xffffffffu, count, from);
        const int e = i % VEC, head = e / (D / 4), d = e % (D / 4) * 4;
        Triple t;
        // Loads in flight together: few segments over many blocks have up to ten in a round; the usual two or three parts
        // are not kept waiting by the longer code (1 to 3 us, mostly of fetching instructions).
        auto gather = [&](auto loads) {
            constexpr int L = decltype(loads)::value;
            for (int i0 = 0; i0 < n; i0 += L) {
                float mi[L], li[L];
                float4 x[L];
#pragma unroll
                for (int k = 0; k < L; ++k) {
                    if (i0 + k >= n) continue;
                    const int64_t at = (int64_t(f0 + i0 + k) * 2 + (i0 + k == 0 ? 1 : 0)) * VEC + e;
                    const float2 ml = __ldcg(p.block_sums + at);
                    mi[k] = ml.x, li[k] = ml.y;
                    x[k] = __ldcg(p.block_parts + at);
                }
                t.add(mi, li, x, n - i0);
            }
        };
        if (n <= 4) gather(Int<4>());
        else gather(Int<7>());
        finish(s_piece[s_run[i / VEC]], head, d, t);
    }
}

// -- host -------------------------------------------------------------------------------------------------------
// Groups of eight query heads a block takes together: two where a key head has more than eight and the registers hold
// both (at 256 they do not: the cache is then read once a group). 48 rows of up to 8192 tokens with 16 heads a key head,
// two groups together against one after the other: 148 / 189 us at 128 in 8 bits, 88 / 112 at 64, 109 / 173 in bfloat16.
inline int groups(const qpack_kv_pool_t &pool, int q_heads) {
    return q_heads / pool.heads > 8 && pool.dim <= 128 ? 2 : 1;
}

template <int KT, int D, int NT> int64_t part_bytes(int grid) {
    using F = Cfg<KT, D, NT>;
    return int64_t(grid) * (2 * F::VEC * 24 + F::W * F::PF * 4);
}

template <int KT, int D, int NT> cudaError_t run(const AttendArgs &a, cudaStream_t s) {
    using F = Cfg<KT, D, NT>;
    static int opted[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    constexpr int smem = F::W * (F::STAGES * F::TILE + F::Q3) + (MAX_ROWS + 1) * 4;
    static_assert(smem <= 227 * 1024 - 5120, "shared memory");
    if (!opted[dev]) {
        e = cudaFuncSetAttribute(attend_kernel<KT, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        opted[dev] = 1;
    }
    const int grid = num_sms();
    Params p;
    p.a = a;
    p.G = a.q_heads / a.pool.heads;
    p.C = (p.G + 8 * NT - 1) / (8 * NT);
    const int HC = a.pool.heads * p.C;
    p.counters = static_cast<int *>(a.ws);
    p.block_parts = reinterpret_cast<float4 *>(p.counters + MAX_COUNTERS);
    p.block_sums = reinterpret_cast<float2 *>(p.block_parts + int64_t(grid) * 2 * F::VEC);
    p.warp_parts = reinterpret_cast<float *>(p.block_sums + int64_t(grid) * 2 * F::VEC);
    // Rows a launch: bounded by the kernel's tables, and tile numbers stay below 2^31 whatever the lengths are.
    const int64_t most = (int64_t(a.t.max_pages) * a.pool.page_tokens + F::TOK - 1) / F::TOK + 1 + SETUP;
    const int64_t fit = 0x7FFF0000 / (most * HC);
    if (fit < 1) return cudaErrorNotSupported;
    int rows = MAX_COUNTERS / (HC * F::SLICES) < MAX_ROWS ? MAX_COUNTERS / (HC * F::SLICES) : MAX_ROWS;
    if (fit < rows) rows = int(fit);
    for (int r = 0; r < a.B; r += rows) {
        p.row0 = r;
        p.B = a.B - r < rows ? a.B - r : rows;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(grid);
        cfg.blockDim = dim3(F::W * 32);
        cfg.dynamicSmemBytes = F::W * (F::STAGES * F::TILE + F::Q3) + (p.B + 1) * 4;
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, attend_kernel<KT, D, NT>, p);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// What each cache type's translation unit defines.
template <int KT> cudaError_t launch(const AttendArgs &a, cudaStream_t s);
template <int KT> int64_t workspace(const qpack_kv_pool_t &pool, int q_heads, int grid);
template <int KT> cudaError_t fault_word(int **word);

#define QPACK_ATTEND_TYPE(KT)                                                                                         \
    namespace qpack {                                                                                                 \
    namespace attend {                                                                                                \
    template <> cudaError_t launch<KT>(const AttendArgs &a, cudaStream_t s) {                                         \
        const int nt = groups(a.pool, a.q_heads);                                                                     \
        if (a.pool.dim == 64) return nt == 2 ? run<KT, 64, 2>(a, s) : run<KT, 64, 1>(a, s);                           \
        if (a.pool.dim == 128) return nt == 2 ? run<KT, 128, 2>(a, s) : run<KT, 128, 1>(a, s);                        \
        return run<KT, 256, 1>(a, s);                                                                                 \
    }                                                                                                                 \
    template <> int64_t workspace<KT>(const qpack_kv_pool_t &pool, int q_heads, int grid) {                           \
        const int nt = groups(pool, q_heads);                                                                         \
        if (pool.dim == 64) return nt == 2 ? part_bytes<KT, 64, 2>(grid) : part_bytes<KT, 64, 1>(grid);               \
        if (pool.dim == 128) return nt == 2 ? part_bytes<KT, 128, 2>(grid) : part_bytes<KT, 128, 1>(grid);            \
        return part_bytes<KT, 256, 1>(grid);                                                                          \
    }                                                                                                                 \
    template <> cudaError_t fault_word<KT>(int **word) {                                                              \
        return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_fault_attend);                                 \
    }                                                                                                                 \
    }                                                                                                                 \
    }

}  // namespace attend
}  // namespace qpack
