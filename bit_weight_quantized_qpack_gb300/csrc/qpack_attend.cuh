// qpack_attend.cuh — attention of one new token a sequence over the paged KV cache: the kernel, instantiated per cache
// type in qpack_attend_i8.cu, qpack_attend_f16.cu and qpack_attend_bf16.cu.
//
// The mathematics. One pass over the cache with a running maximum and sum (base 2): for tokens t, x_t = q~ . k'_t times
// scale log2 e, m' = max(m, x_t), l' = l 2^(m - m') + 2^(x_t - m'), o' = o 2^(m - m') + 2^(x_t - m') v'_t; out = o / l.
// Triples (m, l, o) over parts of a sequence join by the same rule, in any grouping; here always in a fixed order.
//
// What bounds it. Every cached byte is read once: 2 (D + D/16) bytes a token and key/value head in 8 bits, 12.2 clocks
// of an SM's share of the copy rate at D = 128. The two products take 4 D flops a token and query head, too much for
// the CUDA cores with eight heads a key head (2048 FMAs against 1560 issue slots in those 12.2 clocks) and 1% of the
// tensor cores' rate. A query block has 1 to 16 rows where tcgen05.mma has at least 64, and its accumulators would
// have to come back from TMEM for every tile's softmax, so the products run on the warp-level mma.sync (m16n8k16):
// its fragments are registers, the softmax needs no exchange but two shuffles, and 32 instructions per 16 tokens fit
// the budget.
//
//   S = Q K^T:     A = queries (16 rows), B = 16 tokens x D. With up to eight query heads rows 0-7 hold the queries'
//                  leading 16-bit terms and rows 8-15 the remainders of the same heads, so one instruction takes both
//                  and S is the sum of two registers of a thread. With up to sixteen heads the remainders go in a
//                  second instruction.
//   O^T = V^T P^T: A = values transposed by ldmatrix, B = probabilities: S's accumulator layout is B's operand layout
//                  as it stands. Probabilities go in as two terms as well.
//
// Both terms carry 22 bits together (16 where the cache is bfloat16): scores and sums then differ from fp32 arithmetic
// by less than the output's rounding, where a single fp16 term would add errors of that size. Queries are scaled by a
// power of two to a maximum in [2^13, 2^14) and probabilities by 2^12, so neither term meets fp16's range.
//
// 8-bit elements become fp16(scale * code), exactly the cache's definition: a byte permute puts code + 128 under the
// exponent of 1024, one packed subtraction takes 1152 off (exact), one packed product rounds once: 1.75 instructions an
// element. ldmatrix moves pairs of bytes as 16-bit elements: for keys the four bytes of a thread are four consecutive
// d (the queries' fragments use the same order of d), for values two d of two tokens.
//
// Work is cut by tiles of 16 tokens, not by rows: lengths are known on the device only and may be anything, so each
// block adds up the rows' tiles and takes an equal share of all of them (consecutive tiles, through as many segments
// (row, key/value head, group of query heads) as it covers), and each of its warps an equal share of the block's. A
// warp owns a ring of cp.async stages and never waits for another warp until its share is done. A segment inside one
// warp's share is finished by that warp; one inside a block's share is joined in shared memory; one that spans blocks
// goes through the workspace, and the last block to arrive joins it. Where the segments are few and equally long, block
// boundaries are put on theirs.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qpack_dev.cuh"
#include "qpack_launch.h"

namespace qpack {
namespace attend {

constexpr int TOK = 16;                     // tokens a tile
constexpr int MAX_ROWS = 1024;              // rows a launch
constexpr int MAX_SEGS = 65536;             // segments a launch: counters at the front of the workspace
constexpr float P_BIAS = 12.0f;             // probabilities are held as 2^(x - m + 12)

// Shape of an instance: NT groups of eight query heads, W warps, a ring of STAGES tiles each. Registers decide W
// (accumulators D NT / 4 and query fragments D NT / 4 a thread), shared memory the stages.
template <int KT, int D, int NT> struct Cfg {
    static constexpr int ES = KT == QPACK_KV_I8 ? 1 : 2;
    static constexpr int RB = D * ES;                           // bytes of a token's row
    static constexpr int SB = KT == QPACK_KV_I8 ? D / 16 : 0;   // bytes of its scales
    static constexpr int TILE = 2 * TOK * (RB + SB);            // keys, values, their scales
    static constexpr int W = (D == 256 && KT != QPACK_KV_I8) ? 4 : (D * NT >= 256 || RB >= 256) ? 8 : 16;
    static constexpr int STAGES = 212000 / (W * TILE) > 6 ? 6 : 212000 / (W * TILE);
    static constexpr int FR = D * 8 * NT;                       // accumulators of a segment
    static constexpr int PF = FR + 2 * 8 * NT;                  // floats of a partial: accumulators, maxima, sums
    static_assert(STAGES >= 2 && PF * 4 <= STAGES * TILE, "a warp's ring holds a partial");
};

struct Params {
    AttendArgs a;
    int B, C, G;                // rows of this launch, groups of query heads, query heads a key/value head
    int row0;                   // first row of this launch
    int *counters;              // [MAX_SEGS], zero between calls
    float *block_parts;         // [grid][2][PF]
    float *warp_parts;          // [grid][W][PF]
};

static __device__ int g_fault_attend = 0;       // one a translation unit: one a cache type

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
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

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
__device__ __forceinline__ void mma(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
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

// Bytes of w (codes + 128) chosen by `sel` as fp16 codes times their scales: (1024 + u) - 1152 is exact, one rounding.
__device__ __forceinline__ uint32_t dequant2(uint32_t w, uint32_t sel, uint32_t scale) {
    const uint32_t u = __byte_perm(w, 0x64646464u, sel);
    const __half2 off = __half2half2(__ushort_as_half(0x6480));
    const __half2 c = __hsub2(*reinterpret_cast<const __half2 *>(&u), off);
    const __half2 v = __hmul2(c, *reinterpret_cast<const __half2 *>(&scale));
    return *reinterpret_cast<const uint32_t *>(&v);
}

template <int DT> __device__ __forceinline__ void load2(const void *p, int64_t i, float *x) {
    if (DT == DT_F32) {
        const float2 v = *reinterpret_cast<const float2 *>(static_cast<const float *>(p) + i);
        x[0] = v.x;
        x[1] = v.y;
    } else {
        const uint32_t v = *reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(p) + i);
        if (DT == DT_F16) {
            x[0] = h2f_bits(uint16_t(v & 0xFFFFu));
            x[1] = h2f_bits(uint16_t(v >> 16));
        } else {
            x[0] = __uint_as_float(v << 16);
            x[1] = __uint_as_float(v & 0xFFFF0000u);
        }
    }
}
__device__ __forceinline__ void load2(const void *p, int dt, int64_t i, float *x) {
    if (dt == DT_F32) load2<DT_F32>(p, i, x);
    else if (dt == DT_F16) load2<DT_F16>(p, i, x);
    else load2<DT_BF16>(p, i, x);
}
__device__ __forceinline__ void store1(void *p, int dt, int64_t i, float x) {
    if (dt == DT_F32) static_cast<float *>(p)[i] = x;
    else if (dt == DT_F16) static_cast<uint16_t *>(p)[i] = f2h_bits(x);
    else static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(x);
}

// A row's tokens [lo, len), its tiles from the multiple of 16 below lo.
struct Row {
    const int *table;
    unsigned lo, len, base;
    int tiles;
};

__device__ __forceinline__ Row row_of(const Params &p, int b, int *fault) {
    Row r;
    const AttendArgs &a = p.a;
    const int seq = a.seqs ? __ldg(a.seqs + p.row0 + b) : p.row0 + b;
    int64_t len = 0;
    bool bad = seq < 0 || seq >= a.t.seqs;
    if (!bad) {
        len = __ldg(a.t.lens + seq);
        int64_t top = int64_t(a.t.max_pages) * a.pool.page_tokens;
        top = top < 0x7FFFFFFF ? top : 0x7FFFFFFF;
        bad = len < 0 || len > top;
        len = len < 0 ? 0 : (len > top ? top : len);
    }
    if (bad && fault) atomicOr(fault, FAULT_PAGE);
    r.table = a.t.tables + (seq < 0 || seq >= a.t.seqs ? 0 : int64_t(seq) * a.t.stride);
    r.len = unsigned(len);
    r.lo = a.window > 0 && len > a.window ? unsigned(len - a.window) : 0u;
    r.base = r.lo / TOK * TOK;
    r.tiles = int((r.len - r.base + TOK - 1) / TOK);
    return r;
}

// Where a tile lies: row, segment of the row (key/value head x group of query heads), tile of the segment.
struct Cursor {
    int b, hc, ti;
    Row row;
};

__device__ __forceinline__ void seek(const Params &p, const int64_t *cum, int64_t tile, Cursor &c) {
    const int HC = p.a.pool.heads * p.C;
    int lo = 0, hi = p.B;                                  // cum[lo] HC <= tile < cum[hi] HC
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cum[mid] * HC <= tile) lo = mid; else hi = mid;
    }
    c.b = lo;
    c.row = row_of(p, lo, nullptr);
    const int64_t rem = tile - cum[lo] * HC;
    c.hc = int(rem / c.row.tiles);
    c.ti = int(rem - int64_t(c.hc) * c.row.tiles);
}

// The next tile; there is one.
__device__ __forceinline__ void step(const Params &p, const int64_t *cum, Cursor &c) {
    if (++c.ti < c.row.tiles) return;
    c.ti = 0;
    if (++c.hc < p.a.pool.heads * p.C) return;
    c.hc = 0;
    int b = c.b + 1;
    while (cum[b + 1] == cum[b]) ++b;
    c.b = b;
    c.row = row_of(p, b, nullptr);
}

// The share of block i of all tiles: equal pieces of `size` tiles, or (aligned) pieces of `size` tiles of each segment,
// `per` blocks a segment.
struct Plan {
    int64_t total, size;
    int per;                                               // 0: pieces run through the segments
};

__device__ __forceinline__ int64_t seg_start(const Params &p, const int64_t *cum, int b, int hc) {
    return cum[b] * p.a.pool.heads * p.C + hc * (cum[b + 1] - cum[b]);
}

// The blocks that share segment (b, hc), and whether block i reached it in the middle.
__device__ __forceinline__ void sharers(const Params &p, const Plan &pl, const int64_t *cum, int b, int hc, int &first,
                                        int &count) {
    const int64_t s0 = seg_start(p, cum, b, hc), n = cum[b + 1] - cum[b];
    if (pl.per) {
        first = (b * p.a.pool.heads * p.C + hc) * pl.per;
        count = int((n + pl.size - 1) / pl.size);
    } else {
        first = int(s0 / pl.size);
        count = int((s0 + n - 1) / pl.size) - first + 1;
    }
}
__device__ __forceinline__ int64_t block_start(const Params &p, const Plan &pl, const int64_t *cum, int i) {
    if (!pl.per) return i * pl.size < pl.total ? i * pl.size : pl.total;
    const int HC = p.a.pool.heads * p.C, seg = i / pl.per;
    if (seg >= p.B * HC) return pl.total;
    const int64_t n = cum[seg / HC + 1] - cum[seg / HC], at = (i % pl.per) * pl.size;
    return seg_start(p, cum, seg / HC, seg % HC) + (at < n ? at : n);
}
__device__ __forceinline__ int64_t block_end(const Params &p, const Plan &pl, const int64_t *cum, int i) {
    if (!pl.per) return block_start(p, pl, cum, i + 1);
    const int HC = p.a.pool.heads * p.C, seg = i / pl.per;
    if (seg >= p.B * HC) return pl.total;
    const int64_t n = cum[seg / HC + 1] - cum[seg / HC], at = (i % pl.per + 1) * pl.size;
    return seg_start(p, cum, seg / HC, seg % HC) + (at < n ? at : n);
}

// Partials are kept in fragment order: element e = ((chunk * NT + group) * 4 + register) * 32 + lane.
template <int KT, int NT> __device__ __forceinline__ void element(int e, int &d, int &head) {
    const int lane = e & 31, r = (e >> 5) & 3, n = (e >> 7) % NT, c = (e >> 7) / NT;
    const int g = lane >> 2, j = lane & 3;
    head = 8 * n + 2 * j + (r & 1);
    d = KT == QPACK_KV_I8 ? 16 * c + 2 * g + (r >> 1) : 16 * c + 8 * (r >> 1) + g;
}

// 1 / sum, or 0 where no token counted (a sum of NaN stays one).
__device__ __forceinline__ float inverse(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }
__device__ __forceinline__ float finite_base(float m) { return m == -INFINITY ? 0.0f : m; }
__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.0f ? -INFINITY : (m - P_BIAS) * 0.6931471805599453f + logf(l);
}

// Joins partials (part(i), i < n) and hands every element to `sink(e, head, value, base, sum)`, idx of `stride` threads.
template <int FR, int NH, class Part, class Head, class Sink>
__device__ __forceinline__ void join(int n, Part part, Head head_of, Sink sink, int idx, int stride) {
    for (int e = idx; e < FR; e += stride) {
        const int head = head_of(e);
        float m = -INFINITY;
        for (int i = 0; i < n; ++i) m = fmaxf(m, part(i)[FR + head]);
        const float base = finite_base(m);
        float o = 0.0f, l = 0.0f;
        for (int i = 0; i < n; ++i) {
            const float *q = part(i);
            const float f = ex2(q[FR + head] - base);
            o = fmaf(q[e], f, o);
            l = fmaf(q[FR + NH + head], f, l);
        }
        sink(e, head, o, m, l);
    }
}

template <int KT, int D, int NT>
__global__ void __launch_bounds__(Cfg<KT, D, NT>::W * 32, 1) attend_kernel(const __grid_constant__ Params p) {
    using F = Cfg<KT, D, NT>;
    constexpr int W = F::W, STAGES = F::STAGES, TILE = F::TILE, RB = F::RB, SB = F::SB, FR = F::FR, PF = F::PF;
    constexpr int CPR = RB / 16, CH = D / 16, NH = 8 * NT;
    constexpr bool I8 = KT == QPACK_KV_I8;
    extern __shared__ __align__(128) unsigned char smem[];
    int64_t *cum = reinterpret_cast<int64_t *>(smem + W * STAGES * TILE);    // tiles before row b, a segment's worth
    __shared__ int piece_seg[2 * W], piece_far[2 * W], s_max, s_last[2];
    const AttendArgs &a = p.a;
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, j = lane & 3;
    const int H = a.pool.heads, HC = H * p.C, T = a.pool.page_tokens, shift = 31 - __clz(T);

    pdl_launch_dependents();
    pdl_wait();                                            // inputs, cache and workspace may be the previous grid's

    // -- the rows' tiles, and this block's share of them ------------------------------------------------------
    for (int b = tid; b < p.B; b += W * 32) cum[b + 1] = row_of(p, b, blockIdx.x == 0 ? &g_fault_attend : nullptr).tiles;
    if (tid < 2 * W) piece_seg[tid] = -1;
    __syncthreads();
    if (w == 0) {
        int64_t carry = 0;
        int most = 0;
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            const int b = b0 + lane;
            int64_t x = b < p.B ? cum[b + 1] : 0;
            most = max(most, int(x));
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            x += carry;
            if (b < p.B) cum[b + 1] = x;
            carry = __shfl_sync(0xffffffffu, x, 31);
        }
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 0) {
            cum[0] = 0;
            s_max = most;
        }
    }
    __syncthreads();
    Plan pl;
    const int grid = gridDim.x, nseg = p.B * HC;
    pl.total = cum[p.B] * HC;
    pl.size = max((pl.total + grid - 1) / grid, int64_t(W));            // at least a tile a warp
    pl.per = 0;
    if (nseg <= grid) {
        // Few segments: boundaries on theirs save the joins of the pieces, where the shares stay nearly equal.
        const int k = grid / nseg;
        const int64_t size = max(int64_t((s_max + k - 1) / k), int64_t(W));
        if (size <= pl.size + pl.size / 8) {
            pl.size = size;
            pl.per = int((s_max + size - 1) / size);
            if (pl.per < 1) pl.per = 1;
        }
    }
    for (int b = blockIdx.x; b < p.B; b += grid) {
        if (cum[b + 1] != cum[b]) continue;                // an empty row
        for (int i = tid; i < a.q_heads * D; i += W * 32) store1(a.out, a.odt, int64_t(p.row0 + b) * a.ldo + i, 0.0f);
        if (a.lse)
            for (int i = tid; i < a.q_heads; i += W * 32) a.lse[int64_t(p.row0 + b) * a.q_heads + i] = -INFINITY;
    }
    const int64_t start = block_start(p, pl, cum, blockIdx.x), end = block_end(p, pl, cum, blockIdx.x);
    if (start >= end) return;

    // Results of a segment's element, and its log-sum-exp.
    auto put = [&](int b, int hc, int head, int d, float x) {
        const int in = hc % p.C * NH + head;
        if (in < p.G) store1(a.out, a.odt, int64_t(p.row0 + b) * a.ldo + int64_t(hc / p.C * p.G + in) * D + d, x);
    };
    auto put_lse = [&](int b, int hc, int head, float x) {
        const int in = hc % p.C * NH + head;
        if (a.lse && in < p.G) a.lse[int64_t(p.row0 + b) * a.q_heads + hc / p.C * p.G + in] = x;
    };

    // -- this warp's share -------------------------------------------------------------------------------------
    unsigned char *ring = smem + w * STAGES * TILE;
    const int share = int((end - start + W - 1) / W);
    const int64_t w0 = start + int64_t(w) * share;
    const int nt = int(end - w0 < share ? end - w0 : share);
    if (nt > 0) {
        const uint32_t ring32 = smem_u32(ring);
        Cursor ci, cc;
        seek(p, cum, w0, ci);
        cc = ci;
        const unsigned char *kbase = static_cast<const unsigned char *>(a.pool.k) + a.layer * a.pool.layer_stride * F::ES;
        const unsigned char *vbase = static_cast<const unsigned char *>(a.pool.v) + a.layer * a.pool.layer_stride * F::ES;
        const uint16_t *ksbase = I8 ? a.pool.k_scales + a.layer * a.pool.scale_layer_stride : nullptr;
        const uint16_t *vsbase = I8 ? a.pool.v_scales + a.layer * a.pool.scale_layer_stride : nullptr;

        // The page of lane's token of the tile (tokens lane % 16), loaded a tile ahead of its use.
        auto page_of = [&](const Cursor &c) {
            const unsigned t = c.row.base + c.ti * TOK + (lane & 15);
            return t >= c.row.lo && t < c.row.len ? __ldg(c.row.table + (t >> shift)) : -1;
        };
        int entry = page_of(ci);
        // Starts the copies of the cursor's tile into a stage. Rows outside [lo, len) and of pages outside the pool are
        // filled with zeros.
        auto issue = [&](int stage) {
            const uint32_t dst = ring32 + stage * TILE;
            const unsigned t0 = ci.row.base + ci.ti * TOK, mine = t0 + (lane & 15);
            const bool in = mine >= ci.row.lo && mine < ci.row.len;
            const bool ok = in && entry >= 0 && entry < a.pool.pages;
            if (in && !ok && lane < 16) atomicOr(&g_fault_attend, FAULT_PAGE);
            const int page = ok ? entry : 0, h = ci.hc / p.C;
            // element offset of the token's row
            const int64_t row = int64_t(page) * a.pool.page_stride + (int64_t(h) * T + (mine & (T - 1))) * D;
            const unsigned okmask = __ballot_sync(0xffffffffu, ok);
#pragma unroll
            for (int i = 0; i < CPR / 2; ++i) {
                const int idx = i * 32 + lane, r = idx / CPR, c = idx % CPR;
                const int64_t off = __shfl_sync(0xffffffffu, row, r) * F::ES + c * 16;
                const bool live = (okmask >> r) & 1;
                const uint32_t sw = r * RB + ((c ^ (RB % 128 == 0 ? r & 7 : (r >> 1) & 3)) << 4);
                cp16(dst + sw, kbase + off, live);
                cp16(dst + TOK * RB + sw, vbase + off, live);
            }
            if (I8) {
                const int64_t srow = int64_t(page) * a.pool.scale_page_stride + (int64_t(h) * T + (mine & (T - 1))) * (D / 32);
                cp_small<SB ? SB : 16>(dst + 2 * TOK * RB + lane * SB, (lane < 16 ? ksbase : vsbase) + srow, ok);
            }
        };
#pragma unroll
        for (int s = 0; s < STAGES - 1; ++s) {
            if (s < nt) {
                issue(s);
                if (s + 1 < nt) {
                    step(p, cum, ci);
                    entry = page_of(ci);
                }
            }
            cp_commit();
        }

        // ldmatrix: lane addresses row lr of the tile, chunk (even) + lane / 16
        const int lr = (lane & 7) + (lane & 8), lx = ((lane >> 4) ^ (RB % 128 == 0 ? lr & 7 : (lr >> 1) & 3)) << 4;
        const uint32_t lrow = lr * RB;
        uint32_t qf[CH][4 * NT];
        float qs[NT], m[NT], l[NT], acc[CH][NT][4];
        int begun = 0;                                     // the tile of the share with which this segment began
        bool whole = false;
        for (int i = 0; i < nt; ++i) {
            if (i == 0 || cc.ti == 0) {
                // -- a segment begins: its queries, rotated, scaled and split -----------------------------------
                begun = i;
                whole = cc.ti == 0;
                const int h = cc.hc / p.C, first = cc.hc % p.C * NH;
                const int64_t pos = int64_t(cc.row.len) - 1;
                const bool turn = a.rope && pos < a.rope_rows;
                if (a.rope && !turn) atomicOr(&g_fault_attend, FAULT_PAGE);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    m[n] = -INFINITY;
                    l[n] = 0.0f;
                    const int head = first + 8 * n + g;
                    float x[CH][4];
                    const int64_t at = int64_t(p.row0 + cc.b) * a.ldq + int64_t(h * p.G + head) * D;
                    // a thread's four elements of chunk c: 16 c + 4 j .. + 3, or 16 c + 2 j, + 1 and 8 further
                    constexpr int gap = I8 ? 2 : 8;
                    const int d0 = I8 ? 4 * j : 2 * j;
#pragma unroll
                    for (int c = 0; c < CH; ++c) {
                        x[c][0] = x[c][1] = x[c][2] = x[c][3] = 0.0f;
                        if (head < p.G) {
                            load2(a.q, a.qdt, at + 16 * c + d0, x[c]);
                            load2(a.q, a.qdt, at + 16 * c + d0 + gap, x[c] + 2);
                        }
                    }
                    if (turn) {
                        const float *row = a.rope + pos * D;
#pragma unroll
                        for (int c = 0; c < CH / 2; ++c)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int d = 16 * c + d0 + (e >> 1) * gap + (e & 1);
                                const float co = __ldg(row + d), si = __ldg(row + D / 2 + d);
                                const float u = x[c][e], v = x[c + CH / 2][e];
                                x[c][e] = __fsub_rn(__fmul_rn(u, co), __fmul_rn(v, si));
                                x[c + CH / 2][e] = __fadd_rn(__fmul_rn(v, co), __fmul_rn(u, si));
                            }
                    }
                    float big = 0.0f;
#pragma unroll
                    for (int c = 0; c < CH; ++c)
#pragma unroll
                        for (int e = 0; e < 4; ++e) big = fmaxf(big, fabsf(x[c][e]));
                    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
                    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
                    // 2^(13 - exponent of the maximum), within fp32's normal range; 1 for zero, inf and NaN
                    const int ex = __float_as_int(big) >> 23;
                    const int up = big == 0.0f || ex == 255 ? 127 : min(254, 267 - ex);
                    const float f = __int_as_float(up << 23), back = __int_as_float(max(254 - up, 1) << 23);
                    qs[n] = a.scale * 1.4426950408889634f * back * (up == 254 ? 0.5f : 1.0f);
#pragma unroll
                    for (int c = 0; c < CH; ++c) {
                        uint32_t h0, l0, h1, l1;
                        split2<KT>(x[c][0] * f, x[c][1] * f, h0, l0);
                        split2<KT>(x[c][2] * f, x[c][3] * f, h1, l1);
                        if (NT == 1) {
                            qf[c][0] = h0;
                            qf[c][1] = l0;
                            qf[c][2] = h1;
                            qf[c][3] = l1;
                        } else {
                            qf[c][n] = h0;
                            qf[c][2 + n] = h1;
                            qf[c][4 * (NT - 1) + n] = l0;
                            qf[c][4 * (NT - 1) + 2 + n] = l1;
                        }
                    }
#pragma unroll
                    for (int c = 0; c < CH; ++c)
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[c][n][r] = 0.0f;
                }
            }
            cp_wait<STAGES - 2>();
            __syncwarp();                                  // the tile is there, and the stage before it is read
            if (i + STAGES - 1 < nt) {
                issue((i + STAGES - 1) % STAGES);
                if (i + STAGES < nt) {
                    step(p, cum, ci);
                    entry = page_of(ci);
                }
            }
            cp_commit();
            const uint32_t st = ring32 + (i % STAGES) * TILE;

            // -- scores -------------------------------------------------------------------------------------
            float sc[2][4] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
            uint32_t sw[2][SB ? SB / 4 : 1];
            if (I8) {
#pragma unroll
                for (int q = 0; q < SB / 4; ++q)
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        sw[t][q] = *reinterpret_cast<const uint32_t *>(ring + (i % STAGES) * TILE + 2 * TOK * RB + (g + 8 * t) * SB + 4 * q);
#pragma unroll
                for (int c = 0; c < CH; c += 2) {
                    uint32_t r[4];
                    ldsm4(st + lrow + ((c * 16) ^ lx), r);
                    const uint32_t sel = (c / 2) & 1 ? 0x3232u : 0x1010u;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const uint32_t s = __byte_perm(sw[t][c / 4], 0u, sel);
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const uint32_t word = r[2 * u + t] ^ 0x80808080u;
                            const uint32_t b0 = dequant2(word, 0x4140u, s), b1 = dequant2(word, 0x4342u, s);
                            mma<KT>(sc[t], qf[c + u][0], qf[c + u][1], qf[c + u][2], qf[c + u][3], b0, b1);
                            if (NT == 2) mma<KT>(sc[t], qf[c + u][4 * NT - 4], qf[c + u][4 * NT - 3], qf[c + u][4 * NT - 2], qf[c + u][4 * NT - 1], b0, b1);
                        }
                    }
                }
            } else {
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    uint32_t r[4];
                    ldsm4(st + lrow + ((c * 32) ^ lx), r);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        mma<KT>(sc[t], qf[c][0], qf[c][1], qf[c][2], qf[c][3], r[t], r[2 + t]);
                        if (NT == 2) mma<KT>(sc[t], qf[c][4 * NT - 4], qf[c][4 * NT - 3], qf[c][4 * NT - 2], qf[c][4 * NT - 1], r[t], r[2 + t]);
                    }
                }
            }

            // -- softmax ------------------------------------------------------------------------------------
            const unsigned t0 = cc.row.base + cc.ti * TOK;
            const bool edge = t0 < cc.row.lo || cc.row.len - t0 < TOK;
            uint32_t ph[NT][2], plo[NT][2];
            float x[NT][4];
            bool up = false;
            float mt[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float s = NT == 1 ? sc[e >> 1][e & 1] + sc[e >> 1][2 + (e & 1)] : sc[e >> 1][2 * n + (e & 1)];
                    x[n][e] = s * qs[n];
                    if (edge) {
                        const unsigned t = t0 + 8 * (e >> 1) + 2 * j + (e & 1);
                        if (t < cc.row.lo || t >= cc.row.len) x[n][e] = -INFINITY;
                    }
                }
                mt[n] = fmaxf(fmaxf(x[n][0], x[n][1]), fmaxf(x[n][2], x[n][3]));
                mt[n] = fmaxf(mt[n], __shfl_xor_sync(0xffffffffu, mt[n], 1));
                mt[n] = fmaxf(mt[n], __shfl_xor_sync(0xffffffffu, mt[n], 2));
                mt[n] = fmaxf(mt[n], m[n]);
                up |= mt[n] > m[n];
            }
            if (__any_sync(0xffffffffu, up)) {             // rare after the first tiles
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float f = ex2(m[n] - finite_base(mt[n]));
                    m[n] = mt[n];
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
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float base = finite_base(m[n]) - P_BIAS;
#pragma unroll
                for (int e = 0; e < 4; ++e) x[n][e] = ex2(x[n][e] - base);
                l[n] += (x[n][0] + x[n][1]) + (x[n][2] + x[n][3]);
                split2<KT>(x[n][0], x[n][1], ph[n][0], plo[n][0]);
                split2<KT>(x[n][2], x[n][3], ph[n][1], plo[n][1]);
            }

            // -- values -------------------------------------------------------------------------------------
            if (I8) {
                // scales of tokens 2j, 2j + 1 (and 8 further): pairs of the groups
                uint32_t va[2][2][SB ? SB / 4 : 1];
#pragma unroll
                for (int q = 0; q < SB / 4; ++q)
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int u = 0; u < 2; ++u)
                            va[t][u][q] = *reinterpret_cast<const uint32_t *>(ring + (i % STAGES) * TILE + TOK * (2 * RB + SB) +
                                                                              (2 * j + 8 * t + u) * SB + 4 * q);
#pragma unroll
                for (int c = 0; c < CH; c += 2) {
                    uint32_t r[4];
                    ldsm4_t(st + TOK * RB + lrow + ((c * 16) ^ lx), r);
                    const uint32_t sel = (c / 2) & 1 ? 0x7632u : 0x5410u;
                    const uint32_t s0 = __byte_perm(va[0][0][c / 4], va[0][1][c / 4], sel);
                    const uint32_t s1 = __byte_perm(va[1][0][c / 4], va[1][1][c / 4], sel);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint32_t x0 = r[2 * u] ^ 0x80808080u, x1 = r[2 * u + 1] ^ 0x80808080u;
                        const uint32_t a0 = dequant2(x0, 0x4240u, s0), a1 = dequant2(x0, 0x4341u, s0);
                        const uint32_t a2 = dequant2(x1, 0x4240u, s1), a3 = dequant2(x1, 0x4341u, s1);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma<KT>(acc[c + u][n], a0, a1, a2, a3, ph[n][0], ph[n][1]);
                            mma<KT>(acc[c + u][n], a0, a1, a2, a3, plo[n][0], plo[n][1]);
                        }
                    }
                }
            } else {
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    uint32_t r[4];
                    ldsm4_t(st + TOK * RB + lrow + ((c * 32) ^ lx), r);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma<KT>(acc[c][n], r[0], r[2], r[1], r[3], ph[n][0], ph[n][1]);
                        mma<KT>(acc[c][n], r[0], r[2], r[1], r[3], plo[n][0], plo[n][1]);
                    }
                }
            }

            // -- the segment's end, or the share's ----------------------------------------------------------
            const bool done = cc.ti + 1 == cc.row.tiles, last = i + 1 == nt;
            if (done || last) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    l[n] += __shfl_xor_sync(0xffffffffu, l[n], 1);
                    l[n] += __shfl_xor_sync(0xffffffffu, l[n], 2);
                }
                if (done && whole) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float inv = inverse(l[n]);
                        const float f0 = __shfl_sync(0xffffffffu, inv, 8 * j), f1 = __shfl_sync(0xffffffffu, inv, 8 * j + 4);
#pragma unroll
                        for (int c = 0; c < CH; ++c)
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                int d, head;
                                element<KT, NT>(((c * NT + n) * 4 + r) * 32 + lane, d, head);
                                put(cc.b, cc.hc, head, d, acc[c][n][r] * (r & 1 ? f1 : f0));
                            }
                        if (j == 0) put_lse(cc.b, cc.hc, 8 * n + g, lse_of(m[n], l[n]));
                    }
                } else {
                    // The first of two pieces waits in global memory (the ring is in use), the last one in the ring.
                    if (last) {
                        cp_wait<0>();
                        __syncwarp();
                    }
                    float *dst = last ? reinterpret_cast<float *>(ring) : p.warp_parts + (int64_t(blockIdx.x) * W + w) * PF;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
#pragma unroll
                        for (int c = 0; c < CH; ++c)
#pragma unroll
                            for (int r = 0; r < 4; ++r) dst[((c * NT + n) * 4 + r) * 32 + lane] = acc[c][n][r];
                        if (j == 0) {
                            dst[FR + 8 * n + g] = m[n];
                            dst[FR + NH + 8 * n + g] = l[n];
                        }
                    }
                    if (lane == 0) {
                        const int at = 2 * w + (begun == 0 ? 0 : 1);
                        piece_seg[at] = cc.b * HC + cc.hc;
                        piece_far[at] = last ? 0 : 1;
                    }
                }
            }
            if (!last) step(p, cum, cc);
        }
        cp_wait<0>();
    }
    __syncthreads();

    // -- joins ------------------------------------------------------------------------------------------------
    // Pieces in the order of their tiles; runs of one segment are found by ballots, each warp for itself.
    const int seg = lane < 2 * W ? piece_seg[lane] : -1;
    const unsigned valid = __ballot_sync(0xffffffffu, seg >= 0);
    const unsigned below = valid & ((1u << lane) - 1u);
    const int prev = __shfl_sync(0xffffffffu, seg, below ? 31 - __clz(below) : 0);
    const unsigned starts = __ballot_sync(0xffffffffu, seg >= 0 && (!below || prev != seg));
    const bool together = __popc(starts) <= 2;             // all threads on each run, or a warp a run
    auto head_of = [](int e) {
        int d, head;
        element<KT, NT>(e, d, head);
        return head;
    };
    int cross[2] = {-1, -1}, ncross = 0, run = 0;
    for (unsigned mask = starts; mask; mask &= mask - 1, ++run) {
        const int p0 = __ffs(mask) - 1;
        const unsigned rest = mask & (mask - 1);
        const unsigned members = valid & ~((1u << p0) - 1u) & (rest ? (1u << (__ffs(rest) - 1)) - 1u : 0xffffffffu);
        const int s = __shfl_sync(0xffffffffu, seg, p0), b = s / HC, hc = s % HC;
        const int64_t s0 = seg_start(p, cum, b, hc), s1 = s0 + cum[b + 1] - cum[b];
        const bool inside = s0 >= start && s1 <= end;
        if (inside && !together && run % W != w) continue;
        const int idx = inside && !together ? lane : tid, stride = inside && !together ? 32 : W * 32;
        const int n = __popc(members);
        auto part = [&](int i) -> const float * {
            const int at = __fns(members, 0, i + 1);
            return piece_far[at] ? p.warp_parts + (int64_t(blockIdx.x) * W + (at >> 1)) * PF
                                 : reinterpret_cast<const float *>(smem + (at >> 1) * STAGES * TILE);
        };
        if (inside) {
            join<FR, NH>(n, part, head_of, [&](int e, int head, float o, float mm, float ll) {
                int d, hd;
                element<KT, NT>(e, d, hd);
                put(b, hc, head, d, o * inverse(ll));
                if (d == 0) put_lse(b, hc, head, lse_of(mm, ll));
            }, idx, stride);
        } else {
            float *dst = p.block_parts + (int64_t(blockIdx.x) * 2 + (s0 < start ? 0 : 1)) * PF;
            join<FR, NH>(n, part, head_of, [&](int e, int head, float o, float mm, float ll) {
                int d, hd;
                element<KT, NT>(e, d, hd);
                dst[e] = o;
                if (d == 0) {
                    dst[FR + head] = mm;
                    dst[FR + NH + head] = ll;
                }
            }, idx, stride);
            cross[ncross++] = s;
        }
    }
    if (!ncross) return;
    __threadfence();
    __syncthreads();
    if (tid < ncross) {
        const int s = cross[tid];
        int first, count;
        sharers(p, pl, cum, s / HC, s % HC, first, count);
        const int before = atomicAdd(p.counters + s, 1);
        s_last[tid] = before == count - 1;
        if (before == count - 1) p.counters[s] = 0;        // ready for the next call
    }
    __syncthreads();
    for (int c = 0; c < ncross; ++c) {
        if (!s_last[c]) continue;
        __threadfence();
        const int s = cross[c], b = s / HC, hc = s % HC;
        int first, count;
        sharers(p, pl, cum, b, hc, first, count);
        const int64_t s0 = seg_start(p, cum, b, hc);
        auto part = [&](int i) -> const float * {
            return p.block_parts + (int64_t(first + i) * 2 + (s0 < block_start(p, pl, cum, first + i) ? 0 : 1)) * PF;
        };
        join<FR, NH>(count, part, head_of, [&](int e, int head, float o, float mm, float ll) {
            int d, hd;
            element<KT, NT>(e, d, hd);
            put(b, hc, head, d, o * inverse(ll));
            if (d == 0) put_lse(b, hc, head, lse_of(mm, ll));
        }, tid, W * 32);
    }
}

// -- host -------------------------------------------------------------------------------------------------------
inline int groups(const qpack_kv_pool_t &pool, int q_heads) { return q_heads / pool.heads > 8 && pool.dim <= 128 ? 2 : 1; }

template <int KT, int D, int NT> int64_t part_bytes(int grid) {
    using F = Cfg<KT, D, NT>;
    return int64_t(grid) * (2 + F::W) * F::PF * 4;
}

template <int KT, int D, int NT> cudaError_t run(const AttendArgs &a, cudaStream_t s) {
    using F = Cfg<KT, D, NT>;
    static int opted[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    constexpr int smem = F::W * F::STAGES * F::TILE + (MAX_ROWS + 1) * 8;
    static_assert(smem <= 227 * 1024 - 1024, "shared memory");
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
    p.block_parts = reinterpret_cast<float *>(p.counters + MAX_SEGS);
    p.warp_parts = p.block_parts + int64_t(grid) * 2 * F::PF;
    const int rows = MAX_SEGS / HC < MAX_ROWS ? MAX_SEGS / HC : MAX_ROWS;
    for (int r = 0; r < a.B; r += rows) {
        p.row0 = r;
        p.B = a.B - r < rows ? a.B - r : rows;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(grid);
        cfg.blockDim = dim3(F::W * 32);
        cfg.dynamicSmemBytes = F::W * F::STAGES * F::TILE + (p.B + 1) * 8;
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
template <int KT> cudaError_t fetch_fault(int32_t *flags);

#define QPACK_ATTEND_TYPE(KT)                                                                                            \
    namespace qpack {                                                                                                    \
    namespace attend {                                                                                                   \
    template <> cudaError_t launch<KT>(const AttendArgs &a, cudaStream_t s) {                                            \
        const int nt = groups(a.pool, a.q_heads);                                                                        \
        if (a.pool.dim == 64) return nt == 2 ? run<KT, 64, 2>(a, s) : run<KT, 64, 1>(a, s);                              \
        if (a.pool.dim == 128) return nt == 2 ? run<KT, 128, 2>(a, s) : run<KT, 128, 1>(a, s);                           \
        return run<KT, 256, 1>(a, s);                                                                                    \
    }                                                                                                                    \
    template <> int64_t workspace<KT>(const qpack_kv_pool_t &pool, int q_heads, int grid) {                              \
        const int nt = groups(pool, q_heads);                                                                            \
        if (pool.dim == 64) return nt == 2 ? part_bytes<KT, 64, 2>(grid) : part_bytes<KT, 64, 1>(grid);                  \
        if (pool.dim == 128) return nt == 2 ? part_bytes<KT, 128, 2>(grid) : part_bytes<KT, 128, 1>(grid);               \
        return part_bytes<KT, 256, 1>(grid);                                                                             \
    }                                                                                                                    \
    template <> cudaError_t fetch_fault<KT>(int32_t * flags) {                                                           \
        int v = 0;                                                                                                       \
        const cudaError_t e = cudaMemcpyFromSymbol(&v, g_fault_attend, sizeof(int));                                     \
        if (e != cudaSuccess) return e;                                                                                  \
        *flags |= v;                                                                                                     \
        const int zero = 0;                                                                                              \
        return cudaMemcpyToSymbol(g_fault_attend, &zero, sizeof(int));                                                   \
    }                                                                                                                    \
    }                                                                                                                    \
    }

}  // namespace attend
}  // namespace qpack
