// qpack_shared.cuh — attention of one new token a row where groups of rows share a prefix: the kernel over the prefixes,
// instantiated per cache type in qpack_shared_i8.cu, qpack_shared_f16.cu and qpack_shared_bf16.cu.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qpack_dev.cuh"
#include "qpack_launch.h"
#include "qpack_paged.cuh"
#include "qpack_tmem.cuh"

namespace qpack {
namespace shared {

constexpr int ROWS = 128;                   // queries of a block: (row, query head) pairs of a group and key/value head
constexpr int MAX_GROUPS = 1024;
constexpr int MAX_BATCH = 4096;

// Where results go between the launches of a call. Written by the prefix kernel's first block: the plan of the call.
struct Plan {
    int size, total, blocks, ok;            // units of a block, of the call; blocks of the prefix kernel
    int cum[MAX_GROUPS + 1];                // units before group g
    int length[MAX_GROUPS];                 // its prefix, as used
    int from[MAX_BATCH];                    // a row's first token behind its prefix
    int group[MAX_BATCH];                   // its group, -1: none
};
struct Work {
    Plan *plan;
    float *own_out, *own_lse;               // [B, q_heads, D], [B, q_heads]: attention over what rows have of their own
    float *direct;                          // [B, q_heads, D] accumulators of prefixes that one block took
    float2 *direct_ml;                      // [B, q_heads] their maxima (base 2) and sums
    float *piece;                           // [blocks][2][ROWS][D] of prefixes that several took
    float2 *piece_ml;                       // [blocks][2][ROWS]
};
struct Params {
    SharedArgs a;
    Work w;
    int G;                                  // query heads a key/value head
};

// Shape of an instance.
template <int KT, int D> struct Cfg {
    static constexpr int TOK = D == 256 ? 64 : 128;        // tokens of a tile
    static constexpr int BLOCKS = D / 64;                  // 128-byte columns of an operand
    static constexpr int QB = ROWS * 128, KB = TOK * 128;  // bytes of a column of queries, of a tile
    static constexpr int Q_BYTES = BLOCKS * QB, TILE_BYTES = BLOCKS * KB;
    static constexpr bool BF = KT == QPACK_KV_BF16;
    // TMEM columns: accumulators of the output, scores, over whose columns the probabilities go, the probabilities' second terms
    static constexpr int O_COL = 0, S_COL = 256, REST_COL = D == 256 ? 384 : 128;
    // Probabilities are held as 2^(x - m + BIAS), at most 2^(BIAS + GROW): m is a maximum that lags behind by up to GROW.
    static constexpr float BIAS = BF ? 0.0f : 7.0f, GROW = 8.0f;
};

static __device__ int g_fault_shared = 0;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// A (128 x 16, in TMEM) times B.
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
          "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
          "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
          "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]),
          "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Descriptor of an operand whose rows run along the product's sum (tokens) and lie 128 bytes apart, 64 elements of the
// other index (d) a row, 128-byte swizzle: groups of eight rows 1024 bytes apart, columns of 64 elements `column` bytes apart.
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t smem_addr, uint32_t column) {
    uint64_t d = 0;
    d |= uint64_t((smem_addr >> 4) & 0x3FFFu);
    d |= uint64_t(column >> 4) << 16;
    d |= uint64_t(1024 >> 4) << 32;
    d |= uint64_t(1) << 46;
    d |= uint64_t(2) << 61;
    return d;
}
// Instruction descriptors, kind::f16: fp32 sums, M = 128, N, B's layout.
template <bool BF, int N, bool MN> constexpr uint32_t kIdesc =
    (1u << 4) | (BF ? (1u << 7) | (1u << 10) : 0u) | (MN ? 1u << 16 : 0u) | (uint32_t(N >> 3) << 17) | (uint32_t(ROWS >> 4) << 24);

// A pair of fp32 as a pair of 16-bit terms, x in the low half, and what they leave.
template <bool BF> __device__ __forceinline__ uint32_t pack2(float x, float y) {
    if (BF) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <bool BF> __device__ __forceinline__ uint32_t rest2(float x, float y, uint32_t h) {
    if (BF) return pack2<BF>(x - __uint_as_float(h << 16), y - __uint_as_float(h & 0xFFFF0000u));
    return pack2<BF>(x - h2f_bits(uint16_t(h & 0xFFFFu)), y - h2f_bits(uint16_t(h >> 16)));
}

__device__ __forceinline__ float load_elem(const void *p, int dt, int64_t i) {
    if (dt == DT_F32) return static_cast<const float *>(p)[i];
    const uint16_t h = static_cast<const uint16_t *>(p)[i];
    return dt == DT_F16 ? h2f_bits(h) : __uint_as_float(uint32_t(h) << 16);
}

// A row's sequence (-1: out of range) and its length, within the table.
__device__ __forceinline__ int row_seq(const SharedArgs &a, int row) {
    const int seq = a.seqs ? a.seqs[row] : row;
    return seq >= 0 && seq < a.t.seqs ? seq : -1;
}
__device__ __forceinline__ int row_len(const SharedArgs &a, int seq) {
    if (seq < 0) return 0;
    const int64_t cap = int64_t(a.t.max_pages) * a.pool.page_tokens;
    const int64_t len = a.t.lens[seq];
    return int(len < 0 ? 0 : len > cap ? cap : len);
}
// Whether group g's rows are where rows can be.
__device__ __forceinline__ bool group_ok(const SharedArgs &a, int g) {
    const int lo = a.first[g], hi = a.first[g + 1];
    return lo >= 0 && lo <= hi && hi <= a.B;
}
// The prefix that a group shares: as given, at most what its first row holds.
__device__ __forceinline__ int group_prefix(const SharedArgs &a, int g, bool &bad) {
    if (a.first[g] == a.first[g + 1]) return 0;
    const int given = a.prefix[g], len = row_len(a, row_seq(a, a.first[g]));
    bad = given < 0 || given > len;
    return min(max(given, 0), len);
}

// A block's place in the call: a group, its key/value head and block of queries, the tiles of it that are this block's.
struct Segment {
    int g, h, mb, row0, rows, length, tile0, tile1, tiles, page_row;
};

template <int KT, int D> __global__ void __launch_bounds__(256, 1) prefix_kernel(const __grid_constant__ Params p) {
    using F = Cfg<KT, D>;
    constexpr int TOK = F::TOK;
    constexpr bool BF = F::BF, I8 = KT == QPACK_KV_I8;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int cum[MAX_GROUPS + 1];
    __shared__ int s_ok;
    __shared__ int s_lim[ROWS];
    __shared__ float s_scale[ROWS];
    __shared__ uint64_t s_bar;
    __shared__ uint32_t s_tmem;
    const SharedArgs &a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t *sm = smem_raw + (base - smem_u32(smem_raw));
    const uint32_t q_hi = base, q_lo = base + F::Q_BYTES, kt = base + 2 * F::Q_BYTES, vt = kt + F::TILE_BYTES;
    if (tid == 0) mbar_init(&s_bar, 1), fence_mbar_init(), s_ok = 1;
    if (warp == 0) {
        tmem_alloc(&s_tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    pdl_launch_dependents();
    pdl_wait();

    // -- the plan ------------------------------------------------------------------------------------------
    for (int g = tid; g < a.groups; g += 256) {
        bool bad = false;
        int units = 0;
        if (!group_ok(a, g)) {
            s_ok = 0;
        } else {
            const int n = group_prefix(a, g, bad), rows = a.first[g + 1] - a.first[g];
            units = (n + TOK - 1) / TOK * ((rows * p.G + ROWS - 1) / ROWS) * a.pool.heads;
            if (blockIdx.x == 0) p.w.plan->length[g] = n;
        }
        if (bad && blockIdx.x == 0) atomicOr(&g_fault_shared, FAULT_PAGE);
        cum[g + 1] = units;
    }
    __syncthreads();
    const bool ok = s_ok;
    if (warp == 0) {
        int carry = 0;
        for (int g0 = 0; g0 < a.groups; g0 += 32) {
            int x = g0 + lane < a.groups && ok ? cum[g0 + lane + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            x += carry;
            if (g0 + lane < a.groups) cum[g0 + lane + 1] = x;
            carry = __shfl_sync(0xffffffffu, x, 31);
        }
        if (lane == 0) cum[0] = 0;
    }
    __syncthreads();
    const int total = cum[a.groups], size = max(1, (total + int(gridDim.x) - 1) / int(gridDim.x));
    if (blockIdx.x == 0) {
        Plan &pl = *p.w.plan;
        if (tid == 0) {
            pl.size = size, pl.total = total, pl.blocks = gridDim.x, pl.ok = ok;
            if (!ok) atomicOr(&g_fault_shared, FAULT_PAGE);
        }
        for (int g = tid; g <= a.groups; g += 256) pl.cum[g] = cum[g];
        for (int b = tid; b < a.B; b += 256) {
            int g = -1, from = 0;
            if (ok && a.groups > 0 && b >= a.first[0] && b < a.first[a.groups]) {
                int lo = 0, hi = a.groups;                 // first[lo] <= b < first[hi]
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (a.first[mid] <= b) lo = mid; else hi = mid;
                }
                g = lo;
                bool bad;
                from = group_prefix(a, g, bad);
            }
            pl.group[b] = g, pl.from[b] = from;
        }
    }

    // -- this block's units --------------------------------------------------------------------------------
    const int unit1 = min((int(blockIdx.x) + 1) * size, total);
    uint32_t phase = 0;
    bool dead = false;
    const int shift = 31 - __clz(a.pool.page_tokens);
    for (int unit = min(int(blockIdx.x) * size, total); unit < unit1 && !dead;) {
        Segment sg;
        {
            int lo = 0, hi = a.groups;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cum[mid] <= unit) lo = mid; else hi = mid;
            }
            bool bad;
            sg.g = lo;
            sg.length = group_prefix(a, lo, bad), sg.row0 = a.first[lo], sg.rows = a.first[lo + 1] - sg.row0;
            sg.tiles = (sg.length + TOK - 1) / TOK;
            const int item = (unit - cum[lo]) / sg.tiles, blocks = (sg.rows * p.G + ROWS - 1) / ROWS;
            sg.tile0 = unit - cum[lo] - item * sg.tiles;
            sg.h = item / blocks, sg.mb = item - sg.h * blocks;
            sg.tile1 = min(sg.tiles, sg.tile0 + unit1 - unit);
            sg.page_row = row_seq(a, sg.row0);
        }
        const int *table = a.t.tables + int64_t(sg.page_row) * a.t.stride;
        const int live = min(ROWS, sg.rows * p.G - sg.mb * ROWS);   // queries there are
        // queries, rotated, scaled and split: a warp a query
        __syncthreads();
        for (int r = warp; r < ROWS; r += 8) {
            constexpr int NP = D / 64;
            float x[2][NP] = {};
            int lim = 0;
            float factor = 0.0f;
            if (r < live) {
                const int rr = sg.mb * ROWS + r, b = rr / p.G, head = sg.h * p.G + rr - b * p.G, row = sg.row0 + b;
                const int len = row_len(a, row_seq(a, row));
                lim = min(len, sg.length);
                const int64_t at = int64_t(row) * a.ldq + int64_t(head) * D + lane * NP;
                for (int e = 0; e < NP; ++e)
                    x[0][e] = load_elem(a.q, a.qdt, at + e), x[1][e] = load_elem(a.q, a.qdt, at + D / 2 + e);
                if (a.rope && len > 0) {
                    if (len - 1 < a.rope_rows) {
                        const float *t = a.rope + int64_t(len - 1) * D + lane * NP;
                        for (int e = 0; e < NP; ++e) {
                            const float u = x[0][e], v = x[1][e], c = t[e], s = t[D / 2 + e];
                            x[0][e] = __fsub_rn(__fmul_rn(u, c), __fmul_rn(v, s));
                            x[1][e] = __fadd_rn(__fmul_rn(v, c), __fmul_rn(u, s));
                        }
                    } else if (lane == 0) {
                        atomicOr(&g_fault_shared, FAULT_PAGE);
                    }
                }
                float big = 0.0f;
                for (int e = 0; e < NP; ++e) big = fmaxf(big, fmaxf(fabsf(x[0][e]), fabsf(x[1][e])));
                for (int o = 16; o; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
                const int ex = __float_as_int(big) >> 23;
                const int up = BF || big == 0.0f || ex == 255 ? 127 : min(254, 267 - ex);
                const float f = __int_as_float((up << 23) | (__float_as_int(a.scale) & 0x80000000));
                const float back = __int_as_float(max(254 - up, 1) << 23);
                factor = fabsf(a.scale) * 1.4426950408889634f * back * (up == 254 ? 0.5f : 1.0f);
                if (factor == 0.0f) factor = 0x1p-126f;
                for (int e = 0; e < NP; ++e) x[0][e] *= f, x[1][e] *= f;
            }
            if (lane == 0) s_lim[r] = lim, s_scale[r] = factor;
            for (int s = 0; s < 2; ++s)
                for (int e = 0; e < NP; ++e) {
                    const int d = s * (D / 2) + lane * NP + e;
                    const uint32_t to = (d / 64) * F::QB + sw128_off(r, (d % 64) / 8) + (d % 8) * 2;
                    const uint32_t h = pack2<BF>(x[s][e], 0.0f), l = rest2<BF>(x[s][e], 0.0f, h);
                    *reinterpret_cast<uint16_t *>(sm + to) = uint16_t(h);
                    *reinterpret_cast<uint16_t *>(sm + F::Q_BYTES + to) = uint16_t(l);
                }
        }
        float m = -INFINITY, l = 0.0f;                     // of this thread's query (warps 0 to 3)
        for (int tile = sg.tile0; tile < sg.tile1 && !dead; ++tile) {
            const int t0 = tile * TOK;
            for (int i = tid; i < 2 * TOK * (D / 8); i += 256) {
                const int which = i / (TOK * (D / 8)), idx = i % (TOK * (D / 8)), r = idx / (D / 8), c = idx % (D / 8);
                uint4 v = make_uint4(0, 0, 0, 0);
                const int t = t0 + r;
                if (t < sg.length) {
                    const int page = table[t >> shift];
                    if (unsigned(page) < unsigned(a.pool.pages)) {
                        const unsigned slot = unsigned(sg.h * a.pool.page_tokens + (t & (a.pool.page_tokens - 1)));
                        const int64_t at = a.layer * a.pool.layer_stride + int64_t(page) * a.pool.page_stride + int64_t(slot) * D + c * 8;
                        const void *src = which ? a.pool.v : a.pool.k;
                        if (I8) {
                            const int64_t sat = a.layer * a.pool.scale_layer_stride + int64_t(page) * a.pool.scale_page_stride +
                                                int64_t(slot) * (D / 32) + c / 4;
                            const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const int8_t *>(src) + at);
                            const uint32_t sc = (which ? a.pool.v_scales : a.pool.k_scales)[sat], s2 = sc | sc << 16;
                            const uint32_t x = w.x ^ 0x80808080u, y = w.y ^ 0x80808080u;
                            v = make_uint4(dequant2(x, 0x4140u, s2), dequant2(x, 0x4342u, s2), dequant2(y, 0x4140u, s2),
                                           dequant2(y, 0x4342u, s2));
                        } else {
                            v = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(src) + at);
                        }
                    } else if (c == 0 && which == 0) {
                        atomicOr(&g_fault_shared, FAULT_PAGE);
                    }
                }
                *reinterpret_cast<uint4 *>(sm + 2 * F::Q_BYTES + which * F::TILE_BYTES + (c / 8) * F::KB + sw128_off(r, c % 8)) = v;
            }
            fence_proxy_async_smem();
            __syncthreads();
            if (tid == 0) {
                tc_fence_after();
                for (int term = 0; term < a.q_terms; ++term)
                    for (int k = 0; k < D / 16; ++k)
                        umma_f16(tmem + F::S_COL, sw128_kmajor_desc((term ? q_lo : q_hi) + (k / 4) * F::QB + (k % 4) * 32),
                                 sw128_kmajor_desc(kt + (k / 4) * F::KB + (k % 4) * 32), kIdesc<BF, TOK, false>, term || k);
                umma_commit(&s_bar);
            }
            dead = !__syncthreads_and(mbar_wait_bounded(&s_bar, phase));
            phase ^= 1;
            if (dead) break;
            tc_fence_after();
            if (warp < 4) {
                const uint32_t mine = tmem + (uint32_t(32 * warp) << 16);
                const int left = s_lim[tid] - t0;          // tokens of the tile that the query sees
                const float f = s_scale[tid];
                float top = -INFINITY;
                for (int c = 0; c < TOK; c += 32) {
                    uint32_t x[32];
                    tmem_ld32(mine + F::S_COL + c, x);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; ++i) top = c + i < left ? fmaxf(top, __uint_as_float(x[i])) : top;
                }
                // the maximum lags; where it has to follow, what has been added up follows too
                float shrink = 1.0f;
                const bool move = top > m && !((top - m) * f <= F::GROW);
                if (move) {
                    shrink = m == -INFINITY ? 0.0f : ex2((m - top) * f);
                    m = top;
                }
                if (__any_sync(0xffffffffu, move) && tile > sg.tile0) {
                    l *= shrink;
                    for (int c = 0; c < D; c += 32) {
                        uint32_t x[32];
                        tmem_ld32(mine + F::O_COL + c, x);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * shrink);
                        tmem_st32(mine + F::O_COL + c, x);
                    }
                }
                const float zero_at = m == -INFINITY ? 0.0f : m;
                float sum = 0.0f;
                // probabilities over the scores' own columns, first terms in the first half: a chunk is read before it is covered
                for (int c = 0; c < TOK; c += 32) {
                    uint32_t x[32], h[16], g[16];
                    tmem_ld32(mine + F::S_COL + c, x);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float e[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            e[k] = ex2(fmaf(__uint_as_float(x[2 * i + k]) - zero_at, f, F::BIAS));
                            e[k] = c + 2 * i + k < left ? e[k] : 0.0f;
                            sum += e[k];
                        }
                        h[i] = pack2<BF>(e[0], e[1]);
                        g[i] = rest2<BF>(e[0], e[1], h[i]);
                    }
                    tmem_st16(mine + F::S_COL + c / 2, h);
                    if (a.p_terms == 2) tmem_st16(mine + F::REST_COL + c / 2, g);
                }
                l += sum;
                tmem_st_wait();
                tc_fence_before();
            }
            __syncthreads();
            if (tid == 0) {
                tc_fence_after();
                for (int term = 0; term < a.p_terms; ++term)
                    for (int k = 0; k < TOK / 16; ++k)
                        umma_f16_ts(tmem + F::O_COL, tmem + (term ? F::REST_COL : F::S_COL) + k * 8,
                                    sw128_mnmajor_desc(vt + k * 2048, F::KB), kIdesc<BF, D, true>, tile > sg.tile0 || term || k);
                umma_commit(&s_bar);
            }
            dead = !__syncthreads_and(mbar_wait_bounded(&s_bar, phase));
            phase ^= 1;
            tc_fence_after();
        }
        if (warp < 4 && !dead) {
            const bool whole = sg.tile0 == 0 && sg.tile1 == sg.tiles;
            const int rr = sg.mb * ROWS + tid, b = rr / p.G, head = sg.h * p.G + rr - b * p.G;
            const int64_t slot = (int64_t(blockIdx.x) * 2 + (sg.tile0 == 0)) * ROWS + tid;
            const int64_t at = whole ? int64_t(sg.row0 + b) * a.q_heads + head : slot;
            float *o = (whole ? p.w.direct : p.w.piece) + at * D;
            for (int c = 0; c < D; c += 32) {
                uint32_t x[32];
                tmem_ld32(tmem + (uint32_t(32 * warp) << 16) + F::O_COL + c, x);
                tmem_ld_wait();
                if (tid < live)
#pragma unroll
                    for (int i = 0; i < 32; i += 4) *reinterpret_cast<uint4 *>(o + c + i) = make_uint4(x[i], x[i + 1], x[i + 2], x[i + 3]);
            }
            if (tid < live) {
                const float f = s_scale[tid];
                // the maximum as a power of two, the probabilities' height taken off
                (whole ? p.w.direct_ml : p.w.piece_ml)[at] = make_float2(m == -INFINITY ? -INFINITY : m * f - F::BIAS, l);
            }
        }
        tc_fence_before();
        unit += sg.tile1 - sg.tile0;
    }
    if (dead && tid == 0) {
        atomicOr(&g_fault_shared, FAULT_WAIT_MMA);
        (void)mbar_wait_bounded(&s_bar, phase ^ 1, 1u << 16);      // products still running, before their memory is given back
    }
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The parts of a row's query head joined: prefix pieces in the order of their blocks, then what the row has of its own.
template <int D> __global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ Params p, int tok) {
    constexpr int N = D / 32;                              // elements a lane
    const SharedArgs &a = p.a;
    const int lane = threadIdx.x & 31;
    const int64_t i = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);
    pdl_launch_dependents();
    pdl_wait();
    if (i >= int64_t(a.B) * a.q_heads) return;
    const int b = int(i / a.q_heads), head = int(i - int64_t(b) * a.q_heads), h = head / p.G;
    const Plan &pl = *p.w.plan;
    float o[N], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = 0.0f;
    auto add = [&](const float *x, float mi, float li) {
        if (!(li != 0.0f)) return;
        const float top = fmaxf(m, mi), f = m == -INFINITY ? 0.0f : ex2(m - top), g = ex2(mi - top);
        m = top;
        l = fmaf(li, g, l * f);
#pragma unroll
        for (int e = 0; e < N; ++e) o[e] = fmaf(x[lane * N + e], g, o[e] * f);
    };
    const int g = pl.group[b];
    if (g >= 0 && pl.length[g] > 0) {
        const int row0 = a.first[g], rows = a.first[g + 1] - row0, tiles = (pl.length[g] + tok - 1) / tok;
        const int rr = (b - row0) * p.G + head - h * p.G, mb = rr / ROWS, blocks = (rows * p.G + ROWS - 1) / ROWS;
        const int u0 = pl.cum[g] + (h * blocks + mb) * tiles;
        const int f0 = u0 / pl.size, f1 = (u0 + tiles - 1) / pl.size;
        if (f0 == f1) {
            const float2 ml = p.w.direct_ml[i];
            add(p.w.direct + i * D, ml.x, ml.y);
        } else {
            for (int j = f0; j <= f1; ++j) {
                const int64_t at = (int64_t(j) * 2 + (j == f0)) * ROWS + rr % ROWS;
                const float2 ml = p.w.piece_ml[at];
                add(p.w.piece + at * D, ml.x, ml.y);
            }
        }
    }
    const float own = p.w.own_lse[i];
    if (own != -INFINITY) add(p.w.own_out + i * D, own * 1.4426950408889634f, 1.0f);
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t at = int64_t(b) * a.ldo + int64_t(head) * D + lane * N;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const float x = o[e] * inv;
        if (a.odt == DT_F32) static_cast<float *>(a.out)[at + e] = x;
        else if (a.odt == DT_F16) static_cast<uint16_t *>(a.out)[at + e] = f2h_bits(x);
        else static_cast<uint16_t *>(a.out)[at + e] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
    }
    if (a.lse && lane == 0) a.lse[i] = l == 0.0f ? -INFINITY : m * 0.6931471805599453f + logf(l);
}

// -- host -------------------------------------------------------------------------------------------------------
template <int KT, int D> cudaError_t run(const Params &p, cudaStream_t s) {
    using F = Cfg<KT, D>;
    static int opted[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    // one block an SM, whatever the shape: the kernel takes all of the SM's tensor memory
    constexpr int need = 1024 + 2 * F::Q_BYTES + 2 * F::TILE_BYTES, smem = need < 120 * 1024 ? 120 * 1024 : need;
    if (!opted[dev]) {
        e = cudaFuncSetAttribute(prefix_kernel<KT, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        opted[dev] = 1;
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_sms());
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, prefix_kernel<KT, D>, p)) != cudaSuccess) return e;
    // what the rows have of their own: the cache's attention from each row's prefix on
    AttendArgs own = {};
    const SharedArgs &a = p.a;
    own.pool = a.pool, own.t = a.t, own.seqs = a.seqs, own.q = a.q, own.ldq = a.ldq, own.rope = a.rope, own.rope_rows = a.rope_rows;
    own.out = p.w.own_out, own.ldo = int64_t(a.q_heads) * D, own.lse = p.w.own_lse, own.ws = a.ws, own.window = 0;
    own.scale = a.scale, own.layer = a.layer, own.B = a.B, own.q_heads = a.q_heads, own.qdt = a.qdt, own.odt = DT_F32;
    own.from = p.w.plan->from;
    if ((e = launch_kv_attend(own, s)) != cudaSuccess) return e;
    cfg.gridDim = dim3(unsigned((int64_t(a.B) * a.q_heads + 3) / 4));
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, join_kernel<D>, p, F::TOK);
}

// What each cache type's translation unit defines.
template <int KT> cudaError_t launch(const Params &p, cudaStream_t s);
template <int KT> cudaError_t fault_word(int **word);

#define QPACK_SHARED_TYPE(KT)                                                                                         \
    namespace qpack {                                                                                                 \
    namespace shared {                                                                                                \
    template <> cudaError_t launch<KT>(const Params &p, cudaStream_t s) {                                             \
        return p.a.pool.dim == 64 ? run<KT, 64>(p, s) : p.a.pool.dim == 128 ? run<KT, 128>(p, s) : run<KT, 256>(p, s); \
    }                                                                                                                 \
    template <> cudaError_t fault_word<KT>(int **word) {                                                              \
        return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_fault_shared);                                 \
    }                                                                                                                 \
    }                                                                                                                 \
    }

}  // namespace shared
}  // namespace qpack
