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

constexpr int ROWS = 128;                   // queries of a product: (row, query head) pairs of a group and key/value head
constexpr int MAX_GROUPS = 512;
constexpr int MAX_BATCH = 4096;

// Warps: two softmax groups of four (a warp reads the quarter of the tensor memory's lanes that its number mod 4 gives), the
// loaders, the one that issues the products.
constexpr int SOFT = 4, LOADERS = 8, MMA_WARP = 2 * SOFT + LOADERS;
constexpr int THREADS = (MMA_WARP + 1) * 32, LOAD_THREADS = LOADERS * 32;

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
    float *piece;                           // [blocks][2][queries of an item][D] of prefixes that several took
    float2 *piece_ml;                       // [blocks][2][queries of an item]
};
struct Params {
    SharedArgs a;
    Work w;
    int G;                                  // query heads a key/value head
};

// Shape of an instance.
template <int KT, int D> struct Cfg {
    static constexpr bool BF = KT == QPACK_KV_BF16, I8 = KT == QPACK_KV_I8;
    static constexpr bool DUAL = D <= 128;                 // two accumulators fit the tensor memory beside two tiles' scores
    static constexpr int TOK = D == 256 ? 64 : 128;        // tokens of a tile
    static constexpr int ITEM = DUAL ? 2 * ROWS : ROWS;    // queries that a block takes together
    static constexpr int BLOCKS = D / 64;                  // 128-byte columns of an operand
    static constexpr int QB = ROWS * 128, KB = TOK * 128;  // bytes of a column of queries, of a tile
    static constexpr int Q_BYTES = BLOCKS * QB, TILE_BYTES = BLOCKS * KB;
    // TMEM columns: accumulators of the output, two tiles' scores. The probabilities of 32 tokens go over their scores: 16
    // columns of first terms, 16 of second ones.
    static constexpr int O_COL = 0, O_STEP = D, S_COL = 256, S_STEP = TOK;
    // Probabilities are held as 2^(x - m + BIAS), at most 2^(BIAS + GROW): m is a maximum that lags behind by up to GROW.
    static constexpr float BIAS = BF ? 0.0f : 7.0f, GROW = 8.0f;
    // Shared memory: the queries' terms, a ring of tiles (keys or values of TOK tokens each), tables and barriers.
    static constexpr int QUERIES = ITEM / ROWS * Q_BYTES;  // bytes of a term of the item's queries
    static constexpr int REST = (MAX_GROUPS + 1) * 4 + 256;
    static constexpr int ring(int terms) {
        const int n = (227 * 1024 - REST - terms * QUERIES) / TILE_BYTES;
        return n < 8 ? n : 8;
    }
    static constexpr int smem(int terms) { return terms * QUERIES + ring(terms) * TILE_BYTES + REST; }
    static_assert(ring(2) >= 3 && (!DUAL || 3 * TILE_BYTES >= ROWS * D * 4) && TILE_BYTES >= 3 * ITEM * 4, "the ring holds what is exchanged in it");
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

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Pairs of fp32 in one instruction.
__device__ __forceinline__ float2 sub2(float2 a, float b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %4};\n\tadd.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(-b));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float b, float c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %4};\n\tmov.b64 z, {%5, %5};\n\t"
        "fma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

// A block's place in the call: a group, its key/value head and block of queries, the tiles of it that are this block's.
struct Segment {
    int g, h, mb, row0, rows, length, tile0, tile1, tiles, page_row;
};

// A place in the ring: slot, and the parity of the passes over it.
struct Slot {
    int at, phase;
    __device__ __forceinline__ void forward(int n, int ring) {
        at += n;
        if (at >= ring) at -= ring, phase ^= 1;
    }
};

// NP = 1, 2 or 4 consecutive elements of a query as loaded, and as fp32.
template <int NP> struct Elems { uint32_t w[NP]; };
template <int NP> __device__ __forceinline__ void load_elems(const void *p, int dt, int64_t i, Elems<NP> &r) {
    if (dt == DT_F32) {
        const uint32_t *q = static_cast<const uint32_t *>(p) + i;
        if (NP == 1) r.w[0] = q[0];
        else if (NP == 2) {
            const uint2 v = *reinterpret_cast<const uint2 *>(q);
            r.w[0] = v.x, r.w[NP > 1 ? 1 : 0] = v.y;
        } else {
            const uint4 v = *reinterpret_cast<const uint4 *>(q);
            r.w[0] = v.x, r.w[NP > 1 ? 1 : 0] = v.y, r.w[NP > 2 ? 2 : 0] = v.z, r.w[NP > 3 ? 3 : 0] = v.w;
        }
    } else {
        const uint16_t *q = static_cast<const uint16_t *>(p) + i;
        if (NP == 1) r.w[0] = q[0];
        else if (NP == 2) r.w[0] = *reinterpret_cast<const uint32_t *>(q);
        else {
            const uint2 v = *reinterpret_cast<const uint2 *>(q);
            r.w[0] = v.x, r.w[NP > 1 ? 1 : 0] = v.y;
        }
    }
}
template <int NP> __device__ __forceinline__ void widen(const Elems<NP> &r, int dt, float *x) {
#pragma unroll
    for (int e = 0; e < NP; ++e) {
        const uint32_t h = e & 1 ? r.w[e / 2] >> 16 : r.w[e / 2] & 0xFFFFu;
        x[e] = dt == DT_F32 ? __uint_as_float(r.w[e]) : dt == DT_F16 ? h2f_bits(uint16_t(h)) : __uint_as_float(h << 16);
    }
}
// NP elements of 16 bits each into shared memory.
template <int NP> __device__ __forceinline__ void put(uint8_t *p, const uint32_t *w) {
    if (NP == 1) *reinterpret_cast<uint16_t *>(p) = uint16_t(w[0]);
    else if (NP == 2) *reinterpret_cast<uint32_t *>(p) = w[0];
    else *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[NP > 2 ? 1 : 0]);
}

template <int KT, int D> __global__ void __launch_bounds__(THREADS, 1) prefix_kernel(const __grid_constant__ Params p) {
    using F = Cfg<KT, D>;
    constexpr int TOK = F::TOK, ITEM = F::ITEM;
    constexpr bool BF = F::BF, I8 = F::I8, DUAL = F::DUAL;
    extern __shared__ __align__(1024) uint8_t sm[];
    const SharedArgs &a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int R = F::ring(a.q_terms);
    const uint32_t base = smem_u32(sm);
    uint8_t *const ring = sm + a.q_terms * F::QUERIES;
    const uint32_t ring32 = smem_u32(ring);
    int *const cum = reinterpret_cast<int *>(ring + R * F::TILE_BYTES);
    uint64_t *const full = reinterpret_cast<uint64_t *>(cum + MAX_GROUPS + 2), *const empty = full + 8;
    uint64_t *const s_full = empty + 8, *const p_full = s_full + 2, *const pv_done = p_full + 2, *const o_done = pv_done + 1;
    uint32_t *const s_tmem = reinterpret_cast<uint32_t *>(o_done + 1);
    volatile int *const s_ok = reinterpret_cast<volatile int *>(s_tmem + 1), *const s_dead = s_ok + 1;
    // what is exchanged in the ring while it is empty
    int *const x_len = reinterpret_cast<int *>(ring), *const x_lim = x_len + ITEM;
    float *const x_scale = reinterpret_cast<float *>(x_lim + ITEM);

    if (base & 1023) {                                     // operands are laid out from a multiple of 1024 bytes on
        if (tid == 0) atomicOr(&g_fault_shared, FAULT_WAIT_TMEM);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < 8; ++i) mbar_init(&full[i], LOADERS), mbar_init(&empty[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&s_full[i], 1), mbar_init(&p_full[i], SOFT);
        mbar_init(pv_done, 1), mbar_init(o_done, 1);
        fence_mbar_init();
        *s_ok = 1, *s_dead = 0;
    }
    if (warp == MMA_WARP) {
        tmem_alloc(s_tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    pdl_launch_dependents();
    pdl_wait();

    // -- the plan ------------------------------------------------------------------------------------------
    for (int g = tid; g < a.groups; g += THREADS) {
        bool bad = false;
        int units = 0;
        if (!group_ok(a, g)) {
            *s_ok = 0;
        } else {
            const int n = group_prefix(a, g, bad), rows = a.first[g + 1] - a.first[g];
            units = (n + TOK - 1) / TOK * ((rows * p.G + ITEM - 1) / ITEM) * a.pool.heads;
            if (blockIdx.x == 0) p.w.plan->length[g] = n;
        }
        if (bad && blockIdx.x == 0) atomicOr(&g_fault_shared, FAULT_PAGE);
        cum[g + 1] = units;
    }
    __syncthreads();
    const bool ok = *s_ok;
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
        for (int g = tid; g <= a.groups; g += THREADS) pl.cum[g] = cum[g];
        for (int b = tid; b < a.B; b += THREADS) {
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
    const int shift = 31 - __clz(a.pool.page_tokens);
    Slot load = {0, 0}, keys = {0, 0}, values = {0, 0};    // of the loaders; of the products
    int s_phase = 0, s_phase1 = 0, p_phase = 0, p_phase1 = 0, pv_phase = 0, o_phase = 0;
    bool dead = false;
    for (int unit = min(int(blockIdx.x) * size, total); unit < unit1;) {
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
            const int item = (unit - cum[lo]) / sg.tiles, blocks = (sg.rows * p.G + ITEM - 1) / ITEM;
            sg.tile0 = unit - cum[lo] - item * sg.tiles;
            sg.h = item / blocks, sg.mb = item - sg.h * blocks;
            sg.tile1 = min(sg.tiles, sg.tile0 + unit1 - unit);
            sg.page_row = row_seq(a, sg.row0);
        }
        const int live = min(ITEM, sg.rows * p.G - sg.mb * ITEM);   // queries there are
        const bool dual = live > ROWS;                     // two blocks of queries, each with its softmax group; else one, whose
                                                           // tiles the groups take in turn (where there are two accumulators)
        const int nt = sg.tile1 - sg.tile0, jobs = dual ? 2 * nt : nt;

        // -- queries, rotated, scaled and split: a warp a query ---------------------------------------------------
        for (int r = tid; r < ITEM; r += THREADS) {
            int len = 0;
            if (r < live) len = row_len(a, row_seq(a, sg.row0 + (sg.mb * ITEM + r) / p.G));
            x_len[r] = len, x_lim[r] = r < live ? min(len, sg.length) : sg.length;    // rows past the last as if they saw all
        }
        __syncthreads();
        if (warp < MMA_WARP) {
            constexpr int NP = D / 64, U = D == 256 ? 2 : 4;
            const int top = dual ? ITEM : ROWS;
            for (int r0 = warp; r0 < top; r0 += MMA_WARP * U) {
                Elems<NP> raw[U][2];
                float2 turn[U][NP];                        // cos, sin
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int r = r0 + u * MMA_WARP;
#pragma unroll
                    for (int e = 0; e < NP; ++e) raw[u][0].w[e] = raw[u][1].w[e] = 0u, turn[u][e] = make_float2(1.0f, 0.0f);
                    if (r >= live) continue;
                    const int rr = sg.mb * ITEM + r, b = rr / p.G, head = sg.h * p.G + rr - b * p.G, len = x_len[r];
                    const int64_t at = int64_t(sg.row0 + b) * a.ldq + int64_t(head) * D + lane * NP;
                    load_elems<NP>(a.q, a.qdt, at, raw[u][0]);
                    load_elems<NP>(a.q, a.qdt, at + D / 2, raw[u][1]);
                    if (a.rope && len > 0) {
                        if (len - 1 < a.rope_rows) {
                            const float *t = a.rope + int64_t(len - 1) * D + lane * NP;
#pragma unroll
                            for (int e = 0; e < NP; ++e) turn[u][e] = make_float2(t[e], t[D / 2 + e]);
                        } else if (lane == 0) {
                            atomicOr(&g_fault_shared, FAULT_PAGE);
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int r = r0 + u * MMA_WARP;
                    if (r >= top) break;
                    float x[2][NP];
                    widen<NP>(raw[u][0], a.qdt, x[0]);
                    widen<NP>(raw[u][1], a.qdt, x[1]);
                    float big = 0.0f;
#pragma unroll
                    for (int e = 0; e < NP; ++e) {
                        const float i = x[0][e], j = x[1][e], c = turn[u][e].x, s = turn[u][e].y;
                        if (a.rope) {
                            x[0][e] = __fsub_rn(__fmul_rn(i, c), __fmul_rn(j, s));
                            x[1][e] = __fadd_rn(__fmul_rn(j, c), __fmul_rn(i, s));
                        }
                        big = fmaxf(big, fmaxf(fabsf(x[0][e]), fabsf(x[1][e])));
                    }
#pragma unroll
                    for (int o = 16; o; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
                    // a power of two that brings the maximum to [2^13, 2^14), within fp32's normal range; 1 for zero, inf and NaN,
                    // and for bfloat16 terms. The scale's sign goes with it, so that the largest score is the largest sum.
                    const int ex = __float_as_int(big) >> 23;
                    const int up = BF || big == 0.0f || ex == 255 ? 127 : min(254, 267 - ex);
                    const float f = __int_as_float((up << 23) | (__float_as_int(a.scale) & 0x80000000));
                    const float back = __int_as_float(max(254 - up, 1) << 23);
                    float factor = fabsf(a.scale) * 1.4426950408889634f * back * (up == 254 ? 0.5f : 1.0f);
                    if (factor == 0.0f) factor = 0x1p-126f;
                    if (lane == 0) x_scale[r] = factor;
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        uint32_t h[(NP + 1) / 2], l[(NP + 1) / 2];
#pragma unroll
                        for (int e = 0; e < NP; e += 2) {
                            const float y = x[s][e] * f, z = NP > 1 ? x[s][NP > 1 ? e + 1 : e] * f : 0.0f;
                            h[e / 2] = pack2<BF>(y, z);
                            l[e / 2] = rest2<BF>(y, z, h[e / 2]);
                        }
                        const int d = s * (D / 2) + lane * NP;
                        uint8_t *to = sm + (r / ROWS) * F::Q_BYTES + (d / 64) * F::QB + sw128_off(r % ROWS, (d % 64) / 8) + (d % 8) * 2;
                        put<NP>(to, h);
                        if (a.q_terms == 2) put<NP>(to + F::QUERIES, l);
                    }
                }
            }
            fence_proxy_async_smem();
        }
        __syncthreads();
        const int my_row = tid % ROWS + (dual && tid >= ROWS ? ROWS : 0);      // of the softmax groups
        int lim = 0;
        float f = 0.0f;
        if (warp < 2 * SOFT) lim = x_lim[my_row], f = x_scale[my_row];
        __syncthreads();                                   // the ring is free

        float m = -INFINITY, l = 0.0f;                     // of this thread's query
        if (warp == MMA_WARP) {
            // ------------------------------------ products ------------------------------------
            if (lane == 0) {
                auto scores = [&](int j) {
                    const int mb = dual ? j & 1 : 0;
                    if (!dual || mb == 0) dead = dead || !mbar_wait_bounded(&full[keys.at], keys.phase);
                    if (dead) return;
                    tc_fence_after();
                    const uint32_t kt = ring32 + keys.at * F::TILE_BYTES;
                    for (int term = 0; term < a.q_terms; ++term)
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            umma_f16(tmem + F::S_COL + (j & 1) * F::S_STEP,
                                     sw128_kmajor_desc(base + term * F::QUERIES + mb * F::Q_BYTES + (k / 4) * F::QB + (k % 4) * 32),
                                     sw128_kmajor_desc(kt + (k / 4) * F::KB + (k % 4) * 32), kIdesc<BF, TOK, false>, term || k);
                    umma_commit(&s_full[j & 1]);
                    if (!dual || mb == 1) {
                        umma_commit(&empty[keys.at]);
                        keys.forward(!dual && j == 0 && nt > 1 ? 1 : 2, R);
                    }
                };
                // places of the first keys and values; a segment takes 2 nt places
                const Slot begin = keys;
                values = begin;
                values.forward(dual || nt == 1 ? 1 : 2, R);
                scores(0);
                if (jobs > 1) scores(1);
                for (int j = 0; j < jobs && !dead; ++j) {
                    const int mb = dual ? j & 1 : 0, t = dual ? j >> 1 : j;
                    if (!dual || mb == 0) dead = dead || !mbar_wait_bounded(&full[values.at], values.phase);
                    dead = dead || !mbar_wait_bounded(&p_full[j & 1], j & 1 ? p_phase1 : p_phase);
                    if (j & 1) p_phase1 ^= 1; else p_phase ^= 1;
                    if (dead) break;
                    tc_fence_after();
                    const uint32_t vt = ring32 + values.at * F::TILE_BYTES;
                    const uint32_t o = tmem + F::O_COL + (DUAL ? (j & 1) * F::O_STEP : 0);
                    const bool more = DUAL ? j > 1 : j > 0;    // the accumulators hold something
                    for (int term = 0; term < a.p_terms; ++term)
#pragma unroll
                        for (int k = 0; k < TOK / 16; ++k)
                            umma_f16_ts(o, tmem + F::S_COL + (j & 1) * F::S_STEP + (k / 2) * 32 + term * 16 + (k % 2) * 8,
                                        sw128_mnmajor_desc(vt + k * 2048, F::KB), kIdesc<BF, D, true>, more || term || k);
                    if (!dual || mb == 1) {
                        umma_commit(&empty[values.at]);
                        // the last values come right behind their predecessor where tiles are taken in turn
                        values.forward(!dual && t == nt - 2 ? 1 : 2, R);
                    }
                    if (!DUAL) umma_commit(pv_done);
                    if (j + 2 < jobs) scores(j + 2);
                }
                umma_commit(o_done);
                keys = begin;                              // to the next segment's first place
                for (int n = 0; n < 2 * nt; n += 2) keys.forward(2, R);
                if (dead) *s_dead = 1;
            }
            __syncwarp();
        } else if (warp >= 2 * SOFT) {
            // ------------------------------------- loaders -------------------------------------
            const int t = tid - 2 * SOFT * 32;
            const int *table = a.t.tables + int64_t(sg.page_row) * a.t.stride;
            // a segment's tiles in the order of the products: keys of the next tile before values of this one where tiles are
            // taken in turn, keys and values of a tile else
            const int steps = 2 * nt;
            auto place = [&](int n, int &tile) -> bool {   // whether the n-th are values
                if (dual) {
                    tile = n >> 1;
                    return n & 1;
                }
                if (n == 0 || (n == steps - 1)) {
                    tile = n == 0 ? 0 : nt - 1;
                    return n != 0;
                }
                tile = n & 1 ? (n + 1) >> 1 : (n >> 1) - 1;
                return !(n & 1);
            };
            // page of a tile's row, -1 where there is none
            auto page_of = [&](int tile, int r, bool report) -> int {
                const int at = (sg.tile0 + tile) * TOK + r;
                if (at >= sg.length) return -1;
                const int page = table[at >> shift];
                if (unsigned(page) < unsigned(a.pool.pages)) return page;
                if (report) atomicOr(&g_fault_shared, FAULT_PAGE);
                return -1;
            };
            auto slot_of = [&](int tile, int r) -> unsigned {
                return unsigned(sg.h * a.pool.page_tokens) + (unsigned((sg.tile0 + tile) * TOK + r) & (a.pool.page_tokens - 1));
            };
            auto wait_empty = [&] { dead = dead || !mbar_wait_bounded(&empty[load.at], load.phase ^ 1); };
            if constexpr (I8) {
                // 16 codes a thread and row: loaded a place of the ring ahead, their pages two
                constexpr int CPR = D / 16, NC = TOK * CPR / LOAD_THREADS, STEP = LOAD_THREADS / CPR;
                const int row = t / CPR, c = t % CPR;
                struct Raw {
                    uint4 code[NC];
                    uint32_t scale[NC];
                };
                auto pages = [&](int n, int (&pg)[NC]) {
                    int tile;
                    const bool v = place(min(n, steps - 1), tile);
#pragma unroll
                    for (int i = 0; i < NC; ++i) pg[i] = n < steps ? page_of(tile, row + i * STEP, c == 0 && !v) : -1;
                };
                auto fetch = [&](int n, const int (&pg)[NC], Raw &raw) {
                    int tile;
                    const bool v = place(min(n, steps - 1), tile);
                    const int8_t *codes = static_cast<const int8_t *>(v ? a.pool.v : a.pool.k) + a.layer * a.pool.layer_stride + c * 16;
                    const uint16_t *scales = (v ? a.pool.v_scales : a.pool.k_scales) + a.layer * a.pool.scale_layer_stride + c / 2;
#pragma unroll
                    for (int i = 0; i < NC; ++i) {
                        raw.code[i] = make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u);
                        raw.scale[i] = 0;                  // a row without a page: zeros
                        if (pg[i] < 0) continue;
                        const unsigned s = slot_of(tile, row + i * STEP);
                        raw.code[i] = *reinterpret_cast<const uint4 *>(codes + pg[i] * a.pool.page_stride + s * unsigned(D));
                        raw.scale[i] = scales[pg[i] * a.pool.scale_page_stride + s * unsigned(D / 32)];
                    }
                };
                auto convert = [&](const Raw &raw) {
                    wait_empty();
                    if (!dead) {
                        uint8_t *to = ring + load.at * F::TILE_BYTES + (c / 4) * F::KB;
#pragma unroll
                        for (int i = 0; i < NC; ++i) {
                            const uint32_t s = raw.scale[i] | raw.scale[i] << 16;
                            const uint32_t w[4] = {raw.code[i].x ^ 0x80808080u, raw.code[i].y ^ 0x80808080u,
                                                   raw.code[i].z ^ 0x80808080u, raw.code[i].w ^ 0x80808080u};
                            uint4 lo = make_uint4(dequant2(w[0], 0x4140u, s), dequant2(w[0], 0x4342u, s),
                                                  dequant2(w[1], 0x4140u, s), dequant2(w[1], 0x4342u, s));
                            uint4 hi = make_uint4(dequant2(w[2], 0x4140u, s), dequant2(w[2], 0x4342u, s),
                                                  dequant2(w[3], 0x4140u, s), dequant2(w[3], 0x4342u, s));
                            const int r = row + i * STEP, flip = c / 4 & 1;    // odd columns the other half first: other banks
                            *reinterpret_cast<uint4 *>(to + sw128_off(r, (c % 4) * 2 + flip)) = flip ? hi : lo;
                            *reinterpret_cast<uint4 *>(to + sw128_off(r, (c % 4) * 2 + 1 - flip)) = flip ? lo : hi;
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&full[load.at]);
                    }
                    load.forward(1, R);
                };
                Raw x, y;
                int pg[NC];
                pages(0, pg);
                fetch(0, pg, x);
                pages(1, pg);
#pragma unroll 1
                for (int n = 0; n < steps; n += 2) {       // an even number of places
                    fetch(n + 1, pg, y);
                    pages(n + 2, pg);
                    convert(x);
                    fetch(n + 2, pg, x);
                    pages(n + 3, pg);
                    convert(y);
                }
            } else {
                // 16 bytes a thread and row, asynchronously; a place is handed over when `lag` more are under way
                constexpr int CPR = D / 8, NC = TOK * CPR / LOAD_THREADS, STEP = LOAD_THREADS / CPR;
                const int row = t / CPR, c = t % CPR;
                const int lag = min(R - 2, 3);
                Slot done = load;
                auto hand_over = [&] {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&full[done.at]);
                    done.forward(1, R);
                };
                for (int n = 0; n < steps && !dead; ++n) {
                    int tile;
                    const bool v = place(n, tile);
                    const uint16_t *src = static_cast<const uint16_t *>(v ? a.pool.v : a.pool.k) + a.layer * a.pool.layer_stride + c * 8;
                    int pg[NC];
#pragma unroll
                    for (int i = 0; i < NC; ++i) pg[i] = page_of(tile, row + i * STEP, c == 0 && !v);
                    wait_empty();
                    if (dead) break;
                    const uint32_t to = ring32 + load.at * F::TILE_BYTES + (c / 8) * F::KB;
#pragma unroll
                    for (int i = 0; i < NC; ++i) {
                        const int r = row + i * STEP;
                        cp16(to + sw128_off(r, c % 8), src + max(pg[i], 0) * a.pool.page_stride + slot_of(tile, r) * unsigned(D), pg[i] >= 0);
                    }
                    cp_commit();
                    load.forward(1, R);
                    if (n >= lag) {
                        if (lag == 1) cp_wait<1>();
                        else if (lag == 2) cp_wait<2>();
                        else cp_wait<3>();
                        hand_over();
                    }
                }
                cp_wait<0>();
                if (!dead)
                    for (int n = max(0, steps - lag); n < steps; ++n) hand_over();
            }
            if (dead) *s_dead = 1;
        } else {
            // ------------------------------------- softmax -------------------------------------
            const int wg = warp / SOFT;
            const uint32_t lanes = tmem + (uint32_t(32 * (warp % SOFT)) << 16);
            const uint32_t o = lanes + F::O_COL + (DUAL ? wg * F::O_STEP : 0);
            bool any = false;                              // the accumulators hold something
            const bool idle = (dual ? wg * ROWS : 0) + 32 * (warp % SOFT) >= live;     // no queries in this warp's lanes
            for (int j = DUAL ? wg : wg * jobs; j < jobs; j += DUAL ? 2 : 1) {
                const int t0 = (sg.tile0 + (dual ? j >> 1 : j)) * TOK, left = lim - t0;
                const uint32_t sc = lanes + F::S_COL + (j & 1) * F::S_STEP;
                // (a group that has its own score buffer keeps its phase in s_phase)
                const int phase = DUAL || !(j & 1) ? s_phase : s_phase1;
                const bool seen = !dead && mbar_wait_bounded(&s_full[j & 1], phase);
                if (DUAL || !(j & 1)) s_phase ^= 1; else s_phase1 ^= 1;
                if (!__all_sync(0xffffffffu, seen)) {
                    dead = true;
                    break;
                }
                tc_fence_after();
                if (idle) {
                    if (!DUAL) pv_phase ^= 1;
                    if (lane == 0) mbar_arrive(&p_full[j & 1]);
                    continue;
                }
                const bool all = __all_sync(0xffffffffu, left >= TOK);
                float top = -INFINITY;
#pragma unroll 1
                for (int c = 0; c < TOK; c += 32) {
                    uint32_t x[32];
                    tmem_ld32(sc + c, x);
                    tmem_ld_wait();
                    if (all) {
#pragma unroll
                        for (int i = 0; i < 32; i += 2) top = fmaxf(fmaxf(top, __uint_as_float(x[i])), __uint_as_float(x[i + 1]));
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) top = c + i < left ? fmaxf(top, __uint_as_float(x[i])) : top;
                    }
                }
                // the maximum lags; where it has to follow, what has been added up follows too
                const bool move = top > m && !((top - m) * f <= F::GROW);
                if (__any_sync(0xffffffffu, move)) {
                    const float shrink = !move ? 1.0f : m == -INFINITY ? 0.0f : ex2((m - top) * f);
                    m = move ? top : m;
                    if (any) {
                        l *= shrink;
                        if (!DUAL) {                       // the previous tile's product may still be adding
                            const bool there = mbar_wait_bounded(pv_done, pv_phase ^ 1);
                            if (!__all_sync(0xffffffffu, there)) {
                                dead = true;
                                break;
                            }
                            tc_fence_after();
                        }
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            uint32_t x[32];
                            tmem_ld32(o + c, x);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * shrink);
                            tmem_st32(o + c, x);
                        }
                    }
                }
                any = true;
                if (!DUAL) pv_phase ^= 1;
                const float from = m == -INFINITY ? 0.0f : m;
                float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll 1
                for (int c = 0; c < TOK; c += 32) {
                    uint32_t x[32], h[16], g[16];
                    tmem_ld32(sc + c, x);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float2 e = fma2(sub2(make_float2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), from), f, F::BIAS);
                        e = make_float2(ex2(e.x), ex2(e.y));
                        if (!all) {
                            e.x = c + 2 * i < left ? e.x : 0.0f;
                            e.y = c + 2 * i + 1 < left ? e.y : 0.0f;
                        }
                        sum = add2(sum, e);
                        h[i] = pack2<BF>(e.x, e.y);
                        if (BF || a.p_terms == 2) g[i] = rest2<BF>(e.x, e.y, h[i]);
                    }
                    tmem_st16(sc + c, h);
                    if (BF || a.p_terms == 2) tmem_st16(sc + c + 16, g);
                }
                l += sum.x + sum.y;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[j & 1]);
            }
            // ---- the segment's results
            if (!dead) dead = !__all_sync(0xffffffffu, mbar_wait_bounded(o_done, o_phase));
            tc_fence_after();
        }
        o_phase ^= 1;
        if (dead) *s_dead = 1;
        __syncthreads();
        if (*s_dead) break;
        if (warp < 2 * SOFT) {
            const int wg = warp / SOFT, row = tid % ROWS;
            const uint32_t o = tmem + (uint32_t(32 * (warp % SOFT)) << 16) + F::O_COL;
            // one block of queries in two accumulators: each group hands half of its columns to the other through the ring
            const bool merge = DUAL && !dual && jobs > 1;
            float *const swap = reinterpret_cast<float *>(ring);               // [D][ROWS]
            float mine = 1.0f, other = 0.0f;
            if (merge) {
                // maxima and sums first, then accumulators
                float2 *ml = reinterpret_cast<float2 *>(ring);
                ml[wg * ROWS + row] = make_float2(m, l);
                named_bar_sync(1, 2 * SOFT * 32);
                const float2 him = ml[(wg ^ 1) * ROWS + row];
                const float both = fmaxf(m, him.x), at = both == -INFINITY ? 0.0f : both;
                mine = m == -INFINITY ? 0.0f : ex2((m - at) * f), other = him.x == -INFINITY ? 0.0f : ex2((him.x - at) * f);
                m = both, l = l * mine + him.y * other;
                named_bar_sync(1, 2 * SOFT * 32);
                const int theirs = wg ? 0 : D / 2;
                for (int c = 0; c < D / 2; c += 32) {
                    uint32_t x[32];
                    tmem_ld32(o + (wg ? F::O_STEP : 0) + theirs + c, x);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; ++i) swap[(theirs + c + i) * ROWS + row] = __uint_as_float(x[i]);
                }
                named_bar_sync(1, 2 * SOFT * 32);
            }
            const bool whole = sg.tile0 == 0 && sg.tile1 == sg.tiles;
            const int r = dual ? my_row : row;
            const int rr = sg.mb * ITEM + r, b = rr / p.G, head = sg.h * p.G + rr - b * p.G;
            const int64_t at = whole ? int64_t(sg.row0 + b) * a.q_heads + head : (int64_t(blockIdx.x) * 2 + (sg.tile0 == 0)) * ITEM + r;
            float *out = (whole ? p.w.direct : p.w.piece) + at * D;
            // columns that this thread writes: all of its own accumulators, or its half of both; the first group's alone else
            const bool writes = dual || merge || wg == 0;
            const int c0 = merge && wg ? D / 2 : 0, c1 = merge && !wg ? D / 2 : D;
            if (writes)
                for (int c = c0; c < c1; c += 32) {
                    uint32_t x[32];
                    tmem_ld32(o + (wg && DUAL ? F::O_STEP : 0) + c, x);
                    tmem_ld_wait();
                    if (merge)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            x[i] = __float_as_uint(fmaf(swap[(c + i) * ROWS + row], other, __uint_as_float(x[i]) * mine));
                    if (r < live)
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            *reinterpret_cast<uint4 *>(out + c + i) = make_uint4(x[i], x[i + 1], x[i + 2], x[i + 3]);
                }
            // the maximum as a power of two, the probabilities' height taken off
            if (r < live && (dual || wg == 0))
                (whole ? p.w.direct_ml : p.w.piece_ml)[at] = make_float2(m == -INFINITY ? -INFINITY : m * f - F::BIAS, l);
            tc_fence_before();
        }
        __syncthreads();
        unit += nt;
    }
    if (*s_dead && tid == 0) atomicOr(&g_fault_shared, FAULT_WAIT_MMA);
    __syncthreads();
    if (warp == MMA_WARP) {
        tc_fence_after();
        // products still running where a wait gave up, before their memory is given back (a limit again)
        if (lane == 0 && *s_dead) (void)mbar_wait_bounded(o_done, o_phase ^ 1, 1u << 16);
        __syncwarp();
        tmem_dealloc(tmem, 512);
    }
}

// The parts of a row's query head joined: prefix pieces in the order of their blocks, then what the row has of its own.
template <int D> __global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ Params p, int tok, int item) {
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
        const int rr = (b - row0) * p.G + head - h * p.G, mb = rr / item, blocks = (rows * p.G + item - 1) / item;
        const int u0 = pl.cum[g] + (h * blocks + mb) * tiles;
        const int f0 = u0 / pl.size, f1 = (u0 + tiles - 1) / pl.size;
        if (f0 == f1) {
            const float2 ml = p.w.direct_ml[i];
            add(p.w.direct + i * D, ml.x, ml.y);
        } else {
            for (int j = f0; j <= f1; ++j) {
                const int64_t at = (int64_t(j) * 2 + (j == f0)) * item + rr % item;
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
    if (!opted[dev]) {
        const int most = F::smem(1) > F::smem(2) ? F::smem(1) : F::smem(2);
        e = cudaFuncSetAttribute(prefix_kernel<KT, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e != cudaSuccess) return e;
        opted[dev] = 1;
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_sms());
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = F::smem(p.a.q_terms);        // above half of an SM's: one block an SM, which takes all of the tensor memory
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
    return cudaLaunchKernelEx(&cfg, join_kernel<D>, p, F::TOK, F::ITEM);
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
