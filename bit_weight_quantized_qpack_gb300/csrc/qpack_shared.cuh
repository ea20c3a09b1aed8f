// qpack_shared.cuh — attention of one new token a row where groups of rows share a prefix: the kernels over the
// prefixes and for the joins, instantiated per cache type in qpack_shared_i8.cu, qpack_shared_f16.cu and
// qpack_shared_bf16.cu.
//
// The mathematics. Row b of group g sees the tokens 0 .. L_b - 1, of which the first P_g are those of the group's
// first row. For any split of a row's tokens into sets S with m_S = max s_t, l_S = sum e^(s_t - m_S), o_S = sum
// e^(s_t - m_S) v_t, the whole is
//     out = sum_S e^(m_S - m) o_S / sum_S e^(m_S - m) l_S,    m = max m_S,    lse = m + log(sum_S e^(m_S - m) l_S).
// So three launches: o, m and l over the prefixes, for all queries of a group that a key/value head serves in one
// product; over what rows have of their own, by the cache's attention from token P_g on (qpack_attend.cuh); and the
// joins.
//
// What bounds it. A group has R = rows x query heads a key/value head queries, for which each element of its prefix
// is multiplied and added R times: with 8-bit elements the tensor cores at their rate take as long as HBM at R = 142.
// Neither is reached; what limits the prefix kernel is the chain scores -> maximum -> weights -> values: for two
// blocks of 128 queries some 3.8 us a tile of 128 tokens (products of 128 x 128 x 128 are 0.65k clocks each, two for
// the scores and, of two terms, four for the values; weights with their maximum some 2.7k; the rest hand-overs
// between warps; the tensor pipe is 42% busy, the schedulers 58%). 32 rows of 65531 tokens, 64 heads over 8, 8 bits:
// 115 us for 68.7 GFLOP, 32% of the measured bf16 rate; 64 rows of 7999, 32 over 8: 26 us, of which some 12 are the
// call's start (plan, queries, first tiles) and the results' way out. A call of a few rows takes three launches'
// latency, 20 us.
//
// Layout. One block an SM, 17 warps: loaders bring tiles of keys and values into a ring of 128-byte-swizzled operands
// (8-bit codes are unpacked to fp16(scale code) on the way, which is what the cache stands for), one warp issues the
// products on tcgen05, two groups of four hold a query a thread, take scores from tensor memory, and put the weights
// back over them as the A operand of the second product, so that neither leaves the SM nor passes through shared
// memory. Units, a tile for one block of queries, are cut evenly over the blocks whatever the groups' lengths; a
// block that gets part of a prefix leaves a piece.
//   A tile at a time by all warps took 760 us for the 65531 tokens, roles of their own 226, codes staged
// asynchronously 180, addresses by a lane a row 150, products issued by a converged warp and two teams of loaders
// 140, the joins' warps 132 (weights of one term); with weights of two terms and queries' lines asked for ahead it is
// 137. Slower, with one term: halves of 64 tokens with two score buffers a group (149 against 137), one team (150),
// rows' own tokens attended to within the join (fp32, a lane a token out of shared memory: 28 us more for 64 rows of
// up to 200).
//
// Terms. fp32 queries (and rotated ones of 16 bits) are two 16-bit terms; a second term of the queries doubles that
// product, and blocks of 128 queries are then taken one at a time. Weights are always two: of one (fp16: 11 bits, off
// by up to 2^-11 against the sum, which is of unrounded weights) a 16-bit output showed the error, 2.3e-4 to 2.5e-4
// of it where its own rounding alone is 2.1e-4. us a call, one term / two: 64 rows of 7999 tokens 49.2 / 50.2, 32 of
// 65531 124 / 141, heads of 256 45.1 / 45.9.
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

constexpr int ROWS = 128;           // queries of a product: (row, query head) pairs of a group and key/value head
constexpr int MAX_GROUPS = 512;
constexpr int MAX_BATCH = 4096;

// Warps: two softmax groups of four (a warp reads the quarter of the tensor memory's lanes that its number mod 4
// gives), the loaders, the one that issues the products.
constexpr int SOFT = 4, LOADERS = 8, MMA_WARP = 2 * SOFT + LOADERS;
constexpr int THREADS = (MMA_WARP + 1) * 32, LOAD_THREADS = LOADERS * 32;

// Where results go between the launches of a call. Written by the prefix kernel's last block: the plan of the call.
struct Plan {
    int size, item;                         // units of a block; queries that a block takes together
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
    float *piece;                           // [blocks][2][2 ROWS][D] of prefixes that several took
    float2 *piece_ml;                       // [blocks][2][2 ROWS]
};
struct Params {
    SharedArgs a;
    Work w;
    int G;                                  // query heads a key/value head
};

// Shape of an instance.
template <int KT, int D> struct Cfg {
    static constexpr bool BF = KT == QPACK_KV_BF16, I8 = KT == QPACK_KV_I8;
    static constexpr bool TWO = D <= 128;                  // two accumulators fit the tensor memory beside two tiles' scores
    static constexpr int TOK = D == 256 ? 64 : 128;        // tokens of a tile
    // Loaders take a tile together, or, where they convert it, in two teams that take them in turn: with one, the
    // waits and latencies of a tile had nothing to pass under.
    static constexpr int TEAMS = I8 ? 2 : 1, TEAM = LOAD_THREADS / TEAMS;
    static constexpr int BLOCKS = D / 64;                  // 128-byte columns of an operand
    static constexpr int QB = ROWS * 128, KB = TOK * 128;  // bytes of a column of queries, of a tile
    static constexpr int Q_BYTES = BLOCKS * QB, TILE_BYTES = BLOCKS * KB;
    // TMEM columns: accumulators of the output, two tiles' scores. The probabilities of 32 tokens go over their
    // scores: 16 columns of first terms, 16 of second ones.
    static constexpr int O_COL = 0, O_STEP = D, S_COL = 256, S_STEP = TOK;
    // Probabilities are held as 2^(x - m + BIAS), at most 2^(BIAS + GROW): m is a maximum that lags behind by up to
    // GROW.
    static constexpr float BIAS = BF ? 0.0f : 7.0f, GROW = 8.0f;      // (fp16 ends at 2^16)
    // Shared memory: the queries (one or two operands), 8-bit codes on their way (a tile a team), a ring of tiles of
    // 16-bit keys or values, the plan and the barriers. The results of a segment are put together over the first
    // three.
    static constexpr int SMEM = 227 * 1024, REST = (MAX_GROUPS + 1) * 4 + (TWO ? 2 : 1) * ROWS * 4 + 256;
    static constexpr int RAW_BYTES = TOK * D, RAW_ALL = I8 ? TEAMS * RAW_BYTES : 0;
    static constexpr int ring(int operands) {
        const int n = (SMEM - REST - operands * Q_BYTES - RAW_ALL) / TILE_BYTES;
        return n < 8 ? n : 8;
    }
    static constexpr int PS = D + 4;                       // floats of a row of results, padded for the banks
    static_assert(ring(2) >= (I8 ? 2 : 3), "tiles");
    static_assert((TWO ? 2 : 1) * ROWS * PS * 4 <= SMEM - REST, "results");
};

static __device__ int g_fault_shared = 0;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The products are issued by one lane of a warp that runs through their code as a whole: all they are given is the
// same for the warp then, and lies where the instruction wants it (one lane alone in a branch took 135 clocks a
// product).
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}
// Descriptors are given by their low words: between operands and steps only the address field there changes, and one
// addition a descriptor is what the issuing warp can do beside a product. High word: 1024 bytes between groups of
// rows, version 1, 128-byte swizzle.
constexpr uint32_t DESC_HI = 1024 >> 4 | 1u << 14 | 2u << 29;
__device__ __forceinline__ void umma_ss(uint32_t one, uint32_t d_tmem, uint32_t adesc, uint32_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "mov.b64 a, {%1, %6};\n\t"
        "mov.b64 b, {%2, %6};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(adesc), "r"(bdesc), "r"(idesc), "r"(accumulate), "r"(one), "n"(DESC_HI)
        : "memory");
}
// A (128 x 16, in TMEM) times B.
__device__ __forceinline__ void umma_ts(uint32_t one, uint32_t d_tmem, uint32_t a_tmem, uint32_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "mov.b64 b, {%2, %6};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "r"(bdesc), "r"(idesc), "r"(accumulate), "r"(one), "n"(DESC_HI)
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t one, uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)), "r"(one)
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
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Low words of operand descriptors with 128-byte swizzle, groups of eight rows of 128 bytes 1024 bytes apart: rows of
// 64 elements of the product's sum (queries, keys); rows that run along the sum themselves (values by tokens), whose
// columns of 64 elements lie `column` bytes apart.
__device__ __forceinline__ uint32_t desc_k(uint32_t smem_addr) { return (smem_addr >> 4 & 0x3FFFu) | 1u << 16; }
__device__ __forceinline__ uint32_t desc_mn(uint32_t smem_addr, uint32_t column) {
    return (smem_addr >> 4 & 0x3FFFu) | column >> 4 << 16;
}
// Instruction descriptors, kind::f16: fp32 sums, M = 128, N, B's layout.
template <bool BF, int N, bool MN> constexpr uint32_t kIdesc =
    (1u << 4) | (BF ? (1u << 7) | (1u << 10) : 0u) | (MN ? 1u << 16 : 0u) | (uint32_t(N >> 3) << 17) |
    (uint32_t(ROWS >> 4) << 24);

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
__device__ __forceinline__ void prefetch_line(const void *p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }
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
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
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
    int g, length, row0, rows, page_row;    // the group: its prefix, its rows, the sequence whose pages are read
    int blocks, tiles;                      // blocks of queries, tiles of a block
    int h, mb, tile0, nt;
};

// A place in the ring: slot, and the parity of the passes over it.
struct Slot {
    int at, phase;
    __device__ __forceinline__ void forward(int n, int ring) {
        at += n;
        if (at >= ring) at -= ring, phase ^= 1;
    }
};

// N consecutive elements of a query as fp32, N a multiple of 4.
template <int N> __device__ __forceinline__ void load_q(const void *p, int dt, int64_t i, float *x) {
    if (dt == DT_F32) {
#pragma unroll
        for (int e = 0; e < N; e += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i + e);
            x[e] = v.x, x[e + 1] = v.y, x[e + 2] = v.z, x[e + 3] = v.w;
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < N; e += 4) {
        const uint2 v = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + i + e);
        const uint32_t w[2] = {v.x, v.y};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t h = k & 1 ? w[k / 2] >> 16 : w[k / 2] & 0xFFFFu;
            x[e + k] = dt == DT_F16 ? h2f_bits(uint16_t(h)) : __uint_as_float(h << 16);
        }
    }
}

// A bounded wait of a whole warp, which gives up together: lanes that did alone would leave the others in the
// shuffles behind it.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity));
}

template <int KT, int D> __global__ void __launch_bounds__(THREADS, 1) prefix_kernel(const __grid_constant__ Params p) {
    using F = Cfg<KT, D>;
    constexpr int TOK = F::TOK, PS = F::PS;
    constexpr bool BF = F::BF, I8 = F::I8, TWO = F::TWO;
    extern __shared__ __align__(1024) uint8_t sm[];
    const SharedArgs &a = p.a;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t base = smem_u32(sm);
    int *const cum = reinterpret_cast<int *>(sm + F::SMEM - F::REST);
    float *const x_scale = reinterpret_cast<float *>(cum + MAX_GROUPS + 1);
    uint64_t *const full = reinterpret_cast<uint64_t *>(sm + F::SMEM - 248), *const empty = full + 8;
    uint64_t *const s_full = empty + 8, *const p_full = s_full + 2, *const pv_done = p_full + 2, *const o_done = pv_done + 1;
    uint32_t *const s_tmem = reinterpret_cast<uint32_t *>(o_done + 1);
    volatile int *const s_ok = reinterpret_cast<volatile int *>(s_tmem + 1), *const s_dead = s_ok + 1;
    int *const s_group = reinterpret_cast<int *>(s_tmem + 3);      // the first segment's: number, prefix, row, rows, sequence

    if (base & 1023) {                                     // operands are laid out from a multiple of 1024 bytes on
        if (tid == 0) atomicOr(&g_fault_shared, FAULT_WAIT_TMEM);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < 8; ++i) mbar_init(&full[i], LOADERS / F::TEAMS), mbar_init(&empty[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&s_full[i], 1), mbar_init(&p_full[i], SOFT);
        mbar_init(pv_done, 1), mbar_init(o_done, 1);
        fence_mbar_init();
        *s_ok = 1, *s_dead = 0;
    }
    if (warp == MMA_WARP) {
        tmem_alloc(s_tmem, 512);
        tmem_relinquish();
    }
    pdl_launch_dependents();
    pdl_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;

    // -- the plan: a thread a group ---------------------------------------------------------------------------
    static_assert(MAX_GROUPS <= THREADS, "a thread a group");
    int length = 0, row0 = 0, rows = 0, page_row = -1;
    if (tid < a.groups) {
        row0 = a.first[tid], rows = a.first[tid + 1] - row0;
        const int given = a.prefix[tid];
        if (row0 < 0 || rows < 0 || row0 + int64_t(rows) > a.B) {
            *s_ok = 0;
        } else if (rows > 0) {
            page_row = row_seq(a, row0);
            const int len = row_len(a, page_row);
            length = min(max(given, 0), len);
            if ((given < 0 || given > len) && blockIdx.x == 0) atomicOr(&g_fault_shared, FAULT_PAGE);
        }
    }
    const int tiles = (length + TOK - 1) / TOK, queries = rows * p.G;
    // Two blocks of queries at a time share a tile's conversion and its way from L2, where queries are one term each
    // (with two the products take longer than either) and every block gets enough tiles to pay for twice the queries
    // and results.
    const bool pays = queries > ROWS && int64_t(tiles) * ((queries + 2 * ROWS - 1) / (2 * ROWS)) * a.pool.heads >=
                                            6 * int64_t(gridDim.x);
    const int most = TWO && a.q_terms == 1 ? __syncthreads_or(pays) : (__syncthreads(), 0);
    const int item = most ? 2 * ROWS : ROWS;
    const bool ok = *s_ok;
    const int units = ok ? tiles * ((queries + item - 1) / item) * a.pool.heads : 0;
    {                                                      // inclusive sums over the groups
        int x = units;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) x_scale[warp] = __int_as_float(x);
        __syncthreads();
        for (int w = 0; w < warp; ++w) x += __float_as_int(x_scale[w]);
        if (tid < a.groups) cum[tid + 1] = x;
        if (tid == 0) cum[0] = 0;
    }
    __syncthreads();
    const int total = cum[a.groups], size = max(1, (total + int(gridDim.x) - 1) / int(gridDim.x));
    const int unit0 = min(int(blockIdx.x) * size, total), unit1 = min(unit0 + size, total);
    if (tid < a.groups && cum[tid] <= unit0 && unit0 < cum[tid + 1])
        s_group[0] = tid, s_group[1] = length, s_group[2] = row0, s_group[3] = rows, s_group[4] = page_row;
    if (blockIdx.x == gridDim.x - 1) {                     // the block with the least to do
        Plan &pl = *p.w.plan;
        if (tid == 0) {
            pl.size = size, pl.item = item;
            if (!ok) atomicOr(&g_fault_shared, FAULT_PAGE);
        }
        if (tid < a.groups) pl.cum[tid] = cum[tid], pl.length[tid] = length;
        __syncthreads();
        for (int b = tid; b < a.B; b += THREADS) {
            int g = -1, from = 0;
            if (ok && a.groups > 0 && b >= a.first[0] && b < a.first[a.groups]) {
                int lo = 0, hi = a.groups;                 // first[lo] <= b < first[hi]
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (a.first[mid] <= b) lo = mid; else hi = mid;
                }
                g = lo, from = pl.length[lo];
            }
            pl.group[b] = g, pl.from[b] = from;
        }
    }
    __syncthreads();
    if (unit0 >= unit1) {
        if (warp == MMA_WARP) tmem_dealloc(tmem, 512);
        return;
    }

    // -- this block's units --------------------------------------------------------------------------------
    Segment sg;
    sg.g = s_group[0], sg.length = s_group[1], sg.row0 = s_group[2], sg.rows = s_group[3], sg.page_row = s_group[4];
    const int operands = a.q_terms * (item / ROWS), R = F::ring(operands);
    uint8_t *const raw = sm + operands * F::Q_BYTES;
    uint8_t *const ring = raw + F::RAW_ALL;
    const uint32_t ring32 = smem_u32(ring);
    const int shift = 31 - __clz(a.pool.page_tokens);
    Slot load = {I8 && warp >= 2 * SOFT + LOADERS / 2 ? 1 : 0, 0};         // of the loaders
    Slot keys = {0, 0}, values = {0, 0};                   // of the products
    int s_phase = 0, s_phase1 = 0, p_phase = 0, p_phase1 = 0, pv_phase = 0, o_phase = 0;
    bool dead = false;
    for (int unit = unit0;;) {
        sg.blocks = (sg.rows * p.G + item - 1) / item, sg.tiles = (sg.length + TOK - 1) / TOK;
        {
            const int at = unit - cum[sg.g], i = at / sg.tiles;
            sg.tile0 = at - i * sg.tiles, sg.h = i / sg.blocks, sg.mb = i - sg.h * sg.blocks;
            sg.nt = min(sg.tiles - sg.tile0, unit1 - unit);
        }
        const int live = min(item, sg.rows * p.G - sg.mb * item);   // queries there are
        const bool dual = live > ROWS;                     // two blocks of queries, each with its softmax group; else one, whose
                                                           // tiles the groups take in turn (where there are two
                                                           // accumulators)
        const int nt = sg.nt, jobs = dual ? 2 * nt : nt;
        int lim = sg.length;                               // tokens that this thread's query sees (softmax groups)
        float f = 0.0f, m = -INFINITY, l = 0.0f;           // its scale, running maximum and sum
        if (warp < 2 * SOFT || warp == MMA_WARP) {
            // -- queries, rotated, scaled and split: eight lanes a query. Whose they are and where they lie is found by a lane a
            // query first, so that the loads of a pass depend on nothing.
            constexpr int N = D / 16;                      // a lane's elements i and as many i + D / 2
            const int sub = lane & 7, top = (live + 31) / 32 * 32;         // rows behind the last stay as they are, if not of its warp
            if (warp < 2 * SOFT) {
                int my_pos = -1;
                int64_t my_at = 0;
                if (const int r = warp * 4 + (lane & 3) + (lane >> 2) * 32; r < live) {
                    const int rr = sg.mb * item + r, b = rr / p.G, head = sg.h * p.G + rr - b * p.G;
                    my_at = int64_t(sg.row0 + b) * a.ldq + int64_t(head) * D;
                    if (a.rope) my_pos = row_len(a, row_seq(a, sg.row0 + b)) - 1;
                    if (my_pos >= a.rope_rows) {
                        if (a.rope) atomicOr(&g_fault_shared, FAULT_PAGE);
                        my_pos = -1;
                    }
                }
                // all passes' lines are asked for first: registers for their loads there are not (heads of 256:
                // nothing gained)
                if (D <= 128)
#pragma unroll 1
                for (int it = 0; it * 32 < top; ++it) {
                    const int pos = __shfl_sync(0xffffffffu, my_pos, it * 4 + (lane >> 3));
                    const int64_t at = __shfl_sync(0xffffffffu, my_at, it * 4 + (lane >> 3)) + sub * N;
                    if (it * 32 + warp * 4 + (lane >> 3) < live) {
                        const char *from = static_cast<const char *>(a.q) + at * (a.qdt == DT_F32 ? 4 : 2);
                        prefetch_line(from);
                        prefetch_line(from + D / 2 * (a.qdt == DT_F32 ? 4 : 2));
                    }
                    if (pos >= 0) {
                        const float *t = a.rope + int64_t(pos) * D + sub * N;
                        prefetch_line(t);
                        prefetch_line(t + D / 2);
                    }
                }
#pragma unroll 1
                for (int it = 0; it * 32 < top; ++it) {
                    const int r = it * 32 + warp * 4 + (lane >> 3);
                    const int pos = __shfl_sync(0xffffffffu, my_pos, it * 4 + (lane >> 3));
                    const int64_t at = __shfl_sync(0xffffffffu, my_at, it * 4 + (lane >> 3)) + sub * N;
                    float x[2][N];
#pragma unroll
                    for (int e = 0; e < N; ++e) x[0][e] = x[1][e] = 0.0f;
                    if (r < live) {
                        load_q<N>(a.q, a.qdt, at, x[0]);
                        load_q<N>(a.q, a.qdt, at + D / 2, x[1]);
                    }
                    if (pos >= 0) {
                        const float *t = a.rope + int64_t(pos) * D + sub * N;
#pragma unroll
                        for (int e = 0; e < N; e += 4) {
                            const float4 c4 = *reinterpret_cast<const float4 *>(t + e);
                            const float4 s4 = *reinterpret_cast<const float4 *>(t + D / 2 + e);
                            const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float i = x[0][e + k], j = x[1][e + k];
                                x[0][e + k] = __fsub_rn(__fmul_rn(i, c[k]), __fmul_rn(j, s[k]));
                                x[1][e + k] = __fadd_rn(__fmul_rn(j, c[k]), __fmul_rn(i, s[k]));
                            }
                        }
                    }
                    float big = 0.0f;
#pragma unroll
                    for (int e = 0; e < N; ++e) big = fmaxf(big, fmaxf(fabsf(x[0][e]), fabsf(x[1][e])));
#pragma unroll
                    for (int o = 4; o; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
                    // a power of two that brings the maximum to [2^13, 2^14), within fp32's normal range; 1 for zero,
                    // inf and NaN, and for bfloat16 terms. The scale's sign goes with it, so that the largest score
                    // is the largest sum.
                    const int ex = __float_as_int(big) >> 23;
                    const int up = BF || big == 0.0f || ex == 255 ? 127 : min(254, 267 - ex);
                    const float g = __int_as_float((up << 23) | (__float_as_int(a.scale) & 0x80000000));
                    const float back = __int_as_float(max(254 - up, 1) << 23);
                    const float factor = fabsf(a.scale) * 1.4426950408889634f * back * (up == 254 ? 0.5f : 1.0f);
                    // An infinite query is NaN, whatever signs its scores have: were all of them -inf, they would
                    // count as none.
                    if (sub == 0)
                        x_scale[r] = ex == 255 ? __int_as_float(0x7FC00000) : factor == 0.0f ? 0x1p-126f : factor;
                    const int block = r / ROWS, row = r % ROWS;
#pragma unroll
                    for (int s = 0; s < 2; ++s)
#pragma unroll
                        for (int e = 0; e < N; e += 4) {
                            const int d = s * (D / 2) + sub * N + e;
                            uint8_t *to = sm + block * F::Q_BYTES + (d / 64) * F::QB + sw128_off(row, (d % 64) / 8) +
                                          (d % 8) * 2;
                            const float y[4] = {x[s][e] * g, x[s][e + 1] * g, x[s][e + 2] * g, x[s][e + 3] * g};
                            const uint2 h = make_uint2(pack2<BF>(y[0], y[1]), pack2<BF>(y[2], y[3]));
                            *reinterpret_cast<uint2 *>(to) = h;
                            if (a.q_terms == 2)            // one block of queries then
                                *reinterpret_cast<uint2 *>(to + F::Q_BYTES) =
                                    make_uint2(rest2<BF>(y[0], y[1], h.x), rest2<BF>(y[2], y[3], h.y));
                        }
                }
                fence_proxy_async_smem();
            }
            named_bar_sync(1, (2 * SOFT + 1) * 32);
            if (warp < 2 * SOFT) {
                const int r = dual ? tid : tid % ROWS;
                f = x_scale[r];
                if (r < live) lim = min(lim, row_len(a, row_seq(a, sg.row0 + (sg.mb * item + r) / p.G)));
            }
        }
        if (warp == MMA_WARP) {
            // ------------------------------------ products ------------------------------------
            const uint32_t one = elect_one();
            {
                auto scores = [&](int j) {
                    const int mb = dual ? j & 1 : 0;
                    if (!dual || mb == 0) dead = dead || !warp_wait(&full[keys.at], keys.phase);
                    if (dead) return;
                    tc_fence_after();
                    const uint32_t kd = desc_k(ring32 + keys.at * F::TILE_BYTES);
                    const uint32_t to = tmem + F::S_COL + (j & 1) * F::S_STEP;
                    for (int term = 0; term < a.q_terms; ++term) {
                        const uint32_t qd = desc_k(base + (term + mb) * F::Q_BYTES);
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            umma_ss(one, to, qd + ((k / 4) * F::QB + (k % 4) * 32) / 16,
                                    kd + ((k / 4) * F::KB + (k % 4) * 32) / 16, kIdesc<BF, TOK, false>, term || k);
                    }
                    commit(one, &s_full[j & 1]);
                    if (!dual || mb == 1) {
                        commit(one, &empty[keys.at]);
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
                    if (!dual || mb == 0) dead = dead || !warp_wait(&full[values.at], values.phase);
                    dead = dead || !warp_wait(&p_full[j & 1], j & 1 ? p_phase1 : p_phase);
                    if (j & 1) p_phase1 ^= 1; else p_phase ^= 1;
                    if (dead) break;
                    tc_fence_after();
                    const uint32_t vd = desc_mn(ring32 + values.at * F::TILE_BYTES, F::KB);
                    const uint32_t o = tmem + F::O_COL + (TWO ? (j & 1) * F::O_STEP : 0);
                    const uint32_t w = tmem + F::S_COL + (j & 1) * F::S_STEP;
                    const bool more = TWO ? j > 1 : j > 0; // the accumulators hold something
                    for (int term = 0; term < 2; ++term)
#pragma unroll
                        for (int k = 0; k < TOK / 16; ++k)
                            umma_ts(one, o, w + (k / 2) * 32 + term * 16 + (k % 2) * 8, vd + k * (2048 / 16),
                                    kIdesc<BF, D, true>, more || term || k);
                    if (!dual || mb == 1) {
                        commit(one, &empty[values.at]);
                        // the last values come right behind their predecessor where tiles are taken in turn
                        values.forward(!dual && t == nt - 2 ? 1 : 2, R);
                    }
                    if (!TWO) commit(one, pv_done);
                    if (j + 2 < jobs) scores(j + 2);
                }
                commit(one, o_done);
                keys = begin;                              // to the next segment's first place
                keys.phase ^= 2 * nt / R & 1, keys.forward(2 * nt % R, R);
            }
        } else if (warp >= 2 * SOFT) {
            // ------------------------------------- loaders -------------------------------------
            const int team = (warp - 2 * SOFT) / (LOADERS / F::TEAMS), t = tid - 2 * SOFT * 32 - team * F::TEAM;
            const int *table = a.t.tables + int64_t(sg.page_row) * a.t.stride;
            // a segment's tiles in the order of the products: keys of the next tile before values of this one where
            // tiles are taken in turn, keys and values of a tile else
            const int steps = 2 * nt;
            auto place = [&](int n, int &t0) -> bool {     // whether the n-th are values; the tile's first token
                int tile;
                bool v;
                if (dual) tile = n >> 1, v = n & 1;
                else if (n == 0 || n == steps - 1) tile = n == 0 ? 0 : nt - 1, v = n != 0;
                else tile = n & 1 ? (n + 1) >> 1 : (n >> 1) - 1, v = !(n & 1);
                t0 = (sg.tile0 + tile) * TOK;
                return v;
            };
            // A thread has 16 bytes of NC rows of a tile, STEP rows apart; a warp has WR rows. Where a row lies is
            // found by one lane (lane j: the warp's j-th row) and handed to the others by shuffles: by every lane for
            // itself it was most of the loaders' instructions.
            constexpr int CPR = I8 ? D / 16 : D / 8, NC = TOK * CPR / F::TEAM, STEP = F::TEAM / CPR;
            constexpr int SUB = 32 / CPR, WR = SUB * NC;
            static_assert(WR <= 32 && STEP % 8 == 0, "a lane a row; a thread's rows lie alike in the swizzle");
            const int c = t % CPR, row = t / CPR;
            const unsigned slots = sg.h * a.pool.page_tokens, within = a.pool.page_tokens - 1;
            // the page that holds the warp's row j in the n-th tile: -1 none
            auto row_of = [&](int j) { return (t >> 5) * SUB + j % SUB + j / SUB * STEP; };
            auto page_of = [&](int n, int j) -> int {
                if (n >= steps || j >= WR) return -1;
                int t0;
                const bool v = place(n, t0);
                const int at = t0 + row_of(j);
                if (at >= sg.length) return -1;
                const int page = table[at >> shift];
                if (unsigned(page) < unsigned(a.pool.pages)) return page;
                if (!v) atomicOr(&g_fault_shared, FAULT_PAGE);
                return -1;
            };
            auto slot_of = [&](int t0, int j) -> unsigned { return slots + (unsigned(t0 + row_of(j)) & within); };
            auto wait_empty = [&] { dead = dead || !warp_wait(&empty[load.at], load.phase ^ 1); };
            auto arrive = [&](const Slot &at) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[at.at]);
            };
            // starts the copies of the n-th tile's rows, `page` this lane's row's, to `to` and on in steps
            auto copy = [&](int n, int page, uint32_t to, int step) {
                int t0;
                const bool v = place(n, t0);
                constexpr int SIZE = I8 ? 1 : 2;
                const char *from = static_cast<const char *>(v ? a.pool.v : a.pool.k) +
                                   a.layer * a.pool.layer_stride * SIZE + c * 16;
                const int64_t mine = page < 0 ? -1 : (page * a.pool.page_stride + int64_t(slot_of(t0, lane)) * D) * SIZE;
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    const int64_t off = __shfl_sync(0xffffffffu, mine, i * SUB + lane / CPR);
                    cp16(to + i * step, from + (off < 0 ? 0 : off), off >= 0);
                }
            };
            if constexpr (I8) {
                // A tile's codes come asynchronously into places of this thread's own, as soon as it has converted
                // the team's tile before, while the other team's is converted; a row's scales come to the lane that
                // found the row.
                constexpr int WPR = D / 64;                // pairs of scales a row
                const uint8_t *const codes = raw + team * F::RAW_BYTES + t * 16;
                const uint32_t codes32 = smem_u32(codes);
                uint32_t next[WPR];
                auto fetch = [&](int n, int page) {
                    if (n >= steps) return;
                    copy(n, page, codes32, F::TEAM * 16);
                    cp_commit();
                    int t0;
                    const bool v = place(n, t0);
                    const uint16_t *from = (v ? a.pool.v_scales : a.pool.k_scales) + a.layer * a.pool.scale_layer_stride;
#pragma unroll
                    for (int e = 0; e < WPR; ++e) next[e] = 0; // a row without a page: zeros
                    if (page < 0) return;
                    from += page * a.pool.scale_page_stride + int64_t(slot_of(t0, lane)) * (D / 32);
                    if constexpr (WPR == 1) next[0] = *reinterpret_cast<const uint32_t *>(from);
                    else if constexpr (WPR == 2) {
                        const uint2 x = *reinterpret_cast<const uint2 *>(from);
                        next[0] = x.x, next[1] = x.y;
                    } else {
                        const uint4 x = *reinterpret_cast<const uint4 *>(from);
                        next[0] = x.x, next[1] = x.y, next[2] = x.z, next[3] = x.w;
                    }
                };
                fetch(team, page_of(team, lane));
                int page = page_of(team + F::TEAMS, lane);
                const int flip = c / 4 & 1;                // odd columns the other half first: other banks
                const uint32_t off = (c / 4) * F::KB + sw128_off(row, (c % 4) * 2 + flip);
#pragma unroll 1
                for (int n = team; n < steps; n += F::TEAMS) {
                    cp_wait<0>();
                    uint4 code[NC];
                    uint32_t pair[WPR];
#pragma unroll
                    for (int i = 0; i < NC; ++i) code[i] = *reinterpret_cast<const uint4 *>(codes + i * (F::TEAM * 16));
#pragma unroll
                    for (int e = 0; e < WPR; ++e) pair[e] = next[e];
                    wait_empty();
                    if (dead) break;
                    uint8_t *to = ring + load.at * F::TILE_BYTES;
#pragma unroll
                    for (int i = 0; i < NC; ++i) {
                        uint32_t two = __shfl_sync(0xffffffffu, pair[0], i * SUB + lane / CPR);
#pragma unroll
                        for (int e = 1; e < WPR; ++e) {
                            const uint32_t x = __shfl_sync(0xffffffffu, pair[e], i * SUB + lane / CPR);
                            two = c / 4 == e ? x : two;
                        }
                        const uint32_t s = __byte_perm(two, two, c & 2 ? 0x3232u : 0x1010u);
                        const uint32_t w[4] = {
                            (flip ? code[i].z : code[i].x) ^ 0x80808080u, (flip ? code[i].w : code[i].y) ^ 0x80808080u,
                            (flip ? code[i].x : code[i].z) ^ 0x80808080u, (flip ? code[i].y : code[i].w) ^ 0x80808080u};
                        *reinterpret_cast<uint4 *>(to + off + i * (STEP * 128)) =
                            make_uint4(dequant2(w[0], 0x4140u, s), dequant2(w[0], 0x4342u, s),
                                       dequant2(w[1], 0x4140u, s), dequant2(w[1], 0x4342u, s));
                        *reinterpret_cast<uint4 *>(to + (off ^ 16) + i * (STEP * 128)) =
                            make_uint4(dequant2(w[2], 0x4140u, s), dequant2(w[2], 0x4342u, s),
                                       dequant2(w[3], 0x4140u, s), dequant2(w[3], 0x4342u, s));
                    }
                    arrive(load);
                    load.forward(F::TEAMS, R);
                    fetch(n + F::TEAMS, page);
                    page = page_of(n + 2 * F::TEAMS, lane);
                }
                cp_wait<0>();
            } else {
                // a place is handed over when `lag` more are under way
                const int lag = min(R - 2, 3);
                Slot done = load;
                int page = page_of(0, lane);
                const uint32_t off = (c / 8) * F::KB + sw128_off(row, c % 8);
#pragma unroll 1
                for (int n = 0; n < steps; ++n) {
                    wait_empty();
                    if (dead) break;
                    copy(n, page, ring32 + load.at * F::TILE_BYTES + off, STEP * 128);
                    cp_commit();
                    page = page_of(n + 1, lane);
                    load.forward(1, R);
                    if (n >= lag) {
                        if (lag == 1) cp_wait<1>();
                        else if (lag == 2) cp_wait<2>();
                        else cp_wait<3>();
                        arrive(done);
                        done.forward(1, R);
                    }
                }
                cp_wait<0>();
                if (!dead)
                    for (int n = max(0, steps - lag); n < steps; ++n) {
                        arrive(done);
                        done.forward(1, R);
                    }
            }
        } else {
            // ------------------------------------- softmax -------------------------------------
            const int wg = warp / SOFT;
            const uint32_t lanes = tmem + (uint32_t(32 * (warp % SOFT)) << 16);
            const uint32_t o = lanes + F::O_COL + (TWO ? wg * F::O_STEP : 0);
            bool any = false;                              // the accumulators hold something
            const bool idle = (dual ? wg * ROWS : 0) + 32 * (warp % SOFT) >= live;     // no queries in its lanes
            for (int j = TWO ? wg : wg * jobs; j < jobs; j += TWO ? 2 : 1) {
                const int left = lim - (sg.tile0 + (dual ? j >> 1 : j)) * TOK;
                const uint32_t sc = lanes + F::S_COL + (j & 1) * F::S_STEP;
                // (a group that has its own score buffer keeps its phase in s_phase)
                const int phase = TWO || !(j & 1) ? s_phase : s_phase1;
                dead = dead || !warp_wait(&s_full[j & 1], phase);
                if (TWO || !(j & 1)) s_phase ^= 1; else s_phase1 ^= 1;
                if (dead) break;
                tc_fence_after();
                if (!TWO) pv_phase ^= 1;
                if (idle) {
                    if (lane == 0) mbar_arrive(&p_full[j & 1]);
                    continue;
                }
                const bool all = __all_sync(0xffffffffu, left >= TOK);
                float top = -INFINITY;
#pragma unroll 1
                for (int c = 0; c < TOK; c += 64) {
                    uint32_t x[32], y[32];
                    tmem_ld32(sc + c, x);
                    tmem_ld32(sc + c + 32, y);
                    tmem_ld_wait();
                    if (!all)
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            x[i] = c + i < left ? x[i] : 0xFF800000u;          // -inf
                            y[i] = c + 32 + i < left ? y[i] : 0xFF800000u;
                        }
                    float t1 = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        top = max3(top, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
                        t1 = max3(t1, __uint_as_float(y[i]), __uint_as_float(y[i + 1]));
                    }
                    top = fmaxf(top, t1);
                }
                // the maximum lags; where it has to follow, what has been added up follows too
                const bool move = top > m && !((top - m) * f <= F::GROW);
                if (__any_sync(0xffffffffu, move)) {
                    const float shrink = !move ? 1.0f : m == -INFINITY ? 0.0f : ex2((m - top) * f);
                    m = move ? top : m;
                    if (any) {
                        l *= shrink;
                        if (!TWO) {                        // the previous tile's product may still be adding
                            dead = !warp_wait(pv_done, pv_phase);
                            if (dead) break;
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
                const float from = m == -INFINITY ? 0.0f : m;
                float2 sum = make_float2(0.0f, 0.0f), sum1 = sum;
                // two scores' weights, the second of them that of token c + 1 of the tile
                auto weigh = [&](int c, uint32_t u, uint32_t v) -> float2 {
                    float2 e = fma2(sub2(make_float2(__uint_as_float(u), __uint_as_float(v)), from), f, F::BIAS);
                    e = make_float2(ex2(e.x), ex2(e.y));
                    if (!all) e = make_float2(c < left ? e.x : 0.0f, c + 1 < left ? e.y : 0.0f);
                    return e;
                };
                // two terms, 16 scores' loads under the weights of the 16 before: those of 32 tokens go over their
                // scores, the second terms of the first 16 once the other 16 scores are here
                uint32_t x[16], y[16], h[8], g[8];
                auto half = [&](int c, const uint32_t (&z)[16]) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 e = weigh(c + 2 * i, z[2 * i], z[2 * i + 1]);
                        if (i & 1) sum1 = add2(sum1, e); else sum = add2(sum, e);
                        h[i] = pack2<BF>(e.x, e.y);
                        g[i] = rest2<BF>(e.x, e.y, h[i]);
                    }
                };
                tmem_ld16(sc, x);
#pragma unroll 1
                for (int c = 0; c < TOK; c += 32) {
                    tmem_ld_wait();
                    tmem_ld16(sc + c + 16, y);
                    half(c, x);
                    tmem_st8(sc + c, h);
                    tmem_ld_wait();
                    tmem_st8(sc + c + 16, g);
                    if (c + 32 < TOK) tmem_ld16(sc + c + 32, x);
                    half(c + 16, y);
                    tmem_st8(sc + c + 8, h);
                    tmem_st8(sc + c + 24, g);
                }
                l += sum.x + sum.y + (sum1.x + sum1.y);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[j & 1]);
            }
            dead = dead || !warp_wait(o_done, o_phase);
            tc_fence_after();
        }
        o_phase ^= 1;
        if (dead) *s_dead = 1;
        __syncthreads();
        if (*s_dead) break;

        // -- the segment's results: rows of shared memory, then as whole rows to the workspace ----------------------
        float *const rows_out = reinterpret_cast<float *>(sm);
        const bool whole = sg.tile0 == 0 && nt == sg.tiles;
        auto place_of = [&](int r) -> int64_t {            // a query's row there
            const int rr = sg.mb * item + r, b = rr / p.G, head = sg.h * p.G + rr - b * p.G;
            return whole ? int64_t(sg.row0 + b) * a.q_heads + head
                         : (int64_t(blockIdx.x) * 2 + (sg.tile0 == 0)) * (2 * ROWS) + r;
        };
        if (warp < 2 * SOFT) {
            const int wg = warp / SOFT, row = tid % ROWS, r = dual ? tid : row;
            const uint32_t o = tmem + (uint32_t(32 * (warp % SOFT)) << 16) + F::O_COL + (TWO ? wg * F::O_STEP : 0);
            // one block of queries in two accumulators: each group puts down half of the columns, then adds the other
            // half
            const bool merge = TWO && !dual && jobs > 1;
            float mine = 1.0f;
            if (merge) {
                float2 *ml = reinterpret_cast<float2 *>(sm);
                ml[wg * ROWS + row] = make_float2(m, l);
                named_bar_sync(2, 2 * SOFT * 32);
                const float2 him = ml[(wg ^ 1) * ROWS + row];
                const float both = fmaxf(m, him.x), at = both == -INFINITY ? 0.0f : both;
                mine = m == -INFINITY ? 0.0f : ex2((m - at) * f);
                l = l * mine + (him.y == 0.0f ? 0.0f : him.y * ex2((him.x - at) * f));    // (a sum of NaN counts)
                m = both;
                named_bar_sync(2, 2 * SOFT * 32);
            }
            if (dual || merge || wg == 0)
                for (int half = 0; half < (merge ? 2 : 1); ++half) {
                    const int c0 = merge ? (wg ^ half) * (D / 2) : 0, c1 = merge ? c0 + D / 2 : D;
#pragma unroll 1
                    for (int c = c0; c < c1; c += 32) {
                        uint32_t x[32];
                        tmem_ld32(o + c, x);
                        tmem_ld_wait();
                        float4 *to = reinterpret_cast<float4 *>(rows_out + r * PS + c);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            float4 v = make_float4(__uint_as_float(x[4 * i]), __uint_as_float(x[4 * i + 1]),
                                                   __uint_as_float(x[4 * i + 2]), __uint_as_float(x[4 * i + 3]));
                            if (merge) {
                                const float4 w = half ? to[i] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                                v = make_float4(fmaf(v.x, mine, w.x), fmaf(v.y, mine, w.y), fmaf(v.z, mine, w.z),
                                                fmaf(v.w, mine, w.w));
                            }
                            to[i] = v;
                        }
                    }
                    if (merge && half == 0) named_bar_sync(2, 2 * SOFT * 32);
                }
            // the maximum as a power of two, the probabilities' height taken off
            if (r < live && (dual || wg == 0))
                (whole ? p.w.direct_ml : p.w.piece_ml)[place_of(r)] =
                    make_float2(m == -INFINITY ? -INFINITY : m * f - F::BIAS, l);
            tc_fence_before();
        }
        __syncthreads();
#pragma unroll 1
        for (int i = tid; i < live * (D / 4); i += THREADS) {
            const int r = i / (D / 4), c = i % (D / 4) * 4;
            *reinterpret_cast<float4 *>((whole ? p.w.direct : p.w.piece) + place_of(r) * D + c) =
                *reinterpret_cast<const float4 *>(rows_out + r * PS + c);
        }
        unit += nt;
        if (unit >= unit1) break;
        if (unit == cum[sg.g + 1]) {                       // the next group that has units
            do ++sg.g; while (cum[sg.g + 1] == unit);
            sg.row0 = a.first[sg.g], sg.rows = a.first[sg.g + 1] - sg.row0;
            sg.page_row = row_seq(a, sg.row0);
            sg.length = min(max(a.prefix[sg.g], 0), row_len(a, sg.page_row));
        }
        __syncthreads();
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

// The parts of a row's query head joined: prefix pieces in the order of their blocks, then what the row has of its
// own. A block a query head: every warp finds the common maximum and sum, a part a lane, and adds up every JOIN-th
// part's accumulators, four parts' loads at a time and the first four's under way meanwhile; the warps' sums are
// added in shared memory. It is bound by the chain plan -> maxima -> accumulators and by how many blocks pass through
// an SM. us at 1 / 2 / 4 / 8 warps: 64 rows of 32 heads of 128, 10 parts 6.8 / 6.5 / 7.9 / 12.5; 17 rows of 16 heads
// of 256, 28 parts 10.4 / 7.9 / 6.1 / 6.0 (19 by a warp that took one part after another).
template <int D> constexpr int JOIN_WARPS = D == 256 ? 4 : 2;
template <int D> __global__ void __launch_bounds__(JOIN_WARPS<D> * 32) join_kernel(const __grid_constant__ Params p, int tok) {
    constexpr int JOIN = JOIN_WARPS<D>, N = D / 32;        // elements a lane
    __shared__ __align__(16) float s_o[JOIN][D];
    const SharedArgs &a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t i = blockIdx.x;
    const int b = int(i / a.q_heads), head = int(i - int64_t(b) * a.q_heads), h = head / p.G;
    pdl_launch_dependents();
    pdl_wait();
    const Plan &pl = *p.w.plan;
    const float own = p.w.own_lse[i];
    const int g = pl.group[b];
    // parts: n prefix pieces, of which the first block's is in its second place, the others' in their first; then the
    // own one
    int n = 0;
    const float *piece = p.w.direct + i * D;
    const float2 *ml = p.w.direct_ml + i;
    int64_t step = 0, skip = 0;
    if (g >= 0 && pl.length[g] > 0) {
        const int item = pl.item, size = pl.size, tiles = (pl.length[g] + tok - 1) / tok;
        const int row0 = a.first[g], rows = a.first[g + 1] - row0;
        const int rr = (b - row0) * p.G + head - h * p.G, mb = rr / item, blocks = (rows * p.G + item - 1) / item;
        const int u0 = pl.cum[g] + (h * blocks + mb) * tiles, f0 = u0 / size;
        n = (u0 + tiles - 1) / size - f0 + 1;
        if (n > 1) {
            const int64_t first = int64_t(f0) * (4 * ROWS) + rr % item;
            piece = p.w.piece + first * D, ml = p.w.piece_ml + first;
            step = 4 * ROWS, skip = 2 * ROWS;
        }
    }
    // a part's maximum (base 2) and sum (of zero: it has no tokens, and its accumulators may hold anything)
    auto part = [&](int k) -> float2 {
        if (k == n) return make_float2(own * 1.4426950408889634f, own != -INFINITY ? 1.0f : 0.0f);
        return k < n ? ml[k * step + (k ? 0 : skip)] : make_float2(0.0f, 0.0f);
    };
    float2 x[4];
    float v[4][N];
    auto load = [&](int k0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = k0 + j * JOIN;
            x[j] = part(k);
            const float *from = (k < n ? piece + (k * step + (k ? 0 : skip)) * D : p.w.own_out + i * D) + lane * N;
#pragma unroll
            for (int e = 0; e < N; e += 2) {
                const float2 y = k <= n ? *reinterpret_cast<const float2 *>(from + e) : make_float2(0.0f, 0.0f);
                v[j][e] = y.x, v[j][e + 1] = y.y;
            }
        }
    };
    load(warp);                                            // under way while the maximum is found
    float m = -INFINITY, l = 0.0f;
    for (int k = lane; k <= n; k += 32) {
        const float2 y = part(k);
        if (y.y != 0.0f) m = fmaxf(m, y.x);
    }
#pragma unroll
    for (int k = 16; k; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
    for (int k = lane; k <= n; k += 32) {
        const float2 y = part(k);
        if (y.y != 0.0f) l = fmaf(y.y, ex2(y.x - m), l);   // (a sum of NaN counts)
    }
#pragma unroll
    for (int k = 16; k; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
    float o[N];
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = 0.0f;
    for (int k0 = warp; k0 <= n; k0 += 4 * JOIN) {
        if (k0 != warp) load(k0);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float w = x[j].y != 0.0f ? ex2(x[j].x - m) : 0.0f;
#pragma unroll
            for (int e = 0; e < N; ++e) o[e] = w != 0.0f ? fmaf(v[j][e], w, o[e]) : o[e];
        }
    }
#pragma unroll
    for (int e = 0; e < N; e += 2) *reinterpret_cast<float2 *>(&s_o[warp][lane * N + e]) = make_float2(o[e], o[e + 1]);
    __syncthreads();
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    for (int d = threadIdx.x; d < D; d += JOIN * 32) {
        float x = s_o[0][d];
#pragma unroll
        for (int k = 1; k < JOIN; ++k) x += s_o[k][d];
        x *= inv;
        const int64_t at = int64_t(b) * a.ldo + int64_t(head) * D + d;
        if (a.odt == DT_F32) static_cast<float *>(a.out)[at] = x;
        else if (a.odt == DT_F16) static_cast<uint16_t *>(a.out)[at] = f2h_bits(x);
        else static_cast<uint16_t *>(a.out)[at] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
    }
    if (a.lse && threadIdx.x == 0) a.lse[i] = l == 0.0f ? -INFINITY : m * 0.6931471805599453f + logf(l);
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
        e = cudaFuncSetAttribute(prefix_kernel<KT, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, F::SMEM);
        if (e != cudaSuccess) return e;
        opted[dev] = 1;
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_sms());
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = F::SMEM;        // above half of an SM's: one block an SM, which takes all of the tensor memory
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, prefix_kernel<KT, D>, p)) != cudaSuccess) return e;
    // what the rows have of their own: the cache's attention from each row's prefix on
    AttendArgs own = {};
    const SharedArgs &a = p.a;
    own.pool = a.pool, own.t = a.t, own.seqs = a.seqs, own.q = a.q, own.ldq = a.ldq;
    own.rope = a.rope, own.rope_rows = a.rope_rows;
    own.out = p.w.own_out, own.ldo = int64_t(a.q_heads) * D, own.lse = p.w.own_lse, own.ws = a.ws, own.window = 0;
    own.scale = a.scale, own.layer = a.layer, own.B = a.B, own.q_heads = a.q_heads, own.qdt = a.qdt, own.odt = DT_F32;
    own.from = p.w.plan->from;
    if ((e = launch_kv_attend(own, s)) != cudaSuccess) return e;
    // One after the other: blocks that come early, while their predecessors' still run, gather on the SMs that are
    // done first and then wait there for one another's loads (64 samples / 32 rows of 65531 / 17 rows with heads of
    // 256, us in a graph: both early 52.3 / 150.5 / 107, the attention alone 48.5 / 141 / 54.6, neither 46.5 / 135 /
    // 54.5).
    cfg.gridDim = dim3(unsigned(int64_t(a.B) * a.q_heads));
    cfg.blockDim = dim3(JOIN_WARPS<D> * 32);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 0;
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
