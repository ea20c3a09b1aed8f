// qpack_paged.cu — the paged KV cache: appending new tokens (rotary embedding, 8-bit quantization or rounding to 16
// bits, scatter into pages), reading rows back, and the page operators (reserve, fork, free, compact, copy).
//
// Append and read are streams: every element is read and written once, so HBM bounds them at length and the launch at
// a decode step's few tokens. 8191 tokens of 8 heads of 128 in fp16: append into 8 bits 14.6 us (52% of the copy rate),
// read back 11.4 us (66%); at 100000 tokens 74% and 89%. Append is held up by its own chain in each warp (loads, scales,
// codes) with 24 warps an SM (below, at the kernel, what more and fewer cost).
// The page operators move the pages that they have to (HBM bound: 598 MB of pages compacted in 195 us, 91% of the copy
// rate) after a plan on the tables alone (a few us of dependent loads). All of it is deterministic: pages are ranked by
// number and requests by place, never by arrival.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qpack_dev.cuh"
#include "qpack_launch.h"
#include "qpack_paged.cuh"
#include "qpack_quot.cuh"

namespace qpack {
namespace {

__device__ int g_fault_paged = 0;

// ------------------------------------------------------------------------------------------------------------
// Append and read back
// ------------------------------------------------------------------------------------------------------------
template <int DT> __device__ __forceinline__ void store8(void *p, int64_t idx, const float *x) {
    if (DT == DT_F32) {
        float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(p) + idx);
        o[0] = make_float4(x[0], x[1], x[2], x[3]);
        o[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (DT == DT_F16) {
                w[e] = uint32_t(f2h_bits(x[2 * e])) | (uint32_t(f2h_bits(x[2 * e + 1])) << 16);
            } else {
                const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
                w[e] = *reinterpret_cast<const uint32_t *>(&b);
            }
        }
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + idx) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// A warp takes one token, U x RPW heads of its keys and of its values: eight consecutive elements a lane, so a row of D
// takes D / 8 lanes, RPW = 256 / D rows a pass. The token's place (sequence and position, then the page: two dependent
// loads) is found once for all of them, while appended rows are in flight; with a row a warp that chain of loads was
// the time (57 us against 23 for 8191 tokens written and read back).
constexpr int ROW_WARPS = 4, ROW_U = 4;

struct Place {
    int page, pos, slot;   // page -1: nowhere (a skipped token, or one out of range)
};

// First the sequence and the position, loaded together where both are given.
__device__ __forceinline__ int64_t spot_of(const AppendArgs &a, int64_t i, Place &p) {
    p = {-1, -1, 0};
    const int64_t seq = a.seqs ? int64_t(a.seqs[i]) : i;
    if (a.pos) p.pos = a.pos[i];
    if (a.pos && p.pos < 0) {                              // skipped, whatever its sequence
        p.pos = -1;
        return 0;
    }
    if (seq < 0 || seq >= a.t.seqs) {
        p.pos = -1;
        return -1;
    }
    if (!a.pos) p.pos = a.t.lens[seq] - 1;
    p.slot = p.pos & (a.pool.page_tokens - 1);
    return seq;
}
__device__ __forceinline__ void page_of(const AppendArgs &a, int64_t seq, Place &p, bool report) {
    bool bad = seq < 0 || p.pos < -1;                      // a length below 0
    if (p.pos >= 0) {
        const int col = p.pos >> (31 - __clz(a.pool.page_tokens));
        p.page = col < a.t.max_pages ? a.t.tables[seq * a.t.stride + col] : -1;
        bad = p.page < 0 || p.page >= a.pool.pages;
        if (bad) p.page = -1;
    }
    if (bad && report) atomicOr(&g_fault_paged, FAULT_PAGE);
}

// Eight consecutive elements as loaded, and as fp32. Plain loads, as of all that the previous grid may have written: these
// kernels begin while it runs.
template <int DT> struct Raw { uint32_t w[DT == DT_F32 ? 8 : 4]; };
template <int DT> __device__ __forceinline__ void load_raw(const void *p, int64_t idx, Raw<DT> &r) {
    const uint4 *q = DT == DT_F32 ? reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + idx)
                                  : reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + idx);
#pragma unroll
    for (int i = 0; i < (DT == DT_F32 ? 2 : 1); ++i) {
        const uint4 v = q[i];
        r.w[4 * i] = v.x, r.w[4 * i + 1] = v.y, r.w[4 * i + 2] = v.z, r.w[4 * i + 3] = v.w;
    }
}
template <int DT> __device__ __forceinline__ void convert(const Raw<DT> &r, float *x) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (DT == DT_F32) x[e] = __uint_as_float(r.w[e % (DT == DT_F32 ? 8 : 4)]);
        else if (DT == DT_F16) x[e] = h2f_bits(uint16_t(e & 1 ? r.w[e / 2] >> 16 : r.w[e / 2] & 0xFFFFu));
        else x[e] = __uint_as_float(e & 1 ? r.w[e / 2] & 0xFFFF0000u : r.w[e / 2] << 16);
    }
}

// The rotation's partner (i +- D/2) is D/16 lanes away, and the four lanes of a 32-element group reduce its maximum
// with two shuffles.
// Blocks an SM (us; 100000 tokens of 8 heads of 128; bytes that spill at 4, 5, 6, 7, 8 in brackets):
//   fp32 into 8 bits    4 171, 5 167, 6 222, 7 265, 8 244 (0, 0, 248, 456, 472)     into bf16  186, 178, 211, 222, 223
//   fp16 into 8 bits    4 165, 5 144, 6 124, 7 130, 8 137 (0, 0, 24, 68, 176)       into bf16  154, 129, 124, 124, 129
//   bf16 into 8 bits    4 165, 5 144, 6 133, 7 137, 8 143 (0, 0, 28, 112, 196)      into bf16  165, 137, 129, 125, 125
// 8191 tokens, and widths of 64 and 256, fall in the same order but for fp32 into 8 bits, where 4 takes 18.2 us and 5 18.5,
// and bf16 into 8 bits at 256, where 5 and 7 are 5% faster than 6. So 5 from fp32, and from 16 bits 6 into 8 bits, whose few
// spilled bytes cost less than a block fewer, 7 into 16 bits, which do not spill.
template <int KT, int D, int DT>
__global__ void __launch_bounds__(ROW_WARPS * 32, DT == DT_F32 ? 5 : KT == QPACK_KV_I8 ? 6 : 7)
    kv_append_kernel(AppendArgs a, int64_t first, unsigned items, unsigned groups) {
    constexpr int LPR = D / 8, RPW = 32 / LPR, U = ROW_U;
    const int lane = threadIdx.x & 31, sub = lane % LPR, H = a.pool.heads;
    pdl_launch_dependents();
    const unsigned item = blockIdx.x * ROW_WARPS + (threadIdx.x >> 5), tok_in = groups == 1 ? item : item / groups;
    const int head0 = int(item - tok_in * groups) * (U * RPW) + lane / LPR;
    pdl_wait();
    if (item >= items) return;                             // whole warps
    const int64_t tok = first + tok_in;
    Raw<DT> raw[2][U];
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        const int64_t row = tok * (v ? a.ldv : a.ldk) + sub * 8;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (head0 + u * RPW < H) load_raw<DT>(v ? a.v : a.k, row + (head0 + u * RPW) * D, raw[v][u]);
            else raw[v][u] = Raw<DT>{};
    }
    Place pl;
    const int64_t seq = spot_of(a, tok, pl);
    float c[8] = {1, 1, 1, 1, 1, 1, 1, 1}, s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (a.rope && pl.pos >= 0 && pl.pos < a.rope_rows) {
        const int64_t at = int64_t(pl.pos) * D + (sub % (LPR / 2)) * 8;
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
            const float4 x = *reinterpret_cast<const float4 *>(a.rope + at + e);
            const float4 y = *reinterpret_cast<const float4 *>(a.rope + at + D / 2 + e);
            c[e] = x.x, c[e + 1] = x.y, c[e + 2] = x.z, c[e + 3] = x.w;
            s[e] = y.x, s[e + 1] = y.y, s[e + 2] = y.z, s[e + 3] = y.w;
        }
    }
    page_of(a, seq, pl, lane == 0);
    if (pl.page < 0) return;
    const int64_t page = a.layer * a.pool.layer_stride + pl.page * a.pool.page_stride;
    const int64_t spage = a.layer * a.pool.scale_layer_stride + pl.page * a.pool.scale_page_stride;
    const unsigned in_page = (unsigned(head0) * a.pool.page_tokens + pl.slot) * unsigned(D) + sub * 8;
    const unsigned pass = unsigned(RPW) * a.pool.page_tokens * unsigned(D);            // to the next row of the lane
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        float x[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) convert<DT>(raw[v][u], x[u]);
        if (a.rope && v == 0) {
            if (pl.pos >= a.rope_rows && lane == 0) atomicOr(&g_fault_paged, FAULT_PAGE);
            // lower half: x c - y s; upper half: x c + y s; each operation rounded
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] = sub < LPR / 2 ? -s[e] : s[e];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float y = __shfl_xor_sync(0xffffffffu, x[u][e], LPR / 2);
                    x[u][e] = __fadd_rn(__fmul_rn(x[u][e], c[e]), __fmul_rn(y, s[e]));
                }
        }
        if (KT != QPACK_KV_I8) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (head0 + u * RPW < H)
                    store8<KT == QPACK_KV_F16 ? DT_F16 : DT_BF16>(v ? a.pool.v : a.pool.k, page + in_page + u * pass, x[u]);
            continue;
        }
        // The scales: the four lanes of a group hold the maxima of U = 4 rows alike, so lane k of them does row k's two
        // divisions for all.
        static_assert(U == 4, "a lane a row");
        float m[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            m[u] = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) m[u] = fmaxf(m[u], fabsf(x[u][e]));
            m[u] = fmaxf(m[u], __shfl_xor_sync(0xffffffffu, m[u], 1));
            m[u] = fmaxf(m[u], __shfl_xor_sync(0xffffffffu, m[u], 2));
        }
        const int k = lane & 3;
        const float mine = k & 2 ? (k & 1 ? m[3] : m[2]) : (k & 1 ? m[1] : m[0]);
        const uint16_t d16 = f2h_bits(fminf(__fdiv_rn(mine, 127.0f), 65504.0f));
        const float d = h2f_bits(d16), rs = d > 0.0f ? __frcp_rn(d) : 0.0f;     // a scale of 0 gives codes of 0
        // A scale that fp16 holds as a normal number below its largest is off by at most 2^-11 of max / 127, so no quotient
        // is beyond 127.07 and none needs the clamp. The others, subnormal or cut to 65504, take the written definition
        // below (their reciprocal goes negative).
        const float give = d < 0x1p-14f || d >= 65504.0f ? -rs : rs;
        uint32_t w[U][2];
        bool plain[U], any = false;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float r0 = __shfl_sync(0xffffffffu, give, (lane & ~3) + u), r = fabsf(r0);
            // q = rint(x r) read from the low byte of x r + 1.5 2^23. x r is within 2^-24 |x / d| of x / d, and the
            // rounded quotient too, together less than 2^-16: where x r is nearer than 1/2 - 2^-15 to q, q is the
            // quotient's rint.
            float y[8], off = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                y[e] = __fmaf_rn(x[u][e], r, 12582912.0f);
                off = fmaxf(off, fabsf(__fmaf_rn(x[u][e], r, 12582912.0f - y[e])));
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t lo = __byte_perm(__float_as_uint(y[4 * e]), __float_as_uint(y[4 * e + 1]), 0x0040u);
                const uint32_t hi = __byte_perm(__float_as_uint(y[4 * e + 2]), __float_as_uint(y[4 * e + 3]), 0x0040u);
                w[u][e] = __byte_perm(lo, hi, 0x5410u);
            }
            plain[u] = !(off <= 0.5f - 0x1p-15f) || r0 < 0.0f;
            any |= plain[u];
        }
        if (__any_sync(0xffffffffu, any)) {                // rare
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float du = h2f_bits(uint16_t(__shfl_sync(0xffffffffu, int(d16), (lane & ~3) + u)));
                if (!plain[u] || !(du > 0.0f)) continue;
                uint8_t cb[8];
                rint_codes<8>(x[u], du, __frcp_rn(du), 0, -127, 127, 0, cb);
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    w[u][e] = cb[4 * e] | uint32_t(cb[4 * e + 1]) << 8 | uint32_t(cb[4 * e + 2]) << 16 |
                              uint32_t(cb[4 * e + 3]) << 24;
            }
        }
        int8_t *base = static_cast<int8_t *>(v ? a.pool.v : a.pool.k) + page + in_page;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (head0 + u * RPW < H) *reinterpret_cast<uint2 *>(base + u * pass) = make_uint2(w[u][0], w[u][1]);
        if (head0 + k * RPW < H) (v ? a.pool.v_scales : a.pool.k_scales)[spage + (in_page + k * pass) / 32] = d16;
    }
}

// Rows of the cache as they stand for: code x scale rounded to fp16 (the definition of the 8-bit cache), then to DT.
template <int KT, int D, int DT>
__global__ void __launch_bounds__(ROW_WARPS * 32, 8) kv_read_kernel(AppendArgs a, int64_t first, unsigned items, unsigned groups) {
    constexpr int LPR = D / 8, RPW = 32 / LPR, U = ROW_U;
    const int lane = threadIdx.x & 31, sub = lane % LPR, H = a.pool.heads;
    pdl_launch_dependents();
    const unsigned item = blockIdx.x * ROW_WARPS + (threadIdx.x >> 5), tok_in = groups == 1 ? item : item / groups;
    const int head0 = int(item - tok_in * groups) * (U * RPW) + lane / LPR;
    pdl_wait();
    if (item >= items) return;                             // whole warps
    const int64_t tok = first + tok_in;
    Place pl;
    const int64_t seq = spot_of(a, tok, pl);
    page_of(a, seq, pl, lane == 0);
    const int64_t page = a.layer * a.pool.layer_stride + pl.page * a.pool.page_stride;
    const int64_t spage = a.layer * a.pool.scale_layer_stride + pl.page * a.pool.scale_page_stride;
    const unsigned in_page = (unsigned(head0) * a.pool.page_tokens + pl.slot) * unsigned(D) + sub * 8;
    const unsigned pass = unsigned(RPW) * a.pool.page_tokens * unsigned(D);
    constexpr int WORDS = KT == QPACK_KV_I8 ? 2 : 4;
    uint32_t w[2][U][WORDS], sc[2][U];
#pragma unroll
    for (int v = 0; v < 2; ++v)
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int e = 0; e < WORDS; ++e) w[v][u][e] = 0u;
            sc[v][u] = 0u;
            if (pl.page < 0 || head0 + u * RPW >= H || !(v ? a.v : a.k)) continue;
            const void *base = v ? a.pool.v : a.pool.k;
            if (KT == QPACK_KV_I8) {
                const uint2 q = *reinterpret_cast<const uint2 *>(static_cast<const int8_t *>(base) + page + in_page + u * pass);
                w[v][u][0] = q.x, w[v][u][1] = q.y;
                sc[v][u] = (v ? a.pool.v_scales : a.pool.k_scales)[spage + (in_page + u * pass) / 32];
            } else {
                const uint4 q = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + page + in_page + u * pass);
                w[v][u][0] = q.x, w[v][u][1] = q.y, w[v][u][WORDS - 2] = q.z, w[v][u][WORDS - 1] = q.w;
            }
        }
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        void *out = v ? a.v : a.k;
        if (!out) continue;
        const int64_t row = tok * (v ? a.ldv : a.ldk) + sub * 8;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (head0 + u * RPW >= H) continue;
            uint32_t h[4];                                 // eight 16-bit values
            if (KT == QPACK_KV_I8) {
                const uint32_t s = sc[v][u] | sc[v][u] << 16;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t c = w[v][u][e] ^ 0x80808080u;
                    h[2 * e] = dequant2(c, 0x4140u, s), h[2 * e + 1] = dequant2(c, 0x4342u, s);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) h[e] = w[v][u][e % WORDS];
            }
            const int64_t at = row + (head0 + u * RPW) * D;
            constexpr int HT = KT == QPACK_KV_BF16 ? DT_BF16 : DT_F16;
            if (DT == HT) {
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + at) = make_uint4(h[0], h[1], h[2], h[3]);
            } else {
                Raw<HT> r = {h[0], h[1], h[2], h[3]};
                float x[8];
                convert<HT>(r, x);
                store8<DT>(out, at, x);
            }
        }
    }
}

// Launches a kernel that waits for the previous grid itself: its blocks are set up while that one ends.
template <class... A> cudaError_t launch_dependent(void (*kernel)(A...), int64_t grid, int threads, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(grid));
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int KT, int D, int DT> cudaError_t run_rows(const AppendArgs &a, bool read, cudaStream_t s) {
    constexpr int heads = ROW_U * (256 / D);               // a warp's
    const unsigned groups = (a.pool.heads + heads - 1) / heads;
    const int64_t most = (int64_t(1) << 30) / groups;      // tokens a launch: item numbers stay below 2^31
    for (int64_t i = 0; i < a.n; i += most) {
        const int64_t n = a.n - i < most ? a.n - i : most;
        const unsigned items = unsigned(n * groups);
        const cudaError_t e = launch_dependent(read ? kv_read_kernel<KT, D, DT> : kv_append_kernel<KT, D, DT>,
                                               (items + ROW_WARPS - 1) / ROW_WARPS, ROW_WARPS * 32, s, a, i, items, groups);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <int KT, int D> cudaError_t rows_dt(const AppendArgs &a, bool read, cudaStream_t s) {
    if (a.dt == DT_F32) return run_rows<KT, D, DT_F32>(a, read, s);
    if (a.dt == DT_F16) return run_rows<KT, D, DT_F16>(a, read, s);
    return run_rows<KT, D, DT_BF16>(a, read, s);
}

template <int KT> cudaError_t rows_dim(const AppendArgs &a, bool read, cudaStream_t s) {
    if (a.pool.dim == 64) return rows_dt<KT, 64>(a, read, s);
    if (a.pool.dim == 128) return rows_dt<KT, 128>(a, read, s);
    return rows_dt<KT, 256>(a, read, s);
}

cudaError_t rows_kind(const AppendArgs &a, bool read, cudaStream_t s) {
    if (a.pool.type == QPACK_KV_I8) return rows_dim<QPACK_KV_I8>(a, read, s);
    if (a.pool.type == QPACK_KV_F16) return rows_dim<QPACK_KV_F16>(a, read, s);
    return rows_dim<QPACK_KV_BF16>(a, read, s);
}

// ------------------------------------------------------------------------------------------------------------
// Page operators
// ------------------------------------------------------------------------------------------------------------
constexpr int PLAN_THREADS = 1024;

// Exclusive prefix sum of one value a thread over the block; *total gets the sum. Every thread calls it.
template <class V> __device__ __forceinline__ V block_scan(V v, V *warp_sums, V *total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
    V x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const V y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[w] = x;
    __syncthreads();
    if (w == 0) {
        V y = lane < nw ? warp_sums[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const V z = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) y += z;
        }
        if (lane < nw) warp_sums[lane] = y;
    }
    __syncthreads();
    const V before = w ? warp_sums[w - 1] : 0;
    *total = warp_sums[nw - 1];
    __syncthreads();                                       // warp_sums may be written again
    return before + x - v;
}

// Reference counts are ranked in chunks of SCAN a thread, so that a few thousand pages are one pass of the block (a page
// a thread took seven passes of three barriers each, 3 us, at 1600 pages).
constexpr int SCAN = 8;
__device__ __forceinline__ void load_refs(const int *refs, int64_t p, int64_t pages, int (&r)[SCAN]) {
#pragma unroll
    for (int i = 0; i < SCAN; ++i) r[i] = p + i < pages ? refs[p + i] : 0;
}
// Bit i: page p + i exists and passes `test` of its count and number.
template <class Test> __device__ __forceinline__ unsigned pages_where(const int (&r)[SCAN], int64_t p, int64_t pages, Test test) {
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < SCAN; ++i)
        if (p + i < pages && test(r[i], p + i)) m |= 1u << i;
    return m;
}
__device__ __forceinline__ unsigned free_pages(const int *refs, int64_t p, int64_t pages) {
    int r[SCAN];
    load_refs(refs, p, pages, r);
    return pages_where(r, p, pages, [](int n, int64_t) { return n == 0; });
}

// Work of the copy kernel: rows [0, rows) of page src to page dst, in every layer.
struct CopyItem { int src, dst, rows; };

// Workspace of the page operators: the number of items, the items, and compaction's new page numbers.
struct PageWs {
    int *count;        // [4]
    CopyItem *items;   // [cap]
    int *map;          // [pages]
};
__host__ __device__ inline int64_t copy_cap(int64_t pages) { return pages / 2 + 4096; }
__host__ __device__ inline PageWs page_ws(void *ws, int64_t pages) {
    PageWs w;
    w.count = static_cast<int *>(ws);
    w.items = reinterpret_cast<CopyItem *>(w.count + 4);
    w.map = reinterpret_cast<int *>(w.items + copy_cap(pages));
    return w;
}

// One block: the pages that the requests need, in order, are the lowest-numbered free ones. The offsets of the requests
// (how many pages those before need) stay in shared memory, cut to one more than there are pages: what is behind is
// refused alike, and 4096 requests of 2^31 pages fit. The free pages are ranked chunk by chunk and each finds its request by
// a binary search over the offsets.
__global__ void __launch_bounds__(PLAN_THREADS) kv_reserve_kernel(qpack_kv_tables_t t, int page_tokens, const int *seqs,
                                                                  const int *add, int n, int64_t pages) {
    __shared__ long long needs[32];
    __shared__ int sums[32], who[4096];                    // a request's row of the table
    __shared__ unsigned off[4097];                         // pages needed before request i
    auto first_col = [&](int seq) {                        // the column of its first new page (lens is raised last)
        return (int64_t(t.lens[seq]) + page_tokens - 1) / page_tokens;
    };
    auto behind = [&](int seq, int i) {                    // and the one behind its last
        return (int64_t(t.lens[seq]) + add[i] + page_tokens - 1) / page_tokens;
    };
    const long long top = pages + 1;
    const int64_t longest = int64_t(t.max_pages) * page_tokens;
    long long want = 0, all;
    int tot;
    pdl_launch_dependents();
    pdl_wait();
    for (int i0 = 0; i0 < n; i0 += blockDim.x) {
        const int i = i0 + threadIdx.x;
        long long need = 0;
        int s = -1;
        if (i < n) {
            s = seqs[i];
            if (s >= 0 && s < t.seqs && add[i] >= 0 && t.lens[s] >= 0 && t.lens[s] <= longest) {
                const int64_t neu = int64_t(t.lens[s]) + add[i], last = behind(s, i);
                if (last > t.max_pages || neu > 0x7FFFFFFF)
                    s = -2;                                // its row cannot hold them
                else
                    need = last - first_col(s);
            } else {
                s = s < 0 ? -1 : -3;
            }
        }
        const long long before = want + block_scan(need, needs, &all);
        if (i < n) {
            off[i] = unsigned(min(before, top));
            who[i] = s;
            if (s == -2) atomicOr(&g_fault_paged, FAULT_NO_PAGES);
            if (s == -3) atomicOr(&g_fault_paged, FAULT_PAGE);
        }
        want += all;
    }
    want = min(want, top);
    if (threadIdx.x == 0) off[n] = unsigned(want);
    __syncthreads();
    int64_t found = 0;
    for (int64_t p0 = 0; p0 < pages && found < want; p0 += blockDim.x * SCAN) {
        const int64_t p = p0 + threadIdx.x * SCAN;
        unsigned m = free_pages(t.refs, p, pages);
        int64_t rank = found + block_scan(__popc(m), sums, &tot);
        for (; m && rank < want; m &= m - 1, ++rank) {
            int lo = 0, hi = n;                            // off[lo] <= rank < off[lo + 1]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (off[mid] <= rank) lo = mid; else hi = mid;
            }
            // requests that need nothing share their offset with the next one: the last of them owns the rank
            const int page = int(p) + __ffs(m) - 1;
            t.tables[int64_t(who[lo]) * t.stride + first_col(who[lo]) + (rank - off[lo])] = page;
            t.refs[page] = 1;
        }
        found += tot;
    }
    if (found > want) found = want;
    __syncthreads();
    // Requests up to the last that the free pages cover stand; one that they cover in part gives its pages back, before any
    // length is raised: a sequence listed twice, which no call may do, then still finds the places that it wrote to.
    auto stands = [&](int i) { return off[i + 1] <= found || behind(who[i], i) == first_col(who[i]); };
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int s = who[i];
        if (s < 0 || stands(i)) continue;
        atomicOr(&g_fault_paged, FAULT_NO_PAGES);
        for (int64_t j = off[i]; j < found && j < off[i + 1]; ++j) {
            int *e = t.tables + int64_t(s) * t.stride + first_col(s) + (j - off[i]);
            t.refs[*e] = 0;
            *e = -1;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x)
        if (who[i] >= 0 && stands(i)) t.lens[who[i]] += add[i];
}

// One block a child. Its place among the children that need a page is a count over the parents before it, its page the
// free one of that rank. Tables, lengths and counts of live pages are written here; the fresh page's own count is
// written by the copy that follows, since other blocks still read it as free here.
__global__ void __launch_bounds__(256) kv_fork_kernel(qpack_kv_tables_t t, int page_tokens, const int *src,
                                                      const int *dst, int n, int64_t pages, PageWs w) {
    __shared__ int sums[32];
    __shared__ int s_fresh;
    pdl_launch_dependents();
    pdl_wait();
    const int i = blockIdx.x;
    const int s = src[i], d = dst[i];
    auto known = [&](int q) {                              // a sequence, with a length that its row can hold
        return q >= 0 && q < t.seqs && t.lens[q] >= 0 && t.lens[q] <= int64_t(t.max_pages) * page_tokens;
    };
    auto len_of = [&](int q) { return known(q) ? t.lens[q] : 0; };
    int before = 0, tot;
    int mine = 0;
    for (int j = threadIdx.x; j < i; j += blockDim.x) mine += (len_of(src[j]) & (page_tokens - 1)) != 0;
    block_scan(mine, sums, &before);
    if (threadIdx.x == 0) s_fresh = -1;
    __syncthreads();
    const int len = len_of(s), full = len / page_tokens, rows = len & (page_tokens - 1);
    if (rows) {
        int found = 0;
        for (int64_t p0 = 0; p0 < pages && found <= before; p0 += blockDim.x * SCAN) {
            const int64_t p = p0 + threadIdx.x * SCAN;
            unsigned m = free_pages(t.refs, p, pages);
            const int rank = found + block_scan(__popc(m), sums, &tot);
            if (rank <= before && before < rank + __popc(m)) {
                for (int k = rank; k < before; ++k) m &= m - 1;
                s_fresh = int(p) + __ffs(m) - 1;
            }
            found += tot;
        }
        __syncthreads();
    }
    const bool ok_seq = known(s) && d >= 0 && d < t.seqs;
    const int fresh = s_fresh;
    const bool grant = ok_seq && t.lens[d] == 0 && (rows == 0 || fresh >= 0);
    const int last = ok_seq && rows ? t.tables[int64_t(s) * t.stride + full] : -1;
    const bool copy = grant && rows && last >= 0 && last < pages;
    __syncthreads();                                       // every thread has read lens[d]
    if (threadIdx.x == 0) {
        if (!grant) atomicOr(&g_fault_paged, ok_seq ? FAULT_NO_PAGES : FAULT_PAGE);
        if (grant && rows && !copy) atomicOr(&g_fault_paged, FAULT_PAGE);
        w.items[i] = {copy ? last : -1, grant && rows ? fresh : -1, rows};
        if (i == 0) w.count[0] = n;
        if (grant) {
            t.lens[d] = len;
            if (rows) t.tables[int64_t(d) * t.stride + full] = fresh;
        }
    }
    if (!grant) return;
    for (int c = threadIdx.x; c < full; c += blockDim.x) {
        const int p = t.tables[int64_t(s) * t.stride + c];
        t.tables[int64_t(d) * t.stride + c] = p;
        if (p >= 0 && p < pages) atomicAdd(t.refs + p, 1);
        else atomicOr(&g_fault_paged, FAULT_PAGE);
    }
}

__global__ void __launch_bounds__(256) kv_free_kernel(qpack_kv_tables_t t, const int *seqs) {
    pdl_launch_dependents();
    pdl_wait();
    const int s = seqs[blockIdx.x];
    if (s < 0) return;
    if (s >= t.seqs) {
        if (threadIdx.x == 0) atomicOr(&g_fault_paged, FAULT_PAGE);
        return;
    }
    for (int c = threadIdx.x; c < t.max_pages; c += blockDim.x) {
        // exchanged, so that a sequence listed twice gives its pages back once
        const int p = atomicExch(t.tables + int64_t(s) * t.stride + c, -1);
        if (p < 0) continue;
        if (p < t.pages) atomicSub(t.refs + p, 1);
        else atomicOr(&g_fault_paged, FAULT_PAGE);
    }
    if (threadIdx.x == 0) t.lens[s] = 0;
}

// One block: counts the live pages, ranks the holes below and the movers above that number, and writes the moves, the
// new numbers and the new reference counts.
__global__ void __launch_bounds__(PLAN_THREADS) kv_compact_plan_kernel(qpack_kv_tables_t t, int page_tokens,
                                                                       int64_t pages, int *refs_out, int *moved, PageWs w) {
    __shared__ int sums[32];
    int tot, nlive = 0;
    pdl_launch_dependents();
    pdl_wait();
    const int64_t chunk = blockDim.x * SCAN;
    int r[SCAN];
    for (int64_t p0 = 0; p0 < pages; p0 += chunk) {
        const int64_t p = p0 + threadIdx.x * SCAN;
        load_refs(t.refs, p, pages, r);
        block_scan(__popc(pages_where(r, p, pages, [](int n, int64_t) { return n > 0; })), sums, &tot);
        nlive += tot;
    }
    int holes = 0, movers = 0;
    for (int64_t p0 = 0; p0 < pages; p0 += chunk) {
        const int64_t p = p0 + threadIdx.x * SCAN;
        if (pages > chunk) load_refs(t.refs, p, pages, r); // else they are there
        const unsigned hole = pages_where(r, p, pages, [&](int n, int64_t q) { return n <= 0 && q < nlive; });
        const unsigned mover = pages_where(r, p, pages, [&](int n, int64_t q) { return n > 0 && q >= nlive; });
        // both ranks in one scan: at most 2^13 of each a chunk
        const int both = block_scan(__popc(hole) | __popc(mover) << 16, sums, &tot);
        int hr = holes + (both & 0xFFFF), mr = movers + (both >> 16);
        holes += tot & 0xFFFF;
        movers += tot >> 16;
#pragma unroll
        for (int i = 0; i < SCAN; ++i) {
            if (p + i >= pages) break;
            w.map[p + i] = int(p + i);
            if (hole >> i & 1) {
                w.items[hr++].dst = int(p + i);            // its count comes from the page that moves here
            } else if (mover >> i & 1) {
                w.items[mr].src = int(p + i);
                w.items[mr++].rows = r[i];                 // the count, until the lists are matched
                refs_out[p + i] = 0;
            } else {
                refs_out[p + i] = p + i < nlive ? r[i] : 0;
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < movers; i += blockDim.x) {
        const CopyItem it = w.items[i];
        w.items[i].rows = page_tokens;
        w.map[it.src] = it.dst;
        refs_out[it.dst] = it.rows;
    }
    if (threadIdx.x == 0) {
        w.count[0] = movers;
        if (moved) *moved = movers;
    }
}

// Copies the items' rows: 6.2 TB/s over a 32-layer cache. A warp takes one head's rows of keys or values of one layer at a
// time, 16 bytes a lane with eight loads in flight, then the rows' scales. `refs`: fork's fresh pages get their count.
// `tables`: compaction's entries get their new numbers.
__global__ void __launch_bounds__(256) kv_copy_kernel(qpack_kv_pool_t pool, PageWs w, const int *src_list,
                                                      const int *dst_list, int64_t n_list, int *refs, qpack_kv_tables_t t,
                                                      int *tables_out) {
    const int lane = threadIdx.x & 31;
    const int64_t warp = int64_t(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int64_t warps = int64_t(gridDim.x) * (blockDim.x >> 5);
    pdl_launch_dependents();
    pdl_wait();
    const int64_t n = src_list ? n_list : w.count[0];
    const int64_t slabs = n * pool.layers * 2 * pool.heads;
    const int es = pool.type == QPACK_KV_I8 ? 1 : 2;
    const bool narrow = slabs < (int64_t(1) << 31);        // 32-bit divisions do (64 children: 0.4 us less of 28)
    for (int64_t j = warp; j < slabs; j += warps) {
        const int64_t pair = narrow ? int64_t(unsigned(j) / unsigned(pool.heads)) : j / pool.heads;
        const int64_t page = pair >> 1;                    // (item, layer)
        const int64_t item = narrow ? int64_t(unsigned(page) / unsigned(pool.layers)) : page / pool.layers;
        const int64_t layer = page - item * pool.layers;
        const int head = int(j - pair * pool.heads);
        const bool is_v = pair & 1;
        CopyItem it;
        if (src_list) it = {src_list[item], dst_list[item], pool.page_tokens};
        else it = w.items[item];
        if (it.src < 0 || it.dst < 0 || it.src >= pool.pages || it.dst >= pool.pages) {
            if (src_list && lane == 0) atomicOr(&g_fault_paged, FAULT_PAGE);
            continue;
        }
        char *base = static_cast<char *>(is_v ? pool.v : pool.k);
        const int64_t in = layer * pool.layer_stride + int64_t(head) * pool.page_tokens * pool.dim;
        const uint4 *a = reinterpret_cast<const uint4 *>(base + (in + it.src * pool.page_stride) * es);
        uint4 *b = reinterpret_cast<uint4 *>(base + (in + it.dst * pool.page_stride) * es);
        const int vec = it.rows * pool.dim * es / 16;
        int x = lane;
        for (; x + 7 * 32 < vec; x += 8 * 32) {
            uint4 r[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) r[u] = __ldcs(a + x + 32 * u);
#pragma unroll
            for (int u = 0; u < 8; ++u) __stcs(b + x + 32 * u, r[u]);
        }
        for (; x < vec; x += 32) __stcs(b + x, __ldcs(a + x));
        if (es == 1) {
            uint16_t *sb = is_v ? pool.v_scales : pool.k_scales;
            const int64_t si = layer * pool.scale_layer_stride + int64_t(head) * pool.page_tokens * (pool.dim / 32);
            // dim / 32 fp16 a row: whole 4-byte words
            const uint32_t *sa = reinterpret_cast<const uint32_t *>(sb + si + it.src * pool.scale_page_stride);
            uint32_t *sd = reinterpret_cast<uint32_t *>(sb + si + it.dst * pool.scale_page_stride);
            for (int y = lane; y < it.rows * (pool.dim / 64); y += 32) sd[y] = sa[y];
        }
    }
    const int64_t tid = int64_t(blockIdx.x) * blockDim.x + threadIdx.x, threads = int64_t(gridDim.x) * blockDim.x;
    if (refs)
        for (int64_t i = tid; i < n; i += threads)
            if (w.items[i].dst >= 0) refs[w.items[i].dst] = 1;
    if (tables_out)
        for (int64_t i = tid; i < int64_t(t.seqs) * t.max_pages; i += threads) {
            const int64_t at = i / t.max_pages * t.stride + i % t.max_pages;
            const int p = t.tables[at];
            if (p >= t.pages) atomicOr(&g_fault_paged, FAULT_PAGE);
            tables_out[at] = p >= 0 && p < t.pages ? w.map[p] : p;
        }
}

cudaError_t run_copy(const qpack_kv_pool_t &p, const PageWs &w, const int *src, const int *dst, int64_t n, int64_t most,
                     int *refs, const qpack_kv_tables_t &t, int *tables_out, cudaStream_t s) {
    const int64_t warps = most * p.layers * 2 * p.heads, cap = int64_t(num_sms()) * 8;
    int64_t grid = (warps + 7) / 8;
    grid = grid < 1 ? 1 : (grid < cap ? grid : cap);
    return launch_dependent(kv_copy_kernel, grid, 256, s, p, w, src, dst, n, refs, t, tables_out);
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs &a, cudaStream_t s) { return rows_kind(a, false, s); }
cudaError_t launch_kv_read(const AppendArgs &a, cudaStream_t s) { return rows_kind(a, true, s); }

int64_t kv_page_workspace(const qpack_kv_pool_t &p) {
    return 16 + int64_t(sizeof(CopyItem)) * copy_cap(p.pages) + 4 * p.pages;
}

cudaError_t launch_kv_reserve(const qpack_kv_pool_t &p, const qpack_kv_tables_t &t, const int32_t *seqs,
                              const int32_t *add, int n, cudaStream_t s) {
    return launch_dependent(kv_reserve_kernel, 1, PLAN_THREADS, s, t, int(p.page_tokens), seqs, add, n, t.pages);
}

cudaError_t launch_kv_fork(const qpack_kv_pool_t &p, const qpack_kv_tables_t &t, const int32_t *src, const int32_t *dst,
                           int n, void *ws, cudaStream_t s) {
    const PageWs w = page_ws(ws, p.pages);
    const cudaError_t e = launch_dependent(kv_fork_kernel, n, 256, s, t, int(p.page_tokens), src, dst, n, t.pages, w);
    if (e != cudaSuccess) return e;
    return run_copy(p, w, nullptr, nullptr, 0, n, t.refs, t, nullptr, s);
}

cudaError_t launch_kv_free(const qpack_kv_tables_t &t, const int32_t *seqs, int n, cudaStream_t s) {
    return launch_dependent(kv_free_kernel, n, 256, s, t, seqs);
}

cudaError_t launch_kv_compact(const qpack_kv_pool_t &p, const qpack_kv_tables_t &t, int32_t *tables_out,
                              int32_t *refs_out, int32_t *moved, void *ws, cudaStream_t s) {
    const PageWs w = page_ws(ws, p.pages);
    const cudaError_t e = launch_dependent(kv_compact_plan_kernel, 1, PLAN_THREADS, s, t, int(p.page_tokens), t.pages,
                                           refs_out, moved, w);
    if (e != cudaSuccess) return e;
    return run_copy(p, w, nullptr, nullptr, 0, t.pages / 2 + 1, nullptr, t, tables_out, s);
}

cudaError_t launch_kv_copy_pages(const qpack_kv_pool_t &p, const int32_t *src, const int32_t *dst, int64_t n,
                                 cudaStream_t s) {
    return run_copy(p, PageWs{}, src, dst, n, n, nullptr, qpack_kv_tables_t{}, nullptr, s);
}

cudaError_t fault_word_paged(int **word) { return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_fault_paged); }

}  // namespace qpack
