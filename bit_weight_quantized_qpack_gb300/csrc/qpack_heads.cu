// qpack_heads.cu — the root-mean-square norm of query and key heads with the position rotation in the same pass.
//
// The mathematics. A head x of `dim` elements becomes y = x / sqrt(mean(x^2) + eps) * w (or x where it has no weight;
// a head whose squares leave fp32's range is scaled by a power of two for its mean), and of its first `turn` elements
// the pairs (a, b) of position p become (a c - b s, b c + a s), c and s from row p of the table: pairs (i, i + turn /
// 2), or neighbours (2i, 2i + 1). Every operation is fp32 and rounded by itself, products before their sum, as the
// cache's append has it: without a weight the rotated keys are those that append would store.
//
// What bounds it. Each element is read and written once, and one row of the table is read for all heads of a token:
// the copy rate at length (8191 tokens of 40 heads of 128: bfloat16 38 us, 67% of it, fp32 53.5 us, 94%; the chain
// position -> table row -> store in the warps that fit an SM), the launch and that chain at a decode step's few
// tokens (2.1 us in a graph, 10.5 by a call from Python, whose host time that is).
//
// A lane holds two runs of RUN elements, 16 bytes each where the type and the sizes allow it: lane l of a half layout
// the elements RUN l and on and their partners turn / 2 further, so that the rotation needs no shuffle and a lane
// writes what it has read (in place is fine); behind the rotated part, and of neighbouring pairs, 2 RUN elements in a
// row. A head takes dim / (2 RUN) lanes of a group of 4 to 32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cfloat>

#include "qpack_dev.cuh"
#include "qpack_launch.h"
#include "qpack_paged.cuh"

namespace qpack {
namespace {

__device__ int g_fault_heads = 0;

constexpr int WARPS = 4;        // a block
// Heads in flight a group of lanes. us for 16 fp32 tokens / 8191 bfloat16 tokens of 40 heads of 128 (the latter in
// runs of eight): 1 1.8 / 44.4, 2 2.1 / 38.6, 4 2.8 / 38.2; in runs of four 2 2.2 / 40.5, 4 2.8 / 37.6, 6 3.5 / 43.0.
// A grid that stays and asks for the next position a pass ahead took 41 us.
constexpr int ROWS = 2;

// RUN = 4 or 8 consecutive elements, aligned to 8 or 16 bytes. Plain loads: the previous grid may have written them,
// and in place they are written here.
template <int DT, int RUN> struct Raw { uint32_t w[DT == DT_F32 ? RUN : RUN / 2]; };
template <int DT, int RUN> __device__ __forceinline__ void load_run(const void *p, int64_t i, Raw<DT, RUN> &r) {
    constexpr int WORDS = DT == DT_F32 ? RUN : RUN / 2;
    const uint32_t *q = DT == DT_F32 ? static_cast<const uint32_t *>(p) + i
                                     : reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(p) + i);
    if constexpr (WORDS == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(q);
        r.w[0] = v.x, r.w[1] = v.y;
    } else {
#pragma unroll
        for (int e = 0; e < WORDS; e += 4) {
            const uint4 v = *reinterpret_cast<const uint4 *>(q + e);
            r.w[e] = v.x, r.w[e + 1] = v.y, r.w[e + 2] = v.z, r.w[e + 3] = v.w;
        }
    }
}
template <int DT, int RUN> __device__ __forceinline__ void widen(const Raw<DT, RUN> &r, float *x) {
#pragma unroll
    for (int e = 0; e < RUN; ++e) {
        if (DT == DT_F32) x[e] = __uint_as_float(r.w[DT == DT_F32 ? e : 0]);
        else if (DT == DT_F16) x[e] = h2f_bits(uint16_t(e & 1 ? r.w[e / 2] >> 16 : r.w[e / 2] & 0xFFFFu));
        else x[e] = __uint_as_float(e & 1 ? r.w[e / 2] & 0xFFFF0000u : r.w[e / 2] << 16);
    }
}
template <int DT, int RUN> __device__ __forceinline__ void store_run(void *p, int64_t i, const float *x) {
    if (DT == DT_F32) {
#pragma unroll
        for (int e = 0; e < RUN; e += 4)
            *reinterpret_cast<float4 *>(static_cast<float *>(p) + i + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
        return;
    }
    uint32_t w[RUN / 2];
#pragma unroll
    for (int e = 0; e < RUN / 2; ++e) {
        if (DT == DT_F16) {
            w[e] = uint32_t(f2h_bits(x[2 * e])) | uint32_t(f2h_bits(x[2 * e + 1])) << 16;
        } else {
            const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t *>(&b);
        }
    }
    uint16_t *o = static_cast<uint16_t *>(p) + i;
    if constexpr (RUN == 4) *reinterpret_cast<uint2 *>(o) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint4 *>(o) = make_uint4(w[0], w[1], w[RUN / 2 - 2], w[RUN / 2 - 1]);
}

// The token's position: -1 where it is skipped (a negative position, an empty sequence) or its sequence is out of
// range.
__device__ __forceinline__ int position(const HeadsArgs &a, int64_t i, bool report) {
    if (a.pos) return max(a.pos[i], -1);
    if (!a.has_tables) return 0;                           // no rotation: any position will do
    const int64_t seq = a.seqs ? int64_t(a.seqs[i]) : i;
    int len = -1;
    if (seq >= 0 && seq < a.t.seqs) len = a.t.lens[seq];
    if (len < 0 && report) atomicOr(&g_fault_heads, FAULT_PAGE);
    return max(len, 0) - 1;
}

// The sum of a head's squares.
template <int RUN, int G> __device__ __forceinline__ float squares(const float (&y)[2 * RUN]) {
    float sum = 0.0f;
#pragma unroll
    for (int e = 0; e < 2 * RUN; ++e) sum = fmaf(y[e], y[e], sum);
#pragma unroll
    for (int o = G / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
}

// G lanes a head: dim <= 2 RUN G. NEAR: pairs are neighbours.
template <int XT, int OT, int RUN, int G, bool NEAR>
__global__ void __launch_bounds__(WARPS * 32) heads_kernel(HeadsArgs a, int64_t first, unsigned items, unsigned q_groups,
                                                           unsigned groups) {
    constexpr int PER = 32 / G;                            // heads a pass of the warp
    const int lane = threadIdx.x & 31, l = lane % G;
    pdl_launch_dependents();
    const unsigned item = blockIdx.x * WARPS + (threadIdx.x >> 5), tok_in = item / groups;
    const unsigned group = item - tok_in * groups;
    const int side = group >= q_groups;                    // 0: queries, 1: keys
    const int head0 = int(side ? group - q_groups : group) * (ROWS * PER) + lane / G;
    pdl_wait();
    if (item >= items) return;                             // whole warps
    const int64_t tok = first + tok_in;
    const HeadsSide &x = a.side[side];
    const int D = a.dim, half = a.turn / 2;
    const bool holds = l < D / (2 * RUN);
    const bool turned = a.rope && RUN * l < half;          // lane of the rotated part
    // the lane's two runs
    const int at0 = NEAR || !turned ? 2 * RUN * l : RUN * l, at1 = NEAR || !turned ? 2 * RUN * l + RUN : half + RUN * l;
    Raw<XT, RUN> raw[ROWS][2];
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
        const int head = head0 + u * PER;
        raw[u][0] = raw[u][1] = Raw<XT, RUN>{};
        if (holds && head < x.heads) {
            load_run<XT, RUN>(x.x, tok * x.ldx + int64_t(head) * D + at0, raw[u][0]);
            load_run<XT, RUN>(x.x, tok * x.ldx + int64_t(head) * D + at1, raw[u][1]);
        }
    }
    const int pos = position(a, tok, lane == 0 && group == 0);
    if (pos < 0) return;
    float c[RUN], s[RUN];
    const bool in_table = pos < a.rope_rows;
    if (turned && in_table) {
        const float *row = a.rope + int64_t(pos) * a.turn + RUN * l;
#pragma unroll
        for (int e = 0; e < RUN; e += 4) {
            const float4 cc = *reinterpret_cast<const float4 *>(row + e), ss = *reinterpret_cast<const float4 *>(row + half + e);
            c[e] = cc.x, c[e + 1] = cc.y, c[e + 2] = cc.z, c[e + 3] = cc.w;
            s[e] = ss.x, s[e + 1] = ss.y, s[e + 2] = ss.z, s[e + 3] = ss.w;
        }
    }
    if (a.rope && !in_table && lane == 0 && group == 0) atomicOr(&g_fault_heads, FAULT_PAGE);
    float w[2 * RUN] = {};
    if (x.weight && holds)
#pragma unroll
        for (int e = 0; e < RUN; e += 4) {
            const float4 lo = *reinterpret_cast<const float4 *>(x.weight + at0 + e);
            const float4 hi = *reinterpret_cast<const float4 *>(x.weight + at1 + e);
            w[e] = lo.x, w[e + 1] = lo.y, w[e + 2] = lo.z, w[e + 3] = lo.w;
            w[RUN + e] = hi.x, w[RUN + e + 1] = hi.y, w[RUN + e + 2] = hi.z, w[RUN + e + 3] = hi.w;
        }
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
        float y[2 * RUN];
        widen<XT, RUN>(raw[u][0], y);
        widen<XT, RUN>(raw[u][1], y + RUN);
        if (x.weight) {                                    // the same for the whole warp
            float mean = __fdiv_rn(squares<RUN, G>(y), float(D)) + a.eps;
            const bool low = mean < 0x1p-100f;
            const bool rare = low || !(mean <= FLT_MAX);
            if (__any_sync(0xffffffffu, rare)) {
                // Squares that pass fp32, or vanish in it beside an eps that is as small: the head by a power of two
                // that brings its largest element to 1, eps by the square of it. (With an eps, 2^-149 or more, 2^74
                // is enough: what is small then is small beside eps.) A head without a largest element, or with an
                // infinite or NaN one, stays.
                float big = 0.0f;
#pragma unroll
                for (int e = 0; e < 2 * RUN; ++e) big = fmaxf(big, fabsf(y[e]));
#pragma unroll
                for (int o = G / 2; o; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
                const int ex = __float_as_int(big) >> 23;
                const int up = min(max(254 - ex, 1), low && a.eps > 0.0f ? 127 + 74 : 254);
                const float g = !rare || big == 0.0f || ex == 255 ? 1.0f : __int_as_float(up << 23);
#pragma unroll
                for (int e = 0; e < 2 * RUN; ++e) y[e] *= g;
                mean = __fdiv_rn(squares<RUN, G>(y), float(D)) + a.eps * g * g;
            }
            const float r = __frsqrt_rn(mean);
#pragma unroll
            for (int e = 0; e < 2 * RUN; ++e) y[e] = y[e] * r * w[e];
        }
        if (turned && in_table) {
#pragma unroll
            for (int e = 0; e < RUN; ++e) {
                float &p = y[NEAR ? 2 * e : e], &q = y[NEAR ? 2 * e + 1 : RUN + e];
                const float m = p;
                p = __fsub_rn(__fmul_rn(m, c[e]), __fmul_rn(q, s[e]));
                q = __fadd_rn(__fmul_rn(q, c[e]), __fmul_rn(m, s[e]));
            }
        }
        const int head = head0 + u * PER;
        if (holds && head < x.heads) {
            store_run<OT, RUN>(x.out, tok * x.ldo + int64_t(head) * D + at0, y);
            store_run<OT, RUN>(x.out, tok * x.ldo + int64_t(head) * D + at1, y + RUN);
        }
    }
}

template <int XT, int OT, int RUN, int G, bool NEAR> cudaError_t run(const HeadsArgs &a, cudaStream_t s) {
    constexpr int per = ROWS * (32 / G);                   // a warp's heads
    const unsigned q_groups = (a.side[0].heads + per - 1) / per, groups = q_groups + (a.side[1].heads + per - 1) / per;
    const int64_t most = (int64_t(1) << 30) / groups;      // tokens a launch: item numbers stay below 2^31
    for (int64_t i = 0; i < a.n; i += most) {
        const unsigned items = unsigned((a.n - i < most ? a.n - i : most) * groups);
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((items + WARPS - 1) / WARPS);
        cfg.blockDim = dim3(WARPS * 32);
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, heads_kernel<XT, OT, RUN, G, NEAR>, a, i, items, q_groups, groups);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}
template <int XT, int OT, int RUN, int G> cudaError_t run_pairs(const HeadsArgs &a, cudaStream_t s) {
    return a.near_pairs ? run<XT, OT, RUN, G, true>(a, s) : run<XT, OT, RUN, G, false>(a, s);
}
template <int XT, int OT> cudaError_t run_dim(const HeadsArgs &a, cudaStream_t s) {
    // runs of eight where they are 16 bytes on the way in, and both parts of a head are made of pairs of runs
    if constexpr (XT != DT_F32)
        if (a.dim % 16 == 0 && a.turn % 16 == 0)
            return a.dim <= 64    ? run_pairs<XT, OT, 8, 4>(a, s)
                   : a.dim <= 128 ? run_pairs<XT, OT, 8, 8>(a, s)
                                  : run_pairs<XT, OT, 8, 16>(a, s);
    return a.dim <= 64    ? run_pairs<XT, OT, 4, 8>(a, s)
           : a.dim <= 128 ? run_pairs<XT, OT, 4, 16>(a, s)
                          : run_pairs<XT, OT, 4, 32>(a, s);
}
template <int XT> cudaError_t run_out(const HeadsArgs &a, cudaStream_t s) {
    return a.odt == DT_F32   ? run_dim<XT, DT_F32>(a, s)
           : a.odt == DT_F16 ? run_dim<XT, DT_F16>(a, s)
                             : run_dim<XT, DT_BF16>(a, s);
}

}  // namespace

cudaError_t launch_heads(const HeadsArgs &a, cudaStream_t s) {
    return a.dt == DT_F32 ? run_out<DT_F32>(a, s) : a.dt == DT_F16 ? run_out<DT_F16>(a, s) : run_out<DT_BF16>(a, s);
}

cudaError_t fault_word_heads(int **word) {
    return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_fault_heads);
}

}  // namespace qpack
