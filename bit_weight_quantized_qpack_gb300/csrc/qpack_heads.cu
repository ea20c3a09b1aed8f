// qpack_heads.cu — the root-mean-square norm of query and key heads with the position rotation in the same pass.
//
// The mathematics. A head x of `dim` elements becomes y = x / sqrt(mean(x^2) + eps) * w (or x where it has no weight), and
// of its first `turn` elements the pairs (a, b) of position p become (a c - b s, b c + a s), c and s from row p of the
// table: pairs (i, i + turn / 2), or neighbours (2i, 2i + 1). Every operation is fp32 and rounded by itself, products
// before their sum, as the cache's append has it: without a weight the rotated keys are those that append would store.
//
// What bounds it. Each element is read and written once, and one row of the table is read for all heads of a token: the
// copy rate at length, the launch and one chain position -> table row -> store at a decode step's few tokens.
//
// A head takes dim / 8 lanes, in groups of 8, 16 or 32 lanes. A lane holds both elements of its pairs (lane l of a half
// layout the elements 4l .. 4l + 3 and their partners turn / 2 further), so that the rotation needs no shuffle and a lane
// writes what it has read: in place is fine. Behind the rotated part a lane holds eight elements in a row.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qpack_dev.cuh"
#include "qpack_launch.h"
#include "qpack_paged.cuh"

namespace qpack {
namespace {

__device__ int g_fault_heads = 0;

constexpr int WARPS = 4;        // a block
constexpr int ROWS = 4;         // heads in flight a group of lanes

// Four consecutive elements. Plain loads: the previous grid may have written them, and in place they are written here.
template <int DT> struct Four { uint32_t w[DT == DT_F32 ? 4 : 2]; };
template <int DT> __device__ __forceinline__ void load4(const void *p, int64_t i, Four<DT> &r) {
    if (DT == DT_F32) {
        const uint4 v = *reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + i);
        r.w[0] = v.x, r.w[1] = v.y, r.w[DT == DT_F32 ? 2 : 0] = v.z, r.w[DT == DT_F32 ? 3 : 1] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + i);
        r.w[0] = v.x, r.w[1] = v.y;
    }
}
template <int DT> __device__ __forceinline__ void widen(const Four<DT> &r, float *x) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (DT == DT_F32) x[e] = __uint_as_float(r.w[DT == DT_F32 ? e : 0]);
        else if (DT == DT_F16) x[e] = h2f_bits(uint16_t(e & 1 ? r.w[e / 2] >> 16 : r.w[e / 2] & 0xFFFFu));
        else x[e] = __uint_as_float(e & 1 ? r.w[e / 2] & 0xFFFF0000u : r.w[e / 2] << 16);
    }
}
template <int DT> __device__ __forceinline__ void store4(void *p, int64_t i, const float *x) {
    if (DT == DT_F32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(p) + i) = make_float4(x[0], x[1], x[2], x[3]);
        return;
    }
    uint32_t w[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        if (DT == DT_F16) {
            w[e] = uint32_t(f2h_bits(x[2 * e])) | uint32_t(f2h_bits(x[2 * e + 1])) << 16;
        } else {
            const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t *>(&b);
        }
    }
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p) + i) = make_uint2(w[0], w[1]);
}

// The token's position: -1 where it is skipped (a negative position, an empty sequence) or its sequence is out of range.
__device__ __forceinline__ int position(const HeadsArgs &a, int64_t i, bool report) {
    if (a.pos) return max(a.pos[i], -1);
    if (!a.has_tables) return 0;                           // no rotation: any position will do
    const int64_t seq = a.seqs ? int64_t(a.seqs[i]) : i;
    int len = -1;
    if (seq >= 0 && seq < a.t.seqs) len = a.t.lens[seq];
    if (len < 0 && report) atomicOr(&g_fault_heads, FAULT_PAGE);
    return max(len, 0) - 1;
}

// G lanes a head: dim <= 8 G. NEAR: pairs are neighbours.
template <int XT, int OT, int G, bool NEAR>
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
    const bool holds = l < D / 8;
    const bool turned = a.rope && 4 * l < half;            // lane of the rotated part
    // the lane's two runs of four elements
    const int at0 = NEAR || !turned ? 8 * l : 4 * l, at1 = NEAR || !turned ? 8 * l + 4 : half + 4 * l;
    Four<XT> raw[ROWS][2];
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
        const int head = head0 + u * PER;
        raw[u][0] = raw[u][1] = Four<XT>{};
        if (holds && head < x.heads) {
            load4<XT>(x.x, tok * x.ldx + int64_t(head) * D + at0, raw[u][0]);
            load4<XT>(x.x, tok * x.ldx + int64_t(head) * D + at1, raw[u][1]);
        }
    }
    const int pos = position(a, tok, lane == 0 && group == 0);
    if (pos < 0) return;
    float c[4] = {1, 1, 1, 1}, s[4] = {0, 0, 0, 0};
    const bool in_table = pos < a.rope_rows;
    if (turned && in_table) {
        const float *row = a.rope + int64_t(pos) * a.turn + 4 * l;
        const float4 cc = *reinterpret_cast<const float4 *>(row), ss = *reinterpret_cast<const float4 *>(row + half);
        c[0] = cc.x, c[1] = cc.y, c[2] = cc.z, c[3] = cc.w;
        s[0] = ss.x, s[1] = ss.y, s[2] = ss.z, s[3] = ss.w;
    }
    if (a.rope && !in_table && lane == 0 && group == 0) atomicOr(&g_fault_heads, FAULT_PAGE);
    float w[8] = {};
    if (x.weight && holds) {
        const float4 lo = *reinterpret_cast<const float4 *>(x.weight + at0), hi = *reinterpret_cast<const float4 *>(x.weight + at1);
        w[0] = lo.x, w[1] = lo.y, w[2] = lo.z, w[3] = lo.w, w[4] = hi.x, w[5] = hi.y, w[6] = hi.z, w[7] = hi.w;
    }
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
        float y[8];
        widen<XT>(raw[u][0], y);
        widen<XT>(raw[u][1], y + 4);
        if (x.weight) {                                    // the same for the whole warp
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fmaf(y[e], y[e], sum);
#pragma unroll
            for (int o = G / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const float r = __frsqrt_rn(__fdiv_rn(sum, float(D)) + a.eps);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = y[e] * r * w[e];
        }
        if (turned && in_table) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float &p = y[NEAR ? 2 * e : e], &q = y[NEAR ? 2 * e + 1 : 4 + e];
                const float m = p;
                p = __fsub_rn(__fmul_rn(m, c[e]), __fmul_rn(q, s[e]));
                q = __fadd_rn(__fmul_rn(q, c[e]), __fmul_rn(m, s[e]));
            }
        }
        const int head = head0 + u * PER;
        if (holds && head < x.heads) {
            store4<OT>(x.out, tok * x.ldo + int64_t(head) * D + at0, y);
            store4<OT>(x.out, tok * x.ldo + int64_t(head) * D + at1, y + 4);
        }
    }
}

template <int XT, int OT, int G, bool NEAR> cudaError_t run(const HeadsArgs &a, cudaStream_t s) {
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
        const cudaError_t e = cudaLaunchKernelEx(&cfg, heads_kernel<XT, OT, G, NEAR>, a, i, items, q_groups, groups);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}
template <int XT, int OT, int G> cudaError_t run_pairs(const HeadsArgs &a, cudaStream_t s) {
    return a.near_pairs ? run<XT, OT, G, true>(a, s) : run<XT, OT, G, false>(a, s);
}
template <int XT, int OT> cudaError_t run_dim(const HeadsArgs &a, cudaStream_t s) {
    return a.dim <= 64 ? run_pairs<XT, OT, 8>(a, s) : a.dim <= 128 ? run_pairs<XT, OT, 16>(a, s) : run_pairs<XT, OT, 32>(a, s);
}
template <int XT> cudaError_t run_out(const HeadsArgs &a, cudaStream_t s) {
    return a.odt == DT_F32 ? run_dim<XT, DT_F32>(a, s) : a.odt == DT_F16 ? run_dim<XT, DT_F16>(a, s) : run_dim<XT, DT_BF16>(a, s);
}

}  // namespace

cudaError_t launch_heads(const HeadsArgs &a, cudaStream_t s) {
    return a.dt == DT_F32 ? run_out<DT_F32>(a, s) : a.dt == DT_F16 ? run_out<DT_F16>(a, s) : run_out<DT_BF16>(a, s);
}

cudaError_t fault_word_heads(int **word) {
    return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_fault_heads);
}

}  // namespace qpack
