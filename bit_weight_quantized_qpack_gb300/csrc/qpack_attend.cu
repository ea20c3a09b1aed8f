// qpack_attend.cu — attention of one new token a sequence over the paged KV cache.
//
// One pass over the cache with a running maximum and sum (base 2): for tokens t, x_t = q~ . k'_t, m' = max(m, x_t),
// l' = l 2^(m - m') + 2^(x_t - m'), o' = o 2^(m - m') + 2^(x_t - m') v'_t; out = o / l. One block takes a sequence's
// key/value head and up to eight of its query heads, a warp a query head.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qpack_dev.cuh"
#include "qpack_launch.h"

namespace qpack {
namespace {

__device__ int g_fault_attend = 0;

constexpr int HEADS = 8, TILE = 32;

__device__ __forceinline__ float load1(const void *p, int dt, int64_t i) {
    if (dt == DT_F32) return static_cast<const float *>(p)[i];
    if (dt == DT_F16) return h2f_bits(static_cast<const uint16_t *>(p)[i]);
    return __uint_as_float(uint32_t(static_cast<const uint16_t *>(p)[i]) << 16);
}

__device__ __forceinline__ void store1(void *p, int dt, int64_t i, float x) {
    if (dt == DT_F32) static_cast<float *>(p)[i] = x;
    else if (dt == DT_F16) static_cast<uint16_t *>(p)[i] = f2h_bits(x);
    else static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(x);
}

template <int KT, int D>
__global__ void __launch_bounds__(HEADS * 32) attend_kernel(AttendArgs a) {
    extern __shared__ float smem[];
    float *ks = smem, *vs = ks + TILE * (D + 1), *qs = vs + TILE * (D + 1);
    const int H = a.pool.heads, G = a.q_heads / H, chunks = (G + HEADS - 1) / HEADS;
    const int c = blockIdx.x % chunks, h = blockIdx.x / chunks % H, b = blockIdx.x / chunks / H;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, g = c * HEADS + w, qh = h * G + g;
    const int T = a.pool.page_tokens;
    int64_t seq = a.seqs ? a.seqs[b] : b;
    int64_t len = 0;
    if (seq >= 0 && seq < a.t.seqs) len = a.t.lens[seq];
    else if (threadIdx.x == 0) atomicOr(&g_fault_attend, FAULT_PAGE);
    const int64_t top = int64_t(a.t.max_pages) * T;
    if (len < 0 || len > top) {
        if (threadIdx.x == 0) atomicOr(&g_fault_attend, FAULT_PAGE);
        len = len < 0 ? 0 : top;
    }
    const int64_t lo = a.window > 0 && len > a.window ? len - a.window : 0;
    if (g < G) {
        const int64_t p = len - 1;
        const bool turn = a.rope && p >= 0;
        if (turn && p >= a.rope_rows && lane == 0) atomicOr(&g_fault_attend, FAULT_PAGE);
        for (int i = lane; i < D; i += 32) {
            float x = load1(a.q, a.qdt, b * a.ldq + int64_t(qh) * D + i);
            if (turn && p < a.rope_rows) {
                const float y = load1(a.q, a.qdt, b * a.ldq + int64_t(qh) * D + (i ^ (D / 2)));
                const float co = a.rope[p * D + i % (D / 2)], si = a.rope[p * D + D / 2 + i % (D / 2)];
                x = i < D / 2 ? __fsub_rn(__fmul_rn(x, co), __fmul_rn(y, si))
                              : __fadd_rn(__fmul_rn(x, co), __fmul_rn(y, si));
            }
            qs[w * D + i] = x;
        }
    }
    float m = -INFINITY, l = 0.0f, o[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = 0.0f;
    for (int64_t t0 = lo; t0 < len; t0 += TILE) {
        const int n = len - t0 < TILE ? int(len - t0) : TILE;
        __syncthreads();
        for (int i = threadIdx.x; i < n * D; i += HEADS * 32) {
            const int64_t t = t0 + i / D;
            const int e = i % D;
            const int page = a.t.tables[seq * a.t.stride + t / T];
            float kx = 0.0f, vx = 0.0f;
            if (page >= 0 && page < a.pool.pages) {
                const int64_t in = (int64_t(h) * T + t % T) * D + e;
                const int64_t at = a.layer * a.pool.layer_stride + page * a.pool.page_stride + in;
                if (KT == QPACK_KV_I8) {
                    const int64_t sat = a.layer * a.pool.scale_layer_stride + page * a.pool.scale_page_stride + in / 32;
                    kx = h2f_bits(f2h_bits(float(static_cast<const int8_t *>(a.pool.k)[at]) * h2f_bits(a.pool.k_scales[sat])));
                    vx = h2f_bits(f2h_bits(float(static_cast<const int8_t *>(a.pool.v)[at]) * h2f_bits(a.pool.v_scales[sat])));
                } else {
                    kx = load1(a.pool.k, KT == QPACK_KV_F16 ? DT_F16 : DT_BF16, at);
                    vx = load1(a.pool.v, KT == QPACK_KV_F16 ? DT_F16 : DT_BF16, at);
                }
            } else {
                atomicOr(&g_fault_attend, FAULT_PAGE);
            }
            ks[(i / D) * (D + 1) + e] = kx;
            vs[(i / D) * (D + 1) + e] = vx;
        }
        __syncthreads();
        if (g >= G) continue;
        float x = -INFINITY;
        if (lane < n) {
            x = 0.0f;
            for (int e = 0; e < D; ++e) x = fmaf(qs[w * D + e], ks[lane * (D + 1) + e], x);
            x *= a.scale * 1.4426950408889634f;
        }
        float mn = x;
#pragma unroll
        for (int s = 16; s; s >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, s));
        mn = fmaxf(m, mn);
        const float base = mn == -INFINITY ? 0.0f : mn;
        const float p = lane < n ? exp2f(x - base) : 0.0f, f = exp2f(m - base);
        float sum = p;
#pragma unroll
        for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
        l = l * f + sum;
        m = mn;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) o[i] *= f;
        for (int t = 0; t < n; ++t) {
            const float pt = __shfl_sync(0xffffffffu, p, t);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) o[i] = fmaf(pt, vs[t * (D + 1) + 32 * i + lane], o[i]);
        }
    }
    if (g >= G) return;
    const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) store1(a.out, a.odt, b * a.ldo + int64_t(qh) * D + 32 * i + lane, o[i] * inv);
    if (a.lse && lane == 0)
        a.lse[int64_t(b) * a.q_heads + qh] = l > 0.0f || l != l ? m * 0.6931471805599453f + logf(l) : -INFINITY;
}

template <int KT, int D> cudaError_t run(const AttendArgs &a, cudaStream_t s) {
    const int G = a.q_heads / a.pool.heads, chunks = (G + HEADS - 1) / HEADS;
    const int smem = (2 * TILE * (D + 1) + HEADS * D) * 4;
    const cudaError_t e = cudaFuncSetAttribute(attend_kernel<KT, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    attend_kernel<KT, D><<<a.B * a.pool.heads * chunks, HEADS * 32, smem, s>>>(a);
    return cudaGetLastError();
}

template <int KT> cudaError_t run_dim(const AttendArgs &a, cudaStream_t s) {
    if (a.pool.dim == 64) return run<KT, 64>(a, s);
    if (a.pool.dim == 128) return run<KT, 128>(a, s);
    return run<KT, 256>(a, s);
}

}  // namespace

int64_t kv_attend_workspace(const qpack_kv_pool_t &, int, int) { return 16; }

cudaError_t launch_kv_attend(const AttendArgs &a, cudaStream_t s) {
    if (a.pool.type == QPACK_KV_I8) return run_dim<QPACK_KV_I8>(a, s);
    if (a.pool.type == QPACK_KV_F16) return run_dim<QPACK_KV_F16>(a, s);
    return run_dim<QPACK_KV_BF16>(a, s);
}

cudaError_t fetch_fault_attend(int32_t *flags) {
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_fault_attend, sizeof(int));
    if (e != cudaSuccess) return e;
    *flags |= v;
    const int zero = 0;
    return cudaMemcpyToSymbol(g_fault_attend, &zero, sizeof(int));
}

}  // namespace qpack
