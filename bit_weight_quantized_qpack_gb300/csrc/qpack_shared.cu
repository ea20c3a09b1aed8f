// qpack_shared.cu — attention where groups of rows share a prefix: dispatch on the cache's type and the workspace. The
// kernels are in qpack_shared.cuh, one translation unit a type.
#include <cuda_runtime.h>

#include "qpack_shared.cuh"

namespace qpack {

namespace shared {
template <> cudaError_t launch<QPACK_KV_I8>(const Params &, cudaStream_t);
template <> cudaError_t launch<QPACK_KV_F16>(const Params &, cudaStream_t);
template <> cudaError_t launch<QPACK_KV_BF16>(const Params &, cudaStream_t);
template <> cudaError_t fault_word<QPACK_KV_I8>(int **);
template <> cudaError_t fault_word<QPACK_KV_F16>(int **);
template <> cudaError_t fault_word<QPACK_KV_BF16>(int **);

namespace {

// The parts of the workspace behind the attention's own; bytes of all of it.
int64_t lay_out(const qpack_kv_pool_t &pool, int64_t B, int q_heads, unsigned char *ws, Work &w) {
    const int64_t n = B * q_heads, slots = int64_t(num_sms()) * 2 * (2 * ROWS);
    int64_t at = round_up(kv_attend_workspace(pool, q_heads), 16);
    auto part = [&](int64_t bytes) {
        unsigned char *p = ws ? ws + at : nullptr;
        at += round_up(bytes, 16);
        return p;
    };
    w.plan = reinterpret_cast<Plan *>(part(sizeof(Plan)));
    w.own_out = reinterpret_cast<float *>(part(n * pool.dim * 4));
    w.own_lse = reinterpret_cast<float *>(part(n * 4));
    w.direct = reinterpret_cast<float *>(part(n * pool.dim * 4));
    w.direct_ml = reinterpret_cast<float2 *>(part(n * 8));
    w.piece = reinterpret_cast<float *>(part(slots * pool.dim * 4));
    w.piece_ml = reinterpret_cast<float2 *>(part(slots * 8));
    return at;
}

}  // namespace
}  // namespace shared

int64_t kv_shared_workspace(const qpack_kv_pool_t &pool, int64_t B, int q_heads) {
    shared::Work w;
    return shared::lay_out(pool, B, q_heads, nullptr, w);
}

cudaError_t launch_kv_attend_shared(const SharedArgs &a, cudaStream_t s) {
    shared::Params p = {};
    p.a = a;
    p.G = a.q_heads / a.pool.heads;
    // Queries of the products' own type that are not rotated are one term as they stand (a power of two that they are
    // scaled by changes no bit of an fp16 query that is not subnormal after it; see the kernel).
    const bool bf = a.pool.type == QPACK_KV_BF16;
    p.a.q_terms = !a.rope && a.qdt == (bf ? QPACK_BF16 : QPACK_F16) ? 1 : 2;
    shared::lay_out(a.pool, a.B, a.q_heads, static_cast<unsigned char *>(a.ws), p.w);
    // tokens up to the end of a last tile and the units of a call are counted in 31 bits
    const int64_t tokens = int64_t(a.t.max_pages) * a.pool.page_tokens, tiles = (tokens + 63) / 64;
    const int64_t items = (int64_t(a.B) * p.G / shared::ROWS + 1 + a.groups) * a.pool.heads;
    if (tokens > 0x7FFFFF00 || items * tiles >= (int64_t(1) << 30)) return cudaErrorNotSupported;
    if (!kv_attend_fits(a.pool, a.t, a.q_heads)) return cudaErrorNotSupported;      // before anything is launched
    if (a.pool.type == QPACK_KV_I8) return shared::launch<QPACK_KV_I8>(p, s);
    if (a.pool.type == QPACK_KV_F16) return shared::launch<QPACK_KV_F16>(p, s);
    return shared::launch<QPACK_KV_BF16>(p, s);
}

cudaError_t fault_words_shared(int **words) {
    cudaError_t e = shared::fault_word<QPACK_KV_I8>(words);
    if (e == cudaSuccess) e = shared::fault_word<QPACK_KV_F16>(words + 1);
    if (e == cudaSuccess) e = shared::fault_word<QPACK_KV_BF16>(words + 2);
    return e;
}

}  // namespace qpack
