// qpack_attend.cu — attention of one new token over the paged KV cache: dispatch on the cache's type. The kernel is in
// qpack_attend.cuh, one translation unit a type.
#include <cuda_runtime.h>

#include "qpack_attend.cuh"

namespace qpack {

namespace attend {
template <> cudaError_t launch<QPACK_KV_I8>(const AttendArgs &, cudaStream_t);
template <> cudaError_t launch<QPACK_KV_F16>(const AttendArgs &, cudaStream_t);
template <> cudaError_t launch<QPACK_KV_BF16>(const AttendArgs &, cudaStream_t);
template <> int64_t workspace<QPACK_KV_I8>(const qpack_kv_pool_t &, int, int);
template <> int64_t workspace<QPACK_KV_F16>(const qpack_kv_pool_t &, int, int);
template <> int64_t workspace<QPACK_KV_BF16>(const qpack_kv_pool_t &, int, int);
template <> bool fits<QPACK_KV_I8>(const qpack_kv_pool_t &, const qpack_kv_tables_t &, int);
template <> bool fits<QPACK_KV_F16>(const qpack_kv_pool_t &, const qpack_kv_tables_t &, int);
template <> bool fits<QPACK_KV_BF16>(const qpack_kv_pool_t &, const qpack_kv_tables_t &, int);
template <> cudaError_t fault_word<QPACK_KV_I8>(int **);
template <> cudaError_t fault_word<QPACK_KV_F16>(int **);
template <> cudaError_t fault_word<QPACK_KV_BF16>(int **);
}  // namespace attend

int64_t kv_attend_workspace(const qpack_kv_pool_t &pool, int q_heads) {
    const int grid = num_sms();
    int64_t parts;
    if (pool.type == QPACK_KV_I8) parts = attend::workspace<QPACK_KV_I8>(pool, q_heads, grid);
    else if (pool.type == QPACK_KV_F16) parts = attend::workspace<QPACK_KV_F16>(pool, q_heads, grid);
    else parts = attend::workspace<QPACK_KV_BF16>(pool, q_heads, grid);
    return int64_t(attend::MAX_COUNTERS) * 4 + parts;
}

bool kv_attend_fits(const qpack_kv_pool_t &pool, const qpack_kv_tables_t &t, int q_heads) {
    if (pool.type == QPACK_KV_I8) return attend::fits<QPACK_KV_I8>(pool, t, q_heads);
    if (pool.type == QPACK_KV_F16) return attend::fits<QPACK_KV_F16>(pool, t, q_heads);
    return attend::fits<QPACK_KV_BF16>(pool, t, q_heads);
}

cudaError_t launch_kv_attend(const AttendArgs &a, cudaStream_t s) {
    if (a.pool.type == QPACK_KV_I8) return attend::launch<QPACK_KV_I8>(a, s);
    if (a.pool.type == QPACK_KV_F16) return attend::launch<QPACK_KV_F16>(a, s);
    return attend::launch<QPACK_KV_BF16>(a, s);
}

cudaError_t fault_words_attend(int **words) {
    cudaError_t e = attend::fault_word<QPACK_KV_I8>(words);
    if (e == cudaSuccess) e = attend::fault_word<QPACK_KV_F16>(words + 1);
    if (e == cudaSuccess) e = attend::fault_word<QPACK_KV_BF16>(words + 2);
    return e;
}

}  // namespace qpack
