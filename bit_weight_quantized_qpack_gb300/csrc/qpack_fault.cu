// qpack_fault.cu — the library's fault word: the translation units' words taken together and cleared by one small kernel, so
// that a fetch is a launch and a copy whatever their number (16 us; a copy there and back for each of six words took 75).
#include <cuda_runtime.h>

#include "qpack_launch.h"

namespace qpack {
namespace {

constexpr int WORDS = 6;
struct Words {
    int *at[WORDS];
};

__device__ int g_fault = 0;

__global__ void collect_kernel(Words w) {
    const int v = threadIdx.x < WORDS ? atomicExch(w.at[threadIdx.x], 0) : 0;
    const int all = __reduce_or_sync(0xffffffffu, v);
    if (threadIdx.x == 0) g_fault = all;
}

}  // namespace

cudaError_t fetch_faults(int32_t *flags) {
    Words w;
    cudaError_t e = fault_word_gemv(&w.at[0]);
    if (e == cudaSuccess) e = fault_word_prefill(&w.at[1]);
    if (e == cudaSuccess) e = fault_word_paged(&w.at[2]);
    if (e == cudaSuccess) e = fault_words_attend(&w.at[3]);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(32);
    // its own status: an earlier error of the caller's is neither reported here nor cleared
    if ((e = cudaLaunchKernelEx(&cfg, collect_kernel, w)) != cudaSuccess) return e;
    return cudaMemcpyFromSymbol(flags, g_fault, sizeof(int));
}

}  // namespace qpack
