// qpack_paged.cuh — what the paged KV cache's kernels share.
#pragma once

#include "qpack.h"
#include "qpack_dev.cuh"

namespace qpack {

// Bits of the fault word: page numbers, positions, lengths or sequence numbers out of range; requests refused.
enum : int { FAULT_PAGE = QPACK_FAULT_PAGE, FAULT_NO_PAGES = QPACK_FAULT_NO_PAGES };

// 8-bit cache elements: bytes of w (codes + 128, that is the code word xor 0x80808080) chosen by `sel` (second and
// fourth selector 4), times a pair of fp16 scales: the byte under the exponent of 1024 is 1024 + u, less 1152 the code
// (exact), and the product rounds once, so the pair is fp16_rn(scale * code).
__device__ __forceinline__ uint32_t dequant2(uint32_t w, uint32_t sel, uint32_t scale) {
    const uint32_t u = __byte_perm(w, 0x64646464u, sel);
    const __half2 off = __half2half2(__ushort_as_half(0x6480));
    const __half2 c = __hsub2(*reinterpret_cast<const __half2 *>(&u), off);
    const __half2 v = __hmul2(c, *reinterpret_cast<const __half2 *>(&scale));
    return *reinterpret_cast<const uint32_t *>(&v);
}

}  // namespace qpack
