// qpack_shared_bf16.cu — attention over shared prefixes of the bfloat16 paged cache (the kernel is in qpack_shared.cuh).
#include "qpack_shared.cuh"

QPACK_SHARED_TYPE(QPACK_KV_BF16)
