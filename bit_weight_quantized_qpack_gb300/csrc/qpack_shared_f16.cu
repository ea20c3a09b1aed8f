// qpack_shared_f16.cu — attention over shared prefixes of the fp16 paged cache (the kernel is in qpack_shared.cuh).
#include "qpack_shared.cuh"

QPACK_SHARED_TYPE(QPACK_KV_F16)
