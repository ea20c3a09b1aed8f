// qpack_shared_i8.cu — attention over shared prefixes of the 8-bit paged cache (the kernel is in qpack_shared.cuh).
#include "qpack_shared.cuh"

QPACK_SHARED_TYPE(QPACK_KV_I8)
