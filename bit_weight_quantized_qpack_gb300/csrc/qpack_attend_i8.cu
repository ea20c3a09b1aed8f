// qpack_attend_i8.cu — attention over the 8-bit paged cache (the kernel is in qpack_attend.cuh).
#include "qpack_attend.cuh"

QPACK_ATTEND_TYPE(QPACK_KV_I8)
