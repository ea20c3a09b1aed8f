// qpack_attend_f16.cu — attention over the fp16 paged cache (the kernel is in qpack_attend.cuh).
#include "qpack_attend.cuh"

QPACK_ATTEND_TYPE(QPACK_KV_F16)
