// qpack_attend_bf16.cu — attention over the bfloat16 paged cache (the kernel is in qpack_attend.cuh).
#include "qpack_attend.cuh"

QPACK_ATTEND_TYPE(QPACK_KV_BF16)
