"""Host-side checks of the paged KV cache at the limits of its arguments."""
import os


def test_no_read_only_loads_in_dependent_kernels():
    """The decode product and the paged cache's kernels are launched while the grid before them runs and wait for it
    themselves. What it writes (activations, lengths, tables, queries, new rows) is not read-only during their life, so none
    of them uses read-only loads."""
    import re
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_weight_quantized_qpack_gb300", "csrc")
    for name in ("qpack_attend.cuh", "qpack_paged.cu", "qpack_paged.cuh", "qpack_gemv.cu"):
        with open(os.path.join(csrc, name), encoding="utf-8") as f:
            text = f.read()
        assert not re.search(r"__ldg|ld\.global\.nc|\bload8<", text), name


def test_unknown_pool_kind():
    import pytest

    import bit_weight_quantized_qpack_gb300 as qp
    for kind in (3, -1, "i8", None):
        with pytest.raises(qp.QpackError, match="kind: expected KV_I8"):
            qp.alloc_kv_pool(kind, 1, 4, 2, 16, 64, device="cpu")
