"""The decoding example runs its whole path (packed products, append, attend, fork, free, compact) and every attention of
it agrees with a dense one in fp64 over the cache that is read back."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("page,samples", [(16, 4), (8, 1)])
def test_paged_decode_example(qpg, page, samples):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import paged_decode
    got = paged_decode.main(["--layers", "2", "--q-heads", "8", "--kv-heads", "2", "--dim", "128", "--ffn", "2048", "--prompts",
                             "70", "16", "1", "133", "--samples", str(samples), "--steps", "9", "--page", str(page), "--check"])
    assert got["flags"] == 0
    # half a unit of fp16's last place, by element: 2^-11 of the norm at most, and as much again for everything else
    assert 0 < got["worst"] < 2.0 ** -10
    tab = got["decoder"].tab
    lens, refs = tab.lens.tolist(), tab.refs.tolist()
    live = set(got["live"].tolist())
    assert all((n > 0) == (s in live) for s, n in enumerate(lens))
    held = {}
    for row in tab.tables.tolist():
        for p in row:
            if p >= 0:
                held[p] = held.get(p, 0) + 1
    assert held == {p: r for p, r in enumerate(refs) if r}  # every reference is counted, no page leaks
