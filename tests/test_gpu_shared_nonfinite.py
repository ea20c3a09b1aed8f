"""Attention over shared prefixes with keys that are not finite."""
import pytest
import torch

from test_gpu_paged import make_pool
from test_gpu_shared import forked, i32, tables_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_key_that_is_alone_in_its_tile(qpg, kind, D):
    """A NaN key that no other token shares its tile with: out and lse are both NaN, for the rows that see it. As many groups as
    there are SMs, each a row of two tiles, so that a block has one group's two tiles and joins them itself."""
    tok, n = 64 if D == 256 else 128, torch.cuda.get_device_properties(0).multi_processor_count
    first, pref, lens, tab, pages = forked(qpg, [1] * n, [tok + 1] * n, [2, 0], 16, seed=36)
    lens[7] = tok                                           # ends before it
    pref[7] = tok
    pool = make_pool(qpg, kind, 1, pages, 1, 16, D, 36)
    bad = [5, 7, 8, n - 1]
    for b in bad:
        pool.k[0, int(tab[b, tok // 16]), 0, 0, 9] = float("nan")
    q = torch.randn((n, 3, D), device="cuda")
    out, lse = torch.empty((n, 3, D), device="cuda"), torch.empty((n, 3), device="cuda")
    qpg.qpack_kv_attend_shared(pool, 0, tables_of(qpg, tab, lens), q, i32(first), i32(pref), out=out, lse=lse)
    assert qpg.qpack_fetch_fault_flags() == 0
    hit = torch.zeros(n, dtype=torch.bool, device="cuda")
    hit[[5, 8, n - 1]] = True
    assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.isfinite(out[~hit]).all() and torch.isfinite(lse[~hit]).all()
