"""Attention over shared prefixes with queries and keys that are not finite."""
import pytest
import torch

from test_gpu_paged import DT, make_pool
from test_gpu_shared import forked, i32, tables_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,qdt", [("i8", "f16"), ("f16", "f16"), ("bf16", "bf16"), ("i8", "f32"), ("f16", "bf16"), ("bf16", "f16")])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("prefix,own", [(1, 0), (1, 5), (130, 0), (700, 3)])
def test_queries_that_are_not_finite(qpg, kind, qdt, D, prefix, own):
    """An infinite or NaN query makes its own head NaN, as without sharing, whatever the signs of the keys that it meets (of an
    infinity's products alone the largest can be -inf, and every weight 0); the others keep their bits."""
    first, pref, lens, tab, pages = forked(qpg, [5], [prefix], [own], 16, seed=35)
    pool = make_pool(qpg, kind, 1, pages, 2, 16, D, 35)
    pool.k[..., 3] = 50 if kind == "i8" else pool.k[..., 3].abs() + 0.5    # one element has the same sign in all keys
    tables = tables_of(qpg, tab, lens)
    q = torch.randn((5, 6, D), device="cuda").to(DT[qdt])

    def run(q):
        out, lse = torch.empty((5, 6, D), device="cuda"), torch.empty((5, 6), device="cuda")
        qpg.qpack_kv_attend_shared(pool, 0, tables, q, i32(first), i32(pref), out=out, lse=lse)
        return out, lse

    good, good_lse = run(q)
    assert bool(torch.isfinite(good).all()) and bool(torch.isfinite(good_lse).all())
    for bad in (float("nan"), float("inf"), -float("inf")):
        for scale_of in (1.0, 0.0):                         # the other elements as they are, or none
            q2 = q.clone()
            q2[3, 1] *= scale_of
            q2[3, 1, 3] = bad
            got, got_lse = run(q2)
            hit = torch.zeros((5, 6), dtype=torch.bool, device="cuda")
            hit[3, 1] = True
            assert torch.isnan(got[3, 1]).all() and torch.isnan(got_lse[3, 1]), (bad, scale_of, got[3, 1, :4], got_lse[3, 1])
            assert torch.equal(got[~hit], good[~hit]) and torch.equal(got_lse[~hit], good_lse[~hit])
    assert qpg.qpack_fetch_fault_flags() == 0


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
