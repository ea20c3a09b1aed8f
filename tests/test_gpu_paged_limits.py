"""GPU tests of the paged KV cache at the limits of its types and of its arguments."""
import numpy as np
import pytest
import torch

from test_gpu_paged import DT, cache_rows, f64, make_pool, make_tables, pages_for

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("kind", ["i8", "f16", "bf16"])
@pytest.mark.parametrize("D,G", [(64, 1), (64, 16), (128, 3), (128, 11), (256, 8)])
def test_attend_one_token_is_its_value(qpg, kind, D, G):
    """The weight of a lone token is 1: its value comes back unchanged but for the output's one rounding (8-bit values
    often lie halfway between two bf16 numbers), whether the sequence or the window holds a single token."""
    T, lens = 16, [1, 1, 40, 1, 17, 1]
    pages = pages_for(lens, T)
    pool = make_pool(qpg, kind, 1, pages, 2, T, D, 3)
    tab, tables = make_tables(qpg, lens, T, pages, 4)
    last = torch.stack([torch.from_numpy(cache_rows(pool, 0, tab[s], n)[1][-1]) for s, n in enumerate(lens)])
    want = last.repeat_interleave(G, 1).cuda()
    for qdt, odt in (("f32", "bf16"), ("f32", "f16"), ("bf16", "f32"), ("f16", "bf16")):
        q = (torch.randn((len(lens), 2 * G, D), device="cuda") * 2).to(DT[qdt])
        out = torch.empty(q.shape, dtype=DT[odt], device="cuda")
        qpg.qpack_kv_attend(pool, 0, tables, q, window=1, out=out)
        assert torch.equal(out.double(), want.to(DT[odt]).double()), (qdt, odt)
    assert qpg.qpack_fetch_fault_flags() == 0


@pytest.mark.parametrize("kind", ["i8", "f16", "bf16"])
@pytest.mark.parametrize("G", [4, 11])
@pytest.mark.parametrize("top", [1e8, 4.9e7, 1e10, 3e15])
def test_attend_very_large_scores(qpg, kind, G, top):
    """Scores where fp32's spacing passes 1: one token far above the others takes all the weight, equal scores share it,
    and nothing becomes NaN."""
    T, D, H, lens = 16, 128, 2, [1, 2, 100, 700]
    pages = pages_for(lens, T)
    pool = make_pool(qpg, kind, 1, pages, H, T, D, 5)
    tab, tables = make_tables(qpg, lens, T, pages, 6)
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    q = torch.empty((len(lens), H * G, D), device="cuda").uniform_(0.9, 1.1, generator=g) * top
    one = 1                                                 # a code, or a value
    pool.k.zero_()
    if kind == "i8":
        pool.k_scales.fill_(1.0)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    for mode in ("one", "equal"):
        for s, n in enumerate(lens):
            for t in range(n):
                if mode == "equal" or t == n // 2:
                    pool.k[0, int(tab[s, t // T]), :, t % T, 5] = one
        qpg.qpack_kv_attend(pool, 0, tables, q, scale=1.0, out=out, lse=lse)
        for s, n in enumerate(lens):
            v = np.repeat(cache_rows(pool, 0, tab[s], n)[1], G, 1)      # [n, Hq, D]
            want = v[n // 2] if mode == "one" else v.mean(0)
            # a few roundings of the sums, each of at most n terms
            assert np.all(np.abs(f64(out[s]) - want) <= (np.abs(v).mean(0) * (n / 8 + 64) * 2.0 ** -23)), (mode, n)
            assert np.allclose(f64(lse[s]), f64(q[s, :, 5]), rtol=2.0 ** -21, atol=0)
    assert qpg.qpack_fetch_fault_flags() == 0
