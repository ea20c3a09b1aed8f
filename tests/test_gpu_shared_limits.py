"""What attention over shared prefixes does at its limits: offsets past 32 bits, the same sequence many times, graphs that share a
workspace, keys and values that are not finite."""
import numpy as np
import pytest
import torch

from test_gpu_paged import DT, f64, make_pool
from test_gpu_shared import check, forked, i32, tables_of

pytestmark = pytest.mark.gpu


def test_offsets_past_32_bits(qpg):
    """Prefix pages past 2^31 and 2^32 elements, own tokens behind them."""
    T, H, D = 64, 8, 128
    pages = (1 << 32) // (T * H * D) + 70
    k = torch.zeros((1, pages, H, T, D), dtype=torch.int8, device="cuda")
    v = torch.zeros_like(k)
    ks = torch.zeros((1, pages, H, T, D // 32), dtype=torch.float16, device="cuda")
    vs = torch.zeros_like(ks)
    pool = qpg.KVPool(k, v, ks, vs)
    ids = [pages - 1, (1 << 31) // (T * H * D), (1 << 32) // (T * H * D), pages - 9, 3]
    for c in (k, v):
        c[0, ids] = torch.randint(-127, 128, (5, H, T, D), dtype=torch.int8, device="cuda")
    for s in (ks, vs):
        s[0, ids] = 0.02
    tab = np.array([ids[:4], ids[:3] + ids[4:]], np.int32)
    lens = [250, 230]
    tables = tables_of(qpg, tab, lens)
    q = torch.randn((2, 32, D), device="cuda")
    out, lse = torch.zeros((2, 32, D), device="cuda"), torch.zeros((2, 32), device="cuda")
    qpg.qpack_kv_attend_shared(pool, 0, tables, q, i32([0, 2]), i32([190]), out=out, lse=lse)
    assert qpg.qpack_fetch_fault_flags() == 0
    check(out, lse, "f32", "i8", f64(q), pool, 0, tab, lens, [0, 1], [0, 0], [190, 190], D ** -0.5, None)


@pytest.mark.parametrize("kind", ["i8", "bf16"])
def test_a_sequence_many_times(qpg, kind):
    """Several queries of one sequence in a batch, in a group, in two groups and outside of them."""
    first, pref, lens, tab, pages = forked(qpg, [3], [150], [20, 1, 0], 16, seed=31)
    pool = make_pool(qpg, kind, 1, pages, 2, 16, 64, 31, 0, False)
    tables = tables_of(qpg, tab, lens)
    seqs = [0, 0, 1, 0, 2, 2, 1, 1, 0]
    q = torch.randn((9, 6, 64), device="cuda")
    out, lse = torch.zeros((9, 6, 64), device="cuda"), torch.zeros((9, 6), device="cuda")
    qpg.qpack_kv_attend_shared(pool, 0, tables, q, i32([0, 4, 6]), i32([150, 33]), seqs=i32(seqs), out=out, lse=lse)
    assert qpg.qpack_fetch_fault_flags() == 0
    check(out, lse, "f32", kind, f64(q), pool, 0, tab, lens, seqs, [0] * 4 + [2] * 2 + [1, 1, 0], [150] * 4 + [33] * 2 + [0] * 3,
          64 ** -0.5, None)


def test_graphs_that_share_a_workspace(qpg):
    """Two captured calls of different shapes on one workspace and stream, replayed in any order, with plain attention between."""
    first, pref, lens, tab, pages = forked(qpg, [20, 9, 3], [700, 90, 5], [70, 3, 0, 200], 16, seed=32)
    pool = make_pool(qpg, "f16", 1, pages, 2, 16, 128, 32, 0, False)
    tables = tables_of(qpg, tab, lens)
    q = torch.randn((32, 16, 128), device="cuda").half()
    ws = qpg.alloc_kv_shared_workspace(pool, 32, 16)
    calls = [(slice(0, 32), first, pref, None), (slice(0, 7), [1, 6], [300], i32([31, 4, 4, 2, 7, 1, 30])), (slice(0, 20), first[:2], pref[:1], None)]
    want, outs, graphs, keep = [], [], [], []
    for rows, f, p, seqs in calls:
        f, p = i32(f), i32(p)
        keep.append((f, p, seqs))
        want.append(qpg.qpack_kv_attend_shared(pool, 0, tables, q[rows], f, p, seqs=seqs))
        outs.append(torch.zeros_like(want[-1]))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            qpg.qpack_kv_attend_shared(pool, 0, tables, q[rows], f, p, seqs=seqs, out=outs[-1], workspace=ws)
        graphs.append(graph)
    plain = qpg.qpack_kv_attend(pool, 0, tables, q)
    for i in [0, 1, 0, 2, 2, 1, 1, 0, 2, 0]:
        outs[i].zero_()
        graphs[i].replay()
        assert torch.equal(qpg.qpack_kv_attend(pool, 0, tables, q, workspace=ws), plain)
        assert torch.equal(outs[i], want[i]), i
    assert qpg.qpack_fetch_fault_flags() == 0


@pytest.mark.parametrize("kind,D", [("f16", 128), ("bf16", 64), ("f16", 256)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_not_finite(qpg, kind, D, bad):
    """A key that is not finite makes the heads of its group that see it NaN, a value its own element; every other element keeps its
    bits. Rows that are shorter than the prefix do not see a key behind their end; a value there may still make its element NaN."""
    T, H, G = 16, 2, 3
    first, pref, lens, tab, pages = forked(qpg, [40, 4], [300, 60], [9, 0], T, seed=33)
    lens[5] = 120                                           # shorter than its group's prefix
    pool = make_pool(qpg, kind, 1, pages, H, T, D, 33, 0, False)
    tables = tables_of(qpg, tab, lens)
    q = torch.randn((44, H * G, D), device="cuda")
    call = lambda: qpg.qpack_kv_attend_shared(pool, 0, tables, q, i32(first), i32(pref), out=torch.zeros((44, H * G, D), device="cuda"))  # noqa: E731
    good = call()
    assert bool(torch.isfinite(good).all())
    page, slot = int(tab[0, 200 // T]), 200 % T
    kept = pool.k[0, page, 1, slot].clone()
    pool.k[0, page, 1, slot] = bad
    got = call()
    hit = torch.zeros_like(good, dtype=torch.bool)
    hit[:40, G:] = True
    hit[5] = False
    assert bool(torch.isnan(got[hit]).all()) and torch.equal(got[~hit], good[~hit])
    pool.k[0, page, 1, slot] = kept
    pool.v[0, page, 0, slot, 7] = bad
    got = call()
    hit.zero_()
    hit[:40, :G, 7] = True
    got[5, :G, 7] = good[5, :G, 7]                          # NaN where its weight of 0 meets the value in a sum, else its bits
    hit[5] = False
    assert not bool(torch.isfinite(got[hit]).any()) and torch.equal(got[~hit], good[~hit])
    pool.v[0, page, 0, slot, 7] = 0
    assert qpg.qpack_fetch_fault_flags() == 0


@pytest.mark.parametrize("kind", ["i8", "f16"])
@pytest.mark.parametrize("rows,G,prefix,qdt", [(3, 2, 39990, "f32"), (9, 16, 20470, "f16")])
def test_maxima_that_move_in_long_segments(qpg, kind, rows, G, prefix, qdt):
    """Long runs of tiles a block, one and two blocks of queries: scores swell and ebb, so that the running maximum holds in some
    tiles, moves a little in others and far in others, each query in its own."""
    T, H, D = 64, 8, 64
    first, pref, lens, tab, pages = forked(qpg, [rows], [prefix], [20, 3], T, seed=34)
    pool = make_pool(qpg, kind, 1, pages, H, T, D, 34, 0, False)
    t = torch.arange(lens[0], device="cuda")
    ramp = 40 * torch.sin(t / 300.0) + t / 700.0
    page = torch.from_numpy(tab[0]).cuda().long()[t // T]
    for h in range(H):
        x = ramp * (1 + h / 8)
        if kind == "i8":
            pool.k_scales[0, page, h, t % T, 0] = (x.abs() / 127).half()
            pool.k[0, page, h, t % T, 5] = (127 * torch.sign(x)).to(torch.int8)
        else:
            pool.k[0, page, h, t % T, 5] = x.half()
    q = torch.randn((rows, H * G, D), device="cuda") * 0.1
    q[:, :, 5] = torch.linspace(-2, 2, rows * H * G, device="cuda").view(rows, H * G)
    q = q.to(DT[qdt])
    out, lse = torch.empty((rows, H * G, D), dtype=torch.float16, device="cuda"), torch.empty((rows, H * G), device="cuda")
    qpg.qpack_kv_attend_shared(pool, 0, tables_of(qpg, tab, lens), q, i32(first), i32(pref), scale=1.0, out=out, lse=lse)
    assert qpg.qpack_fetch_fault_flags() == 0
    check(out, lse, "f16", kind, f64(q), pool, 0, tab, lens, range(rows), [0] * rows, pref * rows, 1.0, None)
