"""Attention over shared prefixes at the ends of its range: the most rows and groups, many query heads, rows inside wider rows, calls
that run at the same time. Where tables hold the prefixes, as after a fork, attention without sharing gives the same: weights
and queries are off by 2^-22 in each (2^-16 over a bfloat16 cache), which scores of a few units of size raise by their size."""
import pytest
import torch

from test_gpu_paged import DT, make_pool
from test_gpu_shared import forked, i32, tables_of

pytestmark = pytest.mark.gpu


def copy_tails(pool, tab, lens, first, pref):
    """The part of a prefix that ends inside a page, from the first row's page to the others' own, as a fork leaves it."""
    T = pool.page_tokens
    at = [(int(tab[b, p // T]), int(tab[f, p // T]), s) for f, n, p in zip(first, first[1:], pref) if p <= lens[f]
          for b in range(f + 1, n) if lens[b] for s in range(p % T)]
    if not at:
        return
    dst, src, slot = (torch.tensor(x, device="cuda") for x in zip(*at))
    for x in (pool.k, pool.v, pool.k_scales, pool.v_scales):
        if x is not None:
            x[0, dst, :, slot] = x[0, src, :, slot]


def as_without(qpg, kind, pool, tables, q, first, pref, flags=0, **kw):
    """Both calls on the same inputs."""
    one, two = (torch.empty(q.shape, device="cuda") for _ in range(2))
    l1, l2 = (torch.empty(q.shape[:2], device="cuda") for _ in range(2))
    qpg.qpack_kv_attend(pool, 0, tables, q, out=one, lse=l1, **kw)
    qpg.qpack_kv_attend_shared(pool, 0, tables, q, i32(first), i32(pref), out=two, lse=l2, **kw)
    assert qpg.qpack_fetch_fault_flags() == flags
    unit = 2.0 ** -15 if kind == "bf16" else 2.0 ** -17
    seen = torch.isfinite(l1)
    assert torch.equal(seen, torch.isfinite(l2))
    assert (one - two).abs().max() <= unit * 8 * max(1.0, float(one.abs().max()))
    assert (l1[seen] - l2[seen]).abs().max() <= 64 * unit


@pytest.mark.parametrize("kind", ["i8", "bf16"])
@pytest.mark.parametrize("sizes", [[8] * 512, [4096], [1] * 511 + [3585], [0] * 511 + [4096]])
def test_most_rows_and_groups(qpg, kind, sizes):
    prefix = [(7 * i) % 190 for i in range(len(sizes) - 1)] + [170]
    first, pref, lens, tab, pages = forked(qpg, sizes, prefix, [2, 0, 17], 16, seed=51, idle=(3, 4000))
    pref = [0 if n == 0 else p for n, p in zip(sizes, pref)]
    pool = make_pool(qpg, kind, 1, pages, 1, 16, 64, 51)
    assert len(lens) == 4096
    copy_tails(pool, tab, lens, first, pref)
    q = torch.randn((4096, 2, 64), device="cuda")
    # a group whose first row is idle: its prefix is longer than that row, so it is cut to nothing and reported
    cut = any(n and p > lens[f] for n, p, f in zip(sizes, pref, first))
    as_without(qpg, kind, pool, tables_of(qpg, tab, lens), q, first, pref, qpg.FAULT_PAGE if cut else 0)


@pytest.mark.parametrize("kind,D,H,G,rows", [("i8", 64, 1, 2048, 2), ("f16", 128, 2, 777, 1), ("bf16", 256, 1, 300, 3)])
def test_many_query_heads(qpg, kind, D, H, G, rows):
    first, pref, lens, tab, pages = forked(qpg, [rows], [333], [2, 0, 17], 16, seed=52)
    pool = make_pool(qpg, kind, 1, pages, H, 16, D, 52)
    copy_tails(pool, tab, lens, first, pref)
    as_without(qpg, kind, pool, tables_of(qpg, tab, lens), torch.randn((rows, H * G, D), device="cuda"), first, pref)


@pytest.mark.parametrize("kind", ["i8", "f16", "bf16"])
@pytest.mark.parametrize("D,qdt,odt", [(64, "f16", "f16"), (128, "bf16", "f32"), (256, "f32", "bf16"), (128, "f32", "f16")])
def test_rows_inside_wider_rows(qpg, kind, D, qdt, odt):
    """Queries beside keys and values of one product, outputs inside a wider buffer, whose other elements stay."""
    first, pref, lens, tab, pages = forked(qpg, [6, 3], [200, 61], [9, 0, 3], 16, seed=53)
    pool = make_pool(qpg, kind, 1, pages, 2, 16, D, 53)
    tables = tables_of(qpg, tab, lens)
    wide = torch.randn((9, 10, D), device="cuda").to(DT[qdt])
    want = torch.empty((9, 6, D), dtype=DT[odt], device="cuda")
    qpg.qpack_kv_attend_shared(pool, 0, tables, wide[:, 2:8].contiguous(), i32(first), i32(pref), out=want)
    room = torch.full((11, 9, D), 7.0, dtype=DT[odt], device="cuda")
    qpg.qpack_kv_attend_shared(pool, 0, tables, wide[:, 2:8], i32(first), i32(pref), out=room[:, 1:7])
    assert qpg.qpack_fetch_fault_flags() == 0
    assert torch.equal(room[:9, 1:7], want)
    room[:9, 1:7] = 7
    assert (room == 7).all()


def test_calls_at_the_same_time(qpg):
    """Two streams, each with a workspace of its own, sampling and head norms between: every call gives what it gives alone."""
    first, pref, lens, tab, pages = forked(qpg, [30, 2], [1500, 90], [40, 3], 16, seed=54)
    pool = make_pool(qpg, "i8", 1, pages, 4, 16, 128, 54)
    tables = tables_of(qpg, tab, lens)
    f, p = i32(first), i32(pref)
    w, rope, pos = torch.rand(128, device="cuda") + 0.5, torch.randn((2000, 128), device="cuda"), i32([len(lens) + 31 * i for i in range(32)])
    streams = [torch.cuda.Stream() for _ in range(2)]
    sets = []
    for s in streams:
        q, x, u = torch.randn((32, 16, 128), device="cuda"), torch.randn((32, 40000), device="cuda") * 3, torch.rand(32, device="cuda")
        top_p = torch.full((32,), 0.9, device="cuda")
        sets.append((q, x, u, top_p, qpg.alloc_kv_shared_workspace(pool, 32, 16)))

    def step(stream, q, x, u, top_p, ws):
        y, _ = qpg.qpack_qk_norm_rope(q, None, w, rope=rope, pos=pos, stream=stream)
        return (y, qpg.qpack_kv_attend_shared(pool, 0, tables, y, f, p, workspace=ws, stream=stream),
                qpg.qpack_sample(x, u, top_p=top_p, stream=stream))

    want = [step(None, *s) for s in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            got[i].append(step(s, *sets[i]))
    torch.cuda.synchronize()
    assert qpg.qpack_fetch_fault_flags() == 0
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))
