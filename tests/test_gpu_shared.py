"""GPU parity of attention over shared prefixes against the 64-bit restatement of attention (oracle/paged.py), row by row.

The tolerance is that of attention without sharing (derived in test_gpu_paged.py), with the units of this call's terms: over
the prefix a query is off by 2^-22 of itself (fp16 and 8-bit pools) or 2^-16 (bfloat16), a probability by 2^-11 where it is one
fp16 term, 2^-22 where it is two, 2^-16 where it is two of bfloat16; probabilities below fp16's normal numbers by 2^-25 where the
largest is 2^7 or more, so by 2^-32 of that each. Parts are joined in fp32: 2^-22 a join of factors, at most 160 parts,
whose roundings add up like those of a sum. A weight's error scales |v|, its share of all weights."""
import numpy as np
import pytest
import torch

from oracle import paged as ref
from test_gpu_paged import DT, SPLIT, ULP, cache_rows, f64, make_pool, rope_table

pytestmark = pytest.mark.gpu


def forked(qpg, sizes, prefix, own, T, pages_extra=3, seed=0, idle=(), shared=True):
    """Groups of sequences that hold the same full pages of their prefix, as a fork leaves them; the row's own tokens and the
    prefix's last part are in pages of their own. Returns first, prefix, lens, tables (numpy) and KVTables."""
    rng = np.random.default_rng(seed)
    first, rows, lens, at = [0], [], [], 0
    for n, p in zip(sizes, prefix):
        for i in range(n):
            b = len(lens)
            length = 0 if b in idle else p + own[b % len(own)]
            need = -(-length // T)
            same = rows[first[-1]][:min(p // T, need)] if i and shared else []
            rows.append(list(same) + list(range(at, at + need - len(same))))
            at += need - len(same)
            lens.append(length)
        first.append(first[-1] + n)
    pages = at + pages_extra
    perm = rng.permutation(pages)
    width = max(1, max(map(len, rows)) if rows else 1) + 1
    tab = np.full((len(rows), width), -1, np.int32)
    for i, r in enumerate(rows):
        tab[i, :len(r)] = perm[r]
    return first, list(prefix), lens, tab, pages


def tables_of(qpg, tab, lens):
    return qpg.KVTables(torch.from_numpy(tab).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"))


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def tokens_of(pool, layer, tab, lens, lead, p, s):
    """k', v' of row s: the first p tokens from the pages of row `lead`."""
    n = lens[s]
    k, v = cache_rows(pool, layer, tab[s], n)
    m = min(n, p)
    if m:
        ka, va = cache_rows(pool, layer, tab[lead], m)
        k, v = np.concatenate([ka, k[m:]]), np.concatenate([va, v[m:]])
    return k, v


def check(out, lse, odt, kind, q, pool, layer, tab, lens, seqs, lead, pref, scale, rope):
    """Every row: seqs[b] its sequence, lead[b] its group's first sequence, pref[b] its prefix."""
    out, lse = f64(out), f64(lse)
    B, Hq, D = q.shape
    H = pool.heads
    split_p = 2.0 ** -16 if kind == "bf16" else 2.0 ** -22 if odt == "f32" else 2.0 ** -11
    for b in range(B):
        L = lens[seqs[b]]
        if L == 0:
            assert np.all(out[b] == 0) and np.all(lse[b] == -np.inf)
            continue
        k, v = tokens_of(pool, layer, tab, lens, lead[b], pref[b], seqs[b])
        row = None if rope is None else rope[L - 1]
        want, wl = ref.attend(q[b], k, v, scale, 0, row)
        qr = q[b] if row is None else ref.rotate64(q[b][None], row[None])[0]
        qa = np.maximum(np.abs(qr), np.abs(q[b]))
        for h in range(Hq):
            kv = h // (Hq // H)
            x = (k[:, kv] @ qr[h]) * scale
            w = np.exp(x - x.max())
            w /= w.sum()
            mass = (np.abs(k[:, kv]) @ qa[h]).max() * abs(scale)
            dx = mass * (SPLIT[kind] + (D + 8) * 2.0 ** -23)
            va = np.abs(v[:, kv])
            mean = w @ va                                  # of each element, by the weights
            tol = mean * (3 * dx + split_p + 2.0 ** -20 + (L / 8 + 64 + 160) * 2.0 ** -23) + 2.0 ** -32 * va.sum(0)
            tol = tol + np.abs(want[h]) * ULP[odt] + 2.0 ** -25 * (odt != "f32")
            err = np.abs(out[b, h] - want[h])
            assert np.all(err <= tol), (b, h, L, pref[b], float((err / tol).max()))
            ltol = dx + 2.0 ** -20 + np.abs(wl[h]) * 2.0 ** -22 + (L / 8 + 160) * 2.0 ** -23
            assert abs(lse[b, h] - wl[h]) <= ltol, (b, h, L, lse[b, h], wl[h])


def case(qpg, kind, H, G, D, T, sizes, prefix, own, qdt="f32", odt="f16", rope=False, scale=None, seed=0, qscale=2.0, idle=(),
         shared=True, order=None, layers=1, layer=0, page_pad=0, poison=False, plain=True):
    first, pref, lens, tab, pages = forked(qpg, sizes, prefix, own, T, seed=seed, idle=idle, shared=shared)
    pool = make_pool(qpg, kind, layers, pages, H, T, D, seed, page_pad, poison)
    if poison:                                              # real values only where tokens are
        clean = make_pool(qpg, kind, layers, pages, H, T, D, seed, page_pad)
        for s, n in enumerate(lens):
            for c in range(-(-n // T)):
                p, r = int(tab[s, c]), min(T, n - c * T)
                for a, b in ((pool.k, clean.k), (pool.v, clean.v), (pool.k_scales, clean.k_scales), (pool.v_scales, clean.v_scales)):
                    if a is not None:
                        a[:, p, :, :r] = b[:, p, :, :r]
    B = len(lens)
    rows = list(range(B))
    if order is not None:                                   # sequences in another order in the table than in the batch
        perm = np.random.default_rng(seed + 9).permutation(B)
        t2, l2 = np.empty_like(tab), [0] * B
        for b in range(B):
            t2[perm[b]], l2[perm[b]] = tab[b], lens[b]
        tab, lens, rows = t2, l2, [int(x) for x in perm]
    tables = tables_of(qpg, tab, lens)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 2)
    q = (torch.empty((B, H * G, D), device="cuda").normal_(generator=g) * qscale).to(DT[qdt])
    table = rope_table(max(max(lens), 1), D, seed) if rope else None
    out = torch.full((B, H * G, D), 7.0, dtype=DT[odt], device="cuda")
    lse = torch.full((B, H * G), 7.0, device="cuda")
    ws = qpg.alloc_kv_shared_workspace(pool, B, H * G)
    for i in range(2):                                      # the second call finds the workspace as the first left it
        qpg.qpack_kv_attend_shared(pool, layer, tables, q, i32(first), i32(pref), scale=scale, out=out, lse=lse, workspace=ws,
                                   seqs=None if order is None else i32(rows),
                                   rope=None if table is None else torch.from_numpy(table).cuda())
        once = out.clone() if i == 0 else once
    torch.cuda.synchronize()
    assert qpg.qpack_fetch_fault_flags() == 0
    assert torch.equal(once, out), "the same call twice differs"
    of = np.searchsorted(first, np.arange(B), side="right") - 1
    check(out, lse, odt, kind, f64(q), pool, layer, tab, lens, rows, [rows[first[g]] for g in of], [pref[g] for g in of],
          D ** -0.5 if scale is None else scale, table)
    return out


KINDS = ["i8", "f16", "bf16"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_one_tile(qpg, kind, D):
    """A prefix inside one tile, one group, queries of one block."""
    case(qpg, kind, 1, 4, D, 16, [5], [50], [3, 0, 20], seed=D)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 3, 8, 17])
def test_kinds(qpg, kind, D, G):
    """Every cache type, width and group of query heads; prefixes around the tiles' edges; rows without tokens of their own."""
    case(qpg, kind, 2, G, D, 16, [3, 1, 6, 2], [127, 128, 300, 1], [0, 1, 17, 40, 130], seed=D + G, rope=G == 3)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("qdt,odt", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f16", "f32"), ("bf16", "f16"),
                                     ("f32", "bf16")])
def test_types(qpg, kind, qdt, odt):
    case(qpg, kind, 2, 4, 128, 64, [9, 4], [700, 130], [5, 0, 64], qdt, odt, rope=qdt == "f32", seed=3)


@pytest.mark.parametrize("kind", ["i8", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 8, 32, 128, 1024])
def test_page_sizes(qpg, kind, T):
    """Pages that end inside a tile, tiles that end inside a page, prefixes that end inside both."""
    case(qpg, kind, 3, 5, 128, T, [4, 3], [513, 1030], [7, 0, 33], seed=T)


@pytest.mark.parametrize("kind,D", [("i8", 128), ("f16", 64), ("bf16", 256)])
def test_many_queries_and_long_prefixes(qpg, kind, D):
    """Several blocks of queries a group, prefixes that many blocks share, and groups that one block takes whole."""
    case(qpg, kind, 2, 8, D, 64, [70, 1, 33], [3000, 9000, 40], [9, 0, 200], seed=5, rope=True)


def test_one_long_prefix(qpg):
    case(qpg, "i8", 1, 4, 128, 128, [2], [60001], [100], seed=6)


@pytest.mark.parametrize("kind", KINDS)
def test_many_groups(qpg, kind):
    """A group a row, as if nothing were shared, and groups without rows between them."""
    sizes = [1, 0, 2, 0, 0] * 30
    prefix = [(37 * i) % 290 for i in range(len(sizes))]
    case(qpg, kind, 2, 2, 64, 16, sizes, prefix, [0, 3, 50], seed=7)


@pytest.mark.parametrize("kind", KINDS)
def test_idle_rows_strides_and_order(qpg, kind):
    """Rows of length zero, pools with slack between pages, layers, sequences in any order, slots without a token poisoned."""
    case(qpg, kind, 2, 4, 128, 16, [6, 5], [200, 77], [4, 9, 0], idle=(2, 8, 10), order=1, layers=2, layer=1, page_pad=1, seed=8)
    case(qpg, kind, 2, 4, 64, 16, [6, 5], [200, 77], [4, 9, 0], idle=(3,), poison=True, seed=9)


@pytest.mark.parametrize("kind", KINDS)
def test_rows_shorter_than_their_prefix(qpg, kind):
    """A row that has fewer tokens than its group's prefix sees as many of the prefix as it has."""
    first, pref, lens, tab, pages = forked(qpg, [5], [300], [10], 16, seed=10)
    lens[1], lens[2], lens[4] = 1, 128, 299
    pool = make_pool(qpg, kind, 1, pages, 2, 16, 128, 10)
    q = torch.randn((5, 8, 128), device="cuda")
    out, lse = torch.empty_like(q), torch.empty((5, 8), device="cuda")
    rope = rope_table(400, 128)
    qpg.qpack_kv_attend_shared(pool, 0, tables_of(qpg, tab, lens), q, i32(first), i32(pref), out=out, lse=lse,
                               rope=torch.from_numpy(rope).cuda())
    assert qpg.qpack_fetch_fault_flags() == 0
    check(out, lse, "f32", kind, f64(q), pool, 0, tab, lens, range(5), [0] * 5, [300] * 5, 128 ** -0.5, rope)


@pytest.mark.parametrize("scale", [0.0, -0.1, 1.0, 1e-30])
@pytest.mark.parametrize("kind", KINDS)
def test_scales(qpg, kind, scale):
    case(qpg, kind, 1, 4, 64, 16, [7], [290], [5, 0], scale=scale, odt="f32", seed=11)


@pytest.mark.parametrize("kind", KINDS)
def test_rising_maxima(qpg, kind):
    """Scores that rise by thousands along the prefix, so that the running maximum moves in every tile, and fall again."""
    first, pref, lens, tab, pages = forked(qpg, [6], [1500], [20], 64, seed=12)
    pool = make_pool(qpg, kind, 1, pages, 1, 64, 64, 12)
    ramp = torch.tensor([(t if t < 1100 else 2200 - t) / 10.0 for t in range(1520)], device="cuda")
    for s in range(6):
        t = torch.arange(lens[s], device="cuda")
        page = torch.from_numpy(tab[s]).cuda().long()[t // 64]
        if kind == "i8":
            pool.k_scales[0, page, 0, t % 64, 0] = (ramp[:lens[s]] / 127).half()
            pool.k[0, page, 0, t % 64, 5] = 127
        else:
            pool.k[0, page, 0, t % 64, 5] = ramp[:lens[s]].to(pool.k.dtype)
    q = torch.zeros((6, 4, 64), device="cuda")
    q[:, :, 5] = torch.linspace(-3, 30, 24, device="cuda").view(6, 4)
    out, lse = torch.empty_like(q), torch.empty((6, 4), device="cuda")
    qpg.qpack_kv_attend_shared(pool, 0, tables_of(qpg, tab, lens), q, i32(first), i32(pref), scale=1.0, out=out, lse=lse)
    assert qpg.qpack_fetch_fault_flags() == 0
    check(out, lse, "f32", kind, f64(q), pool, 0, tab, lens, range(6), [0] * 6, [1500] * 6, 1.0, None)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_one_token_is_its_value(qpg, kind, D):
    """The weight of a lone token is 1, in the prefix or behind it: its value comes back but for the output's rounding."""
    first, pref, lens, tab, pages = forked(qpg, [3, 2], [1, 0], [0, 0, 0, 1, 1], 16, seed=13)
    pool = make_pool(qpg, kind, 1, pages, 2, 16, D, 13)
    q = torch.randn((5, 6, D), device="cuda") * 3
    for odt in ("f16", "bf16", "f32"):
        out = torch.empty(q.shape, dtype=DT[odt], device="cuda")
        qpg.qpack_kv_attend_shared(pool, 0, tables_of(qpg, tab, lens), q, i32(first), i32(pref), out=out)
        for b in range(5):
            v = cache_rows(pool, 0, tab[0 if b < 3 else b], 1)[1][0]
            assert torch.equal(out[b].double().cpu(), torch.from_numpy(np.repeat(v, 3, 0)).to(DT[odt]).double()), (b, odt)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128])
def test_as_attention_without_sharing(qpg, kind, D):
    """Over sequences that hold the same pages, or copies, the result is qpack_kv_attend's: a fork by the page operators."""
    T, H, G, n, parent = 16, 2, 4, 11, 345
    pages = 200
    pool = make_pool(qpg, kind, 1, pages, H, T, D, 14)
    tables = qpg.alloc_kv_tables(n + 1, 40, pages)
    qpg.qpack_kv_reserve(pool, tables, i32([0]), i32([parent]))
    qpg.qpack_kv_fork(pool, tables, i32([0] * n), i32(list(range(1, n + 1))))
    qpg.qpack_kv_reserve(pool, tables, i32(list(range(1, n + 1))), i32([1 + 3 * i for i in range(n)]))
    seqs = i32(list(range(1, n + 1)))
    q = torch.randn((n, H * G, D), device="cuda")
    rope = torch.from_numpy(rope_table(500, D)).cuda()
    one, two = (torch.empty_like(q) for _ in range(2))
    l1, l2 = (torch.empty((n, H * G), device="cuda") for _ in range(2))
    qpg.qpack_kv_attend(pool, 0, tables, q, seqs=seqs, rope=rope, out=one, lse=l1)
    qpg.qpack_kv_attend_shared(pool, 0, tables, q, i32([0, n]), i32([parent]), seqs=seqs, rope=rope, out=two, lse=l2)
    assert qpg.qpack_fetch_fault_flags() == 0
    unit = 2.0 ** -15 if kind == "bf16" else 2.0 ** -17
    assert (one - two).abs().max() <= unit * 8 * max(1.0, float(one.abs().max())) and (l1 - l2).abs().max() <= 64 * unit
    # without groups it is that call itself
    qpg.qpack_kv_attend_shared(pool, 0, tables, q, i32([0]), i32([]), seqs=seqs, rope=rope, out=two, lse=l2)
    assert torch.allclose(one, two, rtol=1e-6, atol=1e-6) and torch.allclose(l1, l2, rtol=1e-6, atol=1e-6)


def test_rows_of_no_group(qpg):
    """Rows before the first group and behind the last have no prefix."""
    first, pref, lens, tab, pages = forked(qpg, [2, 4, 3], [100, 200, 150], [8, 1], 16, seed=15)
    pool = make_pool(qpg, "f16", 1, pages, 2, 16, 64, 15)
    q = torch.randn((9, 6, 64), device="cuda")
    out, lse = torch.empty_like(q), torch.empty((9, 6), device="cuda")
    qpg.qpack_kv_attend_shared(pool, 0, tables_of(qpg, tab, lens), q, i32(first[1:3]), i32(pref[1:2]), out=out, lse=lse)
    assert qpg.qpack_fetch_fault_flags() == 0
    inside = [2 <= b < 6 for b in range(9)]
    check(out, lse, "f32", "f16", f64(q), pool, 0, tab, lens, range(9), [2 if i else b for b, i in enumerate(inside)],
          [200 if i else 0 for i in inside], 64 ** -0.5, None)


def test_groups_and_prefixes_out_of_range(qpg):
    """Groups that are not rising or pass the batch: reported, and every row goes without a prefix. A prefix longer than its
    first row, or negative, is cut and reported."""
    first, pref, lens, tab, pages = forked(qpg, [4, 4], [100, 60], [8, 1], 16, seed=16)
    pool = make_pool(qpg, "f16", 1, pages, 2, 16, 64, 16)
    tables = tables_of(qpg, tab, lens)
    q = torch.randn((8, 6, 64), device="cuda")
    out, lse = torch.empty_like(q), torch.empty((8, 6), device="cuda")
    for bad in ([0, 9, 8], [4, 2, 8], [-1, 4, 8], [0, 4, 2 ** 31 - 1], [0, -2 ** 31, 8]):
        qpg.qpack_kv_attend_shared(pool, 0, tables, q, i32(bad), i32(pref), out=out, lse=lse)
        assert qpg.qpack_fetch_fault_flags() == qpg.FAULT_PAGE, bad
        check(out, lse, "f32", "f16", f64(q), pool, 0, tab, lens, range(8), range(8), [0] * 8, 64 ** -0.5, None)
    for given, used in (([101 + 8, -5], [lens[0], 0]), ([2 ** 31 - 1, -2 ** 31], [lens[0], 0])):
        qpg.qpack_kv_attend_shared(pool, 0, tables, q, i32(first), i32(given), out=out, lse=lse)
        assert qpg.qpack_fetch_fault_flags() == qpg.FAULT_PAGE
        check(out, lse, "f32", "f16", f64(q), pool, 0, tab, lens, range(8), [0] * 4 + [4] * 4, [used[0]] * 4 + [used[1]] * 4,
              64 ** -0.5, None)


def test_pages_and_sequences_out_of_range(qpg):
    """Bad page numbers in a prefix count as keys and values of zero, unknown sequences as empty ones; reported."""
    first, pref, lens, tab, pages = forked(qpg, [3, 2], [100, 60], [8, 1], 16, seed=17)
    pool = make_pool(qpg, "f16", 1, pages, 2, 16, 64, 17)
    broken = tab.copy()
    broken[0, 2] = pages + 5
    q = torch.randn((5, 6, 64), device="cuda")
    out, lse = torch.empty_like(q), torch.empty((5, 6), device="cuda")
    qpg.qpack_kv_attend_shared(pool, 0, tables_of(qpg, broken, lens), q, i32(first), i32(pref), out=out, lse=lse)
    assert qpg.qpack_fetch_fault_flags() == qpg.FAULT_PAGE
    zero = int(tab[0, 2])
    pool.k[0, zero], pool.v[0, zero] = 0, 0
    check(out, lse, "f32", "f16", f64(q), pool, 0, tab, lens, range(5), [0] * 3 + [3] * 2, [100] * 3 + [60] * 2, 64 ** -0.5, None)
    tables = tables_of(qpg, tab, lens)
    qpg.qpack_kv_attend_shared(pool, 0, tables, q, i32(first), i32(pref), seqs=i32([0, 5, 2, 3, -1]), out=out, lse=lse)
    assert qpg.qpack_fetch_fault_flags() == qpg.FAULT_PAGE
    assert (out[[1, 4]] == 0).all() and (lse[[1, 4]] == -float("inf")).all() and torch.isfinite(lse[[0, 2, 3]]).all()
    qpg.qpack_kv_attend_shared(pool, 0, tables, q, i32(first), i32(pref), rope=torch.from_numpy(rope_table(61, 64)).cuda(), out=out)
    assert qpg.qpack_fetch_fault_flags() == qpg.FAULT_PAGE


def test_stream_graph_and_larger_workspaces(qpg):
    """Other streams, capture and replay with new inputs, workspaces that serve smaller calls and plain attention in turn."""
    first, pref, lens, tab, pages = forked(qpg, [6, 5], [400, 90], [8, 1], 16, seed=18)
    pool = make_pool(qpg, "i8", 1, pages, 2, 16, 128, 18)
    tables = tables_of(qpg, tab, lens)
    q = torch.randn((11, 8, 128), device="cuda")
    f, p = i32(first), i32(pref)
    want = qpg.qpack_kv_attend_shared(pool, 0, tables, q, f, p)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = qpg.qpack_kv_attend_shared(pool, 0, tables, q, f, p, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    ws = qpg.alloc_kv_shared_workspace(pool, 64, 8)
    plain = qpg.qpack_kv_attend(pool, 0, tables, q)
    for _ in range(3):
        assert torch.equal(qpg.qpack_kv_attend_shared(pool, 0, tables, q, f, p, workspace=ws), want)
        assert torch.equal(qpg.qpack_kv_attend(pool, 0, tables, q, workspace=ws), plain)
        assert torch.equal(qpg.qpack_kv_attend_shared(pool, 0, tables, q[:6], f[:2], p[:1], workspace=ws), want[:6])
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qpg.qpack_kv_attend_shared(pool, 0, tables, q, f, p, out=out, workspace=ws)
    q.copy_(torch.randn_like(q))
    tables.lens -= 1                                        # every row a token shorter
    p.copy_(i32([399, 89]))
    want = qpg.qpack_kv_attend_shared(pool, 0, tables, q, f, p)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and qpg.qpack_fetch_fault_flags() == 0


def test_no_rows(qpg):
    pool = make_pool(qpg, "f16", 1, 4, 2, 16, 64, 19)
    tables = qpg.alloc_kv_tables(3, 4, 4)
    q = torch.zeros((0, 6, 64), device="cuda")
    assert qpg.qpack_kv_attend_shared(pool, 0, tables, q, i32([0]), i32([])).shape == (0, 6, 64)
    q = torch.zeros((3, 6, 64), device="cuda")
    out = qpg.qpack_kv_attend_shared(pool, 0, tables, q, i32([0, 3]), i32([0]))
    assert (out == 0).all() and qpg.qpack_fetch_fault_flags() == 0
