"""GPU parity of the paged KV cache: attention of one new token, append, read back and the page operators against the
64-bit restatement (oracle/paged.py).

Attention's tolerance. With e the unit of the two-term split (2^-22 for 8-bit and fp16 pools, 2^-16 for bfloat16 ones,
whose terms have 8 bits each) a score is off by at most dx = scale * sum_i |q_i k_i| * (e + (D + 8) 2^-23): the query's
rounding and D fp32 additions whose rounding is at worst a truncation, the rotation's three included. A probability
is then off by the factor e^(2 dx) - 1 < 3 dx for the ratio of sums, by e for its own split and 2^-20 for the
exponential and the maximum's running updates, and the sum over n tokens, taken 8 or more at a time, adds (n / 8 + 64)
roundings of 2^-23. All of it scales max |v|. The output's own rounding is half a unit in the last place. The
log-sum-exp is off by dx plus a few fp32 roundings of its size."""
import numpy as np
import pytest
import torch

from oracle import paged as ref

pytestmark = pytest.mark.gpu

KIND = {"i8": 0, "f16": 1, "bf16": 2}
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SPLIT = {"i8": 2.0 ** -22, "f16": 2.0 ** -22, "bf16": 2.0 ** -16}
ULP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def make_pool(qpg, kind, layers, pages, heads, T, D, seed, page_pad=0, poison=False):
    """A pool of random values; page_pad pages of slack between pages (a strided pool); poison: NaN and inf everywhere
    (16-bit values, or the 8-bit scales), to be overwritten where tokens are."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    shape = (layers, pages * (1 + page_pad), heads, T, D)
    step = 1 + page_pad
    if kind == "i8":
        k, v = (torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)[:, ::step] for _ in "kv")
        sc = [torch.empty(shape[:-1] + (D // 32,), device="cuda").normal_(-4, 0.5, generator=g).exp_().half()[:, ::step]
              for _ in "kv"]
        if poison:
            for s in sc:
                s.fill_(float("nan"))
                s[..., 0] = float("inf")
        return qpg.KVPool(k, v, *sc)
    k, v = (torch.empty(shape, device="cuda").normal_(generator=g).to(DT[kind])[:, ::step] for _ in "kv")
    if poison:
        for t in (k, v):
            t.fill_(float("nan"))
            t[..., ::2] = float("inf")
            t[..., 1::4] = -torch.finfo(DT[kind]).max
    return qpg.KVPool(k, v)


def cache_rows(pool, layer, table, L):
    """k', v' [L, H, D] fp64 of one sequence."""
    T = pool.page_tokens
    t = np.arange(L)
    page, slot = torch.as_tensor(np.asarray(table))[t // T].long().cuda(), torch.as_tensor(t % T).cuda()
    out = []
    for c, s in ((pool.k, pool.k_scales), (pool.v, pool.v_scales)):
        if L == 0:
            out.append(np.zeros((0, pool.heads, pool.dim)))
        elif s is None:
            out.append(f64(c[layer][page, :, slot]))
        else:
            out.append(ref.values(c[layer][page, :, slot].cpu().numpy(), s[layer][page, :, slot].cpu().numpy()))
    return out


def make_tables(qpg, lens, T, pages, seed, extra=1, refs=None):
    rng = np.random.default_rng(seed)
    perm = rng.permutation(pages)
    width = max(-(-max(lens) // T), 0) + extra
    tab = np.full((len(lens), width), -1, np.int32)
    at = 0
    for i, n in enumerate(lens):
        c = -(-n // T)
        tab[i, :c] = perm[at:at + c]
        at += c
    assert at <= pages
    return tab, qpg.KVTables(torch.from_numpy(tab).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), refs)


def pages_for(lens, T):
    return sum(-(-n // T) for n in lens) + 2


def rope_table(rows, D, seed=0):
    g = np.random.default_rng(seed)
    a = g.uniform(-np.pi, np.pi, (rows, D // 2))
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def check_attend(out, lse, odt, kind, q, pool, layer, tab, lens, seqs, scale, window, rope):
    """Every row against the restatement, within the tolerance derived above."""
    out, lse = f64(out), f64(lse)
    B, Hq, D = q.shape
    H = pool.heads
    for b in range(B):
        s = seqs[b]
        L = lens[s]
        k, v = cache_rows(pool, layer, tab[s], L)
        row = None if rope is None or L == 0 else rope[L - 1]
        want, wl = ref.attend(q[b], k, v, scale, window, row)
        if L == 0:
            assert np.all(out[b] == 0) and np.all(lse[b] == -np.inf)
            continue
        lo = max(0, L - window) if window else 0
        qa = np.abs(ref.rotate64(q[b][None], row[None])[0]) if row is not None else np.abs(q[b])
        qa = np.maximum(qa, np.abs(q[b]))
        for h in range(Hq):
            kv = h // (Hq // H)
            mass = (np.abs(k[lo:, kv]) @ qa[h]).max() * abs(scale)
            dx = mass * (SPLIT[kind] + (D + 8) * 2.0 ** -23)
            vm = np.abs(v[lo:, kv]).max()
            n = L - lo
            tol = vm * (3 * dx + SPLIT[kind] + 2.0 ** -20 + (n / 8 + 64) * 2.0 ** -23)
            tol = tol + np.abs(want[h]) * ULP[odt] + 2.0 ** -25 * (odt != "f32")
            err = np.abs(out[b, h] - want[h])
            assert np.all(err <= tol), (b, h, L, float((err / tol).max()))
            ltol = dx + 2.0 ** -20 + np.abs(wl[h]) * 2.0 ** -22 + n / 8 * 2.0 ** -23
            assert abs(lse[b, h] - wl[h]) <= ltol, (b, h, L, lse[b, h], wl[h])


def attend_case(qpg, kind, H, G, D, T, lens, qdt="f32", odt="f32", window=0, rope=False, seqs=None, layers=1, layer=0,
                page_pad=0, scale=None, seed=0, qscale=2.0, poison=False):
    pages = pages_for(lens, T)
    pool = make_pool(qpg, kind, layers, pages, H, T, D, seed, page_pad, poison)
    tab, tables = make_tables(qpg, lens, T, pages, seed + 1)
    if poison:                                              # real values only where tokens are
        clean = make_pool(qpg, kind, layers, pages, H, T, D, seed, page_pad)
        for s, n in enumerate(lens):
            for c in range(-(-n // T)):
                p, r = int(tab[s, c]), min(T, n - c * T)
                for a, b in ((pool.k, clean.k), (pool.v, clean.v), (pool.k_scales, clean.k_scales),
                             (pool.v_scales, clean.v_scales)):
                    if a is not None:
                        a[:, p, :, :r] = b[:, p, :, :r]
    idx = list(range(len(lens))) if seqs is None else seqs
    B = len(idx)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 2)
    q = (torch.empty((B, H * G, D), device="cuda").normal_(generator=g) * qscale).to(DT[qdt])
    table = rope_table(max(max(lens), 1), D, seed) if rope else None
    out = torch.full((B, H * G, D), 7.0, dtype=DT[odt], device="cuda")
    lse = torch.full((B, H * G), 7.0, dtype=torch.float32, device="cuda")
    ws = qpg.alloc_kv_workspace(pool, B, H * G)
    for _ in range(2):                                      # the second call finds the workspace as the first left it
        qpg.qpack_kv_attend(pool, layer, tables, q, scale=scale, window=window, out=out, lse=lse, workspace=ws,
                            seqs=None if seqs is None else torch.tensor(seqs, dtype=torch.int32, device="cuda"),
                            rope=None if table is None else torch.from_numpy(table).cuda())
        first = out.clone() if _ == 0 else first
    torch.cuda.synchronize()
    assert qpg.qpack_fetch_fault_flags() == 0
    assert torch.equal(first, out), "the same call twice differs"
    check_attend(out, lse, odt, kind, f64(q), pool, layer, tab, lens, idx, D ** -0.5 if scale is None else scale, window,
                 table)
    return out


@pytest.mark.parametrize("kind", ["i8", "f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 3, 4, 8, 11, 17])
def test_attend_kinds(qpg, kind, D, G):
    """Every cache type, width and group of query heads, at lengths around the tiles' edges, an empty row among them."""
    attend_case(qpg, kind, 2, G, D, 16, [1, 0, 15, 16, 17, 33, 250, 129], seed=D + G)


@pytest.mark.parametrize("T", [1, 2, 8, 16, 64, 1024])
@pytest.mark.parametrize("kind", ["i8", "bf16"])
def test_attend_page_sizes(qpg, kind, T):
    """Pages that end inside a tile, and tiles that end inside a page."""
    attend_case(qpg, kind, 3, 5, 128, T, [1, 7, 31, 32, 100, 513, 1024, 1025], seed=T)


@pytest.mark.parametrize("qdt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("odt", ["f32", "f16", "bf16"])
def test_attend_types_and_rotation(qpg, qdt, odt):
    for kind in ("i8", "f16", "bf16"):
        attend_case(qpg, kind, 2, 4, 128, 32, [1, 63, 200], qdt=qdt, odt=odt, rope=True, seed=5)
    attend_case(qpg, "i8", 1, 7, 64, 32, [65], qdt=qdt, odt=odt, rope=True, seed=6)
    attend_case(qpg, "i8", 1, 7, 256, 32, [65], qdt=qdt, odt=odt, rope=True, seed=7)


@pytest.mark.parametrize("window", [1, 15, 16, 64, 100, 5000])
def test_attend_window(qpg, window):
    attend_case(qpg, "i8", 2, 4, 128, 16, [1, 15, 16, 64, 99, 100, 101, 1000], window=window, seed=window)
    attend_case(qpg, "bf16", 2, 3, 64, 32, [1, 64, 1000, 0], window=window, rope=True, seed=window)


@pytest.mark.parametrize("kind", ["i8", "f16", "bf16"])
def test_attend_poisoned_slots(qpg, kind):
    """NaN, infinities and the type's lowest value in every slot that holds no token, in and behind the last page."""
    attend_case(qpg, kind, 2, 4, 128, 16, [1, 5, 16, 31, 77], poison=True, seed=1)
    attend_case(qpg, kind, 2, 9, 64, 64, [1, 63, 64, 65], poison=True, seed=2)


@pytest.mark.parametrize("lens,H,G,D,T", [([20001], 8, 4, 128, 128), ([70000], 1, 8, 64, 64), ([9999, 3, 0, 1200], 4, 4, 128, 64),
                                          ([4097] * 9, 8, 8, 128, 16), ([300] * 150, 5, 2, 64, 32)])
@pytest.mark.parametrize("kind", ["i8", "bf16"])
def test_attend_split(qpg, lens, H, G, D, T, kind):
    """Long lengths split over many blocks and joined; many rows, with block boundaries inside rows."""
    attend_case(qpg, kind, H, G, D, T, lens, seed=3)


def test_attend_sequences_layers_strides(qpg):
    """Rows that take chosen sequences, a middle layer, pages with gaps between them, an own scale."""
    attend_case(qpg, "i8", 2, 4, 128, 16, [40, 7, 0, 100, 3], seqs=[3, 0, 2, 3, 1, 4, 4], layers=3, layer=1, page_pad=2,
                scale=0.3, seed=8)
    attend_case(qpg, "f16", 2, 4, 64, 16, [40, 7, 0, 100, 3], seqs=[4, 3], layers=3, layer=2, page_pad=1, scale=-0.1, seed=9)


@pytest.mark.parametrize("qscale", [1e-30, 1e-6, 60.0, 1e6, 1e30])
def test_attend_query_magnitudes(qpg, qscale):
    """fp32 queries far outside fp16's range: the softmax goes from uniform to a single token."""
    attend_case(qpg, "i8", 2, 4, 128, 16, [50, 1], qscale=qscale, scale=min(1.0, 5.0 / qscale) if qscale > 60 else None, seed=4)


def test_attend_scale_zero(qpg):
    """A scale of 0 (or one that vanishes beside the queries) gives the mean of the values, masked tokens left out."""
    for kind in ("i8", "f16", "bf16"):
        attend_case(qpg, kind, 2, 4, 128, 16, [1, 5, 16, 77, 0], scale=0.0, seed=11)
        attend_case(qpg, kind, 2, 4, 64, 16, [1, 5, 16, 77, 0], scale=0.0, window=3, poison=True, seed=12)
    attend_case(qpg, "i8", 2, 9, 128, 16, [33, 2], scale=1e-38, qscale=1e-30, seed=13)


@pytest.mark.parametrize("H,G,B", [(1, 2, 2300), (40, 1, 700)])
def test_attend_many_rows(qpg, H, G, B):
    """More rows than one launch takes (by their number, and by rows times heads), some empty, chosen in any order."""
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(0, 70, 300)]
    attend_case(qpg, "i8", H, G, 64, 16, lens, seqs=[int(x) for x in rng.integers(0, 300, B)], seed=B)


def test_rotation_table_too_short(qpg):
    """Positions behind the rotation table are left unrotated and reported; the others are not touched by it."""
    lens, D = [10, 40], 64
    pool = make_pool(qpg, "f16", 1, 5, 1, 16, D, 1)
    tab, tables = make_tables(qpg, lens, 16, 5, 2)
    rope = torch.from_numpy(rope_table(20, D)).cuda()
    q = torch.randn((2, 4, D), device="cuda")
    full = torch.cat([rope, torch.cat([torch.ones((20, D // 2)), torch.zeros((20, D // 2))], 1).cuda()])
    want = qpg.qpack_kv_attend(pool, 0, tables, q, rope=full)
    assert qpg.qpack_fetch_fault_flags() == 0
    assert torch.equal(qpg.qpack_kv_attend(pool, 0, tables, q, rope=rope), want)
    assert qpg.qpack_fetch_fault_flags() == qpg.FAULT_PAGE
    x = torch.randn((2, 1, D), device="cuda")
    qpg.qpack_kv_append(pool, 0, tables, x, x, rope=rope)
    assert qpg.qpack_fetch_fault_flags() == qpg.FAULT_PAGE
    k, _ = qpg.qpack_kv_read(pool, 0, tables, n=2)
    x32 = x.cpu().numpy()
    assert np.array_equal(f64(k)[0], ref.rotate32(x32[:1], rope_table(20, D)[9:10])[0].astype(np.float16).astype(np.float64))
    assert np.array_equal(f64(k)[1], x32[1].astype(np.float16).astype(np.float64))


def test_attend_strided_rows(qpg):
    """q and out as slices of wider rows (a fused projection's output), 2-D and 3-D."""
    lens, H, G, D, T = [30, 75, 2], 2, 4, 64, 16
    pool = make_pool(qpg, "i8", 1, pages_for(lens, T), H, T, D, 1)
    tab, tables = make_tables(qpg, lens, T, pages_for(lens, T), 2)
    wide = torch.randn((3, H * G * D + 2 * H * D), device="cuda")
    q = wide[:, :H * G * D]
    outw = torch.zeros((3, H * G * D + 64), dtype=torch.float16, device="cuda")
    a = qpg.qpack_kv_attend(pool, 0, tables, q, out=outw[:, :H * G * D])
    b = qpg.qpack_kv_attend(pool, 0, tables, q.reshape(3, H * G, D).contiguous())
    assert torch.equal(a.reshape(3, H * G, D), b) and torch.all(outw[:, H * G * D:] == 0)
    assert qpg.qpack_fetch_fault_flags() == 0


def test_attend_other_stream(qpg):
    lens = [777, 10]
    pool = make_pool(qpg, "i8", 1, pages_for(lens, 16), 2, 16, 128, 1)
    tab, tables = make_tables(qpg, lens, 16, pages_for(lens, 16), 2)
    q = torch.randn((2, 8, 128), device="cuda")
    want = qpg.qpack_kv_attend(pool, 0, tables, q)
    s = torch.cuda.Stream()
    out, ws = torch.zeros_like(want), qpg.alloc_kv_workspace(pool, 2, 8)
    torch.cuda.synchronize()
    qpg.qpack_kv_attend(pool, 0, tables, q, out=out, workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(out, want)


def test_attend_in_a_graph(qpg):
    """Captured once, replayed after the lengths and the tables changed."""
    lens = [100, 33]
    pool = make_pool(qpg, "i8", 1, 40, 2, 16, 128, 1)
    tab, tables = make_tables(qpg, lens, 16, 40, 2, extra=8)
    q, out = torch.randn((2, 8, 128), device="cuda"), torch.zeros((2, 8, 128), device="cuda")
    lse, ws = torch.zeros((2, 8), device="cuda"), qpg.alloc_kv_workspace(pool, 2, 8)
    call = lambda: qpg.qpack_kv_attend(pool, 0, tables, q, out=out, lse=lse, workspace=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    new = [3, 200]
    used = set(tab[tab >= 0].tolist())
    free = [p for p in range(40) if p not in used]
    tab[1, 3:13] = free[:10]
    tables.tables.copy_(torch.from_numpy(tab))
    tables.lens.copy_(torch.tensor(new, dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    check_attend(out, lse, "f32", "i8", f64(q), pool, 0, tab, new, [0, 1], 128 ** -0.5, 0, None)


def test_attend_long_cache_offsets(qpg):
    """A pool whose element offsets pass 32 bits: pages past 2^31 and 2^32 elements."""
    T, H, D = 64, 8, 128
    pages = (1 << 32) // (T * H * D) + 70
    k = torch.zeros((1, pages, H, T, D), dtype=torch.int8, device="cuda")
    v = torch.zeros_like(k)
    ks = torch.zeros((1, pages, H, T, D // 32), dtype=torch.float16, device="cuda")
    vs = torch.zeros_like(ks)
    pool = qpg.KVPool(k, v, ks, vs)
    ids = [pages - 1, (1 << 31) // (T * H * D), pages - 7, (1 << 32) // (T * H * D)]
    for c in (k, v):
        c[0, ids] = torch.randint(-127, 128, (4, H, T, D), dtype=torch.int8, device="cuda")
    for s in (ks, vs):
        s[0, ids] = 0.02
    tab = np.array([ids], np.int32)
    tables = qpg.KVTables(torch.from_numpy(tab).cuda(), torch.tensor([250], dtype=torch.int32, device="cuda"))
    q = torch.randn((1, 32, D), device="cuda")
    lse = torch.zeros((1, 32), device="cuda")
    out = qpg.qpack_kv_attend(pool, 0, tables, q, lse=lse, out=torch.zeros((1, 32, D), device="cuda"))
    assert qpg.qpack_fetch_fault_flags() == 0
    check_attend(out, lse, "f32", "i8", f64(q), pool, 0, tab, [250], [0], D ** -0.5, 0, None)
    new = torch.randn((1, H, D), device="cuda")
    qpg.qpack_kv_append(pool, 0, tables, new, new, pos=torch.tensor([249], dtype=torch.int32, device="cuda"))
    kr, vr = qpg.qpack_kv_read(pool, 0, tables, pos=torch.tensor([249], dtype=torch.int32, device="cuda"))
    qc, qs = ref.quantize32(new.cpu().numpy())
    assert np.array_equal(f64(kr), ref.values(qc, qs)) and np.array_equal(f64(vr), ref.values(qc, qs))


def test_attend_out_of_range_tables(qpg):
    """Page numbers, lengths and sequence numbers out of range are reported, never followed; other rows keep their
    results."""
    lens, T = [40, 40, 20], 16
    pool = make_pool(qpg, "i8", 1, 12, 2, T, 64, 1)
    tab, tables = make_tables(qpg, lens, T, 12, 2, extra=0)
    q = torch.randn((3, 4, 64), device="cuda")
    want = qpg.qpack_kv_attend(pool, 0, tables, q)
    torch.cuda.synchronize()
    assert qpg.qpack_fetch_fault_flags() == 0
    for bad in (12, -1, 2 ** 31 - 1, -2 ** 31):
        t2 = tab.copy()
        t2[1, 1] = bad
        tables.tables.copy_(torch.from_numpy(t2))
        got = qpg.qpack_kv_attend(pool, 0, tables, q)
        assert torch.equal(got[[0, 2]], want[[0, 2]])
        assert qpg.qpack_fetch_fault_flags() == qpg.FAULT_PAGE
    tables.tables.copy_(torch.from_numpy(tab))
    for bad in (-5, 49, 2 ** 31 - 1):
        tables.lens.copy_(torch.tensor([40, bad, 20], dtype=torch.int32))
        got = qpg.qpack_kv_attend(pool, 0, tables, q)
        assert torch.equal(got[[0, 2]], want[[0, 2]])
        assert qpg.qpack_fetch_fault_flags() == qpg.FAULT_PAGE
    tables.lens.copy_(torch.tensor(lens, dtype=torch.int32))
    got = qpg.qpack_kv_attend(pool, 0, tables, q, seqs=torch.tensor([0, 3, 2], dtype=torch.int32, device="cuda"))
    assert torch.equal(got[[0, 2]], want[[0, 2]]) and torch.all(got[1] == 0)
    assert qpg.qpack_fetch_fault_flags() == qpg.FAULT_PAGE


def test_attend_nonfinite_row_stays_alone(qpg):
    """An infinite or NaN query gives NaN in its own head; the others keep their results."""
    lens = [40, 30]
    pool = make_pool(qpg, "i8", 1, 8, 2, 16, 64, 1)
    tab, tables = make_tables(qpg, lens, 16, 8, 2)
    q = torch.randn((2, 8, 64), device="cuda")
    want = qpg.qpack_kv_attend(pool, 0, tables, q)
    for bad in (float("nan"), float("inf")):
        q2 = q.clone()
        q2[0, 2, 5] = bad
        got = qpg.qpack_kv_attend(pool, 0, tables, q2)
        assert torch.all(torch.isnan(got[0, 2]))
        keep = torch.ones((2, 8), dtype=torch.bool)
        keep[0, 2] = False
        assert torch.equal(got[keep.cuda()], want[keep.cuda()])


# ---------------------------------------------------------------------------------------------------------------
# append, read
# ---------------------------------------------------------------------------------------------------------------
def append_case(qpg, kind, xdt, H, D, T, lens, rope, seed, page_pad=0, layers=1, layer=0, ld_pad=0):
    """Append a shuffled selection of places; every other byte of the pool stays as it was."""
    rng = np.random.default_rng(seed)
    pages = pages_for(lens, T)
    pool = make_pool(qpg, kind, layers, pages, H, T, D, seed, page_pad)
    tab, tables = make_tables(qpg, lens, T, pages, seed)
    places = [(s, p) for s, n in enumerate(lens) for p in range(n)]
    rng.shuffle(places)
    places = places[:max(1, len(places) * 2 // 3)]
    n = len(places)
    seqs, pos = (torch.tensor([x[i] for x in places], dtype=torch.int32, device="cuda") for i in (0, 1))
    wide = (torch.randn((2, n, H * D + ld_pad), device="cuda") * torch.exp(3 * torch.randn((2, n, 1), device="cuda"))).to(DT[xdt])
    k, v = wide[0, :, :H * D], wide[1, :, :H * D]
    table = rope_table(max(lens), D, seed) if rope else None
    before = [None if t is None else t.clone() for t in (pool.k, pool.v, pool.k_scales, pool.v_scales)]
    qpg.qpack_kv_append(pool, layer, tables, k, v, seqs=seqs, pos=pos, rope=None if table is None else torch.from_numpy(table).cuda())
    got = {}
    got["k"], got["v"] = qpg.qpack_kv_read(pool, layer, tables, seqs, pos)
    torch.cuda.synchronize()
    assert qpg.qpack_fetch_fault_flags() == 0
    page = torch.from_numpy(tab[[s for s, _ in places], [p // T for _, p in places]]).long().cuda()
    slot = torch.tensor([p % T for _, p in places], device="cuda")
    after = [pool.k, pool.v, pool.k_scales, pool.v_scales]
    for name, x, c in (("k", k, 0), ("v", v, 1)):
        x32 = x.float().cpu().numpy().reshape(n, H, D)
        fine = np.isfinite(x32).all((1, 2))                 # what fp16 could not hold is infinite: its codes are unspecified
        assert fine.mean() > 0.9
        x32 = x32[fine]
        new, formula = x32, x32.astype(np.float64)
        if name == "k" and rope:
            rows = table[[p for _, p in places]][fine]
            new, formula = ref.rotate32(x32, rows), ref.rotate64(x32.astype(np.float64), rows)
            # three roundings of terms no larger than the pair's norm
            pair = np.hypot(x32[..., :D // 2], x32[..., D // 2:]).astype(np.float64)
            assert np.all(np.abs(new - formula) <= 3 * 2.0 ** -24 * 2 ** 0.5 * np.concatenate([pair, pair], 2) + 1e-45)
        if kind == "i8":
            codes, scales = ref.quantize32(new)
            assert np.array_equal(after[c][layer][page, :, slot].cpu().numpy()[fine], codes), "codes"
            assert np.array_equal(after[c + 2][layer][page, :, slot].cpu().numpy()[fine].view(np.uint16), scales.view(np.uint16))
            want = ref.values(codes, scales)
        else:
            with np.errstate(over="ignore"):
                want = (new.astype(np.float16) if kind == "f16" else ref.bf16(new)).astype(np.float64)
            assert np.array_equal(f64(after[c][layer][page, :, slot])[fine], want)
        assert np.array_equal(f64(got[name])[fine], want)
        before[c][layer][page, :, slot] = after[c][layer][page, :, slot]
        if kind == "i8":
            before[c + 2][layer][page, :, slot] = after[c + 2][layer][page, :, slot]
    for a, b in zip(after, before):
        if a is not None:
            # bytes: 16-bit patterns and codes alike
            w = torch.int16 if a.element_size() == 2 else torch.int8
            assert torch.equal(a.contiguous().view(w), b.contiguous().view(w)), "a byte outside the appended tokens changed"


@pytest.mark.parametrize("kind", ["i8", "f16", "bf16"])
@pytest.mark.parametrize("xdt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_append(qpg, kind, xdt, D):
    append_case(qpg, kind, xdt, 3, D, 16, [1, 40, 17], rope=True, seed=D)
    append_case(qpg, kind, xdt, 1, D, 8, [1], rope=False, seed=D + 1)


def test_append_sizes_and_strides(qpg):
    append_case(qpg, "i8", "f32", 8, 128, 64, [5, 700, 64], rope=True, seed=1, page_pad=1, layers=2, layer=1, ld_pad=40)
    append_case(qpg, "i8", "f16", 5, 128, 1, [33, 2], rope=False, seed=2, ld_pad=8)
    append_case(qpg, "bf16", "bf16", 32, 64, 128, [300, 1], rope=True, seed=3, page_pad=2)
    append_case(qpg, "i8", "f16", 8, 128, 64, [4000, 5000], rope=True, seed=4)


def test_append_matches_flat_quantizer(qpg, orc):
    """fp16 rows without rotation give the codes and scales of the flat 8-bit quantizer, on and next to its rounding
    boundaries, down to subnormal scales."""
    H, D, n = 2, 128, 512
    rng = np.random.default_rng(9)
    m = np.exp(rng.uniform(np.log(1e-6), np.log(6e4), (n * H * D // 32, 1))).astype(np.float16)
    d = (m.astype(np.float32) / np.float32(127)).astype(np.float16).astype(np.float64)
    x = ((rng.integers(-127, 127, (m.shape[0], 31)) + 0.5) * d).astype(np.float16)
    x = np.concatenate([m, x], 1).reshape(n, H, D)
    x[3] = 0
    pool = make_pool(qpg, "i8", 1, 33, H, 16, D, 1)
    _, tables = make_tables(qpg, [n], 16, 33, 2)
    t = torch.from_numpy(x).cuda()
    seqs, pos = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda")
    qpg.qpack_kv_append(pool, 0, tables, t, t, seqs=seqs, pos=pos)
    kr, vr = qpg.qpack_kv_read(pool, 0, tables, seqs, pos)
    rq, rs = orc.kv_quantize(x.view(np.uint16).reshape(-1))
    want = orc.kv_dequant(rq, rs).reshape(-1)
    assert np.array_equal(kr.cpu().numpy().view(np.uint16).reshape(-1), want)
    assert np.array_equal(vr.cpu().numpy().view(np.uint16).reshape(-1), want)


def test_append_defaults_skips_and_reports(qpg):
    """Default sequence and position, skipped tokens, places out of range: nothing else is written."""
    T, H, D = 16, 2, 64
    lens = [5, 0, 33]
    pool = make_pool(qpg, "i8", 1, 8, H, T, D, 1)
    tab, tables = make_tables(qpg, lens, T, 8, 2, extra=0)
    x = torch.randn((3, H, D), device="cuda")
    before = pool.k.clone()
    qpg.qpack_kv_append(pool, 0, tables, x, x)             # sequence 1 is empty: its token is skipped
    assert qpg.qpack_fetch_fault_flags() == 0
    k, v = qpg.qpack_kv_read(pool, 0, tables, n=3)
    want = ref.values(*ref.quantize32(x.cpu().numpy()))
    want[1] = 0
    assert np.array_equal(f64(k), want) and np.array_equal(f64(v), want)
    for s, p in ((0, 4), (2, 32)):
        before[0, tab[s, p // T], :, p % T] = pool.k[0, tab[s, p // T], :, p % T]
    assert torch.equal(before, pool.k)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    for seqs, pos in ((i32(0, 3, 2), i32(-1, 0, -1)), (i32(-1, 0, 0), i32(3, -1, -2)), (i32(0, 0, 0), i32(-1, 48, 2 ** 31 - 1)),
                      (i32(0, 0, 0), i32(-1, 17, -1))):
        qpg.qpack_kv_append(pool, 0, tables, x, x, seqs=seqs, pos=pos)
        assert qpg.qpack_fetch_fault_flags() == qpg.FAULT_PAGE
        assert torch.equal(before, pool.k)
        k, _ = qpg.qpack_kv_read(pool, 0, tables, seqs, pos)
        assert torch.all(k == 0) and qpg.qpack_fetch_fault_flags() == qpg.FAULT_PAGE
    only, none = qpg.qpack_kv_read(pool, 0, tables, k_out=torch.zeros((3, H, D), device="cuda"))
    assert none is None and np.array_equal(f64(only), want)


# ---------------------------------------------------------------------------------------------------------------
# page operators
# ---------------------------------------------------------------------------------------------------------------
def token_view(pool):
    """Pool contents as bytes [pages, tokens, everything else]."""
    parts = []
    for t in (pool.k, pool.v, pool.k_scales, pool.v_scales):
        if t is not None:
            b = t.contiguous().view(torch.int8)             # [L, P, H, T, bytes]
            parts.append(b.permute(1, 3, 0, 2, 4).reshape(t.shape[1], t.shape[3], -1).cpu().numpy())
    return np.concatenate(parts, 2)


def same_state(qpg, pool, tables, sim):
    torch.cuda.synchronize()
    assert tables.lens.cpu().tolist() == sim.lens
    assert tables.tables.cpu().tolist() == sim.tables
    assert tables.refs.cpu().tolist() == sim.refs
    assert np.array_equal(token_view(pool), sim.pool)
    flags = qpg.qpack_fetch_fault_flags()
    assert flags == (qpg.FAULT_NO_PAGES if sim.refused else 0)
    sim.refused = False


@pytest.mark.parametrize("kind,layers,H,T,D,P,S,MP,pad", [("i8", 2, 2, 16, 128, 40, 9, 6, 0), ("f16", 1, 3, 4, 64, 1500, 70, 40, 0),
                                                          ("bf16", 3, 1, 8, 256, 25, 7, 12, 1), ("i8", 1, 5, 1, 64, 90, 12, 30, 2),
                                                          ("i8", 2, 1, 2, 64, 2500, 300, 20, 0)])
def test_page_operators_random_walk(qpg, kind, layers, H, T, D, P, S, MP, pad):
    """A seeded walk of reserve, fork, free and compact, refusals among it, against the lists; pool contents included."""
    rng = np.random.default_rng(P + S)
    pool = make_pool(qpg, kind, layers, P, H, T, D, 1, pad)
    tables = qpg.alloc_kv_tables(S, MP, P)
    ws = qpg.alloc_kv_page_workspace(pool, tables)
    sim = ref.Pages(S, MP, P, T, token_view(pool))
    i32 = lambda a: torch.tensor(list(a), dtype=torch.int32, device="cuda")  # noqa: E731
    for step in range(30):
        op = rng.choice(["reserve", "reserve", "fork", "free", "compact"])
        ids = rng.permutation(S)
        if op == "reserve":
            n = int(rng.integers(1, S + 1))
            seqs, add = ids[:n].tolist(), rng.integers(0, 3 * T + 2, n).tolist()
            seqs = [-1 if rng.random() < 0.1 else s for s in seqs]
            qpg.qpack_kv_reserve(pool, tables, i32(seqs), i32(add))
            sim.reserve(seqs, add)
        elif op == "fork":
            empty = [int(s) for s in ids if sim.lens[s] == 0]
            full = [int(s) for s in ids if sim.lens[s]]
            dst = empty[:int(rng.integers(0, 6))] + (full[:1] if rng.random() < 0.2 and len(full) > 2 else [])
            parents = [s for s in full if s not in dst]
            if not dst or not parents:
                continue
            src = [parents[int(rng.integers(0, min(3, len(parents))))] for _ in dst]
            qpg.qpack_kv_fork(pool, tables, i32(src), i32(dst), workspace=ws)
            sim.fork(src, dst)
        elif op == "free":
            seqs = [int(s) for s in ids[:int(rng.integers(1, max(2, S // 2)))]]
            qpg.qpack_kv_free(tables, i32(seqs + [-1]))
            sim.free(seqs)
        else:
            moved = torch.zeros(1, dtype=torch.int32, device="cuda")
            live = [p for p in range(P) if sim.refs[p] > 0]
            qpg.qpack_kv_compact(pool, tables, moved=moved, workspace=ws)
            assert sim.compact() == int(moved)
            # pages that are no longer live keep what they held; the operator does not say what: compare live ones
            assert len(live) == sum(r > 0 for r in sim.refs)
        same_state(qpg, pool, tables, sim)


def test_page_operators_many_pages(qpg):
    """More pages than one pass of the planning blocks ranks, and free pages that lie behind the first pass."""
    P, S, MP, T = 20011, 40, 900, 1
    pool = make_pool(qpg, "i8", 1, P, 1, T, 64, 1)
    tables = qpg.alloc_kv_tables(S, MP, P)
    ws = qpg.alloc_kv_page_workspace(pool, tables)
    sim = ref.Pages(S, MP, P, T, token_view(pool))
    i32 = lambda a: torch.tensor(list(a), dtype=torch.int32, device="cuda")  # noqa: E731
    rng = np.random.default_rng(3)
    for step in range(4):
        seqs, add = list(range(S)), rng.integers(0, 400, S).tolist()
        qpg.qpack_kv_reserve(pool, tables, i32(seqs), i32(add))
        sim.reserve(seqs, add)
        same_state(qpg, pool, tables, sim)
        gone = rng.permutation(S)[:S // 3].tolist()
        qpg.qpack_kv_free(tables, i32(gone))
        sim.free(gone)
        parents = [s for s in range(S) if s not in gone]
        src, dst = [parents[i % 5] for i in range(len(gone))], gone
        qpg.qpack_kv_fork(pool, tables, i32(src), i32(dst), workspace=ws)
        sim.fork(src, dst)
        same_state(qpg, pool, tables, sim)
    qpg.qpack_kv_free(tables, i32(range(0, S, 2)))
    sim.free(range(0, S, 2))
    moved = torch.zeros(1, dtype=torch.int32, device="cuda")
    qpg.qpack_kv_compact(pool, tables, moved=moved, workspace=ws)
    assert sim.compact() == int(moved) > 0
    same_state(qpg, pool, tables, sim)
    qpg.qpack_kv_reserve(pool, tables, i32([0]), i32([MP]))  # and from behind the live pages
    sim.reserve([0], [MP])
    same_state(qpg, pool, tables, sim)


def test_compact_out_of_place(qpg):
    pool = make_pool(qpg, "f16", 2, 30, 2, 8, 64, 1)
    refs = torch.zeros(30, dtype=torch.int32, device="cuda")
    live = [29, 3, 17, 0, 21]
    refs[live] = torch.tensor([1, 2, 1, 3, 1], dtype=torch.int32, device="cuda")
    tab = torch.tensor([[29, 3, 17, -1], [0, 21, 3, -1]], dtype=torch.int32, device="cuda")
    tables = qpg.KVTables(tab, torch.tensor([24, 24], dtype=torch.int32, device="cuda"), refs)
    t2, r2 = torch.empty_like(tab), torch.empty_like(refs)
    old = pool.k.clone()
    qpg.qpack_kv_compact(pool, tables, tables_out=t2, refs_out=r2)
    assert t2.tolist() == [[4, 3, 1, -1], [0, 2, 3, -1]] and r2[:5].tolist() == [3, 1, 1, 2, 1] and int(r2[5:].sum()) == 0
    assert tab.tolist()[0][0] == 29 and int(refs[29]) == 1          # the inputs stand
    assert torch.equal(pool.k[:, 1], old[:, 17]) and torch.equal(pool.k[:, 2], old[:, 21]) and torch.equal(pool.k[:, 4], old[:, 29])
    assert qpg.qpack_fetch_fault_flags() == 0


def test_copy_pages(qpg):
    for kind in ("i8", "bf16"):
        pool = make_pool(qpg, kind, 3, 20, 3, 16, 64, 1, page_pad=1)
        want = token_view(pool)
        src, dst = [0, 5, 5, 19], [3, 1, 18, 2]
        qpg.qpack_kv_copy_pages(pool, *(torch.tensor(x, dtype=torch.int32, device="cuda") for x in (src, dst)))
        want[dst] = want[src]
        assert np.array_equal(token_view(pool), want) and qpg.qpack_fetch_fault_flags() == 0
        qpg.qpack_kv_copy_pages(pool, *(torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([20, 1, -1], [4, -1, 6])))
        assert np.array_equal(token_view(pool), want) and qpg.qpack_fetch_fault_flags() == qpg.FAULT_PAGE


def test_free_listed_twice_and_out_of_range(qpg):
    pool = make_pool(qpg, "f16", 1, 10, 1, 8, 64, 1)
    tables = qpg.alloc_kv_tables(3, 4, 10)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    qpg.qpack_kv_reserve(pool, tables, i32(0, 1, 7), i32(20, 8, 3))
    assert qpg.qpack_fetch_fault_flags() == qpg.FAULT_PAGE
    qpg.qpack_kv_fork(pool, tables, i32(0, 9), i32(2, 1))
    assert qpg.qpack_fetch_fault_flags() == qpg.FAULT_PAGE
    qpg.qpack_kv_free(tables, i32(0, 0, 1, 5, -1))
    assert qpg.qpack_fetch_fault_flags() == qpg.FAULT_PAGE
    torch.cuda.synchronize()
    assert tables.lens.tolist() == [0, 0, 20] and int(tables.refs.sum()) == 3 and int(tables.refs.min()) == 0
