"""GPU tests of the paged KV cache at the limits of its types and of its arguments."""
import numpy as np
import pytest
import torch

from oracle import paged as ref
from test_gpu_paged import DT, cache_rows, check_attend, f64, make_pool, make_tables, pages_for, rope_table, same_state, token_view

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


@pytest.mark.parametrize("what", ["values", "keys", "small keys"])
@pytest.mark.parametrize("D,G", [(64, 3), (64, 16), (128, 4), (128, 11), (256, 2)])
def test_attend_bf16_magnitudes(qpg, what, D, G):
    """A bf16 cache has fp32's range: values of 2^116, keys of 2^112 beside queries of 2^-112 and the other way round give
    what they give in fp32."""
    T, H, lens = 16, 2, [1, 33, 700, 5000]
    pages = pages_for(lens, T)
    pool = make_pool(qpg, "bf16", 1, pages, H, T, D, 11)
    tab, tables = make_tables(qpg, lens, T, pages, 12)
    q = torch.randn((len(lens), H * G, D), device="cuda")
    if what == "values":
        pool.v.mul_(2.0 ** 116)
    else:
        pool.k.mul_(2.0 ** (112 if what == "keys" else -105))
        q.mul_(2.0 ** (-112 if what == "keys" else 105))
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    qpg.qpack_kv_attend(pool, 0, tables, q, out=out, lse=lse)
    assert qpg.qpack_fetch_fault_flags() == 0
    check_attend(out, lse, "f32", "bf16", f64(q), pool, 0, tab, lens, range(len(lens)), D ** -0.5, 0, None)


@pytest.mark.parametrize("kind", ["i8", "f16", "bf16"])
@pytest.mark.parametrize("D,G,window,rope", [(64, 3, 0, False), (128, 8, 0, True), (128, 11, 300, False), (256, 4, 0, False), (64, 16, 0, True)])
def test_attend_infinite_elements_stay_where_they_are(qpg, kind, D, G, window, rope):
    """A key that is not finite (fp16(scale * code) among them) reaches the heads of its key/value head in its row, a value
    that is not finite its own element of these; all else keeps its bits."""
    T, H, lens = 16, 4, [1, 2, 40, 700, 9000, 33]
    pages = pages_for(lens, T)
    pool = make_pool(qpg, kind, 2, pages, H, T, D, 21)
    tab, tables = make_tables(qpg, lens, T, pages, 22)
    q = torch.randn((len(lens), H * G, D), device="cuda")
    call = dict(window=window, rope=torch.from_numpy(rope_table(max(lens), D, 1)).cuda() if rope else None)
    outs, lses = ([torch.empty(s, device="cuda") for _ in range(2)] for s in (q.shape, q.shape[:2]))
    qpg.qpack_kv_attend(pool, 1, tables, q, out=outs[0], lse=lses[0], **call)
    rng = np.random.default_rng(D + G)
    same, odd = torch.ones(q.shape, dtype=torch.bool), torch.zeros(q.shape, dtype=torch.bool)
    same_lse = torch.ones(q.shape[:2], dtype=torch.bool)
    for s, n in enumerate(lens[:-1]):                       # key/value head 0: a key, 1: a value, 2: both, 3: neither
        for h, what in ((0, "k"), (1, "v"), (2, "kv")):
            for x in what:
                t, d, sign = int(rng.integers(max(0, n - 300), n)), int(rng.integers(0, D)), rng.choice([-1.0, 1.0])
                at, heads = (1, int(tab[s, t // T]), h, t % T), slice(h * G, (h + 1) * G)
                codes, scales = (pool.k, pool.k_scales) if x == "k" else (pool.v, pool.v_scales)
                if kind == "i8":
                    codes[at][d // 32 * 32:d // 32 * 32 + 32] = 0
                    codes[at][d], scales[at][d // 32] = int(127 * sign), 65504.0
                    if x == "v":                            # the group's other values changed too
                        same[s, heads, d // 32 * 32:d // 32 * 32 + 32] = False
                else:
                    codes[at][d] = float(rng.choice(["inf", "nan"])) * sign
                if x == "v":
                    same[s, heads, d], odd[s, heads, d] = False, True
                else:
                    same[s, heads], same_lse[s, heads] = False, False
    for _ in range(2):                                      # the workspace is as it was
        qpg.qpack_kv_attend(pool, 1, tables, q, out=outs[1], lse=lses[1], **call)
    assert qpg.qpack_fetch_fault_flags() == 0
    assert torch.equal(outs[0].cpu()[same], outs[1].cpu()[same]) and torch.equal(lses[0].cpu()[same_lse], lses[1].cpu()[same_lse])
    assert not torch.isfinite(outs[1].cpu()[odd]).any() and torch.isfinite(outs[0]).all()


@pytest.mark.parametrize("kind", ["i8", "f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 8, 11, 16])
def test_attend_scores_keep_the_querys_bits(qpg, kind, D, G):
    """One token whose key is 1 at a single place, every place in turn: the log-sum-exp is that element of the query, to the
    22 bits of two fp16 terms or the 24 of three bfloat16 ones and the roundings of a product by log2 e and one by ln 2 in
    fp32. Two bfloat16 terms (16 bits) would be off by 2^-18 of it on average."""
    pool = make_pool(qpg, kind, 1, D, 1, 1, D, 1)
    pool.k.zero_()
    pool.k[0, torch.arange(D), 0, 0, torch.arange(D)] = 1
    if kind == "i8":
        pool.k_scales.fill_(1.0)
    tables = qpg.KVTables(torch.arange(D, dtype=torch.int32, device="cuda").view(D, 1), torch.ones(D, dtype=torch.int32, device="cuda"))
    g = torch.Generator(device="cuda")
    g.manual_seed(D + G)
    q = torch.empty((D, G, D), device="cuda").uniform_(64, 128, generator=g)
    lse = torch.empty((D, G), device="cuda")
    for scale in (1.0, -1.0):
        qpg.qpack_kv_attend(pool, 0, tables, q, scale=scale, lse=lse)
        want = scale * f64(q)[np.arange(D), :, np.arange(D)]
        tol = 128 * 2.0 ** -22 + 128 * 3 * 2.0 ** -24 + 2.0 ** -19      # a term's last bit, three roundings, the logarithm's
        assert np.all(np.abs(f64(lse) - want) <= tol)
    terms = ref.bf16(want.astype(np.float32))
    two = terms + ref.bf16((want - terms).astype(np.float32))
    assert np.mean(np.abs(two - want) > tol) > 0.5         # what the third term is for
    assert qpg.qpack_fetch_fault_flags() == 0


@pytest.mark.parametrize("kind", ["i8", "f16", "bf16"])
@pytest.mark.parametrize("D,G", [(64, 1), (64, 16), (128, 8), (128, 11), (256, 4)])
def test_attend_fp32_outputs_keep_the_weights_bits(qpg, kind, D, G):
    """Each token's value is 1 at a place of its own, so an fp32 output shows the weights: to the exponential's and the
    division's roundings and to the terms' 22 bits or more, over bf16 caches too (two bfloat16 terms would leave 16)."""
    n, T = 60, 16
    pool = make_pool(qpg, kind, 1, 6, 1, T, D, 1)
    tab, tables = make_tables(qpg, [n], T, 6, 2)
    page, slot = torch.from_numpy(tab[0])[torch.arange(n) // T].long(), torch.arange(n) % T
    for c in (pool.k, pool.v):
        c.zero_()
    if kind == "i8":
        pool.k_scales.fill_(2.0 ** -7), pool.v_scales.fill_(1.0)
    g = torch.Generator()
    g.manual_seed(D + G)
    key = torch.randint(-127, 128, (n,), generator=g)
    pool.k[0, page, 0, slot, 7] = (key.float() * (1 if kind == "i8" else 2.0 ** -7)).to(pool.k.dtype).cuda()
    pool.v[0, page, 0, slot, torch.arange(n)] = 1
    q = torch.zeros((1, G, D), device="cuda")
    q[0, :, 7] = torch.linspace(0.3, 1.5, G)
    out = torch.empty_like(q)
    qpg.qpack_kv_attend(pool, 0, tables, q, scale=1.0, out=out)
    x = f64(q)[0, :, 7, None] * (key.numpy() * 2.0 ** -7)
    e = np.exp(x - x.max(1, keepdims=True))
    want = e / e.sum(1, keepdims=True)
    # scores of at most 1.5: a term's last bit and four roundings, at log2 e; the exponential's 2^-22, the terms' 2^-22, sum and
    # division
    tol = want * (1.5 * 1.443 * (2.0 ** -22 + 4 * 2.0 ** -24) + 2.0 ** -22 + 2.0 ** -22 + 12 * 2.0 ** -24)
    assert np.all(np.abs(f64(out)[0, :, :n] - want) <= tol)
    two = ref.bf16(e.astype(np.float32))
    two = two + ref.bf16((e - two).astype(np.float32)).astype(np.float64)
    assert np.mean(np.abs(two / e.sum(1, keepdims=True) - want) > tol) > 0.1       # what the third term is for
    assert not out[0, :, n:].any() and qpg.qpack_fetch_fault_flags() == 0


# ---------------------------------------------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("xdt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rope", [False, True])
def test_append_saturated_scales(qpg, xdt, D, rope):
    """Groups whose scale ends at fp16's largest number: codes are clamped as the rule says, bit for bit."""
    tops = [8.2e6, 8.319e6, 8.33e6, 8.36e6, 9e6, 1e7, 256 * 65504.0, 257.4 * 65504, 1e9, 2.0 ** 22 * 65504, 2.0 ** 23 * 65504,
            1e12, 1e20, 1e30]
    H, T, n = 3, 16, len(tops)
    rng = np.random.default_rng(D)
    x = rng.uniform(-1, 1, (2, n, H, D)) * np.exp(rng.uniform(-4, 0, (2, n, H, D)))
    x[..., ::32], x[..., 1::32] = 1.0, -1.0                 # every group reaches its magnitude, with both signs
    x = torch.from_numpy(x * np.array(tops)[:, None, None]).float().to(DT[xdt]).cuda()
    pool = make_pool(qpg, "i8", 1, 3, H, T, D, 1)
    tab, tables = make_tables(qpg, [n], T, 3, 2)
    seqs, pos = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda")
    table = rope_table(n, D, 3)
    qpg.qpack_kv_append(pool, 0, tables, x[0], x[1], seqs=seqs, pos=pos, rope=torch.from_numpy(table).cuda() if rope else None)
    page = int(tab[0, 0])
    for c, s, a in ((pool.k, pool.k_scales, x[0]), (pool.v, pool.v_scales, x[1])):
        a = a.float().cpu().numpy()
        if rope and c is pool.k:
            a = ref.rotate32(a, table)
        codes, scales = ref.quantize32(a)
        assert np.array_equal(s[0, page, :, :n].transpose(0, 1).cpu().numpy().view(np.uint16), scales.view(np.uint16))
        assert np.array_equal(c[0, page, :, :n].transpose(0, 1).cpu().numpy(), codes)
    assert qpg.qpack_fetch_fault_flags() == 0


def test_skipped_tokens_of_no_sequence(qpg):
    """A negative position skips a token whatever its sequence number (padding is often -1 in both): nothing is written, nothing
    reported, and reading gives zeros."""
    pool = make_pool(qpg, "i8", 1, 5, 2, 16, 64, 1)
    tab, tables = make_tables(qpg, [20], 16, 5, 2)
    i = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    x, seqs, pos = torch.randn((4, 2, 64), device="cuda"), i(-1, 0, 7, -2 ** 31), i(-1, 3, -5, -2 ** 31)
    before = pool.k.clone()
    qpg.qpack_kv_append(pool, 0, tables, x, x, seqs=seqs, pos=pos)
    k, v = qpg.qpack_kv_read(pool, 0, tables, seqs, pos)
    assert qpg.qpack_fetch_fault_flags() == 0
    want = ref.values(*ref.quantize32(x[1:2].cpu().numpy()))[0]
    for got in (k, v):
        assert np.array_equal(f64(got[1]), want) and not got[[0, 2, 3]].any()
    before[0, int(tab[0, 0]), :, 3] = pool.k[0, int(tab[0, 0]), :, 3]
    assert torch.equal(before, pool.k)


def test_default_position_of_a_negative_length(qpg):
    """A token at the last position of a sequence whose length is negative: left out and reported; of an empty one: skipped."""
    pool = make_pool(qpg, "i8", 1, 5, 2, 16, 64, 1)
    tab, tables = make_tables(qpg, [20, 3], 16, 5, 2)
    x, before = torch.randn((2, 2, 64), device="cuda"), pool.k.clone()
    before[0, int(tab[1, 0]), :, 2] = 0
    for bad, flags in ((0, 0), (-1, 32), (-5, 32), (-2 ** 31, 32)):
        tables.lens[0] = bad
        qpg.qpack_kv_append(pool, 0, tables, x, x)
        assert qpg.qpack_fetch_fault_flags() == flags, bad
        k, v = qpg.qpack_kv_read(pool, 0, tables, n=2)
        assert qpg.qpack_fetch_fault_flags() == flags and not k[0].any() and not v[0].any() and k[1].any()
        after = pool.k.clone()
        after[0, int(tab[1, 0]), :, 2] = 0
        assert torch.equal(after, before)


def test_append_and_attend_at_saturation(qpg):
    """A token whose largest value the 8-bit cache holds as infinite (fp16(65504 * 127)): read back as the rule has it, and
    attention sees it in that element alone, or in its head where it is a key."""
    H, D, T = 2, 128, 16
    pool = make_pool(qpg, "i8", 1, 3, H, T, D, 1)
    _, tables = make_tables(qpg, [3], T, 3, 2)
    k = torch.randn((3, H, D), device="cuda")
    v = torch.randn((3, H, D), device="cuda")
    v[1, 0, 40], k[2, 1, 7] = 9e6, -1e7
    seqs, pos = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.arange(3, dtype=torch.int32, device="cuda")
    qpg.qpack_kv_append(pool, 0, tables, k, v, seqs=seqs, pos=pos)
    kr, vr = qpg.qpack_kv_read(pool, 0, tables, seqs, pos)
    for got, x in ((kr, k), (vr, v)):
        assert np.array_equal(f64(got), ref.values(*ref.quantize32(x.cpu().numpy())))
    assert f64(vr)[1, 0, 40] == np.inf and f64(kr)[2, 1, 7] == -np.inf
    q = torch.randn((1, 2 * H, D), device="cuda")
    out = qpg.qpack_kv_attend(pool, 0, tables, q, out=torch.empty_like(q))
    fine = f64(vr)[:, 0].copy()
    fine[1, 40] = 0
    want, _ = ref.attend(f64(q[0, :2]), f64(kr)[:, :1], fine[:, None], D ** -0.5)
    rest = np.arange(D) != 40
    assert np.allclose(f64(out)[0, :2, rest], want[:, rest].T, rtol=0, atol=2.0 ** -18 * np.abs(fine).max())
    assert not np.isfinite(f64(out)[0, :2, 40]).any() and qpg.qpack_fetch_fault_flags() == 0


# ---------------------------------------------------------------------------------------------------------------
# another stream
# ---------------------------------------------------------------------------------------------------------------
def soil(bytes):
    """Leaves non-zero bytes in what the allocator hands out next on this stream."""
    for n in {bytes, max(bytes // 2, 512)}:
        torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda")


def busy():
    """Keeps the current stream busy for some milliseconds."""
    torch.cuda._sleep(20_000_000)


def test_attend_other_stream_default_workspace(qpg):
    """A call on a stream of the caller's choice, without workspace or output: what it allocates is zeroed, used and
    released in that stream's order, while the current stream is busy and allocates the same sizes."""
    lens = [7777, 10, 3000]
    pages = pages_for(lens, 16)
    pool = make_pool(qpg, "i8", 1, pages, 2, 16, 128, 1)
    _, tables = make_tables(qpg, lens, 16, pages, 2)
    q = torch.randn((3, 8, 128), device="cuda")
    want = qpg.qpack_kv_attend(pool, 0, tables, q)
    size = qpg.alloc_kv_workspace(pool, 3, 8).bytes
    s = torch.cuda.Stream()
    soil(size)
    torch.cuda.synchronize()
    for _ in range(4):
        busy()
        out = qpg.qpack_kv_attend(pool, 0, tables, q, stream=s)
        soil(size)                                          # behind the current stream's work, over what the call gave back
        s.synchronize()
        assert torch.equal(out, want)

    class Handle:                                           # a stream of another library: its handle is all that a launch takes
        cuda_stream = s.cuda_stream
    out = qpg.qpack_kv_attend(pool, 0, tables, q, stream=Handle())
    s.synchronize()
    assert torch.equal(out, want)
    torch.cuda.synchronize()
    assert qpg.qpack_fetch_fault_flags() == 0


def test_read_other_stream_default_outputs(qpg):
    lens = [500]
    pool = make_pool(qpg, "i8", 1, 40, 2, 16, 128, 1)
    _, tables = make_tables(qpg, lens, 16, 40, 2)
    seqs, pos = torch.zeros(500, dtype=torch.int32, device="cuda"), torch.arange(500, dtype=torch.int32, device="cuda")
    want = qpg.qpack_kv_read(pool, 0, tables, seqs, pos)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.full_like(want[0], 3.0)                           # its memory is free again, the fill still to come
    busy()
    torch.full_like(want[0], 3.0)
    got = qpg.qpack_kv_read(pool, 0, tables, seqs, pos, stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_page_operators_other_stream_default_workspace(qpg):
    """Fork and compact on another stream without a workspace: their list of copies is not overwritten by what the current
    stream allocates next."""
    s = torch.cuda.Stream()
    for kind in ("i8", "f16"):
        pool = make_pool(qpg, kind, 4, 600, 2, 16, 128, 1)
        tables = qpg.alloc_kv_tables(60, 20, 600)
        sim = ref.Pages(60, 20, 600, 16, token_view(pool))
        ids = torch.arange(60, dtype=torch.int32, device="cuda")
        seqs, add = list(range(8)), [37, 300, 5, 16, 129, 200, 1, 90]
        qpg.qpack_kv_reserve(pool, tables, ids[:8], torch.tensor(add, dtype=torch.int32, device="cuda"))
        sim.reserve(seqs, add)
        src, dst = [i % 8 for i in range(48)], list(range(8, 56))
        t_src, t_dst, t_gone = ids[:8].repeat(6), ids[8:56], ids[0:40:3].contiguous()
        size = qpg.alloc_kv_page_workspace(pool, tables).bytes
        torch.cuda.synchronize()
        busy()
        qpg.qpack_kv_fork(pool, tables, t_src, t_dst, stream=s)
        soil(size)
        qpg.qpack_kv_free(tables, t_gone, stream=s)
        qpg.qpack_kv_compact(pool, tables, stream=s)
        soil(size)
        sim.fork(src, dst)
        sim.free(range(0, 40, 3))
        assert sim.compact() > 0
        s.synchronize()
        same_state(qpg, pool, tables, sim)


# ---------------------------------------------------------------------------------------------------------------
# fault word
# ---------------------------------------------------------------------------------------------------------------
def test_faults_are_fetched_once(qpg):
    """Every kernel's reports reach the fault word and are gone once they are fetched."""
    for kind in ("i8", "f16", "bf16"):
        pool = make_pool(qpg, kind, 1, 5, 1, 16, 64, 1)
        tab, tables = make_tables(qpg, [20], 16, 5, 2)
        q, bad = torch.randn((1, 2, 64), device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
        qpg.qpack_kv_attend(pool, 0, tables, q, seqs=bad)
        assert [qpg.qpack_fetch_fault_flags() for _ in range(2)] == [qpg.FAULT_PAGE, 0]
        qpg.qpack_kv_attend(pool, 0, tables, q, seqs=bad)
        tables.refs = torch.ones(5, dtype=torch.int32, device="cuda")
        full = qpg.KVTables(tables.tables, tables.lens, tables.refs)
        qpg.qpack_kv_reserve(pool, full, 0 * bad, 16 * bad)
        assert [qpg.qpack_fetch_fault_flags() for _ in range(2)] == [qpg.FAULT_PAGE | qpg.FAULT_NO_PAGES, 0]
        qpg.qpack_kv_attend(pool, 0, tables, q)
        assert qpg.qpack_fetch_fault_flags() == 0


# ---------------------------------------------------------------------------------------------------------------
# page operators
# ---------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("pages", [8, 5000])
def test_reserve_more_pages_than_32_bits_count(qpg, pages):
    """Requests whose pages together pass 2^31 (and 2^32): refused, each without a trace; those before them and those that
    need no page stand."""
    MP = 1 << 30
    pool = make_pool(qpg, "i8", 1, pages, 1, 1, 64, 1)
    tab = torch.empty((6, MP), dtype=torch.int32, device="cuda")
    tab[:, :pages + 8] = -1
    lens = torch.tensor([0, 0, 0, 2, 0, 0], dtype=torch.int32, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    tab[3, :2], refs[:2] = torch.tensor([1, 0], dtype=torch.int32, device="cuda"), 1
    tables = qpg.KVTables(tab, lens, refs)
    seqs = torch.tensor([4, 0, 1, 3, 2, 5], dtype=torch.int32, device="cuda")
    for second in (MP, MP - 5):                             # the sum of the large ones: 2^31, or some less; then past 2^32
        add = torch.tensor([3, MP, second, 0, 7, MP], dtype=torch.int32, device="cuda")
        qpg.qpack_kv_reserve(pool, tables, seqs, add)
        assert qpg.qpack_fetch_fault_flags() == qpg.FAULT_NO_PAGES
        assert lens.tolist() == [0, 0, 0, 2, 3, 0] and refs.tolist() == [1] * 5 + [0] * (pages - 5)
        assert tab[4, :4].tolist() == [2, 3, 4, -1] and tab[3, :3].tolist() == [1, 0, -1]
        assert (tab[[0, 1, 2, 5], :pages + 8] == -1).all()
        qpg.qpack_kv_free(qpg.KVTables(tab[:, :pages], lens, refs), torch.tensor([4], dtype=torch.int32, device="cuda"))
        assert qpg.qpack_fetch_fault_flags() == 0
    big = 4096                                              # as many requests as a call takes, all of one row
    qpg.qpack_kv_reserve(pool, tables, torch.full((big,), -1, dtype=torch.int32, device="cuda"),
                         torch.full((big,), MP, dtype=torch.int32, device="cuda"))
    assert qpg.qpack_fetch_fault_flags() == 0 and lens.tolist() == [0, 0, 0, 2, 0, 0]


def test_reserve_listed_twice_stays_in_its_row(qpg):
    """A sequence listed twice, against the rules, with pages for one request and part of the other: nothing outside its row,
    the reference counts and the lengths is touched."""
    pages, MP, n = 3000, 2000, 600
    pool = make_pool(qpg, "i8", 1, pages, 1, 1, 64, 1)
    for add in ([1200, 1990], [1, 2000] * (n // 2), [5] * n + [1999]):
        tab = torch.full((5, MP), -7, dtype=torch.int32, device="cuda")
        tab[2] = -1
        lens, refs = torch.zeros(5, dtype=torch.int32, device="cuda"), torch.zeros(pages + 64, dtype=torch.int32, device="cuda")
        refs[pages:] = -9
        tables = qpg.KVTables(tab, lens, refs[:pages])
        qpg.qpack_kv_reserve(pool, tables, torch.full((len(add),), 2, dtype=torch.int32, device="cuda"),
                             torch.tensor(add, dtype=torch.int32, device="cuda"))
        assert qpg.qpack_fetch_fault_flags() == qpg.FAULT_NO_PAGES
        assert (tab[[0, 1, 3, 4]] == -7).all() and (refs[pages:] == -9).all()
        assert lens[[0, 1, 3, 4]].tolist() == [0] * 4 and set(refs[:pages].unique().tolist()) <= {0, 1}
        assert ((tab[2] >= -1) & (tab[2] < pages)).all()


def test_page_operators_lengths_out_of_range(qpg):
    """Lengths that are negative or longer than the row: reported, and the request is left out; the others of the call stand."""
    T, MP, pages = 16, 4, 40
    pool = make_pool(qpg, "i8", 2, pages, 1, T, 64, 1)
    for bad in (-1, -2 ** 31, MP * T + 1, 2 ** 31 - 1):
        tables = qpg.alloc_kv_tables(6, MP, pages)
        i = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
        qpg.qpack_kv_reserve(pool, tables, i(0, 1), i(20, 64))
        tables.lens[2] = bad
        before = tables.tables.clone()
        qpg.qpack_kv_reserve(pool, tables, i(2, 0), i(5, 20))
        assert qpg.qpack_fetch_fault_flags() == qpg.FAULT_PAGE
        assert tables.lens.tolist() == [40, 64, bad, 0, 0, 0] and tables.tables[0].tolist() == [0, 1, 6, -1]
        assert torch.equal(tables.tables[1:], before[1:]) and int(tables.refs.sum()) == 7
        held = [t.clone() for t in (tables.tables, tables.refs)]
        qpg.qpack_kv_fork(pool, tables, i(2, 2), i(3, 4))
        assert qpg.qpack_fetch_fault_flags() == qpg.FAULT_PAGE and tables.lens.tolist() == [40, 64, bad, 0, 0, 0]
        assert torch.equal(held[0], tables.tables) and torch.equal(held[1], tables.refs)
        qpg.qpack_kv_fork(pool, tables, i(2, 0, 1), i(3, 4, 5))
        assert qpg.qpack_fetch_fault_flags() == qpg.FAULT_PAGE
        assert tables.lens.tolist() == [40, 64, bad, 0, 40, 64] and tables.tables[4].tolist() == [0, 1, 7, -1]
        assert tables.tables[5].tolist() == tables.tables[1].tolist()


def test_fork_refused_among_others(qpg):
    """Children that are not empty, parents that do not exist and pages that run out, in the middle of a call: the others get
    the pages of their places in it."""
    T, pages = 16, 24
    pool = make_pool(qpg, "i8", 2, pages, 2, T, 64, 1)
    tables, sim = qpg.alloc_kv_tables(16, 6, pages), ref.Pages(16, 6, pages, T, token_view(pool))
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    for op, a, b in (("reserve", [0, 1, 2, 3], [20, 32, 5, 90]), ("fork", [0, 2, 1, 0, 2], [4, 3, 5, 6, 7]), ("free", [6, 1], None),
                     ("fork", [0, 0, 2, 5, 2, 0, 0, 2], [8, 4, 9, 10, 2, 11, 12, 13]), ("reserve", [9, 10, 8], [1, 40, 12])):
        if op == "free":
            qpg.qpack_kv_free(tables, i(a))
            sim.free(a)
            continue
        if op == "reserve":
            qpg.qpack_kv_reserve(pool, tables, i(a), i(b))
        else:
            qpg.qpack_kv_fork(pool, tables, i(a), i(b))
        getattr(sim, op)(a, b)
        same_state(qpg, pool, tables, sim)


def test_fetch_keeps_an_earlier_error(qpg):
    """An error that another library's call left behind is not the fetch's: it succeeds, and the error is still there."""
    import ctypes
    rt = ctypes.CDLL("libcudart.so.13")
    assert rt.cudaGetLastError() == 0
    assert rt.cudaGetDeviceProperties(None, 0) != 0         # invalid argument, on the host
    try:
        assert qpg.qpack_fetch_fault_flags() == 0
        assert rt.cudaPeekAtLastError() != 0
    finally:
        rt.cudaGetLastError()
