"""Attention over shared prefixes that are long enough for every form of its inner loop, against 64 bits.

Which form runs goes by the queries of a group, their type and the tiles that a block of the GPU gets: two blocks of 128 queries
at a time, or one; one accumulator, or two that tiles go to in turn. Lengths here are derived from the number of SMs, and each test
states the conditions of the form that it is about, so that it cannot stop reaching it unnoticed. Tolerances are those of
test_gpu_shared.py."""
import pytest
import torch

from test_gpu_paged import DT, SPLIT, ULP, make_pool
from test_gpu_shared import check as check_rows
from test_gpu_shared import f64, forked, i32, tables_of

pytestmark = pytest.mark.gpu


def held(pool, tab, n):
    """Keys and values of a sequence's first n tokens, [heads, n, dim] in fp64."""
    t, T = torch.arange(n, device="cuda"), pool.page_tokens
    page = torch.from_numpy(tab).cuda().long()[t // T]
    out = []
    for c, s in ((pool.k, pool.k_scales), (pool.v, pool.v_scales)):
        x = c[0, page, :, t % T].double()
        if s is not None:
            x = (x * s[0, page, :, t % T].double().repeat_interleave(32, 2)).half().double()
        out.append(x.transpose(0, 1))
    return out


def check(out, lse, odt, kind, q, pool, tab, lens, prefix, scale):
    """All rows are one group; test_gpu_shared.py's bounds, on the GPU in fp64."""
    B, Hq, D = q.shape
    H = pool.heads
    split_p = 2.0 ** -16 if kind == "bf16" else 2.0 ** -22 if odt == "f32" else 2.0 ** -11
    ka, va = held(pool, tab[0], prefix)
    for b in range(B):
        L = lens[b]
        kb, vb = held(pool, tab[b], L)
        k, v = torch.cat([ka, kb[:, prefix:]], 1), torch.cat([va, vb[:, prefix:]], 1)
        qr = q[b].double().view(H, Hq // H, D)
        x = qr @ k.transpose(1, 2) * scale
        want_lse, w = x.logsumexp(-1), x.softmax(-1)
        mass = (qr.abs() @ k.abs().transpose(1, 2)).amax(-1) * abs(scale)
        dx = mass * (SPLIT[kind] + (D + 8) * 2.0 ** -23)
        tol = (w @ v.abs()) * (3 * dx + split_p + 2.0 ** -20 + (L / 8 + 64 + 160) * 2.0 ** -23)[..., None]
        want = w @ v
        tol = tol + 2.0 ** -32 * v.abs().sum(1)[:, None] + want.abs() * ULP[odt] + 2.0 ** -25 * (odt != "f32")
        err = (out[b].double().view_as(want) - want).abs()
        assert (err <= tol).all(), (b, float((err / tol).max()))
        ltol = dx + 2.0 ** -20 + want_lse.abs() * 2.0 ** -22 + (L / 8 + 160) * 2.0 ** -23
        lerr = (lse[b].double().view_as(want_lse) - want_lse).abs()
        assert (lerr <= ltol).all(), (b, float((lerr / ltol).max()))


def forms(D, H, G, rows, prefix, one_term):
    """Whether two blocks of queries are taken at a time, and the tiles that a softmax group has in a row."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tok, two, queries = 64 if D == 256 else 128, D <= 128, rows * G
    tiles = -(-prefix // tok)
    pair = two and one_term and queries > 128 and tiles * -(-queries // 256) * H >= 6 * sms
    blocks = -(-queries // (256 if pair else 128))
    share = -(-tiles * blocks * H // sms)
    return pair, share if pair or not two else share // 2


# queries' type, output's type: queries are one term where the first is the cache's own product type
@pytest.mark.parametrize("kind,D,G,rows,qdt,odt,pair", [
    ("i8", 64, 64, 3, "f16", "f16", True), ("f16", 64, 64, 3, "f16", "f32", True), ("bf16", 64, 64, 3, "bf16", "bf16", True),
    ("i8", 128, 64, 3, "f16", "f16", True), ("f16", 128, 64, 4, "f16", "bf16", True), ("i8", 128, 33, 5, "f16", "f32", True),
    ("bf16", 128, 64, 3, "bf16", "f32", True), ("bf16", 128, 32, 8, "bf16", "bf16", True),
    ("i8", 64, 4, 3, "f32", "f16", False), ("i8", 128, 4, 3, "f32", "f16", False), ("f16", 128, 4, 3, "f16", "f16", False),
    ("f16", 128, 48, 3, "f32", "f16", False), ("bf16", 128, 4, 3, "f32", "f32", False), ("i8", 256, 4, 3, "f16", "f16", False),
    ("f16", 256, 48, 3, "f32", "f16", False), ("f16", 256, 4, 3, "f16", "f32", False), ("bf16", 256, 4, 3, "bf16", "bf16", False)])
def test_maxima_that_move(qpg, kind, D, G, rows, qdt, odt, pair):
    """Scores swell and ebb along the prefix, each query's in its own way: the running maximum holds in some tiles, moves a little in
    others and far in others, and what has been added up is scaled down behind it."""
    T, H, tok = 64, 2, 64 if D == 256 else 128
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    blocks = -(-rows * G // (256 if pair else 128))
    tiles = -(-(8 if pair or D == 256 else 16) * sms // (H * blocks))
    prefix = tiles * tok - 5
    one_term = qdt == ("bf16" if kind == "bf16" else "f16")
    assert forms(D, H, G, rows, prefix, one_term) == (pair, 8)
    first, pref, lens, tab, pages = forked(qpg, [rows], [prefix], [20, 3, 0], T, seed=D + G)
    pool = make_pool(qpg, kind, 1, pages, H, T, D, D + G)
    t = torch.arange(lens[0], device="cuda")
    ramp = 40 * torch.sin(t / 300.0) + t * (100.0 / prefix)
    page = torch.from_numpy(tab[0]).cuda().long()[t // T]
    for h in range(H):
        x = ramp * (1 + h / 8)
        if kind == "i8":
            pool.k_scales[0, page, h, t % T, 0] = (x.abs() / 127).half()
            pool.k[0, page, h, t % T, 5] = (127 * torch.sign(x)).to(torch.int8)
        else:
            pool.k[0, page, h, t % T, 5] = x.to(DT[kind])
    q = torch.randn((rows, H * G, D), device="cuda") * 0.1
    q[:, :, 5] = torch.linspace(-2, 2, rows * H * G, device="cuda").view(rows, H * G)
    q = q.to(DT[qdt])
    out, lse = torch.empty(q.shape, dtype=DT[odt], device="cuda"), torch.empty(q.shape[:2], device="cuda")
    tables = tables_of(qpg, tab, lens)
    ws = qpg.alloc_kv_shared_workspace(pool, rows, H * G)
    for _ in range(2):                                      # the second call finds the workspace as the first left it
        qpg.qpack_kv_attend_shared(pool, 0, tables, q, i32(first), i32(pref), scale=1.0, out=out, lse=lse, workspace=ws)
        once = out.clone() if _ == 0 else once
    assert qpg.qpack_fetch_fault_flags() == 0 and torch.equal(once, out)
    check(out, lse, odt, kind, q, pool, tab, lens, prefix, 1.0)


@pytest.mark.parametrize("kind", ["i8", "f16", "bf16"])
@pytest.mark.parametrize("D,qdt", [(128, "f32"), (128, "f16"), (256, "f32"), (256, "f16"), (256, "bf16")])
def test_rising_maxima(qpg, kind, D, qdt):
    """Scores that rise by thousands along a prefix, so that the running maximum moves in every tile, and fall again."""
    first, pref, lens, tab, pages = forked(qpg, [6], [1500], [20], 64, seed=12)
    pool = make_pool(qpg, kind, 1, pages, 1, 64, D, 12)
    ramp = torch.tensor([(t if t < 1100 else 2200 - t) / 10.0 for t in range(1520)], device="cuda")
    for s in range(6):
        t = torch.arange(lens[s], device="cuda")
        page = torch.from_numpy(tab[s]).cuda().long()[t // 64]
        if kind == "i8":
            pool.k_scales[0, page, 0, t % 64, 0] = (ramp[:lens[s]] / 127).half()
            pool.k[0, page, 0, t % 64, 5] = 127
        else:
            pool.k[0, page, 0, t % 64, 5] = ramp[:lens[s]].to(pool.k.dtype)
    q = torch.zeros((6, 4, D), device="cuda")
    q[:, :, 5] = torch.linspace(-3, 30, 24, device="cuda").view(6, 4)
    q = q.to(DT[qdt])
    out, lse = torch.empty((6, 4, D), device="cuda"), torch.empty((6, 4), device="cuda")
    qpg.qpack_kv_attend_shared(pool, 0, tables_of(qpg, tab, lens), q, i32(first), i32(pref), scale=1.0, out=out, lse=lse)
    assert qpg.qpack_fetch_fault_flags() == 0
    check_rows(out, lse, "f32", kind, f64(q), pool, 0, tab, lens, range(6), [0] * 6, [1500] * 6, 1.0, None)
