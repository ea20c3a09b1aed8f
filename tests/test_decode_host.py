"""Host-side checks of the operators around the cache (norm and rotation of heads, the draw of tokens): the restatement that the GPU tests
compare with against independent pins, and the refusals of the C ABI and of the binding, which come before any launch."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import decode as ref
from oracle import paged

OK, ARG, SHAPE, ALIGN, UNSUPPORTED = 0, -1, -2, -3, -6
P = 4096            # an address that is never followed: refusals come first


@pytest.fixture(scope="module")
def qp():
    from bit_weight_quantized_qpack_gb300 import _build
    _build.build()
    import bit_weight_quantized_qpack_gb300 as qp
    qp.lib()
    return qp


# ---------------------------------------------------------------------------------------------------------------
# norm and rotation of heads
# ---------------------------------------------------------------------------------------------------------------
def test_norm_restatement():
    """A normed head has a mean square of one, whatever its size; weights scale its elements; torch agrees."""
    rng = np.random.default_rng(0)
    x = rng.normal(size=(5, 3, 40)) * np.exp(rng.uniform(-5, 5, (5, 3, 1)))
    y, _ = ref.norm_rope(x, np.ones(40))
    assert np.allclose((y * y).mean(-1), 1) and np.allclose(ref.norm_rope(7 * x, np.ones(40))[0], y)
    w = rng.normal(size=40)
    want = torch.nn.functional.rms_norm(torch.from_numpy(x), (40,), torch.from_numpy(w), 1e-3)
    assert np.allclose(ref.norm_rope(x, w, 1e-3)[0], want, rtol=1e-12)


def test_rotation_restatement():
    """The half layout is the cache's rotation; neighbours are the half layout of permuted elements; the rest stays."""
    rng = np.random.default_rng(1)
    x, a = rng.normal(size=(4, 2, 48)), rng.uniform(-3, 3, (4, 16))
    rows = np.concatenate([np.cos(a), np.sin(a)], 1)
    y, size = ref.norm_rope(x, rows=rows)
    assert np.allclose(y[..., :32], paged.rotate64(x[..., :32], rows)) and np.array_equal(y[..., 32:], x[..., 32:])
    assert np.all(np.abs(y) <= size * (1 + 1e-15))
    perm = np.concatenate([np.arange(0, 32, 2), np.arange(1, 32, 2)])
    near, _ = ref.norm_rope(x, rows=rows, interleaved=True)
    assert np.allclose(near[..., perm], ref.norm_rope(x[..., perm], rows=rows)[0])


def heads(qp, x=P, out=2 * P, weight=0, ldx=256, ldo=256, n=2, reserved=0):
    return qp._Heads(x or None, out or None, weight or None, ldx, ldo, n, reserved)


def call_heads(qp, q=None, k=None, n=4, dim=128, dt=0, odt=0, eps=1e-6, rope=P, rows=10, turn=128, near=0, t=None, seqs=0,
               pos=P):
    q = heads(qp) if q is None else q
    return qp.lib().qpack_qk_norm_rope(ctypes.byref(q), None if k is None else ctypes.byref(k), n, dim, dt, odt, eps,
                                       rope or None, rows, turn, near, t, seqs or None, pos or None, None)


def test_heads_refusals(qp):
    c = lambda **kw: call_heads(qp, **kw)  # noqa: E731
    h = lambda **kw: heads(qp, **kw)  # noqa: E731
    assert c(n=0) == OK and c(q=h(n=0)) == OK and qp.lib().qpack_qk_norm_rope(
        None, None, 5, 128, 0, 0, 1e-6, None, 0, 0, 0, None, None, None, None) == OK
    for bad in (dict(n=-1), dict(dt=3), dict(odt=-1), dict(eps=-1e-9), dict(eps=float("nan")), dict(eps=float("inf")),
                dict(near=2), dict(pos=0), dict(rows=-1), dict(q=h(x=0)), dict(q=h(out=0)), dict(q=h(n=-1)),
                dict(q=h(reserved=1)), dict(k=h(n=-2)), dict(q=h(out=P), odt=1), dict(q=h(out=P, ldo=264))):
        assert c(**bad) == ARG, bad
    for bad in (dict(dim=4), dict(dim=264), dict(dim=100), dict(turn=136), dict(turn=4), dict(turn=0), dict(turn=60),
                dict(rope=0), dict(q=h(ldx=248)), dict(q=h(ldo=128)), dict(k=h(n=3)), dict(q=h(n=65537))):
        assert c(**bad) == SHAPE, bad
    for bad in (dict(q=h(x=P + 8)), dict(q=h(out=P + 4)), dict(q=h(weight=P + 4)), dict(q=h(ldx=260)), dict(rope=P + 8),
                dict(pos=P + 2), dict(seqs=P + 1)):
        assert c(**bad) == ALIGN, bad
    t = qp._Tables(P, None, None, 4, 0, 2, 4)
    assert c(t=ctypes.byref(t)) == ARG                     # sequences without lengths


def test_heads_binding_refusals(qp):
    x = torch.zeros(4, 2, 64)
    pos = torch.zeros(4, dtype=torch.int32)
    rope = torch.zeros(10, 64)
    bad = [dict(q=x.view(4, 128)), dict(q=x.double()), dict(q=x.transpose(1, 2)), dict(q=x[:, :, ::2]),
           dict(q=x, k=x[:3]), dict(q=x, k=x.half()), dict(q=x, k=torch.zeros(4, 2, 32)), dict(q=x, q_weight=torch.zeros(32)),
           dict(q=x, q_weight=torch.zeros(128)), dict(q=x, q_weight=torch.zeros(64).half()), dict(q=x, rope=rope),
           dict(q=x, rope=rope.half(), pos=pos), dict(q=x, rope=rope[0], pos=pos), dict(q=x, rope=rope[:, ::2], pos=pos),
           dict(q=x, rope=rope, pos=pos.long()), dict(q=x, rope=rope, pos=pos[:3]), dict(q=x, q_out=x[:2]),
           dict(q=x, q_out=x.double()), dict(q=x, rope=rope, pos=pos)]      # the last: not on a GPU
    for kw in bad:
        with pytest.raises(qp.QpackError):
            qp.qpack_qk_norm_rope(**kw)


# ---------------------------------------------------------------------------------------------------------------
# the draw of tokens
# ---------------------------------------------------------------------------------------------------------------
def test_sample_restatement_by_hand():
    """A row whose weights are powers of two: 4 2 1 1 over their sum 8, at tokens 2, 0, 1 and 3."""
    x = np.log(np.array([2.0, 1.0, 4.0, 1.0]))
    at = lambda u, **kw: ref.sample(x, u, **kw)[0]  # noqa: E731
    assert [at(u) for u in (0.0, 0.24, 0.26, 0.37, 0.38, 0.87, 0.88)] == [0, 0, 1, 1, 2, 2, 3]
    assert ref.sample(x, 0.5)[1] == pytest.approx(0.5)
    assert list(ref.sample(x, 0.5, top_k=3)[2]) == [0, 1, 2]           # of equals the lowest index
    assert list(ref.sample(x, 0.5, top_p=0.49)[2]) == [2] and list(ref.sample(x, 0.5, top_p=0.51)[2]) == [0, 2]
    assert list(ref.sample(x, 0.5, top_k=2, top_p=0.7)[2]) == [0, 2]   # p of the two's sum: 4 / 6 < 0.7
    assert list(ref.sample(x, 0.5, top_k=2, top_p=0.66)[2]) == [2]
    assert list(ref.sample(x, 0.5, min_p=0.3)[2]) == [0, 2] and list(ref.sample(x, 0.5, min_p=1.0)[2]) == [2]
    assert ref.sample(x, 0.99, temperature=0.0)[:2] == (2, 1.0)
    assert ref.sample(x, 0.5, temperature=0.5)[1] == pytest.approx(16 / 22)
    x[2] = -np.inf
    assert [at(u) for u in (0.49, 0.51, 0.76)] == [0, 1, 3] and at(0.9, top_k=1) == 0
    assert ref.sample(np.full(3, -np.inf), 0.5)[:2] == (-1, 0.0)


def test_sample_restatement_against_sorting():
    """The filters as they are usually written, on sorted probabilities."""
    rng = np.random.default_rng(3)
    for _ in range(50):
        x = rng.normal(size=200) * 2
        t, k, p, m = rng.uniform(0.3, 2), int(rng.integers(1, 150)), rng.uniform(0.1, 0.99), rng.uniform(0, 0.2)
        q = torch.from_numpy(x / t).softmax(0)
        v, i = q.sort(descending=True)
        v, i = v[:k] / v[:k].sum(), i[:k]
        keep = (v.cumsum(0) - v) < p
        v, i = v[keep], i[keep]
        keep = v >= m * v[0]
        want = sorted(i[keep].tolist())
        assert list(ref.sample(x, rng.random(), t, k, p, m)[2]) == want


def call_sample(qp, logits=P, dt=0, ld=100, V=100, B=3, t=0, k=0, p=0, m=0, u=P, tokens=P, probs=0):
    return qp.lib().qpack_sample(logits or None, dt, ld, V, B, t or None, k or None, p or None, m or None, u or None,
                                 tokens or None, probs or None, None)


def test_sample_refusals(qp):
    c = lambda **kw: call_sample(qp, **kw)  # noqa: E731
    assert c(B=0) == OK and c(B=0, logits=0, u=0, tokens=0) == OK
    for bad in (dict(B=-1), dict(V=-1), dict(dt=3), dict(dt=-1), dict(logits=0), dict(u=0), dict(tokens=0)):
        assert c(**bad) == ARG, bad
    for bad in (dict(V=0), dict(V=2 ** 20 + 1, ld=2 ** 21), dict(ld=99), dict(B=2 ** 31)):
        assert c(**bad) == SHAPE, bad
    for bad in (dict(logits=P + 2), dict(logits=P + 1, dt=1), dict(u=P + 2), dict(tokens=P + 1), dict(probs=P + 2), dict(t=P + 1),
                dict(k=P + 2), dict(p=P + 3), dict(m=P + 2)):
        assert c(**bad) == ALIGN, bad


def test_sample_binding_refusals(qp):
    x, u, i = torch.zeros(4, 10), torch.zeros(4), torch.zeros(4, dtype=torch.int32)
    bad = [dict(logits=x[0], u=u), dict(logits=x.double(), u=u), dict(logits=x.t(), u=u), dict(logits=x[:, ::2], u=u),
           dict(logits=x, u=None), dict(logits=x, u=u[:3]), dict(logits=x, u=u.double()), dict(logits=x, u=u, temperature=u[:2]),
           dict(logits=x, u=u, top_k=i.long()), dict(logits=x, u=u, top_k=u), dict(logits=x, u=u, top_p=u.half()),
           dict(logits=x, u=u, min_p=torch.zeros(8)[::2]), dict(logits=x, u=u, tokens=i[:3]), dict(logits=x, u=u, tokens=u),
           dict(logits=x, u=u, probs=i), dict(logits=x, u=u)]              # the last: not on a GPU
    for kw in bad:
        with pytest.raises(qp.QpackError):
            qp.qpack_sample(**kw)


# ---------------------------------------------------------------------------------------------------------------
# attention over shared prefixes
# ---------------------------------------------------------------------------------------------------------------
def call_shared(qp, layer=0, seqs=0, B=4, first=P, prefix=P, groups=2, q=P, qdt=0, ldq=1024, q_heads=8, scale=0.1, rope=0, rows=0,
                out=P, odt=1, ldo=1024, lse=0, ws=P, ws_bytes=None, type=1, dim=128, heads=2, tables=P, seq=8,
                max_pages=8):
    pool = qp._Pool(P, P, None, None, 1 << 20, 1 << 14, 0, 0, 64, 1, heads, 16, dim, type, 0)
    t = qp._Tables(tables or None, P, None, max_pages, 0, seq, max_pages)
    if ws_bytes is None:
        n = ctypes.c_int64(0)
        good = qp._Pool(P, P, None, None, 1 << 20, 1 << 14, 0, 0, 64, 1, 2, 16, 128, 1, 0)
        assert qp.lib().qpack_kv_shared_workspace(ctypes.byref(good), 4, 8, ctypes.byref(n)) == OK
        ws_bytes = n.value
    return qp.lib().qpack_kv_attend_shared(
        ctypes.byref(pool), layer, ctypes.byref(t), seqs or None, B, first or None, prefix or None, groups, q or None, qdt, ldq,
        q_heads, scale, rope or None, rows, out or None, odt, ldo, lse or None, ws or None, ws_bytes, None)


def test_shared_refusals(qp):
    c = lambda **kw: call_shared(qp, **kw)  # noqa: E731
    assert c(B=0) == OK and c(B=0, q=0, out=0, ws=0, first=0, prefix=0) == OK
    for bad in (dict(layer=1), dict(layer=-1), dict(B=-1), dict(groups=-1), dict(q_heads=0), dict(qdt=3), dict(odt=-1), dict(q=0),
                dict(out=0), dict(ws=0), dict(first=0), dict(prefix=0), dict(rows=-1), dict(tables=0), dict(type=3)):
        assert c(**bad) == ARG, bad
    for bad in (dict(q_heads=7), dict(B=4097), dict(groups=513), dict(ldq=1016), dict(ldo=512), dict(ws_bytes=1 << 20),
                dict(dim=96), dict(q_heads=65536 + 2)):
        assert c(**bad) == SHAPE, bad
    for bad in (dict(q=P + 8), dict(out=P + 8), dict(ldq=1028), dict(ldo=1028), dict(first=P + 2), dict(prefix=P + 1),
                dict(seqs=P + 2), dict(lse=P + 2), dict(ws=P + 8), dict(rope=P + 4)):
        assert c(**bad) == ALIGN, bad
    pool = qp._Pool(P, P, None, None, 1 << 20, 1 << 14, 0, 0, 64, 1, 2, 16, 128, 1, 0)
    size = lambda B, h: qp.lib().qpack_kv_shared_workspace(ctypes.byref(pool), B, h, ctypes.byref(n)) or n.value  # noqa: E731
    n = ctypes.c_int64(0)
    assert size(-1, 8) == ARG and size(4, 0) == ARG and size(4, 7) == SHAPE and size(4097, 8) == SHAPE
    assert size(0, 8) > 1 << 20 and size(64, 8) > size(8, 8)
    assert qp.lib().qpack_kv_shared_workspace(ctypes.byref(pool), 4, 8, None) == ARG


def test_shared_refuses_uncountable_lengths(qp):
    """Tables of 2^31 tokens (16 a page) and tiles of all queries past 2^30: positions and units would pass their 31 bits."""
    for bad in (dict(max_pages=1 << 27), dict(max_pages=1 << 28), dict(max_pages=(1 << 27) - 17, groups=512)):
        assert call_shared(qp, **bad) == UNSUPPORTED, bad


def test_shared_binding_refusals(qp):
    pool = object.__new__(qp.KVPool)
    pool.heads, pool.dim, pool.k = 2, 64, torch.zeros(1)
    tab = object.__new__(qp.KVTables)
    tab.tables, tab.lens = torch.zeros(4, 3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    q, f, p = torch.zeros(4, 6, 64), torch.tensor([0, 2, 4], dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    ok = dict(q=q, first=f, prefix=p)
    bad = [dict(q=q.double()), dict(q=q[:, :, :32]), dict(first=f.long()), dict(first=f[:2]), dict(prefix=p.float()),
           dict(prefix=torch.zeros(4, dtype=torch.int32)[::2]), dict(q=torch.zeros(5, 6, 64)), dict(out=torch.zeros(3, 6, 64)),
           dict(out=torch.zeros(4, 6, 64).double()), dict(lse=torch.zeros(5)), dict(lse=torch.zeros(24).half()),
           dict(seqs=f.long()), dict(seqs=f[:3]), dict(rope=torch.zeros(4, 32)), dict()]      # the last: not on a GPU
    for kw in bad:
        with pytest.raises(qp.QpackError):
            qp.qpack_kv_attend_shared(pool, 0, tab, **{**ok, **kw})
