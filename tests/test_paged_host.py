"""Host-side checks of the paged KV cache: the restatement that the GPU tests compare with against independent pins, and
the refusals of the C ABI and of the binding, which come before any launch."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import paged as ref


@pytest.fixture(scope="module")
def qp():
    from bit_weight_quantized_qpack_gb300 import _build
    _build.build()
    import bit_weight_quantized_qpack_gb300 as qp
    qp.lib()
    return qp


def test_attend_restatement_against_torch():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(6, 64)), rng.normal(size=(50, 2, 64)), rng.normal(size=(50, 2, 64))
    out, lse = ref.attend(q, k, v, 0.2)
    tq, tk, tv = (torch.from_numpy(x) for x in (q, k, v))
    x = torch.einsum("hd,nhd->hn", tq, tk.repeat_interleave(3, 1)) * 0.2
    assert np.allclose(out, torch.einsum("hn,nhd->hd", x.softmax(-1), tv.repeat_interleave(3, 1)), rtol=1e-12, atol=1e-14)
    assert np.allclose(lse, x.logsumexp(-1), rtol=1e-13)
    one, _ = ref.attend(q, k, v, 0.2, window=1)
    assert np.allclose(one, np.repeat(v[-1], 3, 0), rtol=1e-15)


def test_rotation_restatement():
    """A rotation keeps each pair's norm, by angle 0 is the identity, and two turns add up."""
    rng = np.random.default_rng(1)
    x = rng.normal(size=(4, 3, 64)).astype(np.float32)
    a, b = rng.uniform(-3, 3, (2, 4, 32))
    row = lambda t: np.concatenate([np.cos(t), np.sin(t)], 1)  # noqa: E731
    y = ref.rotate64(x, row(a))
    assert np.allclose(np.hypot(y[..., :32], y[..., 32:]), np.hypot(x[..., :32], x[..., 32:]), rtol=1e-6)
    assert np.array_equal(ref.rotate32(x, row(0 * a).astype(np.float32)), x)
    assert np.allclose(ref.rotate64(y, row(b)), ref.rotate64(x, row(a + b)), atol=1e-12)
    assert np.allclose(ref.rotate32(x, row(a).astype(np.float32)), y, atol=1e-5)


def test_quantize_restatement_against_flat_oracle(orc):
    rng = np.random.default_rng(2)
    x = (rng.normal(size=(64, 128)) * np.exp(rng.uniform(-12, 8, (64, 1)))).astype(np.float16)
    rq, rs = orc.kv_quantize(x.view(np.uint16).reshape(-1))
    q, s = ref.quantize32(x.astype(np.float32))
    assert np.array_equal(q.reshape(-1), rq.reshape(-1)) and np.array_equal(s.view(np.uint16).reshape(-1), rs)
    assert np.array_equal(ref.values(q, s).astype(np.float16).view(np.uint16).reshape(-1), orc.kv_dequant(rq, rs).reshape(-1))


def test_bf16_restatement():
    x = np.random.default_rng(3).normal(size=10000).astype(np.float32) * np.float32(1e3)
    assert np.array_equal(ref.bf16(x), torch.from_numpy(x).bfloat16().float().numpy())


def test_page_lists():
    s = ref.Pages(4, 5, 8, 4, np.arange(32).reshape(8, 4).copy())
    s.reserve([0, 1], [6, 4])
    assert s.tables[0][:2] == [0, 1] and s.tables[1][:1] == [2] and s.lens == [6, 4, 0, 0]
    s.fork([0, 1], [2, 3])
    assert s.tables[2][:2] == [0, 3] and s.refs[:4] == [2, 1, 2, 1] and s.pool[3].tolist() == [4, 5, 14, 15]
    s.free([0, 1])
    assert s.refs[:4] == [1, 0, 1, 1] and s.compact() == 1 and s.tables[2][:2] == [0, 1] and s.tables[3][:1] == [2]


def pool_struct(qp, **kw):
    d = dict(k=1 << 20, v=1 << 20, k_scales=1 << 20, v_scales=1 << 20, layer_stride=0, page_stride=2 * 16 * 128,
             scale_layer_stride=0, scale_page_stride=2 * 16 * 4, pages=10, layers=1, heads=2, page_tokens=16, dim=128,
             type=qp.KV_I8, reserved=0)
    d.update(kw)
    return qp._Pool(*(d[f] for f, _ in qp._Pool._fields_))


def table_struct(qp, **kw):
    d = dict(tables=1 << 20, lens=1 << 20, refs=1 << 20, stride=4, pages=10, seqs=3, max_pages=4)
    d.update(kw)
    return qp._Tables(*(d[f] for f, _ in qp._Tables._fields_))


def test_abi_refusals(qp):
    """Null, enum, shape, alignment and workspace errors come back before anything is launched."""
    L, R = qp.lib(), ctypes.byref
    ARG, SHAPE, ALIGN = -1, -2, -3
    good, odd = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 4)
    W = 2 * 128

    def append(pool=None, tab=None, layer=0, n=3, k=good, dt=0, ld=W, rope=None, rows=0, **kw):
        p, t = pool or pool_struct(qp, **kw), tab or table_struct(qp)
        return L.qpack_kv_append(R(p), layer, R(t), None, None, n, k, good, dt, ld, ld, rope, rows, None)

    def attend(layer=0, B=3, q=good, qdt=0, ldq=8 * 128, heads=8, window=0, odt=1, ldo=8 * 128, ws=good, bytes=1 << 40,
               seqs=None, tab=None, **kw):
        return L.qpack_kv_attend(R(pool_struct(qp, **kw)), layer, R(tab or table_struct(qp)), seqs, B, q, qdt, ldq, heads, 0.1,
                                 window, None, 0, good, odt, ldo, None, ws, bytes, None)

    for call in (append, attend):
        assert call(dim=96) == SHAPE and call(page_tokens=24) == SHAPE and call(page_tokens=2048) == SHAPE
        assert call(**({"heads": 0} if call is append else {"heads": 5})) == SHAPE
        assert call(type=3) == ARG and call(pages=-1) == ARG and call(k_scales=None) == ARG
        assert call(layer=1) == ARG and call(layer=-1) == ARG
        assert call(page_stride=2 * 16 * 128 - 16) == SHAPE and call(scale_page_stride=8) == SHAPE
        assert call(page_stride=2 * 16 * 128 + 8) == ALIGN and call(layer_stride=8) == ALIGN
        assert call(tab=table_struct(qp, seqs=-1)) == ARG and call(tab=table_struct(qp, lens=None)) == ARG
        assert call(tab=table_struct(qp, stride=3)) == SHAPE
    assert append(k=None) == ARG and append(k=odd) == ALIGN and append(dt=3) == ARG and append(n=-1) == ARG
    assert append(ld=W - 8) == SHAPE and append(ld=W + 4) == ALIGN and append(rope=odd, rows=5) == ALIGN
    assert attend(heads=7) == SHAPE and attend(B=-1) == ARG and attend(B=4097) == SHAPE and attend(window=-1) == ARG
    assert attend(q=None) == ARG and attend(q=odd) == ALIGN and attend(qdt=7) == ARG and attend(odt=-1) == ARG
    assert attend(ldq=8 * 128 - 8) == SHAPE and attend(ldo=8 * 128 + 4) == ALIGN and attend(seqs=ctypes.c_void_p(2)) == ALIGN
    assert attend(ws=None) == ARG and attend(ws=odd) == ALIGN and attend(bytes=8) == SHAPE
    # empty calls are accepted and launch nothing
    assert append(n=0) == 0 and attend(B=0) == 0
    p, t = pool_struct(qp), table_struct(qp)
    n = ctypes.c_int64(0)
    assert L.qpack_kv_attend_workspace(R(p), 4, 8, R(n)) == 0 and n.value > 0
    assert L.qpack_kv_attend_workspace(R(p), 4, 9, R(n)) == SHAPE and L.qpack_kv_attend_workspace(R(p), 4, 8, None) == ARG
    assert L.qpack_kv_page_workspace(R(p), R(t), R(n)) == 0 and n.value > 0
    assert L.qpack_kv_read(R(p), 0, R(t), None, None, 3, None, None, 0, 0, 0, None) == 0
    assert L.qpack_kv_read(R(p), 0, R(t), None, None, 3, odd, None, 0, W, 0, None) == ALIGN
    big = 1 << 40
    assert L.qpack_kv_reserve(R(p), R(t), None, good, 2, None) == ARG and L.qpack_kv_reserve(R(p), R(t), good, good, 0, None) == 0
    assert L.qpack_kv_reserve(R(p), R(t), good, good, 4097, None) == SHAPE
    assert L.qpack_kv_reserve(R(p), R(table_struct(qp, pages=11)), good, good, 1, None) == SHAPE
    assert L.qpack_kv_fork(R(p), R(t), good, good, 2, None, big, None) == ARG
    assert L.qpack_kv_fork(R(p), R(t), good, good, 2, good, 16, None) == SHAPE
    assert L.qpack_kv_fork(R(p), R(table_struct(qp, refs=None)), good, good, 2, good, big, None) == ARG
    assert L.qpack_kv_free(R(t), None, 1, None) == ARG and L.qpack_kv_free(R(t), good, -1, None) == ARG
    assert L.qpack_kv_free(R(t), good, 0, None) == 0
    assert L.qpack_kv_compact(R(p), R(t), None, good, None, good, big, None) == ARG
    assert L.qpack_kv_compact(R(p), R(t), good, good, None, good, 16, None) == SHAPE
    assert L.qpack_kv_compact(R(p), R(t), ctypes.c_void_p(2), good, None, good, big, None) == ALIGN
    assert L.qpack_kv_copy_pages(R(p), good, None, 1, None) == ARG and L.qpack_kv_copy_pages(R(p), good, good, 0, None) == 0
    assert L.qpack_kv_append(None, 0, R(t), None, None, 1, good, good, 0, W, W, None, 0, None) == ARG
    assert L.qpack_kv_append(R(p), 0, None, None, None, 1, good, good, 0, W, W, None, 0, None) == ARG


def test_binding_refusals(qp):
    z = torch.zeros
    k8, s8 = z((1, 4, 2, 16, 64), dtype=torch.int8), z((1, 4, 2, 16, 2), dtype=torch.float16)
    bad = [
        (lambda: qp.KVPool(k8.int(), k8.int()), "k: expected int8"),
        (lambda: qp.KVPool(k8, k8), "k_scales, v_scales"),
        (lambda: qp.KVPool(k8.half(), k8.half(), s8, s8), "k_scales, v_scales"),
        (lambda: qp.KVPool(k8, k8.half(), s8, s8), "v: expected torch.int8"),
        (lambda: qp.KVPool(k8, k8[:, :3], s8, s8), "v: expected \\[layers"),
        (lambda: qp.KVPool(k8, k8, s8.float(), s8), "k_scales: expected torch.float16"),
        (lambda: qp.KVPool(k8, k8, s8, s8[..., :1]), "v_scales: expected \\[layers"),
        (lambda: qp.KVPool(k8.transpose(2, 3).contiguous().transpose(2, 3), k8, s8, s8), "k: pages are not contiguous"),
        (lambda: qp.KVPool(k8, z((1, 8, 2, 16, 64), dtype=torch.int8)[:, ::2], s8, s8), "v: layer and page strides"),
        (lambda: qp.KVPool(k8, k8, s8, s8), "CUDA tensors"),
        (lambda: qp.KVTables(z((2, 3)), z(2, dtype=torch.int32)), "tables: expected a row-major int32"),
        (lambda: qp.KVTables(z((2, 3), dtype=torch.int32), z(1, dtype=torch.int32)), "lens"),
        (lambda: qp.KVTables(z((2, 3), dtype=torch.int32), z(2, dtype=torch.int64)), "lens: expected torch.int32"),
    ]
    for call, text in bad:
        with pytest.raises(qp.QpackError, match=text):
            call()

    class Fake:                                             # the checks of the calls come before any pointer is taken
        heads, dim, page_tokens, pages, layers = 2, 64, 16, 4, 1
        k = k8
    pool, tab = Fake(), Fake()
    tab.tables, tab.lens, tab.refs = z((2, 3), dtype=torch.int32), z(2, dtype=torch.int32), None
    x = z((2, 2, 64))
    i = z(2, dtype=torch.int32)
    calls = [
        (lambda: qp.qpack_kv_append(pool, 0, tab, x.int(), x), "k: expected float32"),
        (lambda: qp.qpack_kv_append(pool, 0, tab, x, x.half()), "same type"),
        (lambda: qp.qpack_kv_append(pool, 0, tab, x, x[:1]), "same type and number"),
        (lambda: qp.qpack_kv_append(pool, 0, tab, z((2, 3, 64)), x), "k: expected rows of 2 x 64"),
        (lambda: qp.qpack_kv_append(pool, 0, tab, x, x, seqs=i.long()), "seqs: expected torch.int32"),
        (lambda: qp.qpack_kv_append(pool, 0, tab, x, x, pos=i[:1]), "pos: expected a contiguous"),
        (lambda: qp.qpack_kv_append(pool, 0, tab, x, x, rope=z((5, 32))), "rope: expected"),
        (lambda: qp.qpack_kv_read(pool, 0, tab), "n: needed"),
        (lambda: qp.qpack_kv_read(pool, 0, tab, i, i, k_out=x, v_out=x.half()), "same type"),
        (lambda: qp.qpack_kv_read(pool, 0, tab, i, i, k_out=x[:1]), "k_out: expected at least 2"),
        (lambda: qp.qpack_kv_attend(pool, 0, tab, z((2, 100))), "q: expected rows"),
        (lambda: qp.qpack_kv_attend(pool, 0, tab, x, out=z((2, 2, 64), dtype=torch.int8)), "out: expected float32"),
        (lambda: qp.qpack_kv_attend(pool, 0, tab, x, out=x[:1]), "out: expected at least 2 rows"),
        (lambda: qp.qpack_kv_attend(pool, 0, tab, z((3, 2, 64))), "3 rows, but the table has 2"),
        (lambda: qp.qpack_kv_attend(pool, 0, tab, x, lse=z((2, 2), dtype=torch.float16)), "lse: expected torch.float32"),
        (lambda: qp.qpack_kv_reserve(pool, tab, i, i), "reference counts"),
        (lambda: qp.qpack_kv_fork(pool, tab, i, i), "reference counts"),
        (lambda: qp.qpack_kv_free(tab, i), "reference counts"),
        (lambda: qp.qpack_kv_compact(pool, tab), "reference counts"),
        (lambda: qp.qpack_kv_copy_pages(pool, i, i[:1]), "dst"),
    ]
    for call, text in calls:
        with pytest.raises(qp.QpackError, match=text):
            call()
