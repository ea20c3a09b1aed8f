"""GPU tests of the norm and rotation of query and key heads against the formula in 64 bits."""
import numpy as np
import pytest
import torch

from oracle import decode as ref
from test_gpu_paged import DT, make_pool, make_tables, pages_for
from test_gpu_paged import rope_table as host_table

pytestmark = pytest.mark.gpu

HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -133}


def rope_table(rows, dim):
    return torch.from_numpy(host_table(rows, dim)).cuda()


def check(got, x, odt, weight, eps, rows, interleaved):
    """Within the fp32 steps and the output's rounding. The norm's factor: 8 squares summed in order and at most 5 levels
    of pairs, 13 roundings of a sum of positive numbers, halved by the root, the division, the addition of eps and the root:
    10 steps of 2^-24; two products with it, a product and a sum of the rotation: 14."""
    want, size = ref.norm_rope(x, weight, eps, rows, interleaved)
    err = np.abs(got.double().cpu().numpy() - want)
    bound = 15 * 2.0 ** -24 * size
    bound = bound + HALF_STEP[odt] * (np.abs(want) + bound) + TINY[odt]
    assert np.all(err <= bound), (err / bound).max()


def f64(t):
    return t.double().cpu().numpy()


def inputs(n, hq, hk, dim, dt, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.empty((n, hq + 2 * hk, dim), device="cuda").normal_(0, 1.5, generator=g).to(DT[dt])
    w = 1 + 0.3 * torch.empty((2, dim), device="cuda").normal_(0, 1, generator=g)
    return x[:, :hq], x[:, hq:hq + hk], w[0], w[1]


@pytest.mark.parametrize("dim,turn", [(8, 8), (64, 64), (64, 24), (72, 64), (80, 80), (128, 128), (128, 64), (128, 8), (192, 128),
                                      (256, 256), (248, 16)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dt,odt", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f32", "f16"), ("f32", "bf16"),
                                    ("bf16", "f32"), ("f16", "bf16"), ("f16", "f32"), ("bf16", "f16")])
def test_norm_rope(qpg, dim, turn, interleaved, dt, odt):
    n, hq, hk, eps = 7, 9, 3, 1e-5
    q, k, wq, wk = inputs(n, hq, hk, dim, dt, dim + turn)
    rope = rope_table(50, turn)
    pos = torch.tensor([0, 49, 3, 3, 17, 1, 30], dtype=torch.int32, device="cuda")
    qo, ko = (torch.empty((n, h, dim), dtype=DT[odt], device="cuda") for h in (hq, hk))
    got = qpg.qpack_qk_norm_rope(q, k, wq, wk, eps=eps, rope=rope, interleaved=interleaved, pos=pos, q_out=qo, k_out=ko)
    assert got[0] is qo and got[1] is ko
    rows = f64(rope[pos.long()])
    check(qo, f64(q), odt, f64(wq), eps, rows, interleaved)
    check(ko, f64(k), odt, f64(wk), eps, rows, interleaved)
    # one side without a weight; no rotation; one side alone
    qpg.qpack_qk_norm_rope(q, k, None, wk, eps=eps, rope=rope, interleaved=interleaved, pos=pos, q_out=qo, k_out=ko)
    check(qo, f64(q), odt, None, eps, rows, interleaved)
    check(ko, f64(k), odt, f64(wk), eps, rows, interleaved)
    qpg.qpack_qk_norm_rope(q, None, wq, eps=eps, interleaved=interleaved, q_out=qo)
    check(qo, f64(q), odt, f64(wq), eps, None, interleaved)
    assert qpg.qpack_fetch_fault_flags() == 0


@pytest.mark.parametrize("n", [1, 2, 63, 1025])
@pytest.mark.parametrize("hq,hk", [(1, 1), (32, 8), (71, 1), (5, 0), (0, 5)])
def test_counts_of_tokens_and_heads(qpg, n, hq, hk):
    dim = 128
    q, k, wq, wk = inputs(n, hq, hk, dim, "bf16", n)
    rope = rope_table(2000, dim)
    pos = torch.arange(n, dtype=torch.int32, device="cuda") * 1999 // max(n - 1, 1)
    qo, ko = qpg.qpack_qk_norm_rope(q, k, wq, wk, rope=rope, pos=pos)
    assert qo.dtype == ko.dtype == torch.bfloat16
    rows = f64(rope[pos.long()])
    check(qo, f64(q), "bf16", f64(wq), 1e-6, rows, False)
    check(ko, f64(k), "bf16", f64(wk), 1e-6, rows, False)
    assert qpg.qpack_fetch_fault_flags() == 0


def test_no_tokens(qpg):
    q, k, wq, wk = inputs(0, 4, 2, 64, "f16", 0)
    qo, ko = qpg.qpack_qk_norm_rope(q, k, wq, wk, rope=rope_table(4, 64), pos=torch.zeros(0, dtype=torch.int32, device="cuda"))
    assert qo.shape == (0, 4, 64) and ko.shape == (0, 2, 64)


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place(qpg, interleaved):
    """Outputs may be the inputs, inside a row that holds the values too; those stay."""
    n, dim = 33, 128
    x = torch.randn((n, 12, dim), device="cuda").half()
    q, k, before = x[:, :8], x[:, 8:10], x.clone()
    w = torch.rand(dim, device="cuda")
    rope, pos = rope_table(40, dim), torch.arange(n, dtype=torch.int32, device="cuda")
    qpg.qpack_qk_norm_rope(q, k, w, w, rope=rope, interleaved=interleaved, pos=pos, q_out=q, k_out=k)
    rows = f64(rope[pos.long()])
    check(q, f64(before[:, :8]), "f16", f64(w), 1e-6, rows, interleaved)
    check(k, f64(before[:, 8:10]), "f16", f64(w), 1e-6, rows, interleaved)
    assert torch.equal(x[:, 10:], before[:, 10:])


def test_positions_of_sequences_and_skipped_tokens(qpg):
    """Positions from the tables, and rows that nothing is written to: idle sequences, negative positions."""
    lens, dim = [5, 0, 1, 40], 64
    pages = pages_for(lens, 16)
    _, tables = make_tables(qpg, lens, 16, pages, 1)
    q, k, wq, wk = inputs(4, 3, 1, dim, "f32", 2)
    rope = rope_table(64, dim)
    for seqs in (None, [3, 1, 0, 2]):
        order = seqs or [0, 1, 2, 3]
        ids = None if seqs is None else torch.tensor(seqs, dtype=torch.int32, device="cuda")
        qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
        qpg.qpack_qk_norm_rope(q, k, wq, wk, rope=rope, tables=tables, seqs=ids, q_out=qo, k_out=ko)
        for i, s in enumerate(order):
            if lens[s] == 0:
                assert (qo[i] == 7).all() and (ko[i] == 7).all()
            else:
                row = f64(rope[lens[s] - 1:lens[s]])
                check(qo[i:i + 1], f64(q[i:i + 1]), "f32", f64(wq), 1e-6, row, False)
                check(ko[i:i + 1], f64(k[i:i + 1]), "f32", f64(wk), 1e-6, row, False)
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    pos = torch.tensor([3, -1, -2 ** 31, 0], dtype=torch.int32, device="cuda")
    qpg.qpack_qk_norm_rope(q, k, rope=rope, pos=pos, q_out=qo, k_out=ko)
    assert (qo[1:3] == 7).all() and (ko[1:3] == 7).all()
    check(qo[3:], f64(q[3:]), "f32", None, 0, f64(rope[:1]), False)     # the table's angles are random, that of 0 too
    assert qpg.qpack_fetch_fault_flags() == 0


def test_out_of_range_is_reported(qpg):
    lens, dim = [5, 9], 64
    pages = pages_for(lens, 16)
    _, tables = make_tables(qpg, lens, 16, pages, 1)
    q, _, wq, _ = inputs(3, 3, 1, dim, "f32", 2)
    rope = rope_table(8, dim)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out = torch.full_like(q, 7.0)
    qpg.qpack_qk_norm_rope(q, None, wq, rope=rope, tables=tables, seqs=i32([0, 2, -1]), q_out=out)
    assert qpg.qpack_fetch_fault_flags() == qpg.FAULT_PAGE
    assert (out[1:] == 7).all() and not (out[0] == 7).any()
    # behind the table: normed, not rotated
    for pos in ([8, 2 ** 31 - 1, 7],):
        qpg.qpack_qk_norm_rope(q, None, wq, rope=rope, pos=i32(pos), q_out=out)
        assert qpg.qpack_fetch_fault_flags() == qpg.FAULT_PAGE
        check(out[:2], f64(q[:2]), "f32", f64(wq), 1e-6, None, False)
        check(out[2:], f64(q[2:]), "f32", f64(wq), 1e-6, f64(rope[7:]), False)
    tables.lens[0] = -4
    out.fill_(7.0)
    qpg.qpack_qk_norm_rope(q[:2], None, wq, rope=rope, tables=tables, q_out=out[:2])
    assert qpg.qpack_fetch_fault_flags() == qpg.FAULT_PAGE
    assert (out[0] == 7).all()


@pytest.mark.parametrize("kind", ["i8", "f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_keys_rotated_here_are_those_that_append_stores(qpg, kind, dim):
    """Without a norm, rotating first and appending without a table gives the cache that append's own rotation gives."""
    lens, heads = [30, 77], 5
    n = sum(lens)
    pages = pages_for(lens, 16)
    tab, tables = make_tables(qpg, lens, 16, pages, 3)
    seqs = torch.tensor([s for s, m in enumerate(lens) for _ in range(m)], dtype=torch.int32, device="cuda")
    pos = torch.tensor([t for m in lens for t in range(m)], dtype=torch.int32, device="cuda")
    k, v = (torch.randn((n, heads, dim), device="cuda") for _ in range(2))
    rope = rope_table(100, dim)
    one, two = (make_pool(qpg, kind, 1, pages, heads, 16, dim, 5) for _ in range(2))
    qpg.qpack_kv_append(one, 0, tables, k, v, seqs=seqs, pos=pos, rope=rope)
    turned, _ = qpg.qpack_qk_norm_rope(k, rope=rope, pos=pos)
    qpg.qpack_kv_append(two, 0, tables, turned, v, seqs=seqs, pos=pos)
    assert torch.equal(one.k.view(torch.uint8), two.k.view(torch.uint8))
    if kind == "i8":
        assert torch.equal(one.k_scales.view(torch.int16), two.k_scales.view(torch.int16))


def test_zeros_large_and_not_finite(qpg):
    """A head of zeros stays zero with any eps above 0; a value that is not finite stays in its head."""
    dim, w = 128, torch.ones(128, device="cuda")
    q = torch.randn((4, 3, dim), device="cuda")
    q[0, 0] = 0.0
    q[1, 1] *= 1e15
    q[2, 2] *= 1e-18
    q[3, 0, 5] = float("nan")
    q[3, 1, 7] = float("inf")
    out, _ = qpg.qpack_qk_norm_rope(q, None, w, eps=1e-30, rope=rope_table(9, dim),
                                    pos=torch.arange(4, dtype=torch.int32, device="cuda"))
    assert (out[0, 0] == 0).all() and torch.isnan(out[3, 0]).all() and torch.isnan(out[3, 1]).any()
    fine = [(0, 0), (0, 1), (0, 2), (1, 0), (1, 1), (1, 2), (2, 0), (2, 1), (2, 2), (3, 2)]
    rope = f64(rope_table(9, dim))
    for i, h in fine:
        check(out[i:i + 1, h:h + 1], f64(q[i:i + 1, h:h + 1]), "f32", f64(w), np.float32(1e-30), rope[i:i + 1], False)


def test_other_stream_graph_and_strides(qpg):
    n, dim = 19, 96
    buf = torch.randn((n, 2, 10, dim), device="cuda").bfloat16()
    q, k = buf[:, 0, :7], buf[:, 1, :3]
    w = torch.rand(dim, device="cuda")
    rope, pos = rope_table(30, 64), torch.arange(n, dtype=torch.int32, device="cuda")
    want = qpg.qpack_qk_norm_rope(q, k, w, w, rope=rope, pos=pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = qpg.qpack_qk_norm_rope(q, k, w, w, rope=rope, pos=pos, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    wide = torch.full((n, 16, dim), 3.0, device="cuda", dtype=torch.bfloat16)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qpg.qpack_qk_norm_rope(q, k, w, w, rope=rope, pos=pos, q_out=wide[:, 1:8], k_out=wide[:, 9:12])
    buf.copy_(torch.randn_like(buf.float()).bfloat16())
    want = qpg.qpack_qk_norm_rope(q, k, w, w, rope=rope, pos=pos)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(wide[:, 1:8], want[0]) and torch.equal(wide[:, 9:12], want[1])
    assert (wide[:, [0, 8, 12, 13, 14, 15]] == 3).all()
