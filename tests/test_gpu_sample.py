"""GPU tests of the draw of tokens against the definition in 64 bits.

Tokens have to be equal. In exact arithmetic a draw could fall to a neighbour only where u, or top_p, lies within about
2^-40 of a border of the cumulative weights (weights to 2^-43, up to 2^17 of them); random numbers of 24 bits come that
near to a border of some 10^5 with probability 10^5 2^-40 a row, 10^-7. Probabilities: a weight is off by at most 2^-43 of
itself and 2^-42 of the largest for the places that it is held to, the total by as much, and the result is rounded to
fp32, 2^-24 of itself."""
import numpy as np
import pytest
import torch

from oracle import decode as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def dev(x, dt=torch.float32):
    return torch.as_tensor(np.asarray(x)).to("cuda", dt)


def logits_like(rows, vocab, dt, seed, spread=2.0, hot=20):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.empty((rows, vocab), device="cuda").normal_(0, spread, generator=g)
    at = torch.randint(0, vocab, (rows, min(hot, vocab)), device="cuda", generator=g)
    x.scatter_add_(1, at, 6 + 3 * torch.rand(at.shape, device="cuda", generator=g))
    return x.to(DT[dt])


def check(qpg, x, u, temperature=None, top_k=None, top_p=None, min_p=None, flags=0, rows=None):
    """Every row against the definition; returns the tokens."""
    B = x.shape[0]
    probs = torch.full((B,), -7.0, device="cuda")
    as32 = lambda v: None if v is None else dev(v)  # noqa: E731
    tokens = qpg.qpack_sample(x, dev(u), temperature=as32(temperature), top_k=None if top_k is None else dev(top_k, torch.int32),
                              top_p=as32(top_p), min_p=as32(min_p), probs=probs)
    assert qpg.qpack_fetch_fault_flags() == flags
    h, tokens, probs = x.float().cpu().numpy(), tokens.cpu().numpy(), probs.double().cpu().numpy()
    for i in range(B) if rows is None else rows:
        t, p, _ = ref.sample(h[i], np.float32(u[i]), 1.0 if temperature is None else np.float32(temperature[i]),
                             0 if top_k is None else int(top_k[i]), 1.0 if top_p is None else np.float32(top_p[i]),
                             0.0 if min_p is None else np.float32(min_p[i]))
        assert tokens[i] == t, (i, tokens[i], t)
        assert abs(probs[i] - p) <= p * (2.0 ** -24 + 2.0 ** -41) + 2.0 ** -41, (i, probs[i], p)
    return tokens


SIZES = [1, 2, 3, 31, 33, 1000, 4097, 32000, 50257, 128256]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("vocab", SIZES)
def test_each_filter(qpg, vocab, dt):
    rng = np.random.default_rng(vocab)
    B = 9
    x = logits_like(B, vocab, dt, vocab)
    t = rng.uniform(0.3, 1.6, B)
    k, p, m = rng.integers(1, 80, B), rng.uniform(0.05, 0.99, B), rng.uniform(0, 0.3, B)
    u = rng.random(B)
    check(qpg, x, u)
    check(qpg, x, u, t)
    check(qpg, x, u, t, top_k=k)
    check(qpg, x, u, t, top_p=p)
    check(qpg, x, u, t, min_p=m)
    check(qpg, x, u, t, top_k=k, top_p=p)
    check(qpg, x, u, t, top_k=k, top_p=p, min_p=m)
    check(qpg, x, u, None, top_p=p, min_p=m)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_rows_of_all_kinds_together(qpg, dt):
    """Greedy rows, rows without filters, masked ones: 97 rows in one call."""
    rng = np.random.default_rng(5)
    B, V = 97, 5003
    x = logits_like(B, V, dt, 6)
    mask = torch.from_numpy(rng.random((B, V)) < np.linspace(0, 0.9999, B)[:, None]).cuda()
    x = x.masked_fill(mask, float("-inf"))
    x[11] = float("-inf")
    x[12], x[12, 77] = float("-inf"), -3.0
    i = np.arange(B)
    t = np.where(i % 5 == 4, 0.0, rng.uniform(0.2, 2.0, B))
    k = np.where(i % 3 == 0, rng.integers(1, 300, B), 0)
    p = np.where(i % 4 == 1, rng.uniform(0.1, 1.0, B), 1.0)
    m = np.where(i % 7 == 2, rng.uniform(0, 0.5, B), 0.0)
    tokens = check(qpg, x, rng.random(B), t, k, p, m)
    assert tokens[11] == -1 and tokens[12] == 77


@pytest.mark.parametrize("vocab", [5, 4000, 70001])
def test_all_equal(qpg, vocab):
    """Ties throughout: the lowest indices are kept, and the draw is uniform over them."""
    B = 12
    x = torch.full((B, vocab), 1.25, device="cuda")
    u = (np.arange(B) + 0.5) / B
    n = max(1, vocab // 3)
    tokens = check(qpg, x, u, top_k=np.full(B, n))
    assert np.array_equal(tokens, np.floor(np.float32(u).astype(np.float64) * n))
    tokens = check(qpg, x, u, top_p=np.full(B, 0.5))
    assert tokens.max() < (vocab + 1) // 2
    assert np.array_equal(check(qpg, x, u, np.zeros(B)), np.zeros(B))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("vocab", [40000])
def test_many_tokens_in_one_interval(qpg, dt, vocab):
    """Thousands of tokens that lie closer together than an interval of the histogram, some of them alike: the intervals are
    divided by the bits of the logits."""
    rng = np.random.default_rng(8)
    B = 8
    base = 10.0 + 0.01 * rng.random((B, vocab))
    base[:, ::3] = 10.004
    base[4:] *= -1
    x = dev(base).to(DT[dt])
    x[:, 17] += 4
    u = rng.random(B)
    check(qpg, x, u, top_k=rng.integers(1, vocab, B))
    check(qpg, x, u, top_p=rng.uniform(0.3, 0.999, B))
    check(qpg, x, u, np.full(B, 0.01), top_k=rng.integers(1, vocab, B), top_p=rng.uniform(0.3, 0.999, B))


def test_near_zero_of_both_signs(qpg):
    """Logits around 0, -0 and subnormal numbers among them: -0 and 0 are alike."""
    rng = np.random.default_rng(9)
    B, V = 6, 3000
    x = dev(rng.normal(size=(B, V)) * 10.0 ** rng.integers(-45, -35, (B, V)))
    x[:, ::2] = 0.0
    x[:, ::4] = -0.0
    u = rng.random(B)
    check(qpg, x, u, top_k=[1, 2, 700, 1400, 2000, 2999])
    check(qpg, x, u, top_p=rng.uniform(0.1, 0.9, B))
    check(qpg, x, u, np.full(B, 1e-18), top_k=[1, 2, 700, 1400, 2000, 2999])


@pytest.mark.parametrize("temperature", [1e-30, 1e-5, 0.01, 30.0, 1e6, 1e30, float("inf")])
def test_temperatures(qpg, temperature):
    rng = np.random.default_rng(10)
    B, V = 8, 9001
    x = logits_like(B, V, "f32", 11)
    u = rng.random(B)
    t = np.full(B, temperature)
    check(qpg, x, u, t)
    check(qpg, x, u, t, top_k=rng.integers(1, 500, B))
    check(qpg, x, u, t, top_p=rng.uniform(0.1, 0.9, B), min_p=np.full(B, 0.05))


def test_wide_logits(qpg):
    """Differences past fp32's range, and large numbers whose differences lose nothing."""
    rng = np.random.default_rng(12)
    V = 2000
    x = dev(rng.normal(size=(5, V)))
    x[0] = (x[0] * 1e38).clamp(-3e38, 3e38)               # finite: +inf is a fault, tested below
    x[1, 0], x[1, 1] = 3e38, -3e38
    x[2] = 16777216.0 - torch.arange(V, device="cuda")
    x[3] = 1e6 + x[3]
    x[4, :1000] -= 2e4
    u = rng.random(5)
    check(qpg, x, u)
    check(qpg, x, u, top_k=[3, 5, 100, 100, 1500])
    check(qpg, x, u, np.full(5, 40.0), top_p=np.full(5, 0.9))


def test_filters_at_their_ends(qpg):
    """k past the row, p of 0, below 0, above 1 and NaN, min_p of 1 and above, and the random numbers' ends."""
    B, V = 8, 500
    x = logits_like(B, V, "f32", 13)
    top = x.argmax(1).cpu().numpy()
    inf, nan = float("inf"), float("nan")
    u = np.linspace(0, 1 - 2.0 ** -24, B)
    free = check(qpg, x, u)
    first, last = int(free[0]), int(free[-1])
    assert first == 0 and last >= V - 20                   # weights of 2^-46 and more fill all but a few of the places
    for k in (V, V + 1, 2 ** 31 - 1, 0, -1, -2 ** 31):
        assert np.array_equal(check(qpg, x, u, top_k=np.full(B, k)), free)
    get = lambda **kw: qpg.qpack_sample(x, dev(u), **{n: dev(v) for n, v in kw.items()}).cpu().numpy()  # noqa: E731
    assert np.array_equal(get(top_p=np.full(B, nan)), free) and np.array_equal(get(min_p=np.full(B, nan)), free)
    assert np.array_equal(get(top_p=np.full(B, inf)), free) and np.array_equal(get(min_p=np.full(B, -1.0)), free)
    for kw in (dict(top_p=np.zeros(B)), dict(top_p=np.full(B, -3.0)), dict(min_p=np.ones(B)), dict(min_p=np.full(B, inf)),
               dict(temperature=np.full(B, nan)), dict(temperature=np.full(B, -1.0)), dict(top_p=np.full(B, 1e-40))):
        assert np.array_equal(get(**kw), top), kw
    assert np.array_equal(check(qpg, x, u, top_k=np.ones(B)), top)
    ends = qpg.qpack_sample(x, dev([-1.0, -0.0, nan, 1.0, inf, 1 - 2.0 ** -24, 2.0, 0.0])).cpu().numpy()
    start, end = (int(qpg.qpack_sample(x[i:i + 1], dev([v]))[0]) for i, v in ((0, 0.0), (3, 1 - 2.0 ** -24)))
    assert ends[0] == start and ends[3] == end and ends[2] == int(qpg.qpack_sample(x[2:3], dev([0.0]))[0])
    assert qpg.qpack_fetch_fault_flags() == 0


def test_not_finite(qpg):
    x = logits_like(5, 300, "f32", 14)
    x[1, 7] = float("nan")
    x[2, 299] = float("inf")
    x[3, 0] = -float("nan")
    probs = torch.zeros(5, device="cuda")
    tokens = qpg.qpack_sample(x, dev([0.5] * 5), temperature=dev([1, 1, 0, 1, 0]), probs=probs).cpu().numpy()
    assert qpg.qpack_fetch_fault_flags() == qpg.FAULT_NONFINITE_X
    assert np.array_equal(tokens[1:4], [-1, -1, -1]) and torch.isnan(probs[1:4]).all()
    assert tokens[0] >= 0 and tokens[4] == int(x[4].argmax()) and torch.isfinite(probs[[0, 4]]).all()


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_rows_that_start_anywhere(qpg, dt):
    """Rows of an odd width, at every offset inside 16 bytes, with other numbers before and behind them that must not count."""
    rng = np.random.default_rng(15)
    for width, pad, off in ((37, 3, 1), (1001, 0, 3), (64, 5, 7), (1, 2, 1), (7, 1, 5)):
        B = 10
        flat = torch.full((B * (width + pad) + off + 8,), 1000.0, device="cuda").to(DT[dt])
        x = flat[off:off + B * (width + pad)].view(B, width + pad)[:, :width]
        x.copy_(logits_like(B, width, dt, width))
        check(qpg, x, rng.random(B), rng.uniform(0.5, 1.5, B), top_k=rng.integers(0, 30, B), top_p=rng.uniform(0.5, 1.1, B))


def test_largest_vocabulary(qpg):
    rng = np.random.default_rng(16)
    V = 1 << 20
    for dt in ("f32", "bf16"):
        x = logits_like(3, V, dt, 17)
        u = rng.random(3)
        check(qpg, x, u, [1.0, 4.0, 1e9])
        check(qpg, x, u, [1.0, 4.0, 1e9], top_k=[100000, 0, 50], top_p=[0.9, 0.9, 1.0])


def test_same_row_same_token(qpg):
    """The same logits give the same bits, whatever the batch around them."""
    x = logits_like(1, 32000, "f32", 18)
    u, p = dev([0.37]), dev([0.95])
    probs = torch.empty(1, device="cuda")
    one = int(qpg.qpack_sample(x, u, top_p=p, probs=probs))
    for B in (2, 40, 300):
        many = torch.empty(B, device="cuda")
        tokens = qpg.qpack_sample(x.expand(B, -1).contiguous(), u.expand(B).contiguous(), top_p=p.expand(B).contiguous(),
                                  probs=many)
        assert (tokens == one).all() and (many == probs).all()
    for bad in (x.expand(3, -1),):                         # rows that are one row in memory
        with pytest.raises(qpg.QpackError):
            qpg.qpack_sample(bad, u.expand(3).contiguous())


def test_frequencies(qpg):
    """Evenly spaced random numbers draw each token as often as its probability says, to one draw."""
    n, V = 1000, 40
    x = logits_like(1, V, "f32", 19).expand(n, V).contiguous()
    u = (np.arange(n) + 0.5) / n
    tokens = check(qpg, x, u, np.full(n, 0.8), top_k=np.full(n, 12))
    row = x[0].double().cpu().numpy() / np.float64(np.float32(0.8))
    w = np.exp(row - row.max())
    w[np.argsort(-w, kind="stable")[12:]] = 0
    assert np.all(np.abs(np.bincount(tokens, minlength=V) - n * w / w.sum()) <= 1 + 1e-6)


def test_other_stream_graph_and_nothing_to_do(qpg):
    rng = np.random.default_rng(20)
    x = logits_like(6, 32000, "f32", 21)
    u, p = dev(rng.random(6)), dev(rng.uniform(0.3, 0.9, 6))
    want = qpg.qpack_sample(x, u, top_p=p)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = qpg.qpack_sample(x, u, top_p=p, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.full((8,), 99, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qpg.qpack_sample(x, u, top_p=p, tokens=out)
    x.copy_(logits_like(6, 32000, "f32", 22))
    u.copy_(dev(rng.random(6)))
    want = qpg.qpack_sample(x, u, top_p=p)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[:6], want) and (out[6:] == 99).all()
    assert qpg.qpack_sample(x[:0], u[:0]).shape == (0,)
