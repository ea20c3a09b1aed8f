"""The operators of a decode step of many samples of a few prompts, as they are measured: the norm of query and key heads with
the position rotation in the same pass, attention of one new token a row where groups of rows share a prefix, and the draw of
the next token from its logits.

`run` computes the plain form in elementary torch operations where `own` is false, and calls the library where it is true.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------------------------------------------------------
# The cases
# ---------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # A decode step's queries and keys of 16 samples on a 7B-shaped layer with grouped queries, straight from the fp32
        # product of query, key and value together: latency counts.
        dict(name="heads decode", op="heads", tokens=16, q_heads=32, kv_heads=8, dim=128, turn=128, pairs="half", norm=True,
             x="f32", out="f32"),
        # The prompts of that layer, 8191 tokens at once, in the prefill product's type.
        dict(name="heads prompt", op="heads", tokens=8191, q_heads=32, kv_heads=8, dim=128, turn=128, pairs="half",
             norm=True, x="bf16", out="bf16"),
        # A chunk for half-width heads of which half is rotated, in neighbouring pairs, without norms.
        dict(name="heads part", op="heads", tokens=513, q_heads=27, kv_heads=9, dim=64, turn=32, pairs="neighbours",
             norm=False, x="f16", out="f16"),
        # Four samples of a short prompt: latency counts.
        dict(name="shared short", op="shared", kind="i8", rows=4, groups=1, prefix=97, suffix=3, ragged=False, q_heads=32,
             kv_heads=8, dim=128, page=16, rope=True, q="f32", out="f16"),
        # 64 samples of one long prompt, a few hundred tokens into their answers.
        dict(name="shared samples", op="shared", kind="i8", rows=64, groups=1, prefix=7999, suffix=200, ragged=False,
             q_heads=32, kv_heads=8, dim=128, page=64, rope=True, q="f32", out="f16"),
        # Samples of eight prompts of very different lengths in one batch, half-width heads, a 16-bit cache.
        dict(name="shared prompts", op="shared", kind="bf16", rows=61, groups=8, prefix=4000, suffix=300, ragged=True,
             q_heads=27, kv_heads=9, dim=64, page=32, rope=False, q="bf16", out="bf16"),
        # 32 samples of a very long document on a 70B-shaped layer (64 query heads over 8): the largest.
        dict(name="shared 70B long", op="shared", kind="i8", rows=32, groups=1, prefix=65531, suffix=500, ragged=False,
             q_heads=64, kv_heads=8, dim=128, page=128, rope=False, q="f16", out="f16"),
        # Wide heads, few key heads, small pages.
        dict(name="shared wide", op="shared", kind="f16", rows=17, groups=2, prefix=5000, suffix=100, ragged=True,
             q_heads=16, kv_heads=2, dim=256, page=16, rope=True, q="f16", out="f16"),
        # One user's next token: 32000 logits of a 7B model's product, the usual temperature and top-p.
        dict(name="sample one", op="sample", rows=1, vocab=32000, x="f32", filters="p", masked=0.0),
        # A batch of 64 over a large vocabulary.
        dict(name="sample large", op="sample", rows=64, vocab=128256, x="f32", filters="p", masked=0.0),
        # 256 samples without filters: every token can be drawn.
        dict(name="sample free", op="sample", rows=256, vocab=32000, x="f32", filters="none", masked=0.0),
        # Requests of all kinds together, greedy ones among them, half of the tokens masked, 16-bit logits with many ties.
        dict(name="sample mixed", op="sample", rows=33, vocab=50257, x="bf16", filters="mixed", masked=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["heads", "shared", "shared", "sample", "sample"])
    if op == "heads":
        dim = rng.choice([64, 80, 96, 128, 128, 192, 256])
        kv_heads = _log(rng, 1, 16)
        q_heads = kv_heads * rng.choice([1, 2, 3, 4, 8])
        tokens = _log(rng, 1, min(8192, 8191 * 40 * 128 // ((q_heads + kv_heads) * dim)))
        return dict(op=op, tokens=tokens, q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                    turn=rng.choice([dim, dim, dim // 2 // 8 * 8, 16]), pairs=rng.choice(["half", "neighbours"]),
                    norm=rng.random() < 0.7, x=rng.choice(["f32", "f16", "bf16"]), out=rng.choice(["f32", "f16", "bf16"]))
    if op == "shared":
        kv_heads, group, dim = _log(rng, 1, 16), rng.choice([1, 2, 3, 4, 7, 8, 16]), rng.choice([64, 128, 128, 256])
        rows = _log(rng, 1, 96)
        # at most the largest case's products
        room = 32 * 65531 * 64 * 128 // (2 * rows * kv_heads * group * dim)
        prefix = _log(rng, 1, max(1, min(65536, room)))
        return dict(op=op, kind=rng.choice(["i8", "i8", "f16", "bf16"]), rows=rows, groups=_log(rng, 1, min(rows, 12)),
                    prefix=prefix, suffix=_log(rng, 1, 700), ragged=rng.random() < 0.6, q_heads=kv_heads * group,
                    kv_heads=kv_heads, dim=dim, page=rng.choice([8, 16, 32, 64, 128]), rope=rng.random() < 0.5,
                    q=rng.choice(["f32", "f16", "bf16"]), out=rng.choice(["f16", "bf16"]))
    vocab = _log(rng, 50, 152000)
    return dict(op=op, rows=_log(rng, 1, max(1, min(256, 64 * 128256 // vocab))), vocab=vocab,
                x=rng.choice(["f32", "f32", "f16", "bf16"]), filters=rng.choice(["none", "k", "p", "kp", "min", "mixed"]),
                masked=rng.choice([0.0, 0.0, 0.5, 0.99]))


def _rng(case):
    """Lengths belong to the case, so that work() knows them; values come from the seed."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _shape(case):
    """Rows where the groups begin (one more than groups), their prefixes, the rows' lengths."""
    r, n, g = _rng(case), case["rows"], case["groups"]
    if case["ragged"]:
        first = [0] + sorted(r.sample(range(1, n), g - 1)) + [n]
        prefix = [_log(r, 1, case["prefix"]) for _ in range(g)]
        prefix[0] = case["prefix"]
    else:
        first = [n * i // g for i in range(g + 1)]
        prefix = [case["prefix"] - (i > 0) * r.randint(0, case["prefix"] // 4) for i in range(g)]
    lens = [p + r.randint(0, case["suffix"]) for p, a, b in zip(prefix, first, first[1:]) for _ in range(b - a)]
    if case["ragged"] and n // 2 not in first:
        lens[n // 2] = 0                                    # an idle row of the batch
    return first, prefix, lens


def _elem(case):
    """Bytes of a token's keys and values."""
    d = case["dim"]
    return 2 * case["kv_heads"] * (d * 2 if case["kind"] != "i8" else d + d // 16)


def work(case):
    d = case.get("dim")
    if case["op"] == "heads":
        n = case["tokens"] * (case["q_heads"] + case["kv_heads"]) * d
        return {"bytes": n * (SIZE[case["x"]] + SIZE[case["out"]]) + case["tokens"] * (case["turn"] * 4 + 4), "flops": 8 * n}
    if case["op"] == "shared":
        first, prefix, lens = _shape(case)
        own_tokens = sum(max(0, n - p) for p, a, b in zip(prefix, first, first[1:]) for n in lens[a:b])
        rows = case["rows"] * case["q_heads"]
        return {"bytes": (sum(prefix) + own_tokens) * _elem(case) + rows * (d * (SIZE[case["q"]] + SIZE[case["out"]]) + 4),
                "flops": 4 * sum(lens) * case["q_heads"] * d}
    n = case["rows"] * case["vocab"]
    return {"bytes": n * SIZE[case["x"]] + case["rows"] * 28, "flops": 4 * n}


# ---------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------
def _rope_table(rows, dim):
    """cos | sin of position x frequency, base 10000, fp32."""
    f = 10000.0 ** (-torch.arange(0, dim // 2, dtype=torch.float64) * 2 / dim)
    a = torch.arange(rows, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float().cuda()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _normal(gen, *shape):
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0, 1, generator=gen)


def _uniform(gen, *shape):
    return torch.empty(shape, dtype=torch.float32, device="cuda").uniform_(0, 1, generator=gen)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": dict(case), "op": case["op"]}
    return {"heads": _prepare_heads, "shared": _prepare_shared, "sample": _prepare_sample}[case["op"]](case, seed, gen, s)


def _prepare_heads(case, seed, gen, s):
    n, hq, hk, d = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
    # queries, keys and values of a token side by side, as one product gives them
    x = (_normal(gen, n, hq + 2 * hk, d) * 1.5).to(DTYPES[case["x"]])
    s["q"], s["k"] = x[:, :hq], x[:, hq:hq + hk]
    s["q_weight"], s["k_weight"] = ((1 + 0.2 * _normal(gen, d) if case["norm"] else None) for _ in range(2))
    s["eps"] = 1e-6
    s["rope"] = _rope_table(9000, case["turn"])
    s["pos"] = torch.randint(0, 9000, (n,), device="cuda", generator=gen, dtype=torch.int32)
    s["q_out"] = torch.empty((n, hq, d), dtype=DTYPES[case["out"]], device="cuda")
    s["k_out"] = torch.empty((n, hk, d), dtype=DTYPES[case["out"]], device="cuda")
    return s


def _prepare_shared(case, seed, gen, s):
    cpu = torch.Generator()
    cpu.manual_seed(seed)
    first, prefix, lens = _shape(case)
    t, heads, dim = case["page"], case["kv_heads"], case["dim"]
    # samples forked from their prompts: they hold the same full pages, the rest are their own
    held, at = [], 0
    for p, a, b in zip(prefix, first, first[1:]):
        for i in range(a, b):
            need = -(-lens[i] // t)
            same = held[a][:min(p // t, need)] if i > a else []
            held.append(same + list(range(at, at + need - len(same))))
            at += need - len(same)
    pages = at + 3
    perm = torch.randperm(pages, generator=cpu).tolist()
    width = max(1, max(map(len, held)))
    s["tables"] = _i32([[perm[x] for x in row] + [-1] * (width - len(row)) for row in held])
    s["lens"], s["first"], s["prefix"] = _i32(lens), _i32(first), _i32(prefix)
    s["most"] = [max(b - a for a, b in zip(first, first[1:])),       # rows of a group, tokens behind a prefix
                 max(1, max(n - p for p, a, b in zip(prefix, first, first[1:]) for n in lens[a:b]))]
    shape, s["pool"] = (1, pages, heads, t, dim), {}
    for x in ("k", "v"):
        raw = torch.empty(shape, dtype=torch.float16 if case["kind"] != "bf16" else torch.bfloat16, device="cuda")
        raw.normal_(0, 1, generator=gen)
        if case["kind"] == "i8":
            s["pool"][x] = raw.mul_(50).round_().clamp_(-127, 127).to(torch.int8)
            sc = torch.empty(shape[:-1] + (dim // 32,), dtype=torch.float32, device="cuda")
            s["pool"][x + "_scales"] = sc.normal_(-4, 0.3, generator=gen).exp_().half()
        else:
            s["pool"][x], s["pool"][x + "_scales"] = raw, None
    s["q"] = (2 * _normal(gen, case["rows"], case["q_heads"], dim)).to(DTYPES[case["q"]])
    s["scale"] = 1.0 / math.sqrt(dim)
    s["rope"] = _rope_table(max(lens), dim) if case["rope"] else None
    s["out"] = torch.empty(s["q"].shape, dtype=DTYPES[case["out"]], device="cuda")
    s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    if own:
        import bit_weight_quantized_qpack_gb300 as qp
        p = s["pool"]
        s["kv"] = qp.KVPool(p["k"], p["v"], p["k_scales"], p["v_scales"])
        s["tab"] = qp.KVTables(s["tables"], s["lens"])
        s["workspace"] = qp.alloc_kv_shared_workspace(s["kv"], case["rows"], case["q_heads"])
    return s


def _prepare_sample(case, seed, gen, s):
    b, v = case["rows"], case["vocab"]
    # a broad floor of unlikely tokens and a few dozen that the context calls for
    x = 2.0 * _normal(gen, b, v)
    hot = torch.randint(0, v, (b, min(v, 40)), device="cuda", generator=gen)
    x.scatter_add_(1, hot, 6 + 4 * -_uniform(gen, *hot.shape).clamp(min=1e-6).log())
    if case["masked"]:
        x.masked_fill_(_uniform(gen, b, v) < case["masked"], float("-inf"))
        if b > 2:
            x[b // 2] = float("-inf")                       # a grammar that leaves nothing
    s["logits"] = x.to(DTYPES[case["x"]])
    f = case["filters"]
    s["temperature"] = 0.5 + _uniform(gen, b)
    s["top_k"] = torch.randint(1, 100, (b,), device="cuda", generator=gen, dtype=torch.int32) if f in ("k", "kp", "mixed") \
        else None
    s["top_p"] = 0.8 + 0.19 * _uniform(gen, b) if f in ("p", "kp", "mixed") else None
    s["min_p"] = 0.1 * _uniform(gen, b) if f in ("min", "mixed") else None
    if f == "mixed":                                        # each filter left out by two rows of three, every seventh row greedy
        i = torch.arange(b, device="cuda")
        s["top_k"] = torch.where(i % 3 == 0, s["top_k"], torch.zeros_like(s["top_k"]))
        s["top_p"] = torch.where(i % 3 == 1, s["top_p"], torch.ones_like(s["top_p"]))
        s["min_p"] = torch.where(i % 3 == 2, s["min_p"], torch.zeros_like(s["min_p"]))
        s["temperature"] = torch.where(i % 7 == 6, torch.zeros_like(s["temperature"]), s["temperature"])
    s["u"] = _uniform(gen, b).clamp(max=1 - 2.0 ** -24)
    s["tokens"] = torch.empty(b, dtype=torch.int32, device="cuda")
    s["probs"] = torch.empty(b, dtype=torch.float32, device="cuda")
    return s


# ---------------------------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------------------------
def run(state):
    return _RUN[state["op"], own](state)


def _turned(x, rows, pairs):
    """x [..., heads, dim] fp32, its first elements rotated by rows [..., turn] of the cos | sin table."""
    turn = rows.shape[-1]
    c, s = rows[..., None, :].chunk(2, -1)
    part, rest = x[..., :turn], x[..., turn:]
    if pairs == "half":
        a, b = part.chunk(2, -1)
        return torch.cat([a * c - b * s, b * c + a * s, rest], -1)
    a, b = part[..., 0::2], part[..., 1::2]
    return torch.cat([torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2), rest], -1)


def _heads_plain(s):
    case, got = s["case"], {}
    rows = s["rope"][s["pos"].long()]
    for x in ("q", "k"):
        y = s[x].float()
        if s[x + "_weight"] is not None:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + s["eps"]) * s[x + "_weight"]
        got[x] = _turned(y, rows, case["pairs"]).to(s[x + "_out"].dtype)
    return got


def _heads_own(s):
    import bit_weight_quantized_qpack_gb300 as qp
    qp.qpack_qk_norm_rope(s["q"], s["k"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"], rope=s["rope"],
                          interleaved=s["case"]["pairs"] != "half", pos=s["pos"], q_out=s["q_out"], k_out=s["k_out"])
    return {"q": s["q_out"], "k": s["k_out"]}


def _values(codes, scales):
    """The numbers a cache holds, in fp32: an 8-bit element is its code times its group's scale, rounded to fp16."""
    if scales is None:
        return codes.float()
    return (codes.float() * scales.float().repeat_interleave(32, -1)).half().float()


def _shared_plain(s):
    case, pool, t = s["case"], s["pool"], s["case"]["page"]
    b, h, d, n_groups = case["rows"], case["kv_heads"], case["dim"], case["groups"]
    g, (per, more), dev = case["q_heads"] // h, s["most"], s["q"].device
    lens, first, prefix = s["lens"].long(), s["first"].long(), s["prefix"].long()
    row = torch.arange(b, device=dev)
    of = torch.searchsorted(first, row, right=True) - 1     # a row's group, and its place there
    at = row - first[of]
    q = s["q"].float()
    if s["rope"] is not None:
        q = _turned(q, s["rope"][(lens - 1).clamp(min=0)], "half")
    q = q.view(b, h, g, d) * s["scale"]
    # the prefixes, once a group
    wide = -(-case["prefix"] // t)
    pages = s["tables"][first[:-1], :wide].clamp(min=0).long()
    part = lambda x: None if x is None else x[0][pages].transpose(1, 2).reshape(n_groups, h, wide * t, -1)  # noqa: E731
    pos = torch.arange(wide * t, device=dev)
    qs = q.new_zeros((n_groups, per, h, g, d))
    qs[of, at] = q
    qs = qs.transpose(1, 2).reshape(n_groups, h, per * g, d)
    score = (qs @ _values(part(pool["k"]), part(pool["k_scales"])).transpose(2, 3)).view(n_groups, h, per, g, wide * t)
    score = score.transpose(1, 2)[of, at]                   # [rows, h, g, tokens]
    score = score.masked_fill((pos >= torch.minimum(lens, prefix[of])[:, None])[:, None, None], float("-inf"))
    # what the rows have of their own
    mine = prefix[of][:, None] + torch.arange(more, device=dev)
    page = s["tables"].gather(1, (mine // t).clamp(max=s["tables"].shape[1] - 1)).clamp(min=0).long()
    rows = lambda x: None if x is None else x[0].transpose(1, 2)[page, mine % t].transpose(1, 2)  # noqa: E731
    score2 = q @ _values(rows(pool["k"]), rows(pool["k_scales"])).transpose(2, 3)
    beyond = mine >= lens[:, None]
    score2 = score2.masked_fill(beyond[:, None, None], float("-inf"))
    top = torch.maximum(score.amax(-1, keepdim=True), score2.amax(-1, keepdim=True))
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    p, p2 = (score - top).exp(), (score2 - top).exp()
    total = p.sum(-1, keepdim=True) + p2.sum(-1, keepdim=True)
    ps = p.new_zeros((n_groups, per, h, g, wide * t))
    ps[of, at] = p
    v = _values(part(pool["v"]), part(pool["v_scales"]))
    o = (ps.transpose(1, 2).reshape(n_groups, h, per * g, -1) @ v).view(n_groups, h, per, g, d).transpose(1, 2)[of, at]
    o = o + p2 @ _values(rows(pool["v"]), rows(pool["v_scales"])).masked_fill(beyond[:, None, :, None], 0.0)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    return {"out": o.view(b, h * g, d).to(s["out"].dtype), "lse": (total.log() + top).view(b, h * g)}


def _shared_own(s):
    import bit_weight_quantized_qpack_gb300 as qp
    qp.qpack_kv_attend_shared(s["kv"], 0, s["tab"], s["q"], s["first"], s["prefix"], scale=s["scale"], rope=s["rope"],
                              out=s["out"], lse=s["lse"], workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def _sample_plain(s):
    x, v = s["logits"].float(), s["logits"].shape[1]
    col = torch.arange(v, device=x.device)
    top = x.amax(1, keepdim=True)
    greedy = (s["temperature"] <= 0)[:, None]
    heat = torch.where(greedy, 1.0, s["temperature"][:, None]).double()
    lead = torch.where(x == top, col, v).amin(1, keepdim=True)
    # weights and their sums in 64 bits: a token is told from its neighbour by the last place of a sum
    w = torch.where(x == float("-inf"), 0.0, ((x.double() - top.double()) / heat).exp())
    w = torch.where(greedy, (col == lead).double(), w)
    order = x.sort(dim=1, descending=True, stable=True).indices
    down = w.gather(1, order)
    keep = torch.ones_like(down, dtype=torch.bool)
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        keep = keep & ((col < k) | (k <= 0))
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        inside = down * keep
        before = inside.cumsum(1) - inside
        keep = keep & ((before < p * inside.sum(1, keepdim=True)) | (p >= 1) | (col == 0))
    if s["min_p"] is not None:
        keep = keep & (down >= s["min_p"].double()[:, None])
    w = torch.zeros_like(w).scatter_(1, order, down * keep)
    sums = w.cumsum(1)
    total = sums[:, -1:]
    at = (sums <= s["u"].double()[:, None] * total).sum(1, keepdim=True)
    at = torch.minimum(at, torch.where(w > 0, col, 0).amax(1, keepdim=True))
    none = top == float("-inf")
    token = torch.where(none, -1, at)
    prob = torch.where(none, 0.0, w.gather(1, at) / total)
    return {"tokens": token[:, 0].int(), "probs": prob[:, 0].float()}


def _sample_own(s):
    import bit_weight_quantized_qpack_gb300 as qp
    qp.qpack_sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                    min_p=s["min_p"], tokens=s["tokens"], probs=s["probs"])
    return {"tokens": s["tokens"], "probs": s["probs"]}


_RUN = {("heads", False): _heads_plain, ("heads", True): _heads_own, ("shared", False): _shared_plain,
        ("shared", True): _shared_own, ("sample", False): _sample_plain, ("sample", True): _sample_own}


# ---------------------------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def _turn64(x, row, pairs="half"):
    """Heads [..., dim] in fp64 times e^{i angle}, by rows [..., turn] of the table that broadcast over the heads."""
    half = row.shape[-1] // 2
    z = torch.complex(row[..., :half].double(), row[..., half:].double())
    part = x[..., :2 * half]
    part = torch.stack([part[..., :half], part[..., half:]], -1) if pairs == "half" else part.unflatten(-1, (half, 2))
    got = torch.view_as_real(torch.view_as_complex(part.contiguous()) * z)
    got = got.transpose(-1, -2).flatten(-2) if pairs == "half" else got.flatten(-2)
    return torch.cat([got, x[..., 2 * half:]], -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "heads":
        got = {}
        for x in ("q", "k"):
            y = s[x].double()
            if case["norm"]:
                y = s[x + "_weight"].double() * y / (y.pow(2).sum(-1, keepdim=True) / case["dim"] + s["eps"]).sqrt()
            got[x] = _turn64(y, s["rope"][s["pos"].long()][:, None], case["pairs"])
        return got
    if case["op"] == "shared":
        return _exact_shared(case, s)
    return _exact_sample(s)


def _exact_shared(case, s):
    first, prefix, lens = _shape(case)
    t, g, dev = case["page"], case["q_heads"] // case["kv_heads"], "cuda"
    outs, lses = [], []
    for p, a, b in zip(prefix, first, first[1:]):
        for i in range(a, b):
            n = lens[i]
            if n == 0:
                outs.append(torch.zeros(s["q"].shape[1:], dtype=torch.float64, device=dev))
                lses.append(torch.full((case["q_heads"],), float("-inf"), dtype=torch.float64, device=dev))
                continue
            pos = torch.arange(n, device=dev)
            ids = torch.where(pos < p, s["tables"][a][pos // t], s["tables"][i][pos // t]).long()

            def held(x):
                c = s["pool"][x][0][ids, :, pos % t].double()
                d = s["pool"][x + "_scales"]
                return c if d is None else (c * d[0][ids, :, pos % t].double().repeat_interleave(32, 2)).half().double()

            q = s["q"][i].double()
            if s["rope"] is not None:
                q = _turn64(q, s["rope"][n - 1])
            sc = torch.einsum("hgd,nhd->hgn", q.view(-1, g, case["dim"]), held("k")) * s["scale"]
            lses.append(sc.logsumexp(-1).flatten())
            outs.append(torch.einsum("hgn,nhd->hgd", sc.softmax(-1), held("v")).reshape(q.shape))
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}


def _exact_sample(s):
    """Row by row on the host, by the definition's words."""
    x = s["logits"].double().cpu()
    given = {k: None if s[k] is None else s[k].double().tolist() for k in ("temperature", "top_k", "top_p", "min_p", "u")}
    tokens, probs = [], []
    for i, row in enumerate(x):
        one = {k: None if v is None else v[i] for k, v in given.items()}
        top = float(row.max())
        if top == float("-inf"):
            tokens.append(-1), probs.append(0.0)
            continue
        if one["temperature"] <= 0:
            tokens.append(int(torch.nonzero(row == top)[0])), probs.append(1.0)
            continue
        ids = torch.nonzero(row > float("-inf"))[:, 0]
        ids = ids[torch.sort(row[ids], descending=True, stable=True).indices]
        w = ((row[ids] - top) / one["temperature"]).exp()
        if one["top_k"] and one["top_k"] > 0:
            ids, w = ids[:int(one["top_k"])], w[:int(one["top_k"])]
        if one["top_p"] is not None and one["top_p"] < 1:
            few = 1 + int((w.cumsum(0) < one["top_p"] * w.sum()).sum())
            ids, w = ids[:few], w[:few]
        if one["min_p"]:
            ids, w = ids[w >= one["min_p"]], w[w >= one["min_p"]]
        up = ids.sort().indices
        sums = w[up].cumsum(0)
        at = up[min(int((sums <= one["u"] * sums[-1]).sum()), len(up) - 1)]
        tokens.append(int(ids[at])), probs.append(float(w[at] / sums[-1]))
    return {"tokens": torch.tensor(tokens, dtype=torch.int32), "probs": torch.tensor(probs, dtype=torch.float64)}
