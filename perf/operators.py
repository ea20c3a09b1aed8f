"""The paged KV-cache operators as they are measured: attention of one new token over the cache, appending new tokens
(rotary embedding, 8-bit quantization, scatter into pages) and reading them back, and the page operators that share,
release, extend and compact the cache.

A cache pool holds `layers` x `pages` pages of `page` tokens for `kv_heads` heads of `dim` elements: keys and values
[layers, pages, kv_heads, page, dim], in 8 bits with one fp16 scale per 32 elements ("i8"), or in 16 bits ("f16",
"bf16"). A sequence is a row of the page table, its length, and every page has a reference count.

`run` computes the plain form in elementary torch operations where `own` is false, and calls the library where it is
true. Both work on the state's own buffers.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------------------------------------------
# The cases
# ---------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # One user's short prompt on a 7B-shaped layer with grouped queries (32 query heads over 8): latency counts.
        dict(name="attend one short", op="attend", kind="i8", batch=1, longest=97, ragged=False, q_heads=32, kv_heads=8,
             dim=128, page=16, window=0, rope=True, q="f32", out="f16"),
        # Continuous batching on the same layer: 16 sequences of very different lengths, one of them empty.
        dict(name="attend ragged batch", op="attend", kind="i8", batch=16, longest=8191, ragged=True, q_heads=32,
             kv_heads=8, dim=128, page=64, window=0, rope=True, q="f32", out="f16"),
        # A full batch on a 70B-shaped layer (64 query heads over 8) at long contexts: the largest cache read.
        dict(name="attend 70B batch", op="attend", kind="i8", batch=64, longest=8192, ragged=False, q_heads=64,
             kv_heads=8, dim=128, page=64, window=0, rope=False, q="f16", out="f16"),
        # One very long document: few rows, so the cache's length has to be split.
        dict(name="attend one long", op="attend", kind="i8", batch=1, longest=131071, ragged=False, q_heads=32,
             kv_heads=8, dim=128, page=128, window=0, rope=True, q="f32", out="f16"),
        # A 16-bit cache, three query heads a key head, half-width heads, a sliding window and odd lengths.
        dict(name="attend 16-bit window", op="attend", kind="bf16", batch=7, longest=5001, ragged=True, q_heads=27,
             kv_heads=9, dim=64, page=32, window=4095, rope=False, q="bf16", out="bf16"),
        # The decode step's write: one new token for each of 16 sequences, straight from the fp32 products.
        dict(name="append decode", op="append", kind="i8", tokens=16, seqs=16, kv_heads=8, dim=128, page=64, rope=True,
             x="f32"),
        # A prompt of three ragged sequences written after its prefill and read back.
        dict(name="append prefill", op="append", kind="i8", tokens=8191, seqs=3, kv_heads=8, dim=128, page=64,
             rope=True, x="f16"),
        # A chunk of a multi-head (32 heads) model into a 16-bit cache.
        dict(name="append 16-bit chunk", op="append", kind="bf16", tokens=513, seqs=5, kv_heads=32, dim=128, page=32,
             rope=False, x="bf16"),
        # One search step: four beams forked from two prompts, two layers.
        dict(name="fork beams", op="fork", kind="f16", layers=2, parents=2, children=4, longest=301, kv_heads=8, dim=128,
             page=16),
        # 64 samples of eight long prompts through the 32 layers of a 7B-shaped cache.
        dict(name="fork samples", op="fork", kind="f16", layers=32, parents=8, children=64, longest=4000, kv_heads=8,
             dim=128, page=16),
        # A small cache after some sequences ended.
        dict(name="compact small", op="compact", kind="f16", layers=2, pages=150, live=0.6, kv_heads=8, dim=128,
             page=16),
        # A 32-layer cache at half load.
        dict(name="compact 32 layers", op="compact", kind="bf16", layers=32, pages=1200, live=0.5, kv_heads=8, dim=128,
             page=16),
    ]


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))
    return n - (n == 3 << 10)


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "append", "fork", "compact"])
    kind = rng.choice(["i8", "i8", "f16", "bf16"])
    dim = rng.choice([64, 128, 128, 256])
    if op == "attend":
        kv_heads, group = _log(rng, 1, 32), rng.choice([1, 2, 3, 4, 5, 7, 8, 11, 16])
        kv_heads += kv_heads * group * dim == 3 << 10
        batch = _log(rng, 1, 96)
        # cache elements at most half the largest case's, in bytes of either kind
        room = 64 * 8192 * 8 * 128 // 2 // (batch * kv_heads * dim)
        longest = _log(rng, 1, max(1, min(65536, room)))
        window = rng.choice([0, 0, 0, _log(rng, 1, longest)])
        return dict(op=op, kind=kind, batch=batch, longest=longest, ragged=rng.random() < 0.6, q_heads=kv_heads * group,
                    kv_heads=kv_heads, dim=dim, page=rng.choice([8, 16, 32, 64, 128]), window=window,
                    rope=rng.random() < 0.5, q=rng.choice(["f32", "f16", "bf16"]), out=rng.choice(["f16", "bf16"]))
    if op == "append":
        seqs = _log(rng, 1, 64)
        return dict(op=op, kind=kind, tokens=max(seqs, _log(rng, 1, 12000)), seqs=seqs, kv_heads=rng.choice([1, 2, 5, 8, 16]),
                    dim=dim, page=rng.choice([8, 16, 32, 64, 128]), rope=rng.random() < 0.6,
                    x=rng.choice(["f32", "f16", "bf16"]))
    kind = rng.choice(["f16", "bf16"])
    if op == "fork":
        return dict(op=op, kind=kind, layers=_log(rng, 1, 24), parents=_log(rng, 1, 8), children=_log(rng, 1, 60),
                    longest=_log(rng, 2, 1500), kv_heads=rng.choice([1, 2, 5, 8]), dim=dim,
                    page=rng.choice([8, 16, 32]))
    return dict(op=op, kind=kind, layers=_log(rng, 1, 24), pages=_log(rng, 8, 500), live=round(rng.uniform(0.1, 0.95), 3),
                kv_heads=rng.choice([1, 2, 5, 8]), dim=dim, page=rng.choice([8, 16, 32]))


def _rng(case):
    """Lengths and page numbers belong to the case, so that work() knows them; values come from the seed."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _lens(case):
    r, n, top = _rng(case), case["batch"], case["longest"]
    if case["ragged"]:
        lens = [_log(r, 1, top) for _ in range(n)]
        if n > 2:
            lens[n // 2] = 0                                # an idle row of the batch
    else:
        lens = [r.randint((top + 1) // 2, top) for _ in range(n)]
    lens[0] = top
    return lens


def _fork_lens(case):
    r, top = _rng(case), case["longest"]
    return [r.randint(max(1, top // 2), top) for _ in range(case["parents"])]


def _split(case):
    """Tokens a sequence appends, and the length that it had before."""
    r, n = _rng(case), case["seqs"]
    cuts = sorted(r.sample(range(1, case["tokens"]), n - 1)) if n > 1 else []
    new = [b - a for a, b in zip([0] + cuts, cuts + [case["tokens"]])]
    return new, [r.randint(0, 200) for _ in range(n)]


def _live(case):
    r, p = _rng(case), case["pages"]
    ids = list(range(p))
    r.shuffle(ids)
    return ids[:max(1, int(p * case["live"]))]


def _moves(case):
    live = _live(case)
    return sum(i >= len(live) for i in live)


def _page_bytes(case, rows):
    """Bytes of `rows` tokens in keys and values of one layer."""
    per = case["dim"] * 2 if case["kind"] != "i8" else case["dim"] + case["dim"] // 16
    return 2 * rows * case["kv_heads"] * per


SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def work(case):
    op, d = case["op"], case["dim"]
    if op == "attend":
        seen = sum(min(n, case["window"]) if case["window"] else n for n in _lens(case))
        rows = case["batch"] * case["q_heads"]
        return {"bytes": _page_bytes(case, seen) + rows * (d * (SIZE[case["q"]] + SIZE[case["out"]]) + 4),
                "flops": 4 * seen * case["q_heads"] * d}
    if op == "append":                                      # in, to the cache, from the cache, out
        n = 2 * case["tokens"] * case["kv_heads"] * d
        return {"bytes": n * (SIZE[case["x"]] + 2) + 2 * _page_bytes(case, case["tokens"]), "flops": 6 * n}
    if op == "fork":
        lens, t = _fork_lens(case), case["page"]
        got = [lens[i % len(lens)] for i in range(case["children"])]
        rows = sum(n % t for n in got)
        return {"bytes": 2 * case["layers"] * _page_bytes(case, rows) + 8 * sum(-(-n // t) for n in got) + 4096, "flops": 0}
    return {"bytes": 2 * case["layers"] * _page_bytes(case, case["page"] * _moves(case)) + 16 * case["pages"] + 4096,
            "flops": 0}


# ---------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------
def _pool(case, gen, layers, pages):
    """Keys and values as they come: unit normal; 8-bit codes fill their groups' range."""
    dev = "cuda"
    shape = (layers, pages, case["kv_heads"], case["page"], case["dim"])
    pool = {}
    for x in ("k", "v"):
        raw = torch.empty(shape, dtype=torch.float16 if case["kind"] != "bf16" else torch.bfloat16, device=dev)
        raw.normal_(0, 1, generator=gen)
        if case["kind"] == "i8":
            pool[x] = raw.mul_(50).round_().clamp_(-127, 127).to(torch.int8)
            sc = torch.empty(shape[:-1] + (case["dim"] // 32,), dtype=torch.float32, device=dev)
            pool[x + "_scales"] = sc.normal_(-4, 0.3, generator=gen).exp_().half()
        else:
            pool[x] = raw
            pool[x + "_scales"] = None
    return pool


def _rope_table(rows, dim):
    """cos | sin of position x frequency, base 10000, fp32."""
    f = 10000.0 ** (-torch.arange(0, dim // 2, dtype=torch.float64) * 2 / dim)
    a = torch.arange(rows, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float().cuda()


def _tables(lens, page, pages, perm, width=None):
    """Page table [rows, width] on the host: rows take their pages from `perm` in turn."""
    need = [-(-n // page) for n in lens]
    width = max([1] + need) if width is None else width
    t = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        t[i, :n] = perm[at:at + n]
        at += n
    assert at <= pages
    return t


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    cpu = torch.Generator()
    cpu.manual_seed(seed)
    s = {"case": dict(case), "op": case["op"]}
    page, heads, dim = case["page"], case["kv_heads"], case["dim"]
    if case["op"] == "attend":
        lens = _lens(case)
        pages = sum(-(-n // page) for n in lens) + 3
        s["pool"] = _pool(case, gen, 1, pages)
        s["tables"] = _tables(lens, page, pages, torch.randperm(pages, generator=cpu).int()).cuda()
        s["lens"] = _i32(lens)
        q = torch.empty((case["batch"], case["q_heads"], dim), dtype=torch.float32, device="cuda")
        s["q"] = q.normal_(0, 2, generator=gen).to(DTYPES[case["q"]])
        s["scale"] = 1.0 / math.sqrt(dim)
        s["rope"] = _rope_table(max(lens), dim) if case["rope"] else None
        s["out"] = torch.empty(q.shape, dtype=DTYPES[case["out"]], device="cuda")
        s["lse"] = torch.empty(q.shape[:2], dtype=torch.float32, device="cuda")
    elif case["op"] == "append":
        new, had = _split(case)
        lens = [a + b for a, b in zip(new, had)]
        pages = sum(-(-n // page) for n in lens) + 3
        s["pool"] = _pool(case, gen, 1, pages)
        s["tables"] = _tables(lens, page, pages, torch.randperm(pages, generator=cpu).int()).cuda()
        s["lens"] = _i32(lens)
        s["seqs"] = _i32([i for i, n in enumerate(new) for _ in range(n)])
        s["pos"] = _i32([h + j for n, h in zip(new, had) for j in range(n)])
        x = torch.empty((2, case["tokens"], heads, dim), dtype=torch.float32, device="cuda").normal_(0, 1, generator=gen)
        s["k"], s["v"] = x.to(DTYPES[case["x"]]).unbind(0)
        s["rope"] = _rope_table(max(lens), dim) if case["rope"] else None
        s["k_out"] = torch.empty((case["tokens"], heads, dim), device="cuda",
                                 dtype=torch.bfloat16 if case["kind"] == "bf16" else torch.float16)
        s["v_out"] = torch.empty_like(s["k_out"])
    elif case["op"] == "fork":
        lens = _fork_lens(case)
        n, c = len(lens), case["children"]
        width = -(-(max(lens) + 1) // page)
        used = sum(-(-m // page) for m in lens)
        pages = used + 2 * c + 5
        s["pool"] = _pool(case, gen, case["layers"], pages)
        perm = torch.randperm(pages, generator=cpu).int()
        tables = torch.full((n + c, width), -1, dtype=torch.int32)
        tables[:n] = _tables(lens, page, pages, perm, width)
        refs = torch.zeros(pages, dtype=torch.int32)
        refs[perm[:used].long()] = 1
        s["tables"], s["refs"], s["lens"] = tables.cuda(), refs.cuda(), _i32(lens + [0] * c)
        s["src"], s["dst"] = _i32([i % n for i in range(c)]), _i32([n + i for i in range(c)])
        s["add"] = _i32([1] * c)
    else:
        live, pages = _live(case), case["pages"]
        s["pool"] = _pool(case, gen, case["layers"], pages)
        refs = torch.zeros(pages, dtype=torch.int32)
        refs[torch.tensor(live)] = torch.randint(1, 4, (len(live),), generator=cpu, dtype=torch.int32)
        width = 32                                          # eight-page ragged rows, in the shuffled order
        rows, at, r = [], 0, _rng(case)
        while at < len(live):
            m = r.randint(1, width)
            rows.append(live[at:at + m] + [-1] * (width - len(live[at:at + m])))
            at += m
        s["tables"], s["refs"] = _i32(rows), refs.cuda()
        s["lens"] = _i32([sum(x >= 0 for x in row) * page for row in rows])
        s["tables_out"], s["refs_out"] = torch.empty_like(s["tables"]), torch.empty_like(s["refs"])
        s["moved"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if own:
        import bit_weight_quantized_qpack_gb300 as qp
        p = s["pool"]
        s["kv"] = qp.KVPool(p["k"], p["v"], p["k_scales"], p["v_scales"])
        s["tab"] = qp.KVTables(s["tables"], s["lens"], s.get("refs"))
        if case["op"] == "attend":
            s["workspace"] = qp.alloc_kv_workspace(s["kv"], case["batch"], case["q_heads"])
        elif case["op"] != "append":
            s["workspace"] = qp.alloc_kv_page_workspace(s["kv"], s["tab"])
    return s


# ---------------------------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------------------------
def run(state):
    return _RUN[state["op"], own](state)


def _values(codes, scales):
    """The numbers a cache holds, in fp32: an 8-bit element is its code times its group's scale, rounded to fp16."""
    if scales is None:
        return codes.float()
    wide = scales.float().repeat_interleave(32, -1)
    return (codes.float() * wide).half().float()


def _rotate(x, rows):
    """x [..., heads, dim] fp32, rows [..., dim] of the cos | sin table."""
    c, s = rows[..., None, :].chunk(2, -1)
    a, b = x.chunk(2, -1)
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _attend_plain(s):
    case, pool = s["case"], s["pool"]
    b, h, d, t = case["batch"], case["kv_heads"], case["dim"], case["page"]
    g, width = case["q_heads"] // h, s["tables"].shape[1]
    lens = s["lens"].long()
    q = s["q"].float()
    if s["rope"] is not None:
        q = _rotate(q, s["rope"][(lens - 1).clamp(min=0)])
    at = s["tables"].clamp(min=0).long()
    part = lambda x: None if x is None else x[0][at].transpose(1, 2).reshape(b, h, width * t, -1)  # noqa: E731
    pos = torch.arange(width * t, device=q.device)
    seen = pos < lens[:, None]
    if case["window"]:
        seen = seen & (pos >= lens[:, None] - case["window"])
    seen = seen[:, None, None]
    score = q.view(b, h, g, d) @ _values(part(pool["k"]), part(pool["k_scales"])).transpose(2, 3) * s["scale"]
    score = score.masked_fill(~seen, float("-inf"))
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    v = _values(part(pool["v"]), part(pool["v_scales"])).masked_fill(~seen.transpose(2, 3), 0.0)
    o = (p @ v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (total.log() + top).view(b, h * g)
    return {"out": o.view(b, h * g, d).to(s["out"].dtype), "lse": lse}


def _attend_own(s):
    import bit_weight_quantized_qpack_gb300 as qp
    qp.qpack_kv_attend(s["kv"], 0, s["tab"], s["q"], scale=s["scale"], window=s["case"]["window"], rope=s["rope"],
                       out=s["out"], lse=s["lse"], workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def _append_plain(s):
    case, pool, t = s["case"], s["pool"], s["case"]["page"]
    seqs, pos = s["seqs"].long(), s["pos"].long()
    page, slot = s["tables"][seqs, pos // t].long(), pos % t
    got = {}
    for x in ("k", "v"):
        new = s[x].float()
        if x == "k" and s["rope"] is not None:
            new = _rotate(new, s["rope"][pos])
        if case["kind"] == "i8":
            group = new.view(new.shape[:-1] + (-1, 32))
            scale = (group.abs().amax(-1) / 127).half()
            wide = scale.float()[..., None]
            code = torch.where(wide > 0, (group / wide).round().clamp(-127, 127), torch.zeros_like(group))
            pool[x][0].index_put_((page, torch.arange(case["kv_heads"], device=page.device)[:, None], slot),
                                  code.view(new.shape).to(torch.int8).transpose(0, 1))
            pool[x + "_scales"][0].index_put_((page, torch.arange(case["kv_heads"], device=page.device)[:, None], slot),
                                              scale.transpose(0, 1))
        else:
            pool[x][0].index_put_((page, torch.arange(case["kv_heads"], device=page.device)[:, None], slot),
                                  new.to(pool[x].dtype).transpose(0, 1))
        sc = pool[x + "_scales"]
        back = _values(pool[x][0][page, :, slot], None if sc is None else sc[0][page, :, slot])
        got[x] = back.to(s["k_out"].dtype)
    return got


def _append_own(s):
    import bit_weight_quantized_qpack_gb300 as qp
    qp.qpack_kv_append(s["kv"], 0, s["tab"], s["k"], s["v"], seqs=s["seqs"], pos=s["pos"], rope=s["rope"])
    qp.qpack_kv_read(s["kv"], 0, s["tab"], s["seqs"], s["pos"], k_out=s["k_out"], v_out=s["v_out"])
    return {"k": s["k_out"], "v": s["v_out"]}


def _free_order(refs):
    """Every page, the free ones first and in rising order."""
    return (refs > 0).int().argsort(stable=True)


def _fork_plain(s):
    """A search step: the children of the last one are freed, new ones forked and extended by a token each."""
    tables, lens, refs, pool, t = s["tables"], s["lens"], s["refs"], s["pool"], s["case"]["page"]
    src, dst, width = s["src"].long(), s["dst"].long(), s["tables"].shape[1]
    old = tables[dst]
    refs.index_add_(0, old.clamp(min=0).flatten().long(), -(old >= 0).int().flatten())
    col = torch.arange(width, device=tables.device)
    n = lens[src].long()
    full, rows = n // t, n % t
    parent = tables[src]
    share = col < full[:, None]
    free = _free_order(refs)
    refs.index_add_(0, parent.clamp(min=0).flatten().long(), share.int().flatten())
    child = torch.where(share, parent, -1)
    need = rows > 0
    fresh = free[(need.cumsum(0) - 1).clamp(min=0)]
    child = torch.where((col == full[:, None]) & need[:, None], fresh[:, None].int(), child)
    last = parent.gather(1, full.clamp(max=width - 1)[:, None])[:, 0]
    # a child that needs no page copies its first page onto itself
    a = torch.where(need, last, parent[:, 0]).clamp(min=0).long()
    b = torch.where(need, fresh, a)
    keep = (torch.arange(t, device=tables.device) < rows[:, None])[:, None, :, None]
    for x in ("k", "v"):
        pool[x][:, b] = torch.where(keep, pool[x][:, a], pool[x][:, b])
    refs.index_add_(0, fresh, need.int())
    lens[dst] = n.int()
    grow = (n + s["add"] + t - 1) // t > (n + t - 1) // t
    more = _free_order(refs)[(grow.cumsum(0) - 1).clamp(min=0)]
    tables[dst] = torch.where((col == ((n + t - 1) // t)[:, None]) & grow[:, None], more[:, None].int(), child)
    refs.index_add_(0, more, grow.int())
    lens[dst] += s["add"]
    return {"tables": tables, "lens": lens, "refs": refs, "k": pool["k"], "v": pool["v"]}


def _fork_own(s):
    import bit_weight_quantized_qpack_gb300 as qp
    kv, tab, ws = s["kv"], s["tab"], s["workspace"]
    qp.qpack_kv_free(tab, s["dst"])
    qp.qpack_kv_fork(kv, tab, s["src"], s["dst"], workspace=ws)
    qp.qpack_kv_reserve(kv, tab, s["dst"], s["add"])
    return {"tables": s["tables"], "lens": s["lens"], "refs": s["refs"], "k": s["pool"]["k"], "v": s["pool"]["v"]}


def _compact_plain(s):
    refs, tables, pool = s["refs"], s["tables"], s["pool"]
    ids = torch.arange(refs.numel(), device=refs.device)
    live = refs > 0
    n = live.sum()
    a = torch.nonzero(live & (ids >= n))[:, 0]
    b = torch.nonzero(~live & (ids < n))[:, 0]
    new = ids.clone()
    new[a] = b
    for x in ("k", "v"):
        pool[x][:, b] = pool[x][:, a]
    s["refs_out"].copy_(torch.where(ids < n, refs[new.clone().index_copy_(0, b, a)], 0))
    s["tables_out"].copy_(torch.where(tables >= 0, new[tables.clamp(min=0).long()].int(), tables))
    s["moved"].fill_(a.numel())
    return {"tables": s["tables_out"], "refs": s["refs_out"], "moved": s["moved"], "k": pool["k"], "v": pool["v"]}


def _compact_own(s):
    import bit_weight_quantized_qpack_gb300 as qp
    qp.qpack_kv_compact(s["kv"], s["tab"], tables_out=s["tables_out"], refs_out=s["refs_out"], moved=s["moved"],
                        workspace=s["workspace"])
    return {"tables": s["tables_out"], "refs": s["refs_out"], "moved": s["moved"], "k": s["pool"]["k"],
            "v": s["pool"]["v"]}


_RUN = {("attend", False): _attend_plain, ("attend", True): _attend_own, ("append", False): _append_plain,
        ("append", True): _append_own, ("fork", False): _fork_plain, ("fork", True): _fork_own,
        ("compact", False): _compact_plain, ("compact", True): _compact_own}


# ---------------------------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def _turn64(x, row):
    """One token's heads [heads, dim] in fp64 and its fp32 table row."""
    half = x.shape[-1] // 2
    c, s = row[:half].double(), row[half:].double()
    return torch.cat([x[:, :half] * c - x[:, half:] * s, x[:, half:] * c + x[:, :half] * s], 1)


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None                                         # whole numbers, and pages copied bit for bit
    s = prepare(case, seed)
    pool, t = s["pool"], case["page"]

    def held(x, ids, slots):
        """Cache rows [tokens, heads, dim] of layer 0 in fp64."""
        c = pool[x][0][ids, :, slots].double()
        if pool[x + "_scales"] is None:
            return c
        d = pool[x + "_scales"][0][ids, :, slots].double()
        return (c * d.repeat_interleave(32, 2)).half().double()

    if case["op"] == "attend":
        outs, lses = [], []
        g = case["q_heads"] // case["kv_heads"]
        for b, n in enumerate(_lens(case)):
            if n == 0:
                outs.append(torch.zeros(s["q"].shape[1:], dtype=torch.float64, device="cuda"))
                lses.append(torch.full((case["q_heads"],), float("-inf"), dtype=torch.float64, device="cuda"))
                continue
            q = s["q"][b].double()
            if s["rope"] is not None:
                q = _turn64(q, s["rope"][n - 1])
            pos = torch.arange(max(0, n - case["window"]) if case["window"] else 0, n, device="cuda")
            ids, slots = s["tables"][b][pos // t].long(), pos % t
            sc = torch.einsum("hgd,nhd->hgn", q.view(-1, g, case["dim"]), held("k", ids, slots)) * s["scale"]
            lses.append(sc.logsumexp(-1).flatten())
            outs.append(torch.einsum("hgn,nhd->hgd", sc.softmax(-1), held("v", ids, slots)).reshape(q.shape))
        return {"out": torch.stack(outs), "lse": torch.stack(lses)}
    got = {}
    for x in ("k", "v"):
        new = s[x].double()
        if x == "k" and s["rope"] is not None:
            r = s["rope"][s["pos"].long()].double()[:, None]
            c, w = r[..., :case["dim"] // 2], r[..., case["dim"] // 2:]
            lo, hi = new[..., :case["dim"] // 2], new[..., case["dim"] // 2:]
            new = torch.cat([lo * c - hi * w, hi * c + lo * w], 2)
        if case["kind"] == "i8":
            grp = new.unflatten(2, (-1, 32))
            d = (grp.abs().amax(3, keepdim=True) / 127).half().double()
            new = torch.where(d > 0, (grp / d).round().clamp(-127, 127) * d, torch.zeros_like(grp)).flatten(2).half().double()
        else:
            new = new.to(pool[x].dtype).double()
        got[x] = new
    return got
