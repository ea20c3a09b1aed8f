"""Drawing several answers to each of a few prompts, on random weights of a Llama-like shape with query and key norms.

Prompts go in as in paged_decode.py and are forked into samples, a group of consecutive rows for each prompt. A step of all
samples: an embedding, for every layer the fused query/key/value product (qgemm_small), norm and rotation of its query and key
heads (qpack_qk_norm_rope), qpack_kv_append, and qpack_kv_attend_shared, which reads each prompt once for its whole group;
then the logits' product and the next tokens (qpack_sample). A step after the first is captured once and replayed.

    python examples/sampled_decode.py                 # a 7B-shaped model of 4 layers, 4 prompts, 4 samples each
    python examples/sampled_decode.py --check         # and every attention of the first steps against a dense one in fp64
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import bit_weight_quantized_qpack_gb300 as qp  # noqa: E402
from paged_decode import Decoder, Model, dense, i32, norm  # noqa: E402


class Sampler(Decoder):
    """Samples of prompts; rows [first[g], first[g + 1]) of the batch answer prompt g."""

    def __init__(self, model, seqs, max_tokens, page_tokens, pages, vocab, rows, seed=0):
        super().__init__(model, seqs, max_tokens, page_tokens, pages)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rand = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
        self.embedding = rand(vocab, model.hidden)
        self.head = (vocab, model.hidden, *qp.qpack_quantize_pack(model.fmt, rand(vocab, model.hidden) * model.hidden ** -0.5))
        self.norms = [(1 + 0.1 * rand(model.dim), 1 + 0.1 * rand(model.dim)) for _ in model.layers]
        self.shared_ws = qp.alloc_kv_shared_workspace(self.pool, rows, model.q_heads)
        self.gen = g

    def heads(self, layer, qkv, **where):
        """Query, key and value heads of a product, the first two normed and rotated."""
        m = self.m
        q, k, v = (x.view(x.shape[0], -1, m.dim) for x in self.split(qkv))
        qn, kn = self.norms[layer]
        q, k = qp.qpack_qk_norm_rope(q, k, qn, kn, rope=m.rope, **where)
        return q, k, v

    def prompt(self, seqs, lens, x):
        m = self.m
        qp.qpack_kv_reserve(self.pool, self.tab, i32(seqs), i32(lens))
        rows = i32([s for s, n in zip(seqs, lens) for _ in range(n)])
        pos = i32([t for n in lens for t in range(n)])
        for layer, w in enumerate(m.layers):
            q, k, v = self.heads(layer, m.prefill(w["qkv"], norm(x)), pos=pos)
            qp.qpack_kv_append(self.pool, layer, self.tab, k, v, seqs=rows, pos=pos)
            kc, vc = qp.qpack_kv_read(self.pool, layer, self.tab, rows, pos)
            out = [dense(a, b.float(), c.float(), m.dim ** -0.5) for a, b, c in zip(*(t.split(lens) for t in (q, kc, vc)))]
            x = m.mix(m.prefill, w, x, torch.cat(out).flatten(1))
        return x

    def logits(self, x):
        n, k, packed, scales = self.head
        return qp.qgemm_small(self.m.fmt, packed, scales, n, k, norm(x).half())

    def step(self, seqs, tokens, first, prefix, u, out, sampling, check=False):
        """The next token of every row into `out`: `tokens` are the last ones, u random numbers."""
        m = self.m
        x = self.embedding[tokens.long()]
        qp.qpack_kv_reserve(self.pool, self.tab, seqs, torch.ones_like(seqs))
        for layer, w in enumerate(m.layers):
            q, k, v = self.heads(layer, m.small(w["qkv"], norm(x)), tables=self.tab, seqs=seqs)
            qp.qpack_kv_append(self.pool, layer, self.tab, k, v, seqs=seqs)
            got = qp.qpack_kv_attend_shared(self.pool, layer, self.tab, q, first, prefix, seqs=seqs, workspace=self.shared_ws)
            if check:
                self.compare(layer, seqs.tolist(), q, got)
            x = m.mix(m.small, w, x, got.flatten(1))
        logits = self.logits(x)
        qp.qpack_sample(logits, u, tokens=out, **sampling)
        return logits

    def compare(self, layer, seqs, q, out):
        """Against a dense attention over each row's own pages: a fork holds the same tokens there."""
        m = self.m
        for i, s in enumerate(seqs):
            pos = torch.arange(int(self.tab.lens[s]), dtype=torch.int32, device="cuda")
            k, v = qp.qpack_kv_read(self.pool, layer, self.tab, torch.full_like(pos, s), pos)
            want = dense(q[i:i + 1].double(), k.double(), v.double(), m.dim ** -0.5)[0]
            self.worst = max(self.worst, float((out[i].double() - want).norm() / want.norm()))


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--q-heads", type=int, default=32)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--dim", type=int, default=128)
    ap.add_argument("--ffn", type=int, default=11008)
    ap.add_argument("--vocab", type=int, default=32000)
    ap.add_argument("--prompts", type=int, nargs="+", default=[700, 65, 1, 2050])
    ap.add_argument("--samples", type=int, default=4, help="of each prompt; prompts x samples at most 16")
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--page", type=int, default=64)
    ap.add_argument("--temperature", type=float, default=0.8)
    ap.add_argument("--top-k", type=int, default=50)
    ap.add_argument("--top-p", type=float, default=0.95)
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args(argv)
    n, per = len(a.prompts), a.samples
    if min(per, a.steps, *a.prompts) < 1 or n * per > 16:
        ap.error("prompts, samples and steps start at 1; prompts x samples go to 16, what qgemm_small takes")
    rows, top = n * per, max(a.prompts) + a.steps
    model = Model(a.layers, a.q_heads, a.kv_heads, a.dim, a.ffn, top, qp.Q4G32)
    d = Sampler(model, n * (per + 1), top, a.page, n * (per + 1) * -(-top // a.page), a.vocab, rows)
    x = d.prompt(list(range(n)), a.prompts, d.embedding[torch.randint(0, a.vocab, (sum(a.prompts),), device="cuda", generator=d.gen)])
    ends = (torch.tensor(a.prompts).cumsum(0) - 1).cuda()
    src, seqs = i32([i for i in range(n) for _ in range(per)]), i32(list(range(n, n + rows)))
    qp.qpack_kv_fork(d.pool, d.tab, src, seqs, workspace=d.page_ws)
    qp.qpack_kv_free(d.tab, i32(list(range(n))))
    # a group for each prompt, which is what its rows share: full pages by reference, the last one as copies
    first, prefix = i32([g * per for g in range(n + 1)]), i32(a.prompts)
    sampling = dict(temperature=torch.full((rows,), a.temperature, device="cuda"), top_k=torch.full((rows,), a.top_k, dtype=torch.int32, device="cuda"),
                    top_p=torch.full((rows,), a.top_p, device="cuda"))
    u = torch.rand((a.steps, rows), device="cuda", generator=d.gen)
    answers = torch.empty((a.steps, rows), dtype=torch.int32, device="cuda")
    last, now, next_u = (torch.empty(rows, dtype=torch.int32, device="cuda"), torch.empty(rows, dtype=torch.int32, device="cuda"), u[0].clone())
    first_logits = d.logits(x[ends]).repeat_interleave(per, 0)
    qp.qpack_sample(first_logits, u[0], tokens=last, **sampling)
    answers[0] = last
    graph, t0, logits, replayed = None, 0.0, None, max(0, a.steps - 3)
    for i in range(1, a.steps):
        next_u.copy_(u[i])
        if graph is None:
            logits = d.step(seqs, last, first, prefix, next_u, now, sampling, a.check)
            if i == 2:                                      # everything is warm: the rest is replayed
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    logits = d.step(seqs, last, first, prefix, next_u, now, sampling)
                t0 = time.perf_counter()
        else:
            graph.replay()
        answers[i] = now
        last.copy_(now)
    torch.cuda.synchronize()
    speed = f"{(time.perf_counter() - t0) / replayed * 1e3:.2f} ms a replayed step" if replayed else "no step replayed"
    flags = qp.qpack_fetch_fault_flags()
    print(f"{per} answers each to prompts of {a.prompts} tokens, {a.steps} tokens long, {a.layers} layers: {speed}"
          + (f" (worst attention error {d.worst:.2e})" if a.check else "") + f", fault flags {flags}")
    return dict(answers=answers, logits=logits, u=u, last=last, worst=d.worst, flags=flags, decoder=d, first_logits=first_logits, seqs=seqs,
                sampling=sampling, step=lambda t, uu, out: d.step(seqs, t, first, prefix, uu, out, sampling, True))


if __name__ == "__main__":
    main()
