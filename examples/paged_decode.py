"""Decoding with packed weights and a paged 8-bit KV cache, on random weights of a Llama-like shape.

Prompts of different lengths go in at once (qgemm_prefill, then qpack_kv_append, and attention over the rows that
qpack_kv_read gives back); each prompt is forked into samples, and all samples decode together, a token a step:
qpack_kv_reserve, then for every layer the fused query/key/value product (qgemm_small), qpack_kv_append with the rotary
embedding, qpack_kv_attend, and the other products. At the end some samples are freed and the cache is compacted.

    python examples/paged_decode.py                 # a 7B-shaped model of 4 layers
    python examples/paged_decode.py --check         # and every attention against a dense one in fp64
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_weight_quantized_qpack_gb300 as qp  # noqa: E402


class Model:
    """Packed weights of `layers` layers (fused q/k/v, output, gate, up, down) and the rotation table."""

    def __init__(self, layers, q_heads, kv_heads, dim, ffn, positions, fmt, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.q_heads, self.kv_heads, self.dim, self.hidden, self.fmt = q_heads, kv_heads, dim, q_heads * dim, fmt
        shapes = dict(qkv=((q_heads + 2 * kv_heads) * dim, self.hidden), o=(self.hidden, self.hidden),
                      gate=(ffn, self.hidden), up=(ffn, self.hidden), down=(self.hidden, ffn))
        self.layers = []
        for _ in range(layers):
            w = {}
            for name, (n, k) in shapes.items():
                w[name] = (n, k, *qp.qpack_quantize_pack(fmt, torch.randn((n, k), generator=g, device="cuda") * k ** -0.5))
            self.layers.append(w)
        freq = 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
        angle = torch.arange(positions, dtype=torch.float64)[:, None] * freq
        self.rope = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()

    def small(self, w, x):
        n, k, packed, scales = w
        return qp.qgemm_small(self.fmt, packed, scales, n, k, x.half())

    def prefill(self, w, x):
        n, k, packed, scales = w
        return qp.qgemm_prefill(self.fmt, packed, scales, n, k, x.bfloat16()).float()

    def mix(self, product, w, x, attended):
        """The layer after attention: output product, residual, gated feed-forward."""
        x = x + product(w["o"], attended)
        y = norm(x)
        return x + product(w["down"], torch.nn.functional.silu(product(w["gate"], y)) * product(w["up"], y))


def norm(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def dense(q, k, v, scale):
    """Attention of the last len(q) tokens over a sequence's rows: q [n, Hq, D], k and v [L, H, D]."""
    n, L, g = q.shape[0], k.shape[0], q.shape[1] // k.shape[1]
    s = torch.einsum("nhd,lhd->hnl", q, k.repeat_interleave(g, 1)) * scale
    ahead = torch.arange(L, device=q.device) > torch.arange(L - n, L, device=q.device)[:, None]
    return torch.einsum("hnl,lhd->nhd", s.masked_fill(ahead, float("-inf")).softmax(-1), v.repeat_interleave(g, 1))


def rotate(x, rows):
    c, s = rows[:, None].to(x.dtype).chunk(2, -1)
    a, b = x.chunk(2, -1)
    return torch.cat([a * c - b * s, b * c + a * s], -1)


class Decoder:
    def __init__(self, model, seqs, max_tokens, page_tokens, pages):
        self.m = model
        self.pool = qp.alloc_kv_pool(qp.KV_I8, len(model.layers), pages, model.kv_heads, page_tokens, model.dim)
        self.tab = qp.alloc_kv_tables(seqs, -(-max_tokens // page_tokens), pages)
        self.attend_ws = qp.alloc_kv_workspace(self.pool, 16, model.q_heads)
        self.page_ws = qp.alloc_kv_page_workspace(self.pool, self.tab)
        self.worst = 0.0

    def split(self, qkv):
        m = self.m
        q, k, v = qkv.split([m.q_heads * m.dim, m.kv_heads * m.dim, m.kv_heads * m.dim], 1)
        return q, k, v

    def prompt(self, seqs, lens, x):
        """Prompts of `lens` tokens into the empty sequences `seqs`; x [sum lens, hidden]."""
        m = self.m
        qp.qpack_kv_reserve(self.pool, self.tab, i32(seqs), i32(lens))
        rows = i32([s for s, n in zip(seqs, lens) for _ in range(n)])
        pos = i32([t for n in lens for t in range(n)])
        for layer, w in enumerate(m.layers):
            q, k, v = self.split(m.prefill(w["qkv"], norm(x)))
            qp.qpack_kv_append(self.pool, layer, self.tab, k, v, seqs=rows, pos=pos, rope=m.rope)
            kc, vc = qp.qpack_kv_read(self.pool, layer, self.tab, rows, pos)
            q = rotate(q.view(-1, m.q_heads, m.dim), m.rope[pos.long()])
            out = [dense(a, b.float(), c.float(), m.dim ** -0.5) for a, b, c in zip(*(t.split(lens) for t in (q, kc, vc)))]
            x = m.mix(m.prefill, w, x, torch.cat(out).flatten(1))
        return x

    def step(self, seqs, x, check=False):
        """One token each for the sequences `seqs` (int32 tensor, at most 16); x [len(seqs), hidden]."""
        m = self.m
        qp.qpack_kv_reserve(self.pool, self.tab, seqs, torch.ones_like(seqs))
        for layer, w in enumerate(m.layers):
            q, k, v = self.split(m.small(w["qkv"], norm(x)))
            qp.qpack_kv_append(self.pool, layer, self.tab, k, v, seqs=seqs, rope=m.rope)
            out = qp.qpack_kv_attend(self.pool, layer, self.tab, q, seqs=seqs, rope=m.rope, workspace=self.attend_ws)
            if check:
                self.compare(layer, seqs.tolist(), q, out)
            x = m.mix(m.small, w, x, out.flatten(1))
        return x

    def compare(self, layer, seqs, q, out):
        m = self.m
        for i, s in enumerate(seqs):
            n = int(self.tab.lens[s])
            pos = torch.arange(n, dtype=torch.int32, device="cuda")
            k, v = qp.qpack_kv_read(self.pool, layer, self.tab, torch.full_like(pos, s), pos)
            turned = rotate(q[i:i + 1].view(1, m.q_heads, m.dim).double(), m.rope[n - 1:n])
            want = dense(turned, k.double(), v.double(), m.dim ** -0.5).flatten()
            self.worst = max(self.worst, float((out[i].flatten().double() - want).norm() / want.norm()))


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--q-heads", type=int, default=32)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--dim", type=int, default=128)
    ap.add_argument("--ffn", type=int, default=11008)
    ap.add_argument("--prompts", type=int, nargs="+", default=[700, 65, 1, 2050])
    ap.add_argument("--samples", type=int, default=4, help="of each prompt; prompts x samples at most 16")
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--page", type=int, default=64)
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args(argv)
    n, per = len(a.prompts), a.samples
    top = max(a.prompts) + a.steps
    model = Model(a.layers, a.q_heads, a.kv_heads, a.dim, a.ffn, top, qp.Q4G32)
    # every sample could fill its own pages: enough for the worst case
    pages = n * (per + 1) * -(-top // a.page)
    d = Decoder(model, n * (per + 1), top, a.page, pages)
    x = torch.randn((sum(a.prompts), model.hidden), device="cuda")
    x = d.prompt(list(range(n)), a.prompts, x)
    ends = torch.tensor(a.prompts).cumsum(0) - 1
    # samples of prompt i: sequences n + i * per ..; the prompts' own sequences are then released
    src, dst = i32([i for i in range(n) for _ in range(per)]), i32([n + j for j in range(n * per)])
    qp.qpack_kv_fork(d.pool, d.tab, src, dst, workspace=d.page_ws)
    qp.qpack_kv_free(d.tab, i32(list(range(n))))
    x = x[ends.cuda()].repeat_interleave(per, 0) + 0.1 * torch.randn((n * per, model.hidden), device="cuda")
    live, t0 = dst, 0.0
    for step in range(a.steps):
        if step == 1:
            torch.cuda.synchronize()
            t0 = time.perf_counter()
        if step == a.steps // 2:                            # every second sample ends; the cache closes up
            qp.qpack_kv_free(d.tab, live[1::2].contiguous())
            qp.qpack_kv_compact(d.pool, d.tab, workspace=d.page_ws)
            live, x = live[0::2].contiguous(), x[0::2].contiguous()
        x = d.step(live, x, a.check)
    torch.cuda.synchronize()
    ms = (time.perf_counter() - t0) / max(1, a.steps - 1) * 1e3
    flags = qp.qpack_fetch_fault_flags()
    held = int((d.tab.refs > 0).sum())
    print(f"{n * per} samples of prompts {a.prompts}, {a.steps} steps on {a.layers} layers: {ms:.2f} ms a step"
          + (f" (checking: worst attention error {d.worst:.2e})" if a.check else "")
          + f", {held} of {pages} pages held, fault flags {flags}")
    return dict(x=x, worst=d.worst, flags=flags, held=held, decoder=d, live=live)


if __name__ == "__main__":
    main()
