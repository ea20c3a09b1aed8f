"""The operators of a decode step together, as the sampling example runs them: products, norm and rotation of heads, append,
attention over shared prefixes, logits, tokens; captured and replayed. Every attention agrees with a dense one in fp64 over each
row's own pages, and every checked token is the one that the definition gives for its logits."""
import os
import sys

import numpy as np
import pytest
import torch

from oracle import decode as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def tokens_of(logits, u, got):
    h = logits.float().cpu().numpy()
    par = {k: got["sampling"][k].cpu().numpy() for k in got["sampling"]}
    return [ref.sample(h[i], np.float32(u[i]), par["temperature"][i], int(par["top_k"][i]), par["top_p"][i])[0] for i in range(len(h))]


@pytest.mark.parametrize("page,samples", [(16, 4), (8, 1), (64, 3)])
def test_sampled_decode_example(qpg, page, samples):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import sampled_decode
    got = sampled_decode.main(["--layers", "2", "--q-heads", "8", "--kv-heads", "2", "--dim", "128", "--ffn", "2048", "--vocab", "5000",
                               "--prompts", "70", "16", "1", "133", "--samples", str(samples), "--steps", "9", "--page", str(page),
                               "--check"])
    assert got["flags"] == 0
    u = got["u"].cpu().numpy()
    assert np.array_equal(got["answers"][0].cpu().numpy(), tokens_of(got["first_logits"], u[0], got))
    # the graph's last replay left its logits
    assert np.array_equal(got["answers"][-1].cpu().numpy(), tokens_of(got["logits"], u[-1], got))
    d = got["decoder"]
    lens = d.tab.lens.tolist()
    assert [lens[s] for s in got["seqs"].tolist()] == [n + 8 for n in (70, 16, 1, 133) for _ in range(samples)]
    # a step by calls behind the replayed ones: the state they left is whole
    now, uu = torch.empty_like(got["last"]), torch.full_like(got["u"][0], 0.25)
    logits = got["step"](got["last"], uu, now)
    assert np.array_equal(now.cpu().numpy(), tokens_of(logits, uu.cpu().numpy(), got))
    # half a unit of fp16's last place, by element: 2^-11 of the norm at most, and as much again for everything else
    # (probabilities over the prefix are rounded to fp16: 2^-11 of each weight, averaged)
    assert 0 < d.worst < 2.0 ** -10
    assert qpg.qpack_fetch_fault_flags() == 0
