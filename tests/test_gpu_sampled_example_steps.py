"""The sampling example with few steps: it says how long a replayed step took only where one was replayed."""
import os
import re
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("steps", [1, 2, 3, 4])
def test_few_steps(qpg, steps, capsys):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import sampled_decode
    got = sampled_decode.main(["--layers", "1", "--q-heads", "4", "--kv-heads", "2", "--dim", "64", "--ffn", "512", "--vocab", "1000",
                               "--prompts", "9", "20", "--samples", "2", "--steps", str(steps), "--page", "16"])
    assert got["flags"] == 0 and got["answers"].shape == (steps, 4) and bool((got["answers"] >= 0).all())
    said = capsys.readouterr().out
    ms = re.search(r"([0-9.]+) ms a replayed step", said)
    assert (ms is None and "no step replayed" in said) if steps < 4 else 0 < float(ms.group(1)) < 10000
