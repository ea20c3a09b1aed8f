"""Host-side checks of the limits of sampled decoding's operators: waits that run out, calls that are refused as a whole, the example's
arguments."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_weight_quantized_qpack_gb300", "csrc")


def library():
    from bit_weight_quantized_qpack_gb300 import _build
    _build.build()
    import bit_weight_quantized_qpack_gb300 as qp
    qp.lib()
    return qp


def code(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_a_warp_gives_up_together():
    """Whether a barrier was seen is voted on wherever a warp waits in the kernel over prefixes: its lanes meet again in shuffles
    and barriers, which lanes that gave up alone would never reach. The one other wait is a single lane's."""
    text = code("qpack_shared.cuh")
    assert "return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity));" in text
    waits = [text[text.rfind("\n", 0, m.start()):text.find("\n", m.start())] for m in re.finditer(r"\bmbar_wait_bounded\(", text)]
    assert len(waits) == 2 and "__all_sync(0xffffffffu, mbar_wait_bounded" in waits[0] and "if (lane == 0 && *s_dead)" in waits[1]
    assert len(re.findall(r"\bwarp_wait\(", text)) >= 7 and "mbar_try_wait" not in text


def test_shared_refuses_what_the_attention_behind_it_would():
    """Few rows of many query heads over a long table: the tiles of the prefixes can be counted, those of the attention over what
    rows have of their own cannot. The call is refused as a whole, before its first launch (which would fail here, without a GPU)."""
    from test_decode_host import UNSUPPORTED, call_shared
    qp = library()
    many = dict(B=1, heads=1, q_heads=8192, ldq=8192 * 128, ldo=8192 * 128, groups=0, max_pages=(1 << 27) // 16, ws_bytes=1 << 40)
    assert call_shared(qp, **many) == UNSUPPORTED
    assert call_shared(qp, **{**many, "type": 2}) == UNSUPPORTED
    # just inside of what both can count: not refused for its size (without a GPU the launch fails then)
    import torch
    if not torch.cuda.is_available():
        assert call_shared(qp, **{**many, "max_pages": (1 << 27) // 16 // 16}) not in (0, UNSUPPORTED)


@pytest.mark.parametrize("args", [["--samples", "5"], ["--samples", "0"], ["--steps", "0"], ["--prompts", "4", "0"],
                                  ["--prompts"] + ["1"] * 17 + ["--samples", "1"]])
def test_example_refuses_what_it_cannot_run(args, capsys):
    """More rows than qgemm_small takes, and nothing to do: said before anything is set up."""
    import sys
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import sampled_decode
    with pytest.raises(SystemExit):
        sampled_decode.main(args)
    assert "prompts x samples" in capsys.readouterr().err
