"""Host-side checks of the limits of sampled decoding's operators: waits that run out, calls that are refused as a whole, the example's
arguments."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_weight_quantized_qpack_gb300", "csrc")


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
