"""CPU checks of rules that the kernels of the routed feed-forward and the 4-bit weights follow by their
source, where breaking them would show on a GPU only now and then."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp16_gemm_b200", "csrc")


def _code(name):
    """The file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def test_waits_of_the_4bit_products_end_for_a_whole_warp():
    """The lanes of a warp that waits agree on whether it ran out: lanes that left alone would be missing
    at the barriers and in the warp-wide steps that follow."""
    code = _code("sp24_w4_gemv.cuh")
    waits = re.findall(r"[^;{}]*\bmbar_\w*wait\w*\s*\([^;]*;", code)
    assert len(waits) == 1 and "__all_sync(kFull, tc::mbar_wait(bar, parity))" in waits[0]
    assert len(re.findall(r"\bwarp_wait\(", code)) == 3  # itself, the copying warp, the multiplying warps
