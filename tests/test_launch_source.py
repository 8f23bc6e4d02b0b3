"""CPU checks of rules that the kernels of the routed feed-forward and the 4-bit weights follow by their
source, where breaking them would show on a GPU only now and then."""
import os
import re

import pytest

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


FILES = [f for f in sorted(os.listdir(CSRC)) if f.endswith((".cu", ".cuh")) and '#include "sp24_launch.cuh"' in open(os.path.join(CSRC, f)).read()]


def _kernels(code):
    """(parameters, body) of each kernel."""
    for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\((?:[^()]|\([^()]*\))*\)\s*)?(\w+)\s*\(", code):
        ends = []
        at = m.end() - 1
        for pair in ("()", "{}"):
            at = code.index(pair[0], at)
            depth, start = 0, at
            while True:
                depth += (code[at] == pair[0]) - (code[at] == pair[1])
                at += 1
                if depth == 0:
                    break
            ends.append(code[start + 1:at - 1])
        yield m.group(1), ends[0], ends[1]


def test_files_that_launch_ahead():
    assert {"sp24_route.cu", "sp24_sort.cu", "sp24_w4.cu", "sp24_w4_gemv.cuh"} <= set(FILES)
    assert sum(len(list(_kernels(_code(f)))) for f in FILES) >= 11


@pytest.mark.parametrize("name", FILES)
def test_kernels_that_start_early_read_with_ordinary_loads(name):
    """Their predecessor may still write what they are to read, so no load may take the read-only path,
    which is defined for data that nobody writes while the kernel runs, and no pointer may tell the
    compiler that the wait does not concern it."""
    assert not re.search(r"__ldg\b|ld\.global\.nc|ldg_stream16|__restrict__", _code(name))


@pytest.mark.parametrize("name", [f for f in FILES if f != "sp24_w4_gemv.cuh"])
def test_kernels_that_start_early_wait_before_they_read(name):
    """begin() stands once in a kernel, outside of every branch and loop, and no pointer is followed
    before it."""
    for kernel, params, body in _kernels(_code(name)):
        ahead, *rest = body.split("begin();")
        assert len(rest) == 1, kernel
        assert ahead.count("{") == ahead.count("}") and ahead.rstrip()[-1:] in ("", ";"), kernel
        assert not re.search(r"\b(for|while|return)\b", ahead), kernel
        for p in re.findall(r"\*\s*(?:__restrict__\s+)?(\w+)", params):
            assert not re.search(rf"\b{p}\s*\[|\*\s*{p}\b", ahead), (kernel, p)
        assert not re.search(r"\bt\.\w+\s*\[", ahead), kernel


def test_the_4bit_products_wait_before_they_read():
    code = _code("sp24_w4_gemv.cuh")
    assert code.count("begin();") == 1
    run = code[code.index("void run("):code.index("begin();")]
    assert "p." not in run and "return" not in run


@pytest.mark.parametrize("name", FILES)
def test_host_state_of_a_launch_is_atomic(name):
    """What a launch remembers on the host is written by any thread that calls it."""
    held = [m.group(0) for m in re.finditer(r"\bstatic\s+(?!constexpr|__device__|__host__|_?const\b)[\w:<>]+\s+\w+(\[\w+\])?\s*(=|;|\{)", _code(name))]
    assert all("std::atomic<" in h for h in held), held
