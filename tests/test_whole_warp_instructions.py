"""Instructions that all lanes of a warp have to execute together (.aligned) come after a point that brings the warp
together. A warp whose lanes left a loop or a branch at different times is not together by itself, and what such an
instruction then does is undefined. So every function with such an instruction in it begins with __syncwarp(), where
it stands in the way of no caller."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_moe_layout_gb300", "csrc")
FILES = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")))


def strip_comments(text):
    return re.sub(r"//[^\n]*|/\*.*?\*/", lambda m: re.sub(r"[^\n]", " ", m.group()), text, flags=re.S)


def function_around(text, at):
    """The body of the outermost braces around `at` that follow a parameter list."""
    depth, opened, start = 0, [], None
    for i, c in enumerate(text[:at]):
        if c == "{":
            opened.append(i)
        elif c == "}":
            opened.pop()
    for i in opened:
        if re.search(r"\)\s*(const\s*)?$", text[:i]):
            start = i
            break
    assert start is not None
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i]


@pytest.mark.parametrize("name", FILES)
def test_aligned_instructions_follow_a_syncwarp(name):
    text = strip_comments(open(os.path.join(CSRC, name)).read())
    # braces of the asm text itself are balanced within each statement
    for m in re.finditer(r"(?<!setmaxnreg.inc.sync)(?<!setmaxnreg.dec.sync)\.aligned\b", text):
        body = function_around(text, m.start())
        first = body.index(".aligned")
        assert "__syncwarp();" in body[:first], body[:160]


def test_registers_move_straight_after_a_block_barrier():
    """setmaxnreg, the exception: between the last barrier of the block and the warps' own branches, nothing parts a warp."""
    text = strip_comments(open(os.path.join(CSRC, "moe_expert_fp8.cu")).read())
    kernel = text[text.index("grouped_gemm_fp8_kernel("):]
    after = kernel[:kernel.index("regs_release<")].rpartition("__syncthreads();")[2]
    assert re.fullmatch(r"\s*(const int \w+ = [^;{}]*;\s*)*if \(warp == 0\) \{\s*", after), after
    for call in re.finditer(r"regs_(release|claim)<", kernel):
        assert re.search(r"(if \(warp [^{}]*\)|else) \{\s*$", kernel[:call.start()]), kernel[:call.start()][-80:]


@pytest.mark.parametrize("name", FILES)
def test_cluster_barriers_follow_a_syncwarp(name):
    """cluster.sync() is the whole-warp form of the cluster barrier."""
    lines = strip_comments(open(os.path.join(CSRC, name)).read()).split("\n")
    code = [l.strip() for l in lines if l.strip()]
    for i, l in enumerate(code):
        if l.startswith("cluster.sync();"):
            assert code[i - 1] == "__syncwarp();", (name, code[i - 1])
