"""Bounded waits of the kernels whose warps have roles, by their source (a wait that
runs out is not provoked on a GPU).

A wait's answer may differ between the lanes of a warp: some see the barrier, others the
give-up flag or the limit.  A warp whose lanes then go on together, through votes, shuffles or
aligned instructions, would wait for the lanes that left, for good.  So a wait that each
lane makes for itself may stand only where one lane is left of the warp."""
import os
import re

import pytest

from top_activation_sparse_b200 import build

FILES = ["fp4_gemm.cu", "fp4_gemm_wide.cu", "moe_bf16_tensor.cu", "moe_fp4_down.cu", "moe_fp4_factors.cu"]


def lonely_waits(text):
    """(line, waits of one lane's own outside of a block for one lane)."""
    text = re.sub(r"//[^\n]*", "", text)
    stack, since, found = [], 0, []
    for m in re.finditer(r"[{};]|\b[gw]_wait\(", text):
        c = m.group()
        if c == "{":
            stack.append(text[since:m.start()])
        elif c == "}":
            stack.pop()
        elif c != ";":
            inside = " ".join(stack)
            if "lane == 0" not in inside and "__device__" not in inside:
                found.append(text.count("\n", 0, m.start()) + 1)
            if "__device__" in text[since:m.start()]:
                found = [n for n in found if n != text.count("\n", 0, m.start()) + 1]
            continue
        since = m.end()
    return found


def test_the_reader_tells_the_two_apart():
    body = "__global__ void k() { if (warp == 0) { if (lane == 0) { if (!g_wait(a)) return; } } else { %s } }"
    assert lonely_waits(body % "if (!g_wait_warp(a)) return;") == []
    assert lonely_waits(body % "if (!g_wait(a)) return;") == [1]


@pytest.mark.parametrize("name", FILES)
def test_whole_warps_agree_on_a_wait(name):
    with open(os.path.join(build.CSRC, name)) as f:
        assert lonely_waits(f.read()) == []


def test_lists_are_not_read_after_a_give_up():
    """The copying warp of the queue kernel takes a list's length only from a wait that its lanes agree on."""
    with open(os.path.join(build.CSRC, "moe_kernel.cuh")) as f:
        text = f.read()
    sends = re.findall(r"void send_(?:run|down)\(.*?\n}\n", text, re.S)
    assert len(sends) == 2
    assert all("list_wait" in s and not re.search(r"volatile int\*\)&sm\.n", s) for s in sends)
    assert "__all_sync" in re.search(r"int list_wait\(.*?\n}\n", text, re.S).group()
