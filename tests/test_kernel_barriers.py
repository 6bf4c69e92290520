"""Barriers of the kernels, read from their sources (no GPU): a barrier that a warp may miss, or
that its lanes reach apart, would hang the GPU, so none of these is tried out there."""
import os
import re

from rank_compressed_paged_gb300 import build


def source(name):
    with open(os.path.join(build.CSRC, name)) as f:
        text = f.read()
    text = re.sub(r"//[^\n]*", "", text)          # comments and asm strings hold no control flow
    return re.sub(r'"(?:\\.|[^"\\])*"', lambda m: '"' + m.group(0)[1:-1].replace("{", "(").replace(
        "}", ")") + '"', text)


def body(text, head):
    """The brace-enclosed body behind the first match of ``head``."""
    at = text.index("{", re.search(head, text).end() - 1)
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == "{") - (text[i] == "}")
        if depth == 0:
            return text[at + 1:i]
    raise AssertionError(f"no end of {head}")


def test_aligned_barriers_join_the_lanes_of_a_warp_first():
    """bar.sync, bar.red and the cluster barriers are the aligned forms: every lane of a warp has
    to reach them together, whatever branches lie before."""
    text = source("ptx.cuh")
    found = re.findall(r"__device__ __forceinline__ \w+ (named_bar_\w+|cluster_sync_\w+)\(", text)
    assert {"named_bar_sync", "cluster_sync_all"} <= set(found)
    for name in found:
        code = body(text, rf"\b{name}\(")
        assert "asm" in code and "__syncwarp()" in code.split("asm")[0], name
    for name in sorted(os.listdir(build.CSRC)):      # ... and no other place has one
        if name != "ptx.cuh":
            assert not re.search(r'asm[^;]*"[^"]*\b(bar|barrier)\.(sync|red|cta|cluster)', source(name)), name
