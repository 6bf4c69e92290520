"""Barriers of the kernels, read from their sources: one that a warp may miss, or that its lanes
reach apart, would hang the GPU, so that is not tried out there.  On the GPU: a wait that runs
out in some warps of a block, behind bounded waits only."""
import os
import re

import pytest

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
    """bar.sync, bar.red and the cluster barriers marked so are the aligned forms: every lane of a
    warp has to reach them together, whatever branches lie before."""
    text = source("ptx.cuh")
    found = re.findall(r"__device__ __forceinline__ \w+ (named_bar_\w+|cluster_sync_\w+)\(", text)
    assert {"named_bar_sync", "cluster_sync_all"} <= set(found)
    for name in found:
        code = body(text, rf"\b{name}\(")
        assert "asm" in code
        if name.startswith("named") or ".aligned" in code:
            assert "__syncwarp()" in code.split("asm")[0], name
    for name in sorted(os.listdir(build.CSRC)):      # ... and no other place has one
        if name != "ptx.cuh":
            assert not re.search(r'asm[^;]*"[^"]*\b(bar|barrier)\.(sync|red|cta|cluster)', source(name)), name


def test_cluster_barriers_order_memory():
    """Behind a cluster barrier other CTAs overwrite or read what this one loaded or stored."""
    for name in sorted(os.listdir(build.CSRC)):
        for form in re.findall(r"barrier\.cluster\.(?:arrive|wait)[.\w]*", source(name)):
            assert ".release" in form or ".acquire" in form, (name, form)


def test_a_decode_without_pages_waits_for_the_launch_ahead():
    """A launch may start before the one ahead of it has ended, and what comes behind it waits
    for this one alone: its end has to mean that the one ahead has ended too."""
    text = source("decode.cu")
    kernel = text[text.index("decode_main_kernel("):]
    assert "if (writer) griddep_wait();" in body(kernel, r"if \(!active\) \{")
    assert "const bool writer = cta == 0;" in kernel


def test_tensor_memory_loads_join_the_lanes_of_a_warp_behind_a_lanes_own_store():
    """tcgen05.ld is a warp's, not a lane's: where rows of the chunk alone are stored in a loop, its
    next load comes behind lanes that parted."""
    text = source("prefill.cu")
    loops = 0
    for m in re.finditer(r"for \(int c = [^{]*c \+= 16\) \{", text):
        code = body(text[m.start():], r"for \(")
        if "tmem_ld16(" in code and ("if (store)" in code or "if (i0 + r < n)" in code):
            loops += 1
            assert "__syncwarp();" in code.split("tmem_ld16(")[0]
    assert loops == 2


def enclosing(text, at):
    """Heads of the blocks around position ``at``, outermost first, and the statement there."""
    heads, start = [], 0
    for i in range(at):
        if text[i] == "{":
            heads.append(" ".join(text[start:i].split()))
        elif text[i] == "}":
            heads.pop()
        if text[i] in "{};" and text[:i + 1].count("(", start) == text[:i + 1].count(")", start):
            start = i + 1
    return heads, " ".join(text[start:at].split())


def test_softmax_warps_of_the_prefill_meet_whatever_their_waits_said():
    """Waits are bounded and may fail in one warp and not in another, named barriers are neither:
    no branch around one may hang on a wait's outcome or on what a failed wait leaves unread.
    The tiles' number and the item are the same in all of these warps: the item by vote."""
    text = source("prefill.cu")
    kernel = text[text.index("prefill_kernel("):text.index("cudaError_t prepare_prefill")]
    uniform = [r"if constexpr \(.*\)( ok =)?$", r"if \(L::HB == 1\)$", r"if \(!PERS \|\| nkt > 0\)$",
               r"for \(int it = 0, g0 = 0;; \+\+it\)$", r"for \(int j = 0; j < nkt; \+\+j\)$",
               r"auto take_item = .*$"]
    calls = [m.start() for m in re.finditer(r"\bnamed_bar_\w+\(", kernel)]
    assert len(calls) >= 4
    for at in calls:
        heads, statement = enclosing(kernel, at)
        for head in heads + [statement]:
            branch = re.search(r"\b(if|for|while|switch)\b.*", head)
            assert branch is None or any(re.search(u, head) for u in uniform), (head, heads)
    take = body(kernel, r"auto take_item = ")
    assert take.index("named_bar_and(") < take.index("items +") < take.index("ok ? m[0] : -1")


def test_prefill_warps_stay_until_their_copies_and_products_are_done():
    """After a failed wait too: behind its last copy or MMA each of these warps waits (with a
    limit) for what it has under way, before the tensor memory is given back and the CTA leaves."""
    text = source("prefill.cu")
    kernel = text[text.index("prefill_kernel("):text.index("cudaError_t prepare_prefill")]
    keys = body(kernel, r"if \(warp == 0\) \{")
    values = body(kernel, r"else if \(warp == 2 \+ NSW\) \{")
    products = body(kernel, r"else if \(warp == 1\) \{")
    joint = body(values, r"\} else \{")
    rebuilt = values[:values.index(joint)]
    for code, done in ((keys, "drain_copies(k_full, issued)"), (rebuilt, "drain_copies(v_full, issued)"),
                       (joint, "drain_copies(v_full, issued)")):
        assert code.rindex("tma_load_2d(") < code.rindex(done)
    assert keys.rindex("load_queries(") < keys.rindex("mbar_wait_drain(q_full")
    mod = body(products, r"if constexpr \(MOD\) \{")
    plain = body(products, r"if \(!\(MOD && RECON\) && lane == 0\) \{")
    for code in (mod, plain):
        assert code.rindex("umma_f16") < code.rindex("umma_commit(") < code.rindex("mbar_wait_drain(")
    assert kernel.rindex("mbar_wait_drain(") < kernel.rindex("tmem_dealloc(")


@pytest.mark.gpu
@pytest.mark.parametrize("late", [0x00, 0x01, 0x80, 0x7E, 0xFF])
def test_a_wait_that_runs_out_in_some_warps_ends_all_of_them(tmp_path, late):
    """Eight warps that meet at a barrier per item; the wait for item 3 runs out in the warps of
    the mask ``late`` (nothing ever arrives there), after two seconds."""
    import ctypes
    import subprocess
    import torch
    from rank_compressed_paged_gb300 import _lib
    lib = str(tmp_path / "bounded_waits.so")
    subprocess.run([build.nvcc(), *build.ARCH, *build.FLAGS, "-shared", "-o", lib,
                    os.path.join(os.path.dirname(os.path.abspath(__file__)), "bounded_waits.cu")],
                   check=True)
    taken = torch.full((256,), -1, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    run = ctypes.CDLL(lib).run
    run.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_uint, ctypes.c_void_p, ctypes.c_void_p]
    torch.cuda.synchronize()
    assert run(5, 3, late, taken.data_ptr(), err.data_ptr()) == 0
    torch.cuda.synchronize()
    assert bool((taken == (3 if late else 5)).all()), taken
    assert int(err) == (_lib.RCP_DEVERR_TIMEOUT if late else 0)
