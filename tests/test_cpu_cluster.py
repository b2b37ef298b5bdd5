"""The order of cluster operations in the kernels' sources, which no result
shows: a store that comes too early fails only when a CTA of its cluster
happens to start late."""
import os
import re

import pytest

import mxfp8_quantization_gb300 as rn

CSRC = os.path.join(os.path.dirname(os.path.abspath(rn.__file__)), "csrc")


def source(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def body(text, name):
    """The text between the braces of the function `name`."""
    start = text.index("{", re.search(rf"\b{name}\([^;]*?\{{", text).start())
    depth = 0
    for i in range(start, len(text)):
        depth += (text[i] == "{") - (text[i] == "}")
        if depth == 0:
            return text[start:i]
    raise AssertionError(f"{name} does not end")


def test_files_that_store_to_other_ctas():
    """Those whose order the tests below check."""
    found = {f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")) and
             re.search(r"\b(st|red|atom)\.[\w.]*shared::cluster", source(f))}
    assert found == {"rn_ffn.cu", "rn_matvec.cu"}


def test_few_token_kernel_meets_before_its_first_remote_store():
    k = body(source("rn_matvec.cu"), "rn_matvec_kernel")
    # the sums leave in add_up, which acts on a step that was computed ("held"); the first is computed in the
    # loop over a batch's steps, after its tokens were staged
    assert "st.shared::cluster" in k[k.index("const auto add_up"):k.index("Item it[")]
    assert re.search(r"int held = -1\b", k)
    calls = [m.start() for m in re.finditer(r"add_up\(\)", k)]
    guards = [m.start() for m in re.finditer(r"if \(held >= 0\) add_up\(\)", k)]
    assert len(calls) == len(guards) == 3
    first_held = k.index("held = j;")
    meet = k.index("cluster_wait();")
    assert k.index("cluster_arrive();") < k.index("stage_tokens<") < meet < k.index("for (int j = b0") < first_held
    # once, by every thread of a cluster and by no other CTA
    assert re.search(r"if \(pl\.split > 1\) cluster_arrive\(\);", k)
    assert re.search(r"if \(pl\.split > 1 && b0 == 0 && sl == 0\) cluster_wait\(\);", k)
    assert k.count("cluster_arrive();") == k.count("cluster_wait();") == 1


def test_block_kernel_meets_before_its_first_remote_operation():
    k = body(source("rn_ffn.cu"), "rn_ffn_kernel")
    meet = k.index("cluster_sync();")
    for op in ("tma_load_2d(", "mma_bf16_pair(", "mma_commit(", "map_to_rank(", "split_epilogue<"):
        assert meet < k.index(op), op


def test_cluster_barriers_take_whole_warps():
    """barrier.cluster.*.aligned is executed by a converged warp, whatever branch came before it."""
    for half in ("cluster_arrive", "cluster_wait"):
        b = body(source("rn_tc.cuh"), half)
        assert b.index("__syncwarp();") < b.index(".aligned")
    assert "barrier.cluster" not in source("rn_matvec.cu") + source("rn_ffn.cu")


@pytest.mark.parametrize("name", ["rn_matvec.cu", "rn_ffn.cu"])
def test_no_cta_leaves_its_cluster_early(name):
    """The last cluster operation of a kernel is a barrier, after every remote store."""
    k = body(source(name), "rn_matvec_kernel" if name == "rn_matvec.cu" else "rn_ffn_kernel")
    tail = k[k.rindex("cluster_sync();"):]
    for op in ("add_up()", "split_epilogue<", "mbar_arrive_cluster(", "mma_commit("):
        assert op not in tail
