"""The order of cluster barriers and of stores to other CTAs' shared memory in csrc/attn_paged.cu.  A store to a CTA that has not
started can be lost or fault, which no run shows reliably, so the source is read instead."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def kernel():
    text = open(os.path.join(ROOT, "block_sparse_long_gb300", "csrc", "attn_paged.cu")).read()
    body = text[text.index("    paged_kernel("):text.index("// Joins the parts of the items")]
    return re.sub(r"//[^\n]*", lambda m: m[0] if "======" in m[0] else "", body)


def barriers(text):
    return re.findall(r"cluster_(arrive|wait|barrier)\(\)", text)


def test_a_cluster_has_started_before_its_memory_is_written():
    """Every thread arrives before the roles part; the softmax warps wait for it before their first store, and every other warp takes
    the same barriers in the same order."""
    prologue, roles = re.split(r"=+ producer =+", kernel())
    assert barriers(prologue) == ["arrive"] and "store_remote" not in prologue
    softmax = re.split(r"=+ softmax =+", roles)
    assert len(softmax) == 2 and not barriers(softmax[0]) and "store_remote" not in softmax[0]
    mine, others = softmax[1].split("a.cluster > 1 && warp < 4")
    assert barriers(mine) == barriers(others) == ["wait", "barrier", "barrier"]
    assert mine.index("cluster_wait()") < mine.index("store_remote(")


def test_a_warp_that_gave_up_leaves_the_join_out():
    """Behind the pieces `ok` says whether this warp knows its rows: every wait that runs out before has to clear it."""
    softmax = re.split(r"=+ softmax =+", kernel())[1]
    pieces = softmax[softmax.index("more = pieces.next"):softmax.index("cluster_wait()")]
    waits = re.findall(r"if \(!meet\(\)\)([^;]*;)", pieces)
    assert len(waits) == 4 and all("ok = false" in w for w in waits)
    assert "= works && ok;" in softmax
