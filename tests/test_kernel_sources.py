"""Rules of the kernels that a run shows only when it goes wrong (a hang, a stale
read), checked on their source."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_sparse_attention_tsr_gb300",
                    "csrc")


def source(name):
    """A file's text without comments."""
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", open(os.path.join(CSRC, name)).read(), flags=re.S)


def body(text, start):
    """The braces that follow `start`."""
    i = text.index("{", text.index(start))
    depth = 0
    for j in range(i, len(text)):
        depth += (text[j] == "{") - (text[j] == "}")
        if depth == 0:
            return text[i:j + 1]
    raise AssertionError(start)


def test_backward_warps_leave_their_waits_together():
    """The softmax warps use warp-wide instructions (votes, tcgen05.ld / st) behind
    bounded waits that may give up: a wait decides for the whole warp."""
    text = source("bwd.cu")
    softmax = body(text, "void softmax_role(")
    assert "mbar_wait_warp(" in softmax and not re.search(r"\bmbar_wait\(", softmax)
    # the issuers too, but for the last wait, behind which a warp only ends
    issuer = body(text, "void mma_role(")
    assert len(re.findall(r"\bmbar_wait\(", issuer)) == 1
    wait = body(source("ptx.cuh"), "bool mbar_wait_warp(")
    for cond in re.findall(r"if \((.*)\)", wait):
        assert re.match(r"__(all|any)_sync\(0xFFFFFFFFu, ", cond)


def test_forward_warps_leave_their_waits_together():
    """The same in the forward kernels.  A wait by single lanes is left where one lane
    acts (the issuers) and at a warp's end (`dummy`: no abort flag, nothing behind it)."""
    text = source("fwd_kernel.cuh")
    single = [l for l in text.splitlines() if re.search(r"\bmbar_wait\(", l) and "dummy" not in l]
    assert len(single) == 1 and ": mbar_wait(bar, parity" in single[0]      # a single issuing lane's
    text = source("fwd_t_kernel.cuh")
    assert all("dummy" in l for l in text.splitlines() if re.search(r"\bmbar_wait\(", l))
    for cond in re.findall(r"if \((.*)\) return", body(text, "auto wait = [&]")):
        assert re.match(r"__(all|any)_sync\(0xFFFFFFFFu, ", cond)
    issuers = body(text, "if (warp == 1 || warp == 11)")
    one_lane = body(issuers, "if (lane == 0)")
    assert not re.search(r"\bwait\(", issuers) and one_lane.count("wait_one(") == text.count("wait_one(")


@pytest.mark.parametrize("name,first,second", [("select.cu", "struct PoolParams", "struct SelParams"),
                                               ("bwd.cu", None, "struct Params")])
def test_dependent_kernels_read_their_predecessor_with_plain_loads(name, first, second):
    """A kernel started by launch_dependent is resident while the one before it still
    writes; the read-only path (__ldg, const __restrict__) is not for that data."""
    text = source(name)
    assert "launch_dependent(" in text
    fields = re.sub(r"\s+", " ", body(text, second))
    assert "__restrict__" not in fields
    if name == "select.cu":
        # everything behind its parameters reads pool_kernel's output only
        dependent = text[text.index(second):]
    else:
        dependent = "\n".join(l for l in text.splitlines() if re.search(r"p\.(nlse2|ndelta|part|arrived)\b", l))
        assert "p.nlse2[" in dependent
    assert "__ldg" not in dependent and "ld.global.nc" not in dependent
