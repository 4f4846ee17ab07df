"""Rules of the linear layers' and the norm's kernels that a run shows only when it goes
wrong (a hang, a stale read), checked on their source."""
import os
import re

from test_kernel_sources import CSRC, body, source


def test_linear_warps_leave_their_waits_together():
    """Warp-wide instructions stand behind bounded waits that may give up: every wait
    decides for its whole warp."""
    text = source("linear_gemm.cuh")
    assert text.count("mbar_wait_warp(") >= 12 and not re.search(r"\bmbar_wait\(", text)
    assert not re.search(r"mbar_try_wait|mbar_test_wait|while \(true\)", text)


def test_linear_kernels_read_with_plain_loads():
    """They start while the kernel before them may still write; the read-only path is not for
    data that it wrote.  Nothing is read before the wait for it."""
    for name in ("linear_gemm.cuh", "linear.cu"):
        text = source(name)
        assert "__ldg" not in text and "ld.global.nc" not in text and "__restrict__" not in text
    text = source("linear_gemm.cuh")
    for kernel in ("linear_gemm_kernel(", "linear_few_kernel("):
        code = body(text, kernel)
        before = code[:code.index("if (!p.late) grid_wait();")]
        assert "tma_load" not in before and "p.epi" not in before and "p.part" not in before
        # a product that did not wait at its start does at its end
        assert code.rstrip("} \n").endswith("if (p.late) grid_wait();")
    for kernel in ("linear_finish_kernel(", "linear_bias_kernel("):
        code = body(source("linear.cu"), kernel)
        before = code[:code.index("grid_wait();")]
        assert "part[" not in before and "p.part" not in before and "return" not in before


def test_norm_weights_read_their_predecessor_with_plain_loads():
    code = body(source("norm_rope.cu"), "norm_weight_kernel(")
    before = code[:code.index("grid_wait();")]
    assert "__ldg" not in code and "p.part[" not in before and "return" not in before


def test_what_a_late_product_reads_is_passed_on_to_it():
    """A product that does not wait at its start reads what the grid before it has been shown;
    every such grid waits (or was passed it), fences for plain accesses and for the copies, and
    only then lets the next one start."""
    fences = body(source("ptx.cuh"), "void grid_pass_on()")
    assert re.search(r"__threadfence\(\);.*fence\.proxy\.async\.global;", fences, re.S)
    bias = re.sub(r"\s+", " ", body(source("linear.cu"), "linear_bias_kernel("))
    assert "grid_wait(); grid_pass_on(); grid_launch_dependents();" in bias
    for kernel in ("linear_gemm_kernel(", "linear_few_kernel("):
        code = re.sub(r"\s+", " ", body(source("linear_gemm.cuh"), kernel))
        assert "if (!p.late) grid_wait(); if (p.pass_on) grid_pass_on(); grid_launch_dependents();" in code
        assert code.count("grid_launch_dependents") == 1
    calls = re.sub(r"\s+", " ", body(source("linear.cu"), "tsr_status launch_linear_backward("))
    # the products: late only behind the sum of dbias, or dweight behind a dx that is not cut
    assert "bool late = a.dbias != nullptr;" in calls and "late = uncut;" in calls
    assert "late, late || (a.dweight && uncut), st)" in calls and "late, late, st)" in calls


def test_arrivals_on_the_peer_come_before_its_end():
    """The issuer of a pair arrives on barriers of both CTAs; a CTA must not end before the last
    of them: the producer of either CTA waits for each stage that it has filled last."""
    code = re.sub(r"\s+", " ", body(source("linear_gemm.cuh"), "linear_gemm_kernel("))
    producer = code[code.index("if (warp == 0) {"):code.index("} else if (warp == 1)")]
    tail = producer[producer.index("++issued;"):]
    wait = tail.index("ok = mbar_wait_warp(smem_u32(&ctrl.empty[k % C::STAGES])")
    assert "rank" not in tail[:wait]
    # copies in flight are waited for where that was given up
    assert "if (rank == 0 && !ok)" in tail[wait:] and "ctrl.full[k % C::STAGES]" in tail[wait:]
    # the other commits of the pair are waited for by the epilogue of both and by the issuer
    assert code.count("mma_commit_pair(") == 3
    for bar in ("empty[st]", "acc_full[buf]", "final_bar"):
        assert code.count("mma_commit_pair(elect, smem_u32(&ctrl.%s));" % bar) == 1


def test_what_first_calls_note_is_atomic():
    """First calls may come from several threads at once: the flags and numbers that they leave
    behind for the next ones are atomic."""
    for name in sorted(n for n in os.listdir(CSRC) if n.endswith((".cu", ".cuh", ".h"))):
        assert not re.search(r"\bstatic (bool|int|int32_t|int64_t|size_t) \w+(\[\d+\])? *(=|;)", source(name)), name
    assert "std::atomic<bool> done_[64]" in body(source("internal.h"), "class OncePerDevice")


def test_the_products_parameters_are_read():
    """Every field of the kernels' parameters is read by one of them, or by a launch."""
    text = source("linear_gemm.cuh")
    fields = re.findall(r"(\w+)(?=[,;])", re.sub(r"\[[^]]*\]", "", body(text, "struct GemmParams {")))
    assert len(fields) > 20
    read = text.replace(body(text, "struct GemmParams {"), "") + source("linear.cu")
    for name in fields:
        assert re.search(r"\bp\.%s\b(?! = )" % name, read), name
