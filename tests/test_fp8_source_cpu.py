"""Rules of the kernel sources that no run can show (no GPU needed)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "weight_only_bit_gemm_b200", "csrc")


def source(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def body(text, head):
    """The braces' content after the first match of head."""
    at = text.index("{", re.search(head, text).end())
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i + 1]
    raise AssertionError(head)


@pytest.mark.parametrize("name", sorted(os.path.basename(p) for p in glob.glob(CSRC + "/*")))
def test_no_branch_on_a_lanes_own_answer_is_declared_uniform(name):
    assert not re.search(r"@!?\w+\s+bra\.uni", source(name))


def test_warps_are_whole_at_their_barriers():
    # instructions of whole warps (.aligned) reached by lanes that took
    # different ways: the warp's lanes meet first
    assert "__syncwarp();" in body(source("w4_ptx.cuh"), r"void cluster_sync\(\)")
    assert "__syncwarp();" in body(source("w4_fp8_gemm.cuh"), r"void epi_sync\(\)")
    for name in ("w4_fp8_gemm.cuh", "w4_fp8_moe.cuh"):
        text = source(name)
        # a wait that is skipped after an earlier one gave up
        skipped = re.findall(r"if \(ok\)\s*ok = mbar_wait_warp\([^;]*;\s*(\w+)\s*(\w*)", text)
        assert skipped and all(s == ("else", "__syncwarp") for s in skipped)
        # per-lane waits directly before the tensor memory is freed
        assert not re.search(r"[^_]mbar_wait\(done", text)
    # a vote orders no memory: the lanes that did not wait for h themselves
    moe = source("w4_fp8_moe.cuh")
    assert re.search(r"__all_sync\([^;{]*moe_wait_h[^;{]*\{\s*__syncwarp\(\);", moe)


@pytest.mark.parametrize("name", ["w4_fp8.cuh", "w4_fp8_gemm.cuh", "w4_fp8_moe.cuh"])
def test_no_read_only_loads_of_what_a_kernel_ahead_may_write(name):
    # these kernels are resident while the kernel ahead of them runs: a load
    # declared read-only for the kernel's life (ld.global.nc) may be moved ahead
    # of the dependency wait or meet an old line in L1
    text = source(name)
    assert "__ldg(" not in text and "ld.global.nc" not in text and "__restrict__" not in text


# loads whose index is a loop's own (below the bound in the loop's condition) or
# checked on the lines before
LOOP_LOADS = ("a.ids + i", "a.weights + i", "a.active)", "src + (2 * c8 + h) * kFp8Rows + r", "p)", "p + 1)")


@pytest.mark.parametrize("name", ["w4_fp8.cuh", "w4_fp8_gemm.cuh", "w4_fp8_moe.cuh"])
def test_global_accesses_go_through_the_bounds_checks(name):
    # the bounds-checked build can only report an access that asks it
    text = source(name)
    if name == "w4_fp8.cuh":
        for head in (r"\bV ld_in\(", r"\bvoid st_in\("):
            part = body(text, head)
            assert "in_bounds(" in part
            text = text.replace(part, "{}")
    loads = re.findall(r"__ldc[gs]\(([^;]*)", text)
    assert all(l.startswith(LOOP_LOADS) for l in loads), loads
    # vector stores that are left go to shared memory
    for target in re.findall(r"\*reinterpret_cast<u?int\w*\*>\((\w+)", text):
        assert target == "yw", target
    # scalar stores through an operand's pointer: the loop's own index
    for operand in re.findall(r"\b(?:a\.)?(Y|y|q|qm|y_out|residual_out|logits|ids|weights|xq|sx|wt|hq|sh)"
                              r"\[[^\]]*\] = ", text):
        raise AssertionError(operand)
