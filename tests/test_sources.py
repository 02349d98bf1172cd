"""CPU tests of what no run can show: rules of the memory model that the kernels' sources keep."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "layout_general_tensor_gb300", "csrc")


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def test_rows_cleared_in_a_pair_are_announced_at_cluster_scope():
    """The odd CTA's zeros are read by a product that a thread of the even CTA issues: what announces them has to
    release them to that CTA.  (As it runs, the weaker form has not been seen to fail.)"""
    source = _source("gemm_grouped.cu")
    part = source[source.index("rows of the next group\n"):source.index("- results\n")]
    (arrival,) = re.findall(r"(\w+)\(cleared_lead", part)
    body = _source("ptx.cuh").split(f"void {arrival}(")[1].split("\n}")[0]
    assert re.search(r"mbarrier\.arrive\.release\.cluster\.shared::cluster", body)


def test_arrivals_in_another_cta_have_its_scope():
    """What is announced in another CTA's barrier has cluster scope: a release, or, where it says only that tensor
    memory has been read (tcgen05 fences order that), a relaxed arrival."""
    for name in sorted(os.listdir(CSRC)):
        for scope in re.findall(r"mbarrier\.arrive(?:\.expect_tx)?((?:\.\w+)*)\.shared::cluster", _source(name)):
            assert scope in (".release.cluster", ".relaxed.cluster"), (name, scope)


def test_a_look_by_one_lane_is_passed_on_with_its_order():
    """Where one lane of a warp waits for a barrier, the others read and write after it what the barrier announces: a
    shuffle tells them that it has come, and only a barrier of the warp orders their accesses behind it."""
    source = _source("gemm_grouped.cu")
    body = source.split("auto warp_wait = ")[1].split("\n  };")[0]
    assert body.index("lane == 0") < body.index("__syncwarp()")
