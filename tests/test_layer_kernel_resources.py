"""The kernels around the expert products keep everything in registers: the
compiler's own report shows no scratch and no vector spill, and the waves of the
4-bit products' tiles fit a CU as often as they are counted on."""
import os
import shutil

import pytest

from test_kernel_resources import resource_report

pytestmark = pytest.mark.skipif(shutil.which("hipcc") is None and
                                not os.path.exists("/opt/rocm/bin/hipcc"),
                                reason="hipcc needed")


@pytest.fixture(scope="module")
def reports():
    return {src: resource_report(src) for src in ("route.hip", "norm.hip", "mxquant.hip", "mx.hip")}


@pytest.mark.parametrize("src", ["route.hip", "norm.hip", "mxquant.hip", "mx.hip"])
def test_no_scratch_and_no_vector_spill(reports, src):
    assert reports[src]
    for k, r in reports[src].items():
        assert r["ScratchSize [bytes/lane]"] == 0 and r["VGPRs Spill"] == 0, k


@pytest.mark.parametrize("name,waves", [
    ("mx_large_kernel", 2),                    # eight waves, one workgroup a CU
    ("MxTileILi128ELi128E", 4),                # eight waves, two workgroups a CU
    ("MxTileILi64ELi256E", 2),                 # eight waves, one
    ("MxSmallTileILi64ELi64ELi2ELi2ELi3ELi1E", 3),      # four waves, three workgroups a CU
    ("MxSmallTileILi64ELi64ELi2ELi2ELi3ELi2E", 2),      # eight waves, one
    ("MxSmallTileILi32ELi", 2), ("MxSmallTileILi64ELi128E", 2),
    ("mx_skinny_kernelILi1E", 4), ("mx_skinny_kernelILi2E", 4)])
def test_registers_leave_room_for_a_cus_workgroups(reports, name, waves):
    """512 registers a SIMD lane, given out in eights."""
    found = [r for k, r in reports["mx.hip"].items() if name in k]
    assert found
    for r in found:
        regs = -(-(r["VGPRs"] + r.get("AGPRs", 0)) // 8) * 8
        assert regs * waves <= 512, (name, r)
