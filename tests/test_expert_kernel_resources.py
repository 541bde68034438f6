"""The expert products' and the quantiser's kernels keep everything in
registers: the compiler's own report shows no scratch and no vector spill, and
the waves and LDS of each workgroup fit a CU as often as the kernel counts on."""
import os
import shutil

import pytest

from test_kernel_resources import resource_report

pytestmark = pytest.mark.skipif(shutil.which("hipcc") is None and
                                not os.path.exists("/opt/rocm/bin/hipcc"),
                                reason="hipcc needed")


@pytest.fixture(scope="module")
def reports():
    return {src: resource_report(src) for src in ("experts.hip", "skinny.hip", "quant.hip")}


@pytest.mark.parametrize("src,kernels", [("experts.hip", 33), ("skinny.hip", 18), ("quant.hip", 12)])
def test_no_scratch_and_no_vector_spill(reports, src, kernels):
    assert len(reports[src]) == kernels
    for k, r in reports[src].items():
        assert r["ScratchSize [bytes/lane]"] == 0 and r["VGPRs Spill"] == 0, k


@pytest.mark.parametrize("name,waves", [
    ("grouped_large_kernel", 2),                 # eight waves, one workgroup a CU
    ("wgrad_tile_kernelINS0_3F16ELi256", 2), ("wgrad_tile_kernelINS0_4BF16ELi256", 2),
    ("F16ELi128ELi128E", 4),                     # eight waves, two workgroups a CU (both types)
    ("FP8ELi128ELi128E", 2), ("FP8ExactELi128ELi128E", 2),   # eight waves, one
    ("ELi64ELi256E", 2),                         # eight waves, one
    ("ELi64ELi64E", 2)])                         # four waves, two workgroups a CU
def test_registers_leave_room_for_a_cus_workgroups(reports, name, waves):
    """512 registers a SIMD lane, given out in eights."""
    found = [r for k, r in reports["experts.hip"].items() if name in k]
    assert found
    for r in found:
        regs = -(-(r["VGPRs"] + r.get("AGPRs", 0)) // 8) * 8
        assert regs * waves <= 512, (name, r)
