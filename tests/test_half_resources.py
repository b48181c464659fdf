"""The build's register guard of the 16-bit products (no GPU needed)."""
from __future__ import annotations

import pytest

from moe_expert_ffn_amd import build as B


def _remark(name: str, spills: int, scratch: int) -> str:
    lines = (f"Function Name: {name}", "TotalSGPRs: 100", "VGPRs: 250", "AGPRs: 256",
             f"ScratchSize [bytes/lane]: {scratch}", "Occupancy [waves/SIMD]: 1", "SGPRs Spill: 4",
             f"VGPRs Spill: {spills}", "LDS Size [bytes/block]: 139808")
    return "".join(f"half.hip:1:0: remark:     {x} [-Rpass-analysis=kernel-resource-usage]\n" for x in lines)


TILE, FEW = "_ZN7megamoe15half_gmm_kernelINS_6HgGeomILi0EEEEEv", "_ZN7megamoe15half_few_kernelILi2ELb1ELi1EEEv"


def test_kernels_without_spills_pass():
    assert B.check_half_resources(_remark(TILE, 0, 0) + _remark(FEW, 0, 0)) == []


@pytest.mark.parametrize("name", [TILE, FEW])
@pytest.mark.parametrize("spills, scratch", [(1, 8), (0, 16), (17, 72)])
def test_a_spill_fails(name, spills, scratch):
    other = FEW if name == TILE else TILE
    problems = B.check_half_resources(_remark(other, 0, 0) + _remark(name, spills, scratch))
    assert len(problems) == 1 and name in problems[0] and str(spills) in problems[0]


def test_other_kernels_may_spill():
    norm = _remark("_ZN7megamoe16norm_grad_kernelILi0ELi0ELi4EEEv", 25, 100)
    assert B.check_half_resources(norm + _remark(TILE, 0, 0)) == []


def test_an_empty_report_fails():
    assert B.check_half_resources("") != []
