"""The build's register guard looks at every kernel of the 16-bit products (no GPU needed)."""
from __future__ import annotations

import glob
import os

import pytest

from moe_expert_ffn_amd import build as B
from tests.test_half_resources import FEW, TILE, _remark

SMALL = "_ZN7megamoe17half_small_kernelILi1ELi2ELb0EEEvNS_13HalfGmmParamsE"
WEIGHTS = "_ZN7megamoe25half_small_weights_kernelILi2ELi1EEEvNS_13HalfGmmParamsE"
ALL = (TILE, FEW, SMALL, WEIGHTS)
SRCS = sorted(glob.glob(os.path.join(B.CSRC, "*.hip")))


def report(*names, spilling=None):
    return "".join(_remark(n, 40 if n == spilling else 0, 160 if n == spilling else 0) for n in names)


def test_every_kernel_without_spills_passes():
    assert B.check_half_resources(report(*ALL)) == [] and B.check_half_kernels(report(*ALL), SRCS) == []


@pytest.mark.parametrize("name", ALL)
def test_a_spill_in_any_kernel_fails(name):
    problems = B.check_half_resources(report(*ALL, spilling=name))
    assert len(problems) == 1 and name in problems[0] and "40" in problems[0]


@pytest.mark.parametrize("name", ALL)
def test_a_kernel_that_is_not_reported_fails(name):
    problems = B.check_half_kernels(report(*(n for n in ALL if n != name)), SRCS)
    assert len(problems) == 1 and "not in the resource report" in problems[0]


@pytest.mark.parametrize("arguments", ["(HalfGmmParams p)", "(const HalfGmmParams p, int n)", " (\n    HalfGmmParams p)"])
def test_a_kernel_under_another_name_fails(tmp_path, arguments):
    src = tmp_path / "half_other.hip"
    src.write_text(f"template <int T>\n__global__ __launch_bounds__(256) void half_other_kernel{arguments} {{}}\n")
    problems = B.check_half_kernels(report(*ALL), SRCS + [str(src)])
    assert len(problems) == 1 and "half_other_kernel" in problems[0]


def test_the_sources_declare_the_checked_kernels():
    """Without a report every one of them is missed, and none of the sources' is unknown."""
    assert len(B.check_half_kernels("", SRCS)) == len(B.HALF_KERNELS) == len(ALL)
