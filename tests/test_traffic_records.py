"""bench.py's measured HBM traffic: the records under profiles/ are of the kernel sources on file, and
what makes one stale (no GPU needed)."""
from __future__ import annotations

import json
import os

import pytest

import bench

STAGES = {"permute": "permute.hip", "gmm1": "gmm.hip", "swiglu": "swiglu.hip", "gmm2": "gmm.hip",
          "unpermute": "unpermute.hip"}
CSRC = os.path.join(bench.ROOT, "moe_expert_ffn_amd", "csrc")


def test_source_hash_follows_the_includes(tmp_path):
    def write(name, text):
        (tmp_path / name).write_text(text)

    write("k.hip", '#include <vector>\n#include "a.hpp"\n  #  include "sub/../b.hpp"\nint k;\n')
    (tmp_path / "sub").mkdir()
    write("a.hpp", '#pragma once\n#include "c.hpp"\n')
    write("b.hpp", '#include "a.hpp"\n#include "k.hip"\n')  # round again
    write("c.hpp", "int c;\n")
    write("other.hpp", "int other;\n")
    path = str(tmp_path / "k.hip")
    first = bench.source_hash(path)
    write("other.hpp", "int changed;\n")
    write("new.hpp", "int added;\n")
    assert bench.source_hash(path) == first, "a header that the kernel does not include"
    seen = {first}
    for name in ("c.hpp", "b.hpp", "a.hpp", "k.hip"):
        with open(tmp_path / name, "a") as f:
            f.write("// more\n")
        seen.add(bench.source_hash(path))
    assert len(seen) == 5


@pytest.mark.parametrize("workload", ["decode", "mid", "large", "skewed"])
@pytest.mark.parametrize("stage", sorted(STAGES))
def test_traffic_is_of_the_sources_on_file(workload, stage):
    src = os.path.join(CSRC, STAGES[stage])
    got = bench.traffic_from_profile(src, workload, stage)
    with open(os.path.join(bench.ROOT, "profiles", f"traffic_{stage}_{workload}.json")) as f:
        assert got == json.load(f)["hbm_bytes_per_launch"] > 0, "taken from another source: profile again"
