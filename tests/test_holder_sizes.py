"""Sizes that the holder classes rely on (no GPU needed)."""
from __future__ import annotations

import random

import pytest

pytest.importorskip("torch")

from moe_expert_ffn_amd import megamoe as MM  # noqa: E402


def test_few_fits_the_forward_workspace():
    """forward_few of a holder works in forward's memory."""
    rng = random.Random(0)
    for _ in range(2000):
        M, E = rng.randint(1, 16), rng.randint(1, 256)
        d = MM.dims(M, 128 * rng.choice([1, 2, 56, 255, 256]), E, rng.randint(1, min(E, 512 // M)),
                    128 * rng.choice([1, 3, 16, 127, 128]))
        assert MM.megamoe_few_workspace_bytes(d) <= MM.megamoe_workspace_bytes(d), d
