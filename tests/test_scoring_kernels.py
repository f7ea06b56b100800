"""The kernels in the built library, by name, on the CPU: what no call reaches is not built."""
import os
import re

import pytest

from byte_level_bpe_amd import build as libbuild


def test_sixteen_waves_are_of_32_bit_rows():
    """Loss and gradient in one call take sixteen waves for long rows of float32 alone."""
    if not os.path.exists(libbuild.OUT):
        pytest.skip("not built")
    with open(libbuild.OUT, "rb") as f:
        names = set(re.findall(rb"14k_distill_stepI(\w+?)Lj(\d+)ELb([01])E", f.read()))
    waves = {n: {t for t, w, _ in names if int(w) == n} for n in (1, 4, 8, 16)}
    assert all(len(waves[n]) == 3 for n in (1, 4, 8)) and waves[16] == {b"f"}, names
    assert len(names) == 3 * 3 * 2 + 2
