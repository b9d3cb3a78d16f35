"""What holds of the norm and rotation and of cross attention without a GPU."""
import os
import re

import pytest

from precision_attention_fa4fp4_gb300 import build


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(build.CSRC) if f.endswith((".cu", ".cuh"))))
def test_grids_that_start_early_load_plainly(name):
    """A kernel that starts while its predecessor runs reads what that writes: no load of it may need the memory
    unchanged from the kernel's start."""
    with open(os.path.join(build.CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    if re.search(r"\b(wait_for_previous|grid_wait)\(", text) or name in ("cross.cuh", "cache_line.cuh"):
        assert not re.search(r"__ldg\b|__ldca|ld\.global\.nc|__restrict__", text)
