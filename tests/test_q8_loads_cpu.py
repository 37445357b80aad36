"""Which loads the kernels of the block-scaled caches use."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mla_split_kv_gb300", "csrc")


@pytest.mark.parametrize("name", ["append_q8.cu", "decode_q8.cu", "q8_schedule.cuh"])
def test_no_load_assumes_memory_that_never_changes(name):
    """These kernels are resident while the kernel before them runs (the cache's write lets its dependents start at
    its first line, and writes the scales after that). `ld.global.nc`, which `__ldg` is, is defined for memory that
    stays as it is for as long as the reading kernel runs, whatever that waits for in between."""
    with open(os.path.join(CSRC, name)) as f:
        source = re.sub(r"//[^\n]*", "", f.read())
    assert not re.findall(r"\b__ldg\s*\(|ld\.global(?:\.\w+)*\.nc\b|__restrict__", source)
