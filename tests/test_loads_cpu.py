"""Which loads the kernels use that read what the launch before them writes: lists, lengths, tables."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mla_split_kv_gb300", "csrc")


@pytest.mark.parametrize("name,constant", [
    ("prefill.cu", []), ("expand.cu", []), ("step_tables.cu", []), ("decode_shared.cu", ["p.cta_indptr", "unit"]), ("device_common.cuh", ["p.o_indptr"])])
def test_only_a_host_plans_arrays_are_taken_for_memory_that_never_changes(name, constant):
    """A dependent launch is resident while the kernel before it runs: mla_prefill's list is written by the kernel before
    its attention, block tables by mla_update_tables, which lets its dependents start at its first line. `ld.global.nc`,
    which `__ldg` is, is defined for memory that stays as it is for as long as the reading kernel runs, whatever that
    waits for in between. A host plan's arrays do (`constant`)."""
    with open(os.path.join(CSRC, name)) as f:
        source = re.sub(r"//[^\n]*", "", f.read())
    assert not re.findall(r"ld\.global(?:\.\w+)*\.nc\b|__restrict__", source)
    found = re.findall(r"\b__ldg\s*\(\s*([\w.]+)", source)
    assert set(found) <= set(constant) and len(found) == len(re.findall(r"\b__ldg\b", source))
