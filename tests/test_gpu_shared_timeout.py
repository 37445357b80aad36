"""Bounded waits of decode attention over a common prefix: they run out, are reported, and the next call is whole."""
import pytest
import torch

from mla_split_kv_gb300 import binding as nb
from mla_split_kv_gb300 import build as nbuild
from tests.test_gpu_shared import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    nbuild.build()
    nb.load()
    nb.mla_check_device_errors(None)
    yield
    nb.mla_set_wait_timeout_ns(2_000_000_000)
    st, code = nb.mla_check_device_errors(None)
    assert st == nb.MLA_OK, f"device error word {code:#x}"


@pytest.mark.parametrize("lens,shared,H,q_len,dtype", [([40000, 39000], 32768, 16, 1, "f16"), ([20000, 18000, 19000], 16384, 128, 2, "bf16")])
def test_waits_that_run_out_are_reported(lens, shared, H, q_len, dtype):
    case = Case(41, lens, shared, H, q_len, 32, dtype, q_len > 1)
    plan = case.plan()
    case.run(plan)
    st, code = nb.mla_check_device_errors(None)
    assert st == nb.MLA_OK
    nb.mla_set_wait_timeout_ns(1)
    try:
        for _ in range(50):  # (a wait is found too long when the device's timer has moved on and it still lasts)
            case.run(plan)
            st, code = nb.mla_check_device_errors(None)
            if st != nb.MLA_OK:
                break
    finally:
        nb.mla_set_wait_timeout_ns(2_000_000_000)
    assert st == nb.MLA_ERR_TIMEOUT and code & 1, (st, code)
    out, lse = case.run(plan)
    st, code = nb.mla_check_device_errors(None)
    assert st == nb.MLA_OK, code
    case.check(out, lse, heads=[0, H - 1])
