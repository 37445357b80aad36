"""Windowed calls whose contexts have outgrown their plan."""
import numpy as np
import pytest
import torch

from mla_split_kv_gb300 import binding as nb
from mla_split_kv_gb300 import build as nbuild
from mla_split_kv_gb300 import inputs as gen
from mla_split_kv_gb300 import runtime as rt
from tests.test_gpu_window import check, decode, make_plan

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    nbuild.build()
    nb.load()
    nb.mla_check_device_errors(None)
    yield
    st, code = nb.mla_check_device_errors(None)
    assert st == nb.MLA_OK, f"device error word {code:#x}"


@pytest.mark.parametrize("H,q_len,dtype", [(16, 1, "f16"), (16, 4, "bf16"), (128, 1, "bf16"), (16, 1, "e4m3")])
@pytest.mark.parametrize("planned", [[0, 1, 300, 64], [2000, 31, 0, 4999], [40000, 40000, 40000, 40000]])
def test_contexts_longer_or_shorter_than_planned(planned, H, q_len, dtype):
    """No token of a run is lost because the plan was made for a shorter one."""
    window, sinks = 700, 4
    case = gen.make_decode_case(71, [900, 2500, 333, 5003], num_heads=H, q_len=q_len, block_size=32, dtype=dtype, latent_std=0.5,
                                causal=q_len > 1)
    out, lse = decode(case, rt.upload(case), make_plan(case, window, sinks, lens=np.array(planned)))
    check(case, window, sinks, out, lse, [0, H - 1])
