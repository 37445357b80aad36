"""The write into a block-scaled cache and the attention over it, one behind the other as a decode step runs them."""
import numpy as np
import pytest
import torch

from mla_split_kv_gb300 import binding as nb
from mla_split_kv_gb300 import build as nbuild
from mla_split_kv_gb300 import runtime as rt
from tests.test_gpu_q8 import SCALE, Q8Case

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


@pytest.mark.parametrize("H,g", [(16, 32), (64, 32), (16, 8)])
def test_scales_written_by_the_call_before_are_the_ones_read(H, g):
    """Many requests whose last pages are neighbours in the pool, so that eight scales share 32 bytes; every step
    makes every one of them grow, and the attention runs as a dependent of the write. It has the bits of a call made
    when all has long been written."""
    B, bs, steps = 304, 32, 20
    case = Q8Case(91, [33] * B, H=H, bs=bs, g=g, pow2=True)
    table = np.stack([np.arange(B, 2 * B), np.arange(B)], 1).astype(np.int32)  # second pages: 0, 1, 2, ...
    case.table = table
    case.upload()
    plan = case.plan()
    c_in, k_in = (torch.empty(B, 1, n, dtype=torch.float16, device="cuda") for n in (512, 64))
    out, ref = (torch.empty(B, 1, H, 512, device="cuda") for _ in range(2))
    lse, ref_lse = (torch.empty(B, 1, H, device="cuda") for _ in range(2))
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    rt.decode_q8(plan, case.qa, case.qp, case.cache, case.tab, case.ctx, SCALE, ref, ref_lse)
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        case.ctx += 1
        rt.cache_append_q8(case.cache, c_in, k_in, case.tab, case.ctx)
        rt.decode_q8(plan, case.qa, case.qp, case.cache, case.tab, case.ctx, SCALE, out, lse)
    torch.cuda.synchronize()
    r = torch.Generator(device="cuda").manual_seed(92)
    before = case.cache.scales.clone()
    for step in range(steps):
        size = 2.0 ** (step - 10 + torch.arange(B, device="cuda")[:, None, None] % 3)
        c_in.copy_(torch.randn(c_in.shape, device="cuda", generator=r) * size)
        k_in.copy_(torch.randn(k_in.shape, device="cuda", generator=r) * size)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        rt.decode_q8(plan, case.qa, case.qp, case.cache, case.tab, case.ctx, SCALE, ref, ref_lse)
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(lse, ref_lse), step
        assert torch.isfinite(out).all()
    assert (case.cache.scales[:B] > before[:B]).any(1).all()
