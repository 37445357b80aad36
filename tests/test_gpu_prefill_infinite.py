"""Infinite values under keys whose scores are -inf, in prompts whose runs of tokens are cut: a weight of 0 times an infinite
value is NaN in that value's column, whichever piece it lies in."""
import math

import pytest
import torch

from mla_split_kv_gb300 import binding as nb
from mla_split_kv_gb300 import build as nbuild
from tests.test_gpu_prefill import Case

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


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("new,ctx,H,gone", [(513, 30000, 8, 20000), (1, 30000, 2, 29000), (300, 1500, 2, 1100), (200, 200, 2, 0)])
def test_a_long_run_of_scores_of_minus_infinity(new, ctx, H, gone, dtype):
    """The first `gone` tokens of head 0: whole pieces of them, where the run is cut. (Of calls that are not, the same.)"""
    case = Case(31, [new], [ctx], H, dtype)
    case.q_nope[:, 0, 5] = case.q_nope[:, 0, 5].abs().clamp(min=0.01)
    case.k[:gone, 0, 5] = -math.inf
    columns = (7, 64, 127)
    if gone:
        for t, column in zip((100, gone // 2, gone - 1), columns):
            case.v[t, 0, column] = math.inf
    out, lse = case.run()
    torch.cuda.synchronize()
    case.check(out, lse, heads=[H - 1], rows=[0, 127, 128, new - 1])
    half, ulp = torch.finfo(case.dtype).eps / 2, 2.0 ** -23
    at = torch.tensor(sorted({0, new // 3, new // 2, new - 1}), device="cuda")
    q = torch.cat((case.q_nope[at, 0], case.q_pe[at, 0]), 1).double()
    k = torch.cat((case.k[gone:, 0], case.k_pe[gone:]), 1).double()
    v = case.v[gone:, 0].double()
    hidden = torch.arange(gone, ctx, device="cuda")[None] >= (ctx - new + at + 1)[:, None]
    s = (q @ k.T * case.scale).masked_fill(hidden, -math.inf)
    ds = (192 * ulp * case.scale * (q.abs() @ k.abs().T) + 8 * ulp * s.abs()).masked_fill(hidden, 0).amax(1)
    z = torch.logsumexp(s, 1)
    p = torch.exp(s - z[:, None])
    want, size = p @ v, p @ v.abs()
    tol = (half + 2 * ds + 2.0 ** -20 + 2 * ctx * ulp)[:, None] * size + (ctx * 2.0 ** -25 * v.abs().amax() if dtype == "f16" else 0)
    tol = tol + half * (want.abs() + tol) + 2.0 ** -25
    nan = torch.zeros(128, dtype=torch.bool, device="cuda")
    if gone:
        nan[list(columns)] = True
    got, got_lse = out[at, 0].double(), lse[at, 0].double()
    assert bool((got.isnan() == nan).all()), got.isnan().nonzero().tolist()
    assert bool((((got - want).abs() <= tol) | nan).all())
    lse_tol = (ds + ctx * ulp + 2.0 ** -20) / math.log(2.0) + 4 * ulp * (z.abs() / math.log(2.0))
    assert bool(((got_lse - z / math.log(2.0)).abs() <= lse_tol).all())


def test_rows_that_see_nothing_stay_0_in_cut_runs():
    """More rows than tokens beside a long request whose run is cut."""
    case = Case(32, [400, 513], [9, 30000], 4, "bf16", spare=5)
    out, lse = case.run()
    case.check(out, lse, heads=[0, 3], rows=[0, 390, 391, 399, 512])
