"""Steps without new tokens, calls without rows: nothing is launched, nothing is refused."""
import pytest
import torch

from mla_split_kv_gb300 import binding as nb
from mla_split_kv_gb300 import build as nbuild
from mla_split_kv_gb300 import runtime as rt

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


def launches():
    ctr = nb.mla_get_counters()
    return ctr[nb.CTR_STEP], ctr[nb.CTR_PREFILL], ctr[nb.CTR_REJECTED]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_a_step_in_which_requests_only_give_tokens_back(dtype):
    """As many new tokens as there are, none: the same calls as in any other step."""
    new = lambda *s: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
    B, H, bs = 3, 4, 32
    pool = rt.alloc_pool(20, bs)
    step = rt.alloc_step(B, 64, pool=pool)
    table = torch.full((B, 8), -1, dtype=torch.int32, device="cuda")
    changes = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    rt.update_tables(pool, changes(40, 1, 5), step.context_lens, table, step)
    rt.update_tables(pool, changes(-40, -1, -5), step.context_lens, table, step)
    ckv, kpe = torch.ones(20, bs, 512, dtype=dtype, device="cuda"), torch.ones(20, bs, 64, dtype=dtype, device="cuda")
    plan = rt.plan_prefill(B, H, 64)
    w_uk, w_uv_t = new(H, 128, 512), new(H, 512, 128)
    torch.cuda.synchronize()
    assert step.context_lens.tolist() == [0, 0, 0] and pool.count.item() == 20
    nb.mla_reset_counters()
    both = new(0, 576)
    rt.cache_append_slots(ckv, kpe, both[:, :512], both[:, 512:], step.slots)
    rt.cache_append_slots(ckv, kpe, new(0, 512), new(0, 64), step.slots[:0])
    k, v, k_pe = new(0, H, 128), new(0, H, 128), new(0, 64)
    rt.expand_kv(ckv, kpe, table, step.kv_indptr, w_uk, w_uv_t, k, v, k_pe)
    out = new(0, H, 128)
    assert rt.prefill(plan, new(0, H, 128), new(0, H, 64), k, k_pe, v, step.q_indptr, step.kv_indptr, 0.1, out) is out
    k, v, k_pe = new(9, H, 128), new(9, H, 128), new(9, 64)
    q = new(0, H, 192)
    rt.prefill(plan, q[..., :128], q[..., 128:], k, k_pe, v, step.q_indptr, step.kv_indptr, 0.1, out, torch.empty(0, H, device="cuda"))
    torch.cuda.synchronize()
    assert launches() == (0, 0, 0)
    assert bool((ckv == 1).all()) and bool((kpe == 1).all())
    with pytest.raises(ValueError):  # what does not fit together is refused all the same
        rt.prefill(plan, new(0, H, 64), new(0, H, 64), k, k_pe, v, step.q_indptr, step.kv_indptr, 0.1, out)
