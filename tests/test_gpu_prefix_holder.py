"""A common prefix held by a request of its own: the others start with its pages, come by growing and go by shrinking to it."""
import torch
import pytest

from mla_split_kv_gb300 import binding as nb
from mla_split_kv_gb300 import build as nbuild
from mla_split_kv_gb300 import runtime as rt
from tests.test_gpu_shared import Case as SharedCase

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


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_requests_come_and_go_beside_the_prefix(out_dtype):
    g = torch.Generator("cuda").manual_seed(3)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    B, H, bs, P, num_blocks, scale = 3, 16, 32, 128, 40, 192.0 ** -0.5
    pool = rt.alloc_pool(num_blocks, bs)
    step = rt.alloc_step(B + 1, 512, pool=pool)  # request 0 holds the prefix
    table = torch.full((B + 1, 16), -1, dtype=torch.int32, device="cuda")
    ckv, kpe = rand(num_blocks, bs, 512), rand(num_blocks, bs, 64)
    rows = [rand(0, 576) for _ in range(B + 1)]

    def change(*changes):
        new = rand(sum(max(n, 0) for n in changes), 576)
        rt.update_tables(pool, torch.tensor(changes, dtype=torch.int32, device="cuda"), step.context_lens, table, step)
        rt.cache_append_slots(ckv, kpe, new[:, :512], new[:, 512:], step.slots)
        at = 0
        for b, n in enumerate(changes):
            rows[b] = torch.cat((rows[b], new[at:at + n])) if n >= 0 else rows[b][:n]
            at += max(n, 0)

    change(P, 0, 0, 0)
    table[1:, :P // bs] = table[0, :P // bs]
    step.context_lens[1:] = P
    rows[1:] = [rows[0]] * B
    plan = rt.plan_shared([P + 60] * B, P, H, 1, bs, dtype="bf16")  # for three, whoever is there
    out, lse = torch.empty(B, 1, H, 512, dtype=out_dtype, device="cuda"), torch.empty(B, 1, H, device="cuda")

    def decode():
        q_abs, q_pe = rand(B, 1, H, 512), rand(B, 1, H, 64)
        rt.decode_shared(plan, q_abs, q_pe, ckv, kpe, table[1:], step.context_lens[1:], scale, out, lse, shared_table=table[0, :P // bs])
        torch.cuda.synchronize()
        c = SharedCase.__new__(SharedCase)
        c.lens, c.shared, c.H, c.q_len, c.bs, c.dtype, c.causal, c.scale = [len(x) for x in rows[1:]], P, H, 1, bs, torch.bfloat16, False, scale
        c.shared_table, c.table, c.ckv, c.kpe, c.q_abs, c.q_pe = table[0, :P // bs], table[1:], ckv, kpe, q_abs, q_pe
        c.check(out, lse, heads=[0, H - 1])
        assert step.context_lens.tolist() == [len(x) for x in rows]
        for b, x in enumerate(rows):
            t = torch.arange(len(x), device="cuda")
            at = table[b].long()[t // bs] * bs + t % bs
            assert torch.equal(ckv.view(-1, 512)[at], x[:, :512])

    change(0, 70, 33, 0)
    decode()
    change(0, 1, 1, 40)
    decode()
    change(0, P - len(rows[1]), 1, 1)  # the first one ends
    decode()
    change(0, 0, 31, 1)
    change(0, 200, 1, 1)
    decode()
    change(0, *(P - len(x) for x in rows[1:]))
    decode()
    step.context_lens[1:] = 0  # the end: only then may the prefix go
    change(-P, 0, 0, 0)
    assert pool.count.item() == num_blocks and sorted(pool.pages.tolist()) == list(range(num_blocks))
