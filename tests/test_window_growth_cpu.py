"""Plans of windowed calls and contexts that outgrow them."""
import numpy as np
import pytest

from mla_split_kv_gb300 import build as nbuild
from mla_split_kv_gb300 import binding as nb
from mla_split_kv_gb300 import runtime as rt
from tests.test_abi_cpu import fake_gb300


@pytest.fixture(scope="module", autouse=True)
def lib():
    nbuild.build()
    return nb.load()


@pytest.mark.parametrize("max_partitions", [0, 4])
@pytest.mark.parametrize("H,q_len", [(16, 1), (16, 4), (128, 1)])
def test_a_plan_s_last_partitions_take_whatever_a_run_becomes(monkeypatch, H, q_len, max_partitions):
    monkeypatch.setattr(rt, "alloc_partials", lambda *a, **k: (None, None))
    monkeypatch.setattr(rt, "alloc_decode_workspace", lambda *a, **k: None)
    lens = [0, 1, 290, 310, 1000, 9000, 100000]
    plan = rt.plan_window(lens, H, q_len, 32, 6000, 5, causal=q_len > 1, dev=fake_gb300(), device="cpu", max_partitions=max_partitions)
    table, host = plan.chunks.numpy(), np.array(plan.plan.chunks)
    assert np.array_equal(table[:, [0, 1, 3]], host[:, [0, 1, 3]])
    for b in range(len(lens)):
        lo, hi = plan.plan.o_indptr[b], plan.plan.o_indptr[b + 1]
        assert hi > lo and np.array_equal(table[lo:hi - 1, 2], host[lo:hi - 1, 2]) and table[hi - 1, 2] == 2 ** 31 - 1
        assert list(table[lo:hi, 1]) == [0] + list(table[lo:hi - 1, 2])  # one after the other, from the first token
