"""The Python side of the block-scaled caches and windowed plans, without a GPU."""
import pytest

from mla_split_kv_gb300 import binding as nb
from mla_split_kv_gb300 import build as nbuild
from mla_split_kv_gb300 import runtime as rt
from tests.test_abi_cpu import fake_gb300


@pytest.fixture(scope="module", autouse=True)
def lib():
    nbuild.build()
    return nb.load()


@pytest.mark.parametrize("bs", [16, 32, 64])
def test_a_pool_has_the_scale_block_that_was_asked_for(bs):
    for g in range(-1, 2 * bs + 1):
        if g >= 1 and bs % g == 0:
            pool = rt.alloc_q8_cache(3, bs, g, device="cpu")
            assert pool.scale_block == g and tuple(pool.scales.shape) == (3, bs // g)
        else:  # 12 of 32 tokens would have become 16, 24 the whole page
            with pytest.raises(ValueError):
                rt.alloc_q8_cache(3, bs, g, device="cpu")


@pytest.mark.parametrize("H,q_len,causal", [(16, 1, False), (16, 4, True), (64, 1, False), (128, 1, False), (128, 32, True)])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("most", [1, 2, 8, 40, 64, 100, 1024])
def test_a_window_plan_of_any_partition_count_can_be_run(monkeypatch, most, dtype, H, q_len, causal):
    """mla_plan turns to single CTAs where there are more partitions than CTA pairs can share; mla_decode_window
    refuses those, so plan_window must not hand them out."""
    monkeypatch.setattr(rt, "alloc_partials", lambda *a, **k: (None, None))
    monkeypatch.setattr(rt, "alloc_decode_workspace", lambda *a, **k: None)
    for lens in ([20000], [0, 20000], [5000, 100, 7000], [4200] * 3, [9000] + [50] * 40):
        p = rt.plan_window(lens, H, q_len, 32, 4096, 4, dtype=dtype, causal=causal, dev=fake_gb300(), device="cpu", max_partitions=most).plan
        assert p.cluster_ctas >= 2 and (H * q_len <= 16 or p.cluster_ctas == 2)
        assert max(b - a for a, b in zip(p.o_indptr, p.o_indptr[1:])) <= most
