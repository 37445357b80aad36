"""The Python side of the block-scaled caches and windowed plans, without a GPU."""
import pytest

from mla_split_kv_gb300 import binding as nb
from mla_split_kv_gb300 import build as nbuild
from mla_split_kv_gb300 import runtime as rt


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
